// Host side of the sequence operators (rotary positions, decayed linear attention): argument
// checks, the choice of segments, workspace plans and launches.  Included by rehyat.cu after its
// helpers (fail, RH_TRY, cuda_check, Carve).
#pragma once

#include <atomic>

#include "decay.cuh"
#include "decay_bf16.cuh"
#include "rotary.cuh"

namespace {

using rehyat::decay::Pass;
using rehyat::decay::Rows;

struct DecayDims {
  int B, H, Hk, N, D;
  rehyat_dtype dt;
  float scale;
};

int check_decay(const DecayDims& a) {
  if (a.dt != REHYAT_F32 && a.dt != REHYAT_BF16)
    return fail(REHYAT_ERR_DTYPE, "unknown dtype %d", (int)a.dt);
  if (a.B < 1 || a.H < 1 || a.Hk < 1 || a.N < 0 || a.D < 1)
    return fail(REHYAT_ERR_ARG, "need B, H, Hk, D >= 1 and N >= 0 (B=%d H=%d Hk=%d N=%d D=%d)", a.B,
                a.H, a.Hk, a.N, a.D);
  if (a.H % a.Hk) return fail(REHYAT_ERR_ARG, "Hk=%d must divide H=%d", a.Hk, a.H);
  if (a.D % 8 || a.D > rehyat::decay::kMaxD)
    return fail(REHYAT_ERR_SHAPE, "D=%d must be a multiple of 8 up to %d", a.D,
                rehyat::decay::kMaxD);
  if (a.B > 65535 || (long long)a.B * a.H > 65535)
    return fail(REHYAT_ERR_SHAPE, "B*H = %lld exceeds 65535", (long long)a.B * a.H);
  if (a.N > (1 << 30)) return fail(REHYAT_ERR_ARG, "sequence too long");
  if (!std::isfinite(a.scale)) return fail(REHYAT_ERR_ARG, "scale must be finite");
  return REHYAT_OK;
}

// A strided [B, heads, N, D] tensor: aligned, whole 16-byte strides of at least a row.
int check_rows(const char* what, const rehyat_rows& s, const DecayDims& a, int heads) {
  const int el = a.dt == REHYAT_BF16 ? 2 : 4, D = a.D;
  if (a.N == 0) return REHYAT_OK;
  if (!s.p) return fail(REHYAT_ERR_ARG, "null pointer (%s)", what);
  if (!aligned16(s.p)) return fail(REHYAT_ERR_ALIGN, "%s is not 16-byte aligned", what);
  const long long st[3] = {s.batch, s.head, s.row};
  const int size[3] = {a.B, heads, a.N};
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (st[i] < D)
      return fail(REHYAT_ERR_ARG, "%s: stride %lld of a dimension of %d is below D=%d", what, st[i],
                  size[i], D);
    if ((st[i] * el) % 16)
      return fail(REHYAT_ERR_ALIGN, "%s: stride %lld is not a multiple of 16 bytes", what, st[i]);
    if (st[i] * el >= (1LL << 40)) return fail(REHYAT_ERR_ARG, "%s: stride %lld too long", what, st[i]);
  }
  return REHYAT_OK;
}

Rows rows_of(const rehyat_rows& s, int group) {
  return Rows{s.p, s.batch, s.head, s.row, group};
}

// The cut of sequences into segments: one CTA for each and each head, so their number trades whole
// waves of the 148 SMs against each CTA's start, about one chunk of the bf16 kernels (128 rows) and a
// quarter of one of the fp32 kernels (64 rows).  A launch of three passes takes the same cut: each
// pass fills the waves by itself (cut for all three at once, in one wave of 64-chunk segments, the
// 480x832 5 s gradients took 380 us instead of 320).  A ragged batch gets all the slots of its waves,
// and the device cuts the valid rows to fill them; unless whole sequences are one segment each and
// nothing but that cut would need the sums of segments.
rehyat::decay::Cut decay_cut(const DecayDims& a, bool ragged, bool last) {
  rehyat::decay::Cut c{};
  const bool bf16 = a.dt == REHYAT_BF16;
  c.chunk = bf16 ? rehyat::decay::tc::kRows : rehyat::decay::kC;
  const int start = bf16 ? 4 : 1;  // in quarters of a chunk
  const int chunks = a.N > 0 ? (a.N + c.chunk - 1) / c.chunk : 1;
  const long long BH = (long long)a.B * a.H;
  long long best = -1, best_waves = 1;
  for (int n = 1; n <= chunks && n <= 256; ++n) {
    const int per = (chunks + n - 1) / n;
    if ((chunks + per - 1) / per != n) continue;  // the last ones would hold no rows
    const long long waves = (BH * n + 147) / 148, cost = waves * (4 * per + start);
    if ((best < 0 || cost < best) && (n == 1 || (long long)a.B * n <= 65535)) {
      best = cost;
      best_waves = waves;
      c.per_seq = n;
      c.chunks = per;
    }
  }
  c.slots = a.B * c.per_seq;
  c.search = ragged && a.B <= rehyat::decay::kMaxSearch && (c.per_seq > 1 || last);
  if (c.search) {
    const long long fit = best_waves * 148 / a.H;
    if (fit > c.slots) c.slots = (int)(fit < 65535 ? fit : 65535);
  }
  return c;
}

struct DecayPlan {
  rehyat::decay::Cut cut;
  size_t fwd, bwd, part[2], total;
};
DecayPlan plan_decay(const DecayDims& a, bool backward, bool ragged, bool last) {
  DecayPlan p{};
  const size_t BH = (size_t)a.B * a.H;
  p.cut = decay_cut(a, ragged, last);
  Carve cv;
  const size_t states = (size_t)p.cut.slots * a.H * a.D * a.D * 4;
  p.fwd = cv.take(states);
  if (backward) {
    p.bwd = cv.take(states);
    // per query head, where dk and dv are sums over the heads that share a key/value head
    for (size_t& part : p.part) part = cv.take(a.H != a.Hk ? BH * (size_t)a.N * a.D * 4 : 0);
  }
  p.total = cv.off;
  return p;
}

// bf16 [B, heads, N, D] tensor with strides in elements, loaded and stored as 128-row x 64-column
// boxes with 128-byte swizzle; columns past D read zeros and are not written.
int make_map_rows(CUtensorMap* m, const Rows& s, int D, int N, int heads, int B) {
  EncodeTiledFn enc;
  RH_TRY(get_encoder(&enc));
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)heads, (cuuint64_t)B};
  // the stride of a single row, head or sequence is never used; any legal one will do
  const long long one = D;
  cuuint64_t strides[3] = {(cuuint64_t)(N > 1 ? s.sn : one) * 2,
                           (cuuint64_t)(heads > 1 ? s.sh : one) * 2,
                           (cuuint64_t)(B > 1 ? s.sb : one) * 2};
  cuuint32_t box[4] = {64, 128, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(s.p), dims,
                   strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(REHYAT_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return REHYAT_OK;
}
int map_of(CUtensorMap* m, const Rows& t, const Pass& p) {
  return make_map_rows(m, t, p.D, p.N, p.H / t.group, p.B);
}

// A launch behind another of the same call: with `behind`, it may start while that one still runs
// (programmatic stream serialization) and waits for it before it reads what that one writes.
struct Behind {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  Behind(dim3 grid, int threads, size_t smem, cudaStream_t st, bool behind) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 1 : 0;
  }
};

// Lets kernel kKernel use up to `most` bytes of dynamic shared memory, once on each device.
template <auto kKernel>
int allow_smem(int most) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  RH_TRY(cuda_check(cudaGetDevice(&dev), "device"));
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return REHYAT_OK;
  RH_TRY(cuda_check(cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most),
                    "shared memory size"));
  if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return REHYAT_OK;
}

template <int kDp>
int launch_f32_states(const rehyat::decay::Passes& a, dim3 grid, cudaStream_t st) {
  using namespace rehyat::decay;
  const int smem = states_smem_floats(kDp) * 4;
  RH_TRY(allow_smem<decay_states_kernel<kDp>>(smem));
  decay_states_kernel<kDp><<<grid, kThreads, smem, st>>>(a);
  return REHYAT_OK;
}
template <int kDp>
int launch_f32_rows(const rehyat::decay::Passes& a, dim3 grid, bool behind_scan, cudaStream_t st) {
  using namespace rehyat::decay;
  // A grid of one wave asks for more than half of an SM's shared memory: where two CTAs of a narrow
  // head fit one SM, those that start while the scan still runs would pair up on the SMs it has left
  // (4 sequences, 6 heads, 1,151 rows, D = 64: 59.6 us, 43.6 spread out).
  constexpr int kNeeds = rows_smem_floats(kDp) * 4, kAlone = 116 << 10;
  constexpr int kMost = kNeeds > kAlone ? kNeeds : kAlone;
  const int smem = (long long)grid.x * grid.y * grid.z <= 148 ? kMost : kNeeds;
  RH_TRY(allow_smem<decay_rows_kernel<kDp>>(kMost));
  Behind l(grid, kRowThreads, smem, st, behind_scan);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, decay_rows_kernel<kDp>, a), "decay rows launch");
}

// The passes of one launch: the states they need, and the rows.
int launch_decay_states(const Pass* p, int n, rehyat_dtype dt, cudaStream_t st) {
  const dim3 grid(p[0].H, p[0].cut.slots, n);
  if (dt == REHYAT_BF16) {
    using namespace rehyat::decay::tc;
    StatesArgs a{};
    for (int i = 0; i < n; ++i) {
      a.p[i] = p[i];
      RH_TRY(map_of(&a.b[i], p[i].b, p[i]));
      RH_TRY(map_of(&a.c[i], p[i].c, p[i]));
    }
    RH_TRY(allow_smem<decay_states_bf16_kernel>(kStSmem));
    decay_states_bf16_kernel<<<grid, kStThreads, kStSmem, st>>>(a);
  } else {
    using namespace rehyat::decay;
    Passes a{};
    for (int i = 0; i < n; ++i) a.p[i] = p[i];
    switch (padded(p[0].D)) {
      case 32: RH_TRY(launch_f32_states<32>(a, grid, st)); break;
      case 64: RH_TRY(launch_f32_states<64>(a, grid, st)); break;
      case 96: RH_TRY(launch_f32_states<96>(a, grid, st)); break;
      default: RH_TRY(launch_f32_states<128>(a, grid, st)); break;
    }
  }
  return cuda_check(cudaGetLastError(), "decay states launch");
}

// behind_scan: the launch before is this call's scan, whose prefixes the kernel waits for.
int launch_decay_rows(const Pass* p, int n, rehyat_dtype dt, bool behind_scan, cudaStream_t st) {
  const dim3 grid(p[0].H, p[0].cut.slots, n);
  if (dt == REHYAT_F32) {
    using namespace rehyat::decay;
    Passes a{};
    for (int i = 0; i < n; ++i) a.p[i] = p[i];
    switch (padded(p[0].D)) {
      case 32: return launch_f32_rows<32>(a, grid, behind_scan, st);
      case 64: return launch_f32_rows<64>(a, grid, behind_scan, st);
      case 96: return launch_f32_rows<96>(a, grid, behind_scan, st);
      default: return launch_f32_rows<128>(a, grid, behind_scan, st);
    }
  }
  using namespace rehyat::decay::tc;
  RowsArgs a{};
  for (int i = 0; i < n; ++i) {
    a.p[i] = p[i];
    RH_TRY(map_of(&a.a[i], p[i].a, p[i]));
    RH_TRY(map_of(&a.b[i], p[i].b, p[i]));
    RH_TRY(map_of(&a.c[i], p[i].c, p[i]));
    a.out[i] = a.a[i];  // unused with fp32 output
    if (!p[i].out_f32)
      RH_TRY(make_map_rows(&a.out[i], Rows{p[i].out, p[i].ob, p[i].oh, p[i].on, 1}, p[i].D, p[i].N,
                           p[i].H, p[i].B));
  }
  RH_TRY(allow_smem<decay_rows_bf16_kernel>(kRwSmem));
  Behind l(grid, kRwThreads, kRwSmem, st, behind_scan);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, decay_rows_bf16_kernel, a), "decay rows launch");
}

// The state before every segment of n <= 2 passes (rows b, c; time direction and e as in each) from
// S0[i] (or zero), and the state after the last into last[i] unless null.  *scanned: whether a scan
// was launched.
int decay_prefixes(Pass* p, int n, rehyat_dtype dt, const float* const* S0, float* const* last,
                   bool* scanned, cudaStream_t st) {
  const bool many = p[0].cut.per_seq > 1 || p[0].cut.search;
  Pass need[2];
  rehyat::decay::Scans a{};
  int sums = 0, scans = 0;
  for (int i = 0; i < n; ++i) {
    p[i].carried = many || S0[i];
    p[i].exact = last[i] != nullptr;
    if (many || last[i]) need[sums++] = p[i];
    if (p[i].carried || last[i])
      a.s[scans++] = rehyat::decay::Scan{p[i].states, S0[i], last[i], p[i].reverse};
  }
  *scanned = scans > 0;
  if (scans == 0) return REHYAT_OK;
  const bool summed = sums > 0 && p[0].N > 0;
  if (summed) RH_TRY(launch_decay_states(need, sums, dt, st));
  a.log_decay = p[0].log_decay; a.lengths = p[0].lengths;
  a.B = p[0].B; a.H = p[0].H; a.N = p[0].N; a.D = p[0].D; a.cut = p[0].cut;
  const int n4 = a.D * a.D / 4;
  Behind l(dim3((n4 + 255) / 256, p[0].B * p[0].H, scans), 256, 0, st, summed);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, rehyat::decay::decay_scan_kernel, a),
                    "decay scan launch");
}

Pass decay_pass(const DecayDims& a, const float* log_decay, const int* lengths,
                const rehyat::decay::Cut& cut, void* states) {
  Pass p{};
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.B = a.B; p.H = a.H; p.N = a.N; p.D = a.D;
  p.cut = cut;
  p.states = static_cast<float*>(states);
  p.sp = p.si = p.sd = 1.f;
  return p;
}

void set_out(Pass& p, const rehyat_rows& o) {
  p.out = o.p;
  p.ob = o.batch; p.oh = o.head; p.on = o.row;
}

// ---- where the arguments of a call lie ----
// Bytes of one argument: runs of `run` bytes, repeated along up to three dimensions in ascending
// order of their strides.
struct Place {
  const char* what = nullptr;
  bool written = false;
  intptr_t p = 0;
  long long run = 0, size[3], stride[3];
  int dims = 0;

  // Bytes from the first to the last of the runs along the first n dimensions.
  __int128 extent(int n) const {
    __int128 e = run;
    for (int i = 0; i < n; ++i) e += (__int128)(size[i] - 1) * stride[i];
    return e;
  }
  // No byte is reached twice; sufficient, and true of every slice, transpose or stack of a dense
  // tensor.
  bool apart() const {
    for (int i = 0; i < dims; ++i)
      if (stride[i] < extent(i)) return false;
    return true;
  }
};
Place place(const char* what, const void* p, long long bytes, bool written) {
  Place a;
  a.what = what;
  a.written = written;
  a.p = reinterpret_cast<intptr_t>(p);
  a.run = p ? bytes : 0;
  return a;
}
// Runs of `bytes`; counts and strides (in bytes) of three dimensions in any order.
Place place(const char* what, const void* p, long long bytes, const long long (&n)[3],
            const long long (&stride)[3], bool written) {
  Place a = place(what, p, bytes, written);
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 0) a.run = 0;
    if (n[i] <= 1 || (stride[i] == 0 && !written)) continue;  // (an expanded input)
    long long st = stride[i];
    if (st < 0) {
      a.p += (intptr_t)(st * (n[i] - 1));
      st = -st;
    }
    int at = a.dims++;
    for (; at > 0 && a.stride[at - 1] > st; --at) {
      a.stride[at] = a.stride[at - 1];
      a.size[at] = a.size[at - 1];
    }
    a.stride[at] = st;
    a.size[at] = n[i];
  }
  int merged = 0;  // innermost dimensions that continue the run
  while (merged < a.dims && a.stride[merged] == a.run) a.run *= a.size[merged++];
  for (int i = merged; i < a.dims; ++i) {
    a.stride[i - merged] = a.stride[i];
    a.size[i - merged] = a.size[i];
  }
  a.dims -= merged;
  return a;
}
Place place(const char* what, const rehyat_rows& t, int B, int heads, int N, int D, int el,
            bool written) {
  return place(what, t.p, (long long)D * el, {B, heads, N},
               {t.batch * el, t.head * el, t.row * el}, written);
}

// Whether two arguments have a byte in common: whether d = (second's address - first's) is a
// difference of a byte of the first and one of the second, sum over the strides of both of (i - j)
// stride + (x - y), i < size and x < run in the first, j and y in the second.  From the largest stride
// down, what is left of d has to be within reach of the smaller ones, which leaves two or three
// values of i - j where strides are nested; where one argument's runs cover many strides of the
// other, a value in the middle decides.  Never true without a common byte.
bool meet(const Place& a, int na, const Place& b, int nb, __int128 d) {
  const __int128 ra = a.extent(na) - 1, rb = b.extent(nb) - 1;
  if (d > ra || d < -rb) return false;
  if (na == 0 && nb == 0) return true;
  const long long sa = na ? a.stride[na - 1] : -1, sb = nb ? b.stride[nb - 1] : -1;
  const long long s = sa > sb ? sa : sb;
  if (s <= 0) return false;  // (a written dimension expanded: refused before)
  const int ma = sa == s ? na - 1 : na, mb = sb == s ? nb - 1 : nb;
  const __int128 la = a.extent(ma) - 1, lb = b.extent(mb) - 1;  // reach of what is left
  auto floor_div = [](__int128 x, __int128 y) { return x / y - (x % y < 0); };
  __int128 lo = -floor_div(la - d, s), hi = floor_div(d + lb, s);
  const __int128 most = sa == s ? a.size[na - 1] - 1 : 0, least = sb == s ? 1 - b.size[nb - 1] : 0;
  if (lo < least) lo = least;
  if (hi > most) hi = most;
  const __int128 mid = lo + (hi - lo) / 2;
  for (__int128 e = lo; e <= hi; ++e) {
    if (e == lo + 2 && e < mid) e = mid;
    if (e > mid && e < hi - 1) e = hi - 1;
    if (meet(a, ma, b, mb, d - e * s)) return true;
  }
  return false;
}

// No written argument reaches a byte of its own twice, or a byte of another argument: CTAs write
// their parts while others still read or write theirs.
template <int n>
int check_places(const Place (&a)[n]) {
  __int128 end[n];
  for (int i = 0; i < n; ++i) {
    if (a[i].run && a[i].written && !a[i].apart())
      return fail(REHYAT_ERR_ARG, "%s: its rows overlap one another", a[i].what);
    end[i] = a[i].p + a[i].extent(a[i].dims);
  }
  for (const bool same : {true, false})
    for (int i = 1; i < n; ++i)
      for (int j = 0; j < i; ++j) {
        if (!a[i].run || !a[j].run || !(a[i].written || a[j].written)) continue;
        const Place& w = a[i].written ? a[i] : a[j];
        if (same && a[i].p == a[j].p)
          return fail(REHYAT_ERR_ARG, "%s may not be another argument", w.what);
        if (!same && a[i].p < end[j] && a[j].p < end[i] &&
            meet(a[i], a[i].dims, a[j], a[j].dims, (__int128)a[j].p - a[i].p))
          return fail(REHYAT_ERR_ARG, "%s overlaps %s", w.what, a[i].written ? a[j].what : a[i].what);
      }
  return REHYAT_OK;
}

int check_states(const char* what, const float* S) {
  if (S && !aligned16(S)) return fail(REHYAT_ERR_ALIGN, "%s is not 16-byte aligned", what);
  return REHYAT_OK;
}

int check_scratch(const DecayPlan& pl, const void* workspace, size_t ws_bytes) {
  if (!workspace || ws_bytes < pl.total)
    return fail(REHYAT_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", pl.total, ws_bytes);
  if (!aligned16(workspace)) return fail(REHYAT_ERR_ALIGN, "workspace is not 16-byte aligned");
  return REHYAT_OK;
}

}  // namespace

extern "C" {

// The binding packs these blocks by their layout.
static_assert(sizeof(rehyat_rotary_args) == 240 && sizeof(rehyat_decay_forward_args) == 208 &&
                  sizeof(rehyat_decay_backward_args) == 312 && sizeof(rehyat_decay_step_args) == 184,
              "argument block layout");

int rehyat_rotary(const rehyat_rotary_args* args, void* stream) {
  g_msg[0] = 0;
  if (!args) return fail(REHYAT_ERR_ARG, "null pointer (args)");
  const rehyat_rotary_args& a = *args;
  if (a.dtype != REHYAT_F32 && a.dtype != REHYAT_BF16)
    return fail(REHYAT_ERR_DTYPE, "unknown dtype %d", a.dtype);
  if (a.B < 1 || a.n < 0 || a.Hq < 1 || a.Hk < 0 || a.D < 1)
    return fail(REHYAT_ERR_ARG, "need B, Hq, D >= 1 and n, Hk >= 0 (B=%d n=%d Hq=%d Hk=%d D=%d)", a.B,
                a.n, a.Hq, a.Hk, a.D);
  if (a.R < 2 || a.R % 2 || a.R > a.D)
    return fail(REHYAT_ERR_SHAPE, "R=%d must be even, within 2 .. D=%d", a.R, a.D);
  if (a.axes < 1 || a.axes > rehyat::rotary::kMaxAxes)
    return fail(REHYAT_ERR_ARG, "axes=%d outside 1 .. %d", a.axes, rehyat::rotary::kMaxAxes);
  if (!std::isfinite(a.scale)) return fail(REHYAT_ERR_ARG, "scale must be finite");
  if (a.n == 0) return REHYAT_OK;
  if (!a.q.p || !a.q_out.p || !a.freq || (a.Hk > 0 && (!a.k.p || !a.k_out.p)))
    return fail(REHYAT_ERR_ARG, "null pointer");
  const bool bf16 = a.dtype == REHYAT_BF16;
  const int el = bf16 ? 2 : 4;
  rehyat::rotary::Params p{};
  auto tensor = [](const rehyat_rows& x, const rehyat_rows& y, int heads) {
    return rehyat::rotary::Tensor{x.p, y.p, x.batch, x.head, x.row, y.batch, y.head, y.row, heads};
  };
  p.t[0] = tensor(a.q, a.q_out, a.Hq);
  p.t[1] = tensor(a.k, a.k_out, a.Hk);
  bool whole = a.R % 16 == 0 && a.D % 16 == 0, in_place = true;
  for (int i = 0; i < (a.Hk ? 2 : 1); ++i) {
    const rehyat::rotary::Tensor& t = p.t[i];
    in_place &= t.x == t.y;
    if (t.x == t.y && (t.xb != t.yb || t.xh != t.yh || t.xn != t.yn))
      return fail(REHYAT_ERR_ARG, "in place needs the same strides in and out");
    const long long st[6] = {t.xb, t.xh, t.xn, t.yb, t.yh, t.yn};
    const int size[3] = {a.B, t.heads, a.n};
    whole &= aligned16(t.x) && aligned16(t.y);
    for (int j = 0; j < 6; ++j) {
      if (size[j % 3] <= 1) continue;
      whole &= (st[j] * el) % 16 == 0;
      if (j >= 3 && st[j] < a.D)
        return fail(REHYAT_ERR_ARG, "an output's stride %lld of a dimension of %d is below D=%d", st[j],
                    size[j % 3], a.D);
    }
  }
  // an input that is its own output is looked at once, as the output
  rehyat_rows q = a.q, k = a.k;
  if (q.p == a.q_out.p) q.p = nullptr;
  if (k.p == a.k_out.p) k.p = nullptr;
  const int pe = a.pos64 ? 8 : 4;
  RH_TRY(check_places({place("q_out", a.q_out, a.B, a.Hq, a.n, a.D, el, true),
                       place("k_out", a.k_out, a.B, a.Hk, a.n, a.D, el, true),
                       place("q", q, a.B, a.Hq, a.n, a.D, el, false),
                       place("k", k, a.B, a.Hk, a.n, a.D, el, false),
                       place("freq", a.freq, a.R * 4LL, false),
                       place("axis", a.axis, a.R / 2, false),
                       place("pos", a.pos, pe, {a.axes, a.B, a.n},
                             {a.pos_axis * pe, a.pos_batch * pe, a.pos_token * pe}, false)}));
  p.B = a.B; p.n = a.n; p.D = a.D; p.R = a.R;
  p.interleaved = a.interleaved; p.copy_tail = !in_place && a.R < a.D;
  p.freq = a.freq; p.axis = a.axis; p.pos = a.pos; p.pos64 = a.pos64; p.axes = a.axes;
  p.pa = a.pos_axis; p.pb = a.pos_batch; p.pn = a.pos_token;
  p.add_index = a.add_index; p.start = a.start;
  p.scale = a.scale; p.sign = a.inverse ? -1.f : 1.f;
  const int per = whole ? 16 : 2;  // dimensions a thread turns; it copies 16 or 1
  const long long units = a.R / per + (p.copy_tail ? (a.D - a.R) / (whole ? 16 : 1) : 0);
  const long long threads = (long long)a.B * a.n * units;
  const long long blocks = (threads + rehyat::rotary::kThreads - 1) / rehyat::rotary::kThreads;
  if (blocks > 0x7fffffffLL) return fail(REHYAT_ERR_ARG, "too many tokens");
  // heads are dealt out over blocks until the SMs have eight blocks each: the sines and cosines
  // are formed once per block of heads
  const int heads = a.Hq + a.Hk;
  long long split = (148 * 8 + blocks - 1) / blocks;
  if (split > heads) split = heads;
  p.heads_per_block = (int)((heads + split - 1) / split);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + p.heads_per_block - 1) / p.heads_per_block));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using namespace rehyat::rotary;
  if (whole) {
    auto kern = bf16 ? (a.interleaved ? rotary_kernel<__nv_bfloat16, true>
                                      : rotary_kernel<__nv_bfloat16, false>)
                     : (a.interleaved ? rotary_kernel<float, true> : rotary_kernel<float, false>);
    kern<<<grid, kThreads, 0, st>>>(p);
  } else {
    auto kern = bf16 ? rotary_any_kernel<__nv_bfloat16> : rotary_any_kernel<float>;
    kern<<<grid, kThreads, 0, st>>>(p);
  }
  return cuda_check(cudaGetLastError(), "rotary launch");
}

int rehyat_decay_workspace_size(int B, int H, int Hk, int N, int D, int backward, size_t* bytes) {
  g_msg[0] = 0;
  DecayDims d{B, H, Hk, N, D, REHYAT_BF16, 1.f};
  RH_TRY(check_decay(d));
  if (!bytes) return fail(REHYAT_ERR_ARG, "null pointer");
  *bytes = plan_decay(d, backward != 0, true, true).total;  // the most of every kind of call
  d.dt = REHYAT_F32;
  const size_t f32 = plan_decay(d, backward != 0, true, true).total;
  if (f32 > *bytes) *bytes = f32;
  return REHYAT_OK;
}

int rehyat_decay_forward(const rehyat_decay_forward_args* args, void* stream) {
  g_msg[0] = 0;
  if (!args) return fail(REHYAT_ERR_ARG, "null pointer (args)");
  const rehyat_decay_forward_args& a = *args;
  const DecayDims d{a.B, a.H, a.Hk, a.N, a.D, (rehyat_dtype)a.dtype, a.scale};
  RH_TRY(check_decay(d));
  if (!a.log_decay) return fail(REHYAT_ERR_ARG, "null pointer (log_decay)");
  RH_TRY(check_rows("q", a.q, d, a.H));
  RH_TRY(check_rows("k", a.k, d, a.Hk));
  RH_TRY(check_rows("v", a.v, d, a.Hk));
  RH_TRY(check_rows("out", a.out, d, a.H));
  RH_TRY(check_states("S0", a.S0));
  RH_TRY(check_states("S_last", a.S_last));
  const DecayPlan pl = plan_decay(d, false, a.lengths != nullptr, a.S_last != nullptr);
  RH_TRY(check_scratch(pl, a.workspace, a.ws_bytes));
  const int el = d.dt == REHYAT_BF16 ? 2 : 4;
  const long long states = 4LL * a.B * a.H * a.D * a.D;
  RH_TRY(check_places({place("q", a.q, a.B, a.H, a.N, a.D, el, false),
                       place("k", a.k, a.B, a.Hk, a.N, a.D, el, false),
                       place("v", a.v, a.B, a.Hk, a.N, a.D, el, false),
                       place("out", a.out, a.B, a.H, a.N, a.D, el, true),
                       place("S0", a.S0 == a.S_last ? nullptr : a.S0, states, false),
                       place("S_last", a.S_last, states, true),
                       place("log_decay", a.log_decay, 4LL * a.H, false),
                       place("lengths", a.lengths, 4LL * a.B, false),
                       place("workspace", a.workspace, pl.total, true)}));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int group = a.H / a.Hk;
  Pass p = decay_pass(d, a.log_decay, a.lengths, pl.cut, static_cast<uint8_t*>(a.workspace) + pl.fwd);
  p.a = rows_of(a.q, 1);
  p.b = rows_of(a.k, group);
  p.c = rows_of(a.v, group);
  p.e = 1;
  p.sp = p.si = a.scale;
  bool scanned;
  RH_TRY(decay_prefixes(&p, 1, d.dt, &a.S0, &a.S_last, &scanned, st));
  if (a.N == 0) return REHYAT_OK;
  set_out(p, a.out);
  return launch_decay_rows(&p, 1, d.dt, scanned, st);
}

int rehyat_decay_backward(const rehyat_decay_backward_args* args, void* stream) {
  g_msg[0] = 0;
  if (!args) return fail(REHYAT_ERR_ARG, "null pointer (args)");
  const rehyat_decay_backward_args& a = *args;
  const DecayDims d{a.B, a.H, a.Hk, a.N, a.D, (rehyat_dtype)a.dtype, a.scale};
  RH_TRY(check_decay(d));
  if (!a.log_decay) return fail(REHYAT_ERR_ARG, "null pointer (log_decay)");
  RH_TRY(check_rows("q", a.q, d, a.H));
  RH_TRY(check_rows("k", a.k, d, a.Hk));
  RH_TRY(check_rows("v", a.v, d, a.Hk));
  RH_TRY(check_rows("dout", a.dout, d, a.H));
  RH_TRY(check_rows("dq", a.dq, d, a.H));
  RH_TRY(check_rows("dk", a.dk, d, a.Hk));
  RH_TRY(check_rows("dv", a.dv, d, a.Hk));
  RH_TRY(check_states("S0", a.S0));
  RH_TRY(check_states("dS_last", a.dS_last));
  RH_TRY(check_states("dS0", a.dS0));
  const DecayPlan pl = plan_decay(d, true, a.lengths != nullptr, a.dS0 != nullptr);
  RH_TRY(check_scratch(pl, a.workspace, a.ws_bytes));
  const int el = d.dt == REHYAT_BF16 ? 2 : 4;
  const long long states = 4LL * a.B * a.H * a.D * a.D;
  RH_TRY(check_places({place("q", a.q, a.B, a.H, a.N, a.D, el, false),
                       place("k", a.k, a.B, a.Hk, a.N, a.D, el, false),
                       place("v", a.v, a.B, a.Hk, a.N, a.D, el, false),
                       place("dout", a.dout, a.B, a.H, a.N, a.D, el, false),
                       place("dq", a.dq, a.B, a.H, a.N, a.D, el, true),
                       place("dk", a.dk, a.B, a.Hk, a.N, a.D, el, true),
                       place("dv", a.dv, a.B, a.Hk, a.N, a.D, el, true),
                       place("S0", a.S0, states, false),
                       place("dS_last", a.dS_last, states, false),
                       place("dS0", a.dS0, states, true),
                       place("log_decay", a.log_decay, 4LL * a.H, false),
                       place("lengths", a.lengths, 4LL * a.B, false),
                       place("workspace", a.workspace, pl.total, true)}));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int group = a.H / a.Hk;
  const Rows rq = rows_of(a.q, 1), rk = rows_of(a.k, group), rv = rows_of(a.v, group),
             rdo = rows_of(a.dout, 1);

  // states of the prompt, forward in time, for dQ (read transposed); gradient of the state, sum of
  // scale * q dO^T backward in time, for dK (transposed) and dV
  Pass s[2] = {decay_pass(d, a.log_decay, a.lengths, pl.cut, ws + pl.fwd),
               decay_pass(d, a.log_decay, a.lengths, pl.cut, ws + pl.bwd)};
  s[0].e = 1;
  s[0].b = rk;
  s[0].c = rv;
  s[0].sp = s[0].si = a.scale;
  s[1].reverse = 1;
  s[1].b = rq;
  s[1].c = rdo;
  s[1].sp = s[1].sd = a.scale;
  const float* first[2] = {a.S0, a.dS_last};
  float* last[2] = {nullptr, a.dS0};
  bool scanned;
  RH_TRY(decay_prefixes(s, 2, d.dt, first, last, &scanned, st));
  if (a.N == 0) return REHYAT_OK;
  const bool shared = group > 1;
  const long long head = (long long)a.N * a.D;
  Pass p[3] = {s[0], s[1], s[1]};
  p[0].a = rdo;
  p[0].b = rv;
  p[0].c = rk;
  p[0].transposed = 1;
  set_out(p[0], a.dq);
  p[1].a = rv;
  p[1].b = rdo;
  p[1].c = rq;
  p[1].transposed = 1;
  p[2].a = rk;
  for (int i = 1; i < 3; ++i) {
    p[i].out_f32 = shared;
    set_out(p[i], shared ? rehyat_rows{ws + pl.part[i - 1], head * a.H, head, a.D}
                         : (i == 1 ? a.dk : a.dv));
  }
  RH_TRY(launch_decay_rows(p, 3, d.dt, scanned, st));
  if (!shared) return REHYAT_OK;
  rehyat::decay::GroupSum g{};
  for (int i = 0; i < 2; ++i) {
    const rehyat_rows& o = i ? a.dv : a.dk;
    g.part[i] = reinterpret_cast<const float*>(ws + pl.part[i]);
    g.out[i] = o.p;
    g.ob[i] = o.batch; g.oh[i] = o.head; g.on[i] = o.row;
  }
  g.Hk = a.Hk; g.group = group; g.N = a.N; g.D = a.D;
  const long long blocks = head / 4 / 1024 + 1;
  const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096), a.B * a.Hk, 2);
  if (d.dt == REHYAT_BF16)
    rehyat::decay::decay_group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(g);
  else
    rehyat::decay::decay_group_sum_kernel<float><<<grid, 256, 0, st>>>(g);
  return cuda_check(cudaGetLastError(), "decay group sum launch");
}

int rehyat_decay_step(const rehyat_decay_step_args* args, void* stream) {
  g_msg[0] = 0;
  if (!args) return fail(REHYAT_ERR_ARG, "null pointer (args)");
  const rehyat_decay_step_args& a = *args;
  const DecayDims d{a.B, a.H, a.Hk, 1, a.D, (rehyat_dtype)a.dtype, a.scale};
  RH_TRY(check_decay(d));
  if (!a.log_decay || !a.state) return fail(REHYAT_ERR_ARG, "null pointer");
  RH_TRY(check_rows("q", a.q, d, a.H));
  RH_TRY(check_rows("k", a.k, d, a.Hk));
  RH_TRY(check_rows("v", a.v, d, a.Hk));
  RH_TRY(check_rows("out", a.out, d, a.H));
  RH_TRY(check_states("state", a.state));
  if (a.pool < 1 || (!a.slots && a.pool < a.B))
    return fail(REHYAT_ERR_ARG, "a pool of %d states for %d sequences", a.pool, a.B);
  const int el = d.dt == REHYAT_BF16 ? 2 : 4;
  RH_TRY(check_places({place("q", a.q, a.B, a.H, 1, a.D, el, false),
                       place("k", a.k, a.B, a.Hk, 1, a.D, el, false),
                       place("v", a.v, a.B, a.Hk, 1, a.D, el, false),
                       place("out", a.out, a.B, a.H, 1, a.D, el, true),
                       place("state", a.state, 4LL * a.pool * a.H * a.D * a.D, true),
                       place("log_decay", a.log_decay, 4LL * a.H, false),
                       place("slots", a.slots, 4LL * a.B, false)}));
  rehyat::decay::StepParams p{};
  const int group = a.H / a.Hk;
  p.q = rows_of(a.q, 1);
  p.k = rows_of(a.k, group);
  p.v = rows_of(a.v, group);
  p.out = a.out.p;
  p.ob = a.out.batch; p.oh = a.out.head;
  p.log_decay = a.log_decay; p.state = a.state; p.slots = a.slots;
  p.B = a.B; p.H = a.H; p.D = a.D; p.pool = a.pool; p.scale = a.scale;
  using namespace rehyat::decay;
  const dim3 grid((a.D + kStepCols - 1) / kStepCols, a.H, a.B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int passes = (a.D + 15) / 16;  // of 16 rows
  const bool bf16 = d.dt == REHYAT_BF16;
  auto kern = passes <= 4 ? (bf16 ? decay_step_kernel<__nv_bfloat16, 4> : decay_step_kernel<float, 4>)
                          : (bf16 ? decay_step_kernel<__nv_bfloat16, 8> : decay_step_kernel<float, 8>);
  kern<<<grid, kStepThreads, 0, st>>>(p);
  return cuda_check(cudaGetLastError(), "decay step launch");
}

}  // extern "C"
