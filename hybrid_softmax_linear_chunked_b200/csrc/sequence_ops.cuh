// Host side of the sequence operators (rotary positions, decayed linear attention): argument
// checks, the choice of segments, workspace plans and launches.  Included by rehyat.cu after its
// helpers (fail, RH_TRY, cuda_check, Carve).
#pragma once

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

// A strided [B, heads, N, D] tensor: aligned, whole 16-byte strides, rows that do not overlap.
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

// Segments of a sequence: one CTA each, so their number trades whole waves of the 148 SMs against
// the state pass that more than one segment needs (about half the work of the row pass).  `blocks`
// 128-row blocks; +1 block a CTA for its start.
struct Segments {
  int n, rows;
};
Segments decay_segments(int BH, int N, bool states_anyway) {
  const int blocks = (N + rehyat::decay::kBlockRows - 1) / rehyat::decay::kBlockRows;
  Segments best{1, blocks > 0 ? blocks * rehyat::decay::kBlockRows : rehyat::decay::kBlockRows};
  long long best_cost = -1;
  for (int n = 1; n <= blocks && n <= 256; ++n) {
    const int per = (blocks + n - 1) / n;
    const int used = (blocks + per - 1) / per;  // segments that hold rows
    if (used != n) continue;
    const long long waves = ((long long)BH * n + 147) / 148;
    const long long cost = waves * (per + 1) * (n > 1 || states_anyway ? 3 : 2);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = Segments{n, per * rehyat::decay::kBlockRows};
    }
  }
  return best;
}

struct DecayPlan {
  Segments seg;
  size_t fwd, bwd, part, total;
};
DecayPlan plan_decay(const DecayDims& a, bool backward) {
  DecayPlan p{};
  const size_t BH = (size_t)a.B * a.H;
  p.seg = decay_segments((int)BH, a.N, true);
  Carve cv;
  const size_t states = BH * p.seg.n * a.D * a.D * 4;
  p.fwd = cv.take(states);
  if (backward) {
    p.bwd = cv.take(states);
    // per query head, where dk and dv are sums over the heads that share a key/value head
    p.part = cv.take(a.H != a.Hk ? BH * (size_t)a.N * a.D * 4 : 0);
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

// exact: the last state will be given out, so bf16 sums are formed from two-part products.
int launch_decay_states(const Pass& p, rehyat_dtype dt, bool exact, cudaStream_t st) {
  const dim3 grid(p.nseg, p.B * p.H);
  if (dt == REHYAT_BF16) {
    using namespace rehyat::decay::tc;
    CUtensorMap mb, mc;
    RH_TRY(map_of(&mb, p.b, p));
    RH_TRY(map_of(&mc, p.c, p));
    auto k = exact ? decay_states_bf16_kernel<true> : decay_states_bf16_kernel<false>;
    RH_TRY(cuda_check(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)kStSmem), "decay states attr"));
    k<<<grid, kStThreads, kStSmem, st>>>(mb, mc, p);
  } else {
    using namespace rehyat::decay;
    const int smem = states_smem_floats(padded(p.D)) * 4;
    RH_TRY(cuda_check(cudaFuncSetAttribute(decay_states_kernel,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                      "decay states attr"));
    decay_states_kernel<<<grid, kThreads, smem, st>>>(p);
  }
  return cuda_check(cudaGetLastError(), "decay states launch");
}

// behind_scan: the launch before is this call's scan, whose prefix the kernel waits for.
int launch_decay_rows(const Pass& p, rehyat_dtype dt, bool out_f32, bool behind_scan,
                      cudaStream_t st) {
  const dim3 grid(p.nseg, p.B * p.H);
  if (dt == REHYAT_F32) {
    using namespace rehyat::decay;
    const int smem = rows_smem_floats(padded(p.D)) * 4;
    RH_TRY(cuda_check(cudaFuncSetAttribute(decay_rows_kernel,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                      "decay rows attr"));
    decay_rows_kernel<<<grid, kThreads, smem, st>>>(p);
    return cuda_check(cudaGetLastError(), "decay rows launch");
  }
  using namespace rehyat::decay::tc;
  CUtensorMap ma, mb, mc, mo;
  RH_TRY(map_of(&ma, p.a, p));
  RH_TRY(map_of(&mb, p.b, p));
  RH_TRY(map_of(&mc, p.c, p));
  mo = ma;  // unused with fp32 output
  if (!out_f32) RH_TRY(make_map_rows(&mo, Rows{p.out, p.ob, p.oh, p.on, 1}, p.D, p.N, p.H, p.B));
  auto k = p.reverse ? (out_f32 ? decay_rows_bf16_kernel<true, true> : decay_rows_bf16_kernel<true, false>)
                     : decay_rows_bf16_kernel<false, false>;
  RH_TRY(cuda_check(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRwSmem),
                    "decay rows attr"));
  Behind l(grid, kRwThreads, kRwSmem, st, behind_scan);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, k, ma, mb, mc, mo, p), "decay rows launch");
}

int launch_decay_scan(const Pass& p, const float* S0, float* last, bool need_prefix,
                      bool behind_states, cudaStream_t st) {
  const int n4 = p.D * p.D / 4;
  Behind l(dim3((n4 + 255) / 256, p.B * p.H), 256, 0, st, behind_states);
  return cuda_check(cudaLaunchKernelEx(&l.cfg, rehyat::decay::decay_scan_kernel, p.delta, S0, last,
                                       p.log_decay, p.lengths, p.H, p.N, p.D, p.nseg, p.seg_rows,
                                       p.reverse, (int)need_prefix),
                    "decay scan launch");
}

// The state before every segment of a pass (rows b, c; time direction and e as in `p`) from `S0`
// (or zero), and the state after the last into `last` unless null.  *prefix: where the row pass
// reads it ([B*H][nseg][D][D]), null for zero.  *scanned: whether a scan was launched for them.
int decay_prefix(Pass p, rehyat_dtype dt, const float* S0, float* last, const float** prefix,
                 bool* scanned, cudaStream_t st) {
  const bool many = p.nseg > 1, bf16 = dt == REHYAT_BF16;
  *prefix = nullptr;
  *scanned = false;
  if (!many && !last) {
    *prefix = S0;
    return REHYAT_OK;
  }
  if (p.N > 0) {
    p.seg_skip = last ? -1 : (p.reverse ? 0 : p.nseg - 1);
    RH_TRY(launch_decay_states(p, dt, last != nullptr, st));
  }
  // the row pass reads the workspace's copy of S0, since `last` may be S0
  RH_TRY(launch_decay_scan(p, S0, last, many || S0, bf16 && p.N > 0, st));
  if (many || S0) *prefix = p.delta;
  *scanned = true;
  return REHYAT_OK;
}

Pass decay_pass(const DecayDims& a, const float* log_decay, const int* lengths,
                const Segments& s) {
  Pass p{};
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.B = a.B; p.H = a.H; p.N = a.N; p.D = a.D;
  p.nseg = s.n; p.seg_rows = s.rows;
  p.seg_skip = -1;
  p.sp = p.si = p.sd = 1.f;
  return p;
}

void set_out(Pass& p, const rehyat_rows& o) {
  p.out = o.p;
  p.ob = o.batch; p.oh = o.head; p.on = o.row;
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
    for (int j = 0; j < 6; ++j)
      if (size[j % 3] > 1) whole &= (st[j] * el) % 16 == 0;
  }
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
  const DecayDims d{B, H, Hk, N, D, REHYAT_BF16, 1.f};
  RH_TRY(check_decay(d));
  if (!bytes) return fail(REHYAT_ERR_ARG, "null pointer");
  *bytes = plan_decay(d, backward != 0).total;
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
  const DecayPlan pl = plan_decay(d, false);
  RH_TRY(check_scratch(pl, a.workspace, a.ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int group = a.H / a.Hk;
  Pass p = decay_pass(d, a.log_decay, a.lengths, pl.seg);
  p.a = rows_of(a.q, 1);
  p.b = rows_of(a.k, group);
  p.c = rows_of(a.v, group);
  p.e = 1;
  p.sp = p.si = a.scale;
  p.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + pl.fwd);
  bool scanned;
  RH_TRY(decay_prefix(p, d.dt, a.S0, a.S_last, &p.prefix, &scanned, st));
  if (a.N == 0) return REHYAT_OK;
  set_out(p, a.out);
  return launch_decay_rows(p, d.dt, false, scanned, st);
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
  const DecayPlan pl = plan_decay(d, true);
  RH_TRY(check_scratch(pl, a.workspace, a.ws_bytes));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int group = a.H / a.Hk;
  const Rows rq = rows_of(a.q, 1), rk = rows_of(a.k, group), rv = rows_of(a.v, group),
             rdo = rows_of(a.dout, 1);

  // dQ: forward in time over the states of the prompt, transposed
  Pass f = decay_pass(d, a.log_decay, a.lengths, pl.seg);
  f.delta = reinterpret_cast<float*>(ws + pl.fwd);
  f.e = 1;
  bool scanned = false;
  if (a.N > 0) {
    f.b = rk;
    f.c = rv;
    RH_TRY(decay_prefix(f, d.dt, a.S0, nullptr, &f.prefix, &scanned, st));
    f.a = rdo;
    f.b = rv;
    f.c = rk;
    f.transposed = 1;
    f.sp = f.si = a.scale;
    set_out(f, a.dq);
    RH_TRY(launch_decay_rows(f, d.dt, false, scanned, st));
  }

  // dK, dV: backward in time over the gradient of the state, sum of scale * q dO^T
  Pass r = decay_pass(d, a.log_decay, a.lengths, pl.seg);
  r.delta = reinterpret_cast<float*>(ws + pl.bwd);
  r.reverse = 1;
  r.e = 0;
  r.b = rq;
  r.c = rdo;
  r.sp = r.sd = a.scale;
  RH_TRY(decay_prefix(r, d.dt, a.dS_last, a.dS0, &r.prefix, &scanned, st));
  if (a.N == 0) return REHYAT_OK;
  float* part = reinterpret_cast<float*>(ws + pl.part);
  for (int i = 0; i < 2; ++i) {
    Pass p = r;
    p.a = i ? rk : rv;
    p.b = i ? rq : rdo;
    p.c = i ? rdo : rq;
    p.transposed = i ? 0 : 1;
    const rehyat_rows& dst = i ? a.dv : a.dk;
    if (group == 1) {
      set_out(p, dst);
      RH_TRY(launch_decay_rows(p, d.dt, false, scanned && i == 0, st));
      continue;
    }
    const long long head = (long long)a.N * a.D;
    set_out(p, rehyat_rows{part, head * a.H, head, a.D});
    RH_TRY(launch_decay_rows(p, d.dt, true, scanned && i == 0, st));
    const long long vec = head / 4;
    const dim3 grid((unsigned)(vec / 1024 + 1 < 4096 ? vec / 1024 + 1 : 4096), a.B * a.Hk);
    if (d.dt == REHYAT_BF16)
      rehyat::decay::decay_group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
          part, static_cast<__nv_bfloat16*>(dst.p), dst.batch, dst.head, dst.row, a.Hk, group, a.N,
          a.D);
    else
      rehyat::decay::decay_group_sum_kernel<float><<<grid, 256, 0, st>>>(
          part, static_cast<float*>(dst.p), dst.batch, dst.head, dst.row, a.Hk, group, a.N, a.D);
    RH_TRY(cuda_check(cudaGetLastError(), "decay group sum launch"));
  }
  return REHYAT_OK;
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
