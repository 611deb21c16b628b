"""Chunk-by-chunk streaming session over rehyat_chunk_forward_carry ("ReHyAt overview" page, §2.3:
the chunk-wise recurrent form, where only the linear state and the overlap frames are carried).

A session owns every device buffer it needs, allocated once when it is built: the state S
[B,H,F,D] and Z [B,H,F] (fp32), the carry (the last To frames of K and V seen, [B,H,To*L,D]) and
the workspace.  Each step is one library call on the incoming chunk: the library assembles the
softmax window from the carry and the chunk, attends, folds the frames the next window no longer
holds into S and Z, and updates the carry, so memory stays constant however long the video is.

Tc and To are the largest chunk and overlap the session accepts.  A step may pass a shorter
chunk and its own overlap (`To`) and the next step's (`To_next`): a variable schedule of the
"ReHyAt overview" page §5.2 (a longer first chunk, more overlap where motion is strong).

The session's state is its checkpoint: S, Z, the carry and the number of frames seen.
state_dict() copies it to host memory; load_state_dict() puts it back into a fresh session, and
the steps that follow produce the same bits as an uninterrupted run (same kernels, same order).

DecayStream is the same for the pure recurrent layer (linear attention with a decay per head).
"""
from __future__ import annotations

import torch

from . import binding as rb


class ChunkStream:
    def __init__(self, Wq, bq, Wk, bk, *, B: int, P: int, frame_tokens: int, Tc: int, To: int,
                 phi: int = rb.PHI_POLY, dtype: torch.dtype = torch.bfloat16,
                 device: torch.device | None = None):
        dev = device or Wq.device
        H, G, Fg, Dg = Wq.shape
        D, F = Dg * G, Fg * G
        self.Wq, self.bq, self.Wk, self.bk = Wq, bq, Wk, bk
        self.B, self.H, self.D, self.F, self.P, self.phi = B, H, D, F, P, phi
        self.L, self.Tc, self.To = frame_tokens, Tc, To
        self.dtype, self.device = dtype, dev
        self.frames_seen = 0
        self.S = torch.zeros(B, H, F, D, dtype=torch.float32, device=dev)
        self.Z = torch.zeros(B, H, F, dtype=torch.float32, device=dev)
        self.k_carry = torch.zeros(B, H, To * frame_tokens, D, dtype=dtype, device=dev)
        self.v_carry = torch.zeros_like(self.k_carry)
        d = rb.Dims(B, H, D, F, G, P, phi)
        code = rb.REHYAT_BF16 if dtype == torch.bfloat16 else rb.REHYAT_F32
        self.workspace = torch.empty(rb.chunk_carry_workspace_size(d, code, frame_tokens, Tc, To,
                                                                   To),
                                     dtype=torch.uint8, device=dev)

    def reset(self) -> None:
        """Start a new sequence (the buffers are kept)."""
        self.S.zero_()
        self.Z.zero_()
        self.frames_seen = 0

    def step(self, q, k, v, out: torch.Tensor | None = None, To: int | None = None,
             To_next: int | None = None) -> torch.Tensor:
        """Attend the next chunk (q, k, v: [B,H,chunk_frames*L,D], 1 <= chunk_frames <= Tc);
        returns its output [B,H,chunk_frames*L,D].  To / To_next: this chunk's and the next
        chunk's overlap (default: the session's To)."""
        L, cap = self.L, self.To
        To = cap if To is None else To
        n = q.shape[2]
        if n % L or not 1 <= n // L <= self.Tc or k.shape != q.shape or v.shape != q.shape:
            raise ValueError(f"chunk of {n} rows is not 1..{self.Tc} frames of {L} tokens")
        if not 0 <= To <= cap or (To_next is not None and not 0 <= To_next <= cap):
            raise ValueError(f"overlaps must lie in [0, {cap}]")
        out = rb.chunk_forward_carry(q, k, v, self.Wq, self.bq, self.Wk, self.bk, self.S, self.Z,
                                     self.k_carry, self.v_carry, P=self.P, phi=self.phi,
                                     frame_tokens=L, frames_before=self.frames_seen, To=To,
                                     To_next=To_next, out=out, workspace=self.workspace)
        self.frames_seen += n // L
        return out

    def state_dict(self) -> dict:
        """The session's state, copied to host memory."""
        return {"S": self.S.cpu(), "Z": self.Z.cpu(), "k_carry": self.k_carry.cpu(),
                "v_carry": self.v_carry.cpu(), "frames_seen": self.frames_seen,
                "shape": (self.B, self.H, self.D, self.F, self.P, self.L, self.Tc, self.To,
                          self.phi)}

    def load_state_dict(self, st: dict) -> None:
        if tuple(st["shape"]) != (self.B, self.H, self.D, self.F, self.P, self.L, self.Tc,
                                  self.To, self.phi):
            raise ValueError(f"state of shape {st['shape']} does not fit this session")
        self.S.copy_(st["S"])
        self.Z.copy_(st["Z"])
        self.k_carry.copy_(st["k_carry"])
        self.v_carry.copy_(st["v_carry"])
        self.frames_seen = int(st["frames_seen"])


class DecayStream:
    """Decayed linear attention as a session: prompts of any length, then one token at a time, each
    going on from the states the calls before left (decay_forward and decay_step of the binding),
    with rotary positions on q and k counted per sequence.

    The session owns the states [B,H,D,D] fp32 and the number of rows each sequence has seen ([B]
    int32 on the device, so ragged prompts and captured calls need no host value).  Memory does not
    grow with the rows seen.  Scratch is allocated by each prompt: one kept here would be replaced
    by a longer prompt's while a captured prompt still writes to it.

    log_decay [H] fp32; Hk key/value heads (default H); scale defaults to D ** -0.5.  freq (fp64
    [R/2], see rotary_frequencies) turns on rotary positions; rotary_scale and interleaved as in
    `rotary`.  state_dict() / load_state_dict() checkpoint it: the calls that follow a resume
    produce the same bits as an uninterrupted run."""

    def __init__(self, log_decay, *, B: int, D: int, Hk: int | None = None,
                 scale: float | None = None, freq: torch.Tensor | None = None,
                 rotary_scale: float = 1.0, interleaved: bool = False):
        self.log_decay, self.freq = log_decay, freq
        self.B, self.H, self.D = B, log_decay.shape[0], D
        self.Hk = self.H if Hk is None else Hk
        self.scale = D ** -0.5 if scale is None else scale
        self.rotary_scale, self.interleaved = rotary_scale, interleaved
        dev = log_decay.device
        self.state = torch.zeros(B, self.H, D, D, dtype=torch.float32, device=dev)
        self.seen = torch.zeros(B, dtype=torch.int32, device=dev)

    def reset(self) -> None:
        """Start new sequences (the buffers are kept)."""
        self.state.zero_()
        self.seen.zero_()

    def _check(self, q, k, v) -> None:
        B, H, Hk, D = self.B, self.H, self.Hk, self.D
        n = q.shape[2] if q.dim() == 4 else 0
        if tuple(q.shape) != (B, H, n, D) or tuple(k.shape) != (B, Hk, n, D) or v.shape != k.shape:
            raise ValueError(f"q, k, v must be [{B},{H},n,{D}], [{B},{Hk},n,{D}] and the same, got "
                             f"{tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")

    def _turn(self, q, k):
        if self.freq is None:
            return q, k
        return rb.rotary(q, k, self.freq, start=self.seen, scale=self.rotary_scale,
                         interleaved=self.interleaved)

    def prompt(self, q, k, v, lengths: torch.Tensor | None = None) -> torch.Tensor:
        """Outputs [B,H,N,D] of the next N rows of every sequence, or of the first lengths[b]
        (int32 [B] on the device, 0 .. N) of a padded batch, whose other rows are zero."""
        self._check(q, k, v)
        N = q.shape[2]
        q, k = self._turn(q, k)
        out, _ = rb.decay_forward(q, k, v, self.log_decay, scale=self.scale, lengths=lengths,
                                  state=self.state, final_state=self.state)
        self.seen += N if lengths is None else lengths.clamp(0, N)
        return out

    def step(self, q, k, v) -> torch.Tensor:
        """Outputs [B,H,1,D] of the next token of every sequence."""
        self._check(q, k, v)
        q, k = self._turn(q, k)
        out = rb.decay_step(q, k, v, self.log_decay, self.state, scale=self.scale)
        self.seen += 1
        return out

    def _shape(self):
        return (self.B, self.H, self.Hk, self.D)

    def state_dict(self) -> dict:
        """The session's state, copied to host memory."""
        return {"state": self.state.cpu(), "seen": self.seen.cpu(), "shape": self._shape()}

    def load_state_dict(self, st: dict) -> None:
        if tuple(st["shape"]) != self._shape():
            raise ValueError(f"state of shape {st['shape']} does not fit this session")
        self.state.copy_(st["state"])
        self.seen.copy_(st["seen"])
