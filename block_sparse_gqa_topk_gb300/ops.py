"""PyTorch-facing wrappers of the C ABI (device memory and streams only).

Each function checks dtypes/shapes, allocates outputs and a workspace with torch,
and calls the same-named entry point of libmsa.so on the current CUDA stream.
There is no fallback: without the built library or a CUDA device these raise.

Layouts (contiguous): q, o [B,N,H_q,d]; k, v [B,N,H_kv,d]; q_idx [B,N,H_kv,d_idx];
k_idx [B,N,d_idx]; lse [B,H_q,N] f32; lse_idx [B,H_kv,N] f32;
block_idx [B,H_kv,N,topk] int32.
"""
from __future__ import annotations

import dataclasses
import math

import torch
from torch.autograd import forward_ad

from . import _lib

_WS = {}


def _workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    """Per-device scratch buffer, grown on demand (256-byte aligned by torch)."""
    key = (device.type, device.index)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _WS[key] = buf
    return buf


def release_workspace() -> None:
    _WS.clear()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The same handle without a Stream object: a decode step's calls are host-bound (0.1 us for
# 2.0 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(index: int) -> int:
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype=torch.bfloat16, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def make_problem(B, N, H_q, H_kv, d, d_idx, topk, Bk=128, causal=True, scale=None,
                 scale_idx=None) -> _lib.Problem:
    return _lib.Problem(B=B, N=N, H_q=H_q, H_kv=H_kv, d=d, d_idx=d_idx, Bk=Bk, topk=topk,
                        causal=int(bool(causal)),
                        scale=float(scale if scale is not None else 1.0 / math.sqrt(d)),
                        scale_idx=float(scale_idx if scale_idx is not None else 0.0))


def new_plan(B, N, H_q, H_kv, topk, *, d=128, d_idx=64, Bk: int = 128, causal: bool = True,
             device="cuda") -> torch.Tensor:
    """A buffer for one step's inverted lists ("plan").  Pass it as `plan=` to
    msa_index_topk, which builds it, then to msa_fwd and msa_bwd of the same step, which
    read it instead of each building their own (see include/msa.h)."""
    prob = make_problem(B, N, H_q, H_kv, d, d_idx, topk, Bk, causal, None, None)
    n = _lib.msa_plan_size(prob)
    if n == 0:
        raise ValueError("invalid problem for a plan")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _plan_arg(plan):
    if plan.dtype != torch.uint8 or not plan.is_cuda or not plan.is_contiguous():
        raise ValueError("plan must be a contiguous uint8 CUDA tensor from new_plan")
    return _ptr(plan), plan.numel()


def msa_index_topk(q_idx: torch.Tensor, k_idx: torch.Tensor, topk: int = 16, *, H_q=None, d=None,
                   Bk: int = 128, causal: bool = True, scale_idx=None, with_lse: bool = True,
                   plan=None):
    """Index branch: returns (block_idx [B,H_kv,N,topk] int32, lse_idx [B,H_kv,N] f32 or None).
    With `plan` (from new_plan) it also builds the step's shared plan there."""
    _need(q_idx, "q_idx", ndim=4)
    _need(k_idx, "k_idx", ndim=3)
    B, N, H_kv, d_idx = q_idx.shape
    if tuple(k_idx.shape) != (B, N, d_idx):
        raise ValueError(f"k_idx must be {(B, N, d_idx)}, got {tuple(k_idx.shape)}")
    prob = make_problem(B, N, H_q or H_kv, H_kv, d or 128, d_idx, topk, Bk, causal, None, scale_idx)
    dev = q_idx.device
    block_idx = torch.empty((B, H_kv, N, topk), dtype=torch.int32, device=dev)
    lse_idx = torch.empty((B, H_kv, N), dtype=torch.float32, device=dev) if with_lse else None
    nws = _lib.msa_workspace_size(prob, _lib.MSA_WS_INDEX) if with_lse else 0
    ws = _workspace(nws, dev) if with_lse else None
    if plan is None:
        rc = _lib.msa_index_topk(prob, _ptr(q_idx), _ptr(k_idx), _ptr(block_idx), _ptr(lse_idx),
                                 _ptr(ws), nws, _stream(dev))
    else:
        pp, pn = _plan_arg(plan)
        rc = _lib.msa_index_topk_plan(prob, _ptr(q_idx), _ptr(k_idx), _ptr(block_idx),
                                      _ptr(lse_idx), pp, pn, _ptr(ws), nws, _stream(dev))
    _lib.check(rc, "msa_index_topk")
    return block_idx, lse_idx


def msa_fwd(q, k, v, block_idx, *, scale=None, Bk: int = 128, causal: bool = True, d_idx=64,
            plan=None):
    """Main branch forward: returns (o [B,N,H_q,d] bf16, lse [B,H_q,N] f32).  With `plan`
    it reads the step's shared plan (built by msa_index_topk for this block_idx)."""
    _need(q, "q", ndim=4)
    _need(k, "k", ndim=4)
    _need(v, "v", ndim=4)
    _need(block_idx, "block_idx", torch.int32, ndim=4)
    B, N, H_q, d = q.shape
    H_kv = k.shape[2]
    topk = block_idx.shape[3]
    if tuple(k.shape) != (B, N, H_kv, d) or tuple(v.shape) != (B, N, H_kv, d):
        raise ValueError("k, v must be [B,N,H_kv,d] matching q")
    if tuple(block_idx.shape) != (B, H_kv, N, topk):
        raise ValueError("block_idx must be [B,H_kv,N,topk]")
    prob = make_problem(B, N, H_q, H_kv, d, d_idx, topk, Bk, causal, scale, None)
    dev = q.device
    o = torch.empty_like(q)
    lse = torch.empty((B, H_q, N), dtype=torch.float32, device=dev)
    nws = _lib.msa_workspace_size(prob, _lib.MSA_WS_FWD)
    ws = _workspace(nws, dev)
    if plan is None:
        rc = _lib.msa_fwd(prob, _ptr(q), _ptr(k), _ptr(v), _ptr(block_idx), _ptr(o), _ptr(lse),
                          _ptr(ws), nws, _stream(dev))
    else:
        pp, pn = _plan_arg(plan)
        rc = _lib.msa_fwd_plan(prob, _ptr(q), _ptr(k), _ptr(v), _ptr(block_idx), pp, pn, _ptr(o),
                               _ptr(lse), _ptr(ws), nws, _stream(dev))
    _lib.check(rc, "msa_fwd")
    return o, lse


def msa_bwd(q, k, v, o, lse, dO, q_idx, k_idx, block_idx, lse_idx, kl_weight: float, *,
            scale=None, scale_idx=None, Bk: int = 128, causal: bool = True, plan=None):
    """Fused backward: returns dict dq, dk, dv, dq_idx, dk_idx (bf16) and kl (f32 [1]).
    With `plan` it reads the step's shared plan (built by msa_index_topk)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (q_idx, "q_idx")):
        _need(t, n, ndim=4)
    _need(k_idx, "k_idx", ndim=3)
    _need(lse, "lse", torch.float32, ndim=3)
    _need(lse_idx, "lse_idx", torch.float32, ndim=3)
    _need(block_idx, "block_idx", torch.int32, ndim=4)
    B, N, H_q, d = q.shape
    H_kv = k.shape[2]
    d_idx = q_idx.shape[3]
    topk = block_idx.shape[3]
    prob = make_problem(B, N, H_q, H_kv, d, d_idx, topk, Bk, causal, scale, scale_idx)
    dev = q.device
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
           "dq_idx": torch.empty_like(q_idx), "dk_idx": torch.empty_like(k_idx),
           "kl": torch.empty(1, dtype=torch.float32, device=dev)}
    nws = _lib.msa_workspace_size(prob, _lib.MSA_WS_BWD)
    ws = _workspace(nws, dev)
    outs = (_ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dq_idx"]),
            _ptr(out["dk_idx"]), _ptr(out["kl"]), _ptr(ws), nws, _stream(dev))
    ins = (prob, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(q_idx), _ptr(k_idx),
           _ptr(block_idx), _ptr(lse_idx))
    if plan is None:
        rc = _lib.msa_bwd(*ins, kl_weight, *outs)
    else:
        rc = _lib.msa_bwd_plan(*ins, *_plan_arg(plan), kl_weight, *outs)
    _lib.check(rc, "msa_bwd")
    return out


def device_status() -> int:
    """Reads and clears the current device's status word (after syncing the stream)."""
    return _lib.msa_get_device_status(_stream(torch.device("cuda", torch.cuda.current_device())))


class MSAFunction(torch.autograd.Function):
    """o = MSA(q, k, v, q_idx, k_idx).  Backward returns dq, dk, dv from dO and the
    KL-alignment gradients for q_idx, k_idx (teacher detached).  The KL value of
    the last backward is kept in ctx-free storage `MSAFunction.last_kl`."""

    last_kl = None

    @staticmethod
    def forward(ctx, q, k, v, q_idx, k_idx, topk, Bk, scale, scale_idx, kl_coef):
        B, N, H_q, d = q.shape
        # one plan (inverted lists of block_idx) serves the index LSE, forward and backward
        plan = new_plan(B, N, H_q, k.shape[2], topk, d=d, d_idx=q_idx.shape[3], Bk=Bk,
                        device=q.device)
        block_idx, lse_idx = msa_index_topk(q_idx, k_idx, topk, H_q=H_q, d=d, Bk=Bk,
                                            scale_idx=scale_idx, with_lse=True, plan=plan)
        o, lse = msa_fwd(q, k, v, block_idx, scale=scale, Bk=Bk, d_idx=q_idx.shape[3], plan=plan)
        ctx.save_for_backward(q, k, v, q_idx, k_idx, o, lse, block_idx, lse_idx, plan)
        ctx.cfg = (Bk, scale, scale_idx, kl_coef)
        ctx.mark_non_differentiable(block_idx)
        return o, block_idx

    @staticmethod
    def backward(ctx, dO, _dblock):
        q, k, v, q_idx, k_idx, o, lse, block_idx, lse_idx, plan = ctx.saved_tensors
        Bk, scale, scale_idx, kl_coef = ctx.cfg
        B, N, H_q, _ = q.shape
        H_kv = k.shape[2]
        w = kl_coef / float(B * H_kv * N)
        g = msa_bwd(q, k, v, o, lse, dO.contiguous(), q_idx, k_idx, block_idx, lse_idx, w,
                    scale=scale, scale_idx=scale_idx, Bk=Bk, plan=plan)
        MSAFunction.last_kl = g["kl"]
        return g["dq"], g["dk"], g["dv"], g["dq_idx"], g["dk_idx"], None, None, None, None, None


def attention(q, k, v, q_idx, k_idx, topk: int = 16, Bk: int = 128, scale=None, scale_idx=None,
              kl_coef: float = 1.0, *, rope=None, positions=None):
    """MSA attention for training: returns o; backward also trains the index heads.
    Stopping the gradient at the index-branch input is the caller's job (feed the
    projections a detached hidden state).  With `rope` (from new_rope, rot_dim <= d_idx) the
    four operands of the scores get rotary positions first: each token's index in its
    sequence, or positions [B, N]."""
    if rope is not None:
        q, k, q_idx, k_idx = _rotated((q, k, q_idx, k_idx), rope, positions)
    elif positions is not None:
        raise ValueError("positions are those of rope, which is not given")
    o, _ = MSAFunction.apply(q, k, v, q_idx, k_idx, topk, Bk, scale, scale_idx, kl_coef)
    return o


# ---------------------------------------------------------------------------
# Packed variable-length batches (cu_seqlens on the device): each sequence is its own
# causal problem; token axes are packed, per-sequence outputs are stored one sequence
# after another in the single-sequence layout (see include/msa.h).  Every call runs a
# fixed number of kernels whatever the number of sequences; cu_seqlens is checked on
# the device (a bad batch writes nothing and sets the device status).
# ---------------------------------------------------------------------------
def _cu_dev(cu_seqlens, dev):
    if not isinstance(cu_seqlens, torch.Tensor):
        cu_seqlens = torch.tensor([int(x) for x in cu_seqlens], dtype=torch.int32)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.ndim != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of num_seqs + 1 offsets")
    return cu_seqlens.to(dev).contiguous()


def _max_len(cu, max_seqlen):
    """max_seqlen as given, else read from cu_seqlens (one device-to-host copy)."""
    if max_seqlen is not None:
        return int(max_seqlen)
    return int((cu[1:] - cu[:-1]).max()) if cu.numel() > 1 else 0


def varlen_view(flat: torch.Tensor, cu_seqlens, s: int, heads: int, per_row: int = 1):
    """Sequence s of a packed per-sequence output: [heads, L_s, per_row] (block_idx:
    heads = H_kv, per_row = topk; lse_idx: H_kv, 1; lse: H_q, 1)."""
    cu = cu_seqlens.tolist() if isinstance(cu_seqlens, torch.Tensor) else list(cu_seqlens)
    a, b = cu[s] * heads * per_row, cu[s + 1] * heads * per_row
    return flat[a:b].view(heads, cu[s + 1] - cu[s], per_row)


def msa_index_topk_varlen(q_idx, k_idx, cu_seqlens, topk: int = 16, *, max_seqlen=None, H_q=None,
                          d=None, Bk: int = 128, causal: bool = True, scale_idx=None,
                          with_lse: bool = True):
    """q_idx [T,H_kv,d_idx], k_idx [T,d_idx], cu_seqlens (int32, num_seqs + 1) -> packed
    block_idx (int32, H_kv*T*topk) and lse_idx (f32, H_kv*T) or None."""
    _need(q_idx, "q_idx", ndim=3)
    _need(k_idx, "k_idx", ndim=2)
    T, H_kv, d_idx = q_idx.shape
    if tuple(k_idx.shape) != (T, d_idx):
        raise ValueError("q_idx and k_idx must share the token axis")
    dev = q_idx.device
    cu = _cu_dev(cu_seqlens, dev)
    n = cu.numel() - 1
    prob = make_problem(1, _max_len(cu, max_seqlen), H_q or H_kv, H_kv, d or 128, d_idx, topk, Bk,
                        causal, None, scale_idx)
    block_idx = torch.empty(H_kv * T * topk, dtype=torch.int32, device=dev)
    lse_idx = torch.empty(H_kv * T, dtype=torch.float32, device=dev) if with_lse else None
    nws = _lib.msa_workspace_size_varlen(prob, n, T, _lib.MSA_WS_INDEX)
    ws = _workspace(nws, dev)
    rc = _lib.msa_index_topk_varlen(prob, _ptr(cu), n, T, _ptr(q_idx), _ptr(k_idx),
                                    _ptr(block_idx), _ptr(lse_idx), _ptr(ws), nws, _stream(dev))
    _lib.check(rc, "msa_index_topk_varlen")
    return block_idx, lse_idx


def msa_fwd_varlen(q, k, v, block_idx, cu_seqlens, topk: int, *, max_seqlen=None, scale=None,
                   Bk: int = 128, causal: bool = True, d_idx=64):
    """q [T,H_q,d], k, v [T,H_kv,d], packed block_idx -> o [T,H_q,d], packed lse (H_q*T)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, ndim=3)
    _need(block_idx, "block_idx", torch.int32, ndim=1)
    T, H_q, d = q.shape
    H_kv = k.shape[1]
    if block_idx.numel() != H_kv * T * topk:
        raise ValueError("block_idx must hold H_kv*T*topk entries")
    dev = q.device
    cu = _cu_dev(cu_seqlens, dev)
    n = cu.numel() - 1
    prob = make_problem(1, _max_len(cu, max_seqlen), H_q, H_kv, d, d_idx, topk, Bk, causal, scale,
                        None)
    o = torch.empty_like(q)
    lse = torch.empty(H_q * T, dtype=torch.float32, device=dev)
    nws = _lib.msa_workspace_size_varlen(prob, n, T, _lib.MSA_WS_FWD)
    ws = _workspace(nws, dev)
    rc = _lib.msa_fwd_varlen(prob, _ptr(cu), n, T, _ptr(q), _ptr(k), _ptr(v), _ptr(block_idx),
                             _ptr(o), _ptr(lse), _ptr(ws), nws, _stream(dev))
    _lib.check(rc, "msa_fwd_varlen")
    return o, lse


def msa_bwd_varlen(q, k, v, o, lse, dO, q_idx, k_idx, block_idx, lse_idx, kl_weight: float,
                   cu_seqlens, topk: int, *, max_seqlen=None, scale=None, scale_idx=None,
                   Bk: int = 128, causal: bool = True):
    """Fused backward over a packed batch: dict dq, dk, dv, dq_idx, dk_idx and kl (sum over
    every row of every sequence)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (q_idx, "q_idx")):
        _need(t, n, ndim=3)
    _need(k_idx, "k_idx", ndim=2)
    _need(lse, "lse", torch.float32, ndim=1)
    _need(lse_idx, "lse_idx", torch.float32, ndim=1)
    _need(block_idx, "block_idx", torch.int32, ndim=1)
    T, H_q, d = q.shape
    H_kv = k.shape[1]
    d_idx = q_idx.shape[2]
    dev = q.device
    cu = _cu_dev(cu_seqlens, dev)
    n = cu.numel() - 1
    prob = make_problem(1, _max_len(cu, max_seqlen), H_q, H_kv, d, d_idx, topk, Bk, causal, scale,
                        scale_idx)
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
           "dq_idx": torch.empty_like(q_idx), "dk_idx": torch.empty_like(k_idx),
           "kl": torch.empty(1, dtype=torch.float32, device=dev)}
    nws = _lib.msa_workspace_size_varlen(prob, n, T, _lib.MSA_WS_BWD)
    ws = _workspace(nws, dev)
    rc = _lib.msa_bwd_varlen(prob, _ptr(cu), n, T, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                             _ptr(dO), _ptr(q_idx), _ptr(k_idx), _ptr(block_idx), _ptr(lse_idx),
                             kl_weight, _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                             _ptr(out["dq_idx"]), _ptr(out["dk_idx"]), _ptr(out["kl"]), _ptr(ws),
                             nws, _stream(dev))
    _lib.check(rc, "msa_bwd_varlen")
    return out


# ---------------------------------------------------------------------------
# Decode: one new token per sequence against its KV cache (see include/msa.h).
# ---------------------------------------------------------------------------
def msa_decode(q, q_idx, k, v, k_idx, lens, topk: int = 16, *, scale=None, Bk: int = 128):
    """q [B,H_q,d], q_idx [B,H_kv,d_idx] (new token); k, v [B,Lmax,H_kv,d] and
    k_idx [B,Lmax,d_idx] (caches); lens int32 [B] on the device (cache lengths including
    the new token).  Returns (block_idx [B,H_kv,topk] int32, o [B,H_q,d] bf16,
    lse [B,H_q] f32)."""
    _need(q, "q", ndim=3)
    _need(q_idx, "q_idx", ndim=3)
    _need(k, "k", ndim=4)
    _need(v, "v", ndim=4)
    _need(k_idx, "k_idx", ndim=3)
    _need(lens, "lens", torch.int32, ndim=1)
    B, H_q, d = q.shape
    _, Lmax, H_kv, _ = k.shape
    d_idx = q_idx.shape[2]
    if tuple(v.shape) != tuple(k.shape) or tuple(k_idx.shape) != (B, Lmax, d_idx) or lens.numel() != B:
        raise ValueError("cache shapes must agree: k, v [B,Lmax,H_kv,d], k_idx [B,Lmax,d_idx], lens [B]")
    prob = make_problem(B, Lmax, H_q, H_kv, d, d_idx, topk, Bk, True, scale, None)
    dev = q.device
    block_idx = torch.empty((B, H_kv, topk), dtype=torch.int32, device=dev)
    o = torch.empty_like(q)
    lse = torch.empty((B, H_q), dtype=torch.float32, device=dev)
    nws = _lib.msa_decode_workspace_size(prob)
    ws = _workspace(nws, dev)
    rc = _lib.msa_decode(prob, _ptr(q), _ptr(q_idx), _ptr(k), _ptr(v), _ptr(k_idx), _ptr(lens),
                         _ptr(block_idx), _ptr(o), _ptr(lse), _ptr(ws), nws, _stream(dev))
    _lib.check(rc, "msa_decode")
    return block_idx, o, lse


def msa_quantize_kv_fp8(x, *, Bk: int = 128):
    """x [B,Lmax,H_kv,d] bf16 (a k or v cache) -> (codes [B,Lmax,H_kv,d] uint8 E4M3,
    scale [B,Lmax,H_kv] f32): one scale amax/448 per (sequence, token, head) row."""
    _need(x, "x", ndim=4)
    B, Lmax, H_kv, d = x.shape
    prob = make_problem(B, Lmax, H_kv, H_kv, d, 64, 1, Bk, True, None, None)
    x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty((B, Lmax, H_kv), dtype=torch.float32, device=x.device)
    rc = _lib.msa_quantize_kv_fp8(prob, _ptr(x), _ptr(x8), _ptr(scale), _stream(x.device))
    _lib.check(rc, "msa_quantize_kv_fp8")
    return x8, scale


def msa_decode_fp8(q, q_idx, k8, v8, k_scale, v_scale, k_idx, lens, topk: int = 16, *,
                   scale=None, Bk: int = 128):
    """msa_decode over an FP8 cache: k8, v8 [B,Lmax,H_kv,d] uint8 codes and k_scale,
    v_scale [B,Lmax,H_kv] f32 from msa_quantize_kv_fp8.  Returns (block_idx [B,H_kv,topk]
    int32, o [B,H_q,d] bf16, lse [B,H_q] f32)."""
    _need(q, "q", ndim=3)
    _need(q_idx, "q_idx", ndim=3)
    _need(k8, "k8", torch.uint8, ndim=4)
    _need(v8, "v8", torch.uint8, ndim=4)
    _need(k_scale, "k_scale", torch.float32, ndim=3)
    _need(v_scale, "v_scale", torch.float32, ndim=3)
    _need(k_idx, "k_idx", ndim=3)
    _need(lens, "lens", torch.int32, ndim=1)
    B, H_q, d = q.shape
    _, Lmax, H_kv, _ = k8.shape
    d_idx = q_idx.shape[2]
    if (tuple(v8.shape) != tuple(k8.shape) or tuple(k_scale.shape) != (B, Lmax, H_kv)
            or tuple(v_scale.shape) != (B, Lmax, H_kv) or tuple(k_idx.shape) != (B, Lmax, d_idx)
            or lens.numel() != B):
        raise ValueError("cache shapes must agree: k8, v8 [B,Lmax,H_kv,d], scales [B,Lmax,H_kv], "
                         "k_idx [B,Lmax,d_idx], lens [B]")
    prob = make_problem(B, Lmax, H_q, H_kv, d, d_idx, topk, Bk, True, scale, None)
    dev = q.device
    block_idx = torch.empty((B, H_kv, topk), dtype=torch.int32, device=dev)
    o = torch.empty_like(q)
    lse = torch.empty((B, H_q), dtype=torch.float32, device=dev)
    nws = _lib.msa_decode_workspace_size(prob)
    ws = _workspace(nws, dev)
    rc = _lib.msa_decode_fp8(prob, _ptr(q), _ptr(q_idx), _ptr(k8), _ptr(v8), _ptr(k_scale),
                             _ptr(v_scale), _ptr(k_idx), _ptr(lens), _ptr(block_idx), _ptr(o),
                             _ptr(lse), _ptr(ws), nws, _stream(dev))
    _lib.check(rc, "msa_decode_fp8")
    return block_idx, o, lse


# ---------------------------------------------------------------------------
# FP8 (E4M3) main-branch forward for training (d = 128); see include/msa.h.
# ---------------------------------------------------------------------------
def msa_quantize_fwd_fp8(q, k, v, *, Bk: int = 128):
    """bf16 q [B,N,H_q,d], k, v [B,N,H_kv,d] -> the FP8 forward's operands:
    q8 [B,N,H_q,d] uint8 + q_scale [B,N,H_q] (one scale per row), k8 [B,N,H_kv,d] +
    k_scale [B,H_kv,nb] and v8t [B,H_kv,nb,d,Bk] (v transposed per block) + v_scale
    [B,H_kv,nb] (one scale per Bk-key block)."""
    _need(q, "q", ndim=4)
    _need(k, "k", ndim=4)
    _need(v, "v", ndim=4)
    B, N, H_q, d = q.shape
    H_kv = k.shape[2]
    if tuple(k.shape) != (B, N, H_kv, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k, v must be [B, N, H_kv, d] with q's B, N, d")
    nb = (N + Bk - 1) // Bk
    prob = make_problem(B, N, H_q, H_kv, d, 64, 1, Bk, True, None, None)
    dev = q.device
    q8 = torch.empty(q.shape, dtype=torch.uint8, device=dev)
    q_scale = torch.empty((B, N, H_q), dtype=torch.float32, device=dev)
    k8 = torch.empty(k.shape, dtype=torch.uint8, device=dev)
    k_scale = torch.empty((B, H_kv, nb), dtype=torch.float32, device=dev)
    v8t = torch.empty((B, H_kv, nb, d, Bk), dtype=torch.uint8, device=dev)
    v_scale = torch.empty((B, H_kv, nb), dtype=torch.float32, device=dev)
    rc = _lib.msa_quantize_fwd_fp8(prob, _ptr(q), _ptr(k), _ptr(v), _ptr(q8), _ptr(q_scale),
                                   _ptr(k8), _ptr(k_scale), _ptr(v8t), _ptr(v_scale), _stream(dev))
    _lib.check(rc, "msa_quantize_fwd_fp8")
    return q8, q_scale, k8, k_scale, v8t, v_scale


def msa_fwd_fp8(q8, q_scale, k8, k_scale, v8t, v_scale, block_idx, *, scale=None, Bk: int = 128,
                d_idx: int = 64):
    """FP8 forward over the operands of msa_quantize_fwd_fp8 and the block sets
    block_idx [B,H_kv,N,topk]: returns (o [B,N,H_q,d] bf16, lse [B,H_q,N] f32)."""
    _need(q8, "q8", torch.uint8, ndim=4)
    _need(k8, "k8", torch.uint8, ndim=4)
    _need(v8t, "v8t", torch.uint8, ndim=5)
    _need(q_scale, "q_scale", torch.float32, ndim=3)
    _need(k_scale, "k_scale", torch.float32, ndim=3)
    _need(v_scale, "v_scale", torch.float32, ndim=3)
    _need(block_idx, "block_idx", torch.int32, ndim=4)
    B, N, H_q, d = q8.shape
    H_kv = k8.shape[2]
    topk = block_idx.shape[3]
    nb = (N + Bk - 1) // Bk
    if (tuple(k8.shape) != (B, N, H_kv, d) or tuple(v8t.shape) != (B, H_kv, nb, d, Bk)
            or tuple(q_scale.shape) != (B, N, H_q) or tuple(k_scale.shape) != (B, H_kv, nb)
            or tuple(v_scale.shape) != (B, H_kv, nb) or tuple(block_idx.shape[:3]) != (B, H_kv, N)):
        raise ValueError("operand shapes must be those of msa_quantize_fwd_fp8")
    prob = make_problem(B, N, H_q, H_kv, d, d_idx, topk, Bk, True, scale, None)
    dev = q8.device
    o = torch.empty((B, N, H_q, d), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((B, H_q, N), dtype=torch.float32, device=dev)
    nws = _lib.msa_workspace_size(prob, _lib.MSA_WS_FWD)
    ws = _workspace(nws, dev)
    rc = _lib.msa_fwd_fp8(prob, _ptr(q8), _ptr(q_scale), _ptr(k8), _ptr(k_scale), _ptr(v8t),
                          _ptr(v_scale), _ptr(block_idx), _ptr(o), _ptr(lse), _ptr(ws), nws,
                          _stream(dev))
    _lib.check(rc, "msa_fwd_fp8")
    return o, lse


# ---------------------------------------------------------------------------
# Rotary positions (see include/msa.h).
# ---------------------------------------------------------------------------
_ROPE_DTYPES = {torch.bfloat16: _lib.MSA_DTYPE_BF16, torch.float16: _lib.MSA_DTYPE_F16,
                torch.float32: _lib.MSA_DTYPE_F32}
_TWO_PI_E49 = 2 * 31415926535897932384626433832795028841971693993751  # 2 pi 10^49


_Tensor, _BF16, _I32 = torch.Tensor, torch.bfloat16, torch.int32


def _call(index, name, f, *args):
    """f(*args, stream) on the current stream of device `index`, with that device current;
    raises on an error."""
    if index == torch.cuda.current_device():
        rc = f(*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _stream_of(index))
    if rc:
        _lib.check(rc, name)


@dataclasses.dataclass(frozen=True, eq=False)
class Rope:
    """Rotary frequencies on a device (from new_rope)."""
    turns: torch.Tensor  # int64 [rot_dim / 2]: turns a position, in units of 2^-64
    rot_dim: int
    interleaved: bool
    mscale: float


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling=None):
    """Radians a position of the rot_dim / 2 pairs (list of float) and the factor mscale on the
    rotated values.  scaling, to reach past the trained context:
      None                               f_i = base^(-2i / rot_dim)
      {"type": "linear", "factor": s}    f_i / s
      {"type": "ntk", "factor": s}       base s^(rot_dim / (rot_dim - 2)) in place of base
      {"type": "yarn", "factor": s, "original_len": L, "beta_fast": 32, "beta_slow": 1}
          pairs that turn beta_fast times or more over L keep f_i, those that turn beta_slow
          times or fewer take f_i / s, the ones between a linear mix by their turns;
          mscale = 0.1 ln s + 1 (or "mscale") -- YaRN, Peng et al. 2023.  The mix is linear in
          the turns, as the paper has it; a model made with one that is linear in the pair's
          index i has to give its frequencies to new_rope as inv_freq."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not (math.isfinite(base) and base > 0):
        raise ValueError(f"base must be positive, got {base}")
    half = rot_dim // 2
    if scaling is None:
        return [base ** (-2.0 * i / rot_dim) for i in range(half)], 1.0
    known = {"linear": {"factor"}, "ntk": {"factor"},
             "yarn": {"factor", "original_len", "beta_fast", "beta_slow", "mscale"}}
    kind = scaling.get("type")
    if kind not in known:
        raise ValueError(f"unknown scaling type {kind!r}: one of {sorted(known)}")
    extra = set(scaling) - known[kind] - {"type"}
    if extra or "factor" not in scaling:
        raise ValueError(f"scaling {kind!r} takes {sorted(known[kind])}, got {sorted(scaling)}")
    s = float(scaling["factor"])
    if not (math.isfinite(s) and s > 0):
        raise ValueError(f"factor must be positive, got {s}")
    if kind == "ntk":
        if rot_dim == 2:
            raise ValueError("ntk scaling needs rot_dim > 2")
        base *= s ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    if kind == "ntk":
        return f, 1.0
    if kind == "linear":
        return [x / s for x in f], 1.0
    if "original_len" not in scaling:
        raise ValueError("scaling 'yarn' needs original_len")
    L = float(scaling["original_len"])
    fast, slow = float(scaling.get("beta_fast", 32.0)), float(scaling.get("beta_slow", 1.0))
    if not (L > 0 and fast > slow >= 0):
        raise ValueError("yarn needs original_len > 0 and beta_fast > beta_slow >= 0")
    keep = [min(1.0, max(0.0, (L * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
    return ([x * g + x / s * (1.0 - g) for x, g in zip(f, keep)],
            float(scaling.get("mscale", 0.1 * math.log(s) + 1.0)))


def new_rope(rot_dim: int, *, base: float = 10000.0, interleaved: bool = False, scaling=None,
             inv_freq=None, mscale=None, device="cuda") -> Rope:
    """Rotary positions over the first rot_dim values of a head: pairs (i, i + rot_dim / 2), or
    (2i, 2i + 1) with interleaved.  Frequencies from base and scaling (rope_frequencies), or
    given as inv_freq (rot_dim / 2 radians a position); mscale overrides the factor on the
    rotated values.  One handle serves every layer and position."""
    if inv_freq is None:
        freq, m = rope_frequencies(rot_dim, base, scaling)
    else:
        if scaling is not None:
            raise ValueError("inv_freq and scaling exclude one another")
        if rot_dim < 2 or rot_dim % 2:
            raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
        freq, m = [float(x) for x in inv_freq], 1.0
        if len(freq) != rot_dim // 2 or not all(map(math.isfinite, freq)):
            raise ValueError(f"inv_freq must be {rot_dim // 2} finite numbers")
    if rot_dim > 512:
        raise ValueError(f"rot_dim is at most 512, got {rot_dim}")
    m = float(m if mscale is None else mscale)
    if not math.isfinite(m):
        raise ValueError("mscale must be finite")
    turns = []
    for x in freq:  # x / (2 pi) in units of 2^-64, rounded to the nearest, modulo 1
        num, den = x.as_integer_ratio()
        den *= _TWO_PI_E49
        t = ((num * 10 ** 49 << 65) + den) // (2 * den) % (1 << 64)
        turns.append(t - (1 << 64) if t >> 63 else t)
    turns = torch.tensor(turns, dtype=torch.int64)
    return Rope(turns.to(device), rot_dim, bool(interleaved), m)


def msa_rope(xs, rope: Rope, positions=None, *, inverse: bool = False, inplace: bool = False):
    """Rotary positions of one to four tensors in one launch; returns them as a tuple (new
    contiguous tensors, or xs themselves with inplace).  inverse turns back (the gradient).
    Autograd does not see this call: rope is the differentiable one.

    positions None: tokens [B, N, H, d] or [B, N, d] (one head), each at its index in its
    sequence.  positions int32 or int64 [T]: packed tokens [T, H, d] or [T, d];  [B, N] (a
    broadcast row is fine): tokens [B, N, H, d] or [B, N, d].  bf16, fp16 or float32 (all the
    same), d >= rot_dim; any strides (views of a fused projection), the last axis contiguous
    or else copied once.  In place the tensors must not overlap."""
    xs = (xs,) if isinstance(xs, _Tensor) else tuple(xs)
    if not 1 <= len(xs) <= 4:
        raise ValueError(f"one to four tensors, got {len(xs)}")
    if not isinstance(rope, Rope):
        raise TypeError("rope must come from new_rope")
    for x in xs:
        if not isinstance(x, _Tensor):
            raise TypeError("every operand must be a tensor")
    turns, rot = rope.turns, rope.rot_dim
    index, dtype = turns.get_device(), xs[0].dtype
    code = _ROPE_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"tensors must be bf16, fp16 or float32, got {dtype}")
    bits, at, ps = 32, None, (0, 0)
    if positions is None:
        if xs[0].dim() < 3:
            raise ValueError("without positions the tensors are [B, N, H, d] or [B, N, d]")
        lead = xs[0].shape[:2]
    else:
        if not isinstance(positions, _Tensor) or positions.dtype not in (_I32, torch.int64):
            raise TypeError("positions must be an int32 or int64 tensor")
        lead, ps, at = positions.shape, positions.stride(), positions.data_ptr()
        if len(lead) == 1:
            ps = (0, ps[0])
        elif len(lead) != 2:
            raise ValueError(f"positions must be [T] or [B, N], got {tuple(lead)}")
        if positions.dtype != _I32:
            bits = 64
    if index < 0 or (positions is not None and positions.get_device() != index):
        raise ValueError("rope, positions and the tensors must be on one CUDA device (no CPU path exists)")
    n = len(lead)
    B, N = lead if n == 2 else (1, lead[0])
    if inplace:
        _check_in_place(xs)
    # A decode step's time is the host's: each attribute is looked up once.
    ys, packed, keep = [], [], []
    pack, empty, dev = _lib.ROPE_TENSOR.pack, torch.empty, turns.device
    for x in xs:
        shape, sx = x.shape, x.stride()
        more = len(shape) - n
        if shape[:n] != lead or not 1 <= more <= 2:
            raise ValueError(f"every tensor must be {tuple(lead)} + ([H,] d), got {tuple(shape)}")
        if x.dtype != dtype:
            raise TypeError(f"all tensors must be {dtype}, got {x.dtype}")
        if x.get_device() != index:
            raise ValueError("rope, positions and the tensors must be on one CUDA device (no CPU path exists)")
        d = shape[-1]
        if d < rot:
            raise ValueError(f"d = {d} < rot_dim = {rot}")
        H, h = (shape[n], sx[n]) if more == 2 else (1, 0)
        if inplace:
            ys.append(x)
            if B and N and H:
                b, t, p = sx[0] if n == 2 else 0, sx[n - 1], x.data_ptr()
                packed.append(pack(p, p, b, t, h, b, t, h, H, d))
            continue
        if sx[-1] != 1:
            x = x.contiguous()
            keep.append(x)
            sx = x.stride()
            h = sx[n] if more == 2 else 0
        y = empty(shape, dtype=dtype, device=dev)
        ys.append(y)
        if B and N and H:  # strides of batch, token and head; y is contiguous
            packed.append(pack(x.data_ptr(), y.data_ptr(), sx[0] if n == 2 else 0, sx[n - 1], h, N * H * d, H * d, d,
                               H, d))
    if packed:
        r = _lib.ROPE.pack(B, N, rot, rope.interleaved, inverse, code, bits, rope.mscale, *ps)
        _call(index, "msa_rope", _lib.msa_rope, r, turns.data_ptr(), at, b"".join(packed), len(packed))
    return tuple(ys)


def _check_in_place(xs):
    if len({x.data_ptr() for x in xs if x.numel()}) != sum(x.numel() > 0 for x in xs):
        raise ValueError("the same memory is given twice: it would be turned twice")
    for x in xs:
        if any(s == 0 and k > 1 for s, k in zip(x.stride(), x.shape)) or x.stride(-1) != 1:
            raise ValueError("a tensor whose values overlap, or whose last axis is strided, cannot be "
                             "turned in place")
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("a tensor that requires a gradient cannot be turned in place: use rope")
        if _forward_mode() and forward_ad.unpack_dual(x).tangent is not None:
            raise ValueError("a tensor with a tangent cannot be turned in place: use rope")
    for x in xs:
        torch.autograd.graph.increment_version(x)


def _forward_mode() -> bool:
    """Within a level of torch.autograd.forward_ad: tensors may carry tangents, which only an
    autograd function sees."""
    return forward_ad._current_level >= 0


class RopeFunction(torch.autograd.Function):
    """msa_rope with its derivatives: the tangent's turn, and for the gradient the inverse turn
    (linear in x: differentiable again)."""

    @staticmethod
    def forward(ctx, rope, positions, inverse, *xs):
        ctx.rope, ctx.inverse = rope, inverse
        ctx.save_for_backward(positions)
        ctx.save_for_forward(positions)
        ctx.set_materialize_grads(False)
        ctx.like = [(x.shape, x.dtype, x.device) for x in xs] if _forward_mode() else None
        return msa_rope(xs, rope, positions, inverse=inverse)

    @staticmethod
    def jvp(ctx, _rope, _positions, _inverse, *ts):
        (positions,) = ctx.saved_tensors
        got = [i for i, t in enumerate(ts) if t is not None]
        out = [None if t is not None else torch.zeros(s, dtype=dt, device=dev) for t, (s, dt, dev) in zip(ts, ctx.like)]
        for i, y in zip(got, msa_rope([ts[i] for i in got], ctx.rope, positions, inverse=ctx.inverse)):
            out[i] = y
        return tuple(out)

    @staticmethod
    def backward(ctx, *dys):
        (positions,) = ctx.saved_tensors
        got = [i for i, g in enumerate(dys) if g is not None and ctx.needs_input_grad[3 + i]]
        out = [None] * len(dys)
        if got:
            turn = [dys[i] for i in got]
            if torch.is_grad_enabled() or _forward_mode():  # a second derivative may be wanted
                dxs = RopeFunction.apply(ctx.rope, positions, not ctx.inverse, *turn)
            else:
                dxs = msa_rope(turn, ctx.rope, positions, inverse=not ctx.inverse)
            for i, g in zip(got, dxs):
                out[i] = g
        return (None, None, None, *out)


def rope(xs, rope: Rope, positions=None):
    """msa_rope for training: the rotated tensors as a tuple, differentiable in xs (in reverse
    and in forward mode)."""
    xs = (xs,) if isinstance(xs, torch.Tensor) else tuple(xs)
    if _forward_mode() or (torch.is_grad_enabled() and
                           any(isinstance(x, torch.Tensor) and x.requires_grad for x in xs)):
        return RopeFunction.apply(rope, positions, False, *xs)
    return msa_rope(xs, rope, positions)


_rotated = rope  # for attention, whose argument is named rope too


# ---------------------------------------------------------------------------
# Paged cache (see include/msa.h).
# ---------------------------------------------------------------------------
class PagedCache:
    """A pool of pages: k, v [num_pages, page_size, H_kv, d] bf16, or uint8 E4M3 codes with
    k_scale, v_scale [num_pages, page_size, H_kv] float32; k_idx [num_pages, page_size, d_idx]
    bf16, or None for a cache without index keys.  Page tables (int32 [B, max_pages]) and
    lengths (int32 [B]) belong to the calls.  The tensors of a cache are fixed."""

    def __init__(self, k, v, k_idx=None, k_scale=None, v_scale=None):
        fp8 = isinstance(k, torch.Tensor) and k.dtype == torch.uint8
        kind = torch.uint8 if fp8 else torch.bfloat16
        _need(k, "k", kind, ndim=4)
        _need(v, "v", kind, ndim=4)
        P, page, H_kv, d = k.shape
        if v.shape != k.shape:
            raise ValueError(f"v must be {tuple(k.shape)}, got {tuple(v.shape)}")
        if (k_scale is not None or v_scale is not None) != fp8 or (k_scale is None) != (v_scale is None):
            raise ValueError("E4M3 codes (uint8) have k_scale and v_scale; bf16 pages have none")
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _need(t, n, torch.float32, ndim=3)
                if tuple(t.shape) != (P, page, H_kv):
                    raise ValueError(f"{n} must be {(P, page, H_kv)}, got {tuple(t.shape)}")
        d_idx = 0
        if k_idx is not None:
            _need(k_idx, "k_idx", ndim=3)
            d_idx = k_idx.shape[2]
            if tuple(k_idx.shape[:2]) != (P, page):
                raise ValueError(f"k_idx must be {(P, page)} + (d_idx,), got {tuple(k_idx.shape)}")
        if any(t is not None and t.device != k.device for t in (v, k_idx, k_scale, v_scale)):
            raise ValueError("the pages of a cache must be on one device")
        if page < 16 or page % 16:
            raise ValueError(f"page_size must be a multiple of 16, got {page}")
        if d not in (64, 128) or d_idx not in (0, 32, 64):
            raise ValueError(f"d must be 64 or 128 and d_idx 32 or 64, got {d} and {d_idx}")
        if H_kv < 1:
            raise ValueError("a cache has at least one KV head")
        self.k, self.v, self.k_idx, self.k_scale, self.v_scale = k, v, k_idx, k_scale, v_scale
        self._pools = tuple(t for t in (k, v, k_idx, k_scale, v_scale) if t is not None)
        self.num_pages, self.page_size, self.H_kv, self.d, self.d_idx, self.fp8 = P, page, H_kv, d, d_idx, fp8
        self.device, self.index = k.device, k.get_device()
        self._c = _lib.PAGED_CACHE.pack(
            P, page, H_kv, d, d_idx, _lib.MSA_CACHE_E4M3 if fp8 else _lib.MSA_CACHE_BF16,
            *(0 if t is None else t.data_ptr() for t in (k, v, k_idx, k_scale, v_scale)))

    def __setattr__(self, name, value):
        if "_c" in self.__dict__:
            raise AttributeError("the tensors of a PagedCache are fixed: make another one")
        object.__setattr__(self, name, value)

    def __reduce__(self):  # a copy has its own tensors
        return PagedCache, (self.k, self.v, self.k_idx, self.k_scale, self.v_scale)


def new_paged_cache(num_pages: int, H_kv: int, *, page_size: int = 128, d: int = 128, d_idx: int = 64,
                    fp8: bool = False, device="cuda") -> PagedCache:
    """An empty PagedCache (d_idx 0: without index keys)."""
    def pages(*tail, dtype):
        return torch.zeros((num_pages, page_size, *tail), dtype=dtype, device=device)

    kv = torch.uint8 if fp8 else torch.bfloat16
    return PagedCache(pages(H_kv, d, dtype=kv), pages(H_kv, d, dtype=kv),
                      pages(d_idx, dtype=torch.bfloat16) if d_idx else None,
                      pages(H_kv, dtype=torch.float32) if fp8 else None,
                      pages(H_kv, dtype=torch.float32) if fp8 else None)


def _pages_arg(cache, page_table, lens):
    """The packed page table, after the checks that a paged call's arguments share, and its B."""
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    for t, n in ((page_table, "page_table"), (lens, "lens")):
        if not isinstance(t, _Tensor) or t.dtype != _I32:
            raise TypeError(f"{n} must be an int32 tensor")
        if t.get_device() != cache.index:
            raise ValueError(f"{n} must be on the cache's device")
    shape, strides, L = page_table.shape, page_table.stride(), lens.shape
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError("page_table must have 2 dims, the last contiguous")
    B = shape[0]
    if len(L) != 1 or L[0] != B or (B > 1 and lens.stride(0) != 1):
        raise ValueError(f"lens must be a contiguous [{B}], got {tuple(L)}")
    return _lib.PAGE_TABLE.pack(page_table.data_ptr(), B, shape[1], strides[0]), B


def _cu_arg(cu_seqlens, cache, B):
    if not isinstance(cu_seqlens, _Tensor) or cu_seqlens.dtype != _I32:
        raise TypeError("cu_seqlens must be an int32 tensor")
    if cu_seqlens.get_device() != cache.index or cu_seqlens.shape != (B + 1,) or not cu_seqlens.is_contiguous():
        raise ValueError(f"cu_seqlens must be a contiguous [{B + 1}] on the cache's device")
    return cu_seqlens.data_ptr()


def _cache_rows(t, name, cache, shape):
    """A packed input of msa_cache_write (copied where its rows do not start on 16 bytes), its
    address and strides."""
    if not isinstance(t, _Tensor) or t.dtype != _BF16:
        raise TypeError(f"{name} must be a bf16 tensor")
    if t.get_device() != cache.index:
        raise ValueError(f"{name} must be on the cache's device (no CPU path exists)")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    p, s = t.data_ptr(), t.stride()
    if s[-1] != 1 or p % 16 or s[0] % 8 or s[-2] % 8:
        t = t.clone(memory_format=torch.contiguous_format)
        p, s = t.data_ptr(), t.stride()
    return t, p, s


def msa_cache_write(cache: PagedCache, page_table, lens, k, v, k_idx=None, *, cu_seqlens=None) -> None:
    """Writes new tokens into the cache's pages, as E4M3 codes and row scales where it holds
    those: k, v [T, H_kv, d], k_idx [T, d_idx] (given exactly if the cache has index keys), bf16,
    any strides.  lens (int32 [B]): lengths after the call; sequence b's n new tokens go to
    positions lens[b] - n .. lens[b] - 1.  cu_seqlens (int32 [B + 1]) splits the T packed tokens;
    without it there is one token a sequence (T = B), and lens[b] = 0 skips the slot.  A token
    whose place does not exist is dropped and sets the device status."""
    pages, B = _pages_arg(cache, page_table, lens)
    T = k.shape[0] if isinstance(k, _Tensor) and k.dim() == 3 else 0
    k, pk, sk = _cache_rows(k, "k", cache, (T, cache.H_kv, cache.d))
    v, pv, sv = _cache_rows(v, "v", cache, (T, cache.H_kv, cache.d))
    if (k_idx is None) != (cache.k_idx is None):
        raise ValueError("k_idx must be given exactly if the cache has index keys")
    pi, si = None, (0,)
    if k_idx is not None:
        k_idx, pi, si = _cache_rows(k_idx, "k_idx", cache, (T, cache.d_idx))
    cu = None
    if cu_seqlens is not None:
        cu = _cu_arg(cu_seqlens, cache, B)
    elif T != B:
        raise ValueError(f"without cu_seqlens there is one token a sequence: {B}, got {T}")
    if T == 0 or B == 0:
        return
    _call(cache.index, "msa_cache_write", _lib.msa_cache_write, cache._c, pages, lens.data_ptr(), cu, T, pk, pv, pi,
          _lib.CACHE_STRIDES.pack(sk[0], sk[1], sv[0], sv[1], si[0]))
    torch.autograd.graph.increment_version(cache._pools)  # a graph that saved one of them must notice


def msa_cache_read(cache: PagedCache, page_table, lens, cu_seqlens, total_tokens: int):
    """The last cu_seqlens[b + 1] - cu_seqlens[b] tokens of every sequence (up to position
    lens[b] - 1) in packed order: k, v [total_tokens, H_kv, d] and k_idx [total_tokens, d_idx]
    (None without index keys), bf16.  With lens[b] tokens of each it is the whole context, as
    msa_fwd_varlen and its companions take it.  Rows behind cu_seqlens[B] are not written."""
    pages, B = _pages_arg(cache, page_table, lens)
    _cu_arg(cu_seqlens, cache, B)
    T = int(total_tokens)
    if T < 0:
        raise ValueError("total_tokens must not be negative")
    dev = cache.device
    k = torch.empty((T, cache.H_kv, cache.d), dtype=torch.bfloat16, device=dev)
    v = torch.empty((T, cache.H_kv, cache.d), dtype=torch.bfloat16, device=dev)
    k_idx = None
    if cache.k_idx is not None:
        k_idx = torch.empty((T, cache.d_idx), dtype=torch.bfloat16, device=dev)
    if T and B:
        _call(cache.index, "msa_cache_read", _lib.msa_cache_read, cache._c, pages, lens.data_ptr(),
              cu_seqlens.data_ptr(), T, k.data_ptr(), v.data_ptr(), _ptr(k_idx))
    return k, v, k_idx


# ---------------------------------------------------------------------------
# Decode over a paged cache (see include/msa.h).  The workspace is allocated on the calling
# stream: calls on other streams and other captured graphs never share it.
# ---------------------------------------------------------------------------
def _paged_args(q, cache, page_table, lens, topk, scale):
    pages, B = _pages_arg(cache, page_table, lens)
    _need(q, "q", ndim=3)
    shape, H_kv, d = q.shape, cache.H_kv, cache.d
    H_q = shape[1]
    if shape[0] != B or shape[2] != d or H_q == 0 or H_q % H_kv or q.get_device() != cache.index:
        raise ValueError(f"q must be [{B}, a multiple of {H_kv}, {d}] on the cache's device, got {tuple(shape)}")
    if H_q // H_kv > 16:
        raise ValueError(f"at most 16 query heads a group, got {H_q // H_kv}")
    nws = _lib.msa_decode_paged_workspace_size(cache._c, pages, H_q, topk)  # 0: needs none, or the call refuses
    dev = cache.device
    return (pages, B, H_q, d ** -0.5 if scale is None else float(scale), torch.empty_like(q),
            torch.empty((B, H_q), dtype=torch.float32, device=dev),
            torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None, nws)


def msa_decode_paged(q, q_idx, cache: PagedCache, page_table, lens, topk: int = 16, *, scale=None):
    """msa_decode over pages: q [B,H_q,d], q_idx [B,H_kv,d_idx] (new token); page_table int32
    [B,max_pages], lens int32 [B] (lengths including the new token; 0: an empty slot).
    Returns (block_idx [B,H_kv,topk] int32, o [B,H_q,d] bf16, lse [B,H_q] f32)."""
    if not 1 <= topk <= 32:
        raise ValueError(f"topk must be 1 .. 32, got {topk}")
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    if cache.k_idx is None:
        raise ValueError("the cache has no index keys")
    pages, B, H_q, scale, o, lse, ws, nws = _paged_args(q, cache, page_table, lens, topk, scale)
    _need(q_idx, "q_idx", ndim=3)
    if q_idx.shape != (B, cache.H_kv, cache.d_idx) or q_idx.get_device() != cache.index:
        raise ValueError(f"q_idx must be {(B, cache.H_kv, cache.d_idx)} on the cache's device, "
                         f"got {tuple(q_idx.shape)}")
    block_idx = torch.empty((B, cache.H_kv, topk), dtype=_I32, device=cache.device)
    if B:
        _call(cache.index, "msa_decode_paged", _lib.msa_decode_paged, cache._c, pages, lens.data_ptr(), H_q, topk,
              scale, q.data_ptr(), q_idx.data_ptr(), block_idx.data_ptr(), o.data_ptr(), lse.data_ptr(),
              ws.data_ptr() if nws else None, nws)
    return block_idx, o, lse


def msa_decode_paged_dense(q, cache: PagedCache, page_table, lens, *, scale=None):
    """Attention of one new token a sequence over its whole paged cache: arguments as in
    msa_decode_paged.  Returns (o [B,H_q,d] bf16, lse [B,H_q] f32)."""
    pages, B, H_q, scale, o, lse, ws, nws = _paged_args(q, cache, page_table, lens, 0, scale)
    if B:
        _call(cache.index, "msa_decode_paged_dense", _lib.msa_decode_paged_dense, cache._c, pages, lens.data_ptr(),
              H_q, scale, q.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr() if nws else None, nws)
    return o, lse
