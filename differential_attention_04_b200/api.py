"""Python binding of the C ABI in include/diffattn.h.

Argument marshalling only: every step of the computation runs in the CUDA
library.  Tensors are passed by device pointer on the current torch stream;
the functions return immediately (stream-ordered), like the C calls.

The calls that a server makes every step are first offered to the compiled
marshalling module (csrc/marshal.cpp): it makes the call when everything is
plainly right, and otherwise the checks below say what is wrong.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._lib import lib, marshal

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE, ERR_BOUNDS = range(7)
F32, BF16 = 0, 1
# how the two maps are combined: softmax(S1) + c softmax(S2), c = -lambda, 0, +lambda
MODE_DIFF, MODE_LAMBDA_ZERO, MODE_SUM = 0, 1, 2
# which channels a rotation pairs: (2j, 2j + 1) or (j, j + rot / 2)
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
# added to either: rows that are not rotated are written as zeros instead of being left
ROPE_PAD_ZERO = 256
# how a rotary table's frequencies are scaled
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3


class DiffAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().diffattn_status_string(status).decode()
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise DiffAttnError(fn, status)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(*ts: torch.Tensor) -> torch.device:
    """The one CUDA device all of `ts` live on (every tensor contiguous)."""
    dev = ts[0].device
    for t in ts:
        if t.device != dev or not t.is_contiguous():
            break
    else:
        if dev.type == "cuda":
            return dev
    # something is wrong with them: the first fault, tensor by tensor
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if t.device != dev:
            raise ValueError(f"all tensors must be on one device (found {dev} and {t.device})")


def _getters(c):
    """(current device's index, raw current stream of a device): torch's own raw getters where it has them (a Stream
    object and a device context cost more host time than the call itself), else its public ones."""
    return (getattr(c, "_cuda_getDevice", torch.cuda.current_device),
            getattr(c, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream))


_current_device, _raw_stream = _getters(torch._C)


def _launch(name: str, tensors, *args) -> None:
    """Call the C entry point `name` with `args` and the current stream of the
    device that `tensors` (every tensor the call reads or writes) live on, with
    that device current: the library launches on the current device."""
    dev = _dev(*tensors)
    fn = getattr(lib(), name)
    if _current_device() == dev.index:
        status = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev.index))
    if status != OK:
        raise DiffAttnError(name, status)


def _made(name: str, status: int) -> bool:
    """Whether the marshalling module made the call (its status: negative if it was left to the checks here)."""
    if status > 0:
        raise DiffAttnError(name, status)
    return status == 0


# Shape and dtype checks run before the device check, so that every tensor the
# kernels index is known to be large enough before its pointer is passed on.
def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _scalar_f32(name: str, t: torch.Tensor) -> None:
    _need(t.dtype == torch.float32 and t.numel() >= 1, f"{name} must be a float32 device scalar")


def _f32(name: str, t: torch.Tensor, n: int) -> None:
    _need(t.dtype == torch.float32 and t.numel() == n, f"{name} must be float32 with {n} elements")


def _like(name: str, t: torch.Tensor, shape, dtype) -> None:
    _need(tuple(t.shape) == tuple(shape) and t.dtype == dtype, f"{name} must be {dtype} of shape {tuple(shape)}")


def _qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dy: torch.Tensor | None = None):
    """(B, N, H, d) of q, k [B, N, H, 2, d] and v (and dy) [B, N, H, 2d]."""
    _need(q.dim() == 5 and q.shape[3] == 2 and k.shape == q.shape,
          "q and k must be [B, N, H, 2, d] of one shape")
    B, N, H, _, d = q.shape
    _need(tuple(v.shape) == (B, N, H, 2 * d), "v must be [B, N, H, 2d]")
    _need(dy is None or dy.shape == v.shape, "dy must have v's shape")
    return B, N, H, d


def diffattn_lambda(lq1: torch.Tensor, lk1: torch.Tensor, lq2: torch.Tensor, lk2: torch.Tensor,
                    lambda_init: float, out: torch.Tensor | None = None) -> torch.Tensor:
    """lambda = exp(lq1 . lk1) - exp(lq2 . lk2) + lambda_init, as a device fp32 scalar (shape [1])."""
    for name, t in (("lq1", lq1), ("lk1", lk1), ("lq2", lq2), ("lk2", lk2)):
        _f32(name, t, lq1.numel())
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=lq1.device)
    _scalar_f32("out", out)
    _launch("diffattn_lambda", (lq1, lk1, lq2, lk2, out),
            _ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), lq1.numel(), float(lambda_init), _ptr(out))
    return out


def diffattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, lambda_init: float,
                 rms_w: torch.Tensor, eps: float = 1e-5, causal: bool = True,
                 out: torch.Tensor | None = None, mode: int = MODE_DIFF) -> torch.Tensor:
    """Prefill.  q, k: [B, N, H, 2, d]; v: [B, N, H, 2d]; lam: device fp32 scalar; rms_w: fp32 [2d].

    ``mode`` (MODE_DIFF, MODE_LAMBDA_ZERO, MODE_SUM) picks the combination of
    the two maps; MODE_DIFF is the differential attention itself."""
    B, N, H, d = _qkv(q, k, v)
    if q.dtype == torch.bfloat16:
        dt = BF16
    elif q.dtype == torch.float32:
        dt = F32
    else:
        raise ValueError("dtype must be bfloat16 or float32")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype")
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    if out is None:
        out = torch.empty_like(v)
    _like("out", out, v.shape, v.dtype)
    ts = (q, k, v, lam, rms_w, out)
    if mode == MODE_DIFF:
        _launch("diffattn_fwd", ts, _ptr(q), _ptr(k), _ptr(v), _ptr(out), dt, B, N, H, d, int(bool(causal)),
                _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps))
    else:
        _launch("diffattn_fwd_mode", ts, _ptr(q), _ptr(k), _ptr(v), _ptr(out), dt, B, N, H, d, int(bool(causal)),
                _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps), int(mode))
    return out


def quantize_qk(x: torch.Tensor, codes: torch.Tensor | None = None,
                scales: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """e4m3 codes (uint8, x's shape) and float32 scales [B, H, 2] of a bf16 q or k [B, N, H, 2, d]:
    one absmax scale per (batch, head, map)."""
    if x.dtype != torch.bfloat16 or x.dim() != 5 or x.shape[3] != 2:
        raise ValueError("x must be bfloat16 [B, N, H, 2, d]")
    B, N, H, _, d = x.shape
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((B, H, 2), dtype=torch.float32, device=x.device)
    if codes.shape != x.shape or codes.dtype != torch.uint8 or scales.numel() != B * H * 2 or \
            scales.dtype != torch.float32:
        raise ValueError("codes must be uint8 like x and scales float32 [B, H, 2]")
    _launch("diffattn_quantize_qk", (x, codes, scales),
            _ptr(x), B, N, H, d, _ptr(codes), _ptr(scales))
    return codes, scales


def _lowbit_rest(B, N, H, d, q_scales, k_scales, v, lam, rms_w) -> None:
    _f32("q_scales", q_scales, B * H * 2)
    _f32("k_scales", k_scales, B * H * 2)
    _like("v", v, (B, N, H, 2 * d), torch.bfloat16)
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)


def diffattn_fwd_qk8(q_codes: torch.Tensor, q_scales: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor,
                     v: torch.Tensor, lam: torch.Tensor, lambda_init: float, rms_w: torch.Tensor, eps: float = 1e-5,
                     causal: bool = True, out: torch.Tensor | None = None, mode: int = MODE_DIFF) -> torch.Tensor:
    """Prefill with e4m3 queries and keys (as quantize_qk returns them); v, out: bf16 [B, N, H, 2d]."""
    if q_codes.dtype != torch.uint8 or k_codes.dtype != torch.uint8 or k_codes.shape != q_codes.shape or \
            q_codes.dim() != 5 or q_codes.shape[3] != 2:
        raise ValueError("q_codes, k_codes must be uint8 [B, N, H, 2, d]")
    B, N, H, _, d = q_codes.shape
    _lowbit_rest(B, N, H, d, q_scales, k_scales, v, lam, rms_w)
    if out is None:
        out = torch.empty_like(v)
    _like("out", out, v.shape, torch.bfloat16)
    _launch("diffattn_fwd_qk8", (q_codes, q_scales, k_codes, k_scales, v, lam, rms_w, out),
            _ptr(q_codes), _ptr(q_scales), _ptr(k_codes), _ptr(k_scales), _ptr(v), _ptr(out), B, N, H, d,
            int(bool(causal)), _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps), int(mode))
    return out


def quantize_qk4(x: torch.Tensor, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """e2m1 codes, two per byte (uint8 [B, N, H, 2, d / 2], channel 2j in the low nibble), and float32
    scales [B, H, 2] of a bf16 q or k [B, N, H, 2, d]: one absmax scale per (batch, head, map)."""
    if x.dtype != torch.bfloat16 or x.dim() != 5 or x.shape[3] != 2:
        raise ValueError("x must be bfloat16 [B, N, H, 2, d]")
    B, N, H, _, d = x.shape
    if d % 8:
        raise ValueError("d must be a multiple of 8")
    shape = (B, N, H, 2, d // 2)
    if codes is None:
        codes = torch.empty(shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((B, H, 2), dtype=torch.float32, device=x.device)
    if tuple(codes.shape) != shape or codes.dtype != torch.uint8 or scales.numel() != B * H * 2 or \
            scales.dtype != torch.float32:
        raise ValueError("codes must be uint8 [B, N, H, 2, d / 2] and scales float32 [B, H, 2]")
    _launch("diffattn_quantize_qk4", (x, codes, scales),
            _ptr(x), B, N, H, d, _ptr(codes), _ptr(scales))
    return codes, scales


def diffattn_fwd_qk4(q_codes: torch.Tensor, q_scales: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor,
                     v: torch.Tensor, lam: torch.Tensor, lambda_init: float, rms_w: torch.Tensor, eps: float = 1e-5,
                     causal: bool = True, out: torch.Tensor | None = None, mode: int = MODE_DIFF) -> torch.Tensor:
    """Prefill with e2m1 queries and keys (as quantize_qk4 returns them, [B, N, H, 2, d / 2]);
    v, out: bf16 [B, N, H, 2d]."""
    if q_codes.dtype != torch.uint8 or k_codes.dtype != torch.uint8 or k_codes.shape != q_codes.shape or \
            q_codes.dim() != 5 or q_codes.shape[3] != 2:
        raise ValueError("q_codes, k_codes must be uint8 [B, N, H, 2, d / 2]")
    B, N, H, _, half = q_codes.shape
    d = 2 * half
    _lowbit_rest(B, N, H, d, q_scales, k_scales, v, lam, rms_w)
    if out is None:
        out = torch.empty_like(v)
    _like("out", out, v.shape, torch.bfloat16)
    _launch("diffattn_fwd_qk4", (q_codes, q_scales, k_codes, k_scales, v, lam, rms_w, out),
            _ptr(q_codes), _ptr(q_scales), _ptr(k_codes), _ptr(k_scales), _ptr(v), _ptr(out), B, N, H, d,
            int(bool(causal)), _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps), int(mode))
    return out


def bwd_workspace_size(B: int, N: int, H: int, d: int) -> int:
    return int(lib().diffattn_bwd_workspace_size(B, N, H, d))


def diffattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dy: torch.Tensor, lam: torch.Tensor,
                 lambda_init: float, rms_w: torch.Tensor, eps: float = 1e-5, causal: bool = True,
                 mode: int = MODE_DIFF, workspace: torch.Tensor | None = None):
    """Backward of the prefill: (dq, dk, dv, dlambda, drms_w), float32, for the upstream gradient dy
    (shaped like v).  q, k, v, dy share one dtype (bfloat16 or float32)."""
    B, N, H, d = _qkv(q, k, v, dy)
    dt = BF16 if q.dtype == torch.bfloat16 else F32 if q.dtype == torch.float32 else None
    if dt is None or any(t.dtype != q.dtype for t in (k, v, dy)):
        raise ValueError("q, k, v, dy must share one dtype, bfloat16 or float32")
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    _dev(q, k, v, dy, lam, rms_w)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq, dk, dv = torch.empty(q.shape, **f32), torch.empty(k.shape, **f32), torch.empty(v.shape, **f32)
    dlam, dw = torch.empty(1, **f32), torch.empty(2 * d, **f32)
    need = bwd_workspace_size(B, N, H, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _launch("diffattn_bwd", (q, k, v, dy, lam, rms_w, dq, dk, dv, dlam, dw, workspace),
            _ptr(q), _ptr(k), _ptr(v), _ptr(dy), dt, B, N, H, d, int(bool(causal)), _ptr(lam), float(lambda_init),
            _ptr(rms_w), float(eps), int(mode), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), _ptr(dw), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    return dq, dk, dv, dlam, dw


def _grads_out(out, q: torch.Tensor, v: torch.Tensor, d: int):
    """The five float32 gradient outputs (dq, dk, dv, dlambda, drms_w), allocated when `out` is None."""
    f32 = dict(dtype=torch.float32, device=q.device)
    if out is None:
        return (torch.empty(q.shape, **f32), torch.empty(q.shape, **f32), torch.empty(v.shape, **f32),
                torch.empty(1, **f32), torch.empty(2 * d, **f32))
    _need(len(out) == 5, "out must hold (dq, dk, dv, dlambda, drms_w)")
    dq, dk, dv, dlam, dw = out
    _like("dq", dq, q.shape, torch.float32)
    _like("dk", dk, q.shape, torch.float32)
    _like("dv", dv, v.shape, torch.float32)
    _scalar_f32("dlambda", dlam)
    _f32("drms_w", dw, 2 * d)
    _dev(dq, dk, dv, dlam, dw)
    return out


def bwd_tc_workspace_size(B: int, N: int, H: int, d: int) -> int:
    return int(lib().diffattn_bwd_tc_workspace_size(B, N, H, d))


def diffattn_bwd_tc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dy: torch.Tensor, lam: torch.Tensor,
                    lambda_init: float, rms_w: torch.Tensor, eps: float = 1e-5, causal: bool = True,
                    mode: int = MODE_DIFF, workspace: torch.Tensor | None = None, out=None):
    """Tensor-core backward of the prefill: (dq, dk, dv, dlambda, drms_w), float32, for bfloat16 q, k, v and
    upstream gradient dy (shaped like v), d = 64 or 128.  `out` may hold preallocated outputs in that order."""
    B, N, H, d = _qkv(q, k, v, dy)
    if any(t.dtype != torch.bfloat16 for t in (q, k, v, dy)):
        raise ValueError("q, k, v, dy must be bfloat16")
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    dq, dk, dv, dlam, dw = _grads_out(out, q, v, d)
    _dev(q, k, v, dy, lam, rms_w)
    if workspace is None:
        workspace = torch.empty(bwd_tc_workspace_size(B, N, H, d), dtype=torch.uint8, device=q.device)
    _launch("diffattn_bwd_tc", (q, k, v, dy, lam, rms_w, dq, dk, dv, dlam, dw, workspace),
            _ptr(q), _ptr(k), _ptr(v), _ptr(dy), B, N, H, d, int(bool(causal)), _ptr(lam), float(lambda_init),
            _ptr(rms_w), float(eps), int(mode), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), _ptr(dw), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    return dq, dk, dv, dlam, dw


def diffattn_fwd_train(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, lambda_init: float,
                       rms_w: torch.Tensor, eps: float = 1e-5, causal: bool = True, mode: int = MODE_DIFF,
                       workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """Training forward: (o, workspace).  o as diffattn_fwd; the workspace (bwd_tc_workspace_size bytes) holds
    what diffattn_bwd_tc_saved needs for the same q, k, v, lambda and mask."""
    B, N, H, d = _qkv(q, k, v)
    if any(t.dtype != torch.bfloat16 for t in (q, k, v)):
        raise ValueError("q, k, v must be bfloat16")
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    if out is None:
        out = torch.empty_like(v)
    _like("out", out, v.shape, torch.bfloat16)
    if workspace is None:
        workspace = torch.empty(bwd_tc_workspace_size(B, N, H, d), dtype=torch.uint8, device=q.device)
    _launch("diffattn_fwd_train", (q, k, v, lam, rms_w, out, workspace),
            _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, N, H, d, int(bool(causal)), _ptr(lam), float(lambda_init),
            _ptr(rms_w), float(eps), int(mode), _ptr(workspace), workspace.numel() * workspace.element_size())
    return out, workspace


def diffattn_bwd_tc_saved(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dy: torch.Tensor, lam: torch.Tensor,
                          lambda_init: float, rms_w: torch.Tensor, eps: float, causal: bool, mode: int,
                          workspace: torch.Tensor, out=None):
    """diffattn_bwd_tc using the statistics diffattn_fwd_train left in `workspace`."""
    B, N, H, d = _qkv(q, k, v, dy)
    if any(t.dtype != torch.bfloat16 for t in (q, k, v, dy)):
        raise ValueError("q, k, v, dy must be bfloat16")
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    dq, dk, dv, dlam, dw = _grads_out(out, q, v, d)
    _launch("diffattn_bwd_tc_saved", (q, k, v, dy, lam, rms_w, dq, dk, dv, dlam, dw, workspace),
            _ptr(q), _ptr(k), _ptr(v), _ptr(dy), B, N, H, d, int(bool(causal)), _ptr(lam), float(lambda_init),
            _ptr(rms_w), float(eps), int(mode), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), _ptr(dw), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    return dq, dk, dv, dlam, dw


def rope_table(N: int, d: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """(cos, sin) of n * base^(-2j/d) for n < N, j < d/2: float32 [N, d/2, 2] on the device."""
    t = torch.empty((N, d // 2, 2), dtype=torch.float32, device=device or torch.device("cuda"))
    _launch("diffattn_rope_table", (t,), int(N), int(d), float(base), _ptr(t))
    return t


def qkv_proj(x: torch.Tensor, w_qkv: torch.Tensor, B: int, N: int, H: int, d: int, rope: torch.Tensor | None = None,
             out=None):
    """[Q | K | V] = x w_qkv^T with RoPE (from rope_table) on Q and K: q, k [B, N, H, 2, d], v [B, N, H, 2d],
    bfloat16.  x: bfloat16 [B*N, d_model]; w_qkv: bfloat16 [3*H*2d, d_model] (W_q; W_k; W_v)."""
    dm = x.shape[-1]
    if x.dtype != torch.bfloat16 or w_qkv.dtype != torch.bfloat16 or x.numel() != B * N * dm:
        raise ValueError("x must be bfloat16 [B*N, d_model]")
    if tuple(w_qkv.shape) != (3 * H * 2 * d, dm):
        raise ValueError("w_qkv must be bfloat16 [3*H*2d, d_model]")
    if rope is not None and (rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[0] < N or
                             rope.shape[1] * 2 != d or rope.shape[2] != 2):
        raise ValueError("rope must come from rope_table(>= N, d)")
    if out is None:
        bf = dict(dtype=torch.bfloat16, device=x.device)
        out = (torch.empty((B, N, H, 2, d), **bf), torch.empty((B, N, H, 2, d), **bf), torch.empty((B, N, H, 2 * d), **bf))
    _need(len(out) == 3, "out must hold (q, k, v)")
    q, k, v = out
    _like("q", q, (B, N, H, 2, d), torch.bfloat16)
    _like("k", k, (B, N, H, 2, d), torch.bfloat16)
    _like("v", v, (B, N, H, 2 * d), torch.bfloat16)
    _launch("diffattn_qkv_proj", (x, w_qkv, q, k, v, *(() if rope is None else (rope,))),
            _ptr(x), _ptr(w_qkv), B, N, dm, H, d, _ptr(rope) if rope is not None else None, _ptr(q), _ptr(k), _ptr(v))
    return q, k, v


def out_proj(o: torch.Tensor, w_o: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = o w_o^T: o bfloat16 [M, K] (or [B, N, H, 2d]), w_o bfloat16 [n_out, K] -> y bfloat16 [M, n_out]."""
    if w_o.dim() != 2 or o.dtype != torch.bfloat16 or w_o.dtype != torch.bfloat16 or o.numel() % w_o.shape[1]:
        raise ValueError("o and w_o must be bfloat16 with o's rows of width w_o.shape[1]")
    K = w_o.shape[1]
    M, n_out = o.numel() // K, w_o.shape[0]
    if out is None:
        out = torch.empty((M, n_out), dtype=torch.bfloat16, device=o.device)
    _like("out", out, (M, n_out), torch.bfloat16)
    _launch("diffattn_out_proj", (o, w_o, out),
            _ptr(o), _ptr(w_o), M, K, n_out, _ptr(out))
    return out


def diffattn_lambda_bwd(lq1: torch.Tensor, lk1: torch.Tensor, lq2: torch.Tensor, lk2: torch.Tensor,
                        dlam: torch.Tensor):
    """Gradients (dlq1, dlk1, dlq2, dlk2) of the lambda re-parameterisation for a device dlambda."""
    for name, t in (("lq1", lq1), ("lk1", lk1), ("lq2", lq2), ("lk2", lk2)):
        _f32(name, t, lq1.numel())
    _scalar_f32("dlam", dlam)
    _dev(lq1, lk1, lq2, lk2, dlam)
    outs = [torch.empty_like(t) for t in (lq1, lk1, lq2, lk2)]
    _launch("diffattn_lambda_bwd", (lq1, lk1, lq2, lk2, dlam, *outs),
            _ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), lq1.numel(), _ptr(dlam), *[_ptr(t) for t in outs])
    return tuple(outs)


def _decode_shapes(q, k_cache, v_cache, cu_seqlens, lam, rms_w):
    """(S, H, d) of a decode call; checks every shape and dtype the kernels rely on (the offsets in
    cu_seqlens are device data: the caller keeps them within the cache)."""
    _need(q.dim() == 4 and q.shape[2] == 2, "q must be [S, H, 2, d]")
    S, H, _, d = q.shape
    _need(k_cache.dim() == 4 and tuple(k_cache.shape[1:]) == (H, 2, d) and k_cache.dtype == q.dtype,
          "k_cache must be [T, H, 2, d] of q's dtype")
    _like("v_cache", v_cache, (k_cache.shape[0], H, 2 * d), q.dtype)
    _need(cu_seqlens.dtype == torch.int32 and cu_seqlens.numel() == S + 1,
          "cu_seqlens must be int32 with S + 1 entries")
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    _dev(q, k_cache, v_cache, cu_seqlens, lam, rms_w)
    return S, H, d


def decode_workspace_size(S: int, H: int, d: int, max_seqlen: int) -> int:
    return int(lib().diffattn_decode_workspace_size(S, H, d, max_seqlen))


def diffattn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, cu_seqlens: torch.Tensor,
                    max_seqlen: int, lam: torch.Tensor, lambda_init: float, rms_w: torch.Tensor,
                    eps: float = 1e-5, workspace: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, mode: int = MODE_DIFF) -> torch.Tensor:
    """Decode.  q: [S, H, 2, d]; k_cache: [T, H, 2, d]; v_cache: [T, H, 2d]; cu_seqlens: int32 [S + 1].
    ``mode`` as in diffattn_fwd."""
    S, H, d = _decode_shapes(q, k_cache, v_cache, cu_seqlens, lam, rms_w)
    need = decode_workspace_size(S, H, d, max_seqlen)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((S, H, 2 * d), dtype=q.dtype, device=q.device)
    _like("out", out, (S, H, 2 * d), q.dtype)
    ts = (q, k_cache, v_cache, cu_seqlens, lam, rms_w, workspace, out)
    ws_bytes = workspace.numel() * workspace.element_size()
    if mode == MODE_DIFF:
        _launch("diffattn_decode", ts, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens), int(max_seqlen),
                _ptr(out), S, H, d, _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps), _ptr(workspace), ws_bytes)
    else:
        _launch("diffattn_decode_mode", ts, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens),
                int(max_seqlen), _ptr(out), S, H, d, _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps),
                int(mode), _ptr(workspace), ws_bytes)
    return out


NOALLOC_SCRATCH_BYTES = 16 << 20  # DIFFATTN_DECODE_NOALLOC_SCRATCH_BYTES


def diffattn_decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            cu_seqlens: torch.Tensor, max_seqlen: int, lam: torch.Tensor, lambda_init: float,
                            rms_w: torch.Tensor, eps: float = 1e-5, out: torch.Tensor | None = None) -> torch.Tensor:
    """Decode without a workspace, for callers that may not allocate device memory.

    The library's built-in 16 MiB device scratch replaces the workspace; calls
    that overlap on the GPU share it and race.  Pass ``out`` to keep this call
    free of allocations on the Python side as well.
    """
    S, H, d = _decode_shapes(q, k_cache, v_cache, cu_seqlens, lam, rms_w)
    if out is None:
        out = torch.empty((S, H, 2 * d), dtype=q.dtype, device=q.device)
    _like("out", out, (S, H, 2 * d), q.dtype)
    _launch("diffattn_decode_noalloc", (q, k_cache, v_cache, cu_seqlens, lam, rms_w, out),
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens), int(max_seqlen), _ptr(out), S, H, d,
            _ptr(lam), float(lambda_init), _ptr(rms_w), float(eps))
    return out


# ------------------------------------------------ serving from a paged cache --
# These calls are short and made every step, so their checks build a message only when one fails.
def _i32(name: str, t: torch.Tensor, *shape: int) -> None:
    if t.dtype is not torch.int32 or t.shape != shape:
        raise ValueError(f"{name} must be int32 of shape {shape}")


def _int32(name: str, x) -> int:
    """x as the library takes its sizes and switches (ctypes would drop the bits above)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits")
    return x


def _same(name: str, t: torch.Tensor, shape, dtype) -> None:
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}")


def paged_step(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
               pool: torch.Tensor, page_size: int, num_tokens: int, pool_out: torch.Tensor | None = None, out=None):
    """Block tables and slot maps of one step from the requests' lengths: (cu_q, kv_lens, positions, slots, info).

    ctx_lens, new_lens: int32 [S] (new_lens -1: the request is finished); block_table: int32 [S, max_pages],
    updated; free_pages: int32 ring of free pages, updated; pool: int32 [2] (head, count), replaced in place unless
    pool_out is given (in place costs a second launch where the step has more than 512 tokens or 16 requests); num_tokens: rows of positions and slots (-1 behind the last new token).  info: int32 [4]
    (tokens, pages taken, pages returned, 0 or what is wrong; then the step took nothing)."""
    fast = marshal()
    if fast and (out is None or len(out) == 5):
        r = fast.paged_step(ctx_lens, new_lens, block_table, free_pages, pool, pool if pool_out is None else pool_out,
                            page_size, num_tokens, *((None,) * 5 if out is None else out))
        if type(r) is tuple:
            return r
        if _made("diffattn_paged_step", r):
            return tuple(out)
    _need(ctx_lens.dim() == 1 and block_table.dim() == 2 and free_pages.dim() == 1,
          "ctx_lens must be [S], block_table [S, max_pages] and free_pages [ring_size]")
    S, max_pages = block_table.shape
    T, page_size = _int32("num_tokens", num_tokens), _int32("page_size", page_size)
    _need(T >= 0, "num_tokens must not be negative")
    _i32("ctx_lens", ctx_lens, S)
    _i32("new_lens", new_lens, S)
    _i32("block_table", block_table, S, max_pages)
    F = _int32("ring_size", free_pages.numel())
    _int32("max_pages", max_pages)
    _i32("free_pages", free_pages, F)
    _i32("pool", pool, 2)
    if pool_out is None:
        pool_out = pool
    _i32("pool_out", pool_out, 2)
    ts = (ctx_lens, new_lens, block_table, free_pages, pool, pool_out)
    if out is None:  # parts of one allocation
        out = torch.unsafe_split_with_sizes(
            torch.empty(2 * S + 2 * T + 5, dtype=torch.int32, device=ctx_lens.device), (S + 1, S, T, T, 4))
    else:
        _need(len(out) == 5 and all(t is not None for t in out),
              "out must hold (cu_q, kv_lens, positions, slots, info)")
        for name, t, n in zip(("cu_q", "kv_lens", "positions", "slots", "info"), out, (S + 1, S, T, T, 4)):
            _i32(name, t, n)
        ts += tuple(out)
    cu_q, kv_lens, positions, slots, info = out
    _launch("diffattn_paged_step", ts,
            ctx_lens.data_ptr(), new_lens.data_ptr(), S, block_table.data_ptr(), max_pages, free_pages.data_ptr(), F,
            pool.data_ptr(), pool_out.data_ptr(), page_size, T, cu_q.data_ptr(), kv_lens.data_ptr(),
            positions.data_ptr(), slots.data_ptr(), info.data_ptr())
    return cu_q, kv_lens, positions, slots, info


def rope_table_scaled(N: int, rot: int, base: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
                      orig_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                      device=None) -> torch.Tensor:
    """(cos, sin) of n * theta'_j for n < N, j < rot/2 with the frequencies scaled for long contexts
    (ROPE_LINEAR, ROPE_NTK, ROPE_YARN; the last also scales cos and sin): float32 [N, rot/2, 2]."""
    N, rot, scaling = _int32("N", N), _int32("rot", rot), _int32("scaling", scaling)
    orig_len = _int32("orig_len", orig_len)
    t = torch.empty((N, rot // 2, 2), dtype=torch.float32, device=device or torch.device("cuda"))
    _launch("diffattn_rope_table_scaled", (t,), N, rot, float(base), scaling, float(factor), orig_len,
            float(beta_fast), float(beta_slow), _ptr(t))
    return t


def _rope_args(d, positions, table, T):
    ts = table.shape
    if table.dtype is not torch.float32 or len(ts) != 3 or ts[2] != 2 or ts[0] < 1 or not 1 <= ts[1] <= d // 2:
        raise ValueError("table must be float32 [n_pos, rot/2, 2] with rot <= d")
    if positions.dtype is not torch.int32 or positions.numel() != T:
        raise ValueError("positions must be int32 with one entry per row")
    return _int32("n_pos", ts[0]), 2 * ts[1]


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, table: torch.Tensor,
         layout: int = ROPE_INTERLEAVED, inverse: bool = False, out=None):
    """Queries and keys rotated at `positions`: (q', k').  q: [..., H, 2, d], k: [..., H_kv, 2, d] or None, float32
    or bfloat16, with one position (int32) per row of the leading dimensions; table: rope_table or
    rope_table_scaled, whose width says how many channels are rotated.  Rows with a negative position are left as
    they are in `out` (which may be (q, k) itself), or zeros with ROPE_PAD_ZERO added to `layout`; without `out` they
    are zeros.  ``inverse`` is the transposed map: gradients with respect to q', k' go in, those with respect to q, k
    come out.  q and k together stay below 2^31 elements, and so does the table."""
    if out is None:
        out = (torch.empty_like(q), None if k is None else torch.empty_like(k))
        layout = int(layout) | ROPE_PAD_ZERO
    _need(len(out) == 2, "out must hold (q', k')")
    fast = marshal()
    if fast and _made("diffattn_rope", fast.rope(q, k, positions, table, layout, 1 if inverse else 0, *out)):
        return tuple(out)
    qs = q.shape
    _need(len(qs) >= 4 and qs[-2] == 2, "q must be [..., H, 2, d]")
    H, d, layout = qs[-3], qs[-1], _int32("layout", layout)
    T = positions.numel()
    _need(q.numel() == T * H * 2 * d, "positions must be int32 with one entry per row")
    dt = BF16 if q.dtype == torch.bfloat16 else F32 if q.dtype == torch.float32 else None
    _need(dt is not None, "dtype must be bfloat16 or float32")
    H_kv = 0
    if k is not None:
        ks = k.shape
        _need(len(ks) == len(qs) and ks[:-3] == qs[:-3] and ks[-2:] == (2, d) and k.dtype is q.dtype,
              "k must be [..., H_kv, 2, d] with q's rows and dtype")
        H_kv = ks[-3]
    n_pos, rot = _rope_args(d, positions, table, T)
    qo, ko = out
    _same("q'", qo, qs, q.dtype)
    _need((ko is None) == (k is None), "out must hold k' exactly when k is given")
    ts = (q, positions, table, qo)
    if k is not None:
        _same("k'", ko, ks, k.dtype)
        ts += (k, ko)
    _launch("diffattn_rope", ts, q.data_ptr(), _ptr(k), positions.data_ptr(), table.data_ptr(), n_pos, T, H, H_kv, d,
            rot, dt, layout, int(bool(inverse)), qo.data_ptr(), _ptr(ko))
    return qo, ko


def _cache_shapes(k_cache, v_cache, d, dtype):
    """(num_pages, page_size, H_kv) of a paged cache."""
    s = k_cache.shape
    if len(s) != 5 or s[3] != 2 or s[4] != d or k_cache.dtype is not dtype:
        raise ValueError("k_cache must be [num_pages, page_size, H_kv, 2, d] of q's dtype")
    P, ps, H_kv, _, _ = s
    _same("v_cache", v_cache, (P, ps, H_kv, 2 * d), dtype)
    return _int32("num_pages", P), _int32("page_size", ps), H_kv


def _rows(q):
    """(T, H, d) of a step's queries."""
    s = q.shape
    if len(s) != 4 or s[2] != 2 or q.dtype is not torch.bfloat16:
        raise ValueError("q must be bfloat16 [T, H, 2, d]")
    return s[0], s[1], s[3]


def kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None, slots: torch.Tensor,
              table: torch.Tensor | None, k_cache: torch.Tensor, v_cache: torch.Tensor,
              layout: int = ROPE_INTERLEAVED, out: torch.Tensor | None = None) -> torch.Tensor:
    """The cache write of a step: returns q rotated at `positions`, and writes k rotated and v into the pages at
    `slots` (int32 [T], page * page_size + offset; negative: nothing is written).  q: bfloat16 [T, H, 2, d];
    k: [T, H_kv, 2, d]; v: [T, H_kv, 2d]; table None: no rotation (q is copied whole).  Rows with a negative position
    write nothing and are left as they are in `out` (which may be q), or zeros with ROPE_PAD_ZERO added to `layout`;
    without `out` they are zeros.  q and k together stay below 2^31 elements, and the cache below 2^31 tokens."""
    if out is None:
        out = torch.empty_like(q)
        layout = int(layout) | ROPE_PAD_ZERO
    fast = marshal()
    if fast and _made("diffattn_kv_append",
                      fast.kv_append(q, k, v, positions, slots, table, k_cache, v_cache, layout, out)):
        return out
    T, H, d = _rows(q)
    layout = _int32("layout", layout)
    num_pages, page_size, H_kv = _cache_shapes(k_cache, v_cache, d, torch.bfloat16)
    _same("k", k, (T, H_kv, 2, d), torch.bfloat16)
    _same("v", v, (T, H_kv, 2 * d), torch.bfloat16)
    _i32("slots", slots, T)
    n_pos = rot = 0
    _same("out", out, (T, H, 2, d), torch.bfloat16)
    ts = (q, k, v, slots, k_cache, v_cache, out)
    if table is not None:
        _need(positions is not None, "positions must be int32 with one entry per row")
        n_pos, rot = _rope_args(d, positions, table, T)
        ts += (positions, table)
    _launch("diffattn_kv_append", ts, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            None if table is None else positions.data_ptr(), slots.data_ptr(), _ptr(table), n_pos, T, H, H_kv, d, rot,
            layout, num_pages, page_size, out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr())
    return out


class ExtendPlan(NamedTuple):
    """A step's schedule (extend_plan): the device buffer and the sizes it was made for."""
    buf: torch.Tensor
    S: int
    T: int
    H: int
    H_kv: int
    d: int
    max_new: int


def extend_plan(cu_q: torch.Tensor, kv_lens: torch.Tensor, num_tokens: int, H: int, H_kv: int, d: int, max_new: int,
                causal: bool = True, buf: torch.Tensor | None = None) -> ExtendPlan:
    """The schedule of a step's attention, made once and read by every layer.  cu_q: int32 [S + 1]; kv_lens: int32
    [S]; num_tokens: rows of q; max_new: a host bound of the new tokens of a request (close ones are better: one that
    allows more than 16 rows a key head launches the many-row kernel, 4 to 8 us a layer where there is nothing for it)."""
    S = kv_lens.numel()
    _i32("cu_q", cu_q, S + 1)
    _i32("kv_lens", kv_lens, S)
    n = tuple(_int32(name, x) for name, x in (("S", S), ("num_tokens", num_tokens), ("H", H), ("H_kv", H_kv), ("d", d),
                                              ("max_new", max_new)))
    need = int(lib().diffattn_extend_plan_size(*n))
    if buf is None:
        buf = torch.empty(max(need, 16), dtype=torch.uint8, device=kv_lens.device)
    _launch("diffattn_extend_plan", (cu_q, kv_lens, buf), _ptr(cu_q), _ptr(kv_lens), *n, int(bool(causal)), _ptr(buf),
            buf.numel() * buf.element_size())
    return ExtendPlan(buf, *n)


def extend_workspace_size(plan: ExtendPlan) -> int:
    return int(lib().diffattn_extend_workspace_size(*(_int32(n, x) for n, x in zip(plan._fields[1:], plan[1:]))))


def diffattn_extend(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    plan: ExtendPlan, lam: torch.Tensor, lambda_init: float, rms_w: torch.Tensor, eps: float = 1e-5,
                    mode: int = MODE_DIFF, workspace: torch.Tensor | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Differential attention of the step's new tokens over the paged cache.  q: bfloat16 [T, H, 2, d]; k_cache:
    [num_pages, page_size, H_kv, 2, d]; v_cache: [num_pages, page_size, H_kv, 2d]; block_table: int32
    [S, max_pages]; plan: extend_plan's.  Rows behind the last request are left as they are in `out`, and zeros
    without it.  T * H * 2d must stay below 2^31.  A call of a layer passes `workspace` (extend_workspace_size bytes,
    shared by the layers) and `out`: without them both are allocated and `out` is filled with zeros."""
    if out is None or workspace is None:
        T, H, d = _rows(q)
        if workspace is None:
            workspace = torch.empty(max(extend_workspace_size(plan), 16), dtype=torch.uint8, device=q.device)
        if out is None:
            out = torch.zeros((T, H, 2 * d), dtype=q.dtype, device=q.device)
    fast = marshal()
    if fast and _made("diffattn_extend", fast.extend(q, k_cache, v_cache, block_table, *plan, lam, lambda_init, rms_w,
                                                     eps, mode, workspace, out)):
        return out
    T, H, d = _rows(q)
    num_pages, page_size, H_kv = _cache_shapes(k_cache, v_cache, d, q.dtype)
    _need((T, H, H_kv, d) == (plan.T, plan.H, plan.H_kv, plan.d), "the plan was made for other sizes")
    bs = block_table.shape
    if block_table.dtype is not torch.int32 or len(bs) != 2 or bs[0] != plan.S:
        raise ValueError("block_table must be int32 [S, max_pages] with the plan's S")
    S, max_new, max_pages = _int32("S", plan.S), _int32("max_new", plan.max_new), _int32("max_pages", bs[1])
    mode = _int32("mode", mode)
    _scalar_f32("lam", lam)
    _f32("rms_w", rms_w, 2 * d)
    _same("out", out, (T, H, 2 * d), q.dtype)
    _launch("diffattn_extend", (q, k_cache, v_cache, block_table, plan.buf, lam, rms_w, workspace, out),
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), max_pages, num_pages,
            page_size, plan.buf.data_ptr(), plan.buf.nbytes, S, T, H, H_kv, d, max_new, lam.data_ptr(),
            float(lambda_init), rms_w.data_ptr(), float(eps), mode, out.data_ptr(), workspace.data_ptr(),
            workspace.nbytes)
    return out


def device_status() -> int:
    """Synchronise the device and return (and clear) the kernels' status word."""
    v = ctypes.c_int(0)
    _check("diffattn_device_status", lib().diffattn_device_status(ctypes.byref(v)))
    return v.value


def set_wait_limit_ns(limit_ns: int) -> None:
    _check("diffattn_set_wait_limit_ns", lib().diffattn_set_wait_limit_ns(int(limit_ns)))
