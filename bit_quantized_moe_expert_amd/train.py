"""Python binding of the fine-tuning operators around the frozen 4-bit MoE layer:
8-bit activation checkpoints, the gated activation that writes and reads them,
the norms around the block with their gate and residual scale, and the low-rank
adapters of many requests or experts beside a shared projection.

Like the rest of the binding this only marshals arguments; every step runs in the
library's HIP kernels, on the current stream of the tensors' device. Tensors are
contiguous CUDA tensors of one device; sizes, types and devices are checked here,
the rest by the library.

None of these calls is recorded by autograd: inputs that require grad are taken as
values, outputs have no grad_fn, and each forward has a backward call of its own
beside it, for a training loop or a torch.autograd.Function to call.
"""
from __future__ import annotations

import struct
from dataclasses import dataclass

import torch

import bit_quantized_moe_expert_amd as M

CKPT_MXINT8, CKPT_MXFP8 = 0, 1
GATE_IDENTITY, GATE_SIGMOID, GATE_TANH = 0, 1, 2
_SRC = {CKPT_MXINT8: 2, CKPT_MXFP8: 3}
_F32, _BF16, _U8, _I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
_DT = {_F32: M.DT_F32, _BF16: M.DT_BF16}


# A call on a few rows takes the GPU 3 us and its arguments' checks must not take
# longer: one comparison chain per tensor, the reason found only when it fails.
def _dims(t, name, n):
    """The shape of an n-dimensional tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != n:
        M._shape(t, name, (None,) * n)
    return t.shape


def _arg(t, name, shape, dtype, index):
    """The address of tensor t, None for None, after checking that it is a contiguous
    tensor of this shape and type on device `index` (-1: the CPU, which _run refuses
    once shapes and types are known to be right)."""
    if t is None:
        return None
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    M._shape(t, name, tuple(shape))
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, another device than the first tensor's")
    raise ValueError(f"{name} must be contiguous")


def _dt(t, name):
    """nf4moe_dtype_t of a float tensor (0 fp32, 1 bf16)."""
    d = _DT.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return d


def _out_dt(dtype):
    d = _DT.get(dtype)
    if d is None:
        raise TypeError(f"the output type must be torch.float32 or torch.bfloat16, got {dtype}")
    return d


def _run(index, fn, *args):
    """Call an entry point on the current stream of device `index`, that device current."""
    if index < 0:
        raise ValueError("the tensors are on cpu: libnf4moe computes on the GPU only "
                         "(the CPU reference is the test oracle, not a fallback)")
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        M._check(st)


def _p(t):
    return None if t is None else t.data_ptr()


# A new tensor of a checked (so contiguous) one's shape; 0.5 us sooner than new_empty.
_like = torch.empty_like


def _scratch(like, nbytes):
    """(tensor, address, size) of a 256-byte aligned workspace on like's device."""
    ws = like.new_empty(nbytes, dtype=_U8)
    ptr = ws.data_ptr()
    if ptr & 255:  # the caching allocator's blocks are aligned further; another allocator's need not be
        ws = like.new_empty(nbytes + 256, dtype=_U8)
        ptr = (ws.data_ptr() + 255) & ~255
    return ws, ptr, nbytes


@dataclass
class Ckpt8:
    """A tensor [.., K] held in 8 bits: codes uint8 [.., K] (int8 or e4m3 bits) and
    one e8m0 scale byte per 32 values, uint8 [.., K / 32]; fmt CKPT_MXINT8 or
    CKPT_MXFP8."""
    codes: object
    scale: object
    fmt: int

    def args(self, name, shape, index):
        """Addresses of codes (of this shape) and scale, checked."""
        if self.fmt not in (CKPT_MXINT8, CKPT_MXFP8):
            raise ValueError(f"{name}: unknown checkpoint format {self.fmt}")
        if not shape or shape[-1] <= 0 or shape[-1] % 32:
            raise ValueError(f"{name}: the last dimension of {tuple(shape)} must be a positive multiple of 32")
        return (_arg(self.codes, f"{name} codes", shape, _U8, index),
                _arg(self.scale, f"{name} scale", (*shape[:-1], shape[-1] // 32), _U8, index))


def ckpt8_quantize(x, fmt: int = CKPT_MXINT8) -> Ckpt8:
    """fp32 or bf16 x [.., K] (K % 32 == 0) -> its 8-bit checkpoint. Not recorded by
    autograd."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    dt, shape, i = _dt(x, "x"), x.shape, x.get_device()
    if not shape or shape[-1] <= 0 or shape[-1] % 32:
        raise ValueError(f"the last dimension of x {tuple(shape)} must be a positive multiple of 32")
    if fmt not in (CKPT_MXINT8, CKPT_MXFP8):
        raise ValueError(f"unknown checkpoint format {fmt}")
    xp, K = _arg(x, "x", shape, x.dtype, i), shape[-1]
    codes = _like(x, dtype=_U8)
    scale = x.new_empty((*shape[:-1], K // 32), dtype=_U8)
    _run(i, M.lib().nf4moe_ckpt8_quantize, fmt, xp, dt, x.numel() // K, K, codes.data_ptr(), scale.data_ptr())
    return Ckpt8(codes, scale, fmt)


def ckpt8_dequantize(ck: Ckpt8, dtype=_BF16):
    """The values an 8-bit checkpoint stands for, as dtype (bf16 by default, exact).
    Not recorded by autograd."""
    dt = _out_dt(dtype)
    if not isinstance(ck.codes, torch.Tensor):
        raise TypeError("checkpoint codes must be a torch tensor")
    shape, i = ck.codes.shape, ck.codes.get_device()
    cp, sp = ck.args("checkpoint", shape, i)
    K = shape[-1]
    out = _like(ck.codes, dtype=dtype)
    _run(i, M.lib().nf4moe_ckpt8_dequantize, ck.fmt, cp, sp, out.numel() // K, K, out.data_ptr(), dt)
    return out


def _glu_width(cols):
    if cols <= 0 or cols % 64:
        raise ValueError(f"gu has {cols} columns, expected 2 I with I a positive multiple of 32")
    return cols // 2


def glu_forward(gu, glu: int = 0, alpha: float = 0.0, limit: float = 0.0, interleaved: int = 0, ckpt=None):
    """The gated activation of gu [R, 2I] (bf16 or fp32): h bf16 [R, I]. With ckpt
    (CKPT_MXINT8 or CKPT_MXFP8) the same pass saves gu in 8 bits: (h, Ckpt8).
    glu, alpha, limit, interleaved as in MoELayer. Not recorded by autograd: the
    gradient is glu_backward's."""
    R, cols = _dims(gu, "gu", 2)
    dt, I, i = _dt(gu, "gu"), _i32(_glu_width(cols), "I"), gu.get_device()
    if ckpt not in (None, CKPT_MXINT8, CKPT_MXFP8):
        raise ValueError(f"unknown checkpoint format {ckpt}")
    gp = _arg(gu, "gu", gu.shape, gu.dtype, i)
    h = gu.new_empty((R, I), dtype=_BF16)
    if ckpt is None:
        _run(i, M.lib().nf4moe_glu_forward, gp, dt, R, I, glu, alpha, limit, interleaved, h.data_ptr(), 0, None, None)
        return h
    ck = Ckpt8(_like(gu, dtype=_U8), gu.new_empty((R, cols // 32), dtype=_U8), ckpt)
    _run(i, M.lib().nf4moe_glu_forward, gp, dt, R, I, glu, alpha, limit, interleaved, h.data_ptr(), ckpt,
         ck.codes.data_ptr(), ck.scale.data_ptr())
    return h, ck


def glu_backward(dh, gu, glu: int = 0, alpha: float = 0.0, limit: float = 0.0, interleaved: int = 0, row_w=None,
                 need_h: bool = True):
    """Gradient of glu_forward: dh [R, I] (bf16 or fp32), gu as the forward had it (a
    Ckpt8, or bf16 / fp32 [R, 2I]), row_w fp32 [R] or None. Returns a dict: dgu bf16
    [R, 2I]; h bf16 [R, I] recomputed (need_h); drow_w fp32 [R] (with row_w)."""
    R, I = _dims(dh, "dh", 2)
    ddt, i = _dt(dh, "dh"), dh.get_device()
    _glu_width(2 * _i32(I, "I"))
    if isinstance(gu, Ckpt8):
        gp, sp = gu.args("gu", (R, 2 * I), i)
        src = _SRC[gu.fmt]
    else:
        _dims(gu, "gu", 2)
        src, sp = _dt(gu, "gu"), None
        gp = _arg(gu, "gu", (R, 2 * I), gu.dtype, i)
    wp = _arg(row_w, "row_w", (R,), _F32, i)
    dp = _arg(dh, "dh", dh.shape, dh.dtype, i)
    out = dict(dgu=_like(gu.codes if isinstance(gu, Ckpt8) else gu, dtype=_BF16))
    if need_h:
        out["h"] = _like(dh, dtype=_BF16)
    if row_w is not None:
        out["drow_w"] = _like(row_w)
    _run(i, M.lib().nf4moe_glu_backward, dp, ddt, src, gp, sp, R, I, glu, alpha, limit, interleaved, wp,
         out["dgu"].data_ptr(), _p(out.get("h")), _p(out.get("drow_w")))
    return out


# The C descriptors as packed bytes (which a c_void_p argument passes by address):
# nf4moe_block_norm_t (H, x_dtype, w_post, w_pre, gate, gate_kind, gate_dtype, gate_fn,
# alpha, eps) and nf4moe_adapters_t (L, rank, K, N, A, B, scale).
_BLOCK_NORM = struct.Struct("@2i3P3i2f0P")
_ADAPTERS = struct.Struct("@4i3P")


def _i32(v, name):
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name}={v} does not fit 32 bits")
    return v


def _norm_struct(x, f, w_post, w_pre, gate, gate_fn, alpha, eps):
    """The descriptor, the addresses of x and f, and (T, H, device index)."""
    T, H = _dims(x, "x", 2)
    dt, i = _dt(x, "x"), x.get_device()
    kind, gdt, gp = 0, 0, None
    if gate is not None:  # [H] per channel, [T, 1] per row, [T, H] per element
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch tensor")
        kind = {(H,): 1, (T, H): 3, (T, 1): 2}.get(tuple(gate.shape))
        if kind is None:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected ({H},), ({T}, 1) or ({T}, {H})")
        gdt = _dt(gate, "gate")
        gp = _arg(gate, "gate", gate.shape, gate.dtype, i)
    fp = _arg(f, "f", x.shape, _BF16, i)
    st = _BLOCK_NORM.pack(_i32(H, "H"), dt, _arg(w_post, "w_post", (H,), _F32, i) or 0, _arg(w_pre, "w_pre", (H,), _F32, i) or 0,
                          gp or 0, kind, gdt, _i32(gate_fn, "gate_fn"), alpha, eps)
    return st, _arg(x, "x", x.shape, x.dtype, i), fp, T, H, i


def block_norm_forward(x, f=None, *, w_post=None, w_pre=None, gate=None, gate_fn: int = GATE_IDENTITY,
                       alpha: float = 1.0, eps: float = 1e-6, out=None):
    """Post norm, gate, residual and the next block's pre norm in one pass:
        x' = x + alpha * phi(gate) * f * rstd_post * w_post;  y = x' * rstd_pre * w_pre
    x fp32 or bf16 [T, H]; f bf16 [T, H] (None: a pre norm alone); w_post, w_pre fp32
    [H] (None: without that norm); gate fp32 or bf16, [H], [T, 1] or [T, H]; gate_fn
    GATE_IDENTITY, GATE_SIGMOID or GATE_TANH; out: where x' goes (may be x). Returns
    a dict: x (x', or x itself without f), y bf16, rstd_post, rstd_pre fp32 [T] (None
    where there is no such norm); block_norm_backward takes them. Not recorded by
    autograd: the gradients are block_norm_backward's."""
    st, xp, fp, T, H, i = _norm_struct(x, f, w_post, w_pre, gate, gate_fn, alpha, eps)
    if f is None:
        if out is not None:
            raise ValueError("out is for x', which a call without f does not write")
        np_ = None
    else:
        if out is None:
            out = _like(x)
        np_ = _arg(out, "out", x.shape, x.dtype, i)
    y = None if w_pre is None else _like(x, dtype=_BF16)
    rp = x.new_empty((T,), dtype=_F32) if w_post is not None else None
    r = None if w_pre is None else x.new_empty((T,), dtype=_F32) if rp is None else _like(rp)
    _run(i, M.lib().nf4moe_block_norm_forward, st, xp, fp, T, np_, _p(y), _p(rp), _p(r))
    return dict(x=x if f is None else out, y=y, rstd_post=rp, rstd_pre=r)


def block_norm_backward(dx_new, dy, x_new, f=None, *, rstd_post=None, rstd_pre=None, w_post=None, w_pre=None, gate=None,
                        gate_fn: int = GATE_IDENTITY, alpha: float = 1.0):
    """Gradients of block_norm_forward from dx_new (of x', None: zero) and dy (of y,
    with w_pre), at the x' and rstds that it returned. Returns a dict: dx in x's
    type; df bf16 (with f); dw_post, dw_pre fp32 [H], dgate fp32 in gate's shape (for
    those given). The same bits on every run."""
    st, xp, fp, T, H, i = _norm_struct(x_new, f, w_post, w_pre, gate, gate_fn, alpha, 0.0)
    if (dy is None) != (w_pre is None):
        raise ValueError("dy goes with w_pre")
    if dx_new is None and dy is None:
        raise ValueError("neither dx_new nor dy")
    if w_post is not None and rstd_post is None or w_pre is not None and rstd_pre is None:
        raise ValueError("w_post goes with rstd_post, w_pre with rstd_pre")
    dxp = _arg(dx_new, "dx_new", x_new.shape, x_new.dtype, i)
    dyp = _arg(dy, "dy", x_new.shape, _BF16, i)
    rp = None if w_post is None else _arg(rstd_post, "rstd_post", (T,), _F32, i)
    r = None if w_pre is None else _arg(rstd_pre, "rstd_pre", (T,), _F32, i)
    out = dict(dx=_like(x_new))
    if f is not None:
        out["df"] = _like(f)
    if gate is not None:
        out["dgate"] = _like(gate, dtype=_F32)
    if w_post is not None:
        out["dw_post"] = _like(w_post)
    if w_pre is not None:
        out["dw_pre"] = _like(w_pre)
    L = M.lib()
    ws, wsp, nb = _scratch(x_new, L.nf4moe_block_norm_workspace_bytes(H, T))
    _run(i, L.nf4moe_block_norm_backward, st, dxp, dyp, xp, fp, rp, r, T, out["dx"].data_ptr(),
         _p(out.get("df")), _p(out.get("dgate")), _p(out.get("dw_post")), _p(out.get("dw_pre")), wsp, nb)
    return out


@dataclass
class AdapterPlan:
    """The rows of one batch grouped by adapter (adapter_plan); holds for the ids it
    was made from."""
    buffer: object
    ptr: int
    nbytes: int
    R: int
    L: int


def adapter_plan(ids, num_adapters: int) -> AdapterPlan:
    """Group the rows of ids int32 [R] by adapter once, for several calls on the same
    batch (adapter_forward and adapter_backward otherwise do it in each call)."""
    (R,), i = _dims(ids, "ids", 1), ids.get_device()
    _i32(R, "rows"), _i32(num_adapters, "num_adapters")
    ip = _arg(ids, "ids", (R,), _I32, i)
    L = M.lib()
    ws, wsp, nb = _scratch(ids, L.nf4moe_adapter_plan_bytes(R, num_adapters))
    _run(i, L.nf4moe_adapter_plan, ip, R, num_adapters, wsp, nb)
    return AdapterPlan(ws, wsp, nb, R, num_adapters)


def _adapter_struct(A, B, ids, scale, plan, x_row_of, i):
    """The descriptor, (R, K, N, rank, L), and the addresses of ids, the gather, the plan and its size."""
    (L, rank, K), (R,), N = _dims(A, "A", 3), _dims(ids, "ids", 1), _dims(B, "B", 3)[1]
    _i32(R, "rows")
    st = _ADAPTERS.pack(_i32(L, "L"), _i32(rank, "rank"), _i32(K, "K"), _i32(N, "N"), _arg(A, "A", A.shape, _BF16, i),
                        _arg(B, "B", (L, N, rank), _BF16, i), _arg(scale, "scale", (L,), _F32, i) or 0)
    rows = (_arg(x_row_of, "x_row_of", (R,), _I32, i), _arg(ids, "ids", (R,), _I32, i))
    if plan is None:
        return st, (R, K, N, rank, L), rows, (None, 0)
    if plan.R != R or plan.L != L:
        raise ValueError(f"the plan is for {plan.R} rows of {plan.L} adapters, not {R} of {L}")
    if plan.buffer.get_device() != i:
        raise ValueError(f"the plan is on {plan.buffer.device}, expected device {i}")
    return st, (R, K, N, rank, L), rows, (plan.ptr, plan.nbytes)


def _gathered(x_row_of, R, rows):
    _i32(rows, "rows of x")
    if x_row_of is None and rows != R:
        raise ValueError(f"x has {rows} rows, expected {R} (or an x_row_of gather)")


def _one_dtype(what, *choices):
    """The type that the given ones (None left out) agree on, bf16 without any."""
    given = [c for c in choices if c is not None]
    if any(c is not given[0] for c in given):
        raise TypeError(f"{what} must agree on one type, got {given}")
    return given[0] if given else _BF16


def adapter_forward(x, A, B, ids, *, base=None, scale=None, x_row_of=None, out=None, out_dtype=None, plan=None,
                    return_t: bool = False):
    """Low-rank adapters beside a shared projection:
        out[r] = base[r] + scale[l] * B[l] (A[l] x[r]),  l = ids[r]
    x bf16 [rows, K] (row r of the call reads x[x_row_of[r]], or x[r]); A bf16 [L,
    rank, K], B bf16 [L, N, rank] (rank a multiple of 8 up to 128); ids int32 [R], an
    id outside [0, L) means no adapter; scale fp32 [L] or None; base bf16 or fp32 [R,
    N], the shared projection's output, or None (zeros); out: where the result goes
    (may be base), else a new tensor of base's type or out_dtype. Returns out, or
    (out, t) with t = A x fp32 [R, rank] for adapter_backward. Not recorded by autograd:
    the gradients are adapter_backward's."""
    rows, _ = _dims(x, "x", 2)
    i = x.get_device()
    dtype = _one_dtype("base, out and out_dtype", out if out is None else out.dtype, base if base is None else base.dtype,
                       out_dtype)
    dt = _out_dt(dtype)
    st, (R, K, N, rank, _), (rp, ip), (pp, pn) = _adapter_struct(A, B, ids, scale, plan, x_row_of, i)
    xp = _arg(x, "x", (rows, K), _BF16, i)
    _gathered(x_row_of, R, rows)
    bp = _arg(base, "base", (R, N), dtype, i)
    if out is None:
        out = x.new_empty((R, N), dtype=dtype) if base is None else _like(base)
    op = _arg(out, "out", (R, N), dtype, i)
    t = x.new_empty((R, rank), dtype=_F32) if return_t else None
    lib, sp = M.lib(), st
    nb = lib.nf4moe_adapter_workspace_bytes(sp, R, 0)
    ws, wsp, nb = _scratch(x, nb) if nb else (None, None, 0)
    _run(i, lib.nf4moe_adapter_forward, sp, xp, rows, rp, ip, pp, pn, R, bp, op, dt, _p(t), wsp, nb)
    return (out, t) if return_t else out


def adapter_backward(dy, x, t, A, B, ids, *, scale=None, x_row_of=None, dx_base=None, dx=None, dx_dtype=None, plan=None,
                     need=("dx", "dA", "dB")):
    """Gradients of adapter_forward for dy bf16 [R, N]. x as in the forward, bf16 or a
    Ckpt8 of it (read in 8 bits; K % 32 == 0); t the forward's. Returns a dict of
    those in `need`: dx [R, K] = dx_base + A^T u per row (dx_base bf16 or fp32 or None;
    dx: where it goes, may be dx_base), dA fp32 [L, rank, K], dB fp32 [L, N, rank].
    x may be None without dA, t without dB. The weights of all L adapters are read, used
    or not. The same bits on every run."""
    R, _ = _dims(dy, "dy", 2)
    i = dy.get_device()
    if not set(need) <= {"dx", "dA", "dB"}:
        raise ValueError(f"need names {set(need)}, expected some of dx, dA, dB")
    if "dA" in need and x is None:
        raise ValueError("dA needs x")
    if "dB" in need and t is None:
        raise ValueError("dB needs t")
    dtype = _one_dtype("dx_base, dx and dx_dtype", dx if dx is None else dx.dtype, dx_base if dx_base is None else dx_base.dtype,
                       dx_dtype)
    dt = _out_dt(dtype)
    st, (n, K, N, rank, L), (rp, ip), (pp, pn) = _adapter_struct(A, B, ids, scale, plan, x_row_of, i)
    dyp = _arg(dy, "dy", (n, N), _BF16, i)
    src, xp, xs, rows = M.DT_BF16, None, None, R
    if isinstance(x, Ckpt8):
        rows, _ = _dims(x.codes, "x codes", 2)
        xp, xs = x.args("x", (rows, K), i)
        src = _SRC[x.fmt]
    elif x is not None:
        rows, _ = _dims(x, "x", 2)
        xp = _arg(x, "x", (rows, K), _BF16, i)
    _gathered(x_row_of, R, rows)
    tp = _arg(t, "t", (R, rank), _F32, i)
    bp = _arg(dx_base, "dx_base", (R, K), dtype, i)
    out = {}
    if "dx" in need:
        out["dx"] = dx if dx is not None else dy.new_empty((R, K), dtype=dtype) if dx_base is None else _like(dx_base)
        _arg(out["dx"], "dx", (R, K), dtype, i)
    if "dA" in need:
        out["dA"] = _like(A, dtype=_F32)
    if "dB" in need:
        out["dB"] = _like(B, dtype=_F32)
    lib, sp = M.lib(), st
    ws, wsp, nb = _scratch(dy, lib.nf4moe_adapter_workspace_bytes(sp, R, 1))
    _run(i, lib.nf4moe_adapter_backward, sp, dyp, src, xp, xs, max(rows, 1), rp, tp, ip, pp, pn, R, bp, _p(out.get("dx")), dt,
         _p(out.get("dA")), _p(out.get("dB")), wsp, nb)
    return out
