"""Python binding of the fine-tuning operators around the frozen 4-bit MoE layer:
8-bit activation checkpoints, the gated activation that writes and reads them,
the norms around the block with their gate and residual scale, and the low-rank
adapters of many requests or experts beside a shared projection.

Like the rest of the binding this only marshals arguments; every step runs in the
library's HIP kernels, on the current stream of the tensors' device. Tensors are
contiguous CUDA tensors of one device; sizes, types and devices are checked here,
the rest by the library.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import bit_quantized_moe_expert_amd as M

CKPT_MXINT8, CKPT_MXFP8 = 0, 1
GATE_IDENTITY, GATE_SIGMOID, GATE_TANH = 0, 1, 2
_SRC = {CKPT_MXINT8: 2, CKPT_MXFP8: 3}


def _dt(t, name):
    """nf4moe_dtype_t of a float tensor (0 fp32, 1 bf16)."""
    torch = M._torch()
    if t.dtype == torch.bfloat16:
        return M.DT_BF16
    if t.dtype == torch.float32:
        return M.DT_F32
    raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")


def _out_dt(dtype):
    torch = M._torch()
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"the output type must be torch.float32 or torch.bfloat16, got {dtype}")
    return M.DT_BF16 if dtype == torch.bfloat16 else M.DT_F32


def _on(first, **tensors):
    """The tensors (None entries left out) are CUDA, contiguous and on first's device."""
    M._dev(first, "the first tensor")
    for name, t in tensors.items():
        if t is not None:
            M._dev(t, name)
            if t.device != first.device:
                raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _run(device, fn, *args):
    """Call an entry point with the device's current stream, that device current."""
    cuda = M._torch().cuda
    if cuda.current_device() == device.index:
        M._check(fn(*args, cuda.current_stream(device).cuda_stream))
    else:
        with cuda.device(device):
            M._check(fn(*args, cuda.current_stream(device).cuda_stream))


def _p(t):
    return None if t is None else t.data_ptr()


def _empty(shape, dtype, like):
    return M._torch().empty(shape, dtype=dtype, device=like.device)


@dataclass
class Ckpt8:
    """A tensor [.., K] held in 8 bits: codes uint8 [.., K] (int8 or e4m3 bits) and
    one e8m0 scale byte per 32 values, uint8 [.., K / 32]; fmt CKPT_MXINT8 or
    CKPT_MXFP8."""
    codes: object
    scale: object
    fmt: int

    def check(self, name="checkpoint"):
        torch = M._torch()
        if self.fmt not in (CKPT_MXINT8, CKPT_MXFP8):
            raise ValueError(f"{name}: unknown checkpoint format {self.fmt}")
        for what, t in (("codes", self.codes), ("scale", self.scale)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError(f"{name}: {what} must be a torch.uint8 tensor")
        shape = tuple(self.codes.shape)
        if not shape or shape[-1] == 0 or shape[-1] % 32:
            raise ValueError(f"{name}: the last dimension of codes {shape} must be a positive multiple of 32")
        M._shape(self.scale, f"{name} scale", shape[:-1] + (shape[-1] // 32,))
        _on(self.codes, scale=self.scale)
        return self


def ckpt8_quantize(x, fmt: int = CKPT_MXINT8) -> Ckpt8:
    """fp32 or bf16 x [.., K] (K % 32 == 0) -> its 8-bit checkpoint."""
    torch = M._torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    dt = _dt(x, "x")
    if x.dim() < 1 or x.shape[-1] <= 0 or x.shape[-1] % 32:
        raise ValueError(f"the last dimension of x {tuple(x.shape)} must be a positive multiple of 32")
    if fmt not in (CKPT_MXINT8, CKPT_MXFP8):
        raise ValueError(f"unknown checkpoint format {fmt}")
    _on(x)
    K = x.shape[-1]
    codes = _empty(x.shape, torch.uint8, x)
    scale = _empty((*x.shape[:-1], K // 32), torch.uint8, x)
    _run(x.device, M.lib().nf4moe_ckpt8_quantize, fmt, x.data_ptr(), dt, x.numel() // K, K, codes.data_ptr(),
         scale.data_ptr())
    return Ckpt8(codes, scale, fmt)


def ckpt8_dequantize(ck: Ckpt8, dtype=None):
    """The values an 8-bit checkpoint stands for, as dtype (bf16 by default, exact)."""
    torch = M._torch()
    dtype = dtype or torch.bfloat16
    dt = _out_dt(dtype)
    ck.check()
    K = ck.codes.shape[-1]
    out = _empty(ck.codes.shape, dtype, ck.codes)
    _run(out.device, M.lib().nf4moe_ckpt8_dequantize, ck.fmt, ck.codes.data_ptr(), ck.scale.data_ptr(),
         out.numel() // K, K, out.data_ptr(), dt)
    return out


def _glu_width(cols):
    if cols <= 0 or cols % 64:
        raise ValueError(f"gu has {cols} columns, expected 2 I with I a positive multiple of 32")
    return cols // 2


def glu_forward(gu, glu: int = 0, alpha: float = 0.0, limit: float = 0.0, interleaved: int = 0, ckpt=None):
    """The gated activation of gu [R, 2I] (bf16 or fp32): h bf16 [R, I]. With ckpt
    (CKPT_MXINT8 or CKPT_MXFP8) the same pass saves gu in 8 bits: (h, Ckpt8).
    glu, alpha, limit, interleaved as in MoELayer."""
    torch = M._torch()
    M._shape(gu, "gu", (None, None))
    dt = _dt(gu, "gu")
    if ckpt not in (None, CKPT_MXINT8, CKPT_MXFP8):
        raise ValueError(f"unknown checkpoint format {ckpt}")
    R, I = gu.shape[0], _glu_width(gu.shape[1])
    _on(gu)
    h = _empty((R, I), torch.bfloat16, gu)
    ck = None
    if ckpt is not None:
        ck = Ckpt8(_empty((R, 2 * I), torch.uint8, gu), _empty((R, I // 16), torch.uint8, gu), ckpt)
    _run(gu.device, M.lib().nf4moe_glu_forward, gu.data_ptr(), dt, R, I, glu, alpha, limit, interleaved, h.data_ptr(),
         ckpt or 0, _p(ck and ck.codes), _p(ck and ck.scale))
    return h if ck is None else (h, ck)


def glu_backward(dh, gu, glu: int = 0, alpha: float = 0.0, limit: float = 0.0, interleaved: int = 0, row_w=None,
                 need_h: bool = True):
    """Gradient of glu_forward: dh [R, I] (bf16 or fp32), gu as the forward had it (a
    Ckpt8, or bf16 / fp32 [R, 2I]), row_w fp32 [R] or None. Returns a dict: dgu bf16
    [R, 2I]; h bf16 [R, I] recomputed (need_h); drow_w fp32 [R] (with row_w)."""
    torch = M._torch()
    M._shape(dh, "dh", (None, None))
    R, I = dh.shape
    ddt = _dt(dh, "dh")
    if isinstance(gu, Ckpt8):
        gu.check("gu")
        M._shape(gu.codes, "gu codes", (R, 2 * I))
        src, values, scale = _SRC[gu.fmt], gu.codes, gu.scale
    else:
        M._shape(gu, "gu", (R, 2 * I))
        src, values, scale = _dt(gu, "gu"), gu, None
    _glu_width(2 * I)
    M._shape(row_w, "row_w", (R,))
    if row_w is not None and row_w.dtype != torch.float32:
        raise TypeError(f"row_w must be torch.float32, got {row_w.dtype}")
    _on(dh, gu=values, scale=scale, row_w=row_w)
    out = dict(dgu=_empty((R, 2 * I), torch.bfloat16, dh))
    if need_h:
        out["h"] = _empty((R, I), torch.bfloat16, dh)
    if row_w is not None:
        out["drow_w"] = _empty((R,), torch.float32, dh)
    _run(dh.device, M.lib().nf4moe_glu_backward, dh.data_ptr(), ddt, src, values.data_ptr(), _p(scale), R, I, glu,
         alpha, limit, interleaved, _p(row_w), out["dgu"].data_ptr(), _p(out.get("h")), _p(out.get("drow_w")))
    return out


class _BlockNorm(ctypes.Structure):
    """Mirror of nf4moe_block_norm_t."""
    _fields_ = [("H", ctypes.c_int32), ("x_dtype", ctypes.c_int32), ("w_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gate_kind", ctypes.c_int32),
                ("gate_dtype", ctypes.c_int32), ("gate_fn", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float)]


def _norm_struct(x, f, w_post, w_pre, gate, gate_fn, alpha, eps):
    torch = M._torch()
    M._shape(x, "x", (None, None))
    T, H = x.shape
    dt = _dt(x, "x")
    M._shape(f, "f", (T, H))
    if f is not None and f.dtype != torch.bfloat16:
        raise TypeError(f"f must be torch.bfloat16, got {f.dtype}")
    for name, w in (("w_post", w_post), ("w_pre", w_pre)):
        M._shape(w, name, (H,))
        if w is not None and w.dtype != torch.float32:
            raise TypeError(f"{name} must be torch.float32, got {w.dtype}")
    kind = 0
    if gate is not None:
        # [H] per channel, [T, 1] per row, [T, H] per element: told apart by the number of dimensions first
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch tensor")
        if tuple(gate.shape) == (H,):
            kind = 1
        elif gate.dim() == 2 and tuple(gate.shape) == (T, 1):
            kind = 2
        elif tuple(gate.shape) == (T, H):
            kind = 3
        else:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected ({H},), ({T}, 1) or ({T}, {H})")
    _on(x, f=f, w_post=w_post, w_pre=w_pre, gate=gate)
    return _BlockNorm(H, dt, _p(w_post), _p(w_pre), _p(gate), kind, M.DT_F32 if gate is None else _dt(gate, "gate"),
                      gate_fn, alpha, eps), T, H


def block_norm_forward(x, f=None, *, w_post=None, w_pre=None, gate=None, gate_fn: int = GATE_IDENTITY,
                       alpha: float = 1.0, eps: float = 1e-6, out=None):
    """Post norm, gate, residual and the next block's pre norm in one pass:
        x' = x + alpha * phi(gate) * f * rstd_post * w_post;  y = x' * rstd_pre * w_pre
    x fp32 or bf16 [T, H]; f bf16 [T, H] (None: a pre norm alone); w_post, w_pre fp32
    [H] (None: without that norm); gate fp32 or bf16, [H], [T, 1] or [T, H]; gate_fn
    GATE_IDENTITY, GATE_SIGMOID or GATE_TANH; out: where x' goes (may be x). Returns
    a dict: x (x', or x itself without f), y bf16, rstd_post, rstd_pre fp32 [T] (None
    where there is no such norm); block_norm_backward takes them."""
    torch = M._torch()
    st, T, H = _norm_struct(x, f, w_post, w_pre, gate, gate_fn, alpha, eps)
    if f is None:
        if out is not None:
            raise ValueError("out is for x', which a call without f does not write")
        new = None
    elif out is None:
        new = torch.empty_like(x)
    else:
        M._shape(out, "out", (T, H))
        if out.dtype != x.dtype:
            raise TypeError(f"out must be {x.dtype}, got {out.dtype}")
        _on(x, out=out)
        new = out
    y = _empty((T, H), torch.bfloat16, x) if w_pre is not None else None
    rp = _empty((T,), torch.float32, x) if w_post is not None else None
    r = _empty((T,), torch.float32, x) if w_pre is not None else None
    _run(x.device, M.lib().nf4moe_block_norm_forward, ctypes.addressof(st), x.data_ptr(), _p(f), T, _p(new), _p(y),
         _p(rp), _p(r))
    return dict(x=x if new is None else new, y=y, rstd_post=rp, rstd_pre=r)


def block_norm_backward(dx_new, dy, x_new, f=None, *, rstd_post=None, rstd_pre=None, w_post=None, w_pre=None, gate=None,
                        gate_fn: int = GATE_IDENTITY, alpha: float = 1.0):
    """Gradients of block_norm_forward from dx_new (of x', None: zero) and dy (of y,
    with w_pre), at the x' and rstds that it returned. Returns a dict: dx in x's
    type; df bf16 (with f); dw_post, dw_pre fp32 [H], dgate fp32 in gate's shape (for
    those given). The same bits on every run."""
    torch = M._torch()
    st, T, H = _norm_struct(x_new, f, w_post, w_pre, gate, gate_fn, alpha, 0.0)
    M._shape(dx_new, "dx_new", (T, H))
    if dx_new is not None and dx_new.dtype != x_new.dtype:
        raise TypeError(f"dx_new must be {x_new.dtype}, got {dx_new.dtype}")
    if (dy is None) != (w_pre is None):
        raise ValueError("dy goes with w_pre")
    if dx_new is None and dy is None:
        raise ValueError("neither dx_new nor dy")
    M._shape(dy, "dy", (T, H))
    if dy is not None and dy.dtype != torch.bfloat16:
        raise TypeError(f"dy must be torch.bfloat16, got {dy.dtype}")
    for name, r, w in (("rstd_post", rstd_post, w_post), ("rstd_pre", rstd_pre, w_pre)):
        if w is None:
            continue
        if r is None:
            raise ValueError(f"{name} is needed")
        M._shape(r, name, (T,))
        if r.dtype != torch.float32:
            raise TypeError(f"{name} must be torch.float32, got {r.dtype}")
    _on(x_new, dx_new=dx_new, dy=dy, rstd_post=rstd_post, rstd_pre=rstd_pre)
    out = dict(dx=torch.empty_like(x_new))
    if f is not None:
        out["df"] = torch.empty_like(f)
    if gate is not None:
        out["dgate"] = _empty(gate.shape, torch.float32, x_new)
    if w_post is not None:
        out["dw_post"] = _empty((H,), torch.float32, x_new)
    if w_pre is not None:
        out["dw_pre"] = _empty((H,), torch.float32, x_new)
    L = M.lib()
    ws, wsp, nb = M._workspace(L.nf4moe_block_norm_workspace_bytes(H, T), x_new.device)
    _run(x_new.device, L.nf4moe_block_norm_backward, ctypes.addressof(st), _p(dx_new), _p(dy), x_new.data_ptr(), _p(f),
         _p(rstd_post) if w_post is not None else None, _p(rstd_pre) if w_pre is not None else None, T,
         out["dx"].data_ptr(), _p(out.get("df")), _p(out.get("dgate")), _p(out.get("dw_post")), _p(out.get("dw_pre")),
         wsp, nb)
    return out


class _Adapters(ctypes.Structure):
    """Mirror of nf4moe_adapters_t."""
    _fields_ = [("L", ctypes.c_int32), ("rank", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


@dataclass
class AdapterPlan:
    """The rows of one batch grouped by adapter (adapter_plan); holds for the ids it
    was made from."""
    buffer: object
    ptr: int
    nbytes: int
    R: int
    L: int


def _ids(ids):
    torch = M._torch()
    M._shape(ids, "ids", (None,))
    if ids.dtype != torch.int32:
        raise TypeError(f"ids must be torch.int32, got {ids.dtype}")
    return ids.shape[0]


def adapter_plan(ids, num_adapters: int) -> AdapterPlan:
    """Group the rows of ids int32 [R] by adapter once, for several calls on the same
    batch (adapter_forward and adapter_backward otherwise do it in each call)."""
    torch = M._torch()
    R = _ids(ids)
    _on(ids)
    L = M.lib()
    ws, wsp, nb = M._workspace(L.nf4moe_adapter_plan_bytes(R, num_adapters), ids.device)
    _run(ids.device, L.nf4moe_adapter_plan, ids.data_ptr(), R, num_adapters, wsp, nb)
    return AdapterPlan(ws, wsp.value, nb, R, num_adapters)


def _adapter_struct(A, B, ids, scale, plan):
    torch = M._torch()
    M._shape(A, "A", (None, None, None))
    L, rank, K = A.shape
    M._shape(B, "B", (L, None, rank))
    M._shape(scale, "scale", (L,))
    R = _ids(ids)
    for name, t, dt in (("A", A, torch.bfloat16), ("B", B, torch.bfloat16), ("scale", scale, torch.float32)):
        if t is not None and t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if plan is not None and (plan.R != R or plan.L != L):
        raise ValueError(f"the plan is for {plan.R} rows of {plan.L} adapters, not {R} of {L}")
    return _Adapters(L, rank, K, B.shape[1], A.data_ptr(), B.data_ptr(), _p(scale)), R, K, B.shape[1], rank, L


def _gather(x_row_of, R, rows):
    torch = M._torch()
    M._shape(x_row_of, "x_row_of", (R,))
    if x_row_of is not None and x_row_of.dtype != torch.int32:
        raise TypeError(f"x_row_of must be torch.int32, got {x_row_of.dtype}")
    if x_row_of is None and rows != R:
        raise ValueError(f"x has {rows} rows, expected {R} (or an x_row_of gather)")


def adapter_forward(x, A, B, ids, *, base=None, scale=None, x_row_of=None, out=None, out_dtype=None, plan=None,
                    return_t: bool = False):
    """Low-rank adapters beside a shared projection:
        out[r] = base[r] + scale[l] * B[l] (A[l] x[r]),  l = ids[r]
    x bf16 [rows, K] (row r of the call reads x[x_row_of[r]], or x[r]); A bf16 [L,
    rank, K], B bf16 [L, N, rank] (rank a multiple of 8 up to 128); ids int32 [R], an
    id outside [0, L) means no adapter; scale fp32 [L] or None; base bf16 or fp32 [R,
    N], the shared projection's output, or None (zeros); out: where the result goes
    (may be base), else a new tensor of base's type or out_dtype. Returns out, or
    (out, t) with t = A x fp32 [R, rank] for adapter_backward."""
    torch = M._torch()
    st, R, K, N, rank, _ = _adapter_struct(A, B, ids, scale, plan)
    M._shape(x, "x", (None, K))
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x must be torch.bfloat16, got {x.dtype}")
    _gather(x_row_of, R, x.shape[0])
    M._shape(base, "base", (R, N))
    M._shape(out, "out", (R, N))
    dtype = out.dtype if out is not None else base.dtype if base is not None else out_dtype or torch.bfloat16
    dt = _out_dt(dtype)
    if out_dtype is not None and out_dtype != dtype or base is not None and base.dtype != dtype:
        raise TypeError(f"base, out and out_dtype must agree on {dtype}")
    _on(x, A=A, B=B, ids=ids, scale=scale, x_row_of=x_row_of, base=base, out=out, plan=plan and plan.buffer)
    if out is None:
        out = _empty((R, N), dtype, x)
    t = _empty((R, rank), torch.float32, x) if return_t else None
    lib = M.lib()
    ws, wsp, nb = M._workspace(lib.nf4moe_adapter_workspace_bytes(ctypes.addressof(st), R, 0), x.device)
    _run(x.device, lib.nf4moe_adapter_forward, ctypes.addressof(st), x.data_ptr(), x.shape[0], _p(x_row_of),
         ids.data_ptr(), plan and plan.ptr, plan.nbytes if plan else 0, R, _p(base), out.data_ptr(), dt, _p(t), wsp, nb)
    return (out, t) if return_t else out


def adapter_backward(dy, x, t, A, B, ids, *, scale=None, x_row_of=None, dx_base=None, dx=None, dx_dtype=None, plan=None,
                     need=("dx", "dA", "dB")):
    """Gradients of adapter_forward for dy bf16 [R, N]. x as in the forward, bf16 or a
    Ckpt8 of it (read in 8 bits; K % 32 == 0); t the forward's. Returns a dict of
    those in `need`: dx [R, K] = dx_base + A^T u per row (dx_base bf16 or fp32 or None;
    dx: where it goes, may be dx_base), dA fp32 [L, rank, K], dB fp32 [L, N, rank].
    x may be None without dA, t without dB. The same bits on every run."""
    torch = M._torch()
    st, R, K, N, rank, L = _adapter_struct(A, B, ids, scale, plan)
    if not set(need) <= {"dx", "dA", "dB"}:
        raise ValueError(f"need names {set(need)}, expected some of dx, dA, dB")
    M._shape(dy, "dy", (R, N))
    if dy.dtype != torch.bfloat16:
        raise TypeError(f"dy must be torch.bfloat16, got {dy.dtype}")
    src, values, xs = M.DT_BF16, x, None
    if isinstance(x, Ckpt8):
        x.check("x")
        src, values, xs = _SRC[x.fmt], x.codes, x.scale
    elif x is not None and x.dtype != torch.bfloat16:
        raise TypeError(f"x must be torch.bfloat16 or a Ckpt8, got {x.dtype}")
    if "dA" in need and x is None:
        raise ValueError("dA needs x")
    if "dB" in need and t is None:
        raise ValueError("dB needs t")
    M._shape(values, "x", (None, K))
    rows = R if x is None else values.shape[0]
    _gather(x_row_of, R, rows)
    M._shape(t, "t", (R, rank))
    if t is not None and t.dtype != torch.float32:
        raise TypeError(f"t must be torch.float32, got {t.dtype}")
    M._shape(dx_base, "dx_base", (R, K))
    M._shape(dx, "dx", (R, K))
    dtype = dx.dtype if dx is not None else dx_base.dtype if dx_base is not None else dx_dtype or torch.bfloat16
    dt = _out_dt(dtype)
    if dx_dtype is not None and dx_dtype != dtype or dx_base is not None and dx_base.dtype != dtype:
        raise TypeError(f"dx_base, dx and dx_dtype must agree on {dtype}")
    _on(dy, A=A, B=B, ids=ids, scale=scale, x=values, x_scale=xs, x_row_of=x_row_of, t=t, dx_base=dx_base, dx=dx,
        plan=plan and plan.buffer)
    out = {}
    if "dx" in need:
        out["dx"] = _empty((R, K), dtype, dy) if dx is None else dx
    if "dA" in need:
        out["dA"] = _empty((L, rank, K), torch.float32, dy)
    if "dB" in need:
        out["dB"] = _empty((L, N, rank), torch.float32, dy)
    lib = M.lib()
    ws, wsp, nb = M._workspace(lib.nf4moe_adapter_workspace_bytes(ctypes.addressof(st), R, 1), dy.device)
    _run(dy.device, lib.nf4moe_adapter_backward, ctypes.addressof(st), dy.data_ptr(), src, _p(values), _p(xs), max(rows, 1),
         _p(x_row_of), _p(t), ids.data_ptr(), plan and plan.ptr, plan.nbytes if plan else 0, R, _p(dx_base),
         _p(out.get("dx")), dt, _p(out.get("dA")), _p(out.get("dB")), wsp, nb)
    return out
