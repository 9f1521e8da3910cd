"""Python binding of the dense bf16 ends of a training step around the frozen 4-bit MoE
layer: a gated feed-forward's gate and up half (a shared expert's), the losses of a vocabulary head (cross
entropy, distillation from a teacher's top logits) and layer norm.

As in train.py, arguments are contiguous CUDA tensors of one device, sizes, types and
devices are checked here and the rest by the library, calls run on the current stream of
the tensors' device, and none is recorded by autograd: each forward has a backward call
of its own beside it.
"""
from __future__ import annotations

import struct

import torch

import bit_quantized_moe_expert_amd as M

from .train import _BF16, _F32, _I32, _arg, _dims, _dt, _i32, _like, _out_dt, _p, _run, _scratch

# The C descriptors as packed bytes: nf4moe_gated_ffn_t (H, I, w13, glu, alpha, limit,
# interleaved), nf4moe_head_t (H, V, w) and nf4moe_layer_norm_t (H, x_dtype, y_dtype, w, b, eps).
_FFN = struct.Struct("@2iPi2fi0P")
_HEAD = struct.Struct("@2iP")
_LAYER_NORM = struct.Struct("@3i2Pf0P")


def _need(need, names):
    if not set(need) <= set(names) or not need:
        raise ValueError(f"need names {tuple(need)}, expected some of {', '.join(names)}")


def _ffn_args(x, w13, glu, alpha, limit, interleaved):
    """The descriptor, x's address, and (T, H, I, device index)."""
    T, H = _dims(x, "x", 2)
    rows, i = _dims(w13, "w13", 2)[0], x.get_device()
    if rows % 2:
        raise ValueError(f"w13 has {rows} rows, expected 2 I")
    wp = _arg(w13, "w13", (rows, H), _BF16, i)
    st = _FFN.pack(_i32(H, "H"), _i32(rows // 2, "I"), wp or 0, _i32(glu, "glu"), alpha, limit, _i32(interleaved, "interleaved"))
    return st, _arg(x, "x", x.shape, _BF16, i), T, H, rows // 2, i


def gated_ffn_forward(x, w13, *, glu: int = 0, alpha: float = 0.0, limit: float = 0.0, interleaved: int = 0, out=None):
    """The gated feed-forward's first half in one kernel: h = act(x Wg^T, x Wu^T), bf16 [T,
    I]. x bf16 [T, H]; w13 bf16 [2I, H], the gate rows and then the up rows (or
    interleaved); H and I multiples of 8; glu, alpha, limit, interleaved as in MoELayer;
    out: where h goes. Not recorded by autograd: the gradients are gated_ffn_backward's."""
    st, xp, T, _, I, i = _ffn_args(x, w13, glu, alpha, limit, interleaved)
    if out is None:
        out = x.new_empty((T, I))
    _run(i, M.lib().nf4moe_gated_ffn_forward, st, xp, T, _arg(out, "out", (T, I), _BF16, i))
    return out


def gated_ffn_backward(dh, x, w13, *, glu: int = 0, alpha: float = 0.0, limit: float = 0.0, interleaved: int = 0,
                       need=("dx", "dw13")):
    """Gradients of gated_ffn_forward for dh bf16 [T, I], from x and w13 alone (gate and up
    are computed again). Returns a dict of those in `need`: dx bf16 [T, H], dw13 bf16 [2I,
    H] in w13's row order, and beside them h (the forward's output, for the next weight's
    gradient). The same bits on every run of the same call (dx alone may be summed in
    another order than beside dw13)."""
    _need(need, ("dx", "dw13", "h"))
    st, xp, T, H, I, i = _ffn_args(x, w13, glu, alpha, limit, interleaved)
    dp = _arg(dh, "dh", (T, I), _BF16, i)
    out = {}
    if "dx" in need:
        out["dx"] = _like(x)
    if "dw13" in need:
        out["dw13"] = _like(w13)
    if "h" in need:
        out["h"] = _like(dh)
    L = M.lib()
    ws, wsp, nb = _scratch(x, L.nf4moe_gated_ffn_workspace_bytes(st, T))
    _run(i, L.nf4moe_gated_ffn_backward, st, dp, xp, T, _p(out.get("dx")), _p(out.get("dw13")), _p(out.get("h")), wsp, nb)
    return out


def _head_args(x, w):
    """The descriptor, x's address, and (T, device index)."""
    T, H = _dims(x, "x", 2)
    V, i = _dims(w, "w", 2)[0], x.get_device()
    wp = _arg(w, "w", (V, H), _BF16, i)
    return _HEAD.pack(_i32(H, "H"), _i32(V, "V"), wp or 0), _arg(x, "x", x.shape, _BF16, i), T, i


def vocab_ce_forward(x, w, labels):
    """Softmax cross entropy of the logits x w^T, which are never stored: (loss, lse), fp32
    [T]. x bf16 [T, H], w bf16 [V, H] (the head), labels int32 [T]; a label outside [0, V)
    (-100, say) has loss 0. H a multiple of 8. Not recorded by autograd: the gradients are
    vocab_ce_backward's."""
    st, xp, T, i = _head_args(x, w)
    lp = _arg(labels, "labels", (T,), _I32, i)
    loss = x.new_empty((T,), dtype=_F32)
    lse = _like(loss)
    L = M.lib()
    ws, wsp, nb = _scratch(x, L.nf4moe_vocab_workspace_bytes(st, T, 0, 0))
    _run(i, L.nf4moe_vocab_ce_forward, st, xp, T, lp, loss.data_ptr(), lse.data_ptr(), wsp, nb)
    return loss, lse


def _head_backward(x, w, T, k, st, need, call):
    _need(need, ("dx", "dw"))
    out = {}
    if "dx" in need:
        out["dx"] = _like(x)
    if "dw" in need:
        out["dw"] = _like(w)
    ws, wsp, nb = _scratch(x, M.lib().nf4moe_vocab_workspace_bytes(st, T, k, 1))
    call(_p(out.get("dx")), _p(out.get("dw")), wsp, nb)
    return out


def vocab_ce_backward(dloss, x, w, labels, lse, *, need=("dx", "dw")):
    """Gradients of vocab_ce_forward for dloss fp32 [T], with the forward's lse. Returns a
    dict of those in `need`: dx bf16 [T, H], dw bf16 [V, H]. Rows without a label count for
    nothing, whatever x and dloss hold there. The same bits on every run of the same call (dx
    alone may be summed in another order than beside dw)."""
    st, xp, T, i = _head_args(x, w)
    gp, lp, sp = _arg(dloss, "dloss", (T,), _F32, i), _arg(labels, "labels", (T,), _I32, i), _arg(lse, "lse", (T,), _F32, i)
    return _head_backward(x, w, T, 0, st, need, lambda dx, dw, ws, nb: _run(
        i, M.lib().nf4moe_vocab_ce_backward, st, gp, xp, T, lp, sp, dx, dw, ws, nb))


def vocab_distill_forward(x, w, ids, teacher, *, temperature: float = 1.0):
    """Distillation of the head x w^T from a teacher's top logits: ids int32 [T, k] and
    teacher fp32 or bf16 [T, k] (k up to 1024). Returns a dict: loss fp32 [T] =
    temperature^2 KL(teacher || student), the teacher's softmax over the given entries and
    the student's over the whole vocabulary, both at the temperature; lse fp32 [T]; q fp32
    [T, k], the teacher's probabilities; logits fp32 [T, k], the student's at the ids. An
    entry whose id lies outside [0, V) counts for nothing; a row without entries has loss 0
    and lse inf. Not recorded by autograd: the gradients are vocab_distill_backward's."""
    st, xp, T, i = _head_args(x, w)
    shape = _dims(ids, "ids", 2)
    ip = _arg(ids, "ids", (T, shape[1]), _I32, i)
    _dims(teacher, "teacher", 2)
    dt = _dt(teacher, "teacher")
    tp, k = _arg(teacher, "teacher", shape, teacher.dtype, i), _i32(shape[1], "k")
    loss = x.new_empty((T,), dtype=_F32)
    lse, q = _like(loss), _like(ids, dtype=_F32)
    logits = _like(q)
    L = M.lib()
    ws, wsp, nb = _scratch(x, L.nf4moe_vocab_workspace_bytes(st, T, k, 0))
    _run(i, L.nf4moe_vocab_distill_forward, st, xp, T, ip, tp, dt, k, temperature, loss.data_ptr(),
         lse.data_ptr(), q.data_ptr(), logits.data_ptr(), wsp, nb)
    return dict(loss=loss, lse=lse, q=q, logits=logits)


def vocab_distill_backward(dloss, x, w, ids, q, logits, lse, *, temperature: float = 1.0, need=("dx", "dw")):
    """Gradients of vocab_distill_forward for dloss fp32 [T], with the forward's q, logits and
    lse. Returns a dict of those in `need`: dx bf16 [T, H], dw bf16 [V, H]. The same bits as
    in vocab_ce_backward."""
    st, xp, T, i = _head_args(x, w)
    k = _i32(_dims(ids, "ids", 2)[1], "k")
    gp, ip = _arg(dloss, "dloss", (T,), _F32, i), _arg(ids, "ids", (T, k), _I32, i)
    qp, op, sp = _arg(q, "q", (T, k), _F32, i), _arg(logits, "logits", (T, k), _F32, i), _arg(lse, "lse", (T,), _F32, i)
    return _head_backward(x, w, T, k, st, need, lambda dx, dw, ws, nb: _run(
        i, M.lib().nf4moe_vocab_distill_backward, st, gp, xp, T, ip, qp, op, sp, k, temperature, dx, dw, ws, nb))


def _ln_args(x, w, b, y_dtype, eps):
    """The descriptor, x's address, and (T, H, device index)."""
    T, H = _dims(x, "x", 2)
    i = x.get_device()
    st = _LAYER_NORM.pack(_i32(H, "H"), _dt(x, "x"), y_dtype, _arg(w, "w", (H,), _F32, i) or 0, _arg(b, "b", (H,), _F32, i) or 0, eps)
    return st, _arg(x, "x", x.shape, x.dtype, i), T, H, i


def layer_norm_forward(x, w=None, b=None, *, eps: float = 1e-5, out_dtype=None):
    """Layer norm of x [T, H] (fp32 or bf16): y = (x - mean) rstd w + b, w and b fp32 [H] or
    None, y in out_dtype (x's by default). Returns a dict: y, mean, rstd (fp32 [T]; the
    backward takes them). Not recorded by autograd: the gradients are layer_norm_backward's."""
    dtype = x.dtype if out_dtype is None and isinstance(x, torch.Tensor) else out_dtype
    st, xp, T, H, i = _ln_args(x, w, b, _out_dt(dtype), eps)
    y = _like(x, dtype=dtype)
    mean = x.new_empty((T,), dtype=_F32)
    rstd = _like(mean)
    _run(i, M.lib().nf4moe_layer_norm_forward, st, xp, T, y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return dict(y=y, mean=mean, rstd=rstd)


def layer_norm_backward(dy, x, mean, rstd, w=None, *, dx_base=None, dx=None, need=("dx", "dw", "db")):
    """Gradients of layer_norm_forward for dy [T, H] in y's type, at its mean and rstd. Returns
    a dict of those in `need`: dx in x's type, with dx_base (the residual's gradient, x's
    type) added, at dx where given (may be dx_base); dw, db fp32 [H]. The same bits on
    every run."""
    _need(need, ("dx", "dw", "db"))
    if "dx" not in need and (dx_base is not None or dx is not None):
        raise ValueError("dx_base and dx go with need of dx")
    _dims(dy, "dy", 2)
    st, xp, T, H, i = _ln_args(x, w, None, _dt(dy, "dy"), 0.0)
    gp = _arg(dy, "dy", x.shape, dy.dtype, i)
    mp, rp = _arg(mean, "mean", (T,), _F32, i), _arg(rstd, "rstd", (T,), _F32, i)
    bp = _arg(dx_base, "dx_base", x.shape, x.dtype, i)
    out = {}
    if "dx" in need:
        out["dx"] = _like(x) if dx is None else dx
        _arg(out["dx"], "dx", x.shape, x.dtype, i)
    if "dw" in need:
        out["dw"] = x.new_empty((H,), dtype=_F32)
    if "db" in need:
        out["db"] = x.new_empty((H,), dtype=_F32)
    L = M.lib()
    ws, wsp, nb = _scratch(x, L.nf4moe_layer_norm_workspace_bytes(H, T))
    _run(i, L.nf4moe_layer_norm_backward, st, gp, xp, mp, rp, T, bp, _p(out.get("dx")), _p(out.get("dw")), _p(out.get("db")),
         wsp, nb)
    return out
