"""What the dense calls write: their outputs and workspaces to the last byte and nothing beside them,
whatever the workspace held before. Through the C ABI, each array with marked bytes before and
behind it, matrices aligned to 16 bytes and no more."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402
from bit_quantized_moe_expert_amd import dense  # noqa: E402
from test_gpu_train_margins import Out, gen, run  # noqa: E402

DEV = "cuda"
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
L = M.lib()
SIZES = [(1, 8, 8), (3, 72, 40), (17, 136, 1003), (33, 64, 2000), (65, 264, 517), (130, 128, 4099), (300, 72, 1032), (1030, 40, 9001)]


def skewed(t):
    """The same values 16 bytes past a 256-byte boundary, NaN around them."""
    n = t.numel()
    buf = torch.full((n + 512,), float("nan"), dtype=t.dtype, device=DEV) if t.is_floating_point() else \
        torch.full((n + 512,), -1, dtype=t.dtype, device=DEV)
    off = (256 - buf.data_ptr() % 256) % 256 // t.element_size() + 16 // t.element_size()
    buf[off:off + n] = t.reshape(-1)
    return buf[off:off + n].view(t.shape)


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("T,H,I", [(t, h, (i + 7) // 8 * 8) for t, h, i in SIZES])
def test_gated_ffn(T, H, I, inter):
    rn = gen(T + H)
    x, w, dh = (skewed(v) for v in (rn(T, H, dt=BF16), rn(2 * I, H, dt=BF16), rn(T, I, dt=BF16)))
    want = M.gated_ffn_forward(x, w, interleaved=inter)
    back = M.gated_ffn_backward(dh, x, w, interleaved=inter, need=("dx", "dw13", "h"))
    d = dense._FFN.pack(H, I, w.data_ptr(), 0, 0.0, 0.0, inter)
    h = Out((T, I), BF16, 16)
    run(L.nf4moe_gated_ffn_forward, d, x, T, h)
    h.check("h", want)
    n = L.nf4moe_gated_ffn_workspace_bytes(d, T)
    dx, dw, h, ws = Out((T, H), BF16, 16), Out((2 * I, H), BF16, 16), Out((T, I), BF16, 16), Out((n,), U8)
    run(L.nf4moe_gated_ffn_backward, d, dh, x, T, dx, dw, h, ws, n)
    dx.check("dx", back["dx"]), dw.check("dw13", back["dw13"]), h.check("h", back["h"]), ws.check("workspace")
    ws.t.fill_(255)      # NaN, whatever type is read
    run(L.nf4moe_gated_ffn_backward, d, dh, x, T, dx, dw, None, ws, n)
    dx.check("dx", back["dx"]), dw.check("dw13", back["dw13"])


@pytest.mark.parametrize("k", [0, 5])
@pytest.mark.parametrize("T,H,V", SIZES + [(4100, 16, 17001)])
def test_vocabulary_losses(T, H, V, k):
    rn = gen(T + V)
    g = torch.Generator(device=DEV).manual_seed(T)
    x, w = skewed(rn(T, H, dt=BF16)), skewed(rn(V, H, dt=BF16))
    ids = skewed(torch.randint(-V // 8 - 1, V, (T, k) if k else (T,), generator=g, device=DEV).to(I32))
    t, dloss, tau = skewed(rn(T, max(k, 1))), skewed(rn(T)), 1.5 if k else 1.0
    d = dense._HEAD.pack(H, V, w.data_ptr())
    n = L.nf4moe_vocab_workspace_bytes(d, T, k, 0)
    loss, lse, ws = Out((T,), F32, 4), Out((T,), F32, 4), Out((n,), U8)
    for fill in (0xA5, 0xFF):
        ws.t.fill_(fill)
        if k:
            want = M.vocab_distill_forward(x, w, ids, t, temperature=tau)
            q, logits = Out((T, k), F32, 4), Out((T, k), F32, 4)
            run(L.nf4moe_vocab_distill_forward, d, x, T, ids, t, 0, k, tau, loss, lse, q, logits, ws, n)
            q.check("q", want["q"]), logits.check("logits", want["logits"])
        else:
            want = dict(zip(("loss", "lse"), M.vocab_ce_forward(x, w, ids)))
            run(L.nf4moe_vocab_ce_forward, d, x, T, ids, loss, lse, ws, n)
        loss.check("loss", want["loss"]), lse.check("lse", want["lse"]), ws.check("workspace")
    n = L.nf4moe_vocab_workspace_bytes(d, T, k, 1)
    for need in (("dx", "dw"), ("dx",), ("dw",)):
        if k:
            back = M.vocab_distill_backward(dloss, x, w, ids, want["q"], want["logits"], want["lse"], temperature=tau, need=need)
        else:
            back = M.vocab_ce_backward(dloss, x, w, ids, want["lse"], need=need)
        dx, dw = Out((T, H), BF16, 16) if "dx" in need else None, Out((V, H), BF16, 16) if "dw" in need else None
        ws = Out((n,), U8)
        for fill in (0xA5, 0xFF):
            ws.t.fill_(fill)
            if k:
                run(L.nf4moe_vocab_distill_backward, d, dloss, x, T, ids, want["q"], want["logits"], want["lse"], k, tau, dx, dw, ws, n)
            else:
                run(L.nf4moe_vocab_ce_backward, d, dloss, x, T, ids, want["lse"], dx, dw, ws, n)
            if dx:
                dx.check("dx", back["dx"])
            if dw:
                dw.check("dw", back["dw"])
            ws.check("workspace")


@pytest.mark.parametrize("xdt", [0, 1])
@pytest.mark.parametrize("ydt", [0, 1])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 64), (9, 118), (4, 513), (3, 2049), (5, 4100), (2, 8193), (300, 65)])
def test_layer_norm(T, H, xdt, ydt):
    rn, dts = gen(T + H), (F32, BF16)
    x, dy, base, w, b = rn(T, H, dt=dts[xdt]), rn(T, H, dt=dts[ydt]), rn(T, H, dt=dts[xdt]), rn(H), rn(H)
    want = M.layer_norm_forward(x, w, b, out_dtype=dts[ydt])
    d = dense._LAYER_NORM.pack(H, xdt, ydt, w.data_ptr(), b.data_ptr(), 1e-5)
    y, mean, rstd = Out((T, H), dts[ydt], 4 - 2 * ydt), Out((T,), F32, 4), Out((T,), F32, 4)
    run(L.nf4moe_layer_norm_forward, d, x, T, y, mean, rstd)
    y.check("y", want["y"]), mean.check("mean", want["mean"]), rstd.check("rstd", want["rstd"])
    back = M.layer_norm_backward(dy, x, want["mean"], want["rstd"], w, dx_base=base)
    n = L.nf4moe_layer_norm_workspace_bytes(H, T)
    dx, dw, db, ws = Out((T, H), dts[xdt], 4 - 2 * xdt), Out((H,), F32, 4), Out((H,), F32, 4), Out((n,), U8)
    ws.t.fill_(255)
    run(L.nf4moe_layer_norm_backward, d, dy, x, want["mean"], want["rstd"], T, base, dx, dw, db, ws, n)
    dx.check("dx", back["dx"]), dw.check("dw", back["dw"]), db.check("db", back["db"]), ws.check("workspace")
