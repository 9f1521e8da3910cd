"""What the fine-tuning calls write: their outputs and workspaces to the last byte and
nothing beside them. Through the C ABI, each array with marked bytes before and behind it
and no alignment beyond what the call asks for; the values are the binding's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402
from bit_quantized_moe_expert_amd import train  # noqa: E402

DEV = "cuda"
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
L = M.lib()
PAD, MARK = 16384, 0xA5


class Out:
    """An array of this shape with PAD marked bytes on both sides, `skew` bytes past a 256-byte boundary."""

    def __init__(self, shape, dtype, skew=0):
        self.n = torch.Size(shape).numel() * dtype.itemsize
        self.buf = torch.full((2 * PAD + self.n + 512,), MARK, dtype=U8, device=DEV)
        self.off = PAD + (-(self.buf.data_ptr() + PAD)) % 256 + skew
        self.ptr = self.buf.data_ptr() + self.off
        self.t = self.buf[self.off:self.off + self.n]
        if self.n and dtype is not U8:
            self.t = self.t.view(dtype)
        self.t = self.t.view(shape) if dtype is U8 or self.n else torch.empty(shape, dtype=dtype, device=DEV)

    def check(self, name, want=None):
        assert (self.buf[:self.off] == MARK).all(), f"{name}: written before"
        assert (self.buf[self.off + self.n:] == MARK).all(), f"{name}: written behind"
        if want is not None:
            assert torch.equal(self.t, want), name


def run(fn, *args):
    M._check(fn(*[a.ptr if isinstance(a, Out) else a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args],
                torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, dt=F32: torch.randn(*s, generator=g, device=DEV).to(dt)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 2880), (67, 160)])
def test_checkpoints(rows, K, fmt, dt):
    x = gen(rows + K)(rows, K, dt=(F32, BF16)[dt])
    want = M.ckpt8_quantize(x, fmt)
    codes, scale = Out((rows, K), U8, 1), Out((rows, K // 32), U8, 1)
    run(L.nf4moe_ckpt8_quantize, fmt, x, dt, rows, K, codes, scale)
    codes.check("codes", want.codes), scale.check("scale", want.scale)
    out = Out((rows, K), x.dtype, x.element_size())
    run(L.nf4moe_ckpt8_dequantize, fmt, want.codes, want.scale, rows, K, out, dt)
    out.check("out", M.ckpt8_dequantize(want, x.dtype))


@pytest.mark.parametrize("src", [0, 1, 2, 3])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("R,I", [(1, 32), (5, 96), (7, 2880), (600, 64)])
def test_gated_activation(R, I, inter, src):
    rn = gen(R + I + src)
    gu, dh, w = rn(R, 2 * I, dt=BF16 if src == 1 else F32), rn(R, I, dt=BF16 if src & 1 else F32), rn(R)
    fmt = max(src - 2, 0)
    h0, ck = M.glu_forward(gu, interleaved=inter, ckpt=fmt)
    h, codes, scale = Out((R, I), BF16, 2), Out((R, 2 * I), U8, 1), Out((R, I // 16), U8, 1)
    run(L.nf4moe_glu_forward, gu, int(src == 1), R, I, 0, 0.0, 0.0, inter, h, fmt, codes, scale)
    h.check("h", h0), codes.check("codes", ck.codes), scale.check("scale", ck.scale)
    held = ck if src > 1 else gu
    want = M.glu_backward(dh, held, interleaved=inter, row_w=w)
    dgu, h, drow = Out((R, 2 * I), BF16, 2), Out((R, I), BF16, 2), Out((R,), F32, 4)
    run(L.nf4moe_glu_backward, dh, int(dh.dtype is BF16), src, ck.codes if src > 1 else gu, ck.scale if src > 1 else None, R, I, 0,
        0.0, 0.0, inter, w, dgu, h, drow)
    dgu.check("dgu", want["dgu"]), h.check("h", want["h"]), drow.check("drow_w", want["drow_w"])


@pytest.mark.parametrize("kind", [1, 2, 3])
@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("T,H", [(5, h) for h in range(1, 16)] + [(1, 1), (9, 521), (2, 2049), (3, 4094), (2, 8198), (1, 16383), (700, 77)])
def test_block_norm(T, H, dt, kind):
    rn, xt = gen(T * 31 + H + kind), (F32, BF16)[dt]
    x, f, dxn, dy = rn(T, H, dt=xt), rn(T, H, dt=BF16), rn(T, H, dt=xt), rn(T, H, dt=BF16)
    shape = (None, (H,), (T, 1), (T, H))[kind]
    if H == 1 and kind == 3:
        kind = 2                                   # the same gate
    kw = dict(w_post=rn(H), w_pre=rn(H), gate=rn(*shape), gate_fn=kind % 3, alpha=0.5)
    want = M.block_norm_forward(x, f, eps=1e-6, **kw)
    desc = train._BLOCK_NORM.pack(H, dt, kw["w_post"].data_ptr(), kw["w_pre"].data_ptr(), kw["gate"].data_ptr(), kind, 0, kind % 3, 0.5,
                                  1e-6)
    e = x.element_size()
    xn, y, rp, r = Out((T, H), xt, e), Out((T, H), BF16, 2), Out((T,), F32, 4), Out((T,), F32, 4)
    run(L.nf4moe_block_norm_forward, desc, x, f, T, xn, y, rp, r)
    for o, k in ((xn, "x"), (y, "y"), (rp, "rstd_post"), (r, "rstd_pre")):
        o.check(k, want[k])
    back = M.block_norm_backward(dxn, dy, want["x"], f, rstd_post=want["rstd_post"], rstd_pre=want["rstd_pre"], **kw)
    need = L.nf4moe_block_norm_workspace_bytes(H, T)
    dx, df, dg, dwp, dwr, ws = (Out((T, H), xt, e), Out((T, H), BF16, 2), Out(shape, F32, 4), Out((H,), F32, 4), Out((H,), F32, 4),
                                Out((need,), U8))
    run(L.nf4moe_block_norm_backward, desc, dxn, dy, want["x"], f, want["rstd_post"], want["rstd_pre"], T, dx, df, dg, dwp, dwr, ws, need)
    for o, k in ((dx, "dx"), (df, "df"), (dg, "dgate"), (dwp, "dw_post"), (dwr, "dw_pre")):
        o.check(k, back[k])
    ws.check("workspace")


ROWS = [(1, 1, 8, 8, 8), (5, 3, 32, 8, 8), (37, 3, 96, 264, 24), (33, 4, 264, 1032, 72), (70, 2, 64, 40, 128),      # one launch
        (9000, 3, 160, 40, 24), (5000, 5, 1056, 264, 72), (24000, 3, 264, 1032, 8), (9000, 40, 544, 136, 16),       # grouped
        (1100, 3, 3200, 72, 128), (66, 300, 96, 40, 40)]


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("R,Ln,K,N,rank", ROWS)
def test_adapters(R, Ln, K, N, rank, dt, planned):
    rn, yt = gen(R + K + rank), (F32, BF16)[dt]
    ids = torch.randint(-1, Ln, (R,), generator=torch.Generator(device=DEV).manual_seed(R), device=DEV).int()
    x, A, B, scale = rn(R, K, dt=BF16), rn(Ln, rank, K, dt=BF16), rn(Ln, N, rank, dt=BF16), rn(Ln)
    base, dy, dxb = rn(R, N, dt=yt), rn(R, N, dt=BF16), rn(R, K, dt=yt)
    desc = train._ADAPTERS.pack(Ln, rank, K, N, A.data_ptr(), B.data_ptr(), scale.data_ptr())
    plan, pb = None, 0
    if planned:
        pb = L.nf4moe_adapter_plan_bytes(R, Ln)
        plan = Out((pb,), U8)
        run(L.nf4moe_adapter_plan, ids, R, Ln, plan, pb)
        plan.check("plan")
    want, t0 = M.adapter_forward(x, A, B, ids, base=base, scale=scale, return_t=True)
    nb = L.nf4moe_adapter_workspace_bytes(desc, R, 0)
    out, t, ws = Out((R, N), yt, yt.itemsize), Out((R, rank), F32, 16), Out((nb,), U8)
    run(L.nf4moe_adapter_forward, desc, x, R, None, ids, plan, pb, R, base, out, dt, t, ws if nb else None, nb)
    out.check("out", want), t.check("t", t0), ws.check("workspace")
    nb = L.nf4moe_adapter_workspace_bytes(desc, R, 1)
    for src in (1, 2, 3) if K % 32 == 0 else (1,):
        held = x if src == 1 else M.ckpt8_quantize(x, src - 2)
        back = M.adapter_backward(dy, held, t0, A, B, ids, scale=scale, dx_base=dxb)
        dx, dA, dB, ws = Out((R, K), yt, yt.itemsize), Out((Ln, rank, K), F32, 16), Out((Ln, N, rank), F32, 16), Out((nb,), U8)
        run(L.nf4moe_adapter_backward, desc, dy, src, x if src == 1 else held.codes, None if src == 1 else held.scale, R, None, t0, ids,
            plan, pb, R, dxb, dx, dt, dA, dB, ws, nb)
        dx.check("dx", back["dx"]), dA.check("dA", back["dA"]), dB.check("dB", back["dB"]), ws.check("workspace")
        if planned:
            plan.check("plan")
