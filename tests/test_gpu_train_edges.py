"""Edges of the fine-tuning operators on the GPU: unused adapters, rows without one,
and gates far out on the tails of their function."""
import numpy as np
import pytest

import train_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def to_np(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ adapters
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Rn,rank,src", [(1, 8, "bf16"), (40, 16, M.CKPT_MXINT8), (9000, 24, "bf16"), (9000, 72, M.CKPT_MXFP8)])
def test_gradients_of_an_adapter_without_rows_are_zero(Rn, rank, src, bad):
    """Whatever its scale holds (a slot not in use); the others' gradients are what they are without it."""
    g = torch.Generator(device=DEV).manual_seed(Rn + rank)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    Ln, K, N = 7, 96, 136
    used = torch.tensor([1, 4, -1, Ln, 5], device=DEV)
    ids = used[torch.randint(0, 5, (Rn,), generator=g, device=DEV)].int()
    ids[0] = 4
    unused = [l for l in range(Ln) if not (ids == l).any()]
    assert {0, 2, 3, 6} <= set(unused)
    x, A, B = rn(Rn, K).to(BF16), rn(Ln, rank, K).to(BF16), rn(Ln, N, rank).to(BF16)
    dy, scale = rn(Rn, N).to(BF16), rn(Ln).abs() + 0.5
    held = x if src == "bf16" else M.ckpt8_quantize(x, src)
    _, t = M.adapter_forward(x, A, B, ids, scale=scale, return_t=True)
    want = M.adapter_backward(dy, held, t, A, B, ids, scale=scale)
    wild = scale.clone()
    wild[unused] = bad
    got = M.adapter_backward(dy, held, t, A, B, ids, scale=wild)
    assert all(torch.equal(got[k], want[k]) for k in want)
    for l in unused:
        assert torch.count_nonzero(got["dA"][l]) == 0 and torch.count_nonzero(got["dB"][l]) == 0
    assert torch.equal(M.adapter_forward(x, A, B, ids, scale=wild), M.adapter_forward(x, A, B, ids, scale=scale))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Rn,rank", [(9, 8), (30000, 8), (30000, 16), (12000, 24), (12000, 72)])
def test_rows_without_an_adapter_take_base_as_it_is(Rn, rank, dtype):
    """Its bits: a negative zero keeps its sign, in the one-launch form (9 rows) and in the grouped kernels."""
    g = torch.Generator(device=DEV).manual_seed(Rn + rank)
    Ln, K, N = 3, 520, 264
    ids = torch.randint(-2, Ln + 2, (Rn,), generator=g, device=DEV).int()
    ids[:3] = torch.tensor([-1, 0, Ln], device=DEV)
    x = torch.randn(Rn, K, generator=g, device=DEV).to(BF16)
    A = torch.randn(Ln, rank, K, generator=g, device=DEV).to(BF16)
    B = torch.randn(Ln, N, rank, generator=g, device=DEV).to(BF16)
    base = torch.randn(Rn, N, generator=g, device=DEV)
    fi = torch.finfo(dtype)
    base[:, :6] = torch.tensor([-0.0, 0.0, float("inf"), float("-inf"), fi.max, fi.tiny / 4], device=DEV)
    base = base.to(dtype)
    none = (ids < 0) | (ids >= Ln)
    word = torch.int16 if dtype is BF16 else torch.int32
    out = M.adapter_forward(x, A, B, ids, base=base)
    assert torch.equal(out[none].view(word), base[none].view(word))
    dx_base = base.repeat(1, 2)[:, :K].contiguous()
    back = M.adapter_backward(torch.ones(Rn, N, device=DEV, dtype=BF16), None, None, A, B, ids, dx_base=dx_base, need=("dx",))
    assert torch.equal(back["dx"][none].view(word), dx_base[none].view(word))


# ------------------------------------------------------------------ gates on their tails
TAILS = [0.0, 0.5, 2.5, 4.0, 6.0, 8.0, 10.0, 14.0, 17.0, 20.0, 40.0, 60.0, 80.0, 100.0, float("inf")]
TAILS = np.array(TAILS + [-v for v in TAILS])


def tail_phi(v, fn):
    """phi and its slope in 64 bits without cancellation: sigma(v), sigma(v) sigma(-v); tanh(v), 4 sigma(2 v) sigma(-2 v)."""
    s = R._sigma
    return (s(v), s(v) * s(-v)) if fn == 1 else (np.tanh(v), 4 * s(2 * v) * s(-2 * v))


def tail_error(v, fn):
    """Relative error of phi, and of the slope, evaluated in fp32: a sigma of argument a is within (|a| + 8) 2^-23 of
    itself (the exponent's argument is rounded, |a| 1.5 U, then exp2, one addition and a reciprocal, 5 U), the library's
    tanh within 2 units in the last place; a slope is two sigmas and their product."""
    a = np.minimum(np.abs(v) * (1 if fn == 1 else 2), 200.0)
    return (a + 8) * 2 * U if fn == 1 else np.full_like(a, 4 * U), 2 * (a + 8) * 2 * U + 2 * U


@pytest.mark.parametrize("fn", [M.GATE_SIGMOID, M.GATE_TANH])
@pytest.mark.parametrize("kind", ["channel", "row", "full"])
@pytest.mark.parametrize("post", [False, True])
def test_gates_on_their_tails(fn, kind, post):
    """x' and dgate where the gate saturates: phi to its last bits, and a slope that falls like exp(-|v|) (exp(-2 |v|)), not 0.

    x = 0 and no pre norm, so x' = alpha phi z, and g = dx' as it is given. Below 2^-126 the hardware's exp2 and
    reciprocal may give 0: 2^-126 of a sigma, 4 of them in tanh's slope, is allowed on top of the relative error."""
    n = len(TAILS)
    T, H = (n, 9) if kind == "row" else (5, 2 * n)
    g = torch.Generator(device=DEV).manual_seed(7 * fn + post)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    v = dict(channel=np.tile(TAILS, 2), row=TAILS[:, None], full=np.tile(TAILS, (5, 2)))[kind]
    gate = torch.from_numpy(v.astype(np.float32)).to(DEV)
    x, f, dx = torch.zeros(T, H, device=DEV), rn(T, H).to(BF16), rn(T, H)
    w_post = 1 + 0.2 * rn(H) if post else None
    kw = dict(w_post=w_post, gate=gate, gate_fn=fn, alpha=0.625)
    got = M.block_norm_forward(x, f, eps=1e-6, **kw)
    back = M.block_norm_backward(dx, None, got["x"], f, rstd_post=got["rstd_post"], **kw)
    v = to_np(gate)
    phi, slope = tail_phi(v, fn)
    ep, es = tail_error(v, fn)
    z = to_np(f)
    if post:
        z = z * to_np(got["rstd_post"])[:, None] * to_np(w_post)
    tiny = 2.0 ** -123
    # two products of z (rstd, w_post), then phi and alpha: 4 U more
    R.within(to_np(got["x"]), 0.625 * phi * z, 0.625 * np.abs(z) * (np.abs(phi) * (ep + 6 * U) + tiny), "x'")
    term = 0.625 * to_np(dx) * z
    ref, mag = slope * term, np.abs(slope * term) * (es + 8 * U) + np.abs(term) * tiny
    if kind != "full":
        axis = 0 if kind == "channel" else 1
        keep = axis == 1
        # the terms' sum in fp32: H = 9 or T = 5 of them, the lanes, slots and workgroups that hold none add zeros
        ref, mag = ref.sum(axis, keepdims=keep), mag.sum(axis, keepdims=keep) + 16 * U * np.abs(slope * term).sum(axis, keepdims=keep)
    R.within(to_np(back["dgate"]), ref, mag, "dgate")
    if fn == M.GATE_TANH:                       # not lost: the slope at 10 is 8.2e-9
        at = back["dgate"].cpu().numpy()[..., 6:7] if kind != "row" else back["dgate"].cpu().numpy()[6:7]
        assert np.all(at != 0)


def test_a_gate_that_is_not_a_number_stays_its_own():
    T, H = 4, 24
    f, dx = torch.randn(T, H, device=DEV).to(BF16), torch.randn(T, H, device=DEV)
    for fn in (M.GATE_IDENTITY, M.GATE_SIGMOID, M.GATE_TANH):
        gate = torch.randn(T, H, device=DEV)
        gate[2, 5] = float("nan")
        out = M.block_norm_forward(torch.zeros(T, H, device=DEV), f, gate=gate, gate_fn=fn)
        back = M.block_norm_backward(dx, None, out["x"], f, gate=gate, gate_fn=fn)
        one = torch.zeros(T, H, dtype=torch.bool, device=DEV)
        one[2, 5] = True
        assert torch.equal(torch.isnan(out["x"]), one) and torch.equal(torch.isnan(back["df"]), one)
        assert torch.equal(torch.isnan(back["dgate"]), one if fn else torch.zeros_like(one))


# ------------------------------------------------------------------ the widest rows of the gated activation
@pytest.mark.parametrize("inter", [0, 1])
def test_the_widest_row_of_the_gated_activation(inter):
    """2^30 pairs in one row, a pattern of 2^16 repeated: every repeat gives what a row of one repeat gives."""
    P, n = 1 << 16, 1 << 14
    g = torch.Generator(device=DEV).manual_seed(3)
    gu1, dh1 = torch.randn(1, 2 * P, generator=g, device=DEV).to(BF16), torch.randn(1, P, generator=g, device=DEV).to(BF16)
    h1, ck1 = M.glu_forward(gu1, interleaved=inter, ckpt=M.CKPT_MXFP8)
    b1 = M.glu_backward(dh1, ck1, interleaved=inter)
    gu = gu1.repeat(1, n) if inter else torch.cat([gu1[:, :P].repeat(1, n), gu1[:, P:].repeat(1, n)], 1)
    h, ck = M.glu_forward(gu, interleaved=inter, ckpt=M.CKPT_MXFP8)
    del gu

    def same(wide, one, halves):
        if halves and not inter:            # gate columns, then up columns
            k = one.shape[1] // 2
            w = wide.view(2, n, k)
            return all(bool((w[i] == one[0, i * k:(i + 1) * k]).all()) for i in range(2))
        return bool((wide.view(n, -1) == one).all())
    assert same(h, h1, False) and same(ck.codes, ck1.codes, True) and same(ck.scale, ck1.scale, True)
    del h
    b = M.glu_backward(dh1.repeat(1, n), ck, interleaved=inter)
    assert same(b["dgu"], b1["dgu"], True) and same(b["h"], b1["h"], False)


def test_a_small_slope_meets_large_gradients():
    """The slope enters its product first: a gradient that fits is not lost to an infinity on the way."""
    T, H = 3, 16
    f, dx = torch.full((T, H), 1e30, device=DEV).to(BF16), torch.full((T, H), 1e10, device=DEV)
    gate = torch.full((T, H), 20.0, device=DEV)
    gate[1] = -20.0
    out = M.block_norm_forward(torch.zeros(T, H, device=DEV), f, gate=gate, gate_fn=M.GATE_TANH)
    got = to_np(M.block_norm_backward(dx, None, out["x"], f, gate=gate, gate_fn=M.GATE_TANH)["dgate"])
    ref = tail_phi(to_np(gate), 2)[1] * to_np(dx) * to_np(f)
    R.within(got, ref, np.abs(ref) * (tail_error(to_np(gate), 2)[1] + 8 * U), "dgate")
