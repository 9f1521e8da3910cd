"""The dense operators where a rounding or a value that is not finite would show most: a mean loss, whose rows
all have the same gradient; rows sure of their label; rows far from zero; infinities and masked rows in the
forms of few rows. Bounds as in test_gpu_dense.py: u = 2^-24 and b = 2^-8 are half steps of fp32 and bf16."""
import pytest

import dense_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402
from test_gpu_dense import B, BF16, DEV, F32, I32, INF, NAN, U, gen, near  # noqa: E402


# ------------------------------------------------------------------ the gradient of a mean
def mean_case(T, V, k, H=256):
    """Rows unsure of their labels, P of a label all but -dloss."""
    rn = gen(T + V)
    g = torch.Generator(device=DEV).manual_seed(T)
    x, w = rn(T, H, dt=BF16), rn(V, H, std=H ** -0.5, dt=BF16)
    labels = torch.randint(0, V, (T,), generator=g, device=DEV).to(I32)
    return x, w, labels


def head_gradients(x, w, labels, dloss, k):
    """Through the cross entropy, or (k = 1) through the distillation from one sure entry."""
    if not k:
        return M.vocab_ce_backward(dloss, x, w, labels, M.vocab_ce_forward(x, w, labels)[1])
    ids = labels[:, None].contiguous()
    f = M.vocab_distill_forward(x, w, ids, torch.zeros(len(labels), 1, device=DEV))
    return M.vocab_distill_backward(dloss, x, w, ids, f["q"], f["logits"], f["lse"])


@pytest.mark.parametrize("k", [0, 1])
@pytest.mark.parametrize("T,V,rows", [(1020, 8003, 1020), (4080, 4001, 4080), (130, 3001, 127), (1000, 20001, 1019)])
def test_gradients_of_a_mean_loss(T, V, rows, k):
    """dloss is 1 / rows everywhere: no rounding of it may be every row's."""
    x, w, labels = mean_case(T, V, k)
    dloss = torch.full((T,), 1.0 / rows, device=DEV)
    out = head_gradients(x, w, labels, dloss, k)
    P = R.ce_P(dloss, x, w, labels)
    near(out["dx"], P @ w.double(), 2, "dx"), near(out["dw"], P.T @ x.double(), 2, "dw")


@pytest.mark.parametrize("k", [0, 1])
def test_gradients_of_a_mean_loss_behind_masked_rows(k):
    """The mean over the rows with a label; those before them, and rows of weight zero, hold anything."""
    T, V = 3000, 2003
    x, w, labels = mean_case(T, V, k)
    labels[:2100] = -100
    dloss = torch.full((T,), 1.0 / 1020, device=DEV)
    dloss[:2100] = torch.tensor([NAN, INF, 0.7], device=DEV).repeat(700)
    dloss[2100:2103] = 0.0
    out = head_gradients(x, w, labels, dloss, k)
    P = R.ce_P(dloss, x, w, labels)
    near(out["dx"], P @ w.double(), 2, "dx"), near(out["dw"], P.T @ x.double(), 2, "dw")
    assert not out["dx"][:2103].any()


@pytest.mark.parametrize("scale", [2.0 ** -120, 3.0 * 2.0 ** -131, 1.4e-45, 2.0 ** 90])
def test_gradients_of_far_scales(scale):
    """A mean's gradient in proportion to its dloss, whatever size that has; below fp32's normal numbers (and
    bf16's) products go to zero as they like, with nothing but small values."""
    x, w, labels = mean_case(200, 501, 0)
    one = head_gradients(x, w, labels, torch.ones(200, device=DEV), 0)
    out = head_gradients(x, w, labels, torch.full((200,), scale, device=DEV), 0)
    for n in out:
        want = one[n].double() * scale
        R.within(out[n], want, 2 * B * want.abs() + 2.0 ** -124, n)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_gradient_that_is_not_finite_stays_in_its_row(bad):
    x, w, labels = mean_case(150, 501, 0)
    dloss = torch.full((150,), 1.0 / 51, device=DEV)
    want = head_gradients(x, w, labels, dloss, 0)
    dloss[0] = bad
    out = head_gradients(x, w, labels, dloss, 0)
    assert torch.equal(out["dx"][1:], want["dx"][1:])
    assert not torch.isfinite(out["dx"][0]).any() and not torch.isfinite(out["dw"]).any()


@pytest.mark.parametrize("k", [0, 1])
def test_gradients_where_no_row_counts(k):
    x, w, labels = mean_case(100, 300, k)
    out = head_gradients(x, w, torch.full_like(labels, -100), torch.full((100,), NAN, device=DEV), k)
    assert not out["dx"].any() and not out["dw"].any()


# ------------------------------------------------------------------ rows sure of their label
@pytest.mark.parametrize("T,V", [(7, 1000), (30, 9001), (300, 1000), (2500, 301)])
def test_the_loss_of_a_sure_row(T, V):
    """Sums that are exact, logits up to 60, losses down to 0. exp2 of the largest term, the logarithm and the last
    operations are 8 u of 1 together. A sum of about 1 loses no more of a smaller term than the term, so of all
    of them the loss itself; nor than a u a step (300 + V / 512 of them)."""
    H = 64
    g = torch.Generator(device=DEV).manual_seed(T)
    w = torch.randint(-1, 2, (V, H), generator=g, device=DEV).to(BF16)
    labels = torch.randint(0, V, (T,), generator=g, device=DEV).to(I32)
    x = w[labels.long()] * (torch.randint(1, 9, (T, 1), generator=g, device=DEV) / 8).to(BF16)
    loss, lse = R.ce(x, w, labels)
    got, got_lse = M.vocab_ce_forward(x, w, labels)
    assert (loss < 1e-6).any() and (loss > 1e-3).any()
    bound = 8 * U + torch.minimum(loss, torch.full_like(loss, (300 + V / 512) * U)) + 4 * U * loss
    R.within(got, loss, bound, "loss")
    d = M.vocab_distill_forward(x, w, labels[:, None].contiguous(), torch.zeros(T, 1, device=DEV))
    R.within(d["loss"], loss, bound, "distillation from one entry")


# ------------------------------------------------------------------ layer norm far from zero
@pytest.mark.parametrize("T,H", [(5, 2880), (300, 2880), (700, 1000), (3, 129), (300, 6001), (260, 12000), (2, 16384)])
@pytest.mark.parametrize("value", [1000.1, 10000.1, -0.3])
def test_layer_norm_of_constant_rows(T, H, value):
    """The first sum's error, e = s |value| with s = (24 + H / 64) u, is taken out to s of itself: the mean is the
    value, y no more than s e rstd, and the variance's part of rstd s e^2 rstd^2."""
    x = torch.full((T, H), value, device=DEV)
    got = M.layer_norm_forward(x, eps=1e-5)
    v, s, r = float(x[0, 0]), (24 + H / 64) * U, 1e-5 ** -0.5
    e = s * abs(v)
    assert (got["mean"] == v).all()
    assert float(got["y"].abs().max()) <= s * e * r + U * e * r
    assert float((got["rstd"].double() / r - 1).abs().max()) <= 2 * s * e * e * r * r + 8 * U


@pytest.mark.parametrize("T,H", [(5, 2880), (300, 2880), (50, 1000), (300, 6001)])
@pytest.mark.parametrize("shift,spread", [(1000.0, 1.0), (10000.0, 0.01), (-3.0, 1.0)])
def test_layer_norm_of_rows_far_from_zero(T, H, shift, spread):
    """x - mean is exact or off by u of itself, the mean's error e comes out to s of itself and of the spread."""
    x = gen(3)(T, H, std=spread) + shift
    y, mean, rstd = R.layer_norm(x, None, None, 0.0)
    got = M.layer_norm_forward(x, eps=0.0)
    s = (24 + H / 64) * U
    e = s * x.double().abs().mean(1)
    R.within(got["mean"], mean, U * mean.abs() + s * (e + 1 / rstd), "mean")
    rel = 2 * s * (1 + (e * rstd) ** 2) + 8 * U          # of the variance, e^2 of the first mean in it
    R.within(got["rstd"], rstd, rstd * rel, "rstd")
    R.within(got["y"], y, (s * (e * rstd + 1) + 2 * U)[:, None] + y.abs() * (rel + 4 * U)[:, None], "y")


@pytest.mark.parametrize("fill", [NAN, INF, -INF])
@pytest.mark.parametrize("T", [4, 300])
def test_layer_norm_not_finite_stays_in_its_row(T, fill):
    x = gen(4)(T, 1000)
    want = M.layer_norm_forward(x)
    x[2, 7] = fill
    got = M.layer_norm_forward(x)
    rows = torch.arange(T, device=DEV) != 2
    for n in got:
        assert torch.equal(got[n][rows], want[n][rows])
    assert torch.isnan(got["y"][2]).all() and torch.isnan(got["rstd"][2]) and not torch.isfinite(got["mean"][2])


# ------------------------------------------------------------------ the forms of few rows
def kinds(t):
    """0 finite, 1 and -1 infinite, 2 NaN."""
    return torch.where(torch.isnan(t), 2.0, torch.where(torch.isinf(t), torch.sign(t.float()), 0.0))


@pytest.mark.parametrize("glu,inter", [(0, 0), (1, 1)])
@pytest.mark.parametrize("T", [1, 5, 40, 64])
def test_an_infinite_gradient_stays_infinite(T, glu, inter):
    """dh of infinity, and one past bf16's largest value through the slope: what is not finite is what it is in a
    longer batch, whose further rows have no gradient."""
    H, I = 128, 72
    rn = gen(T)
    x, w = rn(65, H, dt=BF16), rn(2 * I, H, std=2.0 * H ** -0.5, dt=BF16)
    how = dict(glu=glu, alpha=1.702, limit=7.0, interleaved=inter)
    slopes = R.ffn(x, w, glu, 1.702, 7.0, inter)[3:]
    assert (slopes[0][0].abs() > 1.1).any()
    for value, col in ((INF, 7), (-INF, 9), (3.3e38, int(slopes[0][0].abs().argmax()))):
        dh = torch.zeros(65, I, device=DEV, dtype=BF16)
        dh[:T] = rn(T, I, std=0.3)
        dh[0, col] = value
        want = M.gated_ffn_backward(dh, x, w, **how)
        got = M.gated_ffn_backward(dh[:T].contiguous(), x[:T].contiguous(), w, **how)
        assert torch.equal(kinds(got["dx"]), kinds(want["dx"][:T])) and torch.equal(kinds(got["dw13"]), kinds(want["dw13"]))
        assert torch.isinf(got["dw13"]).any() and torch.isinf(got["dx"][0]).any()
        assert torch.isfinite(got["dx"][1:]).all()


@pytest.mark.parametrize("k", [0, 1])
@pytest.mark.parametrize("T", [1, 5, 40, 64])
def test_an_infinite_loss_gradient_stays_infinite(T, k):
    x, w, labels = mean_case(65, 601, k, H=128)
    on = torch.arange(65, device=DEV) < T
    labels = torch.where(on, labels, -100).to(I32)
    for value in (INF, -INF):
        dloss = torch.full((65,), 0.1, device=DEV)
        dloss[0] = value
        want = head_gradients(x, w, labels, dloss, k)
        got = head_gradients(x[:T].contiguous(), w, labels[:T].contiguous(), dloss[:T].contiguous(), k)
        assert torch.equal(kinds(got["dw"]), kinds(want["dw"])) and torch.isinf(got["dw"]).all()
        assert not torch.isfinite(got["dx"][0]).any() and torch.isfinite(got["dx"][1:]).all()
    dloss[0] = 3.4e38          # P of the label is past bf16's largest value
    got = head_gradients(x[:T].contiguous(), w, labels[:T].contiguous(), dloss[:T].contiguous(), k)
    assert not torch.isnan(got["dx"]).any() and not torch.isnan(got["dw"]).any()


@pytest.mark.parametrize("fill", [NAN, INF, -INF, 3.3e38])
@pytest.mark.parametrize("T", [2, 17, 40, 64])
def test_few_rows_without_a_target_count_for_nothing(T, fill):
    """Whatever x, dloss and the teacher hold in a masked row or entry."""
    V = 3001
    x, w, labels = mean_case(T, V, 0, H=128)
    labels[::2] = torch.tensor([-100, V], device=DEV, dtype=I32).repeat(T)[:len(labels[::2])]
    dloss = gen(T)(T)
    dead = (labels < 0) | (labels >= V)
    zero = lambda v: torch.where(dead if v.dim() == 1 else dead[:, None], torch.zeros_like(v), v)  # noqa: E731
    put = lambda v: torch.where(dead if v.dim() == 1 else dead[:, None], torch.full_like(v, fill), v)  # noqa: E731
    loss, lse = M.vocab_ce_forward(zero(x), w, labels)
    loss2, lse2 = M.vocab_ce_forward(put(x), w, labels)
    assert torch.equal(loss, loss2) and torch.equal(lse[~dead], lse2[~dead])
    a = M.vocab_ce_backward(zero(dloss), zero(x), w, labels, zero(lse))
    b = M.vocab_ce_backward(put(dloss), put(x), w, labels, put(lse2))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"]) and torch.isfinite(b["dw"]).all()
    assert not b["dx"][dead].any()
    ids = torch.stack([labels, torch.full_like(labels, -1), (labels + 1) % V], 1)
    ids = torch.where(dead[:, None], torch.full_like(ids, -7), ids).contiguous()
    outside = (ids < 0) | (ids >= V)
    t = gen(5)(T, 3)
    t1, t2 = torch.where(outside, 0.0, t), torch.where(outside, fill, t)
    p, r = M.vocab_distill_forward(zero(x), w, ids, t1), M.vocab_distill_forward(put(x), w, ids, t2)
    assert all(torch.equal(p[n], r[n]) for n in p)
    a = M.vocab_distill_backward(zero(dloss), zero(x), w, ids, p["q"], p["logits"], p["lse"])
    b = M.vocab_distill_backward(put(dloss), put(x), w, ids, r["q"], r["logits"], r["lse"])
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"]) and torch.isfinite(b["dw"]).all()
