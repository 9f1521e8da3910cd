"""The dense operators on the GPU against 64-bit references.

Bounds, elementwise, from the arithmetic. u = 2^-24 (fp32), b = 2^-8 (bf16), half a step
each. A product of K terms summed in fp32 in any order is off by at most 2 K u sum |x y|
(a rounding for each product and each sum, twice for the matrix cores' own order and
rounding); the hardware's exp2 and reciprocal are good to 1 ulp, some 8 u through the
formulas here. What is rounded to bf16 on its way into a second product carries b of
itself, and the output its own b."""
import pytest

import dense_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402

DEV = "cuda"
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
U, B = 2.0 ** -24, 2.0 ** -8
INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, std=1.0, dt=F32: (torch.randn(*s, generator=g, device=DEV) * std).to(dt)


def near(got, ref, roundings, what):
    """In the 2-norm a rounding to bf16 is b / sqrt(3) at most where values spread over a binade, 0.6 b with a
    little room, and two of them that do not know of each other sqrt(2) times that: 0.85 b. Of many values only: a
    few that lie at the lower end of a binade come near b, and few sums may cancel (elementwise bounds hold for these)."""
    if ref.numel() >= 4096:
        assert R.off(got, ref) < (0.6, 0.85)[roundings - 1] * B, what


def few(got, ref, T, what):
    """Up to 64 rows nothing is rounded to bf16 but the output: b of the norm at most, whatever the values."""
    if T <= 64 and ref.norm() > 0:
        assert R.off(got, ref) < 1.02 * B, what


def product_bound(x, w):
    """How far fp32 sums of x w^T may be off."""
    return 2 * x.shape[1] * U * (x.double().abs() @ w.double().abs().T)


# ------------------------------------------------------------------ gated feed-forward
FFN_SIZES = [(1, 8, 8), (1, 2048, 1024), (2, 72, 2056), (3, 264, 40), (16, 1024, 264), (17, 128, 72), (31, 64, 136),
             (64, 200, 72), (65, 128, 520), (131, 2048, 768), (257, 520, 264), (1000, 192, 2048), (4099, 64, 1032),
             (8193, 72, 136), (1, 72, 2080), (7, 2048, 8200), (16, 1024, 2056), (17, 40, 8232), (32, 2056, 8192), (4, 2048, 8192)]


def ffn_case(T, H, I, glu, seed=0):
    rn = gen(seed + T + H + I)
    x, w = rn(T, H, dt=BF16), rn(2 * I, H, std=2.0 * H ** -0.5 * (3 if glu else 1), dt=BF16)
    return x, w, rn(T, I, std=0.3, dt=BF16)


def ffn_bounds(x, w, dh, kind, inter):
    """(bound of h, of dg, of du) before their roundings, from those of g and u."""
    g, u, h, by_g, by_u = R.ffn(x, w, kind, 1.702, 7.0, inter)
    wg, wu = R.split(w, inter)
    eg, eu = product_bound(x, wg), product_bound(x, wu)
    # |dh/dg| <= 1.1 |u + 1| (the silu's slope is at most 1.1, alpha's folded in 1.702 * 0.28 + 1), |d2h/dg2| <= alpha |u + 1|
    a = 1.702 if kind else 1.0
    uu = u.abs() + 1
    steep = 1.5 * uu * eg + (g.abs() + 1) * eu
    eh = steep + 16 * U * (g.abs() + 1) * uu
    edg = dh.double().abs() * (2 * a * uu * eg + 1.5 * eu + 16 * U * (g.abs() + 1) * uu)
    edu = dh.double().abs() * (1.5 * eg + 16 * U * (g.abs() + 1))
    if kind:   # a value within its own error of the limit may fall on either side: a whole slope
        near_g, near_u = (g - 7.0).abs() <= eg, (u.abs() - 7.0).abs() <= eu
        edg = edg + near_g * dh.double().abs() * 9 * 1.5
        edu = edu + near_u * dh.double().abs() * 8
    return h, eh, edg, edu


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,H,I", FFN_SIZES)
def test_gated_ffn(T, H, I, kind, inter):
    x, w, dh = ffn_case(T, H, I, kind)
    kw = dict(glu=kind, alpha=1.702, limit=7.0, interleaved=inter)
    h, eh, edg, edu = ffn_bounds(x, w, dh, kind, inter)
    got = M.gated_ffn_forward(x, w, **kw)
    R.within(got, h, B * h.abs() + (1 + B) * eh, "h")
    dg, du, dx, dw = R.ffn_grad(dh, x, w, kind, 1.702, 7.0, inter)
    out = M.gated_ffn_backward(dh, x, w, need=("dx", "dw13", "h"), **kw)
    R.within(out["h"], h, B * h.abs() + (1 + B) * eh, "h again")
    # dgu as an operand: its own error and its rounding, then the sums of the second product
    rg, ru = edg + B * (dg.abs() + edg), edu + B * (du.abs() + edu)
    wg, wu = (v.double().abs() for v in R.split(w, inter))
    xa = x.double().abs()
    ex = rg @ wg + ru @ wu + 4 * I * U * ((dg.abs() + rg) @ wg + (du.abs() + ru) @ wu)
    R.within(out["dx"], dx, B * dx.abs() + (1 + B) * ex, "dx")
    ew = R.join((rg + 2 * T * U * (dg.abs() + rg)).T @ xa, (ru + 2 * T * U * (du.abs() + ru)).T @ xa, inter)
    R.within(out["dw13"], dw, B * dw.abs() + (1 + B) * ew, "dw13")
    near(got, h, 1, "h"), near(out["dx"], dx, 2, "dx"), near(out["dw13"], dw, 2, "dw13")
    few(out["dx"], dx, T, "dx"), few(out["dw13"], dw, T, "dw13")
    again = M.gated_ffn_backward(dh, x, w, need=("dx", "dw13", "h"), **kw)
    assert all(torch.equal(out[n], again[n]) for n in out)
    for n, ref, e in (("dx", dx, ex), ("dw13", dw, ew)):    # alone: the sums may be cut differently
        one = M.gated_ffn_backward(dh, x, w, need=(n,), **kw)
        assert list(one) == [n]
        R.within(one[n], ref, B * ref.abs() + (1 + B) * e, n + " alone")


def test_gated_ffn_without_rows():
    rn = gen(1)
    x, w = rn(0, 64, dt=BF16), rn(48, 64, dt=BF16)
    assert M.gated_ffn_forward(x, w).shape == (0, 24)
    out = M.gated_ffn_backward(rn(0, 24, dt=BF16), x, w, need=("dx", "dw13", "h"))
    assert out["dx"].shape == (0, 64) and not out["dw13"].any() and out["h"].shape == (0, 24)


def test_gated_ffn_into_a_given_tensor_and_from_views():
    x, w, _ = ffn_case(40, 64, 48, 0)
    want = M.gated_ffn_forward(x, w)
    held = torch.full((3, 40, 48), 7.0, device=DEV, dtype=BF16)
    assert M.gated_ffn_forward(x, w, out=held[1]) is not None
    assert torch.equal(held[1], want) and (held[0] == 7).all() and (held[2] == 7).all()
    assert torch.equal(M.gated_ffn_forward(torch.cat([x, x])[40:], w), want)


def test_gated_ffn_not_finite_stays_in_its_row():
    x, w, _ = ffn_case(200, 128, 64, 0)
    want = M.gated_ffn_forward(x, w)
    x[77, 5] = NAN
    got = M.gated_ffn_forward(x, w)
    rows = torch.arange(200, device=DEV) != 77
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[77]).all()


@pytest.mark.parametrize("T", [5, 40, 200])
@pytest.mark.parametrize("inter", [0, 1])
def test_clamped_ffn_shows_a_nan(T, inter):
    """A NaN passes through the clamps, forward and backward, to its row and to the weights' gradient."""
    x, w, dh = ffn_case(T, 128, 64, 1)
    how = dict(glu=1, alpha=1.702, limit=7.0, interleaved=inter)
    want = M.gated_ffn_forward(x, w, **how)
    grad = M.gated_ffn_backward(dh, x, w, need=("dx", "dw13", "h"), **how)
    x[3, 5] = NAN
    got = M.gated_ffn_forward(x, w, **how)
    out = M.gated_ffn_backward(dh, x, w, need=("dx", "dw13", "h"), **how)
    rows = torch.arange(T, device=DEV) != 3
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[3]).all()
    assert torch.equal(out["h"][rows], grad["h"][rows]) and torch.isnan(out["h"][3]).all()
    assert torch.equal(out["dx"][rows], grad["dx"][rows]) and torch.isnan(out["dx"][3]).all() and torch.isnan(out["dw13"]).all()


# ------------------------------------------------------------------ losses of a head
HEAD_SIZES = [(1, 8, 1), (1, 64, 5), (2, 2048, 3001), (17, 2048, 3001), (33, 72, 777), (64, 128, 64), (129, 264, 4099),
              (300, 128, 20001), (515, 1024, 2003), (4096, 64, 20003), (20000, 32, 5003), (520, 264, 32003), (65, 1024, 301),
              (1, 8, 8193), (16, 2048, 8203), (17, 520, 20001), (32, 72, 32003),
              (2048, 1024, 20001)]


def head_case(T, H, V, seed=0, std=2.5):
    rn = gen(seed + T + H + V)
    g = torch.Generator(device=DEV).manual_seed(seed + 3 * T + V)
    x, w = rn(T, H, dt=BF16), rn(V, H, std=std * H ** -0.5, dt=BF16)
    labels = torch.randint(0, V, (T,), generator=g, device=DEV)
    off = torch.rand(T, generator=g, device=DEV)
    labels = torch.where(off < 0.1, -100, torch.where(off > 0.95, V, labels)).to(I32) if T > 1 else labels.to(I32)
    return x, w, labels, torch.rand(T, generator=g, device=DEV) + 0.1


def grad_bounds(P, eP, x, w, need_x=True):
    """Bounds of dx = P W and dw = P^T x where P is off by eP before its rounding."""
    eP = eP + B * (P.abs() + eP)
    T, V = P.shape
    wa, xa = w.double().abs(), x.double().abs()
    ex = (eP + 2 * V * U * (P.abs() + eP)) @ wa
    ew = (eP + 2 * T * U * (P.abs() + eP)).T @ xa
    return ex, ew


@pytest.mark.parametrize("T,H,V", HEAD_SIZES)
def test_vocab_ce(T, H, V):
    x, w, labels, dloss = head_case(T, H, V)
    el = product_bound(x, w)
    loss, lse = R.ce(x, w, labels)
    got_loss, got_lse = M.vocab_ce_forward(x, w, labels)
    # the sum of positive terms: 64 terms a lane, then pairs over the tiles
    e_lse = el.amax(1) + (300 + V / 512) * U + 4 * U * lse.abs()
    R.within(got_lse, lse, e_lse, "lse")
    R.within(got_loss, loss, e_lse + el.amax(1) + 2 * U * (lse.abs() + loss.abs()), "loss")
    P = R.ce_P(dloss, x, w, labels)
    p = torch.softmax(x.double() @ w.double().T, 1)
    eP = dloss.double()[:, None] * (p * (1.2 * (el + e_lse[:, None]) + 16 * U * (1 + lse.abs()[:, None])) + 4 * U)
    ex, ew = grad_bounds(P, eP, x, w)
    dx, dw = P @ w.double(), P.T @ x.double()
    out = M.vocab_ce_backward(dloss, x, w, labels, got_lse)
    R.within(out["dx"], dx, B * dx.abs() + (1 + B) * ex, "dx")
    R.within(out["dw"], dw, B * dw.abs() + (1 + B) * ew, "dw")
    near(out["dx"], dx, 2, "dx"), near(out["dw"], dw, 2, "dw")
    if V > 1:    # (of one class P is a rounding error of 1 - 1)
        few(out["dx"], dx, T, "dx"), few(out["dw"], dw, T, "dw")
    dead = (labels < 0) | (labels >= V)
    assert not out["dx"][dead].any() and not got_loss[dead].any()
    again = M.vocab_ce_backward(dloss, x, w, labels, got_lse)
    assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["dw"], out["dw"])
    for n, ref, e in (("dx", dx, ex), ("dw", dw, ew)):      # alone: the sums may be cut differently
        one = M.vocab_ce_backward(dloss, x, w, labels, got_lse, need=(n,))
        assert list(one) == [n]
        R.within(one[n], ref, B * ref.abs() + (1 + B) * e, n + " alone")


def distill_case(T, H, V, k, tdt, seed=0):
    x, w, _, dloss = head_case(T, H, V, seed + 7)
    g = torch.Generator(device=DEV).manual_seed(seed + T + k)
    ids = torch.randint(-1, V + 1, (T, k), generator=g, device=DEV)      # ids twice in a row, outside on both sides
    ids = torch.where(torch.rand(T, 1, generator=g, device=DEV) < 0.15, -1, ids).to(I32)
    t = (torch.randn(T, k, generator=g, device=DEV) * 3).to(tdt)
    return x, w, ids, t, dloss


@pytest.mark.parametrize("tau,tdt", [(1.0, BF16), (2.5, F32), (0.5, F32)])
@pytest.mark.parametrize("T,H,V,k", [(1, 8, 1, 1), (1, 64, 50, 3), (17, 256, 3001, 16), (65, 72, 333, 65), (129, 128, 4099, 200),
                                     (70, 64, 2000, 1024), (600, 520, 20001, 32), (4096, 32, 17003, 7), (520, 264, 32003, 40), (40, 1040, 500, 9), (100, 1024, 700, 9),
                                     (5, 64, 9001, 20), (16, 1032, 8200, 65), (31, 264, 12001, 130)])
def test_vocab_distill(T, H, V, k, tau, tdt):
    x, w, ids, t, dloss = distill_case(T, H, V, k, tdt)
    el = product_bound(x, w) / tau
    loss, lse, q, logits = R.distill(x, w, ids, t, tau)
    row = torch.isfinite(lse)
    got = M.vocab_distill_forward(x, w, ids, t, temperature=tau)
    on = (ids >= 0) & (ids < V)
    at = torch.where(on, (el * tau).gather(1, torch.where(on, ids, 0).long()), 0.0)
    R.within(got["logits"], logits, at + U * logits.abs(), "logits")
    # (t - m) / tau has two roundings, exp one of 2 u, the sums k and one more; below 2^-126 values go to zero
    tt = torch.where(on, t.double(), 0.0).abs().amax(1)[:, None] / tau
    R.within(got["q"], q, q * (8 * tt + 2 * k + 16) * U + 2.0 ** -120, "q")
    e_lse = el.amax(1) + (300 + V / 512) * U + 4 * U * torch.where(row, lse, 0.0).abs()
    R.within(got["lse"], lse, torch.where(row, e_lse, 0.0), "lse")
    size = torch.where(q > 0, q * (torch.log(torch.where(q > 0, q, 1.0)).abs() + logits.abs() / tau + 1), 0.0).sum(1)
    e_loss = e_lse + el.amax(1) + (size + torch.where(row, lse, 0.0).abs()) * (8 * tt[:, 0] + 4 * k + 32) * U
    R.within(got["loss"], loss, tau * tau * e_loss, "loss")
    P = R.distill_P(dloss, x, w, ids, got["q"], row, tau)
    p = torch.softmax(x.double() @ w.double().T / tau, 1)
    c = (dloss.double() * tau)[:, None]
    eP = c * (p * (1.2 * (el + e_lse[:, None]) + 16 * U * (1 + lse.nan_to_num(0, 0, 0).abs()[:, None])) + 4 * U)
    ex, ew = grad_bounds(P, eP, x, w)
    dx, dw = P @ w.double(), P.T @ x.double()
    args = (dloss, x, w, ids, got["q"], got["logits"], got["lse"])
    out = M.vocab_distill_backward(*args, temperature=tau)
    R.within(out["dx"], dx, B * dx.abs() + (1 + B) * ex, "dx")
    R.within(out["dw"], dw, B * dw.abs() + (1 + B) * ew, "dw")
    assert not out["dx"][~row].any()
    if V > 1:
        few(out["dx"], dx, T, "dx"), few(out["dw"], dw, T, "dw")
    again = M.vocab_distill_backward(*args, temperature=tau, need=("dw", "dx"))
    assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["dw"], out["dw"])
    one = M.vocab_distill_backward(*args, temperature=tau, need=("dx",))
    R.within(one["dx"], dx, B * dx.abs() + (1 + B) * ex, "dx alone")


def test_distill_over_the_largest_vocabulary():
    """2^21 columns and 1024 entries a row: the entries' lists at their largest."""
    T, H, V, k = 18, 8, 1 << 21, 1024
    rn = gen(4)
    x, w = rn(T, H, dt=BF16), rn(V, H, std=1.0, dt=BF16)
    g = torch.Generator(device=DEV).manual_seed(5)
    ids = torch.randint(-1, V, (T, k), generator=g, device=DEV)
    ids[:, 0], ids[:, 1] = V - 1, 0
    ids, t, dloss = ids.to(I32), rn(T, k), torch.ones(T, device=DEV)
    loss, lse, q, logits = R.distill(x, w, ids, t, 1.0)
    got = M.vocab_distill_forward(x, w, ids, t)
    # an H of 8: sums of 8 products, 2^21 terms of the sum of exponentials in chunks of 16 columns and 256 threads
    R.within(got["lse"], lse, 16 * U * 40 + 600 * U + 4 * U * lse.abs(), "lse")
    R.within(got["logits"], logits, 16 * U * (x.double().abs().sum(1).amax() * 5), "logits")
    R.within(got["q"], q, q * (8 * 5 + 2 * k + 16) * U + 2.0 ** -120, "q")
    assert R.off(got["loss"], loss) < 1e-4
    out = M.vocab_distill_backward(dloss, x, w, ids, got["q"], got["logits"], got["lse"])
    P = R.distill_P(dloss, x, w, ids, got["q"], torch.isfinite(lse), 1.0)
    near(out["dw"], P.T @ x.double(), 2, "dw")
    assert R.off(out["dx"], P @ w.double()) < 2 * B     # 144 values: two roundings, each at most b of its sum's terms


@pytest.mark.parametrize("k", [2, 64, 65, 300, 1024])
def test_distill_of_ids_that_a_row_names_often(k):
    """One id everywhere, two ids in turn, each id twice, ids that differ by a power of two, an id with a stranger."""
    H, V = 64, 70001
    rn = gen(9)
    x, w, t = rn(5, H, dt=BF16), rn(V, H, std=0.3, dt=BF16), rn(5, k)
    j = torch.arange(k, device=DEV)
    ids = torch.stack([0 * j + 7, 3 + j % 2 * (V - 4), j // 2 * 65, (j * 4096) % 65536, torch.where(j == k - 1, -1, 69000)]).to(I32)
    loss, lse, q, logits = R.distill(x, w, ids, t, 1.0)
    got = M.vocab_distill_forward(x, w, ids, t)
    tt = t.double().abs().amax(1)[:, None]
    R.within(got["q"], q, q * (8 * tt + 2 * k + 16) * U + 2.0 ** -120, "q")
    assert (got["q"][0, 0] - 1).abs() < 4 * k * U and not got["q"][0, 1:].any() and got["q"][4, k - 1] == 0
    el = product_bound(x, w)
    R.within(got["logits"], logits, torch.where(ids >= 0, el.gather(1, ids.clamp(min=0).long()), 0.0) + U * logits.abs(), "logits")
    again = M.vocab_distill_forward(x, w, ids, t)
    assert all(torch.equal(got[n], again[n]) for n in got)
    dloss = torch.ones(5, device=DEV)
    P = R.distill_P(dloss, x, w, ids, got["q"], torch.isfinite(lse), 1.0)
    out = M.vocab_distill_backward(dloss, x, w, ids, got["q"], got["logits"], got["lse"])
    near(out["dx"], P @ w.double(), 2, "dx"), near(out["dw"], P.T @ x.double(), 2, "dw")


def test_distill_of_one_sure_entry_is_cross_entropy():
    """One entry a row: q is 1, the loss and the gradients are the cross entropy's."""
    x, w, labels, dloss = head_case(140, 128, 2111)
    loss, lse = M.vocab_ce_forward(x, w, labels)
    got = M.vocab_distill_forward(x, w, labels[:, None].contiguous(), torch.full((140, 1), -3.5, device=DEV))
    on = (labels >= 0) & (labels < 2111)
    assert torch.equal(got["q"][:, 0], on.float())
    assert torch.equal(got["loss"], loss) and torch.equal(got["lse"][on], lse[on]) and torch.isinf(got["lse"][~on]).all()
    a = M.vocab_ce_backward(dloss, x, w, labels, lse)
    b = M.vocab_distill_backward(dloss, x, w, labels[:, None].contiguous(), got["q"], got["logits"], got["lse"])
    for n in a:
        assert R.off(b[n], a[n].double()) < 2 * U     # the labels' places are computed apart: a bit of fp32 before the rounding


@pytest.mark.parametrize("fill", [NAN, INF, -INF, 3.3e38])
def test_rows_without_a_target_count_for_nothing(fill):
    """Whatever x, dloss and the teacher hold in a masked row or entry."""
    T, H, V = 200, 128, 3001
    x, w, labels, dloss = head_case(T, H, V)
    dead = (labels < 0) | (labels >= V)
    assert 5 < int(dead.sum()) < T - 5
    zero = lambda v: torch.where(dead if v.dim() == 1 else dead[:, None], torch.zeros_like(v), v)  # noqa: E731
    put = lambda v: torch.where(dead if v.dim() == 1 else dead[:, None], torch.full_like(v, fill), v)  # noqa: E731
    loss, lse = M.vocab_ce_forward(zero(x), w, labels)
    loss2, lse2 = M.vocab_ce_forward(put(x), w, labels)
    assert torch.equal(loss, loss2) and torch.equal(lse[~dead], lse2[~dead])
    a = M.vocab_ce_backward(zero(dloss), zero(x), w, labels, zero(lse))
    b = M.vocab_ce_backward(put(dloss), put(x), w, labels, put(lse2))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    ids = torch.stack([labels, torch.full_like(labels, -1), (labels + 1) % V, torch.full_like(labels, V)], 1)
    ids = torch.where(dead[:, None], torch.full_like(ids, -7), ids).contiguous()
    t = gen(5)(T, 4)
    outside = (ids < 0) | (ids >= V)
    t1, t2 = torch.where(outside, 0.0, t), torch.where(outside, fill, t)
    p, r = M.vocab_distill_forward(zero(x), w, ids, t1), M.vocab_distill_forward(put(x), w, ids, t2)
    assert all(torch.equal(p[n], r[n]) for n in p) and not p["loss"][dead].any() and not r["q"][outside].any()
    a = M.vocab_distill_backward(zero(dloss), zero(x), w, ids, p["q"], p["logits"], p["lse"])
    b = M.vocab_distill_backward(put(dloss), put(x), w, ids, r["q"], r["logits"], r["lse"])
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])


def test_teacher_rows_of_the_lowest_values():
    """Entries at -inf have no probability; a row of them has no target; a row of the type's lowest
    finite value is an even one; NaN in a row's entry is the row's result."""
    x, w, _, _ = head_case(6, 64, 100)
    ids = torch.arange(18, device=DEV, dtype=I32).view(6, 3)
    low = torch.finfo(F32).min
    t = torch.tensor([[0.0, -INF, 1.0], [-INF] * 3, [low] * 3, [low, 0.0, low], [INF, 0.0, 0.0], [NAN, 0.0, 0.0]], device=DEV)
    got = M.vocab_distill_forward(x, w, ids, t)
    q = got["q"].double().cpu()
    assert q[0, 1] == 0 and abs(q[0].sum() - 1) < 4 * U and q[1].tolist() == [0, 0, 0]
    assert (q[2] - 1 / 3).abs().max() < 4 * U and q[3].tolist() == [0, 1, 0]
    assert torch.isnan(q[5]).all() and torch.isnan(q[4]).any()
    lse, loss = got["lse"].cpu(), got["loss"].cpu()
    assert torch.isinf(lse).tolist() == [False, True] + [False] * 4 and loss[1] == 0
    assert torch.isnan(loss).tolist() == [False] * 4 + [True] * 2


def test_logits_far_apart():
    """Logits of hundreds: the running maximum keeps the sums in range."""
    T, H, V = 70, 64, 3000
    x, w, labels, dloss = head_case(T, H, V, std=100.0)
    loss, lse = R.ce(x, w, labels)
    el = product_bound(x, w).amax(1)
    got = M.vocab_ce_forward(x, w, labels)
    assert loss.max() > 200
    R.within(got[1], lse, el + 400 * U + 4 * U * lse.abs(), "lse")
    R.within(got[0], loss, 2 * el + 400 * U + 8 * U * lse.abs() + 4 * U * loss, "loss")
    out = M.vocab_ce_backward(dloss, x, w, labels, got[1])
    P = R.ce_P(dloss, x, w, labels)
    # exp(l - lse) at |l| of hundreds: an error of l log2(e) of 2 u |l| on either side
    assert R.off(out["dx"], P @ w.double()) < 1.2 * B + 8 * U * float(lse.abs().max())


def test_head_without_rows():
    x, w = torch.empty(0, 64, device=DEV, dtype=BF16), gen(1)(30, 64, dt=BF16)
    none, ids = torch.empty(0, device=DEV), torch.empty(0, device=DEV, dtype=I32)
    loss, lse = M.vocab_ce_forward(x, w, ids)
    assert loss.shape == lse.shape == (0,)
    out = M.vocab_ce_backward(none, x, w, ids, lse)
    assert out["dx"].shape == (0, 64) and out["dw"].shape == (30, 64) and not out["dw"].any()
    r = M.vocab_distill_forward(x, w, ids.view(0, 4), none.view(0, 4))
    out = M.vocab_distill_backward(none, x, w, ids.view(0, 4), r["q"], r["logits"], r["lse"])
    assert r["q"].shape == (0, 4) and not out["dw"].any()


def test_head_past_32_bit_offsets():
    """A head of more than 2^32 bytes: its last rows are read and their gradient is written."""
    T, H, V = 3, 4096, 540001
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.zeros(V, H, device=DEV, dtype=BF16)
    w[-8:] = torch.randn(8, H, generator=g, device=DEV) * 0.05
    x = torch.randn(T, H, generator=g, device=DEV).to(BF16)
    labels = torch.tensor([V - 1, V - 8, 0], device=DEV, dtype=I32)
    loss, lse = M.vocab_ce_forward(x, w, labels)
    l = x.double() @ w[-8:].double().T
    full = torch.logsumexp(torch.cat([l, torch.full((T, 1), 0.0, device=DEV).double() + torch.log(torch.tensor(V - 8.0))], 1), 1)
    assert (lse - full).abs().max() < 1e-3 and abs(float(loss[2] - full[2])) < 1e-3
    assert abs(float(loss[0] - (full[0] - l[0, 7]))) < 1e-3
    out = M.vocab_ce_backward(torch.ones(T, device=DEV), x, w, labels, lse, need=("dw",))["dw"]
    P = torch.exp(l - full[:, None])
    P[0, 7] -= 1
    P[1, 0] -= 1
    assert R.off(out[-8:], P.T @ x.double()) < 1.2 * B
    assert R.off(out[1:3], (torch.exp(-full)[:, None] * x.double()).sum(0)[None].expand(2, H)) < 1.2 * B


# ------------------------------------------------------------------ layer norm
@pytest.mark.parametrize("xdt,ydt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 8), (130, 64), (2000, 118), (700, 200), (20003, 24), (515, 1000), (77, 1500), (5, 3500), (33, 5001), (3, 12000), (259, 1500), (300, 3500), (270, 5001), (257, 12000), (4, 513), (300, 2048), (67, 2880), (9, 4100),
                                 (700, 4096), (6, 8191), (5, 8192), (3, 16383), (600, 16384)])
def test_layer_norm(T, H, xdt, ydt):
    rn = gen(T + H)
    x = (rn(T, H, std=2.0) + rn(1, H) + 1.5).to(xdt)
    w, b, dy, base = rn(H), rn(H), rn(T, H, dt=ydt), rn(T, H, dt=xdt)
    e_out, e_dx = (B if ydt is BF16 else U), (B if xdt is BF16 else U)
    sums = (24 + H / 64) * U          # a lane's sum of 8 or 16 values, the wave's, the workgroup's: well below
    for ww, bb in ((w, b), (w, None), (None, None)):
        y, mean, rstd = R.layer_norm(x, ww, bb, 1e-5)
        got = M.layer_norm_forward(x, ww, bb, eps=1e-5, out_dtype=ydt)
        size = x.double().abs().mean(1)
        e_mean = sums * size
        R.within(got["mean"], mean, e_mean + U * mean.abs(), "mean")
        spread = (x.double() - mean[:, None]).abs().amax(1)
        # the variance: twice the mean's error against the spread, where it is at all
        e_r = rstd * (sums + 4 * U + rstd * rstd * (2 * spread * (e_mean + 2 * U * x.double().abs().amax(1)) + e_mean ** 2))
        R.within(got["rstd"], rstd, e_r, "rstd")
        n = (x.double() - mean[:, None]) * rstd[:, None]
        e_n = rstd[:, None] * (e_mean[:, None] + 2 * U * (x.double().abs() + mean.abs()[:, None])) + n.abs() * (e_r / rstd)[:, None] * 1.01
        scale = 1 if ww is None else ww.double().abs()
        R.within(got["y"], y, e_out * y.abs() + scale * e_n * 1.01 + 4 * U * (scale * n.abs() + y.abs()), "y")
    for ww, bs in ((w, base), (None, None)):
        dx, dw, db = R.layer_norm_grad(dy, x, got["mean"], got["rstd"], ww, bs)
        out = M.layer_norm_backward(dy, x, got["mean"], got["rstd"], ww, dx_base=bs)
        n = (x.double() - got["mean"].double()[:, None]) * got["rstd"].double()[:, None]
        a = dy.double().abs() * (1 if ww is None else ww.double().abs())
        e_n = 4 * U * (n.abs() + got["rstd"].double()[:, None] * (x.double().abs() + got["mean"].double().abs()[:, None]))
        r = got["rstd"].double()[:, None]
        terms = a + a.mean(1, keepdim=True) + n.abs() * (a * n.abs()).mean(1, keepdim=True)
        e = r * ((sums + 8 * U) * terms + e_n * (a * n.abs()).mean(1, keepdim=True) + n.abs() * (a * e_n).mean(1, keepdim=True))
        R.within(out["dx"], dx, e_dx * dx.abs() + 1.01 * e + 4 * U * dx.abs(), "dx")
        # at most T / groups rows a slot and 512 workgroups
        rows = (T / 64 + 64) * U
        R.within(out["dw"], dw, (rows * dy.double().abs() * n.abs() + dy.double().abs() * e_n).sum(0) + 2 * U * dw.abs(), "dw")
        R.within(out["db"], db, rows * dy.double().abs().sum(0) + 2 * U * db.abs(), "db")
        again = M.layer_norm_backward(dy, x, got["mean"], got["rstd"], ww, dx_base=bs)
        assert all(torch.equal(out[k], again[k]) for k in out)
        for k in out:
            one = M.layer_norm_backward(dy, x, got["mean"], got["rstd"], ww, dx_base=bs if k == "dx" else None, need=(k,))
            assert list(one) == [k] and torch.equal(one[k], out[k])


def test_layer_norm_far_from_zero():
    """A mean of a thousand spreads: the variance comes from the centred values."""
    x = gen(3)(50, 1000) + 1000.0
    y, mean, rstd = R.layer_norm(x, None, None, 0.0)
    got = M.layer_norm_forward(x, eps=0.0)
    # the mean is off by up to (24 + H / 64) u of 1000, which shifts n by that; its square is lost in the variance
    assert float((got["rstd"].double() / rstd - 1).abs().max()) < 1e-4
    assert float((got["y"].double() - y).abs().max()) < 40 * U * 1000 * float(rstd.max()) + 1e-4


def test_layer_norm_constant_rows_and_in_place_gradient():
    x = torch.full((3, 129), 2.5, device=DEV)
    got = M.layer_norm_forward(x, eps=1e-5)
    assert not got["y"].any() and (got["mean"] == 2.5).all()
    rn = gen(9)
    x, dy, base = rn(33, 200, dt=BF16), rn(33, 200, dt=BF16), rn(33, 200, dt=BF16)
    f = M.layer_norm_forward(x)
    want = M.layer_norm_backward(dy, x, f["mean"], f["rstd"], dx_base=base, need=("dx",))["dx"]
    held = base.clone()
    out = M.layer_norm_backward(dy, x, f["mean"], f["rstd"], dx_base=held, dx=held, need=("dx",))["dx"]
    assert out is held and torch.equal(held, want)


def test_layer_norm_without_rows():
    x = torch.empty(0, 40, device=DEV)
    f = M.layer_norm_forward(x, torch.ones(40, device=DEV))
    out = M.layer_norm_backward(x, x, f["mean"], f["rstd"], torch.ones(40, device=DEV))
    assert out["dx"].shape == (0, 40) and not out["dw"].any() and not out["db"].any()


# ------------------------------------------------------------------ streams and graphs
def everything(x, w13, head, labels, ids, t, dh, dloss, dy):
    """A pass through all of the calls, as a list of tensors."""
    f = M.layer_norm_forward(x, out_dtype=BF16)
    h = M.gated_ffn_forward(f["y"], w13)
    b = M.gated_ffn_backward(dh, f["y"], w13)
    loss, lse = M.vocab_ce_forward(f["y"], head, labels)
    c = M.vocab_ce_backward(dloss, f["y"], head, labels, lse)
    d = M.vocab_distill_forward(f["y"], head, ids, t, temperature=2.0)
    e = M.vocab_distill_backward(dloss, f["y"], head, ids, d["q"], d["logits"], d["lse"], temperature=2.0)
    n = M.layer_norm_backward(dy, x, f["mean"], f["rstd"])
    return [f["y"], h, *b.values(), loss, lse, *c.values(), *d.values(), *e.values(), *n.values()]


def everything_inputs(seed, T=150, H=136, I=72, V=2005, k=9):
    rn = gen(seed)
    x, w, ids, t, dloss = distill_case(T, H, V, k, F32, seed)
    labels = head_case(T, H, V, seed)[2]
    return [x.float(), rn(2 * I, H, std=0.2, dt=BF16), w, labels, ids, t, rn(T, I, dt=BF16), dloss, rn(T, H, dt=BF16)]


def test_captured_passes_replay():
    """Every call in one captured graph (their scratch from the graph's pool): each replay on new inputs
    gives the eager bits, with eager work between the replays; two graphs do not share scratch."""
    held = [everything_inputs(0), everything_inputs(1)]
    graphs = []
    for ins in held:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            everything(*ins)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = everything(*ins)
        graphs.append((g, ins, outs))
    for seed in (2, 3, 4):
        fresh = [everything_inputs(10 * seed + j) for j in range(2)]
        wants = [[v.clone() for v in everything(*f)] for f in fresh]
        for (g, ins, _), f in zip(graphs, fresh):
            for a, b in zip(ins, f):
                a.copy_(b)
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, _, outs), want in zip(graphs, wants):
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_on_two_streams_at_once():
    sets = [everything_inputs(s, T=700, V=4001) for s in (0, 1)]
    wants = [[v.clone() for v in everything(*s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            got.append([everything(*s) for _ in range(3)])
    torch.cuda.synchronize()
    for runs, want in zip(got, wants):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
