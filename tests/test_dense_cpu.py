"""The dense operators without a GPU: their 64-bit references against differences and autograd,
and every refusal of the C ABI and of the binding."""
import os

import pytest

import dense_ref as R

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("bit_quantized_moe_expert_amd")
if not os.path.exists(pkg.LIB_PATH):
    pytest.skip("libnf4moe.so not built", allow_module_level=True)

from bit_quantized_moe_expert_amd import dense  # noqa: E402

L = pkg.lib()
OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = 0, 1, 2, 3, 4
F64, BF16, F32, I32 = torch.float64, torch.bfloat16, torch.float32, torch.int32
BIG = 1 << 62
GPU = torch.cuda.is_available()


def far(i):
    """Addresses far apart, aligned, never dereferenced."""
    return (i + 1) << 40


# ------------------------------------------------------------------ references
def numeric(f, v, eps=1e-6):
    """df/dv of a scalar function by central differences."""
    out = torch.zeros_like(v)
    for i in range(v.numel()):
        d = torch.zeros_like(v).view(-1)
        d[i] = eps
        out.view(-1)[i] = (f(v + d.view(v.shape)) - f(v - d.view(v.shape))) / (2 * eps)
    return out


def rn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g, dtype=F64) * std


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("inter", [0, 1])
def test_ffn_gradient_reference_by_differences(kind, inter):
    x, w, dh = rn(3, 5), rn(8, 5, seed=1, std=2.0), rn(3, 4, seed=2)
    f = lambda x, w: (dh * R.ffn(x, w, kind, 1.702, 7.0, inter)[2]).sum()  # noqa: E731
    g, u = R.ffn(x, w, kind, 1.702, 7.0, inter)[:2]
    assert min((g - 7).abs().min(), (u.abs() - 7).abs().min()) > 1e-3    # no value at a clamp's corner
    _, _, dx, dw = R.ffn_grad(dh, x, w, kind, 1.702, 7.0, inter)
    assert torch.allclose(dx, numeric(lambda v: f(v, w), x), atol=1e-7, rtol=1e-6)
    assert torch.allclose(dw, numeric(lambda v: f(x, v), w), atol=1e-7, rtol=1e-6)
    wg, wu = R.split(w, inter)
    assert torch.equal(R.join(wg, wu, inter), w)
    if kind == 0:
        assert torch.allclose(R.ffn(x, w, 0, 0, 0, inter)[2], torch.nn.functional.silu(x @ wg.T) * (x @ wu.T))


def test_ce_reference_is_torchs_and_its_gradient_by_differences():
    x, w, dloss = rn(6, 4), rn(9, 4, seed=1), rn(6, seed=2).abs()
    labels = torch.tensor([0, 8, -100, 3, 9, 3])
    loss, lse = R.ce(x, w, labels)
    on = (labels >= 0) & (labels < 9)
    want = torch.nn.functional.cross_entropy(x @ w.T, torch.where(on, labels, -100), reduction="none")
    assert torch.allclose(loss, want) and torch.allclose(lse, torch.logsumexp(x @ w.T, 1))
    P = R.ce_P(dloss, x, w, labels)
    f = lambda x, w: (dloss * R.ce(x, w, labels)[0]).sum()  # noqa: E731
    assert torch.allclose(P @ w, numeric(lambda v: f(v, w), x), atol=1e-8) and torch.allclose(P.T @ x, numeric(lambda v: f(x, v), w), atol=1e-8)


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_reference_is_a_divergence_and_its_gradient_by_differences(tau):
    x, w, dloss, t = rn(5, 4), rn(9, 4, seed=1), rn(5, seed=2).abs(), rn(5, 3, seed=3, std=2.0)
    ids = torch.tensor([[0, 4, 8], [2, 2, 5], [-1, -1, 9], [3, -1, 3], [7, 1, 6]])
    loss, lse, q, logits = R.distill(x, w, ids, t, tau)
    Q = torch.zeros(5, 9, dtype=F64)
    for r in range(5):
        e = [(int(i), float(torch.exp(v / tau))) for i, v in zip(ids[r], t[r]) if 0 <= i < 9]
        for i, v in e:
            Q[r, i] += v / sum(v for _, v in e)
    S = torch.log_softmax(x @ w.T / tau, 1)
    want = tau ** 2 * torch.where(Q > 0, Q * (torch.log(Q.clamp(min=1e-300)) - S), 0.0).sum(1)
    assert torch.allclose(loss, want) and loss[2] == 0 and torch.isinf(lse[2])
    assert torch.allclose(q[1], torch.stack([Q[1, 2], torch.tensor(0.0, dtype=F64), Q[1, 5]]))
    P = R.distill_P(dloss, x, w, ids, q, torch.isfinite(lse), tau)
    f = lambda x, w: (dloss * R.distill(x, w, ids, t, tau)[0]).sum()  # noqa: E731
    assert torch.allclose(P @ w, numeric(lambda v: f(v, w), x), atol=1e-7) and torch.allclose(P.T @ x, numeric(lambda v: f(x, v), w), atol=1e-7)


def test_layer_norm_reference_is_torchs_and_its_gradient_by_differences():
    x, w, b, dy, base = rn(3, 7), rn(7, seed=1), rn(7, seed=2), rn(3, 7, seed=3), rn(3, 7, seed=4)
    y, mean, rstd = R.layer_norm(x, w, b, 1e-3)
    assert torch.allclose(y, torch.nn.functional.layer_norm(x, (7,), w, b, 1e-3))
    dx, dw, db = R.layer_norm_grad(dy, x, mean, rstd, w, base)
    f = lambda x, w, b: (dy * R.layer_norm(x, w, b, 1e-3)[0]).sum()  # noqa: E731
    assert torch.allclose(dx - base, numeric(lambda v: f(v, w, b), x), atol=1e-7)
    assert torch.allclose(dw, numeric(lambda v: f(x, v, b), w), atol=1e-7) and torch.allclose(db, numeric(lambda v: f(x, w, v), b), atol=1e-7)


# ------------------------------------------------------------------ refusals of the C ABI
def call(fn, status, *args, msg=""):
    got = fn(*args)
    assert got == status, (got, L.nf4moe_last_error())
    if msg:
        assert msg in L.nf4moe_last_error().decode(), L.nf4moe_last_error()


def ffn_desc(H=64, I=32, w=far(9), glu=0, alpha=0.0, limit=0.0, inter=0):
    return dense._FFN.pack(H, I, w or 0, glu, alpha, limit, inter)


def test_gated_ffn_validation():
    def fwd(d=None, x=far(0), T=4, h=far(1)):
        return L.nf4moe_gated_ffn_forward(ffn_desc() if d is None else d, x, T, h, None)

    def bwd(d=None, dh=far(0), x=far(1), T=4, dx=far(2), dw=far(3), h=far(4), ws=far(5), n=BIG):
        return L.nf4moe_gated_ffn_backward(ffn_desc() if d is None else d, dh, x, T, dx, dw, h, ws, n, None)
    assert L.nf4moe_gated_ffn_forward(None, far(0), 4, far(1), None) == INVALID
    for f in (fwd, bwd):
        for bad in (dict(H=0), dict(H=-8), dict(H=12), dict(H=(1 << 20) + 8), dict(I=0), dict(I=4), dict(I=(1 << 20) + 8),
                    dict(glu=2), dict(glu=-1), dict(inter=2), dict(glu=1), dict(glu=1, alpha=1.0),
                    dict(glu=1, alpha=float("nan"), limit=1.0), dict(glu=1, alpha=1.0, limit=float("inf"))):
            assert f(ffn_desc(**bad)) == INVALID, bad
        assert f(T=-1) == INVALID and f(T=(1 << 30) + 1) == INVALID
        assert f(ffn_desc(w=None)) == INVALID and f(ffn_desc(w=far(9) + 8)) == INVALID
        assert f(x=None) == INVALID and f(x=far(0) + 2) == INVALID
        assert f(ffn_desc(H=1 << 20, I=1 << 20)) == UNSUPPORTED and f(ffn_desc(I=1 << 20), T=1 << 20) == UNSUPPORTED
    assert fwd(h=None) == INVALID and fwd(h=far(1) + 8) == INVALID and fwd(T=0) == OK and fwd(x=None, h=None, T=0) == OK
    assert bwd(dh=None) == INVALID and bwd(dh=far(0) + 8) == INVALID and bwd(dx=None, dw=None) == INVALID
    assert bwd(dx=far(2) + 4) == INVALID and bwd(dw=far(3) + 8) == INVALID and bwd(h=far(4) + 2) == INVALID
    need = L.nf4moe_gated_ffn_workspace_bytes(ffn_desc(), 4)
    assert need > 0 and bwd(n=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE and bwd(ws=far(5) + 128) == INVALID
    assert bwd(T=0, dw=None) == OK and bwd(T=0, dx=None, dw=None) == OK
    assert L.nf4moe_gated_ffn_workspace_bytes(ffn_desc(), 0) == 0 and L.nf4moe_gated_ffn_workspace_bytes(ffn_desc(H=12), 4) == 0
    if not GPU:
        assert fwd() == HIP and bwd(n=need) == HIP and bwd(n=need, dx=None, h=None) == HIP and bwd(n=need, dw=None) == HIP


def head_desc(H=64, V=100, w=far(9)):
    return dense._HEAD.pack(H, V, w or 0)


def ce_fwd(d=None, x=far(0), T=4, labels=far(1), loss=far(2), lse=far(3), ws=far(4), n=BIG):
    return L.nf4moe_vocab_ce_forward(head_desc() if d is None else d, x, T, labels, loss, lse, ws, n, None)


def ce_bwd(d=None, dloss=far(0), x=far(1), T=4, labels=far(2), lse=far(3), dx=far(4), dw=far(5), ws=far(6), n=BIG):
    return L.nf4moe_vocab_ce_backward(head_desc() if d is None else d, dloss, x, T, labels, lse, dx, dw, ws, n, None)


def ds_fwd(d=None, x=far(0), T=4, labels=far(1), t=far(2), tdt=0, k=3, tau=1.0, loss=far(3), lse=far(4), q=far(5), logits=far(6),
           ws=far(7), n=BIG):
    return L.nf4moe_vocab_distill_forward(head_desc() if d is None else d, x, T, labels, t, tdt, k, tau, loss, lse, q, logits, ws, n, None)


def ds_bwd(d=None, dloss=far(0), x=far(1), T=4, labels=far(2), q=far(10), logits=far(11), lse=far(3), k=3, tau=1.0, dx=far(4),
           dw=far(5), ws=far(6), n=BIG):
    return L.nf4moe_vocab_distill_backward(head_desc() if d is None else d, dloss, x, T, labels, q, logits, lse, k, tau, dx, dw, ws, n, None)


def test_head_validation():
    for f, k, back in ((ce_fwd, 0, 0), (ds_fwd, 3, 0), (ce_bwd, 0, 1), (ds_bwd, 3, 1)):
        for bad in (dict(H=0), dict(H=12), dict(H=(1 << 20) + 8), dict(V=0), dict(V=-3), dict(V=(1 << 21) + 1)):
            assert f(head_desc(**bad)) == INVALID, bad
        assert f(T=-1) == INVALID and f(T=(1 << 30) + 1) == INVALID
        assert f(head_desc(V=1 << 21), T=1 << 26) == UNSUPPORTED and f(head_desc(H=1 << 20, V=1 << 21)) == UNSUPPORTED
        assert f(head_desc(w=None)) == INVALID and f(head_desc(w=far(9) + 8)) == INVALID
        for name in ("x", "labels", "lse"):
            assert f(**{name: None}) == INVALID, name
        assert f(x=far(0) + 8) == INVALID and f(labels=far(1) + 2) == INVALID and f(lse=far(3) + 1) == INVALID
        need = L.nf4moe_vocab_workspace_bytes(head_desc(), 4, k, back)
        assert need > 0 and f(n=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE and f(ws=far(20) + 64) == INVALID
        if not GPU:
            assert f(n=need) == HIP
    for f in (ce_fwd, ds_fwd):
        assert f(loss=None) == INVALID and f(loss=far(2) + 2) == INVALID and f(T=0, x=None, labels=None) == OK
    for f in (ce_bwd, ds_bwd):
        assert f(dloss=None) == INVALID and f(dloss=far(0) + 2) == INVALID and f(dx=None, dw=None) == INVALID
        assert f(dx=far(4) + 8) == INVALID and f(dw=far(5) + 4) == INVALID and f(T=0, dw=None) == OK
    for f in (ds_fwd, ds_bwd):
        assert f(k=0) == INVALID and f(k=1025) == INVALID and f(q=None) == INVALID and f(logits=None) == INVALID
        assert f(q=far(5) + 2) == INVALID and f(logits=far(6) + 1) == INVALID
        for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-4, 1e4):
            assert f(tau=tau) == INVALID, tau
    assert ds_fwd(tdt=2) == INVALID and ds_fwd(t=None) == INVALID and ds_fwd(t=far(2) + 2) == INVALID
    assert ds_fwd(t=far(2) + 1, tdt=1) == INVALID
    assert L.nf4moe_vocab_workspace_bytes(head_desc(), 0, 0, 1) == 0 and L.nf4moe_vocab_workspace_bytes(head_desc(V=0), 4, 0, 0) == 0
    assert L.nf4moe_vocab_workspace_bytes(head_desc(), 4, -1, 0) == 0 and L.nf4moe_vocab_workspace_bytes(head_desc(), 4, 1025, 1) == 0


def test_head_backward_workspace_is_bounded():
    """P never takes more than 128 MB or 256 columns, whatever the vocabulary."""
    for T in (1, 100, 4096, 65536, 1 << 20):
        for V in (100, 50304, 1 << 21):
            n = L.nf4moe_vocab_workspace_bytes(head_desc(H=64, V=V), T, 0, 1)
            if not n:       # too many tiles
                continue
            P = max(128 << 20, 2 * 256 * T)
            assert n <= P + 2 * 256 * T + 64 * T * 64 * 4 + T + 4096, (T, V, n)


def test_head_backward_workspace_of_few_rows():
    """Up to 64 rows P has two parts: together at most 128 MB, or 256 columns."""
    for T in (1, 33, 48, 64):
        for V in (100, 50304, 1 << 21):
            n = L.nf4moe_vocab_workspace_bytes(head_desc(H=64, V=V), T, 0, 1)
            # x twice and dx's parts of two rows a row, 64 slices at most
            assert 0 < n <= (128 << 20) + 2 * T * 64 * 2 + 64 * 2 * T * 64 * 4 + 4096, (T, V, n)


def test_head_rows_past_a_dispatch_are_refused():
    for f in (ce_fwd, ce_bwd, ds_fwd, ds_bwd):
        d = head_desc(H=8, V=100)
        assert f(d, T=(1 << 25) + 1) == UNSUPPORTED and "2^25" in L.nf4moe_last_error().decode()
        assert L.nf4moe_vocab_workspace_bytes(d, (1 << 25) + 1, 0, 1) == 0 < L.nf4moe_vocab_workspace_bytes(d, 1 << 25, 0, 1)
        if not GPU:
            # (the arrays lie far apart: none of them is longer than 2^40 bytes)
            assert f(d, T=1 << 25, n=BIG >> 22) == HIP


def ln_desc(H=64, xdt=1, ydt=1, w=far(9), b=far(10), eps=1e-5):
    return dense._LAYER_NORM.pack(H, xdt, ydt, w or 0, b or 0, eps)


def test_layer_norm_validation():
    def fwd(d=None, x=far(0), T=4, y=far(1), mean=far(2), rstd=far(3)):
        return L.nf4moe_layer_norm_forward(ln_desc() if d is None else d, x, T, y, mean, rstd, None)

    def bwd(d=None, dy=far(0), x=far(1), mean=far(2), rstd=far(3), T=4, base=far(4), dx=far(5), dw=far(6), db=far(7), ws=far(8), n=BIG):
        return L.nf4moe_layer_norm_backward(ln_desc() if d is None else d, dy, x, mean, rstd, T, base, dx, dw, db, ws, n, None)
    for f in (fwd, bwd):
        for bad in (dict(H=0), dict(H=16385), dict(xdt=2), dict(ydt=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                    dict(w=far(9) + 2), dict(b=far(10) + 1)):
            assert f(ln_desc(**bad)) == INVALID, bad
        assert f(T=-1) == INVALID and f(T=1 << 31) == INVALID
        for name in ("x", "mean", "rstd"):
            assert f(**{name: None}) == INVALID and f(**{name: far(30) + 1}) == INVALID, name
    assert L.nf4moe_layer_norm_forward(None, far(0), 4, far(1), far(2), far(3), None) == INVALID
    assert fwd(y=None) == INVALID and fwd(T=0, x=None) == OK
    assert bwd(dy=None) == INVALID and bwd(dx=None, dw=None, db=None) == INVALID and bwd(T=0, dw=None, db=None) == OK
    for name in ("dy", "base", "dx"):
        assert bwd(**{name: far(30) + 1}) == INVALID
    assert bwd(dw=far(6) + 2) == INVALID and bwd(db=far(7) + 2) == INVALID
    need = L.nf4moe_layer_norm_workspace_bytes(64, 4)
    assert need > 0 and bwd(n=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE and bwd(ws=far(8) + 8) == INVALID
    assert L.nf4moe_layer_norm_workspace_bytes(64, 0) == 0 and L.nf4moe_layer_norm_workspace_bytes(0, 4) == 0
    if not GPU:
        assert fwd() == HIP and bwd(n=need) == HIP and fwd(ln_desc(w=None, b=None)) == HIP
        assert bwd(n=need, base=far(5)) == HIP         # in place


def overlaps_refused(fn, outs, ins, may_be=()):
    """Every output laid over each input and each other output, by its last and its first bytes: INVALID_ARG."""
    size = {**outs, **ins}
    at = {n: far(i) for i, n in enumerate(size)}
    for o in outs:
        for other in size:
            if other == o or (o, other) in may_be:
                continue
            for shift in {0, size[other] - 256, 256 - size[o]}:
                if shift and (not -size[o] < shift < size[other] or shift % 256):
                    continue
                got = fn(**{**at, o: at[other] + shift})
                assert got == INVALID, (o, other, shift, got)
                msg = L.nf4moe_last_error().decode()
                assert "overlaps" in msg and o in msg.split() and other in msg.split(), msg
    if not GPU:
        assert fn(**at) == HIP, L.nf4moe_last_error()
        o, i = next(iter(outs)), next(iter(ins))
        assert fn(**{**at, o: at[i] + size[i]}) == HIP and fn(**{**at, o: at[i] - size[o]}) == HIP


def test_outputs_over_other_arrays_are_refused():
    T, H, I, V, k = 256, 512, 256, 1024, 16
    d = lambda w13: ffn_desc(H, I, w13)  # noqa: E731
    overlaps_refused(lambda x, w13, h: L.nf4moe_gated_ffn_forward(d(w13), x, T, h, None), dict(h=2 * T * I), dict(x=2 * T * H, w13=4 * I * H))
    need = L.nf4moe_gated_ffn_workspace_bytes(ffn_desc(H, I), T)
    overlaps_refused(lambda dh, x, w13, dx, dw13, h, workspace: L.nf4moe_gated_ffn_backward(d(w13), dh, x, T, dx, dw13, h, workspace, need, None),
                     dict(dx=2 * T * H, dw13=4 * I * H, h=2 * T * I, workspace=need), dict(dh=2 * T * I, x=2 * T * H, w13=4 * I * H))
    d = lambda w: head_desc(H, V, w)  # noqa: E731
    n0, n1, m0, m1 = (L.nf4moe_vocab_workspace_bytes(head_desc(H, V), T, e, b) for e in (0, k) for b in (0, 1))
    xw = dict(x=2 * T * H, w=2 * V * H)
    overlaps_refused(lambda x, w, labels, loss, lse, workspace: ce_fwd(d(w), x, T, labels, loss, lse, workspace, n0),
                     dict(loss=4 * T, lse=4 * T, workspace=n0), dict(**xw, labels=4 * T))
    overlaps_refused(lambda x, w, ids, dloss, lse, dx, dw, workspace: ce_bwd(d(w), dloss, x, T, ids, lse, dx, dw, workspace, n1),
                     dict(dx=2 * T * H, dw=2 * V * H, workspace=n1), dict(**xw, ids=4 * T, dloss=4 * T, lse=4 * T))
    e = 4 * T * k
    overlaps_refused(lambda x, w, ids, teacher, loss, lse, q, logits, workspace: ds_fwd(
        d(w), x, T, ids, teacher, 0, k, 1.0, loss, lse, q, logits, workspace, m0),
        dict(loss=4 * T, lse=4 * T, q=e, logits=e, workspace=m0), dict(**xw, ids=e, teacher=e))
    overlaps_refused(lambda x, w, ids, q, logits, dloss, lse, dx, dw, workspace: ds_bwd(
        d(w), dloss, x, T, ids, q, logits, lse, k, 1.0, dx, dw, workspace, m1),
        dict(dx=2 * T * H, dw=2 * V * H, workspace=m1), dict(**xw, ids=e, q=e, logits=e, dloss=4 * T, lse=4 * T))
    for xdt, ydt in ((0, 1), (1, 0)):
        xb, yb = T * H * (4 - 2 * xdt), T * H * (4 - 2 * ydt)
        d = lambda w, b=None: ln_desc(H, xdt, ydt, w, b)  # noqa: E731, B023
        overlaps_refused(lambda x, w, b, y, mean, rstd: L.nf4moe_layer_norm_forward(d(w, b), x, T, y, mean, rstd, None),
                         dict(y=yb, mean=4 * T, rstd=4 * T), dict(x=xb, w=4 * H, b=4 * H))
        need = L.nf4moe_layer_norm_workspace_bytes(H, T)
        overlaps_refused(lambda dy, x, mean, rstd, dx_base, w, dx, dw, db, workspace: L.nf4moe_layer_norm_backward(
            d(w), dy, x, mean, rstd, T, dx_base, dx, dw, db, workspace, need, None),
            dict(dx=xb, dw=4 * H, db=4 * H, workspace=need), dict(dy=yb, x=xb, mean=4 * T, rstd=4 * T, dx_base=xb, w=4 * H),
            may_be=[("dx", "dx_base")])


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_before_the_device():
    M, z = pkg, lambda *s, dt=BF16: torch.zeros(*s, dtype=dt)  # noqa: E731
    x, w, w13, lab, ids, v = z(4, 16), z(30, 16), z(48, 16), z(4, dt=I32), z(4, 3, dt=I32), z(4, dt=F32)
    e = z(4, 3, dt=F32)
    bad = [
        (TypeError, lambda: M.gated_ffn_forward([1], w13)), (TypeError, lambda: M.gated_ffn_forward(x.float(), w13)),
        (ValueError, lambda: M.gated_ffn_forward(x, z(47, 16))), (ValueError, lambda: M.gated_ffn_forward(x, z(48, 8))),
        (ValueError, lambda: M.gated_ffn_forward(x, w13, out=z(4, 23))), (TypeError, lambda: M.gated_ffn_forward(x, w13, out=z(4, 24, dt=F32))),
        (ValueError, lambda: M.gated_ffn_forward(z(16, 4).T, w13)), (ValueError, lambda: M.gated_ffn_forward(x[0], w13)),
        (ValueError, lambda: M.gated_ffn_backward(z(4, 23), x, w13)), (ValueError, lambda: M.gated_ffn_backward(z(4, 24), x, w13, need=("dw",))),
        (ValueError, lambda: M.gated_ffn_backward(z(4, 24), x, w13, need=())),
        (ValueError, lambda: M.vocab_ce_forward(x, z(30, 8), lab)), (TypeError, lambda: M.vocab_ce_forward(x, w, lab.long())),
        (ValueError, lambda: M.vocab_ce_forward(x, w, lab[:3])), (ValueError, lambda: M.vocab_ce_backward(v[:3], x, w, lab, v)),
        (TypeError, lambda: M.vocab_ce_backward(v.double(), x, w, lab, v)), (ValueError, lambda: M.vocab_ce_backward(v, x, w, lab, v, need=("dh",))),
        (ValueError, lambda: M.vocab_distill_forward(x, w, ids, e[:, :2])), (TypeError, lambda: M.vocab_distill_forward(x, w, ids, e.double())),
        (ValueError, lambda: M.vocab_distill_forward(x, w, ids[:3], e)), (ValueError, lambda: M.vocab_distill_forward(x, w, lab, e)),
        (ValueError, lambda: M.vocab_distill_backward(v, x, w, ids, e, e[:3], v)), (TypeError, lambda: M.vocab_distill_backward(v, x, w, ids, e.bfloat16(), e, v)),
        (TypeError, lambda: M.layer_norm_forward(x.double())), (TypeError, lambda: M.layer_norm_forward(x, out_dtype=torch.float16)),
        (TypeError, lambda: M.layer_norm_forward([1.0])), (ValueError, lambda: M.layer_norm_forward(x, z(15, dt=F32))),
        (TypeError, lambda: M.layer_norm_forward(x, z(16))), (ValueError, lambda: M.layer_norm_backward(x[:3], x, v, v)),
        (TypeError, lambda: M.layer_norm_backward(x, x, v, v, dx_base=x.float())), (ValueError, lambda: M.layer_norm_backward(x, x, v, v, need=("dx", "dg"))),
        (ValueError, lambda: M.layer_norm_backward(x, x, v, v, dx_base=x, need=("dw",))), (ValueError, lambda: M.layer_norm_backward(x, x, v[:2], v)),
    ]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
    good = [lambda: M.gated_ffn_forward(x, w13), lambda: M.gated_ffn_backward(z(4, 24), x, w13), lambda: M.vocab_ce_forward(x, w, lab),
            lambda: M.vocab_ce_backward(v, x, w, lab, v), lambda: M.vocab_distill_forward(x, w, ids, e),
            lambda: M.vocab_distill_backward(v, x, w, ids, e, e, v), lambda: M.layer_norm_forward(x),
            lambda: M.layer_norm_backward(x, x, v, v)]
    for f in good:
        with pytest.raises(ValueError, match="on cpu"):
            f()


def test_names_load_on_first_use():
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__)))
    code = ("import sys, bit_quantized_moe_expert_amd as M\n"
            "assert 'torch' not in sys.modules and 'vocab_ce_forward' in dir(M) and not hasattr(M, 'no_such_name')\n"
            "from bit_quantized_moe_expert_amd import layer_norm_forward, gated_ffn_forward\n"
            "assert M.layer_norm_forward is layer_norm_forward is M.dense.layer_norm_forward and M.train.adapter_plan\n")
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)
