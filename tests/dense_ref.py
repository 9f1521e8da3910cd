"""64-bit references of the dense operators (torch float64, on the inputs' device), written
from their definitions; nothing here is shared with the library."""
import torch

F64 = torch.float64
INF = float("inf")


def within(got, ref, bound, what):
    """Elementwise |got - ref| <= bound; NaN and infinities exactly where the reference has them."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities"
    err = (got - ref).abs()[fine]
    b = torch.as_tensor(bound, dtype=F64, device=ref.device).expand(ref.shape)[fine]
    if (err > b).any():
        i = int((err - b).argmax())
        raise AssertionError(f"{what}: {int((err > b).sum())} of {err.numel()} outside; worst {err[i]:.3e} > {b[i]:.3e} "
                             f"(ref {ref[fine][i]:.6e})")


def off(got, ref):
    """Relative distance in the 2-norm."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    n = ref.norm()
    return float((got - ref).norm() / n) if n > 0 else float(got.abs().max()) if got.numel() else 0.0


# ------------------------------------------------------------------ gated feed-forward
def split(w13, inter):
    return (w13[0::2], w13[1::2]) if inter else (w13[:w13.shape[0] // 2], w13[w13.shape[0] // 2:])


def join(g, u, inter):
    return torch.stack([g, u], 1).flatten(0, 1) if inter else torch.cat([g, u])


def act(g, u, glu, alpha, limit):
    """h and its derivatives by g and u."""
    if glu == 0:
        s = torch.sigmoid(g)
        return g * s * u, u * (s + g * s * (1 - s)), g * s
    gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    s = torch.sigmoid(alpha * gc)
    return (uc + 1) * gc * s, (g <= limit) * (uc + 1) * (s + alpha * gc * s * (1 - s)), (u.abs() <= limit) * gc * s


def ffn(x, w13, glu, alpha, limit, inter):
    """g, u, h and h's derivatives."""
    x, (wg, wu) = x.double(), split(w13.double(), inter)
    g, u = x @ wg.T, x @ wu.T
    return g, u, *act(g, u, glu, alpha, limit)


def ffn_grad(dh, x, w13, glu, alpha, limit, inter):
    """dg, du, dx, dw13."""
    _, _, _, by_g, by_u = ffn(x, w13, glu, alpha, limit, inter)
    x, (wg, wu) = x.double(), split(w13.double(), inter)
    dg, du = dh.double() * by_g, dh.double() * by_u
    return dg, du, dg @ wg + du @ wu, join(dg.T @ x, du.T @ x, inter)


# ------------------------------------------------------------------ losses of a head
def ce(x, w, labels):
    l = x.double() @ w.double().T
    on = (labels >= 0) & (labels < w.shape[0])
    lse = torch.logsumexp(l, 1)
    at = l.gather(1, torch.where(on, labels, 0).long()[:, None])[:, 0]
    return torch.where(on, lse - at, 0.0), lse


def ce_P(dloss, x, w, labels):
    """The gradient of the logits; rows without a label zero whatever they hold."""
    on = (labels >= 0) & (labels < w.shape[0])
    l = torch.where(on[:, None], x.double(), 0.0) @ w.double().T
    P = torch.softmax(l, 1)
    P[torch.arange(len(on), device=on.device)[on], labels[on].long()] -= 1
    return P * torch.where(on, dloss.double(), 0.0)[:, None]


def teacher(ids, t, V, tau):
    """(q with an id's probabilities in its first place, which rows count)."""
    on = (ids >= 0) & (ids < V)
    t = torch.where(on, t.double(), -INF)
    m = t.amax(1, keepdim=True)
    row = m[:, 0] > -INF
    e = torch.where(on & row[:, None], torch.exp((t - torch.where(row[:, None], m, 0.0)) / tau), 0.0)
    e = torch.where(torch.isnan(t).any(1, keepdim=True) & on, torch.nan, e)
    row = row | torch.isnan(e).any(1)
    q = e / torch.where(row, e.sum(1), 1.0)[:, None]
    same = (ids[:, :, None] == ids[:, None, :]) & on[:, :, None]          # [T, k, k]
    first = same.long().argmax(2) == torch.arange(ids.shape[1], device=ids.device)
    return torch.where(on & first, (same * q[:, None, :]).sum(2), 0.0), row


def distill(x, w, ids, t, tau):
    """loss, lse, q, logits."""
    V = w.shape[0]
    q, row = teacher(ids, t, V, tau)
    l = x.double() @ w.double().T
    on = (ids >= 0) & (ids < V)
    at = torch.where(on, l.gather(1, torch.where(on, ids, 0).long()), 0.0)
    lse = torch.where(row, torch.logsumexp(l / tau, 1), INF)
    terms = torch.where(q == 0, 0.0, q * (torch.log(q) - at / tau + torch.where(row, lse, 0.0)[:, None]))
    return tau * tau * terms.sum(1), lse, q, at


def distill_P(dloss, x, w, ids, q, row, tau):
    P = torch.softmax(torch.where(row[:, None], x.double(), 0.0) @ w.double().T / tau, 1)
    P = P.scatter_add(1, torch.where(q != 0, ids, 0).long(), -q.double())
    return P * torch.where(row, dloss.double() * tau, 0.0)[:, None]


# ------------------------------------------------------------------ layer norm
def layer_norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = ((x - mean[:, None]).square().mean(1) + eps) ** -0.5
    y = (x - mean[:, None]) * rstd[:, None]
    y = y if w is None else y * w.double()
    return y if b is None else y + b.double(), mean, rstd


def layer_norm_grad(dy, x, mean, rstd, w, base):
    n, dy = (x.double() - mean.double()[:, None]) * rstd.double()[:, None], dy.double()
    a = dy if w is None else dy * w.double()
    dx = rstd.double()[:, None] * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    return dx if base is None else dx + base.double(), (dy * n).sum(0), dy.sum(0)
