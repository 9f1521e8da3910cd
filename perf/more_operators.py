"""Cases of the dense bf16 ends of a training step around the 4-bit MoE layer:

- the gated feed-forward beside the routed experts (gate and up projection, activation and
  product), forward, for single tokens too, and backward from x and the weights alone;
- the softmax cross entropy of a vocabulary head, forward and gradient, without keeping logits;
- the distillation of that head from a teacher's top logits, forward and gradient;
- layer norm, forward and backward with the weight's and the bias's gradient.

`run` computes them in plain torch operations in 32 bits (own = False) or through
the library (own = True); `exact` computes them from their definitions in 64 bits.
Shapes are those of the library's own workloads (OLMoE-, Qwen3- and
gpt-oss-shaped layers) or generic.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ALPHA, LIMIT = 1.702, 7.0
INF = float("inf")


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of one token through an OLMoE-shaped shared expert
        dict(name="ffn_decode", op="ffn_fwd", T=1, H=2048, I=1024, glu=0, inter=0),
        # a batch of prompts through a gpt-oss-shaped block, its clamped form and interleaved rows
        dict(name="ffn_prompt", op="ffn_fwd", T=4099, H=2880, I=2880, glu=1, inter=1),
        # training a wide dense block: every gradient
        dict(name="ffn_grad", op="ffn_bwd", T=4096, H=2048, I=8192, glu=0, inter=0),
        # a short ragged fine-tuning batch through a Qwen3-shaped expert
        dict(name="ffn_grad_small", op="ffn_bwd", T=131, H=2048, I=768, glu=0, inter=0),
        # scoring a handful of tokens (perplexity of short answers)
        dict(name="ce_score", op="ce_fwd", T=17, H=2048, V=32003),
        # a training micro-batch of 4096 tokens, prompts masked: the loss
        dict(name="ce_loss", op="ce_fwd", T=4096, H=2048, V=50304),
        # and its gradients, of the hidden states and of the head
        dict(name="ce_grad", op="ce_bwd", T=4096, H=2048, V=50304, dw=True),
        # a 4-bit student learns from its parent's 64 top logits: the loss
        dict(name="distill_loss", op="distill_fwd", T=2048, H=2880, V=50304, k=64, tau=2.0, teacher="bf16"),
        # a short batch through a frozen head: the hidden states' gradient alone
        dict(name="distill_grad", op="distill_bwd", T=515, H=1024, V=32003, k=16, tau=1.0, teacher="f32", dw=False),
        # the norm of one decode step of 4 tokens
        dict(name="ln_decode", op="ln_fwd", T=4, H=2048, x="bf16", y="bf16", affine=True),
        # a long prompt on an fp32 residual stream
        dict(name="ln_prompt", op="ln_fwd", T=8190, H=2880, x="f32", y="bf16", affine=True),
        # training: every gradient, the residual's added
        dict(name="ln_grad", op="ln_bwd", T=8192, H=2048, x="bf16", y="bf16", affine=True, base=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_bwd", "ce_fwd", "ce_bwd", "distill_fwd", "distill_bwd", "ln_fwd", "ln_bwd"])
    if op in ("ffn_fwd", "ffn_bwd"):
        return dict(op=op, T=_log(rng, 1, 4096), H=8 * _log(rng, 16, 360), I=8 * _log(rng, 8, 512),
                    glu=rng.choice([0, 1]), inter=rng.choice([0, 1]))
    if op in ("ln_fwd", "ln_bwd"):
        c = dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 64, 2880), x=rng.choice(["bf16", "f32"]),
                 y=rng.choice(["bf16", "f32"]), affine=rng.random() < 0.8)
        if op == "ln_bwd":
            c["base"] = rng.random() < 0.5
        return c
    V, H = _log(rng, 500, 50304), 8 * _log(rng, 16, 360)
    c = dict(op=op, T=_log(rng, 1, min(4096, 4096 * 50304 * 2048 // (V * H))), H=H, V=V)
    if op in ("ce_bwd", "distill_bwd"):
        c["dw"] = rng.random() < 0.6
    if op in ("distill_fwd", "distill_bwd"):
        c.update(k=_log(rng, 1, 128), tau=round(rng.uniform(0.5, 4.0), 2), teacher=rng.choice(["bf16", "f32"]))
    return c


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


def _randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _dtype(name):
    return BF16 if name == "bf16" else F32


def prepare(case, seed):
    g, c = _gen(seed), case
    op, T, H = c["op"], c["T"], c["H"]
    s = dict(case=c)
    if op in ("ffn_fwd", "ffn_bwd"):
        s.update(x=_randn(g, T, H, dtype=BF16), w=_randn(g, 2 * c["I"], H, std=1.5 * H ** -0.5, dtype=BF16))
        if op == "ffn_bwd":
            s["dh"] = _randn(g, T, c["I"], std=0.1, dtype=BF16)
        return s
    if op in ("ln_fwd", "ln_bwd"):
        shift = _randn(g, 1, H, std=0.5)                               # channels with a mean of their own
        s.update(x=(_randn(g, T, H, std=2.0) + shift + 0.3).to(_dtype(c["x"])), eps=1e-5,
                 w=1 + _randn(g, H, std=0.1) if c["affine"] else None, b=_randn(g, H, std=0.1) if c["affine"] else None)
        if op == "ln_bwd":
            _, s["mean"], s["rstd"] = _ln_fwd(s)                       # what the forward returned
            s["dy"] = _randn(g, T, H, std=0.1, dtype=_dtype(c["y"]))
            s["base"] = _randn(g, T, H, std=0.1, dtype=_dtype(c["x"])) if c["base"] else None
        return s
    V = c["V"]
    s.update(x=_randn(g, T, H, dtype=BF16), w=_randn(g, V, H, std=2.0 * H ** -0.5, dtype=BF16))
    masked = torch.rand(T, generator=g, device=DEV) < 0.15             # prompt and padding positions
    if op in ("ce_fwd", "ce_bwd"):
        labels = torch.randint(0, V, (T,), generator=g, device=DEV)
        s["labels"] = torch.where(masked, torch.full_like(labels, -100), labels).int()
        if op == "ce_bwd":
            s["lse"] = _ce_fwd(s)[1]                                   # what the forward returned
            s["dloss"] = torch.full((T,), 1.0 / T, device=DEV) * (0.5 + torch.rand(T, generator=g, device=DEV))
        return s
    k = min(c["k"], V)
    logits = _logits(s) + _randn(g, T, V)                              # a teacher near the student
    top = logits.topk(k, dim=1)
    del logits
    ids, few = top.indices, torch.rand(T, 1, generator=g, device=DEV) < 0.1
    fewer = torch.arange(k, device=DEV)[None, :] >= (2 * k + 2) // 3   # some rows came with fewer entries
    s["ids"] = torch.where(masked[:, None] | (few & fewer), torch.full_like(ids, -1), ids).int()
    s["teacher"] = top.values.to(_dtype(c["teacher"]))
    if op == "distill_bwd":
        s.update({n: v for n, v in _distill_fwd(s).items() if n != "loss"})   # what the forward returned
        s["dloss"] = torch.full((T,), 1.0 / T, device=DEV) * (0.5 + torch.rand(T, generator=g, device=DEV))
    return s


# ------------------------------------------------------------------ plain forms, in 32 bits
def _halves(gu, inter):
    return (gu[..., 0::2], gu[..., 1::2]) if inter else gu.chunk(2, -1)


def _joined(dg, du, inter):
    return torch.stack([dg, du], -1).reshape(*dg.shape[:-1], -1) if inter else torch.cat([dg, du], -1)


def _glu(g, u, glu):
    """h and its derivatives by gate and up."""
    if glu == 0:
        s = 1 / (1 + torch.exp(-g))
        return g * s * u, u * s * (1 + g * (1 - s)), g * s
    g1, u1 = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    s = 1 / (1 + torch.exp(-ALPHA * g1))
    return ((u1 + 1) * g1 * s, torch.where(g <= LIMIT, (u1 + 1) * s * (1 + ALPHA * g1 * (1 - s)), 0.0),
            torch.where(u.abs() <= LIMIT, g1 * s, 0.0))


def _ffn(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    g, u = _halves(x @ w.T, c["inter"])
    h, by_g, by_u = _glu(g, u, c["glu"])
    if c["op"] == "ffn_fwd":
        return h.to(BF16)
    dh = s["dh"].float()
    dgu = _joined(dh * by_g, dh * by_u, c["inter"])
    return dict(dx=(dgu @ w).to(BF16), dw13=(dgu.T @ x).to(BF16), h=h.to(BF16))


def _logits(s):
    return s["x"].float() @ s["w"].float().T


def _lse(z):
    m = z.amax(1, keepdim=True)
    return torch.log(torch.exp(z - m).sum(1)) + m[:, 0]


def _labels(s):
    y = s["labels"].long()
    return y, (y >= 0) & (y < s["case"]["V"])


def _ce_fwd(s):
    z, (y, on) = _logits(s), _labels(s)
    lse = _lse(z)
    picked = z.gather(1, torch.where(on, y, 0)[:, None])[:, 0]
    return torch.where(on, lse - picked, 0.0), lse


def _grads(s, P):
    out = dict(dx=(P @ s["w"].float()).to(BF16))
    if s["case"]["dw"]:
        out["dw"] = (P.T @ s["x"].float()).to(BF16)
    return out


def _ce_bwd(s):
    P, (y, on) = torch.exp(_logits(s) - s["lse"][:, None]), _labels(s)
    P.scatter_add_(1, torch.where(on, y, 0)[:, None], -torch.ones_like(s["lse"])[:, None])
    return _grads(s, P * torch.where(on, s["dloss"], 0.0)[:, None])


def _distill_fwd(s):
    c = s["case"]
    z = _logits(s) / c["tau"]
    ids = s["ids"].long()
    on = (ids >= 0) & (ids < c["V"])
    row = on.any(1)
    t = torch.where(on, s["teacher"].float() / c["tau"], -INF)
    e = torch.where(on, torch.exp(t - torch.where(row, t.amax(1), 0.0)[:, None]), 0.0)
    q = e / torch.where(row, e.sum(1), 1.0)[:, None]
    at = torch.where(on, z.gather(1, torch.where(on, ids, 0)), 0.0)
    lse = torch.where(row, _lse(z), INF)
    terms = torch.where(q > 0, q * (torch.log(torch.where(q > 0, q, 1.0)) - at + torch.where(row, lse, 0.0)[:, None]), 0.0)
    return dict(loss=c["tau"] ** 2 * terms.sum(1), lse=lse, q=q, logits=at * c["tau"])


def _distill_bwd(s):
    c, ids = s["case"], s["ids"].long()
    P = torch.exp(_logits(s) / c["tau"] - s["lse"][:, None])
    P.scatter_add_(1, torch.where(s["q"] > 0, ids, 0), -s["q"])
    on = torch.isfinite(s["lse"])
    return _grads(s, P * torch.where(on, s["dloss"] * c["tau"], 0.0)[:, None])


def _ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + s["eps"])
    y = d * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"] + s["b"]
    return y.to(_dtype(s["case"]["y"])), mean, rstd


def _ln_bwd(s):
    n, dy = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None], s["dy"].float()
    a = dy if s["w"] is None else dy * s["w"]
    dx = s["rstd"][:, None] * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    if s["base"] is not None:
        dx = dx + s["base"].float()
    out = dict(dx=dx.to(s["x"].dtype))
    if s["w"] is not None:
        out.update(dw=(dy * n).sum(0), db=dy.sum(0))
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import bit_quantized_moe_expert_amd as M
        if op in ("ffn_fwd", "ffn_bwd"):
            kw = dict(glu=c["glu"], alpha=ALPHA, limit=LIMIT, interleaved=c["inter"])
            if op == "ffn_fwd":
                return M.gated_ffn_forward(s["x"], s["w"], **kw)
            return M.gated_ffn_backward(s["dh"], s["x"], s["w"], need=("dx", "dw13", "h"), **kw)
        if op == "ce_fwd":
            return list(M.vocab_ce_forward(s["x"], s["w"], s["labels"]))
        need = ("dx", "dw") if c.get("dw") else ("dx",)
        if op == "ce_bwd":
            return M.vocab_ce_backward(s["dloss"], s["x"], s["w"], s["labels"], s["lse"], need=need)
        if op == "distill_fwd":
            return M.vocab_distill_forward(s["x"], s["w"], s["ids"], s["teacher"], temperature=c["tau"])
        if op == "distill_bwd":
            return M.vocab_distill_backward(s["dloss"], s["x"], s["w"], s["ids"], s["q"], s["logits"], s["lse"],
                                            temperature=c["tau"], need=need)
        if op == "ln_fwd":
            r = M.layer_norm_forward(s["x"], s["w"], s["b"], eps=s["eps"], out_dtype=_dtype(c["y"]))
            return [r["y"], r["mean"], r["rstd"]]
        return M.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], dx_base=s["base"],
                                     need=("dx", "dw", "db") if c["affine"] else ("dx",))
    if op in ("ffn_fwd", "ffn_bwd"):
        return _ffn(s)
    if op == "ce_fwd":
        return list(_ce_fwd(s))
    if op == "ce_bwd":
        return _ce_bwd(s)
    if op == "distill_fwd":
        return _distill_fwd(s)
    if op == "distill_bwd":
        return _distill_bwd(s)
    return list(_ln_fwd(s)) if op == "ln_fwd" else _ln_bwd(s)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    op, T, H = c["op"], c["T"], c["H"]
    x = s["x"].double()
    if op in ("ln_fwd", "ln_bwd"):
        w = torch.ones(H, dtype=F64, device=DEV) if s["w"] is None else s["w"].double()
        if op == "ln_fwd":
            var, mean = torch.var_mean(x, 1, unbiased=False)
            rstd = (var + s["eps"]) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None] * w + (0 if s["b"] is None else s["b"].double())
            return [y, mean, rstd]
        r, dy = s["rstd"].double(), s["dy"].double()
        xc = x - s["mean"].double()[:, None]
        v = dy * w
        dx = r[:, None] * v - (r / H * v.sum(1))[:, None] - xc * (r ** 3 / H * (v * xc).sum(1))[:, None]
        out = dict(dx=dx if s["base"] is None else dx + s["base"].double())
        if s["w"] is not None:
            out.update(dw=torch.einsum("th,th,t->h", dy, xc, r), db=dy.sum(0))
        return out
    w = s["w"].double()
    if op in ("ffn_fwd", "ffn_bwd"):
        I = c["I"]
        wg, wu = (w[0::2], w[1::2]) if c["inter"] else (w[:I], w[I:])
        g, u = x @ wg.T, x @ wu.T
        if c["glu"] == 0:
            sg = torch.sigmoid(g)
            h, by_g, by_u = g * sg * u, u * (sg + g * sg * (1 - sg)), g * sg
        else:
            gm, um = torch.clamp(g, max=LIMIT), torch.clamp(u, -LIMIT, LIMIT)
            sg = torch.sigmoid(ALPHA * gm)
            h, by_u = (um + 1) * gm * sg, (u.abs() <= LIMIT) * gm * sg
            by_g = (g <= LIMIT) * (um + 1) * (sg + ALPHA * gm * sg * (1 - sg))
        if op == "ffn_fwd":
            return h
        dg, du = s["dh"].double() * by_g, s["dh"].double() * by_u
        dw = torch.empty(2 * I, H, dtype=F64, device=DEV)
        if c["inter"]:
            dw[0::2], dw[1::2] = dg.T @ x, du.T @ x
        else:
            dw[:I], dw[I:] = dg.T @ x, du.T @ x
        return dict(dx=dg @ wg + du @ wu, dw13=dw, h=h)
    tau = c.get("tau", 1.0)
    z = x @ w.T / tau
    rows = torch.arange(T, device=DEV)
    if op == "ce_fwd":
        lse = torch.logsumexp(z, 1)
        loss = torch.zeros(T, dtype=F64, device=DEV)
        at = rows[(s["labels"] >= 0) & (s["labels"] < c["V"])]
        loss[at] = lse[at] - z[at, s["labels"][at].long()]
        return [loss, lse]
    if op == "distill_fwd":
        out = dict(loss=torch.zeros(T, dtype=F64, device=DEV), lse=torch.full((T,), INF, dtype=F64, device=DEV),
                   q=torch.zeros(s["ids"].shape, dtype=F64, device=DEV), logits=torch.zeros(s["ids"].shape, dtype=F64, device=DEV))
        on = (s["ids"] >= 0) & (s["ids"] < c["V"])
        at = rows[on.sum(1) > 0]
        t = (s["teacher"].double() / tau).masked_fill(~on, -INF)[at]
        logq = torch.log_softmax(t, 1)
        picked = torch.gather(z[at], 1, s["ids"][at].long().clamp(min=0))
        out["lse"][at] = torch.logsumexp(z[at], 1)
        out["q"][at] = logq.exp()
        out["logits"][at] = torch.where(on[at], picked * tau, 0.0)
        kl = torch.where(on[at], logq.exp() * (torch.where(on[at], logq, 0.0) - picked), 0.0).sum(1)
        out["loss"][at] = tau * tau * (kl + out["lse"][at])
        return out
    P = torch.exp(z - s["lse"].double()[:, None])
    if op == "ce_bwd":
        on = (s["labels"] >= 0) & (s["labels"] < c["V"])
        P[rows[on], s["labels"][on].long()] -= 1
        P *= (on * s["dloss"].double())[:, None]
    else:
        on = s["q"] > 0
        P[rows[:, None].expand_as(on)[on], s["ids"][on].long()] -= s["q"][on].double()
        P *= (on.any(1) * tau * s["dloss"].double())[:, None]
    out = dict(dx=P @ w)
    if c["dw"]:
        out["dw"] = P.T @ x
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    op, T, H = c["op"], c["T"], c["H"]
    if op == "ffn_fwd":
        return dict(bytes=2 * T * H + 4 * c["I"] * H + 2 * T * c["I"], flops=4 * T * H * c["I"])
    if op == "ffn_bwd":     # gate and up again, dx, dw13; dh in, h out
        return dict(bytes=4 * T * H + 8 * c["I"] * H + 4 * T * c["I"], flops=12 * T * H * c["I"])
    if op in ("ln_fwd", "ln_bwd"):
        e, d = (2 if c["x"] == "bf16" else 4), (2 if c["y"] == "bf16" else 4)
        if op == "ln_fwd":
            return dict(bytes=(e + d) * T * H + 8 * T + (8 * H if c["affine"] else 0), flops=8 * T * H)
        return dict(bytes=((3 if c["base"] else 2) * e + d) * T * H + 8 * T + (12 * H if c["affine"] else 0), flops=14 * T * H)
    V, k = c["V"], min(c.get("k", 0), c["V"])
    small = (4 + (2 if c["teacher"] == "bf16" else 4) + 8) * T * k if op == "distill_fwd" else 12 * T * k if op == "distill_bwd" else 4 * T
    if op in ("ce_fwd", "distill_fwd"):
        return dict(bytes=2 * (T + V) * H + small + 8 * T, flops=2 * T * V * H)
    n = 2 if c["dw"] else 1   # products after the logits, which the call does not get
    return dict(bytes=4 * T * H + 2 * n * V * H + small + 8 * T, flops=2 * (n + 1) * T * V * H)
