"""A training step's dense ends together, behind a frozen 4-bit routed layer: the routed layer's
output joins the residual stream, layer norm -> shared gated feed-forward -> down projection
-> residual -> layer norm -> vocabulary head with cross entropy and distillation from a teacher's
top logits; then back through all of it. Against 64-bit autograd of the same block.

What separates the two in a tensor's 2-norm: a rounding to bf16 is 2^-8 / sqrt(3) = 0.23 % or
less. Forward, the longest path to a logit has four (y1, h, the down projection's output, y2),
backward six more (P, dy2, d x2, dh, dgu, dy1): ten that do not know of each other, 0.23 % sqrt(10)
= 0.7 %; twice that for what the activation's and the norms' slopes add."""
import pytest

import dense_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402

DEV = "cuda"
BF16, F64 = torch.bfloat16, torch.float64


class Step:
    def __init__(self, glu, inter, T=193, H=128, I=264, V=3001, k=12):
        g = torch.Generator(device=DEV).manual_seed(17 + glu + 2 * inter)
        rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
        E, Ir = 4, 64
        p13, s13 = M.quantize(rn(E, 2 * Ir, H, std=0.15))
        p2, s2 = M.quantize(rn(E, H, Ir, std=0.15))
        self.layer = M.MoELayer(fmt=0, E=E, H=H, I=Ir, top_k=2, w13=p13, w13_scale=s13, w2=p2, w2_scale=s2, router_w=rn(E, H, std=0.2))
        self.T, self.V, self.tau, self.mix = T, V, 2.0, 0.7
        self.kw = dict(glu=glu, alpha=1.702 if glu else 0.0, limit=7.0 if glu else 0.0, interleaved=inter)
        self.x0 = rn(T, H).to(BF16)
        self.w13, self.w2 = rn(2 * I, H, std=1.2 * H ** -0.5).to(BF16), rn(H, I, std=I ** -0.5).to(BF16)
        self.ln = [1 + rn(H, std=0.1), rn(H, std=0.1), 1 + rn(H, std=0.1), rn(H, std=0.1)]
        self.head = rn(V, H, std=2 * H ** -0.5).to(BF16)
        labels = torch.randint(0, V, (T,), generator=g, device=DEV)
        self.on = torch.rand(T, generator=g, device=DEV) > 0.2
        self.labels = torch.where(self.on, labels, -100).int()
        ids = torch.rand(T, V, generator=g, device=DEV).topk(k, 1).indices
        self.ids = torch.where(self.on[:, None], ids, -1).int()
        self.teacher = rn(T, k, std=2.0)

    def run(self):
        """Loss and gradients through the library."""
        n = self.on.sum()
        x1 = self.x0.float() + M.moe_forward(self.layer, self.x0).float()
        a = M.layer_norm_forward(x1, self.ln[0], self.ln[1], out_dtype=BF16)
        h = M.gated_ffn_forward(a["y"], self.w13, **self.kw)
        x2 = x1 + (h @ self.w2.T).float()
        b = M.layer_norm_forward(x2, self.ln[2], self.ln[3], out_dtype=BF16)
        loss, lse = M.vocab_ce_forward(b["y"], self.head, self.labels)
        d = M.vocab_distill_forward(b["y"], self.head, self.ids, self.teacher, temperature=self.tau)
        total = (loss.sum() + self.mix * d["loss"].sum()) / n
        dloss = torch.ones_like(loss) / n
        p = M.vocab_ce_backward(dloss, b["y"], self.head, self.labels, lse)
        q = M.vocab_distill_backward(dloss * self.mix, b["y"], self.head, self.ids, d["q"], d["logits"], d["lse"], temperature=self.tau)
        dy2 = p["dx"].float() + q["dx"].float()
        nb = M.layer_norm_backward(dy2, x2, b["mean"], b["rstd"], self.ln[2])
        dx2 = nb["dx"]
        dout = dx2.to(BF16)
        g = M.gated_ffn_backward(dout @ self.w2, a["y"], self.w13, need=("dx", "dw13", "h"), **self.kw)
        na = M.layer_norm_backward(g["dx"], x1, a["mean"], a["rstd"], self.ln[0], dx_base=dx2)
        assert torch.equal(g["h"], h)
        return x1, total, dict(x1=na["dx"], w13=g["dw13"], w2=dout.T @ h, ln0=na["dw"], ln1=na["db"], ln2=nb["dw"], ln3=nb["db"],
                               head=p["dw"].double() + q["dw"].double())

    def reference(self, x1):
        v = dict(x1=x1, w13=self.w13, w2=self.w2, head=self.head, **{f"ln{i}": t for i, t in enumerate(self.ln)})
        v = {n: t.double().requires_grad_() for n, t in v.items()}
        norm = lambda x, w, b: torch.nn.functional.layer_norm(x, (x.shape[1],), w, b, 1e-5)  # noqa: E731
        wg, wu = R.split(v["w13"], self.kw["interleaved"])
        y = norm(v["x1"], v["ln0"], v["ln1"])
        g, u = y @ wg.T, y @ wu.T
        h = R.act(g, u, self.kw["glu"], self.kw["alpha"], self.kw["limit"])[0]
        x2 = v["x1"] + h @ v["w2"].T
        logits = (norm(x2, v["ln2"], v["ln3"]) @ v["head"].T)[self.on]
        ce = torch.nn.functional.cross_entropy(logits, self.labels[self.on].long())
        t = torch.log_softmax(self.teacher[self.on].double() / self.tau, 1)
        s = torch.log_softmax(logits / self.tau, 1).gather(1, self.ids[self.on].long())
        total = ce + self.mix * self.tau ** 2 * (t.exp() * (t - s)).sum() / self.on.sum()
        total.backward()
        return total, {n: t.grad for n, t in v.items()}


@pytest.mark.parametrize("glu,inter", [(0, 0), (1, 1)])
def test_training_step(glu, inter):
    s = Step(glu, inter)
    x1, total, got = s.run()
    want_total, want = s.reference(x1)
    assert abs(float(total) / float(want_total) - 1) < 1e-2
    for n, ref in want.items():
        assert R.off(got[n], ref) < 0.015, (n, R.off(got[n], ref))
    again = s.run()
    assert torch.equal(total, again[1]) and all(torch.equal(got[n], again[2][n]) for n in got if n not in ("w2",))
