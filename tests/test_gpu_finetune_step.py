"""One fine-tuning step of a whole block on frozen 4-bit experts, through the
library's calls only where it has them: pre norm -> routing -> 4-bit gate_up with an
adapter per expert -> gated activation (saved in 8 bits) -> 4-bit down with an adapter
per expert -> combine -> post norm, gate, residual and the next pre norm; then back
through all of it. Against 64-bit autograd of the same block on the decoded weights.

What separates the two, relative to a tensor's norm: a bf16 rounding is 2^-8 / sqrt(3)
or less of each value (0.23 %, about eight of them on the longest path: 0.65 %), and an
MXINT8 value is off by a step 2^(X - 6) uniformly, 2^-6 / sqrt(12) = 0.45 % of the
block's largest power of two, which is at most 2.6 rms for blocks of 32 of these
near-normal values: 1.2 % for each of the two tensors held (the layer input and
gate_up; gate_up enters twice, as g and u). Together below 2.3 %; the bounds are 1 % for
the forward and 3 % for the gradients."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402

DEV = "cuda"


def off(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    return float((got - ref).norm() / ref.norm())


class Block:
    def __init__(self, fmt, glu, inter, seed, T=72, H=128, I=64, E=6, k=2, rank=8):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
        self.fmt, self.T, self.H, self.I, self.E, self.k = fmt, T, H, I, E, k
        self.glu = dict(glu=glu, alpha=1.702 if glu else 0.0, limit=7.0 if glu else 0.0, interleaved=inter)
        self.p13, self.s13 = M.quantize(rn(E, 2 * I, H, std=0.1), fmt)
        self.p2, self.s2 = M.quantize(rn(E, H, I, std=0.1), fmt)
        self.router_w = rn(E, H, std=0.2)
        self.A13, self.B13 = rn(E, rank, H, std=0.1).bfloat16(), rn(E, 2 * I, rank, std=0.2).bfloat16()
        self.A2, self.B2 = rn(E, rank, I, std=0.1).bfloat16(), rn(E, H, rank, std=0.2).bfloat16()
        self.scale = torch.full((E,), 0.5, device=DEV)
        self.w_in, self.w_post, self.w_next = (1 + rn(H, std=0.1) for _ in range(3))
        self.gate, self.alpha, self.eps = rn(H), 0.7, 1e-6
        self.x = rn(T, H).bfloat16()
        self.dx_new, self.dy_next = rn(T, H).bfloat16(), rn(T, H).bfloat16()

    def step(self):
        T, H, I, E, k = self.T, self.H, self.I, self.E, self.k
        kw = dict(scale=self.scale)
        pre = M.block_norm_forward(self.x, w_pre=self.w_in, eps=self.eps)
        y = pre["y"]
        held_y = M.ckpt8_quantize(y)
        r = M.route_permute(M.router_logits(y, self.router_w), k)
        slots = r["sorted_slots"].long()
        tok, ids = (slots // k).int(), r["topk_ids"].reshape(-1)[slots].contiguous()
        w = r["topk_w"].reshape(-1)[slots].contiguous()
        off_, plan = r["expert_offsets"], M.adapter_plan(ids, E)
        gu = M.grouped_gemm(y, self.p13, self.s13, off_, H, T * k, a_row_of=tok, fmt=self.fmt, out_dtype=torch.bfloat16)
        gu, t13 = M.adapter_forward(y, self.A13, self.B13, ids, base=gu, out=gu, x_row_of=tok, plan=plan, return_t=True, **kw)
        h, held = M.glu_forward(gu, ckpt=M.CKPT_MXINT8, **self.glu)
        dn = M.grouped_gemm(h, self.p2, self.s2, off_, I, T * k, fmt=self.fmt)
        dn, t2 = M.adapter_forward(h, self.A2, self.B2, ids, base=dn, plan=plan, return_t=True, **kw)
        by_slot = torch.empty_like(dn)
        by_slot[slots] = dn * w[:, None]
        f = by_slot.view(T, k, H).sum(1).bfloat16()
        nkw = dict(w_post=self.w_post, w_pre=self.w_next, gate=self.gate, gate_fn=M.GATE_SIGMOID, alpha=self.alpha)
        out = M.block_norm_forward(self.x, f, eps=self.eps, **nkw)
        # back
        nb = M.block_norm_backward(self.dx_new, self.dy_next, out["x"], f, rstd_post=out["rstd_post"], rstd_pre=out["rstd_pre"], **nkw)
        d = nb["df"][tok.long()].contiguous()
        dh = M.grouped_dgrad(d, self.p2, self.s2, off_, I, fmt=self.fmt)
        dh = M.adapter_backward(d, None, None, self.A2, self.B2, ids, dx_base=dh, dx=dh, plan=plan, need=("dx",), **kw)["dx"]
        gb = M.glu_backward(dh, held, row_w=w, **self.glu)
        g2 = M.adapter_backward((d * w[:, None]).bfloat16(), gb["h"], t2, self.A2, self.B2, ids, plan=plan, need=("dA", "dB"), **kw)
        dr = M.grouped_dgrad(gb["dgu"], self.p13, self.s13, off_, H, fmt=self.fmt)
        g13 = M.adapter_backward(gb["dgu"], held_y, t13, self.A13, self.B13, ids, x_row_of=tok, dx_base=dr, plan=plan, **kw)
        rows = torch.empty_like(g13["dx"])
        rows[slots] = g13["dx"]
        dy = rows.view(T, k, H).sum(1).bfloat16()
        first = M.block_norm_backward(nb["dx"], dy, self.x, rstd_pre=pre["rstd_pre"], w_pre=self.w_in)
        self.routing = (tok, ids, w)
        return dict(x=out["x"], y=out["y"], dx=first["dx"], dw_in=first["dw_pre"], dw_post=nb["dw_post"], dw_next=nb["dw_pre"],
                    dgate=nb["dgate"], drow_w=gb["drow_w"], dA13=g13["dA"], dB13=g13["dB"], dA2=g2["dA"], dB2=g2["dB"])

    def reference(self):
        """The same block in 64 bits on the CPU, differentiated by autograd (the routing as the GPU had it)."""
        D = lambda t: t.detach().double().cpu()  # noqa: E731
        leaf = lambda t: D(t).requires_grad_()  # noqa: E731
        W13, W2 = D(M.dequantize(self.p13, self.s13, self.H, self.fmt)), D(M.dequantize(self.p2, self.s2, self.I, self.fmt))
        tok, ids, w = (t.cpu() for t in self.routing)
        tok, ids = tok.long(), ids.long()
        v = {n: leaf(getattr(self, n)) for n in ("x", "A13", "B13", "A2", "B2", "w_in", "w_post", "w_next", "gate")}
        w = w.double().requires_grad_()
        norm = lambda a: a / torch.sqrt((a * a).mean(1, keepdim=True) + self.eps)  # noqa: E731
        y = norm(v["x"]) * v["w_in"]
        yr = y[tok]
        lin = lambda a, Wt, A, B: (torch.einsum("rk,rnk->rn", a, Wt[ids])  # noqa: E731
                                   + 0.5 * torch.einsum("rj,rnj->rn", torch.einsum("rk,rjk->rj", a, A[ids]), B[ids]))
        gu = lin(yr, W13, v["A13"], v["B13"])
        g, u = (gu[:, 0::2], gu[:, 1::2]) if self.glu["interleaved"] else (gu[:, :self.I], gu[:, self.I:])
        if self.glu["glu"]:
            g, u = g.clamp(max=7.0), u.clamp(-7.0, 7.0)
            h = (u + 1) * g * torch.sigmoid(1.702 * g)
        else:
            h = torch.nn.functional.silu(g) * u
        f = torch.zeros(self.T, self.H, dtype=torch.float64).index_add(0, tok, w[:, None] * lin(h, W2, v["A2"], v["B2"]))
        x = v["x"] + self.alpha * torch.sigmoid(v["gate"]) * norm(f) * v["w_post"]
        out = norm(x) * v["w_next"]
        ((x * D(self.dx_new)).sum() + (out * D(self.dy_next)).sum()).backward()
        return dict(x=x, y=out, dx=v["x"].grad, dw_in=v["w_in"].grad, dw_post=v["w_post"].grad, dw_next=v["w_next"].grad,
                    dgate=v["gate"].grad, drow_w=w.grad, dA13=v["A13"].grad, dB13=v["B13"].grad, dA2=v["A2"].grad,
                    dB2=v["B2"].grad)


@pytest.mark.parametrize("fmt,glu,inter", [(M.FMT_NF4, 0, 0), (M.FMT_MXFP4, 1, 1)])
def test_step_against_autograd(fmt, glu, inter):
    b = Block(fmt, glu, inter, seed=41 + fmt)
    got = b.step()
    ref = b.reference()
    errs = {n: off(got[n], ref[n]) for n in ref}
    print({n: round(e, 4) for n, e in errs.items()})
    for n, e in errs.items():
        assert e <= (0.01 if n in ("x", "y") else 0.03), (n, errs)


def test_step_repeats_bit_for_bit():
    b = Block(M.FMT_NF4, 0, 0, seed=7)
    one, two = b.step(), b.step()
    assert all(torch.equal(one[n], two[n]) for n in one)
    assert all(np.isfinite(float(one[n].double().sum())) for n in one)
