"""Adapters of many requests or experts on the GPU against 64-bit references.

Inputs are bf16, products of two bf16 values are exact in fp32, and the low-rank
intermediates enter their second product exactly, so an output differs from the
reference by half a step of its type plus the roundings of fp32 additions: at most
(number of terms) 2^-24 of the sum of the terms' magnitudes, whatever their order."""
import numpy as np
import pytest

import train_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def to_np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(rows, Rn, L, K, N, rank, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    row_of, T = None, Rn
    if rows == "mixed":
        ids = torch.randint(-1, L, (Rn,), generator=g, device=DEV)
    elif rows == "one":
        ids = torch.full((Rn,), L - 1, device=DEV)
    elif rows == "none":
        ids = torch.tensor([-1, L, -7, L + 5, 2 ** 31 - 1, -2 ** 31] * (Rn // 6 + 1), device=DEV)[:Rn]
    else:  # experts: sorted ids, x gathered with repeats
        T = Rn // 4 + 1
        ids = torch.randint(0, L, (Rn,), generator=g, device=DEV).sort().values
        row_of = torch.randint(0, T, (Rn,), generator=g, device=DEV).int()
    return dict(ids=ids.int(), row_of=row_of, x=rn(T, K).bfloat16(), A=(rn(L, rank, K) * K ** -0.5).bfloat16(),
                B=rn(L, N, rank).bfloat16(), scale=torch.rand(L, generator=g, device=DEV) + 0.5, base=rn(Rn, N).to(DT[dt]),
                dy=rn(Rn, N).bfloat16(), dx_base=rn(Rn, K).to(DT[dt]))


CASES = [("mixed", 1, 1, 8, 8, 8, "bf16"), ("mixed", 7, 3, 64, 40, 16, "f32"), ("mixed", 32, 5, 2048, 264, 32, "bf16"),
         ("mixed", 33, 5, 2048, 264, 32, "bf16"), ("experts", 64, 2, 136, 72, 8, "f32"), ("one", 65, 4, 264, 512, 16, "bf16"),
         ("mixed", 129, 40, 320, 1032, 24, "bf16"), ("experts", 1000, 16, 768, 1536, 16, "bf16"),
         ("one", 515, 1, 512, 520, 64, "f32"), ("mixed", 300, 300, 96, 64, 72, "bf16"), ("none", 70, 2, 64, 64, 16, "f32"),
         ("mixed", 200, 3, 2880, 96, 128, "bf16"), ("none", 9, 2, 64, 64, 16, "bf16"), ("experts", 2500, 4, 64, 96, 40, "f32")]


# enough rows for the grouped kernels (the smaller forward calls run in one launch; every backward groups)
GROUPED = [("mixed", 25000, 9, 512, 264, 8, "f32"), ("experts", 9000, 16, 768, 512, 16, "bf16"),
           ("mixed", 5000, 40, 1032, 320, 24, "bf16"), ("one", 2100, 1, 520, 512, 64, "f32"),
           ("mixed", 2600, 300, 520, 264, 72, "bf16"), ("mixed", 700, 3, 2880, 96, 128, "bf16"),
           ("none", 25001, 2, 512, 264, 8, "bf16"), ("mixed", 40000, 50, 104, 520, 32, "f32")]


@pytest.mark.parametrize("rows,Rn,L,K,N,rank,dt", CASES + GROUPED)
def test_forward(rows, Rn, L, K, N, rank, dt):
    v = make(rows, Rn, L, K, N, rank, dt, Rn + K)
    n = {k: to_np(t) for k, t in v.items()}
    ids, row_of = v["ids"].cpu().numpy(), None if v["row_of"] is None else v["row_of"].cpu().numpy()
    ref, t, dm, tm = R.adapter_forward(n["x"], n["A"], n["B"], ids, n["scale"], n["base"], row_of)
    out, tg = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], base=v["base"], scale=v["scale"], x_row_of=v["row_of"],
                                return_t=True)
    R.within(to_np(tg), t, K * U * tm + 1e-37, "t")
    bound = np.abs(ref) * R.half_step(dt) + (K + 3 * rank + 8) * U * dm + 2 * U * np.abs(n["base"]) + 1e-37
    R.within(to_np(out), ref, bound, "out")
    none = (ids < 0) | (ids >= L)
    assert torch.equal(out[torch.from_numpy(none).to(DEV)], v["base"][torch.from_numpy(none).to(DEV)])
    # without a base, without scales, in the other type
    other = "f32" if dt == "bf16" else "bf16"
    ref, _, dm, _ = R.adapter_forward(n["x"], n["A"], n["B"], ids, np.ones(L), None, row_of)
    out2 = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], x_row_of=v["row_of"], out_dtype=DT[other])
    R.within(to_np(out2), ref, np.abs(ref) * R.half_step(other) + (K + 3 * rank + 8) * U * dm + 1e-37, "without a base")
    # into the base, with a plan
    plan = M.adapter_plan(v["ids"], L)
    base = v["base"].clone()
    got = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], base=base, out=base, scale=v["scale"], x_row_of=v["row_of"],
                            plan=plan)
    assert got is base and torch.equal(got, out)


@pytest.mark.parametrize("src", ["bf16", M.CKPT_MXINT8, M.CKPT_MXFP8])
@pytest.mark.parametrize("rows,Rn,L,K,N,rank,dt", CASES)
def test_backward(rows, Rn, L, K, N, rank, dt, src):
    if src != "bf16" and K % 32:
        K += 32 - K % 32
    v = make(rows, Rn, L, K, N, rank, dt, Rn + K + 1)
    n = {k: to_np(t) for k, t in v.items()}
    ids, row_of = v["ids"].cpu().numpy(), None if v["row_of"] is None else v["row_of"].cpu().numpy()
    _, t = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], x_row_of=v["row_of"], return_t=True)
    x, xn = v["x"], n["x"]
    if src != "bf16":
        x = M.ckpt8_quantize(v["x"], src)
        xn = R.ckpt8(n["x"], src)[2]
    ref, mag = R.adapter_backward(n["dy"], xn, to_np(t), n["A"], n["B"], ids, n["scale"], n["dx_base"], row_of)
    kw = dict(scale=v["scale"], x_row_of=v["row_of"])
    got = M.adapter_backward(v["dy"], x, t, v["A"], v["B"], v["ids"], dx_base=v["dx_base"], **kw)
    terms = N + 3 * rank + 8
    R.within(to_np(got["dx"]), ref["dx"], np.abs(ref["dx"]) * R.half_step(dt) + terms * U * mag["dx"] + 2 * U * np.abs(n["dx_base"]) + 1e-37, "dx")
    most = max([len(r) for r in R.adapter_rows(ids, L).values()], default=0)
    R.within(to_np(got["dA"]), ref["dA"], (N + 3 * most + 8) * U * mag["dA"], "dA")
    R.within(to_np(got["dB"]), ref["dB"], (3 * most + 8) * U * mag["dB"], "dB")
    plan = M.adapter_plan(v["ids"], L)
    again = M.adapter_backward(v["dy"], x, t, v["A"], v["B"], v["ids"], dx_base=v["dx_base"], plan=plan, **kw)
    assert all(torch.equal(got[k], again[k]) for k in got)        # a fixed order of every sum, with a plan or without
    for need in (("dx",), ("dA",), ("dB",)):
        one = M.adapter_backward(v["dy"], x if "dA" in need else None, t if "dB" in need else None, v["A"], v["B"], v["ids"],
                                 scale=v["scale"], x_row_of=v["row_of"], dx_base=v["dx_base"], need=need)
        assert set(one) == set(need) and torch.equal(one[need[0]], got[need[0]])


# every number of K slices, both heights of an expansion block, several chunks of an adapter
LARGE = [("mixed", 9000, 9, 1032, 264, 48, "bf16"), ("experts", 17000, 12, 776, 280, 40, "f32"),
         ("one", 16500, 3, 1544, 136, 16, "bf16"), ("mixed", 4100, 5, 3208, 264, 32, "f32"),
         ("mixed", 1300, 3, 3208, 520, 8, "bf16"), ("mixed", 5000, 7, 1032, 2056, 64, "bf16"),
         ("experts", 8200, 6, 640, 136, 128, "f32"), ("one", 20000, 2, 520, 392, 24, "bf16")]


@pytest.mark.parametrize("rows,Rn,L,K,N,rank,dt", LARGE)
def test_forward_of_many_rows(rows, Rn, L, K, N, rank, dt):
    test_forward(rows, Rn, L, K, N, rank, dt)


@pytest.mark.parametrize("src", ["bf16", M.CKPT_MXINT8, M.CKPT_MXFP8])
@pytest.mark.parametrize("rows,Rn,L,K,N,rank,dt", LARGE)
def test_backward_of_many_rows(rows, Rn, L, K, N, rank, dt, src):
    test_backward(rows, Rn, L, K, N, rank, dt, src)


@pytest.mark.parametrize("Rn,L", [(1500, 7), (5000, 4096), (70000, 900), (70000, 4096)])
def test_grouping_of_many_rows_and_adapters(Rn, L):
    """Every row meets its own adapter, and sums over rows see each row once."""
    g = torch.Generator(device=DEV).manual_seed(Rn + L)
    ids = torch.randint(-1, L, (Rn,), generator=g, device=DEV).int()
    x = torch.zeros(Rn, 8, device=DEV, dtype=torch.bfloat16)
    x[:, 0] = 1
    A = torch.zeros(L, 8, 8, device=DEV, dtype=torch.bfloat16)
    A[:, 0, 0] = 1
    B = torch.zeros(L, 8, 8, device=DEV, dtype=torch.bfloat16)
    lid = torch.arange(L, device=DEV)
    B[:, 0, 0], B[:, 1, 0] = (lid // 64).bfloat16(), (lid % 64 + 1).bfloat16()      # the id in two exact digits
    out, t = M.adapter_forward(x, A, B, ids, out_dtype=torch.float32, return_t=True)
    live = ids >= 0
    assert torch.equal(out[:, 0], torch.where(live, ids // 64, 0).float())
    assert torch.equal(out[:, 1], torch.where(live, ids % 64 + 1, 0).float())
    back = M.adapter_backward(out.bfloat16(), x, t, A, B, ids, need=("dB",))
    counts = torch.bincount(ids[live].long(), minlength=L).float()
    assert torch.equal(back["dB"][:, 1, 0], counts * (lid % 64 + 1))
    assert torch.equal(back["dB"][:, 0, 0], counts * (lid // 64))


def test_nonfinite_rows_stay_their_own():
    """A NaN or an infinity in one row's x reaches that row's output and its own adapter's gradients only."""
    for Rn in (20, 8000):       # in one launch, and grouped
        v = make("mixed", Rn, 4, 512, 1024, 16, "bf16", 5)
        v["ids"][:] = torch.arange(Rn, device=DEV) % 4
        v["x"][6, 3] = float("nan")        # adapter 2
        v["x"][Rn - 1, 5] = float("inf")   # adapter 3, the last place of its tile
        out, t = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], base=v["base"], return_t=True)
        bad = ~torch.isfinite(out).all(1)
        assert bad.nonzero().flatten().tolist() == [6, Rn - 1]
        dy = torch.ones_like(v["dy"])
        g = M.adapter_backward(dy, v["x"], t, v["A"], v["B"], v["ids"])
        assert torch.isfinite(g["dx"]).all()
        assert [bool(torch.isfinite(g["dA"][l]).all()) for l in range(4)] == [True, True, False, False]
        # column 5 is not finite: u = h + m + l in three parts, and h inf + m inf + l inf is a NaN where the parts
        # differ in sign or one is 0, else an infinity
        assert torch.isfinite(g["dA"][3][:, 6:]).all() and not torch.isfinite(g["dA"][3][:, 5]).any()
        assert [bool(torch.isfinite(g["dB"][l]).all()) for l in range(4)] == [True, True, False, False]
    # an infinite weight of one adapter stays with that adapter
    v = make("mixed", 8000, 3, 512, 1024, 24, "bf16", 6)
    v["B"][1, 7, 23] = float("inf")
    out = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], base=v["base"])
    assert torch.isfinite(out[v["ids"] != 1]).all() and torch.isfinite(out[:, :7]).all() and torch.isfinite(out[:, 8:]).all()


def test_gather_indices_are_clamped():
    for Rn in (100, 9000):
        _gather_clamped(make("experts", Rn, 4, 512, 1024, 16, "bf16", 8))


def _gather_clamped(v):
    ok = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], x_row_of=v["row_of"])
    T = v["x"].shape[0]
    wild = v["row_of"].clone()
    wild[3], wild[50] = -5, T + 1000
    got = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], x_row_of=wild)
    same = torch.ones(len(wild), dtype=torch.bool, device=DEV)
    same[[3, 50]] = False
    assert torch.equal(got[same], ok[same])


def test_empty():
    v = make("mixed", 8, 3, 64, 64, 16, "f32", 9)
    e = {k: (t[:0] if k in ("ids", "x", "base", "dy", "dx_base") else t) for k, t in v.items()}
    out, t = M.adapter_forward(e["x"], e["A"], e["B"], e["ids"], base=e["base"], return_t=True)
    assert tuple(out.shape) == (0, 64) and tuple(t.shape) == (0, 16)
    g = M.adapter_backward(e["dy"], e["x"], t, e["A"], e["B"], e["ids"])
    assert torch.count_nonzero(g["dA"]) == 0 and torch.count_nonzero(g["dB"]) == 0 and tuple(g["dx"].shape) == (0, 64)
    assert M.adapter_plan(e["ids"], 3).R == 0


def test_misaligned_views():
    v = make("mixed", 4000, 5, 1032, 520, 24, "bf16", 11)

    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)
    o = {k: off(t) if t is not None and t.dtype == torch.bfloat16 else t for k, t in v.items()}
    for k in (4000, 20):    # the grouped kernels and the one for few rows
        a = M.adapter_forward(v["x"][:k], v["A"], v["B"], v["ids"][:k], base=v["base"][:k])
        b = M.adapter_forward(o["x"][:k], o["A"], o["B"], o["ids"][:k], base=o["base"][:k])
        assert torch.equal(a, b)
    _, t = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], return_t=True)
    a = M.adapter_backward(v["dy"], v["x"], t, v["A"], v["B"], v["ids"], dx_base=v["dx_base"])
    b = M.adapter_backward(o["dy"], o["x"], t, o["A"], o["B"], o["ids"], dx_base=o["dx_base"])
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_captured_and_replayed():
    v = make("experts", 7000, 9, 1024, 320, 16, "bf16", 12)
    few = make("mixed", 6, 9, 1024, 320, 16, "bf16", 13)

    def step():
        out, t = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], base=v["base"], scale=v["scale"], x_row_of=v["row_of"],
                                   return_t=True)
        g = M.adapter_backward(v["dy"], v["x"], t, v["A"], v["B"], v["ids"], scale=v["scale"], x_row_of=v["row_of"],
                               dx_base=v["dx_base"])
        small = M.adapter_forward(few["x"], v["A"], v["B"], few["ids"], base=few["base"])
        return [out, t, small, *[g[k] for k in sorted(g)]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):          # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for k in range(4):
        v["x"].copy_(torch.randn_like(v["x"]))
        v["ids"].copy_(torch.randint(-1, 9, (7000,), device=DEV).int())      # other groups, other tables
        few["ids"].copy_(torch.randint(-1, 9, (6,), device=DEV).int())
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, eager)), k


def test_two_streams_at_once():
    vs = [make("mixed", 12000, 12, 512, 512, 16, "bf16", 20 + i) for i in range(2)]

    def step(v):
        out, t = M.adapter_forward(v["x"], v["A"], v["B"], v["ids"], base=v["base"], return_t=True)
        g = M.adapter_backward(v["dy"], v["x"], t, v["A"], v["B"], v["ids"])
        return [out, *[g[k] for k in sorted(g)]]
    want = [step(v) for v in vs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in vs]
    for _ in range(3):
        got = []
        for st, v in zip(streams, vs):
            with torch.cuda.stream(st):
                got.append(step(v))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


def test_offsets_past_32_bits():
    """Base and out of more than 2^31 elements: the last rows are right."""
    Rn, N, K, rank = 70000, 32768, 32, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(Rn, K, generator=g, device=DEV).bfloat16()
    A, B = torch.randn(2, rank, K, generator=g, device=DEV).bfloat16(), torch.randn(2, N, rank, generator=g, device=DEV).bfloat16()
    ids = (torch.arange(Rn, device=DEV) % 2).int()
    base = torch.ones(Rn, N, device=DEV, dtype=torch.bfloat16)
    M.adapter_forward(x, A, B, ids, base=base, out=base)
    rows = [0, 1, 65535, 65536, Rn - 2, Rn - 1]
    for r in rows:
        l = r % 2
        ref = 1.0 + to_np(B[l]) @ (to_np(A[l]) @ to_np(x[r]))
        mag = np.abs(to_np(B[l])) @ (np.abs(to_np(A[l])) @ np.abs(to_np(x[r])))
        R.within(to_np(base[r]), ref, np.abs(ref) * 2.0 ** -8 + (K + 32) * U * (mag + 1), f"row {r}")
