"""8-bit checkpoints, the gated activation with its backward, and the block norms
on the GPU against 64-bit references.

Codes and scales are exact (compared as integers). A computed output may be off
by half a step of its type, |ref| 2^-8 for bf16 and 2^-24 for fp32, plus the fp32
evaluation error, which scales with the magnitudes of the terms it adds: 2^-24 of
their sum for each rounding on the longest chain (the bound is written at each
check)."""
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


def to_gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(DT[dtype])


def to_np(t):
    return t.detach().double().cpu().numpy()


def off_by_one(t):
    """The same values at an address one element past an aligned one (contiguous, not 16-byte aligned)."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


# ------------------------------------------------------------------ 8-bit checkpoints
def planted(rows, K, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, K)) * np.exp(2 * rng.standard_normal((rows, 1)))).astype(np.float32)
    x[0, :32] = 0.0
    x[0, 1] = -0.0
    if K >= 64 and rows >= 6:
        x[0, 32:64] = np.float32(2.0 ** -140) * rng.integers(-9, 9, 32)     # subnormal block
        x[1, :32] = np.float32(1.7e38) * rng.uniform(-2, 2, 32).astype(np.float32)   # top of the range
        x[1, 32:64] = np.arange(32) / 64 + 1 / 128                           # ties of both formats around 2^-6 ..
        x[1, 63] = 1.0
        x[2, 5] = np.inf
        x[2, 40] = np.nan
        x[3, 7] = -np.inf
        x[4, :32] = np.linspace(440, 511, 32)                                # past e4m3's largest code
        x[5, :32] = np.arange(32) * 2.0 ** -11                               # e4m3 subnormal codes
        x[5, 31] = 1.0
    return x


@pytest.mark.parametrize("fmt", [M.CKPT_MXINT8, M.CKPT_MXFP8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 96), (6, 64), (37, 2048), (5, 2880), (1, 32 * 1031)])
def test_ckpt8_exact(fmt, dtype, rows, K):
    with np.errstate(over="ignore"):
        x = planted(rows, K, rows * 31 + K + fmt)
    xg = to_gpu(x, dtype)
    codes, scale, vals = R.ckpt8(to_np(xg), fmt)
    for t in (xg, off_by_one(xg)):
        ck = M.ckpt8_quantize(t, fmt)
        assert np.array_equal(ck.scale.cpu().numpy(), scale)
        assert np.array_equal(ck.codes.cpu().numpy(), codes)
        back = to_np(M.ckpt8_dequantize(ck, torch.float32))
        assert np.array_equal(back, vals, equal_nan=True)
        b16 = to_np(M.ckpt8_dequantize(ck))
        assert np.array_equal(b16, R.bf16(vals), equal_nan=True)
        big = np.abs(vals) >= 2.0 ** -126
        assert np.array_equal(b16[big], vals[big])                           # exact in bf16


def test_ckpt8_every_e4m3_code_and_int8_code():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).reshape(8, 32).to(DEV)
    for b in (0, 1, 6, 7, 100, 127, 200, 246, 255):
        scale = torch.full((8, 1), b, dtype=torch.uint8, device=DEV)
        f8 = to_np(M.ckpt8_dequantize(M.Ckpt8(codes, scale, M.CKPT_MXFP8), torch.float32))
        i8 = to_np(M.ckpt8_dequantize(M.Ckpt8(codes, scale, M.CKPT_MXINT8), torch.float32))
        n = np.arange(256)
        mag = np.append(R.E4M3, np.nan)[n & 127].reshape(8, 32)
        sgn = np.where(n >= 128, -1.0, 1.0).reshape(8, 32)
        two = np.nan if b == 255 else 2.0 ** (b - 127)
        assert np.array_equal(f8, mag * sgn * two, equal_nan=True), b
        assert np.array_equal(i8, n.astype(np.uint8).view(np.int8).reshape(8, 32) * two / 64, equal_nan=True), b


def test_ckpt8_empty_and_shapes():
    for shape in ((0, 64), (2, 0, 32), (3, 2, 64), (64,)):
        x = torch.randn(shape, device=DEV)
        ck = M.ckpt8_quantize(x)
        assert tuple(ck.codes.shape) == shape and tuple(ck.scale.shape) == shape[:-1] + (shape[-1] // 32,)
        assert tuple(M.ckpt8_dequantize(ck).shape) == shape


# ------------------------------------------------------------------ gated activation
GLU = [(0, 0, 0.0, 0.0), (0, 1, 0.0, 0.0), (1, 0, 1.702, 7.0), (1, 1, 1.702, 7.0)]
LIM = float(np.float32(1.702))


@pytest.mark.parametrize("kind,inter,alpha,limit", GLU)
@pytest.mark.parametrize("Rn,I", [(1, 32), (3, 96), (65, 768), (9, 1024), (7, 2880)])
def test_glu_forward_and_backward(kind, inter, alpha, limit, Rn, I):
    rng = np.random.default_rng(Rn * 131 + I + kind * 7 + inter)
    gu = rng.standard_normal((Rn, 2 * I)) * 4
    gu[0, :8] = [0.0, -0.0, 7.0, -7.0, 60.0, -60.0, 100.0, -100.0]
    gu[0, -8:] = [7.0, 7.0625, -7.0, 6.9375, 0.0, 1.0, -1.0, 30.0]
    dh = rng.standard_normal((Rn, I))
    w = rng.random(Rn)
    wg = to_gpu(w, "f32")
    w = to_np(wg)
    kw = dict(glu=kind, alpha=alpha, limit=limit, interleaved=inter)
    al = LIM if kind else 0.0
    for dt in ("bf16", "f32"):
        g = to_gpu(gu, dt)
        g64 = to_np(g)
        ref = R.glu(g64, kind, al, limit, inter)
        share = (np.abs(R.split(g64, inter)[0]) * 1.702 + 8) * 2.0 ** -23
        bound = np.abs(ref) * (2.0 ** -8 + share) + 1e-37
        R.within(to_np(M.glu_forward(g, **kw)), ref, bound, "h")
        for fmt in (M.CKPT_MXINT8, M.CKPT_MXFP8):
            h, ck = M.glu_forward(off_by_one(g), ckpt=fmt, **kw)
            R.within(to_np(h), ref, bound, "h with a checkpoint")
            codes, scale, vals = R.ckpt8(g64, fmt)
            assert np.array_equal(ck.codes.cpu().numpy(), codes) and np.array_equal(ck.scale.cpu().numpy(), scale)
            d = to_gpu(dh, dt)
            for held, at in ((ck, vals), (g, g64)):
                (dgu, h2, drow), (ed, eh) = R.glu_grad(at, to_np(d), w, kind, al, limit, inter)
                got = M.glu_backward(d, held, row_w=wg, **kw)
                # d = w dh is rounded once more: 2 U of each term
                R.within(to_np(got["dgu"]), dgu, np.abs(dgu) * 2.0 ** -8 + 1.01 * ed + 1e-37, "dgu")
                R.within(to_np(got["h"]), h2, np.abs(h2) * 2.0 ** -8 + 1.01 * eh + 1e-37, "h again")
                # a lane adds ceil(I / 64) terms, then 6 levels of lanes
                chain = (I // 64 + 8) * U
                R.within(to_np(got["drow_w"]), drow, (np.abs(to_np(d)) * (eh + chain * np.abs(h2))).sum(1) + 1e-37, "drow")
                alone = M.glu_backward(d, held, need_h=False, **kw)
                assert set(alone) == {"dgu"}
                (dgu1, _, _), (ed1, _) = R.glu_grad(at, to_np(d), np.ones(Rn), kind, al, limit, inter)
                R.within(to_np(alone["dgu"]), dgu1, np.abs(dgu1) * 2.0 ** -8 + ed1 + 1e-37, "dgu without weights")


def test_glu_nan_block_stays_nan():
    gu = torch.randn(2, 128, device=DEV, dtype=torch.bfloat16)
    gu[0, 3] = float("nan")
    for kind, al, lim in ((0, 0.0, 0.0), (1, 1.702, 7.0)):
        h, ck = M.glu_forward(gu, glu=kind, alpha=al, limit=lim, ckpt=M.CKPT_MXINT8)
        assert torch.isnan(h[0, 3]) and torch.isfinite(h[1]).all() and int(torch.isnan(h).sum()) == 1
        back = M.glu_backward(torch.ones_like(h), ck, glu=kind, alpha=al, limit=lim)
        assert torch.isnan(back["dgu"][0, :32]).all() and torch.isnan(back["h"][0, :32]).all()
        assert torch.isfinite(back["dgu"][1]).all() and torch.isfinite(back["h"][0, 32:]).all()


def test_glu_empty():
    gu = torch.empty(0, 128, device=DEV, dtype=torch.bfloat16)
    h, ck = M.glu_forward(gu, ckpt=M.CKPT_MXFP8)
    assert tuple(h.shape) == (0, 64)
    back = M.glu_backward(h, ck, row_w=torch.empty(0, device=DEV))
    assert tuple(back["dgu"].shape) == (0, 128) and tuple(back["drow_w"].shape) == (0,)


# ------------------------------------------------------------------ block norms
def norm_inputs(T, H, xdt, post, pre, gate, gdt, seed):
    rng = np.random.default_rng(seed)
    v = dict(x=to_gpu(rng.standard_normal((T, H)) * 2, xdt), f=to_gpu(rng.standard_normal((T, H)), "bf16"),
             w_post=to_gpu(1 + 0.2 * rng.standard_normal(H), "f32") if post else None,
             w_pre=to_gpu(1 + 0.2 * rng.standard_normal(H), "f32") if pre else None)
    shape = dict(none=None, channel=(H,), row=(T, 1), full=(T, H))[gate]
    v["gate"] = None if shape is None else to_gpu(np.clip(rng.standard_normal(shape), -2.5, 2.5), gdt)
    v["dx_new"] = to_gpu(rng.standard_normal((T, H)), xdt)
    v["dy"] = to_gpu(rng.standard_normal((T, H)), "bf16") if pre else None
    if T > 2:
        v["f"][1] = 0                       # a row of zeros: rstd = eps^-1/2
    return v


NORM = [(1, 1, "bf16", True, True, "none", "f32", 0), (4, 2048, "bf16", True, True, "none", "f32", 0),
        (3, 7, "f32", True, True, "full", "bf16", 2), (33, 513, "bf16", True, True, "channel", "f32", 1),
        (300, 64, "f32", True, True, "row", "bf16", 1), (17, 2049, "bf16", True, False, "channel", "f32", 2),
        (70, 2880, "f32", False, True, "row", "f32", 2), (1030, 512, "bf16", True, True, "channel", "bf16", 0),
        (5, 4097, "bf16", True, True, "full", "f32", 1), (3, 8193, "f32", True, True, "channel", "f32", 0),
        (2, 16384, "bf16", True, True, "row", "f32", 0), (600, 1021, "bf16", False, False, "full", "f32", 0)]


@pytest.mark.parametrize("T,H,xdt,post,pre,gate,gdt,fn", NORM)
def test_block_norm_forward_and_backward(T, H, xdt, post, pre, gate, gdt, fn):
    v = norm_inputs(T, H, xdt, post, pre, gate, gdt, T * 17 + H)
    n = {k: None if t is None else to_np(t) for k, t in v.items()}
    alpha, eps = 0.625, float(np.float32(1e-5))
    kw = dict(w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"], gate_fn=fn, alpha=alpha)
    got = M.block_norm_forward(v["x"], v["f"], eps=eps, **kw)
    store = R.bf16 if xdt == "bf16" else (lambda a: a.astype(np.float32).astype(np.float64))
    x, _, rp, _ = R.norm_forward(n["x"], n["f"], n["w_post"], n["w_pre"], n["gate"], fn, alpha, eps, store)
    # rstd: the sum of squares has at most 32 roundings on a chain, rstd half of that plus the division and root
    rel = 24 * U
    if post:
        R.within(to_np(got["rstd_post"]), rp, rp * rel, "rstd_post")
    # z: rstd, two products; the gate function within (|v| + 8) 2^-23 of itself
    zmag = np.abs(x - n["x"])
    R.within(to_np(got["x"]), x, np.abs(x) * R.half_step(xdt) + zmag * 64 * U + np.abs(n["x"]) * U, "x'")
    xs = to_np(got["x"])                    # the pre norm is that of the stored stream
    if pre:
        r = 1 / np.sqrt((xs ** 2).mean(1) + eps)
        y = xs * r[:, None] * n["w_pre"]
        R.within(to_np(got["rstd_pre"]), r, r * rel, "rstd_pre")
        R.within(to_np(got["y"]), y, np.abs(y) * (2.0 ** -8 + 32 * U), "y")
    # backward at what the forward returned
    rp_, r_ = (None if got[k] is None else to_np(got[k]) for k in ("rstd_post", "rstd_pre"))
    ref, mag = R.norm_backward(n["dx_new"], n["dy"], xs, n["f"], rp_, r_, n["w_post"], n["w_pre"], n["gate"], fn, alpha)
    call = lambda: M.block_norm_backward(v["dx_new"], v["dy"], got["x"], v["f"], rstd_post=got["rstd_post"],  # noqa: E731
                                         rstd_pre=got["rstd_pre"], **kw)
    back = call()
    assert set(back) == set(ref)
    # row sums: 64 roundings on a chain; the gate's slope near its tails loses up to 2^9 U; column sums:
    # a slot's rows (T / 256 at most), 16 slots, 16 + 16 partial sums
    gate_u = 512 * U if gate != "none" and fn else 64 * U
    for k in ref:
        chain = gate_u + (T / 256 + 48) * U
        step = {"dx": R.half_step(xdt), "df": 2.0 ** -8}.get(k, U)
        R.within(to_np(back[k]), ref[k], np.abs(ref[k]) * step + mag[k] * chain + 1e-37, k)
    again = call()
    assert all(torch.equal(back[k], again[k]) for k in back)      # a fixed order of every sum


@pytest.mark.parametrize("T,H", [(1, 64), (5, 2047), (40, 4096)])
def test_pre_norm_alone_and_in_place(T, H):
    v = norm_inputs(T, H, "bf16", True, True, "none", "f32", T + H)
    one = M.block_norm_forward(v["x"], w_pre=v["w_pre"], eps=1e-6)
    assert one["x"] is v["x"] and one["rstd_post"] is None
    xs = to_np(v["x"])
    r = 1 / np.sqrt((xs ** 2).mean(1) + np.float32(1e-6))
    R.within(to_np(one["y"]), xs * r[:, None] * to_np(v["w_pre"]), np.abs(xs * r[:, None] * to_np(v["w_pre"])) * (2.0 ** -8 + 32 * U), "y")
    back = M.block_norm_backward(None, v["dy"], v["x"], rstd_pre=one["rstd_pre"], w_pre=v["w_pre"])
    ref, mag = R.norm_backward(None, to_np(v["dy"]), xs, None, None, to_np(one["rstd_pre"]), None, to_np(v["w_pre"]), None, 0, 1.0)
    for k in ref:
        R.within(to_np(back[k]), ref[k], np.abs(ref[k]) * 2.0 ** -8 + mag[k] * (112 + T / 256) * U + 1e-37, k)
    kw = dict(w_post=v["w_post"], w_pre=v["w_pre"], alpha=0.5)
    a = M.block_norm_forward(v["x"], v["f"], **kw)
    x = v["x"].clone()
    b = M.block_norm_forward(x, v["f"], out=x, **kw)
    assert b["x"] is x and torch.equal(a["x"], x) and torch.equal(a["y"], b["y"])


def test_block_norm_empty_and_misaligned():
    v = norm_inputs(0, 96, "bf16", True, True, "channel", "f32", 1)
    got = M.block_norm_forward(v["x"], v["f"], w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"])
    back = M.block_norm_backward(v["dx_new"], v["dy"], got["x"], v["f"], rstd_post=got["rstd_post"],
                                 rstd_pre=got["rstd_pre"], w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"])
    assert all(torch.count_nonzero(back[k]) == 0 and back[k].shape == (96,) for k in ("dw_post", "dw_pre", "dgate"))
    v = norm_inputs(6, 96, "bf16", True, True, "channel", "f32", 2)
    o = {k: None if t is None else off_by_one(t) for k, t in v.items()}
    a = M.block_norm_forward(v["x"], v["f"], w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"])
    b = M.block_norm_forward(o["x"], o["f"], w_post=o["w_post"], w_pre=o["w_pre"], gate=o["gate"])
    assert torch.equal(a["x"], b["x"]) and torch.equal(a["y"], b["y"])


def test_captured_and_replayed():
    """Checkpoint, activation and norms in one captured graph, replayed on new inputs with eager work between."""
    R_, I, H = 70, 96, 160
    gu = torch.randn(R_, 2 * I, device=DEV, dtype=torch.bfloat16)
    dh = torch.randn(R_, I, device=DEV, dtype=torch.bfloat16)
    v = norm_inputs(R_, H, "bf16", True, True, "channel", "f32", 9)

    def step():
        h, ck = M.glu_forward(gu, ckpt=M.CKPT_MXINT8)
        back = M.glu_backward(dh, ck)
        n = M.block_norm_forward(v["x"], v["f"], w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"], gate_fn=1)
        nb = M.block_norm_backward(v["dx_new"], v["dy"], n["x"], v["f"], rstd_post=n["rstd_post"], rstd_pre=n["rstd_pre"],
                                   w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"], gate_fn=1)
        return [h, back["dgu"], back["h"], n["x"], n["y"], *[nb[k] for k in sorted(nb)]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        gu.copy_(torch.randn_like(gu))
        v["f"].copy_(torch.randn_like(v["f"]))
        g.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), k


def test_two_streams_at_once():
    gu = [torch.randn(4000, 512, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    dh = [torch.randn(4000, 256, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    v = [norm_inputs(3000, 256, "bf16", True, True, "channel", "f32", k) for k in range(2)]

    def step(i):
        _, ck = M.glu_forward(gu[i], ckpt=M.CKPT_MXFP8)
        d = M.glu_backward(dh[i], ck)
        w = dict(w_post=v[i]["w_post"], w_pre=v[i]["w_pre"], gate=v[i]["gate"])
        n = M.block_norm_forward(v[i]["x"], v[i]["f"], **w)
        nb = M.block_norm_backward(v[i]["dx_new"], v[i]["dy"], n["x"], v[i]["f"], rstd_post=n["rstd_post"],
                                   rstd_pre=n["rstd_pre"], **w)
        return [d["dgu"], d["h"], n["y"], *[nb[k] for k in sorted(nb)]]
    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append(step(i))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


@pytest.mark.parametrize("H", [2, 3, 4, 5, 6, 8, 9, 10, 11, 12, 13, 14, 15, 521, 2052, 4094, 8198])
@pytest.mark.parametrize("xdt,gdt", [("bf16", "f32"), ("f32", "bf16")])
def test_block_norm_every_length_of_a_last_piece(H, xdt, gdt):
    test_block_norm_forward_and_backward(9, H, xdt, True, True, "full", gdt, 1)


def test_block_norm_neighbours_of_a_last_piece():
    """A row's partial piece is read with the values before it: those, not finite, stay out of it, and no row reaches another."""
    T, H = 6, 21
    v = norm_inputs(T, H, "bf16", True, True, "none", "f32", 3)
    w = dict(w_post=v["w_post"], w_pre=v["w_pre"])
    want = M.block_norm_forward(v["x"], v["f"], **w)
    bad = v["f"].clone()
    bad[2, 15] = float("nan")
    bad[3, 13] = float("inf")
    got = M.block_norm_forward(v["x"], bad, **w)
    keep = [0, 1, 4, 5]
    assert all(torch.equal(got[k][keep], want[k][keep]) for k in want)
    w1 = dict(w_pre=v["w_pre"])                 # without the post norm each value of f reaches its own place of x' only
    a, b = M.block_norm_forward(v["x"], v["f"], **w1), M.block_norm_forward(v["x"], bad, **w1)
    same = torch.ones(T, H, dtype=torch.bool, device=DEV)
    same[2, 15] = same[3, 13] = False
    assert torch.equal(a["x"][same], b["x"][same]) and not torch.isfinite(b["x"][~same]).any()


def test_rows_behind_the_last_are_left_alone():
    """Through the C ABI with room behind each output: nothing past the last row is written."""
    Rn, I = 5, 64
    L = M.lib()
    gu = torch.randn(Rn, 2 * I, device=DEV, dtype=torch.bfloat16)
    h = torch.full((Rn + 2, I), 7.0, device=DEV, dtype=torch.bfloat16)
    codes = torch.full((Rn + 2, 2 * I), 0xAB, device=DEV, dtype=torch.uint8)
    scale = torch.full((Rn + 2, 2 * I // 32), 0xAB, device=DEV, dtype=torch.uint8)
    st = torch.cuda.current_stream().cuda_stream
    M._check(L.nf4moe_glu_forward(gu.data_ptr(), 1, Rn, I, 0, 0.0, 0.0, 0, h.data_ptr(), 0, codes.data_ptr(),
                                  scale.data_ptr(), st))
    x = torch.randn(Rn, 96, device=DEV)
    q = torch.full((Rn + 1, 96), 0xAB, device=DEV, dtype=torch.uint8)
    qs = torch.full((Rn + 1, 3), 0xAB, device=DEV, dtype=torch.uint8)
    M._check(L.nf4moe_ckpt8_quantize(1, x.data_ptr(), 0, Rn, 96, q.data_ptr(), qs.data_ptr(), st))
    torch.cuda.synchronize()
    assert (h[Rn:] == 7.0).all() and (codes[Rn:] == 0xAB).all() and (scale[Rn:] == 0xAB).all()
    assert (q[Rn:] == 0xAB).all() and (qs[Rn:] == 0xAB).all()
    assert not (h[:Rn] == 7.0).all()


def test_rows_past_one_launch():
    """More rows than one launch takes: every piece's rows, and nothing between them, against the same rows alone."""
    T, H, I = (1 << 22) + 5, 8, 32
    g = torch.Generator(device=DEV).manual_seed(4)
    rn = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g, device=DEV).to(dt)  # noqa: E731
    cuts = [(0, 4), ((1 << 21) - 3, (1 << 21) + 3), ((1 << 22) - 3, T)]
    x, f, gate = rn(T, H), rn(T, H), rn(T, 1, dt=torch.float32)
    w = dict(w_post=rn(H, dt=torch.float32), w_pre=rn(H, dt=torch.float32), gate_fn=M.GATE_TANH)
    for gt in (gate, rn(T, H)):
        a = M.block_norm_forward(x, f, gate=gt, **w)
        for lo, hi in cuts:
            b = M.block_norm_forward(x[lo:hi].clone(), f[lo:hi].clone(), gate=gt[lo:hi].clone(), **w)
            assert all(torch.equal(a[k][lo:hi], b[k]) for k in a), (lo, hi)
    del x, f, gate, gt, a, b
    gu, dh, rw = rn(T, 2 * I), rn(T, I), rn(T, dt=torch.float32)
    h, ck = M.glu_forward(gu, ckpt=M.CKPT_MXFP8)
    a = M.glu_backward(dh, ck, row_w=rw)
    for lo, hi in cuts:
        b, c = M.glu_forward(gu[lo:hi].clone(), ckpt=M.CKPT_MXFP8)
        assert torch.equal(b, h[lo:hi]) and torch.equal(c.codes, ck.codes[lo:hi]) and torch.equal(c.scale, ck.scale[lo:hi])
        d = M.glu_backward(dh[lo:hi].clone(), c, row_w=rw[lo:hi].clone())
        # drow_w: one wave a row against four for so few; 32 columns lie in one wave either way, the rest adds zeros
        assert all(torch.equal(a[k][lo:hi], d[k]) for k in a), (lo, hi)
