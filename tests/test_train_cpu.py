"""The fine-tuning operators without a GPU: their 64-bit references against
independent facts, and every refusal of the C ABI and of the binding."""
import os

import numpy as np
import pytest

import train_ref as R

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("bit_quantized_moe_expert_amd")
if not os.path.exists(pkg.LIB_PATH):
    pytest.skip("libnf4moe.so not built", allow_module_level=True)

L = pkg.lib()
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000          # aligned, never dereferenced
ODD = FAKE + 1


# ------------------------------------------------------------------ references
def test_e4m3_reference_is_torchs_float8():
    codes = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v[:127], R.E4M3)
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 64)) * np.exp(rng.standard_normal((40, 1)))).astype(np.float32)
    codes, scale, vals = R.ckpt8(x, R.MXFP8)
    X = scale.astype(int).repeat(32, 1).reshape(x.shape) - 127
    # torch does not saturate: compare where the scaled value is inside the range
    v = np.ldexp(x.astype(np.float64), -X)
    t = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ok = np.abs(v) <= 448
    assert np.array_equal(codes[ok], t[ok])
    assert np.all((codes[~ok] & 127) == 126)


@pytest.mark.parametrize("fmt,step", [(R.MXINT8, 2.0 ** -6), (R.MXFP8, None)])
def test_checkpoint_reference_error_and_idempotence(fmt, step):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((64, 128)).astype(np.float32)
    codes, scale, vals = R.ckpt8(x, fmt)
    X = scale.astype(int).repeat(32, 1).reshape(x.shape) - 127
    if fmt == R.MXINT8:     # half a step of 2^(X - 6); a whole one where the top code saturates
        assert np.all(np.abs(vals - x) <= np.ldexp(0.5, X - 6) + (np.abs(x) > np.ldexp(127.0, X - 6)) * np.ldexp(0.5, X - 6))
    else:                   # half a step of 3 fraction bits, saturation at 448 2^X
        big = np.abs(x) > np.ldexp(448.0, X)
        assert np.all(np.abs(vals - x)[~big] <= np.maximum(np.abs(x) * 2.0 ** -4, np.ldexp(1.0, X - 10))[~big])
    again = R.ckpt8(vals, fmt)
    assert np.array_equal(again[2], vals)


def test_glu_gradient_reference_by_differences():
    rng = np.random.default_rng(2)
    for kind, inter in ((0, 0), (0, 1), (1, 0), (1, 1)):
        gu = rng.standard_normal((3, 64)) * 4
        gu = np.where(np.abs(np.abs(gu) - 7.0) < 1e-3, 6.5, gu)
        dh, w = rng.standard_normal((3, 32)), rng.random(3)
        (dgu, _, drow), _ = R.glu_grad(gu, dh, w, kind, 1.702, 7.0, inter)
        num = np.zeros_like(gu)
        for r in range(3):
            for c in range(64):
                for sgn in (1, -1):
                    p = gu.copy()
                    p[r, c] += sgn * 1e-6
                    num[r, c] += sgn * (w[:, None] * dh * R.glu(p, kind, 1.702, 7.0, inter)).sum() / 2e-6
        assert np.allclose(dgu, num, rtol=1e-6, atol=1e-6)
        assert np.allclose(drow, (dh * R.glu(gu, kind, 1.702, 7.0, inter)).sum(1))


@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_norm_gradient_reference_by_differences(gate):
    rng = np.random.default_rng(3)
    T, H = 3, 5
    shape = dict(none=None, channel=(H,), row=(T, 1), full=(T, H))[gate]
    for fn in (0, 1, 2):
        v = dict(x=rng.standard_normal((T, H)), f=rng.standard_normal((T, H)), w_post=rng.standard_normal(H),
                 w_pre=rng.standard_normal(H))
        if shape:
            v["gate"] = rng.standard_normal(shape)
        cx, cy = rng.standard_normal((T, H)), rng.standard_normal((T, H))

        def loss(v):
            x, y, _, _ = R.norm_forward(v["x"], v["f"], v["w_post"], v["w_pre"], v.get("gate"), fn, 0.7, 1e-5, lambda a: a)
            return (cx * x).sum() + (cy * y).sum()
        x, y, rp, r = R.norm_forward(v["x"], v["f"], v["w_post"], v["w_pre"], v.get("gate"), fn, 0.7, 1e-5, lambda a: a)
        got, _ = R.norm_backward(cx, cy, x, v["f"], rp, r, v["w_post"], v["w_pre"], v.get("gate"), fn, 0.7)
        for name, key in (("x", "dx"), ("f", "df"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("gate", "dgate")):
            if name not in v:
                continue
            num = np.zeros_like(v[name])
            for i in np.ndindex(*num.shape):
                for sgn in (1, -1):
                    q = {k: a.copy() for k, a in v.items()}
                    q[name][i] += sgn * 1e-6
                    num[i] += sgn * loss(q) / 2e-6
            # eps > 0: the reference's gradient uses the rstd with eps, as the formula does
            assert np.allclose(got[key], num, rtol=2e-5, atol=2e-5), (fn, name)


def test_adapter_gradient_reference_by_differences():
    rng = np.random.default_rng(4)
    L_, r, K, N, ids, row_of = 3, 2, 4, 5, np.array([1, -1, 0, 1, 9, 0]), np.array([0, 1, 1, 2, 0, 2])
    v = dict(x=rng.standard_normal((3, K)), A=rng.standard_normal((L_, r, K)), B=rng.standard_normal((L_, N, r)))
    scale, cy = rng.random(L_) + 0.5, rng.standard_normal((6, N))

    def loss(v):
        return (cy * R.adapter_forward(v["x"], v["A"], v["B"], ids, scale, None, row_of)[0]).sum()
    t = R.adapter_forward(v["x"], v["A"], v["B"], ids, scale, None, row_of)[1]
    got, _ = R.adapter_backward(cy, v["x"], t, v["A"], v["B"], ids, scale, None, row_of)
    dx = np.zeros((3, K))
    np.add.at(dx, row_of, got["dx"])
    for name, g in (("x", dx), ("A", got["dA"]), ("B", got["dB"])):
        num = np.zeros_like(v[name])
        for i in np.ndindex(*num.shape):
            for sgn in (1, -1):
                q = {k: a.copy() for k, a in v.items()}
                q[name][i] += sgn * 1e-6
                num[i] += sgn * loss(q) / 2e-6
        assert np.allclose(g, num, rtol=1e-6, atol=1e-7), name
    assert np.all(got["dA"][2] == 0) and np.all(got["dx"][[1, 4]] == 0)


# ------------------------------------------------------------------ refusals of the C ABI
def test_ckpt8_validation():
    for q in (lambda f, x, dt, rows, K, c, s: L.nf4moe_ckpt8_quantize(f, x, dt, rows, K, c, s, None),
              lambda f, x, dt, rows, K, c, s: L.nf4moe_ckpt8_dequantize(f, c, s, rows, K, x, dt, None)):
        assert q(2, FAKE, 0, 4, 64, FAKE, FAKE) == INVALID          # unknown format
        assert q(-1, FAKE, 0, 4, 64, FAKE, FAKE) == INVALID
        assert q(0, FAKE, 2, 4, 64, FAKE, FAKE) == INVALID          # unknown dtype
        assert q(0, FAKE, 0, -1, 64, FAKE, FAKE) == INVALID
        assert q(0, FAKE, 0, 4, 48, FAKE, FAKE) == INVALID          # K % 32
        assert q(0, FAKE, 0, 4, 0, FAKE, FAKE) == INVALID
        assert q(0, FAKE, 0, 1 << 45, 64, FAKE, FAKE) == UNSUPPORTED
        assert q(0, None, 0, 4, 64, FAKE, FAKE) == INVALID
        assert q(0, FAKE, 0, 4, 64, None, FAKE) == INVALID
        assert q(0, FAKE, 0, 4, 64, FAKE, None) == INVALID
        assert q(0, FAKE + 2, 0, 4, 64, FAKE, FAKE) == INVALID      # fp32 misaligned
        assert q(0, ODD, 1, 4, 64, FAKE, FAKE) == INVALID           # bf16 misaligned
        assert q(0, None, 0, 0, 64, None, None) == OK               # empty: no-op


def test_glu_validation():
    def fwd(gu=FAKE, dt=1, R=4, I=64, glu=0, al=0.0, lim=0.0, inter=0, h=FAKE, ck=0, codes=None, scale=None):
        return L.nf4moe_glu_forward(gu, dt, R, I, glu, al, lim, inter, h, ck, codes, scale, None)

    def bwd(dh=FAKE, dt=1, src=1, gu=FAKE, sc=None, R=4, I=64, glu=0, al=0.0, lim=0.0, inter=0, w=None, dgu=FAKE, h=None,
            dw=None):
        return L.nf4moe_glu_backward(dh, dt, src, gu, sc, R, I, glu, al, lim, inter, w, dgu, h, dw, None)

    for call in (fwd, bwd):
        assert call(dt=3) == INVALID
        assert call(R=-1) == INVALID
        assert call(I=48) == INVALID and call(I=0) == INVALID
        assert call(R=1 << 35, I=64) == UNSUPPORTED
        assert call(glu=2) == INVALID
        assert call(glu=1) == INVALID                               # clamped without alpha, limit
        assert call(glu=1, al=1.7, lim=float("inf")) == INVALID
        assert call(glu=1, al=float("nan"), lim=7.0) == INVALID
        assert call(inter=2) == INVALID
        assert call(gu=None) == INVALID
        assert call(gu=ODD) == INVALID
        assert call(R=0, gu=None) == OK
    assert fwd(h=None) == INVALID
    assert fwd(codes=FAKE) == INVALID                               # codes without scale
    assert fwd(codes=FAKE, scale=FAKE, ck=2) == INVALID
    assert bwd(dh=None) == INVALID and bwd(dgu=None) == INVALID
    assert bwd(src=4) == INVALID and bwd(src=-1) == INVALID
    assert bwd(src=2) == INVALID                                    # checkpoint without scales
    assert bwd(w=ODD) == INVALID and bwd(dw=ODD) == INVALID and bwd(h=ODD) == INVALID


def _norm(H=64, x_dtype=1, w_post=FAKE, w_pre=FAKE, gate=None, kind=0, gdt=0, fn=0, alpha=1.0, eps=1e-6):
    from bit_quantized_moe_expert_amd import train
    st = train._BLOCK_NORM.pack(H, x_dtype, w_post or 0, w_pre or 0, gate or 0, kind, gdt, fn, alpha, eps)
    return st, st


def test_block_norm_validation():
    def both(T=4, f=FAKE, **kw):
        st, a = _norm(**kw)
        H = max(1, min(kw.get("H", 64), 16384))
        need = L.nf4moe_block_norm_workspace_bytes(H, max(T, 1))
        return (L.nf4moe_block_norm_forward(a, FAKE, f, T, FAKE, FAKE, FAKE, FAKE, None),
                L.nf4moe_block_norm_backward(a, FAKE, FAKE, FAKE, f, FAKE, FAKE, T, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                             need, None))
    assert L.nf4moe_block_norm_forward(None, FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    bad = [dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=16385), dict(x_dtype=2), dict(gdt=2), dict(kind=4, gate=FAKE),
           dict(fn=3), dict(kind=1), dict(gate=FAKE), dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("inf")),
           dict(w_post=FAKE + 2), dict(gate=ODD, kind=1, gdt=1), dict(f=None), dict(f=None, w_post=None, gate=FAKE, kind=1),
           dict(f=None, w_post=None, w_pre=None), dict(f=ODD)]
    for kw in bad:
        assert both(**kw) == (INVALID, INVALID), kw
    st, a = _norm()
    fw = L.nf4moe_block_norm_forward
    assert fw(a, None, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert fw(a, FAKE, FAKE, 4, None, FAKE, FAKE, FAKE, None) == INVALID
    assert fw(a, FAKE, FAKE, 4, FAKE, None, FAKE, FAKE, None) == INVALID
    assert fw(a, FAKE, FAKE, 4, FAKE, FAKE, None, FAKE, None) == INVALID
    assert fw(a, FAKE, FAKE, 4, FAKE, FAKE, FAKE, None, None) == INVALID
    assert fw(a, ODD, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert fw(a, None, None, 0, None, None, None, None, None) == OK             # empty tensors may have no address
    need = L.nf4moe_block_norm_workspace_bytes(64, 4)
    assert need > 0 and L.nf4moe_block_norm_workspace_bytes(64, 0) == 0 and L.nf4moe_block_norm_workspace_bytes(0, 4) == 0
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, None, FAKE, FAKE, FAKE, need]
    bw = lambda i, v: L.nf4moe_block_norm_backward(a, *(args[:i] + [v] + args[i + 1:]), None)  # noqa: E731
    for i in (1, 2, 4, 5, 7, 8, 10, 11):
        assert bw(i, None) == INVALID, i
    assert bw(12, None) == WORKSPACE and bw(13, need - 1) == WORKSPACE
    assert bw(12, FAKE + 16) == INVALID


def test_adapter_validation():
    from bit_quantized_moe_expert_amd import train

    def desc(L_=4, rank=16, K=64, N=64, A=FAKE, B=FAKE, scale=None):
        st = train._ADAPTERS.pack(L_, rank, K, N, A or 0, B or 0, scale or 0)
        return st, st
    st, a = desc()
    assert L.nf4moe_adapter_plan_bytes(0, 4) == 0 and L.nf4moe_adapter_plan_bytes(8, 0) == 0
    assert L.nf4moe_adapter_plan_bytes(8, 4097) == 0 and L.nf4moe_adapter_plan_bytes(8, 4096) > 0
    n = 200000          # enough rows for the grouped kernels
    pb, wf, wb = (L.nf4moe_adapter_plan_bytes(n, 4), L.nf4moe_adapter_workspace_bytes(a, n, 0),
                  L.nf4moe_adapter_workspace_bytes(a, n, 1))
    assert pb > 0 and wf >= pb and wb > wf
    assert L.nf4moe_adapter_workspace_bytes(a, 8, 0) == 0 and L.nf4moe_adapter_workspace_bytes(a, 8, 1) > 0
    assert L.nf4moe_adapter_workspace_bytes(a, 0, 0) == 0 and L.nf4moe_adapter_workspace_bytes(None, 8, 0) == 0
    plan = L.nf4moe_adapter_plan
    assert plan(FAKE, n, 0, FAKE, pb, None) == INVALID and plan(FAKE, n, 4097, FAKE, pb, None) == INVALID
    assert plan(FAKE, -1, 4, FAKE, pb, None) == INVALID and plan(None, n, 4, FAKE, pb, None) == INVALID
    assert plan(FAKE + 2, n, 4, FAKE, pb, None) == INVALID and plan(FAKE, n, 4, FAKE + 16, pb, None) == INVALID
    assert plan(FAKE, n, 4, None, pb, None) == WORKSPACE and plan(FAKE, n, 4, FAKE, pb - 1, None) == WORKSPACE
    assert plan(None, 0, 4, None, 0, None) == OK

    names = ["x", "x_rows", "row_of", "ids", "plan", "pb", "R", "base", "out", "dt", "t", "ws", "wsb"]
    dflt = dict(x=FAKE, x_rows=n, row_of=None, ids=FAKE, plan=None, pb=0, R=n, base=FAKE, out=FAKE, dt=1, t=None,
                ws=FAKE, wsb=wf)

    def fwd(d=None, **kw):
        keep = d or desc()
        return L.nf4moe_adapter_forward(keep[1], *[dict(dflt, **kw)[n] for n in names], None)
    bnames = ["dy", "src", "x", "xs", "x_rows", "row_of", "t", "ids", "plan", "pb", "R", "dxb", "dx", "dt", "dA", "dB", "ws", "wsb"]
    bdflt = dict(dy=FAKE, src=1, x=FAKE, xs=None, x_rows=n, row_of=None, t=FAKE, ids=FAKE, plan=None, pb=0, R=n, dxb=None,
                 dx=FAKE, dt=1, dA=FAKE, dB=FAKE, ws=FAKE, wsb=wb)

    def bwd(d=None, **kw):
        keep = d or desc()
        return L.nf4moe_adapter_backward(keep[1], *[dict(bdflt, **kw)[n] for n in bnames], None)
    for call in (fwd, bwd):
        for bad in (dict(L_=0), dict(L_=4097), dict(rank=0), dict(rank=4), dict(rank=20), dict(rank=136), dict(K=4), dict(K=60),
                    dict(N=0), dict(N=12), dict(K=1 << 21), dict(A=None), dict(B=None), dict(A=ODD), dict(scale=FAKE + 2)):
            assert call(desc(**bad)) == INVALID, bad
        assert call(R=-1) == INVALID and call(R=(1 << 30) + 1) == INVALID
        assert call(dt=2) == INVALID and call(ids=None) == INVALID and call(ids=ODD) == INVALID
        assert call(x_rows=n - 1) == INVALID and call(x_rows=0, row_of=FAKE) == INVALID and call(row_of=ODD) == INVALID
        assert call(plan=FAKE, pb=pb - 1) == WORKSPACE and call(plan=FAKE + 16, pb=pb) == INVALID
        assert call(ws=None) == WORKSPACE and call(wsb=10) == WORKSPACE and call(ws=FAKE + 16) == INVALID
        assert call(t=FAKE + 4) == INVALID and call(x=ODD) == INVALID
    assert L.nf4moe_adapter_forward(None, *[dflt[n] for n in names], None) == INVALID
    assert fwd(x=None) == INVALID and fwd(out=None) == INVALID and fwd(out=ODD) == INVALID and fwd(base=ODD) == INVALID
    assert fwd(R=0, x=None, ids=None, out=None, ws=None, wsb=0) == OK
    assert bwd(src=0) == INVALID and bwd(src=4) == INVALID and bwd(src=2) == INVALID      # fp32; unknown; no scales
    assert bwd(desc(K=40), src=2, xs=FAKE) == INVALID                                     # 8-bit x: K % 32
    assert bwd(dy=None) == INVALID and bwd(x=None) == INVALID and bwd(t=None) == INVALID
    assert bwd(dA=FAKE + 4) == INVALID and bwd(dB=FAKE + 4) == INVALID and bwd(dx=ODD) == INVALID
    assert bwd(dx=None, dA=None, dB=None) == OK
    assert bwd(R=0, dA=None, dB=None) == OK


@pytest.mark.parametrize("n", [4, 200000])          # the one-launch form and the grouped kernels
def test_adapter_refuses_overlapping_outputs(n):
    """An output over an input that other rows still read; the exceptions are base and dx_base themselves."""
    from bit_quantized_moe_expert_amd import train
    K = N = 64
    desc = train._ADAPTERS.pack(4, 16, K, N, FAKE, FAKE, 0)
    big, far, bytes_ = 1 << 40, 1 << 41, n * N * 2
    wf, wb = L.nf4moe_adapter_workspace_bytes(desc, n, 0), L.nf4moe_adapter_workspace_bytes(desc, n, 1)

    def fwd(x, base, out):
        return L.nf4moe_adapter_forward(desc, x, n, None, FAKE, None, 0, n, base, out, 1, None, FAKE, wf, None)

    def bwd(dy, x, dxb, dx):
        return L.nf4moe_adapter_backward(desc, dy, 1, x, None, n, None, FAKE, FAKE, None, 0, n, dxb, dx, 1, FAKE, FAKE, FAKE, wb,
                                         None)
    for d in (0, 2, bytes_ - 2, 2 - bytes_):
        assert fwd(big, None, big + d) == INVALID and fwd(big, big, big) == INVALID
        assert bwd(big, far, None, big + d) == INVALID and bwd(far, big, None, big + d) == INVALID
        if d:
            assert fwd(far, big, big + d) == INVALID and bwd(far, 1 << 42, big, big + d) == INVALID
    assert "overlaps" in L.nf4moe_last_error().decode()


def test_block_norm_refuses_overlapping_outputs():
    big, far = 1 << 40, 1 << 41
    st, a = _norm()
    fw = lambda x, f, out: L.nf4moe_block_norm_forward(a, x, f, 4, out, FAKE, FAKE, FAKE, None)  # noqa: E731
    for d in (2, 4 * 64 * 2 - 2, 2 - 4 * 64 * 2):
        assert fw(big, far, big + d) == INVALID and fw(far, big, big + d) == INVALID
    assert fw(far, big, big) == INVALID


def test_adapter_refuses_more_than_a_dispatch():
    """Grids past 2^32 threads are refused before anything runs."""
    from bit_quantized_moe_expert_amd import train
    n = 1 << 30
    desc = train._ADAPTERS.pack(4, 16, 64, 1 << 14, FAKE, FAKE, 0)
    assert L.nf4moe_adapter_forward(desc, FAKE, n, None, FAKE, None, 0, n, None, FAKE, 1, None, FAKE, 0, None) == UNSUPPORTED
    wide = train._ADAPTERS.pack(4096, 8, 1 << 18, 1 << 18, FAKE, FAKE, 0)     # dA and dB of many adapters, one row
    assert L.nf4moe_adapter_backward(wide, FAKE, 1, FAKE, None, 1, None, FAKE, FAKE, None, 0, 1, None, None, 1, FAKE, FAKE, FAKE, 0,
                                     None) == UNSUPPORTED
    assert L.nf4moe_adapter_backward(wide, FAKE, 1, FAKE, None, 1, None, FAKE, FAKE, None, 0, 1, None, FAKE, 1, None, None, FAKE, 0,
                                     None) == WORKSPACE


def test_binding_refuses_sizes_past_32_bits():
    """Row counts that a 32-bit argument cannot hold are refused, not cut."""
    meta = dict(device="meta")
    A, B = torch.empty(2, 8, 64, dtype=torch.bfloat16, **meta), torch.empty(2, 64, 8, dtype=torch.bfloat16, **meta)
    rows = (1 << 32) + 4
    x, ids = torch.empty(rows, 64, dtype=torch.bfloat16, **meta), torch.empty(rows, dtype=torch.int32, **meta)
    few = torch.empty(4, dtype=torch.int32, **meta)
    with pytest.raises(ValueError, match="32 bits"):
        pkg.adapter_forward(x, A, B, ids)
    with pytest.raises(ValueError, match="32 bits"):
        pkg.adapter_forward(x, A, B, few, x_row_of=few)
    with pytest.raises(ValueError, match="32 bits"):
        pkg.adapter_plan(ids, 2)
    with pytest.raises(ValueError, match="32 bits"):
        pkg.adapter_plan(few, rows)
    with pytest.raises(ValueError, match="32 bits"):
        pkg.glu_forward(torch.empty(2, 1 << 33, dtype=torch.bfloat16, **meta))


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_before_the_device():
    M = pkg
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cpu"):
        M.ckpt8_quantize(bf)
    with pytest.raises(ValueError, match="multiple of 32"):
        M.ckpt8_quantize(bf[:, :40])
    with pytest.raises(TypeError):
        M.ckpt8_quantize(bf.half())
    with pytest.raises(ValueError, match="format"):
        M.ckpt8_quantize(bf, 5)
    with pytest.raises(ValueError, match="shape"):
        M.ckpt8_dequantize(M.Ckpt8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 3, dtype=torch.uint8), 0))
    with pytest.raises(TypeError):
        M.ckpt8_dequantize(M.Ckpt8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8), 0))
    with pytest.raises(ValueError, match="columns"):
        M.glu_forward(bf[:, :48])
    with pytest.raises(ValueError, match="cpu"):
        M.glu_forward(bf)
    with pytest.raises(ValueError, match="shape"):
        M.glu_backward(bf, bf)
    with pytest.raises(ValueError, match="shape"):
        M.glu_backward(bf[:, :32], bf, row_w=torch.zeros(5))
    w = torch.ones(64)
    with pytest.raises(ValueError, match="gate has shape"):
        M.block_norm_forward(bf, bf, w_pre=w, gate=torch.zeros(4))
    with pytest.raises(TypeError):
        M.block_norm_forward(bf, bf.float(), w_pre=w)
    with pytest.raises(TypeError):
        M.block_norm_forward(bf, bf, w_pre=w.bfloat16())
    with pytest.raises(ValueError, match="cpu"):
        M.block_norm_forward(bf, bf, w_pre=w)
    with pytest.raises(ValueError, match="cpu"):
        M.block_norm_backward(bf, bf, bf, bf, w_pre=w, rstd_pre=torch.ones(4))


def test_binding_refuses_bad_adapters():
    M = pkg
    x, ids = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    A, B = torch.zeros(3, 16, 64, dtype=torch.bfloat16), torch.zeros(3, 32, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, 16)
    dy = torch.zeros(4, 32, dtype=torch.bfloat16)
    for err, kw in ((ValueError, dict(B=B[:2])), (ValueError, dict(B=torch.zeros(3, 32, 8, dtype=torch.bfloat16))),
                    (TypeError, dict(A=A.float())), (TypeError, dict(ids=ids.long())), (ValueError, dict(x=x[:, :32])),
                    (ValueError, dict(x=x[:3])), (TypeError, dict(x=x.float())), (ValueError, dict(scale=torch.ones(4))),
                    (TypeError, dict(scale=torch.ones(3).double())), (ValueError, dict(base=torch.zeros(4, 31))),
                    (TypeError, dict(base=torch.zeros(4, 32), out_dtype=torch.bfloat16)),
                    (TypeError, dict(x_row_of=ids.long())), (ValueError, dict(x_row_of=ids[:3])),
                    (TypeError, dict(out_dtype=torch.float16)),
                    (ValueError, dict(plan=M.AdapterPlan(x, 0, 0, 5, 3))), (ValueError, dict())):
        with pytest.raises(err):
            M.adapter_forward(**dict(dict(x=x, A=A, B=B, ids=ids), **kw))
    for err, kw in ((ValueError, dict(need=("dz",))), (ValueError, dict(dy=dy[:, :16])), (TypeError, dict(dy=dy.float())),
                    (ValueError, dict(x=None)), (ValueError, dict(t=None)), (TypeError, dict(t=t.double())),
                    (ValueError, dict(t=t[:3])), (ValueError, dict(x=x[:3])), (TypeError, dict(x=x.float())),
                    (TypeError, dict(dx_base=torch.zeros(4, 64), dx_dtype=torch.bfloat16)), (ValueError, dict())):
        with pytest.raises(err):
            M.adapter_backward(**dict(dict(dy=dy, x=x, t=t, A=A, B=B, ids=ids), **kw))
    with pytest.raises(ValueError, match="cpu"):
        M.adapter_plan(ids, 3)
