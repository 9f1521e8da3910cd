"""Refusals of the fine-tuning operators at the edges of their sizes and arguments,
without a GPU: addresses are made up and never dereferenced, every refused call
returns before anything is enqueued."""
import os

import pytest

torch = pytest.importorskip("torch")
pkg = pytest.importorskip("bit_quantized_moe_expert_amd")
if not os.path.exists(pkg.LIB_PATH):
    pytest.skip("libnf4moe.so not built", allow_module_level=True)

L = pkg.lib()
OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = 0, 1, 2, 3, 4
FAKE = 0x10000


def far(i):
    """Made-up addresses 8 TB apart."""
    return (i + 1) << 43


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses, which a GPU would dereference")
@pytest.mark.parametrize("glu,alpha,limit", [(0, 0.0, 0.0), (1, 1.702, 7.0)])
def test_glu_refuses_rows_whose_columns_pass_32_bits(glu, alpha, limit):
    """Columns of a row of gu are counted in 32 bits: 2 I is at most 2^31."""
    for inter in (0, 1):
        for wide in ((1 << 30) + 32, (1 << 31) - 32):
            assert L.nf4moe_glu_forward(far(0), 1, 1, wide, glu, alpha, limit, inter, far(1), 0, None, None, None) == UNSUPPORTED
            assert L.nf4moe_glu_forward(far(0), 0, 3, wide, glu, alpha, limit, inter, far(1), 1, far(2), far(3), None) == UNSUPPORTED
            for src in range(4):
                assert L.nf4moe_glu_backward(far(0), 1, src, far(1), far(2), 1, wide, glu, alpha, limit, inter, None, far(3),
                                             far(4), None, None) == UNSUPPORTED
        # the widest row is taken: without a device its launch fails
        assert L.nf4moe_glu_forward(far(0), 1, 1, 1 << 30, glu, alpha, limit, inter, far(1), 0, None, None, None) == HIP


def test_package_imports_without_torch():
    """Constants, the library's path and the build are there without torch, as before; the operators come with it."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(pkg.__file__)))
    code = ("import sys; sys.modules['torch'] = None\n"
            "import bit_quantized_moe_expert_amd as M, bit_quantized_moe_expert_amd.build as b\n"
            "assert M.FMT_MXFP4 == 1 and M.LIB_PATH and b.sources() and 'adapter_forward' in dir(M)\n"
            "assert not hasattr(M, 'no_such_name')\n")
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=120)
    code = ("import sys, bit_quantized_moe_expert_amd as M\n"
            "assert 'torch' not in sys.modules\n"
            "from bit_quantized_moe_expert_amd import Ckpt8, adapter_forward\n"
            "assert M.adapter_forward is adapter_forward is M.train.adapter_forward and M.CKPT_MXFP8 == 1\n")
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)


def test_adapter_backward_without_dA_takes_no_x():
    """x is read for dA only: dx and dB are made without its rows."""
    from bit_quantized_moe_expert_amd import train
    n = 100
    desc = train._ADAPTERS.pack(4, 16, 64, 64, far(0), far(1), 0)
    need = L.nf4moe_adapter_workspace_bytes(desc, n, 1)

    def bwd(dA, ws_bytes, x=None, x_rows=0):
        return L.nf4moe_adapter_backward(desc, far(2), 1, x, None, x_rows, None, far(3), far(4), None, 0, n, None, far(5), 1, dA,
                                         far(6), far(7), ws_bytes, None)
    assert bwd(None, need - 1) == WORKSPACE         # the next check after those of the rows
    assert bwd(None, need - 1, x_rows=n - 1) == WORKSPACE
    assert bwd(far(8), need, x=far(9), x_rows=n - 1) == INVALID
    assert bwd(far(8), need, x=None, x_rows=n) == INVALID


def test_sources_compile_without_format_warnings():
    """Error messages print each argument by its own type (printf formats, checked by the compiler)."""
    import subprocess
    from bit_quantized_moe_expert_amd import build
    src = os.path.join(build.CSRC, "api_train.hip")
    subprocess.run([build._hipcc(), *build.FLAGS, "--offload-host-only", "-Werror=format", "-fsyntax-only", src], check=True, timeout=300)


# ------------------------------------------------------------------ arrays that share bytes
def overlaps_refused(call, outs, ins, may_be=(), base=None):
    """Every output laid over each input and each other output, by its last and its first
    element: INVALID_ARG. may_be: (output, input) pairs that may be one array, not two in part."""
    at = {n: far(i) for i, n in enumerate({**outs, **ins})}
    size = {**outs, **ins}

    def status(**over):
        return call(**{**at, **over})
    for o in outs:
        for other in size:
            if other == o or (other in outs and list(outs).index(other) < list(outs).index(o)):
                continue
            for shift in (size[other] - 256, 256 - size[o], 0):
                if shift % 256 or (shift == 0 and (o, other) in may_be):
                    continue
                if shift and not -size[o] < shift < size[other]:
                    continue
                assert status(**{o: at[other] + shift}) == INVALID, (o, other, shift)
                msg = L.nf4moe_last_error().decode()
                assert "overlaps" in msg and o in msg.split() and other in msg.split(), msg
    for o, other in may_be:
        if not torch.cuda.is_available():
            assert status(**{o: at[other]}) == HIP, (o, other)      # every check passed: no device to run on
    if not torch.cuda.is_available():
        assert status() == HIP
        # side by side is not over one another
        o, i = next(iter(outs)), next(iter(ins))
        assert status(**{o: at[i] + size[i]}) == HIP and status(**{o: at[i] - size[o]}) == HIP


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dt", [0, 1])
def test_ckpt8_refuses_overlapping_outputs(fmt, dt):
    rows, K = 64, 1024
    dense, n = rows * K * (4 if dt == 0 else 2), rows * K
    overlaps_refused(lambda x, codes, scale: L.nf4moe_ckpt8_quantize(fmt, x, dt, rows, K, codes, scale, None),
                     dict(codes=n, scale=n // 32), dict(x=dense))
    overlaps_refused(lambda out, codes, scale: L.nf4moe_ckpt8_dequantize(fmt, codes, scale, rows, K, out, dt, None),
                     dict(out=dense), dict(codes=n, scale=n // 32))


@pytest.mark.parametrize("dt", [0, 1])
def test_glu_refuses_overlapping_outputs(dt):
    R, I = 256, 1024
    e, n = (4 if dt == 0 else 2), 256 * 1024
    overlaps_refused(lambda gu, h, codes, scale: L.nf4moe_glu_forward(gu, dt, R, I, 0, 0.0, 0.0, 0, h, 0, codes, scale, None),
                     dict(h=2 * n, codes=2 * n, scale=n // 16), dict(gu=2 * n * e))
    for src, width in ((0, 4), (1, 2), (2, 1), (3, 1)):
        ins = dict(dh=n * e, gu=2 * n * width, row_w=4 * R, **(dict(gu_scale=n // 16) if src > 1 else {}))
        overlaps_refused(lambda dh, gu, row_w, dgu, h, drow_w, gu_scale=None: L.nf4moe_glu_backward(  # noqa: E731
            dh, dt, src, gu, gu_scale, R, I, 0, 0.0, 0.0, 0, row_w, dgu, h, drow_w, None),
            dict(dgu=4 * n, h=2 * n, drow_w=4 * R), ins)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("kind", [1, 2, 3])
def test_block_norm_refuses_overlapping_arrays(dt, kind):
    from bit_quantized_moe_expert_amd import train
    T, H = 256, 1024
    xb, hb, gate = T * H * (4 if dt == 0 else 2), T * H * 2, 4 * (0, H, T, T * H)[kind]

    def desc(w_post, w_pre, g):
        return train._BLOCK_NORM.pack(H, dt, w_post, w_pre, g, kind, 0, 0, 1.0, 1e-6)
    w = dict(w_post=4 * H, w_pre=4 * H, gate=gate)
    overlaps_refused(lambda x, f, w_post, w_pre, gate, x_new, y, rstd_post, rstd_pre: L.nf4moe_block_norm_forward(
        desc(w_post, w_pre, gate), x, f, T, x_new, y, rstd_post, rstd_pre, None),
        dict(x_new=xb, y=hb, rstd_post=4 * T, rstd_pre=4 * T), dict(x=xb, f=hb, **w), may_be=[("x_new", "x")])
    need = L.nf4moe_block_norm_workspace_bytes(H, T)
    overlaps_refused(lambda dx_new, dy, x_new, f, rstd_post, rstd_pre, w_post, w_pre, gate, dx, df, dgate, dw_post, dw_pre, workspace:
                     L.nf4moe_block_norm_backward(desc(w_post, w_pre, gate), dx_new, dy, x_new, f, rstd_post, rstd_pre, T, dx, df,
                                                  dgate, dw_post, dw_pre, workspace, need, None),
                     dict(dx=xb, df=hb, dgate=gate, dw_post=4 * H, dw_pre=4 * H, workspace=need),
                     dict(dx_new=xb, dy=hb, x_new=xb, f=hb, rstd_post=4 * T, rstd_pre=4 * T, **w))


@pytest.mark.parametrize("R", [256, 65536])         # the one-launch form and the grouped kernels
@pytest.mark.parametrize("dt", [0, 1])
def test_adapters_refuse_overlapping_arrays(R, dt):
    from bit_quantized_moe_expert_amd import train
    Ln, rank, K, N, T = 64, 16, 128, 256, 128
    e = 4 if dt == 0 else 2
    d = lambda A, B, scale: train._ADAPTERS.pack(Ln, rank, K, N, A, B, scale)  # noqa: E731
    w = dict(A=2 * Ln * rank * K, B=2 * Ln * rank * N, scale=4 * Ln)
    pb = L.nf4moe_adapter_plan_bytes(R, Ln)
    wf, wb = (L.nf4moe_adapter_workspace_bytes(d(far(0), far(1), 0), R, k) for k in (0, 1))
    overlaps_refused(lambda ids, plan: L.nf4moe_adapter_plan(ids, R, Ln, plan, pb, None), dict(plan=pb), dict(ids=4 * R))
    outs = dict(out=R * N * e, t=4 * R * rank, **(dict(workspace=wf) if wf else {}))
    overlaps_refused(lambda x, x_row_of, ids, plan, base, A, B, scale, out, t, workspace=None: L.nf4moe_adapter_forward(
        d(A, B, scale), x, T, x_row_of, ids, plan, pb, R, base, out, dt, t, workspace, wf, None),
        outs, dict(x=2 * T * K, x_row_of=4 * R, ids=4 * R, plan=pb, base=R * N * e, **w), may_be=[("out", "base")])
    for src, width in ((1, 2), (2, 1)):
        more = dict(x_scale=T * K // 32) if src == 2 else {}
        overlaps_refused(lambda dy, x, x_row_of, t, ids, plan, dx_base, A, B, scale, dx, dA, dB, workspace, x_scale=None:
                         L.nf4moe_adapter_backward(d(A, B, scale), dy, src, x, x_scale, T, x_row_of, t, ids, plan, pb, R, dx_base, dx,
                                                   dt, dA, dB, workspace, wb, None),
                         dict(dx=R * K * e, dA=4 * Ln * rank * K, dB=4 * Ln * rank * N, workspace=wb),
                         dict(dy=2 * R * N, x=width * T * K, x_row_of=4 * R, t=4 * R * rank, ids=4 * R, plan=pb,
                              dx_base=R * K * e, **more, **w), may_be=[("dx", "dx_base")])


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses, which a GPU would dereference")
@pytest.mark.parametrize("plan_bytes", [1 << 46, (1 << 64) - 1])
def test_a_plan_counts_for_its_own_bytes_alone(plan_bytes):
    """A caller may state any size from nf4moe_adapter_plan_bytes up: what lies behind the plan is free for outputs."""
    from bit_quantized_moe_expert_amd import train
    R, Ln = 65536, 64
    d = train._ADAPTERS.pack(Ln, 16, 128, 256, far(0), far(1), 0)
    wf, wb = (L.nf4moe_adapter_workspace_bytes(d, R, k) for k in (0, 1))
    plan, behind = far(3), far(3) + L.nf4moe_adapter_plan_bytes(R, Ln)
    assert L.nf4moe_adapter_forward(d, far(2), R, None, far(4), plan, plan_bytes, R, None, behind, 1, None, far(6), wf, None) == HIP
    assert L.nf4moe_adapter_backward(d, far(2), 1, far(4), None, R, None, far(5), far(6), plan, plan_bytes, R, None, behind, 1,
                                     far(8), far(9), far(10), wb, None) == HIP
    assert L.nf4moe_adapter_forward(d, far(2), R, None, far(4), plan, plan_bytes, R, None, behind - 256, 1, None, far(6), wf,
                                    None) == INVALID
