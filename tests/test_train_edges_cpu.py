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
