"""Edges of the fine-tuning operators on the GPU: unused adapters, rows without one,
and gates far out on the tails of their function."""
import numpy as np
import pytest

import train_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_moe_expert_amd as M  # noqa: E402

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def to_np(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ adapters
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Rn,rank,src", [(1, 8, "bf16"), (40, 16, M.CKPT_MXINT8), (9000, 24, "bf16"), (9000, 72, M.CKPT_MXFP8)])
def test_gradients_of_an_adapter_without_rows_are_zero(Rn, rank, src, bad):
    """Whatever its scale holds (a slot not in use); the others' gradients are what they are without it."""
    g = torch.Generator(device=DEV).manual_seed(Rn + rank)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    Ln, K, N = 7, 96, 136
    used = torch.tensor([1, 4, -1, Ln, 5], device=DEV)
    ids = used[torch.randint(0, 5, (Rn,), generator=g, device=DEV)].int()
    ids[0] = 4
    unused = [l for l in range(Ln) if not (ids == l).any()]
    assert {0, 2, 3, 6} <= set(unused)
    x, A, B = rn(Rn, K).to(BF16), rn(Ln, rank, K).to(BF16), rn(Ln, N, rank).to(BF16)
    dy, scale = rn(Rn, N).to(BF16), rn(Ln).abs() + 0.5
    held = x if src == "bf16" else M.ckpt8_quantize(x, src)
    _, t = M.adapter_forward(x, A, B, ids, scale=scale, return_t=True)
    want = M.adapter_backward(dy, held, t, A, B, ids, scale=scale)
    wild = scale.clone()
    wild[unused] = bad
    got = M.adapter_backward(dy, held, t, A, B, ids, scale=wild)
    assert all(torch.equal(got[k], want[k]) for k in want)
    for l in unused:
        assert torch.count_nonzero(got["dA"][l]) == 0 and torch.count_nonzero(got["dB"][l]) == 0
    assert torch.equal(M.adapter_forward(x, A, B, ids, scale=wild), M.adapter_forward(x, A, B, ids, scale=scale))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Rn,rank", [(9, 8), (30000, 8), (30000, 16), (12000, 24), (12000, 72)])
def test_rows_without_an_adapter_take_base_as_it_is(Rn, rank, dtype):
    """Its bits: a negative zero keeps its sign, in the one-launch form (9 rows) and in the grouped kernels."""
    g = torch.Generator(device=DEV).manual_seed(Rn + rank)
    Ln, K, N = 3, 520, 264
    ids = torch.randint(-2, Ln + 2, (Rn,), generator=g, device=DEV).int()
    ids[:3] = torch.tensor([-1, 0, Ln], device=DEV)
    x = torch.randn(Rn, K, generator=g, device=DEV).to(BF16)
    A = torch.randn(Ln, rank, K, generator=g, device=DEV).to(BF16)
    B = torch.randn(Ln, N, rank, generator=g, device=DEV).to(BF16)
    base = torch.randn(Rn, N, generator=g, device=DEV)
    fi = torch.finfo(dtype)
    base[:, :6] = torch.tensor([-0.0, 0.0, float("inf"), float("-inf"), fi.max, fi.tiny / 4], device=DEV)
    base = base.to(dtype)
    none = (ids < 0) | (ids >= Ln)
    word = torch.int16 if dtype is BF16 else torch.int32
    out = M.adapter_forward(x, A, B, ids, base=base)
    assert torch.equal(out[none].view(word), base[none].view(word))
    dx_base = base.repeat(1, 2)[:, :K].contiguous()
    back = M.adapter_backward(torch.ones(Rn, N, device=DEV, dtype=BF16), None, None, A, B, ids, dx_base=dx_base, need=("dx",))
    assert torch.equal(back["dx"][none].view(word), dx_base[none].view(word))
