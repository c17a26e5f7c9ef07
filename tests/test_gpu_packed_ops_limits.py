"""The building blocks of packed layers at the limits of their inputs and of float32: values that are not
finite, the largest ones, long sums, tails (GPU).  What is expected is the definition in 64 bits.

Tolerances are counted: u = torch.finfo(t).eps / 2 is the largest relative error of one rounding to t.
"""
import pytest
import torch

from diffusion_transformer_denoiser_dit_b200 import attention_packed

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def offsets(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


# ------------------------------------------------------------------ attention


# lengths and heads that reach each way through the keys: single tokens (short, and over several CTAs), few rows
# with too many heads for that, one tile over several CTAs, many tiles
FORMS = {
    "single": ([1, 1, 1], [17, 300, 90], 4, 2), "single_long": ([1, 1], [2500, 5], 4, 1), "few_rows": ([1, 1], [400, 33], 20, 1),
    "few_rows_long": ([1], [9000], 40, 2), "pieces": ([70, 300], [210, 300], 4, 2), "one_piece": ([40], [3000], 4, 4),
    "whole": ([500] * 12, [500] * 12, 16, 16),
}


def inputs(form, d, dtype, seed, std=1.0):
    ql, kl, h, hk = FORMS[form]
    g = gen(seed)
    q = normal(g, sum(ql), h, d, dtype=dtype, std=std)
    q = torch.where(q == 0, torch.full_like(q, 0.5), q)
    return q, normal(g, sum(kl), hk, d, dtype=dtype, std=std), normal(g, sum(kl), hk, d, dtype=dtype), ql, kl


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (72, BF16), (128, FP16)])
@pytest.mark.parametrize("form", ["pieces", "one_piece", "whole"])
def test_attention_masked_values_have_no_weight(form, d, dtype):
    """Values next to the type's largest at keys that a row does not see change no bit of it."""
    q, k, v, ql, kl = inputs(form, d, dtype, d)
    run = lambda v: attention_packed(q, k, v, offsets(ql), offsets(kl), max(ql), max(kl), causal=True, return_lse=True)  # noqa: E731
    want, lse_want = run(v)
    large, blind, a, b = v.clone(), torch.zeros(sum(ql), dtype=torch.bool, device="cuda"), 0, 0
    for nq, nk in zip(ql, kl):
        a, b = a + nq, b + nk
        large[b - nq // 2:b] = torch.finfo(dtype).max * torch.sign(large[b - nq // 2:b])
        blind[a - nq:a - nq // 2] = True
    got, lse = run(large)
    assert torch.equal(got[blind], want[blind]) and torch.equal(lse, lse_want)
