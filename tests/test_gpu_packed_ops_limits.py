"""The building blocks of packed layers at the limits of their inputs and of float32: values that are not
finite, the largest ones, long sums, tails (GPU).  What is expected is the definition in 64 bits.

Tolerances are counted: u = torch.finfo(t).eps / 2 is the largest relative error of one rounding to t.
"""
import math

import pytest
import torch

from diffusion_transformer_denoiser_dit_b200 import attention_packed, linear_fused

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = math.nan, math.inf


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def offsets(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


# ------------------------------------------------------------------ linear


def same_signed(m, n, k, dtype, std, dx, dw):
    """Operands of one sign, in rows dx and dw elements longer than K."""
    g = gen(m + n + k)
    x = normal(g, m, k + dx, dtype=F32, std=std).abs().to(dtype)[:, :k]
    w = normal(g, n, k + dw, dtype=F32, std=std).abs().to(dtype)[:, :k]
    return x, w


def long_sum(x, w):
    """In 64 bits, in parts of K."""
    return sum(a.double() @ b.double().t() for a, b in zip(x.split(8192, 1), w.split(8192, 1)))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("m,n,k,dx,dw", [
    (6, 256, 65536, 0, 0), (130, 700, 65536, 0, 0), (1024, 1152, 16384, 0, 0), (1024, 1152, 65536, 0, 0),
    (1024, 1152, 65535, 0, 0), (1024, 1152, 65536, 4, 2), (2100, 1100, 16390, 1, 0), (4096, 4096, 8190, 0, 0), (9, 72, 40000, 3, 0),
    (300, 2000, 4672, 0, 0), (1024, 1152, 17000, 0, 8), (2048, 4608, 32768, 0, 0),
])
def test_linear_long_float32_sums(m, n, k, dx, dw, dtype):
    """Products of one sign.  The tensor cores cut off what lies below the sum's last place, of the sum and of each of
    the 16 products of a step (fp16's reach lower than bf16's), which is one-sided: a sum taken over every 512 products has
    the mean error of one of 512 products, however long K is.  The roundings to nearest beside it (2^-24 each, at most
    k / 512 + 8 of them) are of either sign and leave less than one 2^-24 in the mean of a thousand outputs; the
    last place varies with the value inside a factor of two, which a mean over parts evens out: 1.1.  A single value is off
    by at most 2^-22 of the sum at each of 32 steps, (33 / 2) 2^-22 of a sum that grows evenly, and all the roundings."""
    x, w = same_signed(m, n, k, dtype, 0.25, dx, dw)

    def off(x, w):
        want = long_sum(x, w)
        return (linear_fused(x, w, out_dtype=F32).double() - want) / want

    # many rows of K = 512: each output's products are in one accumulator (of few, K is cut between CTAs as well)
    whole, one = off(x, w), off(*same_signed(4096, 4096, 512, dtype, 0.25, 0, 0)).mean().abs()
    assert whole.mean().abs() <= 1.1 * one + 2.0 ** -24, (whole.mean().item(), one.item())
    assert whole.abs().max() <= 33 * 2.0 ** -23 + (k / 512 + 8) * 2.0 ** -24, whole.abs().max().item()


@pytest.mark.parametrize("m,n,k,dx", [(6, 256, 65536, 0), (1024, 1152, 20000, 0), (1024, 1152, 20001, 1)])
def test_linear_long_float32_sums_repeat_and_add_the_rest(m, n, k, dx):
    x, w = same_signed(m, n, k, BF16, 0.25, dx, 0)
    b, r = normal(gen(1), n, std=100.0), normal(gen(2), m, n, std=100.0)
    first = linear_fused(x, w, b, act="silu", residual=r, out_dtype=F32)
    want = long_sum(x, w) + b.double()
    want = want * torch.sigmoid(want) + r.double()
    assert ((first.double() - want).abs() / want.abs()).max() <= 40 * 2.0 ** -23 + (k / 512 + 12) * 2.0 ** -24
    for _ in range(3):
        assert torch.equal(first, linear_fused(x, w, b, act="silu", residual=r, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("m,n,k,dx", [(512, 512, 262144, 0), (500, 600, 131077, 1), (2048, 1024, 131072, 0), (1024, 4608, 70000, 0),
                                      (512, 512, 8192, 0), (2048, 1024, 8200, 0), (1024, 4608, 16384, 0)])
def test_linear_long_16_bit_sums(m, n, k, dx, dtype):
    """The sum is taken over every 8192 products: 512 steps of at most 2^-22 of a sum that grows evenly, 513 / 2 2^-22 of the
    whole, however long K is.  The rounding of an output is of either sign, at most u, 0.6 u in the root mean square: five
    deviations of its mean over all outputs."""
    x, w = same_signed(m, n, k, dtype, 0.25, dx, 0)
    want = long_sum(x, w)
    for _ in range(2):
        off = (linear_fused(x, w).double() - want) / want
        u = torch.finfo(dtype).eps / 2
        assert off.mean().abs() <= 513 * 2.0 ** -23 + 5 * 0.6 * u / math.sqrt(m * n), off.mean().item()
        assert off.abs().max() <= 513 * 2.0 ** -23 + u * (1 + 2.0 ** -10) + (k / 8192 + 8) * 2.0 ** -24, off.abs().max().item()


def activation(act, z, sixteen):
    """Value in 64 bits and relative tolerance of the float32 one.  The sigmoid's exponent -z log2 e is rounded, by |z| 2^-24
    of the result, as is its constant; two units of 2^-22 each and a few roundings: (|z| + 8) 2^-23.  Under the
    tanh form its z is 2u, itself off by five roundings of 2^-24.  The erf form: 4.3e-7 of the polynomial, the
    exponential and twice the reciprocal unit's 2^-22 and 2^-23, and six roundings make 1.3e-6 < 2^-19; for 16 bits 8.5e-6
    of the polynomial and the exponent's rounding, at most 120 2^-24, besides: 1.7e-5 < 2^-15."""
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2.0)) / 2, torch.full_like(z, 2.0 ** -15 if sixteen else 2.0 ** -19)
    w = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(w), ((1 if act == "silu" else 3.5) * w.abs() + 8) * 2.0 ** -23


@pytest.mark.parametrize("act,low", [("gelu", -12.5), ("silu", -80.0), ("gelu_tanh", -9.0)])
@pytest.mark.parametrize("m", [1, 3, 200, 4096])
def test_linear_activations_keep_their_tails(m, act, low):
    """The argument is the bias alone, exact, from where the result leaves float32's range of digits up to 30."""
    n = 4096
    z = torch.cat([torch.linspace(low, 0, n // 2, device="cuda"), torch.linspace(0, 30, n // 2, device="cuda")])
    for dtype in (BF16, FP16):
        x, w = torch.zeros(m, 64, dtype=dtype, device="cuda"), torch.ones(n, 64, dtype=dtype, device="cuda")
        want, tol = activation(act, z.double(), False)
        got = linear_fused(x, w, z, act=act, out_dtype=F32).double()
        assert ((got - want).abs() <= want.abs() * tol).all(), ((got - want) / want).abs().max().item()
        want, tol = activation(act, z.double(), True)
        got = linear_fused(x, w, z, act=act).double()
        small = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2   # half a step of the subnormal values
        assert ((got - want).abs() <= want.abs() * (tol + torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -10)) + small).all()


def test_linear_activations_of_what_is_not_finite():
    z = torch.tensor([NAN, INF, -INF, 1e30, -1e30, 0.0], device="cuda")
    x, w = torch.zeros(2, 8, dtype=BF16, device="cuda"), torch.ones(6, 8, dtype=BF16, device="cuda")
    for act in ("gelu", "silu", "gelu_tanh"):
        for t in (F32, BF16):
            y = linear_fused(x, w, z, act=act, out_dtype=t)[0]
            assert torch.isnan(y[0]) and y[1] == INF and torch.isnan(y[2]) and y[3] == z[3].to(t) and y[4] == 0 and y[5] == 0


# ------------------------------------------------------------------ attention


def attention_want(q, k, v, ql, kl, causal, scale):
    """out, its tolerance, lse, its tolerance in 64 bits; a row that sees a NaN or +inf score is NaN, one whose
    scores are all -inf (or that sees no key) is 0 with lse -inf.

    A score is off by ds <= scale sum|q||k| 2^-22 (dh / 16 + 2) (the products' sum in the tensor cores) and by 2^-22
    of itself and of the row's maximum (scale log2 e in float32, the product, the subtraction of the maximum).  The
    base-2 exponential is off by 3e-6 of its value (the quartic 2.8e-6, the exponential unit 2^-22), the float32 sum by
    2^-24 for each of at most nk / 128 + 48 additions.  In the output each of these counts in numerator and
    sum; a probability is rounded to the type for the product with v: by u of its value, or for fp16 below 2^-14 by 2^-25
    of a reference that is at most the row's sum; that product's sum drops 2^-22 per 16 keys; then one rounding."""
    h, hk = q.shape[1], k.shape[1]
    u = half_step(q.dtype)
    small = 2.0 ** -25 if q.dtype == FP16 else 0.0
    outs, tols, logs, ltols = [], [], [], []
    a = b = 0
    for nq, nk in zip(ql, kl):
        qq = q[a:a + nq].double().transpose(0, 1)
        kk = k[b:b + nk].double().repeat_interleave(h // hk, 1).transpose(0, 1)
        vv = v[b:b + nk].double().repeat_interleave(h // hk, 1).transpose(0, 1)
        a, b = a + nq, b + nk
        s = qq @ kk.transpose(1, 2) * scale
        if causal:
            i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")
            s = s.masked_fill(j > i + nk - nq, -INF)
        top = s.amax(-1, keepdim=True) if nk else torch.full((h, nq, 1), -INF, dtype=torch.float64, device="cuda")
        bad = torch.isnan(top) | (top == INF)
        none = top == -INF
        z = torch.logsumexp(s.masked_fill(bad, 0), -1, keepdim=True) if nk else top
        p = torch.exp(s - z.masked_fill(none, 0)).masked_fill(bad, 0)
        fin = lambda t: torch.nan_to_num(t.abs(), 0, 0, 0)  # noqa: E731
        ds = fin(qq) @ fin(kk).transpose(1, 2) * scale * 2.0 ** -22 * (q.shape[2] / 16 + 2) + (fin(s) + fin(top)) * 2.0 ** -22
        add = (nk / 128 + 48) * 2.0 ** -24
        # a weight of exactly 0 takes nothing of its value, however large that is
        o = torch.where(p[..., None] > 0, p[..., None] * vv[:, None], 0).sum(-2) if nk < 600 else p @ vv
        each = p * (2 * (ds + 3e-6 + add) + u + 2.0 ** -22 * (nk / 16 + 4)) + small * (p > 0)
        err = torch.where(each[..., None] > 0, each[..., None] * vv.abs()[:, None], 0).sum(-2) if nk < 600 else each @ vv.abs()
        nan = torch.full_like(o, NAN)
        outs.append(torch.where(bad, nan, torch.where(none, 0 * nan.nan_to_num(0), o)).transpose(0, 1))
        tols.append((err + (o.abs() + err) * u + torch.finfo(q.dtype).tiny).transpose(0, 1))
        logs.append(torch.where(bad, torch.full_like(z, NAN), z)[..., 0])
        ltols.append((p * (ds + 3e-6)).sum(-1) + add + fin(z[..., 0]) * 2.0 ** -21 + 1e-6)
    return torch.cat(outs), torch.cat(tols), torch.cat(logs, 1), torch.cat(ltols, 1)


def same(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (what, "NaN", int(torch.isnan(got).sum()), int(torch.isnan(want).sum()))
    fine = torch.isfinite(want)
    rest = ~fine & ~torch.isnan(want)
    assert torch.equal(got[rest], want[rest]), (what, "inf")
    off = (got[fine] - want[fine]).abs() - tol[fine]
    assert off.numel() == 0 or off.max() <= 0, (what, off.max().item(), int((off > 0).sum()))


def check_attention(q, k, v, ql, kl, causal, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, tol, lse_want, lse_tol = attention_want(q, k, v, ql, kl, causal, scale)
    got, lse = attention_packed(q, k, v, offsets(ql), offsets(kl), max(ql), max(kl), causal=causal, scale=scale, return_lse=True)
    same(got, want, tol, "out")
    same(lse, lse_want, lse_tol, "lse")
    return got, lse


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


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, FP16), (72, BF16)])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_attention_nan_in_a_query_or_a_key_is_seen(form, d, dtype, causal):
    q, k, v, ql, kl = inputs(form, d, dtype, d)
    check_attention(q, k, v, ql, kl, causal)
    bad = q.clone()
    bad[0, 0, 1], bad[-1, -1, d - 1] = NAN, NAN
    got, lse = check_attention(bad, k, v, ql, kl, causal)
    assert torch.isnan(got[0, 0]).all() and torch.isnan(lse[0, 0]) and torch.isnan(got[-1, -1]).all()
    # one key at a time, at places of every kind inside a tile; then all of a sequence's
    for at in (0, 8, 9, 16, kl[0] - 1):
        bad = k.clone()
        bad[at, 0, 3] = NAN
        check_attention(q, bad, v, ql, kl, causal)
    bad = k.clone()
    bad[:kl[0], :, 0] = NAN
    check_attention(q, bad, v, ql, kl, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_attention_infinite_scores(form, d, dtype, causal):
    """A key with an infinite feature scores +inf or -inf by the sign of the query's: the first makes the row NaN, the
    second leaves the key out; a row whose scores are all -inf has no weight on any key."""
    q, k, v, ql, kl = inputs(form, d, dtype, d + 1)
    for at in (0, 8, 16, kl[0] - 1):
        bad = k.clone()
        bad[at, :, 5] = INF
        check_attention(q, bad, v, ql, kl, causal)
    bad = k.clone()
    bad[:kl[0], :, 5] = INF
    got, lse = check_attention(q, bad, v, ql, kl, causal)
    left_out = (q[0, :, 5] < 0)
    assert left_out.any() and (got[0][left_out] == 0).all() and (lse[left_out, 0] == -INF).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_attention_scores_that_overflow(form, sign):
    """A score that is finite until it is scaled (64 equal products, 1e38 in all, times 8): as an infinite one.  Of
    mixed signs, partial sums of such products may overflow on the way, so that nothing is said of those."""
    q, k, v, ql, kl = inputs(form, 64, BF16, 7)
    q, k = q.clone(), k.clone()
    q[0], k[3] = 1.25e18, sign * 1.25e18
    k[:3], k[4:kl[0]] = k[:3].abs() * 1e-18, k[4:kl[0]].abs() * 1e-18
    got, lse = attention_packed(q, k, v, offsets(ql), offsets(kl), max(ql), max(kl), scale=8.0, return_lse=True)
    if sign > 0:
        assert torch.isnan(got[0]).all() and torch.isnan(lse[:, 0]).all()
        return
    keep = [j for j in range(kl[0]) if j != 3]       # that key has no weight, the others theirs
    want, tol, lse_want, lse_tol = attention_want(q[:1], k[:kl[0]][keep], v[:kl[0]][keep], [1], [kl[0] - 1], False, 8.0)
    same(got[:1], want, tol, "out")
    same(lse[:, :1], lse_want, lse_tol, "lse")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_attention_one_key_with_nearly_all_weight(form, d):
    """Scores of 10 at one key and small ones elsewhere: the log-sum-exp shows the error of that key's exponential alone, at
    places that every unit computes.  Its tolerance (4.1e-5 at most by the count above) is far below 7e-5: an exponential
    that is off by that at 2^0, as a cubic fitted on [-1/2, 1/2] is, does not pass."""
    q, k, v, ql, kl = inputs(form, d, BF16, 21)
    k = (k.float() * 0.05).to(BF16)
    for at in (0, 3, 8, 9, 16):
        one = k.clone()
        one[at] = 0.25
        qq = torch.full_like(q, 10 * d ** 0.5 / (0.25 * d))   # 10 = scale d 0.25 q
        _, _, lse, tol = attention_want(qq, one, v, ql, kl, False, d ** -0.5)
        assert tol[:, :ql[0]].max() < 5e-5
        check_attention(qq, one, v, ql, kl, False)
        check_attention(qq, one, v, ql, kl, True)
