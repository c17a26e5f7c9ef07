"""The building blocks of a layer over packed sequences against their definitions in 64 bits (GPU).

Tolerances are counted, not fitted.  u = torch.finfo(t).eps / 2 is the largest relative error
of one rounding to t.  The tensor cores add 16 products at a time to a 32-bit sum and may drop
what is below its last place, at most 2^-22 of the sum of magnitudes per step.
"""
import math

import pytest
import torch

from diffusion_transformer_denoiser_dit_b200 import DitError, Rotary, attention_packed, binding, linear_fused

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def close(got, want, tol, what=""):
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(got.double()).any(), what
    assert (off <= 0).all(), (what, off.max().item(), int((off > 0).sum()))


# ------------------------------------------------------------------ linear


ACTS = {
    "none": lambda z: z,
    "relu": lambda z: z.clamp(min=0),
    "gelu_tanh": lambda z: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)),
    "gelu": lambda z: z * torch.special.ndtr(z),
    "silu": lambda z: z * torch.sigmoid(z),
}


def linear_want(x, w, bias, act, residual, out_dtype):
    """(value, tolerance) in 64 bits: the sum's own error reaches the output through a slope of
    at most 1.13 (the activations' steepest); the activation itself is good to 2^-18 of its
    argument (exponential and reciprocal units); then one rounding."""
    k = x.shape[1]
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    err = mag * 2.0 ** -22 * (k / 16 + 4)
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    y = ACTS[act](z)
    err = 1.13 * (err + z.abs() * 2.0 ** -18)
    if residual is not None:
        y = y + residual.double()
    return y, err + (y.abs() + err) * (half_step(out_dtype) + 2.0 ** -22) + torch.finfo(out_dtype).tiny


def check_linear(x, w, bias=None, act="none", residual=None, out_dtype=None, out=None):
    t = out_dtype or x.dtype
    want, tol = linear_want(x, w, bias, act, residual, t)
    got = linear_fused(x, w, bias, act=act, residual=residual, out_dtype=out_dtype, out=out)
    assert got.dtype == t and got.shape == want.shape
    close(got, want, tol, (tuple(x.shape), tuple(w.shape), act))
    return got


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 4608, 1152), (1, 130, 4608), (2, 33, 7), (3, 1000, 588), (5, 64, 8), (8, 1152, 1152), (9, 257, 64),
    (16, 384, 1536), (17, 1153, 588), (32, 6912, 1152), (64, 96, 63), (100, 31, 4096), (127, 129, 65), (128, 128, 128),
    (129, 256, 200), (200, 1152, 4608), (256, 256, 64), (257, 513, 1000), (300, 2, 72), (1024, 1152, 1152),
    (1111, 1153, 588), (2048, 2304, 768), (1, 70000, 16), (70000, 8, 16),
])
def test_linear_shapes(dtype, m, n, k):
    g = gen(m * 7 + n * 3 + k)
    x, w = normal(g, m, k, dtype=dtype), normal(g, n, k, dtype=dtype, std=k ** -0.5)
    check_linear(x, w)
    b, r = normal(g, n), normal(g, m, n)
    check_linear(x, w, b, "gelu_tanh")
    check_linear(x, w, b, residual=r, out_dtype=F32)
    check_linear(x, w, None, "silu", residual=r.to(dtype))


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("m", [4, 70, 640])
def test_linear_activations(act, m):
    """Sums from -30 to 30, where the activations' tails are, in every output type."""
    g = gen(m)
    for dtype in (BF16, FP16):
        x, w = normal(g, m, 96, dtype=dtype), normal(g, 200, 96, dtype=dtype)
        b = normal(g, 200, std=5.0)
        check_linear(x, w, b, act)
        check_linear(x, w, b, act, out_dtype=F32)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("m,n,k,dx,dw", [(3, 100, 96, 1, 0), (300, 200, 96, 0, 1), (300, 200, 97, 3, 5),
                                         (260, 130, 640, 4, 4), (150, 520, 72, 8, 0), (40, 70, 1000, 2, 1)])
def test_linear_strides_and_alignment(dtype, m, n, k, dx, dw):
    """Slices of wider matrices that start anywhere, and an output inside a wider one whose
    other values stay as they were."""
    g = gen(k)
    x = normal(g, m, k + 24, dtype=dtype)[:, dx:dx + k]
    w = normal(g, n, k + 24, dtype=dtype)[:, dw:dw + k] * k ** -0.5
    wide = torch.full((n, k + 24), 7.0, dtype=dtype, device="cuda")
    wide[:, dw:dw + k] = w
    for t in (dtype, F32):
        for at in (0, 1, 8):
            whole = torch.full((m + 2, n + 16), -5.0, dtype=t, device="cuda")
            r = normal(g, m, n + 3).to(t)[:, 1:1 + n]
            check_linear(x, wide[:, dw:dw + k], normal(g, n), "relu", residual=r, out_dtype=t,
                         out=whole[1:-1, at:at + n])
            outside = whole.clone()
            outside[1:-1, at:at + n] = -5.0
            assert (outside == -5.0).all()


@pytest.mark.parametrize("m", [2, 50, 400])
def test_linear_broadcast_and_in_place(m):
    g = gen(m)
    x, w, b = normal(g, m, 128, dtype=BF16), normal(g, 136, 128, dtype=BF16, std=0.1), normal(g, 136)
    row = normal(g, 1, 136)
    check_linear(x, w, b, residual=row.expand(m, 136), out_dtype=F32)          # one row for all
    check_linear(x[:1].expand(m, 128), w, b)                                   # rows of x that share memory
    check_linear(x, w[:1].expand(136, 128), b)
    h = normal(g, m, 136)
    want, tol = linear_want(x, w, b, "none", h, F32)
    close(linear_fused(x, w, b, residual=h, out=h), want, tol)                 # the residual stream, in place
    h16 = normal(g, m, 136, dtype=BF16)
    want, tol = linear_want(x, w, b, "gelu", h16, BF16)
    close(linear_fused(x, w, b, act="gelu", residual=h16, out=h16), want, tol)


def test_linear_long_sums_keep_32_bits():
    """A float32 output: same-signed products, whose truncated sum would drift with K.  Chunks of
    512 products are at most 32 steps of truncation each."""
    g = gen(1)
    for m in (6, 256):
        x, w = normal(g, m, 16384, dtype=BF16).abs(), normal(g, 256, 16384, dtype=BF16).abs()
        want = x.double() @ w.double().t()
        got = linear_fused(x, w, out_dtype=F32)
        assert ((got.double() - want).abs() / want).max() < 32 * 2.0 ** -22 + 34 * 2.0 ** -24


@pytest.mark.parametrize("m", [3, 40, 300])
def test_linear_nan_and_inf_stay_in_their_rows(m):
    g = gen(m)
    x, w = normal(g, m, 200, dtype=BF16), normal(g, 150, 200, dtype=BF16)
    x[1, 5], x[2, 7], w[9, 3] = float("nan"), float("inf"), float("nan")
    y = linear_fused(x, w)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any() and torch.isnan(y[:, 9]).all()
    keep = torch.ones(m, 150, dtype=torch.bool, device="cuda")
    keep[1], keep[2], keep[:, 9] = False, False, False
    want, tol = linear_want(x.nan_to_num(0, 0, 0), w.nan_to_num(0, 0, 0), None, "none", None, BF16)
    close(y[keep], want[keep], tol[keep])


def test_linear_empty():
    w = torch.zeros(8, 16, dtype=BF16, device="cuda")
    assert linear_fused(torch.zeros(0, 16, dtype=BF16, device="cuda"), w).shape == (0, 8)
    with pytest.raises(DitError):
        linear_fused(torch.zeros(3, 0, dtype=BF16, device="cuda"), torch.zeros(8, 0, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("m,n,k", [(1, 1152, 4608), (24, 1152, 4608), (1000, 1152, 1152)])
def test_linear_repeats_bit_for_bit(m, n, k):
    g = gen(k)
    x, w, b = normal(g, m, k, dtype=BF16), normal(g, n, k, dtype=BF16), normal(g, n)
    first = linear_fused(x, w, b, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(first, linear_fused(x, w, b, out_dtype=F32))


# ------------------------------------------------------------------ attention


def offsets(lengths, start=0):
    return torch.tensor([start] + lengths, device="cuda").cumsum(0).to(torch.int32)


def attention_want(q, k, v, ql, kl, causal, scale, q0=0, k0=0):
    """out, tolerance, lse, its tolerance: [tokens, heads, dh] and [heads, tokens] in 64 bits.

    A score is off by ds <= scale sum|q||k| 2^-22 (dh / 16 + 2) and the base-2 exponential by
    1e-4 of its value (a cubic on part of them), in numerator and sum: 2 (ds + 1e-4); each
    probability is rounded to the type for the product with v: u; the sum over the keys drops
    2^-22 per 16 keys; then one rounding."""
    h, hk = q.shape[1], k.shape[1]
    u = half_step(q.dtype)
    outs, tols, logs, ltols = [], [], [], []
    a, b = q0, k0
    for nq, nk in zip(ql, kl):
        qq = q[a:a + nq].double().transpose(0, 1)
        kk = k[b:b + nk].double().repeat_interleave(h // hk, 1).transpose(0, 1)
        vv = v[b:b + nk].double().repeat_interleave(h // hk, 1).transpose(0, 1)
        a, b = a + nq, b + nk
        s = qq @ kk.transpose(1, 2) * scale
        ds = (qq.abs() @ kk.abs().transpose(1, 2) * scale * 2.0 ** -22 * (q.shape[2] / 16 + 2)) + s.abs() * 2.0 ** -22
        if causal:
            i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")
            s = s.masked_fill(j > i + nk - nq, -math.inf)
        z = torch.logsumexp(s, -1) if nk else torch.full((h, nq), -math.inf, dtype=torch.float64, device="cuda")
        p = torch.exp(s - z.masked_fill(z == -math.inf, 0)[..., None])
        each = 2 * (ds + 1e-4) + u + 2.0 ** -22 * (nk / 16 + 4)
        o = p @ vv
        err = (p * each) @ vv.abs() + p.sum(-1, keepdim=True) * 0
        outs.append(o.transpose(0, 1))
        tols.append((err + (o.abs() + err) * u + torch.finfo(q.dtype).tiny).transpose(0, 1))
        logs.append(z)
        ltols.append((p * (ds + 1e-4)).sum(-1) + z.abs().masked_fill(z == -math.inf, 0) * 2.0 ** -21 + 1e-6)
    return torch.cat(outs), torch.cat(tols), torch.cat(logs, 1), torch.cat(ltols, 1)


def check_attention(q, k, v, ql, kl, causal, scale=None, out=None):
    want, tol, lse_want, lse_tol = attention_want(q, k, v, ql, kl, causal, q.shape[2] ** -0.5 if scale is None else scale)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = attention_packed(q, k, v, offsets(ql), offsets(kl), max(ql), max(kl), causal=causal, scale=scale, out=out,
                                return_lse=True, status=status)
    assert int(status.item()) == 0
    n = sum(ql)
    close(got[:n], want, tol, "out")
    lse = lse[:, :n]
    none = lse_want == -math.inf
    assert torch.equal(lse == -math.inf, none)
    close(lse[~none], lse_want[~none], lse_tol[~none], "lse")
    return got


def qkv(g, ql, kl, h, hk, d, dtype, std=1.0):
    return (normal(g, sum(ql), h, d, dtype=dtype, std=std), normal(g, sum(kl), hk, d, dtype=dtype, std=std),
            normal(g, sum(kl), hk, d, dtype=dtype))


LENGTHS = [
    ([1], [1]), ([5], [5]), ([1], [300]), ([128], [128]), ([129], [257]), ([300], [77]), ([256], [1024]),
    ([1, 0, 7, 130, 1], [1, 3, 0, 130, 900]), ([64, 200, 333], [64, 200, 333]), ([0, 0, 2], [5, 0, 2]),
    ([1, 1, 1, 1, 1, 1], [1, 17, 128, 129, 640, 2000]), ([2, 3, 1], [511, 4, 1025]),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("ql,kl", LENGTHS)
def test_attention_lengths(ql, kl, causal):
    for dtype, h, hk, d in ((BF16, 4, 2, 64), (FP16, 6, 2, 128), (BF16, 3, 3, 72)):
        g = gen(sum(ql) + sum(kl) + d)
        check_attention(*qkv(g, ql, kl, h, hk, d, dtype), ql, kl, causal)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 64, 72, 80, 96, 104, 112, 120, 128])
def test_attention_head_dims(d, dtype):
    for ql, kl in (([200, 31], [200, 400]), ([1, 2], [700, 90])):
        g = gen(d)
        check_attention(*qkv(g, ql, kl, 4, 2, d, dtype), ql, kl, True)


@pytest.mark.parametrize("h,hk", [(1, 1), (8, 1), (5, 1), (14, 2), (24, 8), (64, 1), (128, 1), (100, 2), (127, 1)])
def test_attention_groups(h, hk):
    for ql, kl in (([70, 1, 40], [150, 260, 40]), ([1, 1], [1000, 3])):
        g = gen(h)
        check_attention(*qkv(g, ql, kl, h, hk, 64, BF16), ql, kl, True)
        check_attention(*qkv(g, ql, kl, h, hk, 72, FP16), ql, kl, False)


def test_attention_strides():
    """q, k and v inside one projection's output, heads before tokens, and an output inside a wider one."""
    g = gen(5)
    ql = kl = [100, 1, 299]
    n, h, hk, d = sum(ql), 6, 2, 64
    fused = normal(g, n, (h + 2 * hk) * d + 8, dtype=BF16)
    q = fused[:, :h * d].unflatten(1, (h, d))
    k, v = (fused[:, (h + i * hk) * d:(h + (i + 1) * hk) * d].unflatten(1, (hk, d)) for i in (0, 1))
    whole = torch.full((n + 3, h + 1, d + 8), 3.0, dtype=BF16, device="cuda")
    check_attention(q, k, v, ql, kl, True, out=whole[:n, :h, :d])
    assert (whole[n:] == 3).all() and (whole[:, h] == 3).all() and (whole[:, :, d:] == 3).all()
    q, k, v = (normal(g, c, n, d, dtype=BF16).transpose(0, 1) for c in (h, hk, hk))
    check_attention(q, k, v, ql, kl, False)


@pytest.mark.parametrize("ql,kl", [([130, 60], [130, 200]), ([1, 1], [77, 500]), ([3], [40])])
def test_attention_leaves_and_ignores_what_is_outside(ql, kl):
    """Rows before, behind and between the sequences' ends: NaN and infinite keys and values
    there change nothing, output rows there stay as they were."""
    for d in (64, 128, 72):
        g = gen(d)
        q, k, v = qkv(g, ql, kl, 4, 2, d, BF16)
        want = attention_packed(q, k, v, offsets(ql), offsets(kl), max(ql), max(kl), causal=True)
        pad = lambda t, a, b, f: torch.cat((torch.full_like(t[:1], f).expand(a, -1, -1), t,  # noqa: E731
                                            torch.full_like(t[:1], f).expand(b, -1, -1)))
        nan, inf = float("nan"), float("inf")
        out = torch.full((sum(ql) + 200, 4, d), 9.0, dtype=BF16, device="cuda")
        for fk, fv in ((nan, nan), (inf, -inf)):
            got = attention_packed(pad(q, 60, 140, nan), pad(k, 33, 300, fk), pad(v, 33, 300, fv), offsets(ql, 60),
                                   offsets(kl, 33), max(ql), max(kl), causal=True, out=out)
            assert torch.equal(got[60:60 + sum(ql)], want)
            assert (got[:60] == 9).all() and (got[60 + sum(ql):] == 9).all()


@pytest.mark.parametrize("h,hk", [(2, 2), (8, 2)])
def test_attention_other_sequences_do_not_leak(h, hk):
    g = gen(11)
    ql, kl = [33, 1, 140], [33, 90, 140]
    q, k, v = qkv(g, ql, kl, h, hk, 64, FP16)
    want = attention_packed(q, k, v, offsets(ql), offsets(kl), 140, 140)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    k2[33:123], v2[33:123], q2[33:34] = float("nan"), float("inf"), float("nan")
    got = attention_packed(q2, k2, v2, offsets(ql), offsets(kl), 140, 140)
    assert torch.equal(got[:33], want[:33]) and torch.equal(got[34:], want[34:])


@pytest.mark.parametrize("ql,kl", [([256], [1024]), ([1, 2], [1500, 700])])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_growing_scores(ql, kl, causal):
    """Keys that grow along the sequence: the running maximum climbs by far more than the
    exponential's comfortable range, again and again; and falling ones, whose later weights vanish."""
    for dtype in (BF16, FP16):
        g = gen(3)
        q, k, v = qkv(g, ql, kl, 4, 2, 64, dtype)
        ramp = torch.cat([torch.linspace(0.1, 12, n, device="cuda") for n in kl])[:, None, None]
        check_attention(q, (k * ramp).to(dtype), v, ql, kl, causal)
        check_attention(q, (k * ramp.flip(0)).to(dtype), v, ql, kl, causal)
        check_attention((q * 0).to(dtype), k, v, ql, kl, causal)                  # flat: the mean of v
        check_attention(q, k, v, ql, kl, causal, scale=3.0)


def test_attention_long_cache():
    for ql, kl, h, hk, d in (([1], [33000], 8, 2, 128), ([1, 1], [20001, 5], 4, 4, 72), ([5], [9999], 8, 1, 64)):
        g = gen(kl[0])
        check_attention(*qkv(g, ql, kl, h, hk, d, BF16), ql, kl, True)


def test_attention_many_sequences():
    g = gen(2)
    ql = [(i * 7) % 5 for i in range(5000)]
    kl = [(i * 3) % 9 for i in range(5000)]
    check_attention(*qkv(g, ql, kl, 2, 1, 64, BF16), ql, kl, False)
    ql = [1] * 3000
    kl = [1 + i % 40 for i in range(3000)]
    check_attention(*qkv(g, ql, kl, 4, 2, 128, BF16), ql, kl, True)


def test_attention_no_keys_at_all():
    q = torch.ones(9, 2, 64, dtype=BF16, device="cuda")
    k = torch.empty(0, 1, 64, dtype=BF16, device="cuda")
    out, lse = attention_packed(q, k, k, offsets([4, 5]), offsets([0, 0]), 5, 0, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert attention_packed(q[:0], k, k, offsets([0]), offsets([0]), 0, 0).shape == (0, 2, 64)


def test_attention_hints_only_choose_the_split():
    """max_q and max_k that are too small or too large give the same values within the tolerance."""
    g = gen(8)
    ql, kl = [1, 200, 3], [900, 200, 64]
    q, k, v = qkv(g, ql, kl, 4, 2, 64, BF16)
    want, tol, _, _ = attention_want(q, k, v, ql, kl, True, 0.125)
    for mq, mk in ((200, 900), (1, 1), (0, 0), (10000, 100000), (1, 100000), (200, 1)):
        close(attention_packed(q, k, v, offsets(ql), offsets(kl), mq, mk, causal=True), want, tol, (mq, mk))


@pytest.mark.parametrize("ql,kl", [([1, 1], [3000, 100]), ([300, 77], [300, 500])])
def test_attention_repeats_bit_for_bit(ql, kl):
    g = gen(4)
    q, k, v = qkv(g, ql, kl, 8, 2, 128, BF16)
    run = lambda: attention_packed(q, k, v, offsets(ql), offsets(kl), max(ql), max(kl), causal=True)  # noqa: E731
    first = run()
    for _ in range(5):
        assert torch.equal(first, run())


# few rows per sequence: by clusters of one, two, four and eight (few items, many keys), more sequences than
# are ordered at one time, sequences of no queries whose keys are NaN, and hints of one query where there are more
FEW = [
    ([1], [1], 1), ([1], [16], 1), ([1, 1, 1], [16, 0, 17], 1), ([1, 0, 1, 1], [63, 64, 65, 513], 1), ([2, 1], [1, 4], 2),
    ([1] * 5, [1000, 1, 130, 999, 64], 1), ([1, 1], [300, 4000], 1), ([3, 7, 1, 0], [200, 3, 640, 20], 1),
    ([1, 0, 2, 1, 1] * 14, [3, 70, 33, 128, 260] * 14, 2), ([1] * 40, list(range(0, 400, 10)), 1),
]


@pytest.mark.parametrize("ql,kl,hint", FEW)
@pytest.mark.parametrize("h,hk,d,dtype", [(1, 1, 8, BF16), (4, 4, 64, FP16), (12, 4, 72, BF16), (16, 1, 128, FP16), (10, 2, 104, BF16),
                                          (16, 2, 40, BF16)])
def test_attention_of_few_rows(ql, kl, hint, h, hk, d, dtype):
    g = gen(12)
    q, k, v = qkv(g, ql, kl, h, hk, d, dtype)
    at = 0
    for nq, nk in zip(ql, kl):
        if nq == 0:
            k[at:at + nk], v[at:at + nk] = float("nan"), float("inf")
        at += nk
    room = 3                                         # keys and queries behind the last sequence
    k, v = (torch.cat([x, torch.full_like(x[:1].expand(room, -1, -1), float("nan"))]) for x in (k, v)) if sum(kl) else (k, v)
    for causal in (False, True):
        want, tol, lse_want, lse_tol = attention_want(q, k, v, ql, kl, causal, d ** -0.5)
        out = torch.full((sum(ql) + room, h, d), 7.0, device="cuda", dtype=dtype)
        qq = torch.cat([q, q.new_full((room, h, d), float("nan"))])
        got, lse = attention_packed(qq, k, v, offsets(ql), offsets(kl), hint, max(kl), causal=causal, out=out, return_lse=True)
        n = sum(ql)
        close(got[:n], want, tol, causal)
        assert (got[n:] == 7).all()
        none = lse_want == -math.inf
        assert torch.equal(lse[:, :n] == -math.inf, none)
        close(lse[:, :n].masked_fill(none, 0), lse_want.masked_fill(none, 0), lse_tol, "lse")
        again = attention_packed(qq, k, v, offsets(ql), offsets(kl), hint, max(kl), causal=causal)
        assert torch.equal(again[:n], got[:n])


def test_attention_of_few_rows_with_strides_and_large_scores():
    """Heads and tokens interleaved in memory; scores whose maximum moves by far more than 2^8."""
    g = gen(13)
    ql, kl, d = [1, 2, 1], [70, 400, 1], 72
    buf = normal(g, sum(kl), 2, 4, 80, dtype=BF16, std=6.0)
    k, v = buf[:, 0, :, :d], buf[:, 1, :, :d]
    q = normal(g, 12, sum(ql), 96, dtype=BF16, std=6.0).transpose(0, 1)[:, :, :d]
    out = torch.zeros(sum(ql), 12, 88, device="cuda", dtype=BF16)[:, :, :d]
    for causal in (False, True):
        check_attention(q, k, v, ql, kl, causal, out=out)
        check_attention(q, k, v, ql, kl, causal, scale=3.0, out=out)


# ------------------------------------------------------------------ rotary


def rotary_want(x, pos, freqs, part, axes, interleaved, amp, transpose=False):
    """Value and tolerance: the angle is good to 2^-25 turns and cos, sin to 2^-22; two products and one
    sum in 32 bits; one rounding."""
    t = pos.double().reshape(-1, axes, 1) * freqs
    t = t.flatten(1)[:, None]
    c, s = torch.cos(t) * amp, torch.sin(t) * amp * (-1 if transpose else 1)
    y = x.double().clone()
    a, b = (slice(0, part, 2), slice(1, part, 2)) if interleaved else (slice(0, part // 2), slice(part // 2, part))
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    mag = torch.zeros_like(y)
    mag[..., a] = mag[..., b] = xa.abs() + xb.abs()
    err = mag * amp * (2 * math.pi * 2.0 ** -25 + 3 * 2.0 ** -22)
    return y, err + y.abs() * half_step(x.dtype) * (mag > 0) + torch.finfo(x.dtype).tiny


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
@pytest.mark.parametrize("n,h,d,part,axes,inter", [
    (1, 1, 2, 2, 1, False), (1, 40, 128, 128, 1, False), (7, 3, 72, 72, 3, True), (33, 2, 72, 36, 1, False),
    (5, 16, 128, 64, 1, False), (300, 4, 64, 64, 2, True), (50, 5, 80, 10, 1, True), (17, 3, 9, 6, 3, False),
    (4, 2, 512, 512, 1, False), (1000, 20, 96, 96, 1, True), (3, 1, 7, 2, 1, True), (129, 1, 256, 64, 4, False),
])
def test_rotary(dtype, n, h, d, part, axes, inter):
    g = gen(n + d)
    each = part // 2 // axes
    freqs = 10000.0 ** (-torch.arange(each, dtype=torch.float64, device="cuda") / each)
    x = normal(g, n, h, d, dtype=dtype)
    rot = Rotary(d, rotary_dim=part, interleaved=inter, axes=axes)
    for low, high, t in ((0, 4096, torch.int32), (-(2 ** 20), 2 ** 20, torch.int64)):
        pos = torch.randint(low, high, (n, axes), device="cuda", generator=g).to(t)
        for tr in (False, True):
            want, tol = rotary_want(x, pos, freqs, part, axes, inter, 1.0, tr)
            close(rot.apply(x, pos, transpose=tr), want, tol)
    same = x.clone()
    assert torch.equal(rot.apply(same, pos, out=same), rot.apply(x, pos))


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
def test_rotary_scalings(scaling, factor):
    g = gen(9)
    x, pos = normal(g, 40, 3, 64), torch.randint(0, 60000, (40,), device="cuda", generator=g)
    i = torch.arange(32, dtype=torch.float64, device="cuda") / 32
    f, amp = 10000.0 ** -i, 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ntk":
        f = (10000.0 * factor ** (32 / 31)) ** -i
    else:
        keep = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f, amp = keep * f + (1 - keep) * f / factor, 0.1 * math.log(factor) + 1
    want, tol = rotary_want(x, pos, f, 64, 1, False, amp)
    rot = Rotary(64, scaling=scaling, factor=factor, original_length=4096)
    close(rot.apply(x, pos), want, tol)
    own = Rotary(64, freqs=(f.tolist()))
    if scaling != "yarn":
        close(own.apply(x, pos), want, tol)


def test_rotary_strides_and_offsets():
    """Queries and keys inside one projection turn in place; unaligned slices; heads before tokens."""
    g = gen(6)
    n, h, d = 65, 5, 64
    freqs = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    pos = torch.randint(0, 9999, (n,), device="cuda", generator=g)
    rot = Rotary(d)
    fused = normal(g, n, (h + 2) * d, dtype=BF16)
    before = fused.clone()
    view = fused[:, :h * d].unflatten(1, (h, d))
    want, tol = rotary_want(view.clone(), pos, freqs, d, 1, False, 1.0)
    close(rot.apply(view, pos, out=view), want, tol)
    assert torch.equal(fused[:, h * d:], before[:, h * d:])
    for off in (1, 2, 4):
        x = normal(g, n, h, d + 8, dtype=FP16)[..., off:off + d]
        want, tol = rotary_want(x, pos, freqs, d, 1, False, 1.0)
        close(rot.apply(x, pos), want, tol)
    x = normal(g, h, n, d).transpose(0, 1)
    want, tol = rotary_want(x, pos, freqs, d, 1, False, 1.0)
    close(rot.apply(x, pos, out=torch.empty_strided(x.shape, x.stride(), device="cuda")), want, tol)


def test_rotary_transpose_is_the_gradient():
    """sum(w * turn(x)) changes along a direction e by e . transpose(w), by differences; the map
    is linear, so a difference of any size is exact but for rounding (|terms| * 2^-20)."""
    g = gen(10)
    rot = Rotary(48, rotary_dim=32, interleaved=True, scaling="yarn", factor=8.0, original_length=100)
    x, w, e = (normal(g, 30, 4, 48) for _ in range(3))
    pos = torch.randint(0, 5000, (30,), device="cuda", generator=g)
    up, down = rot.apply(x + e, pos).double(), rot.apply(x - e, pos).double()
    num = ((up - down) / 2 * w.double())
    ana = e.double() * rot.apply(w, pos, transpose=True).double()
    assert abs(num.sum() - ana.sum()) < (num.abs().sum() + ana.abs().sum()) * 2.0 ** -20


def test_rotary_turns_like_the_forward_of_the_video_model():
    """Three axes, adjacent pairs: the library's own convention for spacetime tokens."""
    from oracle import dit_oracle as O
    x = torch.randn(2 * 3 * 4, 1, 72, device="cuda", generator=gen(12))
    coords = torch.cartesian_prod(torch.arange(2), torch.arange(3), torch.arange(4)).cuda()
    got = Rotary(72, axes=3, interleaved=True).apply(x, coords)
    freqs = 10000.0 ** (-2 * torch.arange(12, dtype=torch.float64, device="cuda") / 24)
    want, tol = rotary_want(x, coords, freqs, 72, 3, True, 1.0)
    close(got, want, tol)
    rope = getattr(O, "rope_3d", None)
    if rope is not None:
        ref = torch.as_tensor(rope(x[:, 0].double().cpu().numpy(), coords.cpu().numpy()))
        close(got[:, 0].cpu(), ref, tol[:, 0].cpu())


# ------------------------------------------------------------------ together, streams, graphs


def layer(x, w, cu, longest, pos, h, hk, d, rot, causal, stream=None):
    """One layer over packed sequences on the residual stream x (float32), in place."""
    kw = dict(stream=stream)
    t = x.to(BF16)
    proj = linear_fused(t, w["qkv"], w["qkv_b"], **kw)
    qk = proj[:, :(h + hk) * d].unflatten(1, (h + hk, d))
    rot.apply(qk, pos, out=qk, **kw)
    o = attention_packed(qk[:, :h], qk[:, h:], proj[:, (h + hk) * d:].unflatten(1, (hk, d)), cu, cu, longest, longest,
                         causal=causal, **kw)
    linear_fused(o.flatten(1), w["o"], w["o_b"], residual=x, out=x, **kw)
    u = linear_fused(x.to(BF16), w["up"], w["up_b"], act="gelu_tanh", **kw)
    return linear_fused(u, w["down"], w["down_b"], residual=x, out=x, **kw)


def layer_weights(g, width, h, hk, d):
    shapes = {"qkv": ((h + 2 * hk) * d, width), "o": (width, h * d), "up": (4 * width, width), "down": (width, 4 * width)}
    w = {n: normal(g, *s, dtype=BF16, std=s[1] ** -0.5) for n, s in shapes.items()}
    w.update({n + "_b": normal(g, s[0], std=0.1) for n, s in shapes.items()})
    return w


def layer_want(x, w, lengths, pos, h, hk, d, causal):
    """The layer in 64 bits, rounded to bf16 exactly where the layer hands a tensor on in bf16."""
    r = lambda t: t.to(BF16).double()  # noqa: E731
    lin = lambda t, n: t @ w[n].double().t() + w[n + "_b"].double()  # noqa: E731
    x = x.double()
    proj = r(lin(r(x), "qkv"))
    f = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    qk = proj[:, :(h + hk) * d].unflatten(1, (h + hk, d))
    t = (pos.double()[:, None] * f)[:, None]
    a, b = qk[..., :d // 2], qk[..., d // 2:]
    qk = r(torch.cat((a * torch.cos(t) - b * torch.sin(t), b * torch.cos(t) + a * torch.sin(t)), -1)).to(BF16)
    v = proj[:, (h + hk) * d:].unflatten(1, (hk, d)).to(BF16)
    o = attention_want(qk[:, :h], qk[:, h:], v, lengths, lengths, causal, d ** -0.5)[0]
    x = x + lin(r(o).flatten(1), "o")
    u = r(ACTS["gelu_tanh"](lin(r(x), "up")))
    return x + lin(u, "down")


@pytest.mark.parametrize("lengths,h,hk,d,causal", [([100, 1, 256, 31], 4, 2, 64, True), ([225, 64, 400], 4, 4, 72, False),
                                                   ([1, 1, 1], 8, 2, 128, True)])
def test_layer_of_all_three(lengths, h, hk, d, causal):
    """Rounding points are the same on both sides, so what is left are values next to a rounding
    border that fall the other way: a bf16 step (2^-7 relative) on a small share of the
    intermediate values, whose effect on a sum of n of them grows like sqrt(n).  Four tensors are handed
    on, each off by at most 2^-8 in the root mean square: 4 * 2^-8 of the result's."""
    g = gen(h + d)
    n, width = sum(lengths), 320
    w, x = layer_weights(g, width, h, hk, d), normal(g, n, width)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lengths])
    want = layer_want(x, w, lengths, pos, h, hk, d, causal)
    got = layer(x.clone(), w, offsets(lengths), max(lengths), pos, h, hk, d, Rotary(d), causal)
    assert (got.double() - want).norm() <= 4 * 2.0 ** -8 * want.norm()


def test_first_calls_inside_a_capture():
    """In a fresh process, so that the kernels' one-time set-up happens while the stream is captured."""
    import subprocess
    import sys
    code = """
import torch
from diffusion_transformer_denoiser_dit_b200 import Rotary, attention_packed, linear_fused
x = torch.randn(600, 4, 64, device="cuda").bfloat16()
w = torch.randn(512, 256, device="cuda").bfloat16()
cu, pos = torch.tensor([0, 600], device="cuda").int(), torch.arange(600, device="cuda")
rot = Rotary(64)
run = lambda: [linear_fused(attention_packed(rot.apply(x, pos), x, x, cu, cu, m, 600, causal=True).flatten(1)[:n], w)
               for m, n in ((600, 600), (1, 1), (1, 40))] + [linear_fused(torch.cat([x.flatten(1)] * 9), w)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
for a, b in zip(got, run()):
    assert torch.equal(a, b) and torch.isfinite(a).all()
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_captured_replayed_and_on_other_streams():
    """The layer captured once and replayed on new inputs, twice at once on two streams, and on a
    side stream, gives the direct call's bits."""
    g = gen(1)
    h, hk, d, width = 4, 2, 64, 256
    lengths = [60, 1, 200]
    n, rot = sum(lengths), Rotary(d)
    w = layer_weights(g, width, h, hk, d)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lengths])
    cu = offsets(lengths)
    inputs = [normal(g, n, width) for _ in range(4)]
    want = [layer(x.clone(), w, cu, 200, pos, h, hk, d, rot, True) for x in inputs]
    graphs = []
    for _ in range(2):
        x = inputs[0].clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(x, w, cu, 200, pos, h, hk, d, rot, True)
        graphs.append((graph, x, y))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(2):
        torch.cuda.synchronize()
        for i, (graph, x, y) in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                x.copy_(inputs[2 * turn + i])
                graph.replay()
        torch.cuda.synchronize()
        for i, (graph, x, y) in enumerate(graphs):
            assert torch.equal(y, want[2 * turn + i])
    side = torch.cuda.Stream()
    x, cache = inputs[1].clone(), inputs[2].clone()
    side.wait_stream(torch.cuda.current_stream())
    xb, wq = x.to(BF16), w["qkv"]
    torch.cuda.synchronize()
    got = linear_fused(xb, wq, w["qkv_b"], stream=side)           # passed as an argument
    side.synchronize()
    assert torch.equal(got, linear_fused(xb, wq, w["qkv_b"]))
    with torch.cuda.stream(side):                                  # or current
        y = layer(cache, w, cu, 200, pos, h, hk, d, rot, True)
    side.synchronize()
    assert torch.equal(y, want[2])


# ------------------------------------------------------------------ the two ways from Python


def both_ways(call, monkeypatch):
    """(result by the short way, by the long one, whether the short one took the call)."""
    rt = binding._rt()
    taken, fast = [], rt.fast

    class Watch:
        def __getattr__(self, name):
            def run(*args):
                y = getattr(fast, name)(*args)
                taken.append(y is not None)
                return y
            return run

    with monkeypatch.context() as m:
        m.setattr(rt, "fast", Watch())
        a = call()
        m.setattr(rt, "fast", None)
        b = call()
    assert len(taken) == 1
    return a, b, taken[0]


def need_short_way():
    if binding._rt().fast is None:
        pytest.skip("the short way was not built here")


def test_short_way_of_linear(monkeypatch):
    need_short_way()
    g = gen(5)
    x, w, b, r = normal(g, 70, 136, dtype=BF16), normal(g, 96, 136, dtype=BF16), normal(g, 96), normal(g, 70, 96, dtype=BF16)
    wide = normal(g, 70, 200, dtype=BF16)
    out = torch.empty(70, 96, device="cuda", dtype=BF16)
    calls = {
        "plain": lambda: linear_fused(x, w),
        "all": lambda: linear_fused(x, w, b, "gelu", r),
        "row": lambda: linear_fused(x, w, residual=r[:1].expand(70, 96)),
        "strided": lambda: linear_fused(wide[:, 8:144], w, b, out=torch.zeros_like(wide)[:, 40:136]),
        "one": lambda: linear_fused(x[3:4], w, b, "silu"),
        "none": lambda: linear_fused(x[:0], w, b),
        "f32": lambda: linear_fused(x, w, b, out_dtype=F32),
        "fp16": lambda: linear_fused(x.to(FP16), w.to(FP16), b, out_dtype=F32, residual=r.to(F32)),
        "parameter": lambda: linear_fused(x, torch.nn.Parameter(w), torch.nn.Parameter(b)),
    }
    for what, call in calls.items():
        a, want, short = both_ways(call, monkeypatch)
        assert short and a.dtype == want.dtype and a.stride() == want.stride() and torch.equal(a, want), what
        assert not a.requires_grad
    a, _, short = both_ways(lambda: linear_fused(x, w, b, out=out), monkeypatch)
    assert short and a is out
    stream = torch.cuda.current_stream()
    assert torch.equal(linear_fused(x, w, b, stream=stream), linear_fused(x, w, b))


def test_short_way_of_attention_and_rotary(monkeypatch):
    need_short_way()
    g = gen(6)
    qkv = normal(g, 90, 8, 64, dtype=BF16)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    cu = offsets([40, 0, 50])
    calls = {
        "plain": lambda: attention_packed(q, k, v, cu, cu, 50, 50),
        "causal": lambda: attention_packed(q, k, v, cu, cu, 50, 50, True, 0.2),
        "out": lambda: attention_packed(q, k, v, cu, cu, 50, 50, out=torch.zeros_like(qkv)[:, 2:6]),
    }
    for what, call in calls.items():
        a, want, short = both_ways(call, monkeypatch)
        assert short and a.stride() == want.stride() and torch.equal(a, want), what
    (a, la), (want, lw), short = both_ways(lambda: attention_packed(q, k, v, cu, cu, 50, 50, return_lse=True), monkeypatch)
    assert short and torch.equal(a, want) and torch.equal(la, lw) and la.dtype == F32
    pos = torch.arange(90, device="cuda")
    grid = torch.stack([pos // 9, pos % 9], 1).int()
    for rot, p in ((Rotary(64), pos), (Rotary(64, rotary_dim=32, interleaved=True, axes=2), grid)):
        for call in (lambda: rot.apply(q, p), lambda: rot.apply(q.float(), p, transpose=True),
                     lambda: rot.apply(k, p, out=torch.zeros_like(qkv)[:, :2])):
            a, want, short = both_ways(call, monkeypatch)
            assert short and a.stride() == want.stride() and torch.equal(a, want)


def test_short_way_leaves_refusals_to_the_long_one(monkeypatch):
    """What the short way does not take raises what the long way raises; a refusal of the library
    is raised by both."""
    need_short_way()
    g = gen(7)
    x, w = normal(g, 8, 64, dtype=BF16), normal(g, 32, 64, dtype=BF16)
    q, cu = normal(g, 8, 2, 64, dtype=BF16), offsets([8])
    rot, pos = Rotary(64), torch.arange(8, device="cuda")
    bad = [
        lambda: linear_fused(x, w[:, :32]),
        lambda: linear_fused(x.float(), w.float()),
        lambda: linear_fused(x, w.cpu()),
        lambda: linear_fused(x, w, act="square"),
        lambda: linear_fused(x, w, bias=torch.zeros(32, device="cuda", dtype=BF16)),
        lambda: linear_fused(x, w, residual=torch.zeros(8, 32, device="cuda")),
        lambda: linear_fused(x, w.t().contiguous().t()),
        lambda: linear_fused(x, w, out=torch.empty(8, 32, device="cuda", dtype=BF16), out_dtype=F32),
        lambda: linear_fused(x, w, out_dtype=torch.int32),
        lambda: attention_packed(q, q[:, :, :32], q, cu, cu, 8, 8),
        lambda: attention_packed(q, q, q, cu.long(), cu.long(), 8, 8),
        lambda: attention_packed(q, q, q, cu, cu, -1, 8),
        lambda: attention_packed(q, q, q, cu, cu, 2 ** 40, 8),
        lambda: attention_packed(q[:, :1], q, q, cu, cu, 8, 8),
        lambda: rot.apply(q, pos.float()),
        lambda: rot.apply(q, pos[:4]),
        lambda: rot.apply(q[:, :, :32], pos),
    ]
    rt = binding._rt()
    for i, call in enumerate(bad):
        raised = []
        for fast in (rt.fast, None):
            with monkeypatch.context() as m:
                m.setattr(rt, "fast", fast)
                with pytest.raises(Exception) as e:
                    call()
                raised.append((e.type, str(e.value)))
        assert raised[0] == raised[1], i
    torch.cuda.synchronize()
