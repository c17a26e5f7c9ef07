"""Argument checks and host arithmetic of the packed-layer building blocks (no GPU): every
refusal comes back before anything is launched, with no device present."""
import ctypes
import math

import numpy as np
import pytest
import torch

from diffusion_transformer_denoiser_dit_b200 import Rotary, attention_packed, binding, linear_fused

OK, BAD, UNS = binding.DIT_OK, binding.DIT_ERR_INVALID_ARG, binding.DIT_ERR_UNSUPPORTED
F32, BF16, FP16 = binding.DIT_DTYPE_F32, binding.DIT_DTYPE_BF16, binding.DIT_DTYPE_FP16
A = 1 << 20    # an aligned address that nothing reads: each call below is refused first


def linear(**kw):
    a = dict(dtype=BF16, x=A, ldx=64, w=A, ldw=64, bias=None, act=0, residual=None, ldr=0, y=A, ldy=32, out=BF16, M=4,
             N=32, K=64, status=None, stream=None)
    a.update(kw)
    return binding.load().dit_op_linear_fused(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(dtype=F32), UNS), (dict(dtype=9), UNS), (dict(out=FP16), UNS), (dict(M=-1), BAD), (dict(N=0), BAD),
    (dict(K=0), BAD), (dict(act=-1), BAD), (dict(act=5), BAD), (dict(x=None), BAD), (dict(w=None), BAD),
    (dict(y=None), BAD), (dict(ldx=-1), BAD), (dict(ldw=-8), BAD), (dict(ldr=-8), BAD), (dict(ldy=31), BAD),
    (dict(x=A + 1), BAD), (dict(w=A + 1), BAD), (dict(y=A + 1), BAD), (dict(bias=A + 2), BAD),
    (dict(residual=A + 1), BAD), (dict(out=F32, y=A + 2), BAD), (dict(out=F32, residual=A + 2), BAD),
    (dict(M=0), OK), (dict(M=0, x=None, y=None), OK), (dict(residual=A, ldr=40), BAD),
    (dict(M=2 ** 31 - 1), UNS), (dict(N=2 ** 31 - 4096, ldy=2 ** 31), UNS), (dict(K=2 ** 31 - 1), UNS),
])
def test_linear_refusals(change, code):
    assert linear(**change) == code


def attention(**kw):
    strides = kw.pop("strides", (256, 64, 128, 64, 128, 64, 256, 64))
    a = dict(dtype=BF16, q=A, k=A, v=A, o=A, lse=None, cu_q=A, cu_k=A, n=2, tq=8, tk=8, mq=4, mk=4, h=4, hk=2, dh=64,
             strides=None if strides is None else (ctypes.c_longlong * 8)(*strides), scale=0.125, causal=1, status=None,
             stream=None)
    a.update(kw)
    return binding.load().dit_op_attention_packed(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(dtype=F32), UNS), (dict(dh=60), UNS), (dict(dh=136), UNS), (dict(h=129 * 2, hk=2), UNS), (dict(n=-1), BAD),
    (dict(tq=-1), BAD), (dict(tk=-1), BAD), (dict(mq=-1), BAD), (dict(mk=-1), BAD), (dict(h=3), BAD), (dict(h=0), BAD),
    (dict(hk=0), BAD), (dict(dh=0), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(q=None), BAD), (dict(k=None), BAD),
    (dict(v=None), BAD), (dict(o=None), BAD), (dict(cu_q=None), BAD), (dict(cu_k=None), BAD), (dict(q=A + 8), BAD),
    (dict(k=A + 2), BAD), (dict(v=A + 4), BAD), (dict(o=A + 8), BAD), (dict(lse=A + 2), BAD), (dict(cu_q=A + 1), BAD),
    (dict(strides=None), BAD), (dict(strides=(252, 64, 128, 64, 128, 64, 256, 64)), BAD),
    (dict(strides=(-256, 64, 128, 64, 128, 64, 256, 64)), BAD),
    (dict(strides=(256, 64, 0, 64, 128, 64, 256, 64)), BAD),      # keys that share a row
    (dict(strides=(256, 64, 128, 64, 128, 0, 256, 64)), BAD),     # key heads that share a row
    (dict(strides=(256, 64, 128, 64, 128, 64, 256, 56)), BAD),    # output heads overlap
    (dict(strides=(256, 64, 128, 64, 128, 64, 192, 64)), BAD),    # output tokens overlap
    (dict(n=0), OK), (dict(tq=0), OK), (dict(tq=2 ** 30 + 2 ** 20), UNS), (dict(tk=2 ** 31 - 1), UNS),
])
def test_attention_refusals(change, code):
    assert attention(**change) == code


def plan(pairs=32, axes=1):
    r = binding.RotaryPlan()
    f = (ctypes.c_double * pairs)(*[1.0] * pairs)
    assert binding.load().dit_rotary_init(ctypes.byref(r), f, pairs, axes, 1.0) == OK
    return r


def rotary(r=None, **kw):
    a = dict(dtype=BF16, x=A, xt=256, xh=64, pos=A, p64=0, y=A, yt=256, yh=64, n=8, h=4, dh=64, inter=0, tr=0,
             stream=None)
    a.update(kw)
    return binding.load().dit_op_rotary(ctypes.byref(r or plan()), *a.values())


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), UNS), (dict(n=-1), BAD), (dict(h=0), BAD), (dict(dh=62), BAD), (dict(x=None), BAD),
    (dict(y=None), BAD), (dict(pos=None), BAD), (dict(x=A + 1), BAD), (dict(dtype=F32, y=A + 2), BAD),
    (dict(pos=A + 2), BAD), (dict(p64=1, pos=A + 4), BAD), (dict(xt=-1), BAD), (dict(yh=-64), BAD),
    (dict(yh=63), BAD), (dict(yt=255), BAD), (dict(xt=512), BAD), (dict(h=1 << 19, y=2 * A, yt=1 << 26), UNS),
    (dict(n=0), OK), (dict(n=2 ** 31 - 1), UNS),
])
def test_rotary_refusals(change, code):
    assert rotary(**change) == code


def test_rotary_plan_refusals():
    lib, r = binding.load(), binding.RotaryPlan()
    f, amp = (ctypes.c_double * 300)(*[1.0] * 300), ctypes.c_float()
    assert lib.dit_rotary_init(None, f, 4, 1, 1.0) == BAD
    assert lib.dit_rotary_init(ctypes.byref(r), None, 4, 1, 1.0) == BAD
    assert lib.dit_rotary_init(ctypes.byref(r), f, 0, 1, 1.0) == BAD
    assert lib.dit_rotary_init(ctypes.byref(r), f, 4, 0, 1.0) == BAD
    assert lib.dit_rotary_init(ctypes.byref(r), f, 4, 1, float("inf")) == BAD
    assert lib.dit_rotary_init(ctypes.byref(r), f, 257, 1, 1.0) == UNS
    assert lib.dit_rotary_init(ctypes.byref(r), f, 129, 2, 1.0) == UNS
    f[3] = float("nan")
    assert lib.dit_rotary_init(ctypes.byref(r), f, 4, 1, 1.0) == BAD
    bad = binding.RotaryPlan()
    assert rotary(bad) == BAD                                        # never filled
    for kind, pairs, base, factor, length in [(-1, 4, 1e4, 1.0, 0), (4, 4, 1e4, 1.0, 0), (0, 0, 1e4, 1.0, 0),
                                              (0, 4, 0.0, 1.0, 0), (0, 4, 1e4, 0.0, 0), (2, 1, 1e4, 2.0, 0),
                                              (3, 4, 1e4, 2.0, 0), (0, 4, float("inf"), 1.0, 0)]:
        assert lib.dit_rotary_frequencies(kind, pairs, base, factor, length, f, ctypes.byref(amp)) == BAD


@pytest.mark.parametrize("pairs", [1, 12, 32, 64])
@pytest.mark.parametrize("kind,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
def test_rotary_frequencies(pairs, kind, factor):
    if kind == "ntk" and pairs < 2:
        return
    lib, f, amp = binding.load(), (ctypes.c_double * pairs)(), ctypes.c_float()
    assert lib.dit_rotary_frequencies(binding.ROTARY_SCALINGS[kind], pairs, 1e4, factor, 4096, f, ctypes.byref(amp)) == OK
    base = np.array([1e4 ** (-i / pairs) for i in range(pairs)])
    want, a = base, 1.0
    if kind == "linear":
        want = base / factor
    elif kind == "ntk":
        want = np.array([(1e4 * factor ** (pairs / (pairs - 1))) ** (-i / pairs) for i in range(pairs)])
        assert math.isclose(want[0], 1.0) and math.isclose(want[-1], base[-1] / factor, rel_tol=1e-12)
    elif kind == "yarn":
        turns = 4096 * base / (2 * np.pi)        # rotations over the trained length
        g = np.clip((turns - 1) / 31, 0, 1)
        want, a = g * base + (1 - g) * base / factor, 0.1 * math.log(factor) + 1
    assert np.allclose(np.array(f), want, rtol=1e-13, atol=0) and math.isclose(amp.value, a, rel_tol=1e-6)
    # the plan holds them as turns * 2^64
    r = binding.RotaryPlan()
    assert lib.dit_rotary_init(ctypes.byref(r), f, pairs, 1, amp) == OK
    got = np.array([t / 2.0 ** 64 for t in r.turns[:pairs]]) * 2 * np.pi
    assert np.allclose(got, want, rtol=1e-13, atol=2e-18)


def test_quartic_exponential_of_the_attention_kernel():
    """Its coefficients, read from the source, replayed in float32: 2.7e-6 at most, next to nothing on
    average, and masked scores (clamped to -126) vanish."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(binding.__file__), "csrc", "op_attention.cu")).read()
    body = src[src.index("ex2_quartic_f2"):]
    c = [np.float32(re.search(rf"c{i} = ([0-9.]+)f", body).group(1)) for i in range(5)]
    x = np.linspace(-125.5, 8.0, 400001, dtype=np.float32)
    big = np.float32(12582912.0)
    n = (x + big) - big
    f = x - n
    assert np.abs(f).max() <= 0.5
    p = np.full_like(x, c[4])
    for k in (3, 2, 1, 0):
        p = p * f + c[k]
    got = (p.view(np.int32) + (n.astype(np.int32) << 23)).view(np.float32)
    rel = got.astype(np.float64) / np.exp2(x.astype(np.float64)) - 1
    assert np.abs(rel).max() < 2.8e-6 and abs(rel.mean()) < 1e-7


def test_fixed_point_angles_are_exact_far_out():
    """(position * turns) mod 2^64, as the kernel forms it, against integer arithmetic on the exact frequency."""
    from fractions import Fraction
    r = binding.RotaryPlan()
    f = (ctypes.c_double * 1)(0.3)
    binding.load().dit_rotary_init(ctypes.byref(r), f, 1, 1, 1.0)
    two_pi = Fraction(62831853071795864769252867665590057684, 10 ** 37)
    for pos in (1, -1, 99991, 2 ** 31 - 1, -(2 ** 31)):
        turn = ((pos * r.turns[0]) % 2 ** 64) / 2.0 ** 64
        want = float((Fraction(0.3) * pos / two_pi) % 1)
        assert min(abs(turn - want), 1 - abs(turn - want)) < 1e-9 * max(1, abs(pos) / 2 ** 31) + 1e-15


def test_binding_refuses_before_the_library():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    for bad in (lambda: linear_fused(x[0], w), lambda: linear_fused(x, w[:, :32]), lambda: linear_fused(x, w.half()),
                lambda: linear_fused(x, w, act="tanh"), lambda: linear_fused(x, w, torch.zeros(31)),
                lambda: linear_fused(x, w, torch.zeros(32).half()), lambda: linear_fused(x, w.t().contiguous().t()),
                lambda: linear_fused(x, w, residual=torch.zeros(4, 32)),
                lambda: linear_fused(x, w, out=torch.zeros(4, 33).bfloat16()), lambda: linear_fused(x, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        linear_fused(x.float(), w.float())
    with pytest.raises(TypeError):
        linear_fused(x, w, out_dtype=torch.float64)
    q, k = torch.zeros(8, 4, 64).half(), torch.zeros(8, 2, 64).half()
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for bad in (lambda: attention_packed(q[0], k, k, cu, cu, 8, 8), lambda: attention_packed(q, k, k[1:], cu, cu, 8, 8),
                lambda: attention_packed(q, k.bfloat16(), k, cu, cu, 8, 8),
                lambda: attention_packed(q, k, k, cu.long(), cu, 8, 8), lambda: attention_packed(q, k, k, cu, cu[1:], 8, 8),
                lambda: attention_packed(q, k, k, cu, cu.float(), 8, 8),
                lambda: attention_packed(q, k, k, cu, cu, 8, 8, out=q.bfloat16()),
                lambda: attention_packed(q, k, k, cu, cu, 8, 8)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: Rotary(64, rotary_dim=63), lambda: Rotary(64, rotary_dim=66), lambda: Rotary(64, axes=3),
                lambda: Rotary(64, scaling="exp"), lambda: Rotary(64, freqs=[1.0]),
                lambda: Rotary(64).apply(q.transpose(1, 2), cu), lambda: Rotary(64).apply(q, torch.zeros(8)),
                lambda: Rotary(64).apply(q, torch.arange(7)), lambda: Rotary(64).apply(q, torch.arange(8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.DitError):
        Rotary(64, scaling="yarn", factor=2.0)       # needs original_length


@pytest.mark.parametrize("far", [2 ** 31, 2 ** 32 + 5, 2 ** 40])
def test_binding_refuses_sizes_beyond_the_interface(far):
    """Sizes go to the library as int; more must not arrive as their lower bits."""
    x, w = torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    many = x.expand(far, 64)
    for call in (lambda: linear_fused(many, w), lambda: linear_fused(w, many)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    q, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for limits in ((far, 4), (4, far), (-far, 4)):
        with pytest.raises(ValueError, match="32 bits"):
            attention_packed(q, q, q, cu, cu, *limits)
    with pytest.raises(ValueError, match="32 bits"):
        attention_packed(q[:1].expand(far, 2, 64), q, q, cu, cu, 4, 4)
    with pytest.raises(ValueError, match="32 bits"):
        Rotary(64).apply(q[:1].expand(far, 2, 64), torch.empty(far, dtype=torch.int32, device="meta"))
