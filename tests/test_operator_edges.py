"""Edges of the operators around the cache that the host decides or computes (no GPU needed)."""

import ctypes

import pytest

FAKE, NULL = 0x1000, None
OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    from kv_cache_attention_gqa_b200 import _lib

    return _lib._lib


def _mod(key_range, cap=0.0):
    from kv_cache_attention_gqa_b200 import _lib

    return ctypes.pointer(_lib._ScoreMod(cap, None, key_range))


@pytest.mark.parametrize("dtype", [0, 1])
def test_key_ranges_off_their_alignment_are_refused(lib, dtype):
    """A row's range is read as one pair of 8 bytes; a view that starts at an odd element would fault."""
    calls = {
        "prefill": lambda m: lib.gqa_prefill_mod(FAKE, FAKE, FAKE, FAKE, NULL, NULL, NULL, m, 1, 4, 2, 8, 8, 64, 0.0, 1, 0,
                                                 dtype, NULL, 0, NULL),
        "backward": lambda m: lib.gqa_prefill_backward_mod(*[FAKE] * 9, NULL, NULL, m, 1, 4, 2, 8, 8, 64, 0.0, 1, 0, dtype,
                                                           NULL, 0, NULL),
        "decode": lambda m: lib.gqa_decode_mod(FAKE, FAKE, FAKE, FAKE, NULL, NULL, NULL, m, 1, 4, 2, 8, 64, 0.0, 0, dtype,
                                               NULL, 0, 1, NULL),
        "paged": lambda m: lib.gqa_decode_paged_mod(FAKE, FAKE, FAKE, FAKE, NULL, NULL, NULL, FAKE, m, 1, 4, 2, 8, 16, 4, 64,
                                                    0.0, 0, dtype, NULL, 0, 1, NULL),
    }
    for name, call in calls.items():
        assert call(_mod(FAKE + 4)) == INVALID, name
        if name != "prefill" or dtype == 0:  # an aligned one gets to the next refusal, the workspace's
            assert call(_mod(FAKE + 8)) == WORKSPACE, name


def test_bf16_outputs_off_their_alignment_are_refused(lib):
    """They are written in vectors of 16 bytes; a view that starts inside one would fault."""
    plain = lambda o, dtype: lib.gqa_prefill(FAKE, FAKE, FAKE, o, NULL, NULL, NULL, 1, 4, 2, 8, 8, 64, 0.0, 1, 0, dtype,  # noqa: E731
                                             NULL)
    assert plain(FAKE + 2, 0) == INVALID and plain(FAKE + 8, 0) == INVALID
    mod = lambda o: lib.gqa_prefill_mod(FAKE, FAKE, FAKE, o, NULL, NULL, NULL, _mod(FAKE, 5.0), 1, 4, 2, 8, 8, 64, 0.0, 1, 0, 0,  # noqa: E731
                                        NULL, 0, NULL)
    assert mod(FAKE + 2) == INVALID and mod(FAKE) == WORKSPACE
    for call in (lambda a, dtype: lib.gqa_prefill_backward(*a, NULL, NULL, 1, 4, 2, 8, 8, 64, 0.0, 1, 0, dtype, NULL, 0, NULL),
                 lambda a, dtype: lib.gqa_prefill_backward_mod(*a, NULL, NULL, _mod(FAKE), 1, 4, 2, 8, 8, 64, 0.0, 1, 0, dtype,
                                                               NULL, 0, NULL)):
        for i in (6, 7, 8):  # dq, dk, dv
            a = [FAKE] * 9
            a[i] += 4
            assert call(a, 0) == INVALID and call(a, 1) == WORKSPACE  # fp32 is written element by element
        assert call([FAKE] * 9, 0) == WORKSPACE
    mla = lambda o: lib.gqa_mla_decode(FAKE, FAKE, o, NULL, NULL, NULL, 1, 16, 64, 576, 512, 0.1, 0, NULL, 0, 1, NULL)  # noqa: E731
    assert mla(FAKE + 2) == INVALID and mla(FAKE) == WORKSPACE


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def test_rotation_onto_overlapping_rows_is_refused(lib):
    """A block reads rows that another has rotated already, unless every row goes onto itself. (Sets that lie between
    each other's rows are allowed: the GPU tests call those.)"""
    x = 1 << 30
    call = lambda out, xs=NULL, os=NULL, dtype=0, B=2, h=4, S=3: lib.gqa_rope(  # noqa: E731
        x, out, FAKE, FAKE, 0, B, h, S, 64, 64, 0, xs, os, 0, 0, 1.0, dtype, NULL)
    row = 64 * 2
    for shift in (2, row, -row, 3 * row, -5 * row, 2 * 4 * 3 * row - 2, -(2 * 4 * 3 * row - 2)):
        assert call(x + shift) == INVALID, shift
    # a fused projection (2, 3, 10, 64): 4 query heads; out among them, shifted by one head, by one token, or across
    fused = _strides(3 * 10 * 64, 64, 10 * 64)
    for shift in (row, 3 * row, -row, 10 * row, (10 + 2) * row, (30 - 3) * row, 64, 7 * row):
        assert call(x + shift, fused, fused) == INVALID, shift
    assert call(x + row, fused, NULL) == INVALID and call(x, fused, NULL) == INVALID
    assert call(x + 4 * 64, dtype=1) == INVALID
    names = "q k v q_out kc vc inv_freq pos positions per_token B h_q h_kv S T d d_rot offset qs ks vs interleaved scale dtype stream"
    args = dict(zip(names.split(), [x, 2 * x, 3 * x, 4 * x, 5 * x, 6 * x, FAKE, FAKE, NULL, 0, 2, 4, 2, 3, 16, 64, 64, 0, NULL,
                                    NULL, NULL, 0, 1.0, 0, NULL]))
    for change in (dict(q_out=x + row), dict(q_out=2 * x), dict(q_out=3 * x - 2 * row), dict(k=4 * x + 6 * row), dict(v=4 * x)):
        assert lib.kv_rope_append(*(args | change).values()) == INVALID, change


@pytest.mark.parametrize("d_rot,base,factor,length", [(64, 10000.0, 4.0, 4096), (128, 500000.0, 8.0, 8192), (64, 10000.0, 40.0, 4096),
                                                      (32, 1e6, 2.0, 32768)])
def test_the_middle_of_the_yarn_ramps(d_rot, base, factor, length):
    """Pair by pair in 64 bits: linear in the turns over the original length, or in the index between two whole bounds."""
    import math

    import kv_cache_attention_gqa_b200 as gqa

    how = dict(scaling="yarn", factor=factor, original_length=length, device="cpu")
    turns, s = gqa.rope_frequencies(d_rot, base, **how)
    index, s2 = gqa.rope_frequencies(d_rot, base, ramp="index", **how)
    assert s == s2 == 0.1 * math.log(factor) + 1.0
    f = [base ** (-2.0 * i / d_rot) for i in range(d_rot // 2)]
    n = [length * x / (2 * math.pi) for x in f]
    first = max(max([i for i in range(-4 * d_rot, 4 * d_rot) if length * base ** (-2.0 * i / d_rot) / (2 * math.pi) >= 32.0]), 0)
    last = min(min(i for i in range(-4 * d_rot, 4 * d_rot) if length * base ** (-2.0 * i / d_rot) / (2 * math.pi) <= 1.0), d_rot - 1)
    assert 0 <= first < last and any(1.0 < x < 32.0 for x in n)
    for i in range(d_rot // 2):
        a = min(max((n[i] - 1.0) / 31.0, 0.0), 1.0)
        b = 1.0 - min(max((i - first) / (last - first), 0.0), 1.0)
        assert abs(float(turns[i]) / (f[i] * (a + (1 - a) / factor)) - 1) < 1e-12, i
        assert abs(float(index[i]) / (f[i] * (b + (1 - b) / factor)) - 1) < 1e-12, i
    assert float((turns / index - 1).abs().max()) > 0.01  # not the same angles
    for bad in (dict(ramp="both"), dict(ramp="index", beta_slow=0.0)):
        with pytest.raises(ValueError):
            gqa.rope_frequencies(d_rot, base, **how, **bad)
    with pytest.raises(ValueError):
        gqa.rope_frequencies(d_rot, 1.0, ramp="index", **how)


def _tanh_coefficients(name):
    """(first factor, addend) literals of the Horner steps of a function in common.cuh, in the order they stand."""
    import os
    import re

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_attention_gqa_b200", "csrc",
                        "common.cuh")
    with open(path) as f:
        body = f.read().split(f"float2 {name}(float2 x)")[1].split("\n}")[0]
    return [float.fromhex(a) if "x" in a else float(a) for a in re.findall(r"make_float2\((-?(?:0x[0-9a-f.]+p-?\d+|1\.))f,", body)]


def _lawson(x, n, m, steps):
    """P (degree n) / Q (degree m, Q(0) = 1) in z = x^2 for tanh(x) / x of least maximum relative error on the points x."""
    import numpy as np

    z, f = (x / x.max()) ** 2, np.tanh(x) / x
    w, q, best = np.ones_like(x) / len(x), np.ones_like(x), (np.inf, None)
    for _ in range(steps):
        a = np.concatenate([z[:, None] ** np.arange(n + 1), -f[:, None] * z[:, None] ** np.arange(1, m + 1)], 1)
        weight = np.sqrt(w) / (f * np.abs(q))
        c = np.linalg.lstsq(a * weight[:, None], f * weight, rcond=None)[0]
        q = 1.0 + z[:, None] ** np.arange(1, m + 1) @ c[n + 1:]
        off = np.abs(z[:, None] ** np.arange(n + 1) @ c[:n + 1] / q / f - 1.0)
        if off.max() < best[0]:
            best = (off.max(), c / np.concatenate([x.max() ** (2.0 * np.arange(n + 1)), x.max() ** (2.0 * np.arange(1, m + 1))]))
        w = w * (off / off.max() + 1e-6)
        w /= w.sum()
    return best


def _horner(c, z):
    import numpy as np

    r = np.full_like(z, np.float32(c[0]))
    for x in c[1:]:  # a fused multiply-add: one rounding
        r = (r.astype(np.float64) * z.astype(np.float64) + np.float64(np.float32(x))).astype(np.float32)
    return r


def test_the_polynomial_for_the_tanh_of_small_scores():
    import numpy as np

    p = _tanh_coefficients("pair_tanh_small")  # highest power first
    assert len(p) == 5
    least, fit = _lawson(0.6 * np.cos(np.linspace(0.0, np.pi / 2, 400, endpoint=False)), 4, 0, 3000)
    assert 7.2e-8 < least < 7.4e-8
    assert np.allclose(p[::-1], fit, rtol=1e-4, atol=0)  # the fit, up to where Lawson's steps have come
    x = np.linspace(0.6, 0.0, 400000, endpoint=False)
    # rounding the coefficients: half an ulp of each term, and the terms past the first add up to less than a fifth of it
    half = 2.0 ** -24
    assert np.abs(x * np.polyval(p, x * x) / np.tanh(x) - 1.0).max() < least + 1.3 * half
    x = np.concatenate([x, np.logspace(-30, -2, 100000)]).astype(np.float32)
    y = _horner(p, x * x) * x  # rounded: z (a tenth of it passes on), the last two sums (one, and a fifth), the product
    assert np.abs(y / np.tanh(x.astype(np.float64)) - 1.0).max() < least + (1.3 + 0.1 + 1.2 + 1.0) * half


def test_the_rational_function_for_the_tanh_of_any_score():
    import numpy as np

    c = _tanh_coefficients("pair_tanh_any")
    # as they stand: P and Q by turns, the highest powers first; Q is one degree longer
    p, q = [c[0], c[1], c[4], c[6]], [c[2], c[3], c[5], c[7], c[8]]
    assert len(c) == 9 and q[-1] == 1.0 and min(c) > 0
    t = np.linspace(0.0, np.pi / 2, 1500)[1:]
    least, fit = _lawson(np.unique(np.concatenate([7.8 * np.sin(t), 7.8 * (1 - np.cos(t))])), 3, 4, 1500)
    assert 1.1e-7 < least < 1.2e-7
    ref = lambda v: np.tanh(v.astype(np.float64))  # noqa: E731
    x = np.linspace(7.8, 0.0, 400000, endpoint=False)
    # rounding the coefficients: no term is negative, so P and Q are each off by half an ulp at most
    half = 2.0 ** -24
    assert np.abs(x * np.polyval(p, x * x) / np.polyval(q, x * x) / ref(x) - 1.0).max() < least + 2 * half
    assert np.allclose([*p[::-1], *q[-2::-1]], fit, rtol=3e-3, atol=0)
    x = np.concatenate([np.linspace(0.0, 20.0, 400001)[1:], np.logspace(-30, 30, 200000)]).astype(np.float32)
    v = np.minimum(x, np.float32(7.8))
    for ulp in (-1.2e-7, 0.0, 1.2e-7):  # the reciprocal's
        r = (1.0 / _horner(q, v * v).astype(np.float64) * (1.0 + ulp)).astype(np.float32)
        y = v * _horner(p, v * v) * r
        # roundings, each of half an ulp: z (three times in P, four in Q), three sums of P, four of Q, the reciprocal (and
        # its ulp, two halves), two products
        assert np.abs(y / ref(x) - 1.0).max() < least + (2 + 7 + 7 + 3 + 2) * half and y.max() <= 1.0


def test_the_binding_does_without_private_helpers_of_torch():
    """They are shortcuts for the current device, its stream and whether that captures."""
    import os
    import subprocess
    import sys

    names = ["_cuda_getCurrentRawStream", "_cuda_isCurrentStreamCapturing", "_cuda_getDevice"]
    code = f"""
import torch
for n in {names}:
    if hasattr(torch._C, n):
        delattr(torch._C, n)
from kv_cache_attention_gqa_b200 import _lib
assert _lib._capturing is torch.cuda.is_current_stream_capturing and _lib._device is torch.cuda.current_device
torch.cuda.current_stream = lambda index: type("S", (), dict(cuda_stream=40 + index))
assert _lib._raw_stream(2) == 42
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr


def test_eviction_counts_its_rows_in_32_bits(lib):
    """Threads step past the last row, so the limit lies that far below 2^31."""
    far, most = 1 << 44, 2**31 - 2**16
    call = lambda T, To, budget: lib.kv_evict(far, 2 * far, 3 * far, 4 * far, 5 * far, 6 * far, 7 * far, 8 * far, 9 * far, 1, 1,  # noqa: E731
                                              T, To, budget, 0, 0, 1, 0, NULL)
    for T, To in ((most, 64), (2**31 - 1, 64), (64, most), (64, 2**31 - 1)):
        assert call(T, To, 16) == UNSUPPORTED, (T, To)
    paged = lambda max_pages, max_out: lib.kv_evict_paged(far, 2 * far, 3 * far, 4 * far, 5 * far, 6 * far, 7 * far, 8 * far,  # noqa: E731
                                                          9 * far, 1, 1, 8, 1, max_pages, max_out, 4, 0, 0, 1, 0, NULL)
    assert paged(most, 8) == UNSUPPORTED and paged(8, most) == UNSUPPORTED
