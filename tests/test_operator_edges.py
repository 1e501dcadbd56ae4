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
