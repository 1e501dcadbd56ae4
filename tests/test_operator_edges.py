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
