"""The oracles of the operators around the cache, pinned without a GPU: closed forms, differences, brute force."""

import numpy as np
import pytest
import torch

import oracle


def test_rope_oracle_turns_pairs():
    x = np.zeros((1, 1, 2, 6))
    x[..., 1], x[..., 3] = 1.0, 2.0
    half = oracle.rope_ref(x, [np.pi / 2], [[0, 1]], offset=1)          # pair (1, 2)
    assert np.allclose(half[0, 0, 0], x[0, 0, 0]) and np.allclose(half[0, 0, 1], [0, 0, 1, 2, 0, 0])
    wide = oracle.rope_ref(x, [np.pi / 2, 0.0], [[1, 3]], offset=1, scale=2.0)  # pairs (1, 3), (2, 4)
    assert np.allclose(wide[0, 0, 0], [0, -4, 0, 2, 0, 0]) and np.allclose(wide[0, 0, 1], [0, 4, 0, -2, 0, 0])
    near = oracle.rope_ref(x, [np.pi / 2, np.pi], [[1, 1]], offset=0, interleaved=True)  # pairs (0, 1), (2, 3)
    assert np.allclose(near[0, 0, 0], [-1, 0, 0, -2, 0, 0])


def test_weights_oracle_is_the_column_sum_of_the_softmax():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(2, 4, 3, 8)), rng.normal(size=(2, 2, 7, 8)), rng.normal(size=(2, 2, 7, 8))
    lens = [7, 5]
    _, lse = oracle.attention_ref(q, k, v, q_start=np.array([4, 2]), kv_len=np.array(lens))
    w = oracle.kv_weights_ref(q, k, lse, kv_len=lens)
    assert np.allclose(w.sum(-1), 2 * 3) and (w[1, :, 5:] == 0).all() and (w[0, :, 6] > 0).all()
    # the weighted sum of the values over a group equals the sum of its outputs
    o, _ = oracle.attention_ref(q, k, v, q_start=np.array([4, 2]), kv_len=np.array(lens))
    assert np.allclose(np.einsum("bgj,bgjd->bgd", w, v), o.reshape(2, 2, 2, 3, 8).sum((2, 3)))


def test_evict_oracle_by_hand():
    w = np.array([[[5, 1, 9, 9, 0, 9, 2, 7]]], float)
    kept, n = oracle.kv_evict_ref(w, [8], 4)
    assert kept.tolist() == [[[2, 3, 5, 7]]] and n.tolist() == [4]
    kept, _ = oracle.kv_evict_ref(w, [8], 4, sink=1, recent=1)
    assert kept.tolist() == [[[0, 2, 3, 7]]]
    kept, _ = oracle.kv_evict_ref(w, [3], 4)
    assert kept.tolist() == [[[0, 1, 2, -1]]]
    w[0, 0, 2] = np.nan
    assert oracle.kv_evict_ref(w, [8], 3)[0].tolist() == [[[3, 5, 7]]]


@pytest.mark.parametrize("how", [dict(softcap=2.0), dict(slopes=np.array([0.5, 0.1, 0.0, 1.0])),
                                 dict(softcap=3.0, slopes=np.array([0.5, 0.1, 0.0, 1.0]), window=3),
                                 dict(softcap=1.0, causal=False, ranged=True)])
def test_modified_attention_gradients_against_differences(how):
    rng = np.random.default_rng(1)
    how = dict(how)
    q, k, v = rng.normal(size=(1, 4, 5, 6)), rng.normal(size=(1, 2, 6, 6)), rng.normal(size=(1, 2, 6, 6))
    up = rng.normal(size=q.shape)
    if how.pop("ranged", False):
        how["key_range"] = np.array([[[0, 3], [1, 6], [2, 2], [5, 6], [-4, 60]]])
    how["q_start"] = [1]
    *_, dq, dk, dv = oracle.modified_attention_ref(q, k, v, d_o=up, **how)
    loss = lambda a, b, c: (oracle.modified_attention_ref(a, b, c, **how)[0] * up).sum()  # noqa: E731
    e = 1e-5
    for x, grad, put in ((q, dq, lambda y: (y, k, v)), (k, dk, lambda y: (q, y, v)), (v, dv, lambda y: (q, k, y))):
        for at in [tuple(rng.integers(0, n) for n in x.shape) for _ in range(12)]:
            hi, lo = x.copy(), x.copy()
            hi[at] += e
            lo[at] -= e
            assert abs((loss(*put(hi)) - loss(*put(lo))) / (2 * e) - grad[at]) < 1e-8


def test_plain_scores_are_the_plain_oracle():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(2, 4, 5, 6)), rng.normal(size=(2, 2, 9, 6)), rng.normal(size=(2, 2, 9, 6))
    a = oracle.modified_attention_ref(q, k, v, q_start=[2, 3], kv_len=[9, 8], window=4)
    b = oracle.attention_ref(q, k, v, q_start=np.array([2, 3]), kv_len=np.array([9, 8]), window=4)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_key_ranges_write_documents_and_prefixes():
    import kv_cache_attention_gqa_b200 as gqa

    ids = torch.tensor([[3, 3, 3, 1, 1, 7, -1, -1], [-1, 2, 2, 2, 2, 2, 3, 3]])
    for causal, prefix in ((True, None), (False, None), (True, 2), (True, 100)):
        got = gqa.key_ranges(ids, prefix_len=prefix, causal=causal)
        assert got.dtype == torch.int32 and got.is_contiguous()
        for b in range(2):
            for p in range(8):
                same = [j for j in range(8) if ids[b, j] == ids[b, p]]
                see = [j for j in same if not causal or j <= p or j - same[0] < (prefix or 0)] if ids[b, p] >= 0 else []
                assert list(range(*got[b, p].tolist())) == see
    per_row = torch.tensor([[1, 1, 1, 2, 2, 0, 0, 0], [0, 3, 3, 3, 3, 3, 1, 1]])
    assert gqa.key_ranges(ids, prefix_len=per_row)[1].tolist()[1] == [1, 4]


def test_rope_frequencies():
    import kv_cache_attention_gqa_b200 as gqa

    f, s = gqa.rope_frequencies(8, 100.0, device="cpu")
    assert s == 1.0 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    g, s = gqa.rope_frequencies(8, 100.0, scaling="linear", factor=4.0, device="cpu")
    assert s == 1.0 and torch.allclose(g, f / 4)
    g, _ = gqa.rope_frequencies(8, 100.0, scaling="ntk", factor=4.0, device="cpu")
    assert g[0] == f[0] and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12
    g, s = gqa.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    f, _ = gqa.rope_frequencies(64, device="cpu")
    assert g[0] == f[0] and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12 and abs(s - 1.1386294361119891) < 1e-12
    assert gqa.rope_frequencies(2, scaling="ntk", factor=2.0, device="cpu")[0].tolist() == [1.0]
    for bad in (dict(d_rot=7), dict(d_rot=8, factor=0.5), dict(d_rot=8, scaling="other"), dict(d_rot=8, base=-1.0),
                dict(d_rot=8, scaling="yarn", original_length=0), dict(d_rot=8, scaling="yarn", beta_fast=1.0)):
        with pytest.raises(ValueError):
            gqa.rope_frequencies(device="cpu", **bad)
