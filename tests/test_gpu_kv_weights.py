"""Attention weights of cached keys (gqa_kv_weights, gqa_kv_weights_paged) on the GPU against the fp64 oracle.

Every weight is a sum of positive terms exp2(c s - lse2), so a relative bound on the exponent's error bounds
the weight's. In units of 2^-24: rounding c, lse2 (constant and product) and the fused multiply-add costs at
most |c s| + 2 |lse2| + |c s - lse2|; the dot product, summed in fp32 in 16-term steps of the matrix unit (fp32
mode: term by term), at most (d / 16 + 1) steps (d steps) of 2 units of the sum A of the magnitudes |c q_i k_i|; exp2 is
off by 2^-22, and the sums over rows (32 at a time, then compensated) by less than 40 units.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(B, h_q, h_kv, S, T, d, dtype, seed, lens=None, nan_tail=True):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, h_q, S, d, generator=g).to(dtype)
    k = torch.randn(B, h_kv, T, d, generator=g).to(dtype)
    if lens is not None and nan_tail:
        for b, n in enumerate(lens):
            k[b, :, n:] = float("nan")
    return q, k


def _lse(q, k, lens, start, causal, window):
    """lse (fp32) of every row, -inf where a row sees no key."""
    B, h_q, S, d = q.shape
    r = h_q // k.shape[1]
    out = torch.empty(B, h_q, S)
    for b in range(B):
        n = lens[b]
        at, key = start[b] + torch.arange(S)[:, None], torch.arange(n)[None, :]
        seen = torch.ones(S, n, dtype=torch.bool)
        if causal:
            seen = (key <= at) & ((key > at - window) if window else True)
        s = torch.einsum("hid,hjd->hij", q[b].double(), k[b, :, :n].double().repeat_interleave(r, 0)) / d ** 0.5
        out[b] = torch.logsumexp(s.masked_fill(~seen, float("-inf")), -1)
    return out


def _tol(q, k, lse, dtype):
    d = q.shape[-1]
    c = 1.4426950408889634 / d ** 0.5
    kf, qf = torch.nan_to_num(k.double()).abs(), q.double().abs()
    A = c * float(qf.max(-1).values.max() * kf.max(-1).values.max()) * d / 6  # ~ sum |q_i k_i|, generous for normal rows
    A = max(A, c * float((qf.norm(dim=-1).max() * kf.norm(dim=-1).max())))
    l2 = 1.45 * float(lse[torch.isfinite(lse)].abs().max()) if torch.isfinite(lse).any() else 0.0
    steps = d / 16 + 1 if dtype == torch.bfloat16 else d
    return 0.7 * U * (2 * A + 3 * l2 + 2 * steps * A) + 4 * U + 40 * U


def _run(q, k, lse, **how):
    import kv_cache_attention_gqa_b200 as gqa

    return gqa.kv_weights(q.cuda(), k.cuda(), lse.cuda(), **how)


CASES = [  # B, h_q, h_kv, S, T, d
    (1, 1, 1, 1, 1, 64), (2, 4, 2, 1, 129, 128), (3, 32, 1, 1, 700, 128), (2, 8, 8, 1, 300, 64), (1, 40, 1, 1, 257, 128),
    (2, 14, 2, 3, 131, 64), (2, 4, 4, 32, 160, 128), (1, 8, 2, 33, 515, 128), (2, 6, 2, 128, 384, 64),
    (1, 4, 1, 130, 130, 128), (1, 12, 4, 300, 1111, 128), (1, 160, 1, 2, 200, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", ["causal", "full", "window"])
@pytest.mark.parametrize("B,h_q,h_kv,S,T,d", CASES)
def test_weights(dtype, mode, B, h_q, h_kv, S, T, d):
    import kv_cache_attention_gqa_b200 as gqa

    lens = [max(S, T - (T - S) * b // max(1, B - 1) * 2 // 3) for b in range(B)]
    q, k = _inputs(B, h_q, h_kv, S, T, d, dtype, T + S, lens)
    causal, window = mode != "full", max(1, T // 5) if mode == "window" else 0
    start = [n - S for n in lens]
    lse = _lse(q, k, lens, start, causal, window)
    ref = oracle.kv_weights_ref(q.double(), k.double(), lse, kv_len=lens, causal=causal, window=window)
    how = dict(kv_len=lens, causal=causal, window=window)
    out = _run(q, k, lse, **how)
    tol = _tol(q, k, lse, dtype)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol * ref).all(), (np.abs(got - ref)[ref > 0] / ref[ref > 0]).max() / tol
    for b, n in enumerate(lens):
        assert (got[b, :, n:] == 0).all()
    np.testing.assert_allclose(got.sum(-1), h_q // h_kv * S, rtol=2e-5)  # every row's softmax sums to one
    assert torch.equal(out, _run(q, k, lse, **how))                      # the same bits again
    w = torch.rand(B, h_kv, T, generator=torch.Generator().manual_seed(9)).cuda()
    w0 = w.clone()
    assert _run(q, k, lse, weights=w, **how) is w
    want = w0.clone()
    for b, n in enumerate(lens):
        want[b, :, :n] += out[b, :, :n]
    assert torch.equal(w, want)
    assert gqa.get_device_error() == 0


def test_one_token_form_equals_one_row():
    q, k = _inputs(3, 8, 2, 1, 400, 128, torch.bfloat16, 5)
    lens = [400, 77, 1]
    lse = _lse(q, k, lens, [n - 1 for n in lens], True, 0)
    a = _run(q, k, lse, kv_len=lens)
    assert torch.equal(a, _run(q[:, :, 0], k, lse[:, :, 0], kv_len=lens))


def test_rows_before_the_end_and_past_it():
    """Explicit q_start: rows in the middle of the cache, and rows past its last key."""
    q, k = _inputs(2, 4, 2, 70, 500, 64, torch.bfloat16, 6)
    lens, start = [500, 300], [111, 260]
    lse = _lse(q, k, lens, start, True, 0)
    ref = oracle.kv_weights_ref(q.double(), k.double(), lse, kv_len=lens, q_start=start)
    got = _run(q, k, lse, kv_len=lens, q_start=start).double().cpu().numpy()
    assert (np.abs(got - ref) <= _tol(q, k, lse, torch.bfloat16) * ref).all()
    assert (got[0, :, 111 + 70:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S", [1, 40, 140])
def test_rows_without_lse_add_nothing(dtype, S):
    """lse = -inf and NaN rows (padding) are left out even when their queries hold NaN; +inf weighs nothing."""
    q, k = _inputs(2, 6, 2, S, 300, 64, dtype, 8)
    lens = [300, 200]
    lse = _lse(q, k, lens, [n - S for n in lens], True, 0)
    lse[0, 1, S // 2], lse[1, 5, 0], lse[1, 2, S - 1] = float("-inf"), float("nan"), float("inf")
    ref = oracle.kv_weights_ref(q.double(), k.double(), lse, kv_len=lens)
    q[0, 1, S // 2], q[1, 5, 0] = float("nan"), float("inf")
    got = _run(q, k, lse, kv_len=lens).double().cpu().numpy()
    assert (np.abs(got - ref) <= _tol(q[:, :1], k, lse, dtype) * ref).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 48, 64, 128])
@pytest.mark.parametrize("S", [1, 5, 200])
def test_paged_equals_contiguous(dtype, page, S):
    """Shuffled pages; entries past a sequence's last page are out of the pool and never read."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, d, n = 3, 8, 2, 128, 720 // page + 1
    T = n * page
    lens = [T - 3, 333, max(S, 17)]
    q, k = _inputs(B, h_q, h_kv, S, T, d, dtype, page + S, lens)
    lse = _lse(q, k, lens, [m - S for m in lens], True, 0)
    order = torch.randperm(B * n + 2, generator=torch.Generator().manual_seed(2))[:B * n]
    pool = torch.full((B * n + 2, h_kv, page, d), float("nan")).to(dtype)
    pool[order] = k.view(B, h_kv, n, page, d).transpose(1, 2).reshape(B * n, h_kv, page, d)
    table = order.view(B, n).to(torch.int32).clone()
    for b, m in enumerate(lens):
        table[b, (m + page - 1) // page:] = 10 ** 6
    a = _run(q, k, lse, kv_len=lens)
    p = gqa.kv_weights_paged(q.cuda(), pool.cuda(), table.cuda(), lse.cuda(), kv_len=lens)
    assert torch.equal(a, p)
    assert gqa.get_device_error() == 0
    table[0, 0] = -1  # a page that is needed: flagged, replaced by page 0, the other sequences unharmed
    p = gqa.kv_weights_paged(q.cuda(), torch.nan_to_num(pool).cuda(), table.cuda(), lse.cuda(), kv_len=lens)
    assert gqa.get_device_error() == 5
    assert torch.equal(a[1:], p[1:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_lengths_and_starts_are_flagged(dtype):
    import kv_cache_attention_gqa_b200 as gqa

    q, k = _inputs(3, 4, 2, 9, 200, 64, dtype, 3)
    lse = _lse(q, k, [200] * 3, [191] * 3, True, 0)
    good = _run(q, k, lse)
    for lens, code in (([0, 200, 200], 1), ([201, 200, 200], 1), ([8, 200, 200], 2)):  # 8 < S: no start
        out = _run(q, k, lse, kv_len=lens)
        assert gqa.get_device_error() == code
        assert out[0].abs().sum() == 0 and torch.equal(out[1:], good[1:])
        w = torch.ones_like(out)
        _run(q, k, lse, kv_len=lens, weights=w)
        assert gqa.get_device_error() == code and (w[0] == 1).all()


def test_captured_twice_and_replayed_on_two_streams():
    """The scratch of a call (its row parts) belongs to the capture: two graphs do not share it."""
    import kv_cache_attention_gqa_b200 as gqa

    sets = []
    for seed in (1, 2):
        q, k = _inputs(1, 4, 1, 600, 600, 128, torch.bfloat16, seed)
        lse = _lse(q, k, [600], [0], True, 0)
        sets.append([t.cuda() for t in (q, k, lse)])
    want = [gqa.kv_weights(*s) for s in sets]
    assert gqa._lib._lib.gqa_kv_weights_workspace_size(1, 4, 1, 600, 600, 0) > 0
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gqa.kv_weights(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_after_prefill_and_decode():
    """With the lse of the library's own forward calls: the columns of the softmax it applied."""
    import kv_cache_attention_gqa_b200 as gqa

    q, k = _inputs(2, 8, 2, 256, 256, 128, torch.bfloat16, 4)
    q, k = q.cuda(), k.cuda()
    _, lse = gqa.prefill(q, k, k, return_lse=True)
    w = gqa.kv_weights(q, k, lse)
    # the forward's lse is good to 2e-4 (its exponentials are approximations summed in fp32)
    torch.testing.assert_close(w.sum(-1), torch.full((2, 2), 4.0 * 256, device="cuda"), rtol=2e-4, atol=0)
    one = q[:, :, -1].contiguous()
    _, lse1 = gqa.decode(one, k, k, return_lse=True)
    w1 = gqa.kv_weights(one, k, lse1)
    torch.testing.assert_close(w1.sum(-1), torch.full((2, 2), 4.0, device="cuda"), rtol=2e-4, atol=0)
    assert gqa.get_device_error() == 0
