"""Modified scores (softcap, alibi_slopes, key_range) in prefill, its backward and the decode calls, on the GPU against
the fp64 oracle.

Forward tolerance, bf16: the output is rounded once (eps / 2 of it) and the probabilities are rounded to bf16 before
the second product (eps / 2 of the weighted |v|); the rest is fp32 (2e-4 of the weighted |v|, which covers a cap of
50 at 3e-7). lse is fp32: 1e-4, and the cap's tanh (3e-7 of the cap). fp32 check mode: 1e-5 of the largest value, as in
the other check-mode tests. Gradients: the bounds of the plain backward's tests."""

import math

import numpy as np
import pytest
import torch

import oracle
from _tol import assert_fp32_close, assert_grad_close

pytestmark = pytest.mark.gpu


def _randn(shape, dtype, seed, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _check(o, lse, ref, dtype, what=""):
    ro, rl, mag = ref[:3]
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    if dtype == torch.float32:
        assert_fp32_close(o, ro, what)
    else:
        tol = 2.0 ** -8 * (np.abs(ro) + mag) + 2e-4 * mag
        assert (np.abs(o - ro) <= tol).all(), (what, (np.abs(o - ro) / np.maximum(tol, 1e-30)).max())
    assert (np.isneginf(lse) == np.isneginf(rl)).all(), what
    seen = np.isfinite(rl)
    assert np.abs(lse[seen] - rl[seen]).max(initial=0) <= (1e-4 if dtype == torch.bfloat16 else 1e-5 * max(1, np.abs(rl[seen]).max(initial=0))), what


def _slopes(h):
    return 2.0 ** (-8.0 * (1 + torch.arange(h, dtype=torch.float32)) / h)


def _mask(kind, B, S, T, start, seed):
    """Keyword arguments of a mask, and the ranges for the oracle."""
    g = torch.Generator().manual_seed(seed)
    if kind == "causal":
        return dict()
    if kind == "full":
        return dict(causal=False)
    if kind == "window":
        return dict(window=max(1, T // 6))
    import kv_cache_attention_gqa_b200 as gqa

    if kind in ("documents", "prefixes"):
        cut = torch.rand(B, T, generator=g) < 6 / T
        ids = cut.int().cumsum(1)
        ids[:, T - T // 9:] = -1  # padding at the end
        rg = gqa.key_ranges(ids, prefix_len=T // 12 if kind == "prefixes" else None)
        rows = torch.stack([rg[b, start[b]:start[b] + S] for b in range(B)])
        return dict(causal=False, key_range=rows.contiguous())
    # unordered ranges, some empty, some past every limit
    lo = torch.randint(-5, T, (B, S), generator=g)
    hi = lo + torch.randint(-20, T, (B, S), generator=g)
    return dict(causal=kind == "random causal", key_range=torch.stack([lo, hi], -1).to(torch.int32))


MODS = {"cap": dict(softcap=5.0), "cap50": dict(softcap=50.0), "bias": dict(slopes=True),
        "both": dict(softcap=2.0, slopes=True), "none": dict()}
SHAPES = [(2, 4, 2, 70, 131, 64), (1, 8, 1, 300, 300, 128), (3, 32, 32, 300, 300, 64), (1, 6, 2, 1, 257, 128),
          (1, 40, 2, 150, 400, 64), (20, 16, 8, 260, 260, 128)]


@pytest.mark.parametrize("mask", ["causal", "full", "window", "documents", "prefixes", "random", "random causal"])
@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("B,h_q,h_kv,S,T,d", SHAPES)
def test_prefill_bf16(B, h_q, h_kv, S, T, d, mod, mask):
    _prefill(B, h_q, h_kv, S, T, d, mod, mask, torch.bfloat16, grad=B * h_q * S * T <= 3000000)


@pytest.mark.parametrize("mask", ["causal", "full", "window", "documents", "prefixes", "random", "random causal"])
@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("B,h_q,h_kv,S,T,d", [(2, 4, 2, 40, 60, 96), (1, 3, 1, 67, 67, 20)])
def test_prefill_fp32(B, h_q, h_kv, S, T, d, mod, mask):
    _prefill(B, h_q, h_kv, S, T, d, mod, mask, torch.float32, grad=True)


def _prefill(B, h_q, h_kv, S, T, d, mod, mask, dtype, grad):
    import kv_cache_attention_gqa_b200 as gqa

    if mod == "none" and mask in ("causal", "full", "window"):
        pytest.skip("the plain call")
    std = 3.0 if mod.startswith("cap") else 1.0
    q, k, v = _randn((B, h_q, S, d), dtype, 1, std), _randn((B, h_kv, T, d), dtype, 2), _randn((B, h_kv, T, d), dtype, 3)
    up = _randn((B, h_q, S, d), dtype, 4)
    lens = [T - (3 * b) % 7 if S < T else T for b in range(B)]
    start = [n - S for n in lens]
    how = _mask(mask, B, S, T, start, 5)
    m = dict(MODS[mod])
    slopes = _slopes(h_q) if m.pop("slopes", False) else None
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")
    if mask in ("documents", "prefixes"):  # no row sees the padding at the end
        k[:, :, T - T // 9:], v[:, :, T - T // 9:] = float("nan"), float("nan")
        kr, vr = torch.nan_to_num(k), torch.nan_to_num(v)
    else:
        kr, vr = k, v
    rg = how.get("key_range")
    args = dict(q_start=start, kv_len=lens, causal=how.get("causal", True), window=how.get("window", 0), **m)
    ref = oracle.modified_attention_ref(q.double(), kr.double(), vr.double(), slopes=None if slopes is None else slopes.numpy(),
                                        key_range=None if rg is None else rg.numpy(), d_o=up.double() if grad else None, **args)
    args.update(alibi_slopes=None if slopes is None else slopes.cuda(), key_range=None if rg is None else rg.cuda())
    q, k, v, up = q.cuda(), k.cuda(), v.cuda(), up.cuda()
    o, lse = gqa.prefill(q, k, v, return_lse=True, **args)
    _check(o, lse, ref, dtype, "prefill")
    assert torch.equal(o, gqa.prefill(q, k, v, **args))
    if grad:
        for name, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, k, v, o, up, lse, **args), ref[3:]):
            assert_grad_close(got.double().cpu().numpy(), want, name, fp32=dtype == torch.float32)
            if name != "dq":
                for b, n in enumerate(lens):
                    assert (got[b, :, n:] == 0).all()
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("mask", ["causal", "window", "ranges"])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (3, 3, 64), (40, 1, 64), (20, 1, 128)])
def test_decode(h_q, h_kv, d, mod, mask, page, dtype):
    import kv_cache_attention_gqa_b200 as gqa

    if mod == "none" and mask != "ranges":
        pytest.skip("the plain call")
    B, T = 5, 704
    lens, at = [704, 333, 1, 700, 50], [703, 331, 0, 200, 400]
    std = 3.0 if mod.startswith("cap") else 1.0
    q, k, v = _randn((B, h_q, d), dtype, 1, std), _randn((B, h_kv, T, d), dtype, 2), _randn((B, h_kv, T, d), dtype, 3)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")
    m = dict(MODS[mod])
    slopes = _slopes(h_q) if m.pop("slopes", False) else None
    window = 100 if mask == "window" else 0
    rg = torch.tensor([[0, 704], [17, 200], [0, 1], [100, 90], [-3, 10**9]], dtype=torch.int32) if mask == "ranges" else None
    ref = oracle.modified_attention_ref(q.double()[:, :, None], k.double(), v.double(), q_start=at, kv_len=lens, window=window,
                                        slopes=None if slopes is None else slopes.numpy(),
                                        key_range=None if rg is None else rg.numpy()[:, None], **m)
    how = dict(kv_len=lens, q_pos=at, window=window, alibi_slopes=None if slopes is None else slopes.cuda(),
               key_range=None if rg is None else rg.cuda(), return_lse=True, **m)
    if mask == "window":  # sequence 4's window [301, 400] starts past its 50 keys: flagged, zeros
        ref[1][4], ref[0][4], ref[2][4] = -np.inf, 0, 0
    for splits in (0, 3):
        if page:
            n = T // page
            order = torch.randperm(B * n, generator=torch.Generator().manual_seed(7))
            pools = []
            for x in (k, v):
                pool = torch.empty(B * n, h_kv, page, d, dtype=dtype)
                pool[order] = x.view(B, h_kv, n, page, d).transpose(1, 2).reshape(B * n, h_kv, page, d)
                pools.append(pool.cuda())
            o, lse = gqa.decode_paged(q.cuda(), *pools, order.view(B, n).to(torch.int32), num_splits=splits, **how)
        else:
            o, lse = gqa.decode(q.cuda(), k.cuda(), v.cuda(), num_splits=splits, **how)
        _check(o[:, :, None], lse[:, :, None], ref, dtype, f"decode splits {splits}")
        assert gqa.get_device_error() == (3 if mask == "window" else 0)


def test_scores_far_past_the_cap():
    """Scores of hundreds against a cap of 1: tanh saturates, the row is a softmax over +-1."""
    import kv_cache_attention_gqa_b200 as gqa

    for dtype, d in ((torch.bfloat16, 64), (torch.float32, 40)):
        q, k, v = _randn((1, 2, 130, d), dtype, 1, 40.0), _randn((1, 1, 200, d), dtype, 2, 40.0), _randn((1, 1, 200, d), dtype, 3)
        ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), q_start=[70], softcap=1.0)
        o, lse = gqa.prefill(q.cuda(), k.cuda(), v.cuda(), q_start=[70], softcap=1.0, return_lse=True)
        _check(o, lse, ref, dtype)


def test_padded_batch_in_a_captured_step():
    """A training step over packed documents, captured: the forward, its gradients, twice replayed with other documents."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S, d = 2, 8, 2, 384, 64
    q, k, v = _randn((B, h_q, S, d), torch.bfloat16, 1).cuda(), _randn((B, h_kv, S, d), torch.bfloat16, 2).cuda(), _randn((B, h_kv, S, d), torch.bfloat16, 3).cuda()
    up, slopes = _randn((B, h_q, S, d), torch.bfloat16, 4).cuda(), _slopes(h_q).cuda()

    def ranges(cuts):
        ids = torch.full((B, S), -1)
        for b, c in enumerate(cuts):
            for i, (lo, hi) in enumerate(zip(c, c[1:])):
                ids[b, lo:hi] = i
        return gqa.key_ranges(ids).cuda()

    a, b = ranges([[0, 100, 384], [0, 5, 200]]), ranges([[0, 384], [0, 129, 130, 300]])
    rg = a.clone()

    def step():
        how = dict(causal=False, key_range=rg, alibi_slopes=slopes, softcap=20.0)
        o, lse = gqa.prefill(q, k, v, return_lse=True, **how)
        return (o, lse, *gqa.prefill_backward(q, k, v, o, up, lse, **how))

    want = {}
    for name, r in (("a", a), ("b", b)):
        rg.copy_(r)
        want[name] = [t.clone() for t in step()]
    assert not torch.equal(want["a"][0], want["b"][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for name, r in (("a", a), ("b", b), ("a", a)):
        rg.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[name])), name
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0)])
def test_ranges_at_the_limits_of_an_int(causal, window, dtype):
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S, d = 1, 4, 2, 200, 64
    least, most = -2 ** 31, 2 ** 31 - 1
    rows = torch.tensor([[least, most], [0, least], [most, most], [most, least], [5, most], [least, 9], [least, least],
                         [3, 150]], dtype=torch.int64)
    rg = rows[torch.arange(S) % len(rows)].to(torch.int32)[None].contiguous()
    q, k, v = _randn((B, h_q, S, d), dtype, 1), _randn((B, h_kv, S, d), dtype, 2), _randn((B, h_kv, S, d), dtype, 3)
    up = _randn((B, h_q, S, d), dtype, 4)
    ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), key_range=rg.numpy(), d_o=up.double(),
                                        causal=causal, window=window)
    q, k, v, up, rg = q.cuda(), k.cuda(), v.cuda(), up.cuda(), rg.cuda()
    how = dict(causal=causal, window=window, key_range=rg)
    o, lse = gqa.prefill(q, k, v, return_lse=True, **how)
    _check(o, lse, ref, dtype, "prefill")
    for name, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, k, v, o, up, lse, **how), ref[3:]):
        assert_grad_close(got.double().cpu().numpy(), want, name, fp32=dtype == torch.float32)
    for i in range(len(rows)):  # the same range for every head of a step at the end of the cache
        q1 = q[:, :, -1].contiguous()
        ro, rl, mag = oracle.modified_attention_ref(q1[:, :, None].double().cpu(), k.double().cpu(), v.double().cpu(),
                                                    key_range=rg[:, i:i + 1].cpu().numpy(), q_start=[S - 1])[:3]
        o, lse = gqa.decode(q1, k, v, kv_len=[S], return_lse=True, key_range=rg[:, i].contiguous())
        _check(o[:, :, None], lse[..., None], (ro, rl, mag), dtype, f"decode {i}")
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("how", [dict(alibi=True), dict(softcap=8.0), dict(docs=True)])
def test_gradients_keep_to_two_roundings(how, d):
    """Peaked scores (standard deviation 3) make dS = P (dP - D) a small difference. dS is rounded to bf16 once and so
    are dQ and dK: each rounding is off by at most 2^-8 of the value, uniformly, so by 2^-8 / sqrt(3) in the mean square;
    two of them by sqrt(2) times that of the gradient's norm."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S = 1, 8, 2, 700
    mods, cpu = {}, {}
    if how.get("alibi"):
        slopes = 2.0 ** (-8.0 * (1 + torch.arange(h_q)) / h_q)
        mods["alibi_slopes"], cpu["slopes"] = slopes.cuda(), slopes.numpy()
    if how.get("softcap"):
        mods["softcap"] = cpu["softcap"] = how["softcap"]
    if how.get("docs"):
        rg = torch.tensor([[lo, hi] for lo, hi in ((0, 300), (300, 333), (333, S)) for _ in range(hi - lo)],
                          dtype=torch.int32)[None].contiguous()
        mods["key_range"], cpu["key_range"] = rg.cuda(), rg.numpy()
    q = (3.0 * _randn((B, h_q, S, d), torch.float32, 1)).to(torch.bfloat16)
    k, v = _randn((B, h_kv, S, d), torch.bfloat16, 2), _randn((B, h_kv, S, d), torch.bfloat16, 3)
    up = _randn((B, h_q, S, d), torch.bfloat16, 4)
    ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), d_o=up.double(), causal=True, **cpu)
    q, k, v, up = q.cuda(), k.cuda(), v.cuda(), up.cuda()
    o, lse = gqa.prefill(q, k, v, return_lse=True, **mods)
    grads = gqa.prefill_backward(q, k, v, o, up, lse, **mods)
    for name, got, want in zip(("dq", "dk"), grads, ref[3:5]):
        off = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert off <= 2.0 ** -8 * math.sqrt(2 / 3), (name, off)
    assert gqa.get_device_error() == 0


def test_expired_wait_with_drawn_items():
    """More work than CTAs, so that items are drawn from the counter: the CTA that gives up hands none on to itself, the
    others draw the rest, and its rows are zeros."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S, d = 1, 32, 8, 2600, 64
    q, k, v = (_randn((B, h, S, d), torch.bfloat16, i).cuda() for i, h in ((1, h_q), (2, h_kv), (3, h_kv)))
    rg = torch.tensor([[p // 500 * 500, S] for p in range(S)], dtype=torch.int32)[None].contiguous().cuda()
    want, want_lse = gqa.prefill(q, k, v, return_lse=True, key_range=rg)
    assert gqa.get_device_error() == 0
    gqa.debug_expire_waits(True)
    try:
        o, lse = gqa.prefill(q, k, v, out=torch.full_like(q, float("nan")), return_lse=True, key_range=rg)
        code = gqa.get_device_error()
    finally:
        gqa.debug_expire_waits(False)
    assert code == 4  # GQA_DEVERR_TIMEOUT
    gone = torch.isneginf(lse)
    assert 0 < int(gone.sum()) <= 256
    assert not o[gone].any() and torch.equal(o[~gone], want[~gone]) and torch.equal(lse[~gone], want_lse[~gone])
    for _ in range(3):
        o, lse = gqa.prefill(q, k, v, return_lse=True, key_range=rg)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert gqa.get_device_error() == 0


def test_two_captured_decodes_at_once():
    """Two graphs captured on one stream, replayed together on two: neither uses the other's partial results, also after
    the stream's own workspace has grown."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, T, d = 4, 8, 2, 4000, 128
    slopes = torch.linspace(0.01, 0.2, h_q, device="cuda")
    calls = []
    side = torch.cuda.Stream()
    for seed in (1, 10):
        q = _randn((B, h_q, d), torch.bfloat16, seed).cuda()
        k, v = (_randn((B, h_kv, T, d), torch.bfloat16, seed + i).cuda() for i in (1, 2))
        how = dict(softcap=20.0, alibi_slopes=slopes, return_lse=True)
        want = gqa.decode(q, k, v, **how)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = gqa.decode(q, k, v, **how)
        calls.append((graph, got, want, (q, k, v)))
    with torch.cuda.stream(side):
        gqa.workspace(1 << 26, "cuda").fill_(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, (graph, *_) in zip(streams, calls):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in calls:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("d", [24, 96, 200])
def test_check_mode_with_many_tiles(d):
    """More 32-row tiles than SMs: the check mode's large tiles (smaller calls take tiles of 8)."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S = 2, 12, 4, 213
    slopes = torch.linspace(0.0, 0.3, h_q)
    rg = torch.tensor([[lo, hi] for lo, hi in ((0, 90), (90, 90), (60, 140), (140, S)) for _ in range(54)],
                      dtype=torch.int32)[None, :S].repeat(B, 1, 1).contiguous()
    q, k, v, up = (_randn((B, h, S, d), torch.float32, i) for i, h in ((1, h_q), (2, h_kv), (3, h_kv), (4, h_q)))
    kv = [S, 170]
    ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), kv_len=kv, causal=False, softcap=9.0,
                                        slopes=slopes.numpy(), key_range=rg.numpy(), d_o=up.double())
    k[1, :, 170:], v[1, :, 170:] = float("nan"), float("nan")
    q, k, v, up = q.cuda(), k.cuda(), v.cuda(), up.cuda()
    how = dict(kv_len=torch.tensor(kv, dtype=torch.int32).cuda(), causal=False, softcap=9.0, alibi_slopes=slopes.cuda(),
               key_range=rg.cuda())
    o, lse = gqa.prefill(q, k, v, return_lse=True, **how)
    _check(o, lse, ref, torch.float32, "prefill")
    for name, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, k, v, o, up, lse, **how), ref[3:]):
        assert_grad_close(got.double().cpu().numpy(), want, name, fp32=True)
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,T_max,page", [(1, 1, 0), (5, 5, 0), (37, 4096, 0), (20, 64, 16)])
def test_decode_of_many_short_sequences(T, T_max, page, dtype):
    """More units than a chunk of 128 keys holds: chunks of at least 16 keys spread them, some cut into pieces."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, d = 9, 64, 4, 64
    lens = [max(1, T - b % 4) for b in range(B)]
    slopes = torch.linspace(0.0, 0.5, h_q)
    q = _randn((B, h_q, d), dtype, 1, 3.0)
    k, v = _randn((B, h_kv, T_max, d), dtype, 2), _randn((B, h_kv, T_max, d), dtype, 3)
    ref = oracle.modified_attention_ref(q[:, :, None].double(), k.double(), v.double(), kv_len=lens,
                                        q_start=[n - 1 for n in lens], softcap=20.0, slopes=slopes.numpy())
    how = dict(kv_len=torch.tensor(lens, dtype=torch.int32).cuda(), softcap=20.0, alibi_slopes=slopes.cuda(),
               return_lse=True)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    if page:
        n = T_max // page
        pool = [x.view(B, h_kv, n, page, d).transpose(1, 2).reshape(B * n, h_kv, page, d).contiguous() for x in (k, v)]
        table = torch.arange(B * n, dtype=torch.int32).view(B, n).cuda()
        call = lambda **x: gqa.decode_paged(q, *pool, table, **how, **x)  # noqa: E731
    else:
        call = lambda **x: gqa.decode(q, k, v, **how, **x)  # noqa: E731
    need = gqa.decode_workspace_size(B, h_q, h_kv, T_max, d, dtype, 0, True)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for how_ws in (dict(), dict(ws=ws), dict(num_splits=3)):
        o, lse = call(**how_ws)
        _check(o[:, :, None], lse[..., None], ref, dtype, str(how_ws))
    assert gqa.get_device_error() == 0
