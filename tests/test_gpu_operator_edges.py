"""Edges of the operators around the cache, on the GPU: memory that may hold anything, flags, capped scores at the ends
of their range, captured calls, copies with odd shapes. Tolerances: those of the operators' own tests."""

import numpy as np
import pytest
import torch

import oracle
from _tol import assert_grad_close

pytestmark = pytest.mark.gpu


def _randn(shape, dtype, seed, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _forward_close(o, lse, ref, what=""):
    """bf16: two roundings of at most 2^-8 (of the output, and of the probabilities against |v|), the rest fp32."""
    ro, rl, mag = ref[:3]
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = 2.0 ** -8 * (np.abs(ro) + mag) + 2e-4 * mag
    assert (np.abs(o - ro) <= tol).all(), (what, np.abs(o - ro).max())
    assert (np.isneginf(lse) == np.isneginf(rl)).all(), what
    seen = np.isfinite(rl)
    assert np.abs(lse[seen] - rl[seen]).max(initial=0) <= 1e-4, what


# Keys that a tile of 128 rows sees, for the two tiles that one item holds (one head a KV head, more items than SMs),
# and the rows of K and V that neither sees.
GAPS = {"padding between documents": ([[0, 100]], [[130, 256]], 256), "blocks apart": ([[0, 100]], [[500, 600]], 768),
        "later tile sees earlier keys": ([[500, 600]], [[3, 40]], 768), "first tile sees none": ([[9, 9]], [[300, 400]], 512),
        "second tile sees none": ([[300, 400]], [[0, 0]], 512), "two documents a tile": ([[5, 60], [70, 90]], [[400, 410], [380, 390]], 512)}


@pytest.mark.parametrize("mods", [dict(), dict(softcap=6.0), dict(slopes=True)])
@pytest.mark.parametrize("name", list(GAPS))
def test_rows_that_no_tile_sees_may_hold_anything(name, mods):
    import kv_cache_attention_gqa_b200 as gqa

    B, h, S, d = 5, 32, 256, 64
    first, second, T = GAPS[name]
    rows = [first[i % len(first)] for i in range(128)] + [second[i % len(second)] for i in range(128)]
    rg = torch.tensor(rows, dtype=torch.int32).expand(B, S, 2).contiguous()
    q, up = _randn((B, h, S, d), torch.bfloat16, 1, 2.0), _randn((B, h, S, d), torch.bfloat16, 4)
    k, v = _randn((B, h, T, d), torch.bfloat16, 2), _randn((B, h, T, d), torch.bfloat16, 3)
    m = dict(mods)
    slopes = torch.linspace(0.0, 0.3, h) if m.pop("slopes", False) else None
    ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), causal=False, key_range=rg.numpy(),
                                        slopes=None if slopes is None else slopes.numpy(), d_o=up.double(), **m)
    free = torch.ones(T, dtype=torch.bool)
    for tile in (first, second):
        tile = [r for r in tile if r[0] < r[1]]
        if tile:
            free[min(r[0] for r in tile):max(r[1] for r in tile)] = False
    how = dict(causal=False, key_range=rg.cuda(), alibi_slopes=None if slopes is None else slopes.cuda(), **m)
    q, up = q.cuda(), up.cuda()
    for fill in (float("nan"), float("inf")):
        k[:, :, free], v[:, :, free] = fill, fill
        kd, vd = k.cuda(), v.cuda()
        o, lse = gqa.prefill(q, kd, vd, return_lse=True, **how)
        _forward_close(o, lse, ref, name)
        for what, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, kd, vd, o, up, lse, **how), ref[3:]):
            assert_grad_close(got.double().cpu().numpy(), want, what)
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("mods", [dict(), dict(softcap=6.0), dict(slopes=True)])
def test_a_second_tile_without_a_key_is_flagged(mods):
    """The boundary between rows whose window holds a cached key and rows whose does not falls between the two tiles of
    an item: flagged as in the plain call."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h, S, d, n, window = 5, 32, 256, 64, 100, 29  # row 127 sees key 99, row 128 none
    q, k, v = (_randn((B, h, S, d), torch.bfloat16, i).cuda() for i in (1, 2, 3))
    m = dict(mods)
    if m.pop("slopes", False):
        m["alibi_slopes"] = torch.linspace(0.0, 0.3, h).cuda()
    o, lse = gqa.prefill(q, k, v, kv_len=[n] * B, window=window, return_lse=True, **m)
    assert gqa.get_device_error() == 3
    assert not o[:, :, 128:].any() and torch.isneginf(lse[:, :, 128:]).all() and torch.isfinite(lse[:, :, :128]).all()
    # every row sees a key: no flag
    gqa.prefill(q, k, v, kv_len=[n] * B, window=window + 200, return_lse=True, **m)
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_capped_results_do_not_depend_on_masked_memory(d):
    """Keys past the length, and keys that no row sees, may hold anything: the bits of the results stay the same."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S, T = 2, 6, 2, 200, 333
    lens, start = torch.tensor([T - 40, T - 9], dtype=torch.int32), None
    q, up = _randn((B, h_q, S, d), torch.bfloat16, 1).cuda(), _randn((B, h_q, S, d), torch.bfloat16, 4).cuda()
    k, v = _randn((B, h_kv, T, d), torch.bfloat16, 2), _randn((B, h_kv, T, d), torch.bfloat16, 3)
    rg = torch.tensor([[20, 250]], dtype=torch.int32).expand(B, S, 2).contiguous().cuda()
    start = (lens - S).cuda()
    want = None
    for fill in (0.0, 1000.0, float("inf"), float("nan")):
        for b, n in enumerate(lens.tolist()):
            k[b, :, n:], v[b, :, n:] = fill, fill
        kd, vd = k.cuda(), v.cuda()
        # scratch of other kernels, and rows of shared memory that no query fills, differ from run to run
        torch.full((1 << 20,), fill, device="cuda")
        gqa.prefill(torch.full((1, 40, 300, d), 9.0 if fill else 0.1, dtype=torch.bfloat16, device="cuda"), *(
            torch.full((1, 40, 300, d), 9.0 if fill else 0.1, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        how = dict(q_start=start, kv_len=lens.cuda(), softcap=30.0)
        got = list(gqa.prefill(q, kd, vd, return_lse=True, **how))
        got += gqa.prefill_backward(q, kd, vd, got[0], up, got[1], **how)
        k2, v2 = k.clone(), v.clone()
        k2[:, :, :20], v2[:, :, :20], k2[:, :, 250:], v2[:, :, 250:] = fill, fill, fill, fill
        k2, v2 = k2.cuda(), v2.cuda()
        o, lse = gqa.prefill(q, k2, v2, return_lse=True, key_range=rg, **how)
        got += [o, lse, *gqa.prefill_backward(q, k2, v2, o, up, lse, key_range=rg, **how)]
        got += gqa.decode(q[:, :, -1].contiguous(), kd, vd, kv_len=lens.cuda(), softcap=30.0, return_lse=True)
        if want is None:
            want = [x.clone() for x in got]
        assert all(torch.equal(x, y) for x, y in zip(got, want)), (fill, [torch.equal(x, y) for x, y in zip(got, want)])
    assert gqa.get_device_error() == 0


def _capped_inputs(dtype, B, h_q, h_kv, S, d):
    q, k, v = (_randn((B, h, S, d), dtype, i) for i, h in ((1, h_q), (2, h_kv), (3, h_kv)))
    return q, k, v, _randn((B, h_q, S, d), dtype, 4)


@pytest.mark.parametrize("cap", [20.0, 1e4, 1e7])
def test_small_scores_beside_large_ones_keep_their_accuracy(cap):
    """One key's scores reach the cap, the others are of order one: these keep their relative accuracy (a tanh formed as
    1 - 2 / (e^2x + 1) is off by 3e-7 of the cap). The large scores are negative, so that they weigh nothing."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S, d = 1, 4, 2, 150, 64
    q, k, v, up = _capped_inputs(torch.bfloat16, B, h_q, h_kv, S, d)
    q[..., 0], k[..., 0] = 64.0, 0.0
    k[:, :, 3, 0] = -2.0 * cap / 8.0 if cap > 1e3 else -256.0  # q.k scale: -2 cap and less
    ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), softcap=cap, d_o=up.double())
    q, k, v, up = q.cuda(), k.cuda(), v.cuda(), up.cuda()
    o, lse = gqa.prefill(q, k, v, softcap=cap, return_lse=True)
    _forward_close(o[:, :, 4:], lse[:, :, 4:], [x[:, :, 4:] for x in ref[:3]])
    for what, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, k, v, o, up, lse, softcap=cap), ref[3:]):
        assert_grad_close(got.double().cpu().numpy(), want, what)
    o, lse = gqa.decode(q[:, :, -1].contiguous(), k, v, softcap=cap, return_lse=True)
    _forward_close(o[:, :, None], lse[..., None], [x[:, :, -1:] for x in ref[:3]])
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap", [1e-45, 1e-39, 1e-30, 1e30, 2.5e38, 3.4028234e38])
def test_caps_at_the_ends_of_their_range(cap, dtype):
    """Any finite cap above zero is allowed. A vast one changes nothing, a tiny one makes every score zero."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, S, d = 1, 4, 2, 150, 64
    q, k, v = (_randn((B, h, S, d), dtype, i) for i, h in ((1, h_q), (2, h_kv), (3, h_kv)))
    q[:, :, 5] = 0  # scores of exactly zero
    up = _randn((B, h_q, S, d), dtype, 4)
    ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), softcap=cap, d_o=up.double())
    q, k, v, up = q.cuda(), k.cuda(), v.cuda(), up.cuda()
    o, lse = gqa.prefill(q, k, v, softcap=cap, return_lse=True)
    _forward_close(o, lse, ref)
    for what, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, k, v, o, up, lse, softcap=cap), ref[3:]):
        if what == "dv" or cap > 1:
            assert_grad_close(got.double().cpu().numpy(), want, what)
        else:  # scores at the cap: nothing flows to q and k (a score of zero passes its gradient on)
            assert torch.isfinite(got).all()
    o, lse = gqa.decode(q[:, :, -1].contiguous(), k, v, softcap=cap, return_lse=True)
    _forward_close(o[:, :, None], lse[..., None], [x[:, :, -1:] for x in ref[:3]])
    assert gqa.get_device_error() == 0


def _evict_case(B, h_kv, T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(B, h_kv, T, generator=g)
    return w, *(torch.randn(B, h_kv, T, d, generator=g).to(dtype) for _ in range(2))


def _rows_moved(dense, out, kept):
    out = out.clone()
    for b in range(kept.shape[0]):
        for h in range(kept.shape[1]):
            at = torch.from_numpy(kept[b, h][kept[b, h] >= 0]).long()
            out[b, h, :len(at)] = dense[b, h, at]
    return out


@pytest.mark.parametrize("d,dtype", [(8, torch.bfloat16), (4, torch.float32), (2, torch.bfloat16), (1, torch.float32),
                                     (1, torch.bfloat16), (16, torch.bfloat16), (3, torch.float32)])
def test_eviction_of_narrow_rows(d, dtype):
    """Rows of one vector: a batch of the move fills its table of addresses, which the next but one overwrites."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_kv, T, budget = 2, 3, 20000, 9001
    w, k, v = _evict_case(B, h_kv, T, d, dtype, d)
    lens = [T, 15001]
    ref, new = oracle.kv_evict_ref(w.numpy(), lens, budget, sink=3, recent=70)
    ko, vo = torch.zeros(B, h_kv, budget, d, dtype=dtype), torch.zeros(B, h_kv, budget, d, dtype=dtype)
    want = [_rows_moved(k, ko, ref), _rows_moved(v, vo, ref), _rows_moved(k, k, ref), _rows_moved(v, v, ref)]
    for _ in range(5):
        kd, vd, wd, kod, vod = k.cuda(), v.cuda(), w.cuda(), ko.cuda(), vo.cuda()
        wo = torch.empty(B, h_kv, budget, device="cuda")
        how = dict(kv_len=lens, sink=3, recent=70)
        kept, n = gqa.kv_evict(kd, vd, wd, budget, k_out=kod, v_out=vod, weights_out=wo, **how)
        assert np.array_equal(kept.cpu().numpy(), ref) and n.tolist() == new.tolist()
        assert torch.equal(kod.cpu(), want[0]) and torch.equal(vod.cpu(), want[1])
        gqa.kv_evict(kd, vd, wd, budget, **how)
        assert torch.equal(kd.cpu(), want[2]) and torch.equal(vd.cpu(), want[3])
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("fresh", [[0], [1], [0, 2], [0, 1, 2, 3, 5]])
@pytest.mark.parametrize("page", [16, 7])
def test_eviction_into_new_and_own_pages(fresh, page):
    """A table that replaces some of a sequence's pages and keeps the others: the move keeps its order."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_kv, d, n = 1, 2, 64, 300
    T, budget = n * page, 60 * page - 3
    m = 60
    w, k, v = _evict_case(B, h_kv, T, d, torch.bfloat16, page)
    ref, _ = oracle.kv_evict_ref(w.numpy(), [T], budget, recent=9)
    order = torch.randperm(n + m, generator=torch.Generator().manual_seed(3))
    table = order[:n].view(B, n)
    out = table[:, :m].clone()
    out[0, fresh] = order[n:n + len(fresh)]

    def pool(dense):
        p = torch.zeros(n + m, h_kv, page, d, dtype=torch.bfloat16)
        p[table.reshape(-1)] = dense.view(B, h_kv, n, page, d).transpose(1, 2).reshape(n, h_kv, page, d)
        return p

    kp, vp = pool(k), pool(v)
    for _ in range(3):
        kd, vd = kp.cuda(), vp.cuda()
        wo = torch.empty(B, h_kv, m * page, device="cuda")
        kept, _ = gqa.kv_evict_paged(kd, vd, table.int().cuda(), w.cuda(), budget, kv_len=[T], recent=9,
                                     block_table_out=out.int().cuda(), weights_out=wo)
        assert np.array_equal(kept.cpu().numpy(), ref)
        for got, before, dense in ((kd, kp, k), (vd, vp, v)):
            want = before.clone()
            rows = before[out.reshape(-1)].view(B, m, h_kv, page, d).transpose(1, 2).reshape(B, h_kv, m * page, d)
            rows = _rows_moved(dense, rows, ref)
            want[out.reshape(-1)] = rows.view(B, h_kv, m, page, d).transpose(1, 2).reshape(m, h_kv, page, d)
            assert torch.equal(got.cpu(), want)
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("kind", ["contiguous", "paged", "fp32", "mla", "mla 128 heads", "many splits"])
def test_two_captured_plain_decodes_at_once(kind):
    """Two graphs captured on one stream, the second replayed first, then both together on two streams: neither uses the
    other's partial results or counters, also after the stream's own workspace has grown."""
    import kv_cache_attention_gqa_b200 as gqa
    from kv_cache_attention_gqa_b200 import _lib

    side = torch.cuda.Stream()
    calls = []
    cached = dict(_lib._ws_cache)
    for seed in (1, 10):
        rand = lambda shape, i, dtype=torch.bfloat16: _randn(shape, dtype, seed + i).cuda()  # noqa: E731
        if kind.startswith("mla"):
            h = 128 if "128" in kind else 16
            q, cache = rand((4, h, 576), 0), rand((4, 3000, 576), 1)
            call = lambda q=q, cache=cache: gqa.mla_decode(q, cache, scale=0.05, return_lse=True)  # noqa: E731
        elif kind == "paged":
            q, k, v = rand((4, 8, 128), 0), rand((800, 2, 16, 128), 1), rand((800, 2, 16, 128), 2)
            table = torch.arange(800, dtype=torch.int32).view(4, 200).cuda()
            call = lambda q=q, k=k, v=v, t=table: gqa.decode_paged(q, k, v, t, return_lse=True)  # noqa: E731
        else:
            dtype = torch.float32 if kind == "fp32" else torch.bfloat16
            q, k, v = rand((4, 8, 128), 0, dtype), rand((4, 2, 3000, 128), 1, dtype), rand((4, 2, 3000, 128), 2, dtype)
            splits = 600 if kind == "many splits" else 0  # more chunks than blocks: drawn from the counter
            call = lambda q=q, k=k, v=v, s=splits: gqa.decode(q, k, v, num_splits=s, return_lse=True)  # noqa: E731
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call()
        calls.append((graph, got, call))
    assert _lib._ws_cache.keys() == cached.keys()  # a capture leaves the streams' workspaces alone
    with torch.cuda.stream(side):
        gqa.workspace(1 << 27, "cuda").fill_(0)
    torch.cuda.synchronize()
    calls[1][0].replay()
    torch.cuda.synchronize()
    wants = [call() for _, _, call in calls]
    assert all(torch.equal(a, b) for a, b in zip(calls[1][1], wants[1]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (graph, _, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, got, _), want in zip(calls, wants):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gqa.get_device_error() == 0


def _odd_weights(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "equal":
        return torch.full(shape, 0.5)
    if kind == "ties":  # 0, 1/4, 1/2, 3/4
        return torch.randint(0, 4, shape, generator=g) / 4
    w = torch.randn(shape, generator=g)
    if kind == "odd":
        for i, x in enumerate((float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-42)):
            w[..., i::13] = x
    return w


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("page", [0, 16])
def test_selection_shared_by_a_cluster(kind, page):
    """Few long rows: four blocks share one row's keys. Equal weights across their borders, lengths just above the budget
    (blocks without a key), at it and below it."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_kv, T, d, budget, sink, recent = 4, 2, 20000, 8, 5000, 3, 40
    w = _odd_weights(kind, (B, h_kv, T), 3)
    k = torch.arange(B * h_kv * T * d, dtype=torch.float32).view(B, h_kv, T, d)
    lens = [T, budget + 1, 12345, budget]
    ref, new = oracle.kv_evict_ref(w.numpy(), lens, budget, sink=sink, recent=recent)
    want = _rows_moved(k, k, ref)
    how = dict(kv_len=lens, sink=sink, recent=recent)
    if page:
        n = T // page
        order = torch.randperm(B * n, generator=torch.Generator().manual_seed(1))
        pool = torch.empty(B * n, h_kv, page, d)
        pool[order] = k.view(B, h_kv, n, page, d).transpose(1, 2).reshape(B * n, h_kv, page, d)
        kd, vd, wd = pool.cuda(), (pool + 0.5).cuda(), w.cuda()
        kept, n_ = gqa.kv_evict_paged(kd, vd, order.view(B, n).int().cuda(), wd, budget, **how)
        kd, vd = (x.cpu()[order].view(B, n, h_kv, page, d).transpose(1, 2).reshape(B, h_kv, T, d) for x in (kd, vd))
    else:
        kd, vd, wd = k.cuda(), (k + 0.5).cuda(), w.cuda()
        kept, n_ = gqa.kv_evict(kd, vd, wd, budget, **how)
    assert np.array_equal(kept.cpu().numpy(), ref) and n_.tolist() == new.tolist()
    assert torch.equal(kd.cpu(), want) and torch.equal(vd.cpu(), want + 0.5)
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("kind", ["ties", "odd"])
def test_selection_of_rows_too_long_for_shared_memory(kind):
    """So many rows that each has one block, and more keys than it holds: every pass reads the weights again."""
    import kv_cache_attention_gqa_b200 as gqa

    B, T, budget, sink, recent = 80, 50001, 7000, 5, 100
    w = _odd_weights(kind, (B, 1, T), 5)
    k = torch.arange(B * T, dtype=torch.float32).view(B, 1, T, 1)
    lens = [T - 7 * (b % 9) for b in range(B)]
    some = [0, 1, 8, 37, 79]
    ref, _ = oracle.kv_evict_ref(w[some].numpy(), [lens[b] for b in some], budget, sink=sink, recent=recent)
    kd, vd, wd = k.cuda(), (k + 0.5).cuda(), w.cuda()
    kept, new = gqa.kv_evict(kd, vd, wd, budget, kv_len=lens, sink=sink, recent=recent)
    assert np.array_equal(kept.cpu().numpy()[some], ref) and new.tolist() == [budget] * B
    want = _rows_moved(k, k, kept.cpu().numpy())
    assert torch.equal(kd.cpu()[:, :, :, 0], want[:, :, :, 0]) and gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotation_between_slices_of_one_buffer(dtype):
    """Rows that lie between each other's rows share no memory: they are rotated from one slice into another."""
    import kv_cache_attention_gqa_b200 as gqa

    B, S, H, d = 3, 5, 10, 64
    f, _ = gqa.rope_frequencies(d)
    buf = _randn((B, S, H, d), dtype, 1).cuda()
    for lo, hi in (((0, 4), (4, 8)), ((5, 9), (1, 5)), ((0, 1), (9, 10)), ((2, 6), (2, 6))):
        b = buf.clone()
        x, out = (b[:, :, s[0]:s[1]].transpose(1, 2) for s in (lo, hi))
        want = gqa.rope(x.clone(), f, [7, 0, 100])
        assert gqa.rope(x, f, [7, 0, 100], out=out) is out
        assert torch.equal(out, want)
        rest = [h for h in range(H) if not hi[0] <= h < hi[1]]
        assert torch.equal(b[:, :, rest], buf[:, :, rest])
    # halves of the rows, halves of the tokens, one token's rows
    wide = _randn((B, 4, S, 2 * d), dtype, 2).cuda()
    want = gqa.rope(wide[..., :d].contiguous(), f, [1, 2, 3])
    gqa.rope(wide[..., :d], f, [1, 2, 3], out=wide[..., d:])
    assert torch.equal(wide[..., d:], want)
    dense = _randn((1, 4, 6, d), dtype, 3).cuda()
    want = gqa.rope(dense[:, :, 0::2].contiguous(), f, [4])
    gqa.rope(dense[:, :, 0::2], f, [4], out=dense[:, :, 1::2])
    assert torch.equal(dense[:, :, 1::2], want)
    with pytest.raises(gqa.GQAError):
        gqa.rope(dense[:, :, :3], f, [4], out=dense[:, :, 1:4])
    # a fused projection of one step, appended from where it lies
    qkv = _randn((B, S, 8, d), dtype, 4).cuda()
    q, k, v = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 6), (6, 8)))
    kc, vc = torch.zeros(B, 2, 16, d, dtype=dtype, device="cuda"), torch.zeros(B, 2, 16, d, dtype=dtype, device="cuda")
    got = gqa.kv_rope_append(q, k, v, kc, vc, [0, 3, 6], f)
    assert torch.equal(got, gqa.rope(q.contiguous(), f, [0, 3, 6])) and torch.equal(vc[1, :, 3:8], v[1])
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("large", [False, True])
def test_nan_in_a_key_stays_visible_under_a_cap(large):
    """A row that reads a NaN is NaN, whatever the sizes of the scores beside it; the other heads keep their bits."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h, S, d = 1, 3, 200, 64
    q, k, v = (_randn((B, h, S, d), torch.bfloat16, i, 30.0 if large else 1.0) for i in (1, 2, 3))
    how = dict(softcap=5.0 if large else 1000.0, return_lse=True)
    want = gqa.prefill(q.cuda(), k.cuda(), v.cuda(), **how)
    k[0, 2, 90, 7] = float("nan")
    o, lse = gqa.prefill(q.cuda(), k.cuda(), v.cuda(), **how)
    gone = torch.zeros(h, S, dtype=torch.bool)
    gone[2, 90:] = True
    assert torch.equal(torch.isnan(o[0]).all(-1).cpu(), gone) and torch.equal(torch.isnan(lse[0]).cpu(), gone)
    assert torch.equal(o[0, :2], want[0][0, :2]) and torch.equal(lse[0, :2], want[1][0, :2])
    o, _ = gqa.decode(q[:, :, -1].cuda().contiguous(), k.cuda(), v.cuda(), **how)
    assert torch.isnan(o[0]).all(-1).tolist() == [False, False, True]
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_tiles_of_very_different_lengths_take_their_turns(seed):
    """Pairs of tiles whose keys span none to 64 blocks each, in any order: the chains' turns never hold one another for
    good (a wait that ran out would be flagged)."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h, S, T, d = 1, 16, 2560, 8192, 64
    g = torch.Generator().manual_seed(seed)
    rows = []
    for tile in range(S // 128):
        kind = int(torch.randint(0, 4, (1,), generator=g))
        lo = int(torch.randint(0, T, (1,), generator=g))
        hi = [lo, min(T, lo + 100), T, int(torch.randint(lo, T + 1, (1,), generator=g))][kind]
        rows += [[0 if kind == 2 else lo, hi]] * 128
    rg = torch.tensor(rows, dtype=torch.int32)[None].contiguous().cuda()
    q, k, v = (_randn((B, h, n, d), torch.bfloat16, seed + i).cuda() for i, n in ((1, S), (2, T), (3, T)))
    key = torch.arange(T, device="cuda")
    seen = (key >= rg[0, :, :1]) & (key < rg[0, :, 1:])
    first = None
    for _ in range(3):
        o, lse = gqa.prefill(q, k, v, causal=False, key_range=rg, softcap=4.0, return_lse=True)
        assert gqa.get_device_error() == 0
        first = (o.clone(), lse.clone()) if first is None else first
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    for a in range(0, h, 5):
        s = 4.0 * torch.tanh(q[0, a].double() @ k[0, a].double().T / 8.0 / 4.0)
        s = s.masked_fill(~seen, -float("inf"))
        rl = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(torch.isfinite(rl), rl, 0.0)[:, None])
        x, mag = p @ v[0, a].double(), p @ v[0, a].double().abs()
        _forward_close(o[0, a], lse[0, a], [t.cpu().numpy() for t in (x, rl, mag)], a)


def test_check_mode_reads_nothing_into_keys_without_weight():
    """Key ranges in fp32: NaN in keys that a tile's rows span but none sees, and in queries that see no key."""
    import kv_cache_attention_gqa_b200 as gqa

    for S, T, d in ((90, 160, 40), (700, 300, 64)):
        B, h_q, h_kv = 1, 6, 2
        q, k, v = (_randn((B, h, n, d), torch.float32, i) for i, h, n in ((1, h_q, S), (2, h_kv, T), (3, h_kv, T)))
        up = _randn((B, h_q, S, d), torch.float32, 4)
        rg = torch.tensor([[0, 42] if i < 42 else [7, 7] if i < 50 else [100, 150] for i in range(S)], dtype=torch.int32)[None]
        ref = oracle.modified_attention_ref(q.double(), k.double(), v.double(), causal=False, key_range=rg.numpy(),
                                            softcap=8.0, d_o=up.double())
        for x in (k, v):
            x[:, :, 42:100], x[:, :, 150:] = float("nan"), float("inf")
        q[:, :, 42:50], up[:, :, 42:50] = float("nan"), float("nan")
        q, k, v, up = q.cuda(), k.cuda(), v.cuda(), up.cuda()
        how = dict(causal=False, key_range=rg.contiguous().cuda(), softcap=8.0)
        o, lse = gqa.prefill(q, k, v, return_lse=True, **how)
        assert not o[:, :, 42:50].any()
        _forward_close(o, lse, ref)
        for what, got, want in zip(("dq", "dk", "dv"), gqa.prefill_backward(q, k, v, o, up, lse, **how), ref[3:]):
            assert_grad_close(got.double().cpu().numpy(), want, what, fp32=True)
        assert gqa.get_device_error() == 0


@pytest.mark.parametrize("B,h", [(1, 3), (5, 32)])
@pytest.mark.parametrize("mods", [dict(softcap=20.0), dict(slopes=True), dict(ranges=True)])
def test_a_nan_query_gives_a_nan_row(mods, B, h):
    """All scores of the row are NaN: it is no row without a key. Few tiles (two chains share one) and many."""
    import kv_cache_attention_gqa_b200 as gqa

    S, d = 200, 64
    q, k, v = (_randn((B, h, S, d), torch.bfloat16, i) for i in (1, 2, 3))
    q[0, 1, 50, 3] = float("nan")
    how = dict(softcap=mods.get("softcap", 0.0), return_lse=True)
    if mods.get("slopes"):
        how["alibi_slopes"] = torch.linspace(0.0, 0.3, h).cuda()
    if mods.get("ranges"):
        how["key_range"] = torch.tensor([[0, S]], dtype=torch.int32).expand(B, S, 2).contiguous().cuda()
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    gone = torch.zeros(B, h, S, dtype=torch.bool, device="cuda")
    gone[0, 1, 50] = True
    o, lse = gqa.prefill(q, k, v, **how)
    assert torch.equal(torch.isnan(o).all(-1), gone) and torch.equal(torch.isnan(o).any(-1), gone)
    assert torch.equal(torch.isnan(lse), gone) and torch.isfinite(lse[~gone]).all()
    if mods.get("ranges"):
        how["key_range"] = how["key_range"][:, 0].contiguous()
    o, lse = gqa.decode(q[:, :, 50].contiguous(), k, v, **how)
    assert torch.equal(torch.isnan(o).all(-1), gone[:, :, 50]) and torch.isfinite(o[~gone[:, :, 50]]).all()
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_biased_decode_after_an_eviction_counts_rows(dtype):
    """Weights from a plain call, eviction, then a decode with a bias, a window and a key range: all count the rows that
    are left."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, T, d, budget = 2, 8, 2, 400, 64, 96
    q, k, v = (_randn((B, h, n, d), dtype, i) for i, h, n in ((1, h_q, 1), (2, h_kv, T), (3, h_kv, T)))
    lens = [T, 250]
    kd, vd, q1 = k.cuda(), v.cuda(), q[:, :, 0].cuda().contiguous()
    _, lse = gqa.decode(q1, kd, vd, kv_len=lens, return_lse=True)
    w = gqa.kv_weights(q1, kd, lse, kv_len=lens)
    assert np.abs(w.double().sum(-1).cpu().numpy() - h_q / h_kv).max() < 1e-4
    kept, new = gqa.kv_evict(kd, vd, w, budget, kv_len=lens, sink=2, recent=20)
    assert new.tolist() == [budget, budget]
    left = [torch.stack([torch.stack([x[b, g, kept[b, g].long().cpu()] for g in range(h_kv)]) for b in range(B)]) for x in (k, v)]
    slopes, rg = torch.linspace(0.0, 0.3, h_q), torch.tensor([[10, 90], [0, 96]], dtype=torch.int32)
    ref = oracle.modified_attention_ref(q.double(), *(x.double() for x in left), q_start=[budget - 1] * B, window=70,
                                        slopes=slopes.numpy(), key_range=rg[:, None].numpy())
    o, lse = gqa.decode(q1, kd, vd, kv_len=new, window=70, alibi_slopes=slopes.cuda(), key_range=rg.cuda(), return_lse=True)
    _forward_close(o[:, :, None], lse[..., None], ref)
    assert gqa.get_device_error() == 0
