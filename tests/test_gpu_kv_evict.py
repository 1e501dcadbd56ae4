"""Eviction (kv_evict, kv_evict_paged) on the GPU: kept rows against the oracle's rule, moved rows bit for bit."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def _weights(B, h_kv, T, kind, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(3 * torch.randn(B, h_kv, T, generator=g)) / T
    if kind == "ties":  # a few distinct values, most of them zero
        w = torch.randint(0, 3, w.shape, generator=g).float().clamp(max=1) * 0.25
    elif kind == "equal":
        w = torch.zeros_like(w)
    elif kind == "odd":  # negative, infinite and missing weights, both zeros
        w = torch.randn(w.shape, generator=g)
        for i, x in enumerate((float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-42)):
            w[..., i::11] = x
    return w


def _cache(B, h_kv, T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, h_kv, T, d, generator=g).to(dtype)


def _expect(dense, out, kept):
    """out with row i of every head replaced by dense's row kept[i]."""
    out = out.clone()
    for b in range(kept.shape[0]):
        for g in range(kept.shape[1]):
            at = torch.from_numpy(kept[b, g][kept[b, g] >= 0]).long()
            out[b, g, :len(at)] = dense[b, g, at]
    return out


def _expect_w(w, T_out, kept):
    out = torch.zeros(w.shape[0], w.shape[1], T_out)
    return _expect(w[..., None], out[..., None], kept)[..., 0]


def _same(a, b):
    a, b = a.cpu(), b.cpu()
    view = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


CASES = [  # B, h_kv, T, d, budget, sink, recent, lens
    (1, 1, 1, 64, 1, 0, 0, [1]), (2, 3, 40, 8, 7, 0, 0, [40, 7]), (3, 2, 333, 80, 101, 1, 16, [333, 57, 102]),
    (2, 2, 700, 128, 256, 4, 252, [700, 300]), (2, 1, 500, 128, 499, 0, 100, [500, 499]), (1, 2, 130, 3, 64, 64, 0, [130]),
    (2, 2, 300, 5, 32, 2, 3, [0, 299]), (1, 1, 5000, 64, 1, 0, 0, [5000]), (2, 4, 3000, 128, 2000, 0, 1, [3000, 2001]),
]


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,h_kv,T,d,budget,sink,recent,lens", CASES)
def test_evict(kind, dtype, B, h_kv, T, d, budget, sink, recent, lens):
    import kv_cache_attention_gqa_b200 as gqa

    w = _weights(B, h_kv, T, kind, T)
    k, v = _cache(B, h_kv, T, d, dtype, 1), _cache(B, h_kv, T, d, dtype, 2)
    ref, new = oracle.kv_evict_ref(w.numpy(), lens, budget, sink=sink, recent=recent)
    how = dict(kv_len=lens, sink=sink, recent=recent)
    # into a smaller cache
    T_out = budget + 3
    ko, vo = _cache(B, h_kv, T_out, d, dtype, 3), _cache(B, h_kv, T_out, d, dtype, 4)
    kd, vd, wd, kod, vod = k.cuda(), v.cuda(), w.cuda(), ko.cuda(), vo.cuda()
    wo = torch.full((B, h_kv, T_out), 7.0, device="cuda")
    kept, new_len = gqa.kv_evict(kd, vd, wd, budget, k_out=kod, v_out=vod, weights_out=wo, **how)
    assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(new_len.cpu().numpy(), new)
    assert _same(kod, _expect(k, ko, ref)) and _same(vod, _expect(v, vo, ref))
    assert _same(wo, _expect_w(w, T_out, ref))
    assert _same(kd, k) and _same(wd, w)
    # in place
    kept, new_len = gqa.kv_evict(kd, vd, wd, budget, **how)
    assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(new_len.cpu().numpy(), new)
    assert _same(kd, _expect(k, k, ref)) and _same(vd, _expect(v, v, ref)) and _same(wd, _expect_w(w, T, ref))
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("where", ["in place", "first pages", "other pages"])
@pytest.mark.parametrize("page,d", [(16, 128), (5, 64), (64, 24)])
def test_evict_paged(dtype, where, page, d):
    import kv_cache_attention_gqa_b200 as gqa

    B, h_kv, n = 3, 2, 640 // page
    T, budget, sink, recent = n * page, 203, 2, 31
    lens = [T, 204, 150]
    w = _weights(B, h_kv, T, "ties", page)
    k, v = _cache(B, h_kv, T, d, dtype, 1), _cache(B, h_kv, T, d, dtype, 2)
    ref, new = oracle.kv_evict_ref(w.numpy(), lens, budget, sink=sink, recent=recent)
    m = (budget + page - 1) // page
    order = torch.randperm(B * (n + m), generator=torch.Generator().manual_seed(3))
    table, other = order[:B * n].view(B, n), order[B * n:].view(B, m)

    def pool(dense, seed):
        p = _cache(B * (n + m), h_kv, page, d, dtype, seed)
        p[table.reshape(-1)] = dense.view(B, h_kv, n, page, d).transpose(1, 2).reshape(B * n, h_kv, page, d)
        return p

    def rows(p, t):
        return p[t.reshape(-1)].view(B, t.shape[1], h_kv, page, d).transpose(1, 2).reshape(B, h_kv, t.shape[1] * page, d)

    kp, vp = pool(k, 5), pool(v, 6)
    to = {"in place": table, "first pages": table[:, :m], "other pages": other}[where]
    T_out = to.shape[1] * page
    used = table.to(torch.int32).clone()
    for b, x in enumerate(lens):
        used[b, (x + page - 1) // page:] = -5  # entries behind a sequence are not read
    wd, kd, vd = w.cuda(), kp.cuda(), vp.cuda()
    wo = None if where == "in place" else torch.full((B, h_kv, T_out), 7.0, device="cuda")
    out = None if where == "in place" else to.to(torch.int32).contiguous().cuda()
    kept, new_len = gqa.kv_evict_paged(kd, vd, used.cuda(), wd, budget, kv_len=lens, sink=sink, recent=recent,
                                       block_table_out=out, weights_out=wo)
    assert gqa.get_device_error() == 0
    assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(new_len.cpu().numpy(), new)
    assert _same(wd if wo is None else wo, _expect_w(w, T_out, ref))
    for got, before, dense in ((kd, kp, k), (vd, vp, v)):
        assert _same(rows(got.cpu(), to), _expect(dense, rows(before, to), ref))
        others = [p for p in range(B * (n + m)) if p not in set(to.reshape(-1).tolist())]
        assert _same(got.cpu()[others], before[others])


def test_long_rows_do_not_fit_shared_memory():
    import kv_cache_attention_gqa_b200 as gqa

    T, budget = 70001, 5000
    w = _weights(1, 2, T, "spread", 1)
    k = torch.arange(2 * T, dtype=torch.float32).view(1, 2, T, 1)
    ref, _ = oracle.kv_evict_ref(w.numpy(), [T], budget, sink=3, recent=50)
    kd, vd, wd = k.cuda(), (k + 0.5).cuda(), w.cuda()
    kept, new_len = gqa.kv_evict(kd, vd, wd, budget, sink=3, recent=50)
    assert np.array_equal(kept.cpu().numpy(), ref) and new_len.tolist() == [budget]
    assert _same(kd, _expect(k, k, ref)) and _same(vd, _expect(k + 0.5, k + 0.5, ref))


def test_bad_lengths_leave_the_sequence_alone():
    import kv_cache_attention_gqa_b200 as gqa

    w = _weights(3, 2, 100, "spread", 2).cuda()
    k, v = _cache(3, 2, 100, 16, torch.bfloat16, 1).cuda(), _cache(3, 2, 100, 16, torch.bfloat16, 2).cuda()
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    kept, new_len = gqa.kv_evict(k, v, w, 10, kv_len=[101, 60, -1])
    assert gqa.get_device_error() == 1
    assert new_len.tolist() == [101, 10, -1] and (kept[0] == -1).all() and (kept[2] == -1).all()
    for got, was in ((k, k0), (v, v0), (w, w0)):
        assert torch.equal(got[0], was[0]) and torch.equal(got[2], was[2]) and not torch.equal(got[1], was[1])
    pool = torch.zeros(4, 2, 16, 16, dtype=torch.bfloat16, device="cuda")
    gqa.kv_evict_paged(pool, pool.clone(), [[0, 7]], w[:1, :, :32].contiguous(), 3)
    assert gqa.get_device_error() == 5


def test_steady_state_in_a_graph():
    """Append, attend, weigh, evict: one captured step replayed equals the same step run eagerly."""
    import kv_cache_attention_gqa_b200 as gqa

    B, h_q, h_kv, d, T, budget = 2, 8, 2, 128, 80, 64
    f, _ = gqa.rope_frequencies(d)
    g = torch.Generator().manual_seed(1)
    qs, ks, vs = (torch.randn(40, B, h, 1, d, generator=g).to(torch.bfloat16).cuda() for h in (h_q, h_kv, h_kv))

    def state():
        return dict(k=torch.zeros(B, h_kv, T, d, dtype=torch.bfloat16, device="cuda"),
                    v=torch.zeros(B, h_kv, T, d, dtype=torch.bfloat16, device="cuda"),
                    w=torch.zeros(B, h_kv, T, device="cuda"), n=torch.tensor([60, 37], dtype=torch.int32, device="cuda"),
                    at=torch.tensor([60, 37], dtype=torch.int32, device="cuda"))

    def step(s, q, k, v):
        qr = gqa.kv_rope_append(q, k, v, s["k"], s["v"], s["n"], f, positions=s["at"])
        s["n"] += 1
        s["at"] += 1
        o, lse = gqa.decode(qr[:, :, 0], s["k"], s["v"], kv_len=s["n"], return_lse=True)
        gqa.kv_weights(qr[:, :, 0], s["k"], lse, kv_len=s["n"], weights=s["w"])
        _, new = gqa.kv_evict(s["k"], s["v"], s["w"], budget, kv_len=s["n"], sink=2, recent=16)
        s["n"].copy_(new)
        return o

    a, b = state(), state()
    eager = [step(a, qs[i], ks[i], vs[i]).clone() for i in range(40)]
    q, k, v = qs[0].clone(), ks[0].clone(), vs[0].clone()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(state(), q, k, v)  # warm-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(b, q, k, v)
    for name, x in state().items():
        b[name].copy_(x)
    for i in range(40):
        q.copy_(qs[i]), k.copy_(ks[i]), v.copy_(vs[i])
        graph.replay()
        assert torch.equal(o, eager[i]), i
    assert b["n"].tolist() == [64, 64] and all(torch.equal(a[m], b[m]) for m in a)
    assert gqa.get_device_error() == 0
