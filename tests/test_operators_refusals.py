"""Refusals of the operators around the cache, decided on the host before any CUDA call (no GPU needed)."""

import ctypes

import pytest
import torch

FAKE, NULL = 0x1000, None
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    from kv_cache_attention_gqa_b200 import _lib

    return _lib._lib


def _caller(fn, names, values):
    def call(**change):
        assert set(change) <= set(names), change
        return fn(*[change.get(n, v) for n, v in zip(names, values)])

    return call


def test_rope(lib):
    names = "x out inv_freq positions per_token B h S d d_rot offset xs os interleaved inverse scale dtype stream".split()
    call = _caller(lib.gqa_rope, names, [FAKE, FAKE, FAKE, FAKE, 0, 2, 4, 3, 64, 32, 8, NULL, NULL, 0, 0, 1.0, 0, NULL])
    for bad in (dict(x=NULL), dict(out=NULL), dict(inv_freq=NULL), dict(positions=NULL), dict(per_token=2), dict(B=0),
                dict(h=0), dict(S=-1), dict(d=0), dict(d_rot=0), dict(d_rot=7), dict(d_rot=-2), dict(offset=-1),
                dict(offset=33), dict(offset=2**31 - 1), dict(interleaved=2), dict(inverse=-1), dict(dtype=5),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == INVALID, bad
    assert call(d=5000, offset=0) == UNSUPPORTED
    assert call(B=65536, S=65536) == UNSUPPORTED
    assert call(S=0, x=NULL, out=NULL) == OK  # nothing to do


def test_rope_append(lib):
    names = ("q k v q_out kc vc inv_freq pos positions per_token B h_q h_kv S T d d_rot offset qs ks vs interleaved scale "
             "dtype stream").split()
    call = _caller(lib.kv_rope_append, names, [FAKE] * 8 + [NULL, 0, 2, 4, 2, 3, 16, 64, 64, 0, NULL, NULL, NULL, 0, 1.0,
                                                            0, NULL])
    for bad in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(q_out=NULL), dict(kc=NULL), dict(vc=NULL), dict(pos=NULL),
                dict(inv_freq=NULL), dict(h_kv=0), dict(T=0), dict(S=17), dict(d_rot=66), dict(dtype=2),
                dict(positions=FAKE, per_token=3)):
        assert call(**bad) == INVALID, bad
    assert call(S=0, k=NULL, v=NULL, pos=NULL, q=NULL, q_out=NULL) == OK
    names = ("q k v q_out kc vc inv_freq pos positions per_token bt B h_q h_kv S num_pages page max_pages d d_rot offset qs ks "
             "vs interleaved scale dtype stream").split()
    call = _caller(lib.kv_rope_append_paged, names, [FAKE] * 8 + [NULL, 0, FAKE, 2, 4, 2, 3, 8, 16, 4, 64, 64, 0, NULL,
                                                                  NULL, NULL, 0, 1.0, 0, NULL])
    for bad in (dict(bt=NULL), dict(num_pages=0), dict(page=0), dict(max_pages=0), dict(S=65), dict(kc=NULL)):
        assert call(**bad) == INVALID, bad
    assert call(page=1 << 16, max_pages=1 << 16) == UNSUPPORTED


def test_weights(lib):
    names = "q k lse w qs kl B h_q h_kv S T d scale causal window acc dtype ws bytes stream".split()
    call = _caller(lib.gqa_kv_weights, names, [FAKE, FAKE, FAKE, FAKE, NULL, NULL, 2, 4, 2, 3, 64, 128, 0.0, 1, 0, 0, 0,
                                               NULL, 0, NULL])
    for bad in (dict(q=NULL), dict(k=NULL), dict(lse=NULL), dict(w=NULL), dict(B=0), dict(h_q=5), dict(h_kv=0), dict(S=0),
                dict(T=0), dict(d=0), dict(scale=-1.0), dict(scale=float("nan")), dict(causal=2), dict(window=-1),
                dict(window=4, causal=0), dict(acc=2), dict(dtype=3)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(d=300, dtype=1), dict(B=1024, h_q=64, h_kv=64, T=65536), dict(B=40000)):
        assert call(**bad) == UNSUPPORTED, bad
    names = ("q k lse w qs kl bt B h_q h_kv S num_pages page max_pages d scale causal window acc dtype ws bytes "
             "stream").split()
    call = _caller(lib.gqa_kv_weights_paged, names, [FAKE, FAKE, FAKE, FAKE, NULL, NULL, FAKE, 2, 4, 2, 3, 8, 16, 4, 128, 0.0,
                                                     1, 0, 0, 0, NULL, 0, NULL])
    for bad in (dict(bt=NULL), dict(num_pages=0), dict(page=0), dict(max_pages=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(page=24), dict(page=1 << 16, max_pages=1 << 16), dict(num_pages=1 << 27)):
        assert call(**bad) == UNSUPPORTED, bad
    assert lib.gqa_kv_weights_workspace_size(0, 4, 2, 3, 64, 0) == 0
    assert lib.gqa_kv_weights_workspace_size(2, 4, 3, 3, 64, 0) == 0


def test_evict(lib):
    m = 1 << 20  # buffers far enough apart
    names = "k v ko vo w wo kept new kl B h_kv T To budget sink recent d dtype stream".split()
    call = _caller(lib.kv_evict, names, [1 * m, 2 * m, 3 * m, 4 * m, 5 * m, 6 * m, 7 * m, 8 * m, 9 * m, 2, 2, 64, 32, 16, 2, 4, 64,
                                         0, NULL])
    for bad in (dict(k=NULL), dict(v=NULL), dict(ko=NULL), dict(vo=NULL), dict(w=NULL), dict(wo=NULL), dict(kept=NULL),
                dict(new=NULL), dict(B=0), dict(h_kv=0), dict(T=0), dict(To=0), dict(budget=0), dict(budget=33), dict(sink=-1),
                dict(recent=-1), dict(sink=10, recent=7), dict(sink=2**31 - 1, recent=2**31 - 1), dict(d=0), dict(dtype=9)):
        assert call(**bad) == INVALID, bad
    # overlaps: half in place, in place with another row count, shifted, crossed, weights, lengths
    for bad in (dict(ko=1 * m), dict(ko=1 * m, vo=2 * m), dict(ko=1 * m + 256), dict(ko=2 * m), dict(vo=1 * m),
                dict(vo=3 * m + 512), dict(wo=5 * m), dict(wo=5 * m + 16), dict(new=9 * m), dict(new=9 * m + 4)):
        assert call(**bad) == INVALID, bad
    far = 1 << 44
    assert call(k=far, v=2 * far, ko=3 * far, vo=4 * far, w=5 * far, wo=6 * far, B=70000, h_kv=1) == UNSUPPORTED
    names = "k v bt bto w wo kept new kl B h_kv num_pages page max_pages max_out budget sink recent d dtype stream".split()
    call = _caller(lib.kv_evict_paged, names, [1 * m, 2 * m, 3 * m, NULL, 5 * m, 5 * m, 7 * m, 8 * m, 9 * m, 2, 2, 8, 16, 4, 0, 16, 2, 4,
                                               64, 0, NULL])
    for bad in (dict(bt=NULL), dict(num_pages=0), dict(page=0), dict(max_pages=0), dict(bto=4 * m), dict(bto=4 * m, max_out=-1),
                dict(v=1 * m), dict(budget=65), dict(bto=4 * m, max_out=2, wo=5 * m)):
        assert call(**bad) == INVALID, bad
    assert call(page=1 << 16, max_pages=1 << 16) == UNSUPPORTED


def test_modified_scores(lib):
    from kv_cache_attention_gqa_b200 import _lib

    mod = lambda **k: ctypes.pointer(_lib._ScoreMod(k.get("cap", 0.0), k.get("slopes"), k.get("range")))  # noqa: E731
    names = "q k v o lse qs kl mod B h_q h_kv S T d scale causal window dtype ws bytes stream".split()
    fwd = _caller(lib.gqa_prefill_mod, names, [FAKE, FAKE, FAKE, FAKE, NULL, NULL, NULL, mod(cap=5.0), 1, 4, 2, 8, 8, 64, 0.0, 1, 0, 0,
                                               NULL, 0, NULL])
    names = "q k v o do lse dq dk dv qs kl mod B h_q h_kv S T d scale causal window dtype ws bytes stream".split()
    bwd = _caller(lib.gqa_prefill_backward_mod, names, [FAKE] * 9 + [NULL, NULL, mod(cap=5.0), 1, 4, 2, 8, 8, 64, 0.0, 1, 0, 0, FAKE,
                                                                     1 << 20, NULL])
    names = "q k v o lse kl qp mod B h_q h_kv T d scale window dtype ws bytes splits stream".split()
    dec = _caller(lib.gqa_decode_mod, names, [FAKE, FAKE, FAKE, FAKE, NULL, NULL, NULL, mod(cap=5.0), 1, 4, 2, 8, 64, 0.0, 0, 0, FAKE,
                                              1 << 20, 1, NULL])
    for call in (fwd, bwd, dec):
        for cap in (-1.0, float("nan"), float("inf")):
            assert call(mod=mod(cap=cap)) == INVALID
        assert call(q=NULL) == INVALID and call(h_kv=3) == INVALID and call(dtype=4) == INVALID
        assert call(d=96) == UNSUPPORTED
    assert fwd(causal=0, window=3) == INVALID and bwd(causal=0, window=3) == INVALID
    # key ranges need the workspace (bf16 prefill; the backward a larger one)
    need = lib.gqa_prefill_mod_workspace_size(1, 4, 2, 8)
    assert need > 0 and lib.gqa_prefill_mod_workspace_size(1, 4, 3, 8) == 0
    rg = mod(range=FAKE)
    assert fwd(mod=rg) == WORKSPACE and fwd(mod=rg, ws=FAKE, bytes=need - 1) == WORKSPACE
    assert fwd(mod=rg, ws=FAKE + 16, bytes=need) == WORKSPACE
    plain, more = lib.gqa_prefill_backward_workspace_size(1, 4, 8), lib.gqa_prefill_backward_mod_workspace_size(1, 4, 2, 8)
    assert more > plain and bwd(mod=rg, bytes=plain) == WORKSPACE
    assert dec(ws=NULL) == WORKSPACE


@pytest.mark.gpu
def test_binding_refusals():
    import kv_cache_attention_gqa_b200 as gqa

    def bf(*shape, device="cuda"):
        return torch.zeros(shape, dtype=torch.bfloat16, device=device)

    f, _ = gqa.rope_frequencies(64)
    x = bf(2, 4, 3, 64)
    for args, how in (((x.cpu(), f, [0, 0]), {}), ((x[0], f, [0, 0]), {}), ((x.transpose(2, 3), f, [0, 0]), {}),
                      ((x, f, [0]), {}), ((x, f, torch.zeros(2, 4, dtype=torch.int32)), {}), ((x, f, [0, 0]), dict(offset=1)),
                      ((x, f, [0, 0]), dict(out=bf(2, 4, 3, 32))), ((x, f, [0, 0]), dict(out=bf(2, 1, 3, 64).expand(2, 4, 3, 64))),
                      ((x, f[::2], [0, 0]), {})):
        with pytest.raises(ValueError):
            gqa.rope(*args, **how)
    for args in ((x.half(), f, [0, 0]), (x, f.float(), [0, 0])):
        with pytest.raises(TypeError):
            gqa.rope(*args)
    kc = bf(2, 2, 8, 64)
    q, k = bf(2, 4, 1, 64), bf(2, 2, 1, 64)
    for change in (dict(k=bf(2, 3, 1, 64)), dict(v=bf(2, 2, 2, 64)), dict(kc=bf(2, 2, 9, 64)), dict(pos=None), dict(pos=[0]),
                   dict(kc=bf(3, 2, 8, 64), vc=bf(3, 2, 8, 64))):
        a = dict(q=q, k=k, v=k, kc=kc, vc=kc.clone(), pos=[0, 0]) | change
        with pytest.raises(ValueError):
            gqa.kv_rope_append(a["q"], a["k"], a["v"], a["kc"], a["vc"], a["pos"], f)
    lse = torch.zeros(2, 4, 1, device="cuda")
    for args, how in (((q, kc, lse[:, :, 0]), {}), ((q, bf(3, 2, 8, 64), lse), {}), ((q, kc, lse), dict(kv_len=[1])),
                      ((q, kc, lse), dict(weights=torch.zeros(2, 2, 9, device="cuda"))),
                      ((q.transpose(1, 2), kc, lse.transpose(1, 2)), {})):  # (one head for two KV heads: the library's refusal)
        with pytest.raises((ValueError, gqa.GQAError)):
            gqa.kv_weights(*args, **how)
    with pytest.raises(TypeError):
        gqa.kv_weights(q, kc.float(), lse)
    w = torch.zeros(2, 2, 8, device="cuda")
    vc = kc.clone()
    for how in (dict(budget=0), dict(budget=9), dict(k_out=bf(2, 2, 4, 64)), dict(k_out=bf(2, 2, 4, 64), v_out=bf(2, 2, 4, 64)),
                dict(k_out=bf(2, 2, 4, 64), v_out=bf(2, 2, 5, 64), weights_out=w), dict(kv_len=[1]),
                dict(k_out=bf(2, 2, 6, 64), v_out=bf(2, 2, 6, 64), weights_out=w)):
        with pytest.raises(ValueError):
            gqa.kv_evict(kc, vc, w, how.pop("budget", 4), **how)
    with pytest.raises(gqa.GQAError):
        gqa.kv_evict(kc, vc, w, 4, sink=3, recent=2)
    with pytest.raises(gqa.GQAError):  # the last rows of the source as the destination
        gqa.kv_evict(kc[:1], vc[:1], w[:1], 4, k_out=kc[:1].view(1, 2, 8, 64), v_out=bf(1, 2, 8, 64), weights_out=w[1:].clone())
    slopes, rg = torch.zeros(4, device="cuda"), torch.zeros(2, 1, 2, dtype=torch.int32, device="cuda")
    for how in (dict(alibi_slopes=slopes[:3]), dict(alibi_slopes=slopes.double()), dict(key_range=rg[:, 0]), dict(key_range=rg.long()),
                dict(alibi_slopes=slopes.cpu())):
        with pytest.raises(ValueError):
            gqa.prefill(q, kc, vc, **how)
    with pytest.raises(ValueError):
        gqa.decode(q[:, :, 0], kc, vc, key_range=rg)
    for how in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf"))):
        with pytest.raises(gqa.GQAError):
            gqa.prefill(q, kc, vc, **how)
    assert gqa.get_device_error() == 0
