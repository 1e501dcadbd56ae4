"""Rotary positions (gqa_rope, kv_rope_append, kv_rope_append_paged) on the GPU against the fp64 oracle.

Tolerance: the result is rounded once (eps / 2 of its size). Before that, the reduced angle is rounded
to fp32 (pi 2^-24 rad), sin and cos are off by at most 2 ulp (2^-22 of one), the product with the scale
and the two products and their sum round once each (2^-24): below 1e-6 scale (|x0| + |x1|) in all.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _check(out, x, inv_freq, positions, dtype, *, scale=1.0, **how):
    x64 = x.double().cpu().numpy()
    ref = oracle.rope_ref(x64, inv_freq.cpu().numpy(), positions, scale=scale, **how)
    pair = oracle.rope_ref(np.abs(x64), np.zeros(inv_freq.numel()), positions, **how)  # |x| (angle 0)
    size = pair.max(axis=-1, keepdims=True)
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + 2e-6 * abs(scale) * size
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()


CASES = [  # B, h, S, d, d_rot, offset
    (1, 1, 1, 2, 2, 0), (2, 3, 1, 128, 128, 0), (3, 5, 7, 80, 20, 12), (2, 2, 33, 64, 32, 32), (1, 4, 5, 130, 6, 3),
    (2, 1, 9, 576, 64, 512), (1, 40, 65, 72, 72, 0), (1, 2, 3, 7, 4, 1), (2, 3, 4, 4096, 4096, 0), (5, 9, 300, 16, 8, 4),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,h,S,d,d_rot,offset", CASES)
def test_rope(dtype, interleaved, B, h, S, d, d_rot, offset):
    import kv_cache_attention_gqa_b200 as gqa

    x = _rand((B, h, S, d), dtype, d + S).cuda()
    f, _ = gqa.rope_frequencies(d_rot)
    first = [(37 * b) % 101 for b in range(B)]
    at = [[p + t for t in range(S)] for p in first]
    how = dict(offset=offset, interleaved=interleaved)
    _check(gqa.rope(x, f, first, **how), x, f, at, dtype, **how)
    _check(gqa.rope(x, f, first, inverse=True, scale=1.25, **how), x, f, at, dtype, inverse=True, scale=1.25, **how)
    assert gqa.get_device_error() == 0


def test_positions_per_token_far_away_and_scalings():
    import kv_cache_attention_gqa_b200 as gqa

    x = _rand((2, 3, 4, 64), torch.float32, 1).cuda()
    at = [[0, 1, 2**31 - 1, 5], [999999, 123456789, 3, 3]]
    for how in (dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
                dict(scaling="yarn", factor=32.0, original_length=4096)):
        f, scale = gqa.rope_frequencies(64, 1e6, **how)
        out = gqa.rope(x, f, torch.tensor(at, dtype=torch.int32, device="cuda"), scale=scale)
        _check(out, x, f, at, torch.float32, scale=scale)


def test_strided_inputs_outputs_and_in_place():
    import kv_cache_attention_gqa_b200 as gqa

    f, _ = gqa.rope_frequencies(64)
    at = [[5 + t for t in range(11)], [9 + t for t in range(11)]]
    fused = _rand((2, 11, 7, 64), torch.bfloat16, 3).cuda()      # (B, S, heads, d)
    x = fused[:, :, 1:5].transpose(1, 2)
    ref = gqa.rope(x.contiguous(), f, [5, 9])
    _check(ref, x, f, at, torch.bfloat16)
    assert torch.equal(gqa.rope(x, f, [5, 9]), ref)
    shifted = torch.empty(2 * 4 * 11 * 64 + 3, dtype=torch.bfloat16, device="cuda")[3:].view(2, 4, 11, 64)
    shifted.copy_(x)                                             # rows on 2-byte boundaries only
    assert torch.equal(gqa.rope(shifted, f, [5, 9]), ref)
    odd = torch.zeros(2, 4, 11, 67, dtype=torch.bfloat16, device="cuda")[..., 1:65]
    odd.copy_(x)                                                 # odd row stride
    assert torch.equal(gqa.rope(odd, f, [5, 9]), ref)
    before = fused.clone()
    assert gqa.rope(x, f, [5, 9], out=x) is x                    # in place, between other heads
    assert torch.equal(x, ref)
    assert torch.equal(fused[:, :, :1], before[:, :, :1]) and torch.equal(fused[:, :, 5:], before[:, :, 5:])
    back = gqa.rope(gqa.rope(ref.float(), f, [5, 9]), f, [5, 9], inverse=True)
    assert (back - ref.float()).abs().max() <= 4e-6 * ref.float().abs().max()
    many = _rand((1, 1, 11, 64), torch.bfloat16, 4).cuda().expand(2, 4, 11, 64)  # broadcast input
    assert torch.equal(gqa.rope(many, f, [5, 9]), gqa.rope(many.contiguous(), f, [5, 9]))


def test_gradient_is_the_inverse_rotation():
    """<rope(x + e v) - rope(x - e v), w> / 2e = <v, inverse(w)>: rope is linear, so the difference is exact."""
    import kv_cache_attention_gqa_b200 as gqa

    f, _ = gqa.rope_frequencies(48)
    x, v, w = (_rand((2, 3, 5, 64), torch.float32, s).cuda() for s in (5, 6, 7))
    for inter in (False, True):
        how = dict(offset=8, interleaved=inter, scale=1.5)
        up, down = (gqa.rope(x + e * v, f, [3, 90], **how) for e in (0.5, -0.5))
        diff = ((up - down).double() * w.double()).sum()
        grad = (gqa.rope(w, f, [3, 90], inverse=True, **how).double() * v.double()).sum()
        assert abs(diff - grad) <= 1e-5 * (v.norm() * w.norm())


def test_negative_position_is_flagged_and_zero():
    import kv_cache_attention_gqa_b200 as gqa

    x = _rand((2, 2, 3, 64), torch.bfloat16, 8).cuda()
    f, _ = gqa.rope_frequencies(32)
    out = gqa.rope(x, f, torch.tensor([[0, -1, 2], [3, 4, 5]], dtype=torch.int32, device="cuda"))
    assert gqa.get_device_error() == 2
    assert out[0, :, 1].abs().sum() == 0
    good = gqa.rope(x, f, [0, 3])
    assert torch.equal(out[0, :, 0], good[0, :, 0]) and torch.equal(out[1], good[1])
    assert gqa.rope(x[:, :, :0], f, [0, 0]).shape == (2, 2, 0, 64)
    assert gqa.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [0, 16, 5])
@pytest.mark.parametrize("B,h_q,h_kv,S,d,d_rot", [(3, 4, 2, 1, 128, 128), (2, 6, 3, 9, 64, 32), (1, 3, 3, 70, 10, 6)])
def test_append(dtype, page, B, h_q, h_kv, S, d, d_rot):
    """q_out and the cached k equal rope's bits, v and every other cache row are untouched copies."""
    import kv_cache_attention_gqa_b200 as gqa

    T = 80
    qkv = _rand((B, S, h_q + 2 * h_kv, d), dtype, 11).cuda()
    q, k, v = (t.transpose(1, 2) for t in qkv.split([h_q, h_kv, h_kv], dim=2))
    f, _ = gqa.rope_frequencies(d_rot)
    pos = torch.tensor([(13 * b) % (T - S + 1) for b in range(B)], dtype=torch.int32, device="cuda")
    pos[-1] = T - S
    kc, vc = _rand((B, h_kv, T, d), dtype, 12).cuda(), _rand((B, h_kv, T, d), dtype, 13).cuda()
    for positions in (None, pos + 1000, pos[:, None] * 3 + torch.arange(S, device="cuda", dtype=torch.int32)):
        at = pos if positions is None else positions
        kr, vr = kc.clone(), vc.clone()
        qr = gqa.rope(q, f, at, interleaved=True, scale=1.1)
        gqa.kv_append(kr, vr, gqa.rope(k, f, at, interleaved=True, scale=1.1), v.contiguous(), pos)
        how = dict(positions=positions, interleaved=True, scale=1.1)
        if page:
            n = T // page
            order = torch.randperm(B * n, generator=torch.Generator().manual_seed(1)).cuda()
            table = order.view(B, n).to(torch.int32)

            def paged(dense):
                pool = torch.empty(B * n, h_kv, page, d, dtype=dtype, device="cuda")
                pool[order] = dense.view(B, h_kv, n, page, d).transpose(1, 2).reshape(B * n, h_kv, page, d)
                return pool

            kd, vd = paged(kc), paged(vc)
            qo = gqa.kv_rope_append_paged(q, k, v, kd, vd, pos, table, f, **how)
            kr, vr = paged(kr), paged(vr)
        else:
            kd, vd = kc.clone(), vc.clone()
            qo = gqa.kv_rope_append(q, k, v, kd, vd, pos, f, **how)
        assert torch.equal(qo, qr) and torch.equal(kd, kr) and torch.equal(vd, vr)
    qc = q.contiguous()
    assert gqa.kv_rope_append(qc, k, v, kc.clone(), vc.clone(), pos, f, q_out=qc) is qc  # in place
    assert torch.equal(qc, gqa.rope(q, f, pos))
    assert gqa.get_device_error() == 0


def test_append_outside_the_cache_or_the_pool_is_flagged():
    import kv_cache_attention_gqa_b200 as gqa

    f, _ = gqa.rope_frequencies(64)
    q, k = _rand((2, 4, 2, 64), torch.bfloat16, 1).cuda(), _rand((2, 2, 2, 64), torch.bfloat16, 2).cuda()
    kc = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    out = gqa.kv_rope_append(q, k, k, kc, vc, [7, 0], f)
    assert gqa.get_device_error() == 2
    assert kc[0].abs().sum() == 0 and vc[0].abs().sum() == 0 and torch.equal(vc[1, :, :2], k[1])
    assert torch.equal(out, gqa.rope(q, f, [7, 0]))  # the queries have positions all the same
    pool, vpool = torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    gqa.kv_rope_append_paged(q, k, k, pool, vpool, [0, 4], [[0, 3], [0, 2]], f)
    assert gqa.get_device_error() == 0
    gqa.kv_rope_append_paged(q, k, k, pool, vpool, [3, 4], [[0, 3], [-1, 2]], f)  # token 1 of sequence 0 has no page
    assert gqa.get_device_error() == 5
    assert torch.equal(vpool[0, :, 3], k[0, :, 0]) and vpool[1].abs().sum() == 0
    gqa.kv_rope_append(q, k, k, kc, vc, [0, 0], f, positions=[-4, 0])  # no position: zeros, not cached
    assert gqa.get_device_error() == 2 and kc[0].abs().sum() == 0


def test_captured_and_on_another_stream():
    import kv_cache_attention_gqa_b200 as gqa

    f, _ = gqa.rope_frequencies(128)
    q, k, v = (_rand((4, h, 1, 128), torch.bfloat16, h).cuda() for h in (8, 2, 3))
    v = v[:, :2].contiguous()
    kc, vc = torch.zeros(4, 2, 32, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 2, 32, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    qo = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gqa.kv_rope_append(q, k, v, kc, vc, pos, f, q_out=qo)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gqa.kv_rope_append(q, k, v, kc, vc, pos, f, q_out=qo)
        pos += 1
    for step in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for step in range(5):
        assert torch.equal(kc[:, :, step], gqa.rope(k, f, [step] * 4)[:, :, 0]) and torch.equal(vc[:, :, step], v[:, :, 0])
    assert torch.equal(qo, gqa.rope(q, f, [4] * 4)) and kc[:, :, 5:].abs().sum() == 0
