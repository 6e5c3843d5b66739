"""GPU parity of the head norms with rotation (forward, backward, cache form)
against plain 64-bit arithmetic.

Tolerances, from the roundings alone.  The kernels compute in fp32 and round
once: a bf16 value is off by half a step, 2^-9 of its binade's upper end, at
most 2^-8 of the value.  The fp32 part: the mean of squares (a sum of D <= 128
terms of one sign, in a tree of depth <= 11: 12 * 2^-24), rsqrt (2 ulp), the
products and the rotation (six roundings on terms of the pair's size) stay
below 32 * 2^-24 of the pair's norm; a bf16 result is therefore within
2^-8 |y| + 2^-19 (|u_a| + |u_b|).
"""
import math

import pytest
import torch

from tiled_attention_blackwell_b200 import attn, build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    attn.lib()
    yield
    assert attn.device_status() == attn.ATTN_OK


def rotate(u, c, s, rot, interleaved):
    """The rotation by its matrix [rot, rot] per token: u [T, H, D], c, s [T, rot / 2] (64 bits)."""
    T, half = c.shape
    R = torch.zeros(T, rot, rot, dtype=torch.float64)
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    R[:, a, a] = c
    R[:, a, b] = -s
    R[:, b, b] = c
    R[:, b, a] = s
    y = u.clone()
    y[..., :rot] = torch.einsum("tij,thj->thi", R, u[..., :rot])
    return y, R


def reference(x, w, c, s, rot, eps, interleaved):
    x, w = x.double().cpu(), w.double().cpu()
    u = w * x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    y, R = rotate(u, c, s, rot, interleaved)
    _, size = rotate(u.abs(), torch.ones_like(c), torch.zeros_like(s), rot, interleaved)
    bound = u.abs()
    half = rot // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    pair = u[..., a].abs() + u[..., b].abs()
    bound[..., a] = pair
    bound[..., b] = pair
    return y, 2.0 ** -8 * y.abs() + 2.0 ** -19 * bound, R


def inputs(T, Hq, Hkv, D, rot, seed, *, w_dtype=torch.bfloat16, max_pos=4096):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(w_dtype).to(DEV) for _ in range(2))
    cos, sin = attn.rope_table(max_pos, rot, device=DEV)
    pos = torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32)
    pos[0], pos[-1] = 0, max_pos - 1
    c, s = cos.double().cpu()[pos.long()], sin.double().cpu()[pos.long()]
    return q, k, v, qw, kw, cos, sin, pos.to(DEV), c, s


def within(got, want, bound):
    err = (got.double().cpu() - want).abs()
    assert not torch.isnan(err).any()
    assert (err <= bound).all(), float((err - bound).max())


SHAPES = [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (2, 3, 1, 128, 16), (33, 6, 2, 64, 48), (257, 5, 5, 128, 96),
          (1000, 40, 2, 64, 32), (17, 16, 16, 128, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float32])
def test_forward(shape, interleaved, w_dtype):
    T, Hq, Hkv, D, rot = shape
    q, k, _, qw, kw, cos, sin, pos, c, s = inputs(*shape, seed=T + Hq, w_dtype=w_dtype)
    for eps in (1e-6, 0.5):
        qo, ko = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, eps=eps, interleaved=interleaved)
        for got, x, w in ((qo, q, qw), (ko, k, kw)):
            want, bound, _ = reference(x, w, c, s, rot, eps, interleaved)
            within(got, want, bound)


def test_in_place_batched_and_bit_identical_again():
    q, k, _, qw, kw, cos, sin, pos, _, _ = inputs(60, 6, 2, 128, 128, seed=5)
    want = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos)
    again = attn.qk_norm_rope(q.unflatten(0, (3, 20)), k.unflatten(0, (3, 20)), qw, kw, cos, sin, pos.view(3, 20))
    assert all(torch.equal(a.flatten(0, 1), b) for a, b in zip(again, want))
    rest = k.as_strided((60, 2, 128), k.stride(), k.storage_offset() + 2 * 128).clone()  # V, in the same rows
    out = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, q_out=q, k_out=k)
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rest, k.as_strided((60, 2, 128), k.stride(), k.storage_offset() + 2 * 128))


def test_views_that_are_taken_and_refused():
    qkv = torch.randn(2, 5, 8 * 64, device=DEV).to(torch.bfloat16)
    qw = kw = torch.ones(64, device=DEV)
    cos, sin = attn.rope_table(8, 64, device=DEV)
    pos = torch.arange(5, dtype=torch.int32, device=DEV).repeat(2, 1)
    q, k = qkv[..., :256].unflatten(-1, (4, 64)), qkv[..., 256:384].unflatten(-1, (2, 64))
    want = attn.qk_norm_rope(q.contiguous(), k.contiguous(), qw, kw, cos, sin, pos)

    def same(got, rows):
        assert all(torch.equal(a, b[rows]) for a, b in zip(got, want))

    everything = (slice(None), slice(None))
    same(attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos), everything)
    # one token of each row, one token at all, one head, one key head of several
    same(attn.qk_norm_rope(q[:, 2:3], k[:, 2:3], qw, kw, cos, sin, pos[:, 2:3].contiguous()), (slice(None), slice(2, 3)))
    same(attn.qk_norm_rope(q[1:, 2:3], k[1:, 2:3], qw, kw, cos, sin, pos[1:, 2:3].contiguous()), (slice(1, 2), slice(2, 3)))
    got = attn.qk_norm_rope(q[..., 3:, :], k[..., :1, :], qw, kw, cos, sin, pos)
    assert torch.equal(got[0], want[0][..., 3:, :]) and torch.equal(got[1], want[1][..., :1, :])
    for bad in (q[:, :3], q.transpose(0, 1).contiguous().transpose(0, 1)[:, :3], q[..., ::2, :], q[..., ::2]):
        with pytest.raises((TypeError, attn.AttnError)):
            attn.qk_norm_rope(bad, k[:, :bad.shape[1]], qw, kw, cos, sin, pos[:, :bad.shape[1]].contiguous())
    with pytest.raises(attn.AttnError) as e:  # tokens that share one row
        attn.qk_norm_rope(q[:1, :1].expand(2, 5, 4, 64), k, qw, kw, cos, sin, pos)
    assert e.value.status == attn.ATTN_ERR_INVALID_ARG
    with pytest.raises(TypeError, match="q_out"):
        attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, q_out=q[:, :, :2])


def test_zero_row_and_special_values():
    q, k, _, qw, kw, cos, sin, pos, _, _ = inputs(4, 2, 2, 64, 64, seed=6)
    q = q.contiguous()
    q[1] = 0.0
    q[2, 0, 3] = float("nan")
    qo, _ = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos)
    assert (qo[1] == 0).all()
    assert torch.isnan(qo[2, 0]).all() and not torch.isnan(qo[2, 1]).any()
    # with eps = 0 a row of zeros is 0 * inf, as in the formula
    qo, _ = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, eps=0.0)
    assert torch.isnan(qo[1]).all() and not torch.isnan(qo[3]).any()


def test_positions_outside_the_table_are_clamped_and_reported():
    q, k, _, qw, kw, cos, sin, pos, _, _ = inputs(4, 2, 1, 64, 32, seed=7, max_pos=50)
    pos[:] = torch.tensor([-1, 49, 50, 2 ** 31 - 1], dtype=torch.int32)
    got = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos)
    assert attn.device_status() == attn.ATTN_ERR_RANGE
    pos[:] = torch.tensor([0, 49, 49, 49], dtype=torch.int32)
    want = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos)
    assert attn.device_status() == attn.ATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------- backward

def backward_reference(dy, x, w, R, rot, eps):
    dy, x, w = dy.double().cpu(), x.double().cpu(), w.double().cpu()
    D = x.shape[-1]
    g = dy.clone()
    g[..., :rot] = torch.einsum("tji,thj->thi", R, dy[..., :rot])
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    dot = (w * g * x).sum(-1, keepdim=True)
    dx = r * w * g - r ** 3 * x * dot / D
    terms = g * x * r
    # fp32 part of dx: the sums over the head may cancel, so by the sizes of their terms
    size = r * (w * g).abs() + r ** 3 * x.abs() * (w * g * x).abs().sum(-1, keepdim=True) / D
    pair = r * w.abs() * dy.abs().amax(-1, keepdim=True) * 2
    return dx, 2.0 ** -8 * dx.abs() + 2.0 ** -18 * (size + pair), terms.flatten(0, 1).sum(0), \
        terms.abs().flatten(0, 1).sum(0)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("types", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_backward(shape, interleaved, types):
    T, Hq, Hkv, D, rot = shape
    q, k, _, qw, kw, cos, sin, pos, c, s = inputs(*shape, seed=T + Hq, w_dtype=torch.float32)
    g = torch.Generator().manual_seed(9)
    dq, dk = (torch.randn(x.shape, generator=g).to(t).to(DEV) for x, t in zip((q, k), types))
    dqi, dki, dqw, dkw = attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos, interleaved=interleaved)
    for dy, x, w, dx, dw in ((dq, q, qw, dqi, dqw), (dk, k, kw, dki, dkw)):
        _, _, R = reference(x, w, c, s, rot, 1e-6, interleaved)
        want, bound, want_w, size_w = backward_reference(dy, x, w, R, rot, 1e-6)
        within(dx, want, bound)
        # dw: every term is off by less than 24 * 2^-24 of the sizes in it (the rotation mixes a pair),
        # and a sum in fp32 of n terms in chains of length L by L * 2^-24 of the terms' sizes.
        mixed = size_w + (dy.double().cpu().abs().amax(-1, keepdim=True) * 2 * x.double().cpu().abs() *
                          (x.double().cpu().pow(2).mean(-1, keepdim=True)).rsqrt()).flatten(0, 1).sum(0)
        within(dw, want_w, 2.0 ** -24 * (24 * mixed + 128 * size_w))


def test_backward_against_differences():
    """The gradients of sum(y * t) by central differences of the 64-bit formula."""
    shape = (3, 2, 1, 64, 48)
    q, k, _, qw, kw, cos, sin, pos, c, s = inputs(*shape, seed=21, w_dtype=torch.float32)
    g = torch.Generator().manual_seed(2)
    dq, dk = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    dqi, dki, dqw, dkw = attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos)

    def value(x, w, dy):
        u = w * x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
        return float((rotate(u, c, s, 48, False)[0] * dy).sum())

    h = 1e-4  # differences are off by h^2 times third derivatives of order 10: 1e-7
    for dy, x, w, dx, dw in ((dq, q, qw, dqi, dqw), (dk, k, kw, dki, dkw)):
        x, w, dy = x.double().cpu(), w.double().cpu(), dy.double().cpu()
        for at in ((0, 0, 0), (1, 0, 23), (2, 0, 24), (2, 0, 47), (0, 0, 63)):
            up, down = x.clone(), x.clone()
            up[at] += h
            down[at] -= h
            want = (value(up, w, dy) - value(down, w, dy)) / (2 * h)
            assert abs(float(dx[at]) - want) <= 2.0 ** -8 * abs(want) + 1e-4
        for d in (0, 25, 63):
            up, down = w.clone(), w.clone()
            up[d] += h
            down[d] -= h
            want = (value(x, up, dy) - value(x, down, dy)) / (2 * h)
            assert abs(float(dw[d]) - want) <= 1e-4


@pytest.mark.parametrize("size,eps", [(1e-17, 0.0), (1e-13, 0.0), (1e-13, 1e-6), (1e14, 1e-6), (1e15, 1e-6), (1e17, 1e-6)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_far_from_one(size, eps, D):
    """Inputs whose squares fp32 still holds (sums of 128 of them included), but
    not the cube of their norm: the bounds are those of ordinary inputs."""
    shape = (5, 3, 2, D, D)
    q, k, _, qw, kw, cos, sin, pos, c, s = inputs(*shape, seed=31, w_dtype=torch.float32)
    q, k = ((x.double() * size).to(torch.bfloat16) for x in (q, k))
    g = torch.Generator().manual_seed(32)
    dq, dk = (torch.randn(x.shape, generator=g).to(DEV) for x in (q, k))
    out = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, eps=eps)
    dqi, dki, dqw, dkw = attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos, eps=eps)
    for y, dy, x, w, dx, dw in ((out[0], dq, q, qw, dqi, dqw), (out[1], dk, k, kw, dki, dkw)):
        want, bound, R = reference(x, w, c, s, D, eps, False)
        within(y, want, bound)
        want, bound, want_w, size_w = backward_reference(dy, x, w, R, D, eps)
        within(dx, want, bound)
        x = x.double().cpu()
        r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
        mixed = size_w + (dy.double().cpu().abs().amax(-1, keepdim=True) * 2 * x.abs() * r).flatten(0, 1).sum(0)
        within(dw, want_w, 2.0 ** -24 * (24 * mixed + 128 * size_w))


def test_backward_into_a_packed_gradient_deterministic():
    T, Hq, Hkv, D = 700, 6, 2, 128
    q, k, _, qw, kw, cos, sin, pos, _, _ = inputs(T, Hq, Hkv, D, 128, seed=30)
    dq, dk = torch.randn(T, Hq, D, device=DEV), torch.randn(T, Hkv, D, device=DEV).to(torch.bfloat16)
    want = attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos)
    packed = torch.full((T, (Hq + 2 * Hkv) * D), 7.0, dtype=torch.bfloat16, device=DEV)
    views = [x.unflatten(-1, (-1, D)) for x in packed.split([Hq * D, Hkv * D, Hkv * D], -1)]
    got = attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos, dq_in=views[0], dk_in=views[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (views[2] == 7).all()


# ----------------------------------------------------------------- cache form

@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_cache_form(shape, dtype):
    T, Hq, Hkv, D, rot = shape
    q, k, v, qw, kw, cos, sin, pos, c, s = inputs(*shape, seed=T + 1)
    page = 16
    pages = T // page + 3
    fp8 = dtype == torch.float8_e4m3fn
    kd, vd = (1 / 96, 1 / 50) if fp8 else (1.0, 1.0)
    raw = torch.uint8 if fp8 else torch.int16
    kc, vc = (torch.full((pages, page, Hkv, D), 3, dtype=raw, device=DEV).view(dtype) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    pad = torch.rand(T, generator=g) < 0.2
    pad[0] = T > 1
    pad[-1] = False
    slots[pad] = -1
    qo = torch.full_like(q.contiguous(), 5.0)
    interleaved = T % 2 == 0
    attn.qk_norm_rope_cache(q, k, v, qw, kw, cos, sin, pos, slots.to(DEV), kc, vc, k_descale=kd, v_descale=vd,
                            q_out=qo, interleaved=interleaved)
    qn, kn = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, interleaved=interleaved)
    keep = ~pad
    assert torch.equal(qo[keep.to(DEV)], qn[keep.to(DEV)])
    assert (qo[pad.to(DEV)] == 5).all()
    at = slots[keep].long()
    other = torch.ones(pages * page, dtype=torch.bool)
    other[at] = False
    for cache in (kc, vc):
        assert (cache.view(raw).flatten(0, 1).cpu()[other] == 3).all(), "slots of no token were written"
    got_k, got_v = (x.flatten(0, 1)[at.to(DEV)] for x in (kc.view(raw), vc.view(raw)))
    if not fp8:
        assert torch.equal(got_k.view(dtype), kn[keep.to(DEV)])
        assert torch.equal(got_v.view(dtype), v[keep.to(DEV)])
        return
    # V: the division and the rounding to e4m3 are exact operations of their own
    want = (v[keep.to(DEV)].float() / torch.tensor(vd, device=DEV)).clamp(-448, 448).to(dtype)
    assert torch.equal(got_v, want.view(raw))
    # K: half a step of e4m3 (2^-4 of the value, 2^-10 of a subnormal one) beside the fp32 part
    y, bound, _ = reference(k, kw, c, s, rot, 1e-6, interleaved)
    y, bound = (y / kd)[keep], (bound / kd)[keep]
    fp32_part = bound - 2.0 ** -8 * y.abs()
    within(got_k.view(dtype).float(), y.clamp(-448, 448), 2.0 ** -4 * y.abs() + 2.0 ** -10 + 1.1 * fp32_part)


def test_cache_slots_out_of_range_are_reported_and_skipped():
    q, k, v, qw, kw, cos, sin, pos, _, _ = inputs(3, 2, 1, 64, 64, seed=8)
    kc, vc = (torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.tensor([32, 2 ** 31 - 1, 31], dtype=torch.int32, device=DEV)
    attn.qk_norm_rope_cache(q, k, v, qw, kw, cos, sin, pos, slots, kc, vc)
    assert attn.device_status() == attn.ATTN_ERR_RANGE
    assert torch.equal(vc.flatten(0, 1)[31], v[2]) and (vc.flatten(0, 1)[:31] == 0).all()


def test_captured_and_on_a_side_stream():
    q, k, v, qw, kw, cos, sin, pos, _, _ = inputs(40, 8, 2, 128, 128, seed=12)
    dq, dk = torch.randn(40, 8, 128, device=DEV), torch.randn(40, 2, 128, device=DEV)
    want = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos) + \
        attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos, stream=side) + \
        attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.qk_norm_rope(q, k, qw, kw, cos, sin, pos) + \
            attn.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
