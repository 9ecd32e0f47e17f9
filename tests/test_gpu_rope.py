"""Rotary positions and the norm + rotation + cache write (``pa_rope``,
``pa_rope_and_cache``) against float64.

Tolerance of an output y0 = f (x0 cos a - x1 sin a): its own rounding to bf16,
half a step, is at most 2^-8 |y|.  Before it, in fp32: the angle reduced to a
turn is off by 2^-25 turns (1.9e-7 rad), cos and sin by a few 2^-24, the norm's
sum of D squares, its rsqrt and the two products by less than 16 * 2^-24 of the
value: together below 4e-6 f (|x0| + |x1|) of the normed pair."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import drafting
from oracle.paged_attention import bf16_bits_to_f64
from workloads.synth import f32_to_bf16_bits

import gpu_helpers as H

pytestmark = pytest.mark.gpu


def pa():
    import paged_kv_cache_454_b200 as m
    return m


def freqs(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))


def bits(rng, *shape):
    return f32_to_bf16_bits((2 * rng.standard_normal(shape)).astype(np.float32))


def dev_f64(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.float64))).cuda()


def close(got, x, positions, f, interleaved, factor, what):
    """``x``: the float64 rows that are rotated."""
    want = drafting.rope(x, positions, f, interleaved, factor)
    got = H.host_f64(got)
    half = len(f)
    room = np.zeros_like(want)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        room[..., a] = room[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    room[..., 2 * half:] = np.abs(x[..., 2 * half:])
    tol = 2.0 ** -8 * np.abs(want) + 4e-6 * max(factor, 1.0) * room
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, np.argwhere(bad)[:3], np.abs(got - want).max())


ROPE = [  # tokens, hq, hkv, d, rot, interleaved, factor, furthest position
    (1, 1, 0, 64, 64, False, 1.0, 10),
    (1, 8, 1, 128, 128, False, 1.0, 5000),
    (2, 7, 7, 128, 32, True, 1.0, 100000),
    (17, 5, 1, 64, 48, False, 1.25, 1000000),
    (33, 40, 8, 128, 96, True, 1.0, 30),
    (300, 3, 3, 64, 16, True, 0.5, 10 ** 9),
    (300, 64, 8, 128, 112, False, 1.2, 10 ** 9),
    (1501, 2, 1, 128, 64, False, 1.0, 4096),
    (5, 16, 16, 128, 0, False, 3.0, 50),
]


@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,factor,far", ROPE)
def test_rope(t, hq, hkv, d, rot, inter, factor, far):
    rng = np.random.default_rng(t * 1000 + d + rot)
    q, k = bits(rng, t, hq, d), bits(rng, t, hkv, d)
    pos = rng.integers(-far, far, t)
    f = freqs(rot)
    dq = H.dev_bf16(q)
    dk = H.dev_bf16(k) if hkv else None
    qo, ko = pa().pa_rope(dq, dk, H.dev_i64(pos), dev_f64(f), interleaved=inter, factor=factor)
    close(qo, bf16_bits_to_f64(q), pos, f, inter, factor, "q")
    if hkv:
        close(ko, bf16_bits_to_f64(k), pos, f, inter, factor, "k")
    else:
        assert ko is None
    assert np.array_equal(H.host_bits(dq), q)  # inputs untouched
    # in place: the same bits
    q2, k2 = pa().pa_rope(dq, dk, H.dev_i64(pos), dev_f64(f), interleaved=inter, factor=factor,
                          q_out=dq, k_out=dk)
    assert q2 is dq and np.array_equal(H.host_bits(dq), H.host_bits(qo))
    if hkv:
        assert np.array_equal(H.host_bits(k2), H.host_bits(ko))


def test_rope_strides_and_slices():
    import torch
    rng = np.random.default_rng(4)
    t, hq, hkv, d, rot = 70, 6, 2, 64, 32
    x = bits(rng, t + 1, hq + 2 * hkv + 1, d)
    pos = rng.integers(0, 9000, t + 1)
    f = freqs(rot)
    dx = H.dev_bf16(x)[1:]
    q, k = dx[:, :hq], dx[:, hq:hq + hkv]
    wide = torch.full((t, hq + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    # positions start at an 8-byte boundary
    qo, ko = pa().pa_rope(q, k, H.dev_i64(pos)[1:], dev_f64(f), q_out=wide[:, 2:2 + hq])
    xf = bf16_bits_to_f64(x)[1:]
    close(qo, xf[:, :hq], pos[1:], f, False, 1.0, "q")
    close(ko, xf[:, hq:hq + hkv], pos[1:], f, False, 1.0, "k")
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + hq:] == 7).all())


def test_rope_leaves_the_rest_of_the_head_alone():
    # infinities, NaN and the sign of zero past rot_dim come out as they went in
    import torch
    q = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    q[:, :, 64] = float("inf")
    q[:, :, 65] = -float("inf")
    q[:, :, 66] = float("nan")
    q[:, :, 67] = -0.0
    out, _ = pa().pa_rope(q, None, H.dev_i64([1, 2, 3]), dev_f64(freqs(64)))
    assert bool(torch.isposinf(out[:, :, 64]).all()) and bool(torch.isneginf(out[:, :, 65]).all())
    assert bool(torch.isnan(out[:, :, 66]).all()) and bool((out[:, :, :64] == 0).all())
    assert bool(torch.signbit(out[:, :, 67]).all())


CACHE = [  # tokens, hq, hkv, d, rot, interleaved, q weight, k weight, padded
    (1, 64, 8, 128, 128, False, True, True, 0),
    (1, 4, 4, 64, 64, True, False, False, 0),
    (19, 8, 1, 128, 64, True, True, False, 3),
    (130, 40, 8, 128, 128, False, True, True, 10),
    (777, 5, 5, 64, 48, False, False, True, 77),
    (64, 16, 2, 128, 0, False, True, True, 64),
    (1300, 7, 1, 128, 16, False, True, True, 1),
]


@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,with_q,with_k,pad", CACHE)
def test_rope_and_cache(t, hq, hkv, d, rot, inter, with_q, with_k, pad):
    import torch
    rng = np.random.default_rng(t + hq + rot)
    x = bits(rng, t, hq + 2 * hkv, d)
    nb = -(-t // 16) + 3
    kp, vp = bits(rng, nb, hkv, 16, d), bits(rng, nb, hkv, 16, d)
    slots = rng.permutation(nb * 16)[:t].astype(np.int64)
    slots[rng.permutation(t)[:pad]] = rng.choice([-1, -7])
    pos = rng.integers(0, 200000, t)
    f = freqs(rot)
    qw = f32_to_bf16_bits((1 + 0.3 * rng.standard_normal(d)).astype(np.float32))
    kw = f32_to_bf16_bits((1 + 0.3 * rng.standard_normal(d)).astype(np.float32))
    dx, dk, dv = H.dev_bf16(x), H.dev_bf16(kp), H.dev_bf16(vp)
    qo = pa().pa_rope_and_cache(
        dx[:, :hq], dx[:, hq:hq + hkv], dx[:, hq + hkv:], dk, dv, H.dev_i64(slots),
        H.dev_i64(pos), dev_f64(f), interleaved=inter, factor=1.1 if rot else 1.0,
        q_weight=H.dev_bf16(qw) if with_q else None, k_weight=H.dev_bf16(kw) if with_k else None,
        eps=1e-5)
    factor = float(np.float32(1.1)) if rot else 1.0
    xf = bf16_bits_to_f64(x)
    q, k = xf[:, :hq], xf[:, hq:hq + hkv]
    if with_q:
        q = drafting.head_norm(q, bf16_bits_to_f64(qw), float(np.float32(1e-5)))
    if with_k:
        k = drafting.head_norm(k, bf16_bits_to_f64(kw), float(np.float32(1e-5)))
    close(qo, q, pos, f, inter, factor, "q")
    # every written slot, and nothing else
    flat = lambda p: np.swapaxes(p, 1, 2).reshape(-1, hkv, d)  # noqa: E731
    gk, gv = flat(H.host_bits(dk)), flat(H.host_bits(dv))
    want_v = flat(vp).copy()
    live = np.nonzero(slots >= 0)[0]
    want_v[slots[live]] = x[live, hq + hkv:]
    assert np.array_equal(gv, want_v)
    rest = np.setdiff1d(np.arange(nb * 16), slots[live])
    assert np.array_equal(gk[rest], flat(kp)[rest])
    if len(live):
        got = torch.from_numpy(gk[slots[live]].view(np.int16)).view(torch.bfloat16)
        close(got, k[live], pos[live], f, inter, factor, "k")
    assert pa().pa_get_device_error() == 0


def test_rope_and_cache_flags_slots_outside_the_pool():
    import torch
    rng = np.random.default_rng(8)
    x = bits(rng, 4, 3, 64)
    dk = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros_like(dk)
    dx = H.dev_bf16(x)
    qo = pa().pa_rope_and_cache(dx[:, :1], dx[:, 1:2], dx[:, 2:], dk, dv,
                                H.dev_i64([0, 32, 2 ** 40, 31]), H.dev_i64([0, 1, 2, 3]),
                                dev_f64(freqs(64)))
    assert pa().pa_get_device_error() == pa().PA_DEV_ERR_SLOT
    close(qo, bf16_bits_to_f64(x)[:, :1], [0, 1, 2, 3], freqs(64), False, 1.0, "q")
    got = H.host_bits(dv)
    assert np.array_equal(got[0, 0, 0], x[0, 2]) and np.array_equal(got[1, 0, 15], x[3, 2])
    got[0, 0, 0] = got[1, 0, 15] = 0
    assert not got.any()


def test_rope_on_a_side_stream_and_in_a_graph():
    import torch
    rng = np.random.default_rng(9)
    x = H.dev_bf16(bits(rng, 50, 4, 128))
    pos, f = H.dev_i64(rng.integers(0, 999, 50)), dev_f64(freqs(128))
    want, _ = pa().pa_rope(x, None, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = pa().pa_rope(x, None, pos, f, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = pa().pa_rope(x, None, pos, f)
    x.copy_(H.dev_bf16(bits(rng, 50, 4, 128)))
    g.replay()
    again, _ = pa().pa_rope(x, None, pos, f)
    assert torch.equal(out, again) and not torch.equal(out, want)


@pytest.mark.parametrize("d,rot,inter", [(64, 0, False), (64, 48, False), (128, 32, True),
                                         (128, 0, True), (128, 112, False)])
def test_dims_past_the_rotation_keep_their_bits(d, rot, inter):
    # any bits: subnormals, NaN of every payload, both zeros
    rng = np.random.default_rng(d + rot)
    t, hq, hkv = 65, 3, 3
    x = bits(rng, t, hq + 2 * hkv, d)
    x[..., rot:] = rng.integers(0, 1 << 16, (t, hq + 2 * hkv, d - rot))
    x[:40, :, rot:] &= 0x807F     # subnormals
    x[40:50, :, rot:] |= 0x7F80   # infinities and NaN
    dx, pos, f = H.dev_bf16(x), H.dev_i64(rng.integers(0, 999, t)), dev_f64(freqs(rot))
    q, k = dx[:, :hq], dx[:, hq:hq + hkv]
    qo, ko = pa().pa_rope(q, k, pos, f, interleaved=inter, factor=1.5)
    assert np.array_equal(H.host_bits(qo)[..., rot:], x[:, :hq, rot:])
    assert np.array_equal(H.host_bits(ko)[..., rot:], x[:, hq:hq + hkv, rot:])
    dk = H.dev_bf16(np.zeros((5, hkv, 16, d), np.uint16))
    dv = H.dev_bf16(np.zeros((5, hkv, 16, d), np.uint16))
    slots = rng.permutation(80)[:t]
    qo = pa().pa_rope_and_cache(q, k, dx[:, hq + hkv:], dk, dv, H.dev_i64(slots), pos, f,
                                interleaved=inter, factor=1.5)
    assert np.array_equal(H.host_bits(qo)[..., rot:], x[:, :hq, rot:])
    flat = lambda p: np.swapaxes(H.host_bits(p), 1, 2).reshape(-1, hkv, d)  # noqa: E731
    assert np.array_equal(flat(dk)[slots][..., rot:], x[:, hq:hq + hkv, rot:])
    assert np.array_equal(flat(dv)[slots], x[:, hq + hkv:])
