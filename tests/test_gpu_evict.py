"""Eviction (``pa_evict``) and the move of kept tokens (``pa_compact_tokens``): exact
against the definition, token by token and bit by bit."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import drafting
from workloads import synth

import gpu_helpers as H

pytestmark = pytest.mark.gpu


def pa():
    import paged_kv_cache_454_b200 as m
    return m


def dev_f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.float32))).cuda()


class Batch:
    """Sequences over a pool of random bits, and as many free blocks again."""

    def __init__(self, seed, lens, hkv, d, width=None, ties=False):
        self.rng = rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        need = -(-self.lens // 16)
        total = int(need.sum())
        self.nb = nb = 2 * total + 3
        order = rng.permutation(nb)
        w = max(1, int(need.max())) + 1
        self.tables = np.full((len(lens), w), synth.INT32_MAX, np.int32)
        self.fresh = np.full((len(lens), w), synth.INT32_MAX, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = order[at:at + k]
            self.fresh[s, :k] = order[total + at:total + at + k]
            at += k
        self.hkv, self.d = hkv, d
        self.k, self.v = (rng.integers(0, 1 << 16, (nb, hkv, 16, d)).astype(np.uint16)
                          for _ in range(2))
        self.width = width or max(1, int(self.lens.max()))
        m = np.exp(3 * rng.standard_normal((len(lens), hkv, self.width))).astype(np.float32)
        if ties:
            m = np.floor(np.minimum(m, 4.0))
        self.mass = m.astype(np.float32)

    def choices(self, budgets, sink, recent, most):
        return [[drafting.evict_choice(self.mass[s, g], int(self.lens[s]),
                                       min(int(budgets[s]), most), sink, recent)
                 for g in range(self.hkv)] for s in range(len(self.lens))]

    def run(self, budgets, sink, recent, new, most=None, in_place_mass=False):
        dk, dv = H.dev_bf16(self.k), H.dev_bf16(self.v)
        mass = dev_f32(self.mass)
        kw = {}
        if in_place_mass:
            kw["mass_out"] = mass
        got = pa().pa_evict(mass, dk, dv, H.dev_i32(self.tables), H.dev_i32(self.lens),
                            H.dev_i32(budgets), sink=sink, recent=recent,
                            new_tables=H.dev_i32(self.fresh) if new else None, max_keep=most, **kw)
        return got, dk, dv

    def check(self, budgets, sink, recent, new, most=None, in_place_mass=False):
        import torch
        budgets = np.asarray(budgets, np.int32)
        (kept, lens, mass), dk, dv = self.run(budgets, sink, recent, new, most, in_place_mass)
        cap = kept.shape[2]
        want = self.choices(budgets, sink, recent, min(cap, mass.shape[2]))
        k, v = self.k, self.v
        kept, lens, mass = kept.cpu().numpy(), lens.cpu().numpy(), mass.cpu().numpy()
        for s in range(len(self.lens)):
            n = len(want[s][0])
            assert lens[s] == n
            for g in range(self.hkv):
                assert np.array_equal(kept[s, g, :n], want[s][g]), (s, g)
                m = self.mass[s, g][want[s][g]]
                assert np.array_equal(mass[s, g, :n].view(np.uint32) if not np.isnan(m).any()
                                      else np.isnan(mass[s, g, :n]),
                                      (m + 0.0).view(np.uint32) if not np.isnan(m).any()
                                      else np.isnan(m)), (s, g)
            if in_place_mass:
                assert np.array_equal(mass[s, :, n:], self.mass[s, :, n:], equal_nan=True)
            table = self.fresh[s] if new else None
            k = drafting.compact(k, self.tables[s], 0, want[s], table)
            v = drafting.compact(v, self.tables[s], 0, want[s], table)
        assert np.array_equal(H.host_bits(dk), k) and np.array_equal(H.host_bits(dv), v)
        assert pa().pa_get_device_error() == 0


CASES = [  # lens, hkv, d, budgets, sink, recent
    ([1], 1, 64, [1], 0, 0),
    ([1], 1, 128, [0], 1, 1),
    ([17, 33, 16], 2, 64, [5, 40, 16], 1, 2),
    ([300, 40, 1000], 3, 128, [100, 10, 999], 4, 32),
    ([1024, 1025, 1023], 2, 128, [512, 512, 512], 0, 0),
    ([4097, 2000], 1, 64, [2049, 1], 3, 3),          # eight tokens a thread
    ([9000], 2, 128, [1531], 16, 256),               # sixteen
    ([20011, 31], 1, 128, [4096, 8], 4, 64),         # thirty-two
    ([33000, 500], 1, 64, [3001, 500], 5, 77),
    ([70001], 2, 64, [65000], 0, 1),
    ([100] * 20, 2, 64, [50] * 20, 2, 5),            # a CTA per row: up to 2048 tokens
    ([5000, 100, 8192] + [64] * 37, 1, 64, [700] * 40, 2, 5),   # and up to 8192
    ([140000], 1, 64, [30000], 4, 1000),             # past what a cluster holds
]


@pytest.mark.parametrize("new", [True, False], ids=["fresh", "in_place"])
@pytest.mark.parametrize("lens,hkv,d,budgets,sink,recent", CASES)
def test_evict(lens, hkv, d, budgets, sink, recent, new):
    Batch(sum(lens) + hkv, lens, hkv, d).check(budgets, sink, recent, new)


@pytest.mark.parametrize("length", [700, 5000, 40000, 132000])
def test_evict_ties_go_to_the_lowest_index(length):
    b = Batch(3, [length, length // 2], 2, 64, ties=True)
    b.check([length // 3, length // 3], 2, 9, new=True)
    b.mass[:] = 0.0  # nothing was looked at: the first ones stay
    b.mass[:, :, ::2] = -0.0
    b.check([length // 3, length // 4], 0, 5, new=False)


@pytest.mark.parametrize("length", [500, 6000, 6001, 36000, 133000])
def test_evict_unusual_weights(length):
    # NaN is the least, infinities and denormals keep their order
    b = Batch(5, [length] + [1] * 40, 2, 64) if length == 6001 else Batch(5, [length], 2, 64)
    m = b.mass[0, 0]
    m[:] = b.rng.choice(np.array([np.nan, np.inf, -np.inf, 1e-45, 3e-45, -1e-45, 0.0, -2.5, 7.0],
                                 np.float32), length)
    order = np.argsort(b.rng.random(length))
    b.mass[0, 1] = (order * np.float32(1e-45)).astype(np.float32)  # denormals only
    for budget in (length // 5, length // 2, length - 3):
        b.check([budget] * len(b.lens), 1, 1, new=True)
    b.check([length // 2] * len(b.lens), 0, 0, new=False, in_place_mass=True)


def test_evict_bounds_and_strides():
    b = Batch(7, [200, 100], 2, 128, width=333)
    b.check([50, 1000], 1000, 1000, new=True, most=64)      # kept holds 64, all sinks
    b.check([-5, 3], 0, 7, new=False, most=64)              # nothing, and the last three
    b.check([90, 90], 4, 4, new=False, in_place_mass=True)  # mass packed where it is
    b = Batch(8, [40000], 1, 64, width=41111)
    b.check([20000], 4, 4, new=True, in_place_mass=True)


def test_evict_leaves_a_bad_length_and_block_alone():
    import torch
    b = Batch(11, [64, 48, 80], 1, 64)
    lens = b.lens.copy()
    lens[1] = 16 * b.tables.shape[1] + 1
    tables = b.tables.copy()
    tables[2, 1] = b.nb + 5
    dk, dv = H.dev_bf16(b.k), H.dev_bf16(b.v)
    kept, new_lens, _ = pa().pa_evict(dev_f32(b.mass), dk, dv, H.dev_i32(tables), H.dev_i32(lens),
                                      H.dev_i32([20, 20, 20]), new_tables=H.dev_i32(b.fresh))
    err = pa().pa_get_device_error()
    assert err == pa().PA_DEV_ERR_CONTEXT | pa().PA_DEV_ERR_BLOCK_ID
    assert new_lens.tolist() == [20, 0, 20]
    want = b.choices([20, 20, 20], 0, 0, 80)
    k = drafting.compact(b.k, b.tables[0], 0, want[0], b.fresh[0])
    moved = [(i, int(t)) for i, t in enumerate(want[2][0])]
    for i, t in moved:
        if not 16 <= t < 32:  # those of the bad block stay
            k[b.fresh[2, i // 16], 0, i % 16] = b.k[b.tables[2, t // 16], 0, t % 16]
    assert np.array_equal(H.host_bits(dk), k)


@pytest.mark.parametrize("new", [True, False], ids=["fresh", "in_place"])
@pytest.mark.parametrize("heads", [1, 3], ids=["shared", "per_head"])
def test_compact_accepted_branches(new, heads):
    # base: the cached tokens; kept: the accepted drafted tokens, packed behind them
    b = Batch(13, [130, 17, 64, 5], 3, 128)
    base = np.array([100, 10, 64, 0], np.int32)
    counts = np.array([7, 3, 0, 5], np.int32)
    kept = np.full((4, heads, 9), -1, np.int32)
    for s in range(4):
        for g in range(heads):
            room = int(b.lens[s] - base[s])
            kept[s, g, :counts[s]] = np.sort(b.rng.permutation(room)[:counts[s]])
    dk, dv = H.dev_bf16(b.k), H.dev_bf16(b.v)
    pa().pa_compact_tokens(dk, dv, H.dev_i32(b.tables), H.dev_i32(kept), H.dev_i32(counts),
                           base=H.dev_i32(base), new_tables=H.dev_i32(b.fresh) if new else None)
    k, v = b.k, b.v
    for s in range(4):
        lists = [kept[s, g % heads, :counts[s]] for g in range(3)]
        table = b.fresh[s] if new else None
        k = drafting.compact(k, b.tables[s], int(base[s]), lists, table)
        v = drafting.compact(v, b.tables[s], int(base[s]), lists, table)
    assert np.array_equal(H.host_bits(dk), k) and np.array_equal(H.host_bits(dv), v)
    assert pa().pa_get_device_error() == 0


def test_compact_refuses_rows_outside_the_table():
    b = Batch(17, [40], 1, 64)
    w = b.tables.shape[1]
    dk, dv = H.dev_bf16(b.k), H.dev_bf16(b.v)
    kept = np.array([[[0, 3, 16 * w, 2 ** 31 - 1]]], np.int32)
    pa().pa_compact_tokens(dk, dv, H.dev_i32(b.tables), H.dev_i32(kept), H.dev_i32([9]),
                           base=H.dev_i32([1]))
    assert pa().pa_get_device_error() & pa().PA_DEV_ERR_CONTEXT
    want = drafting.compact(b.k, b.tables[0], 1, [[0, 3]])
    assert np.array_equal(H.host_bits(dk), want)


def test_long_moves_in_place():
    # many chunks of rows per CTA: every source lies just ahead of its target
    b = Batch(19, [6000, 3000], 2, 64)
    b.mass[:] = -np.arange(6000, dtype=np.float32)[::-1]  # the last ones are the heaviest
    b.check([5900, 2000], 0, 0, new=False)
    b.mass[:] = b.rng.random(b.mass.shape)
    b.check([5000, 2999], 1, 1, new=False)


def test_evict_in_a_graph_and_on_a_stream():
    import torch
    b = Batch(23, [900, 1200], 2, 128)
    args = lambda: (dev_f32(b.mass), H.dev_bf16(b.k), H.dev_bf16(b.v),  # noqa: E731
                    H.dev_i32(b.tables), H.dev_i32(b.lens), H.dev_i32([300, 301]))
    new = H.dev_i32(b.fresh)
    a = args()
    want = pa().pa_evict(*a, sink=4, recent=16, new_tables=new, max_keep=400)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = args()
    torch.cuda.synchronize()
    got = pa().pa_evict(*c, sink=4, recent=16, new_tables=new, max_keep=400, stream=side)
    g = torch.cuda.CUDAGraph()
    e = args()
    with torch.cuda.graph(g):
        again = pa().pa_evict(*e, sink=4, recent=16, new_tables=new, max_keep=400)
    g.replay()
    torch.cuda.synchronize()
    for x in (got, again):
        assert torch.equal(x[1], want[1])
        for s, n in enumerate(want[1].tolist()):
            assert torch.equal(x[0][s, :, :n], want[0][s, :, :n])
            assert torch.equal(x[2][s, :, :n], want[2][s, :, :n])
    for x, y in ((c, a), (e, a)):
        assert torch.equal(x[1].view(torch.int16), y[1].view(torch.int16))
        assert torch.equal(x[2].view(torch.int16), y[2].view(torch.int16))


@pytest.mark.parametrize("length,rows", [(500, 1), (500, 41), (6000, 1), (6000, 41), (36000, 1),
                                         (133000, 1)])
def test_every_kept_weight_keeps_its_value(length, rows):
    # bit by bit, in rows that hold NaN of any payload among infinities, denormals and
    # zeros: -0 becomes 0, a NaN the canonical one
    b = Batch(29, [length] + [1] * (rows - 1), 2, 64)
    pool = np.array([np.inf, -np.inf, 1e-45, 3e-45, -1e-45, 0.0, -0.0, -2.5, 7.0, 1e38], np.float32)
    m = b.rng.choice(pool, (2, length))
    nan = (b.rng.integers(1, 1 << 23, (2, length)) | 0x7F800000).astype(np.uint32)
    nan |= b.rng.integers(0, 2, (2, length)).astype(np.uint32) << 31
    b.mass[0] = np.where(b.rng.random((2, length)) < 0.3, nan.view(np.float32), m)
    for budget in (length // 4, length - 5):  # the second keeps some NaN
        (kept, lens, mass), _, _ = b.run([budget] * rows, 3, 11, True)
        want = b.choices([budget] * rows, 3, 11, kept.shape[2])
        got = mass.cpu().numpy()
        for g in range(2):
            n = len(want[0][g])
            assert lens[0] == n
            assert np.array_equal(kept[0, g, :n].cpu().numpy(), want[0][g])
            w = b.mass[0, g][want[0][g]]
            bits = np.where(np.isnan(w), np.uint32(0x7FC00000),
                            (np.where(np.isnan(w), 0, w) + np.float32(0)).view(np.uint32))
            assert np.array_equal(got[0, g, :n].view(np.uint32), bits)
        assert np.isnan(b.mass[0, 0][want[0][0]]).any()
    assert pa().pa_get_device_error() == 0
