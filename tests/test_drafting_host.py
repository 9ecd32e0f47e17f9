"""Host side of the drafting and eviction calls, without a GPU: refusals of the
C ABI before anything is launched, the frequencies, and pins of the oracle."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import oracle
from oracle import drafting
from paged_kv_cache_454_b200 import _abi
import paged_kv_cache_454_b200 as pa

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: the calls fail first
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def pool(nb=8, hkv=2, bs=16, d=128):
    return _abi.PoolDesc(nb, hkv, bs, d)


def refuse(call, status, **kw):
    assert call(**kw) == status, kw


# ----------------------------------------------------------------------------
# Rotation
# ----------------------------------------------------------------------------
def test_rope_refusals(lib):
    def call(q=FAKE, qs=512, qo=FAKE, qos=512, hq=4, k=FAKE, ks=256, ko=FAKE, kos=256, hkv=2,
             d=128, pos=FAKE, f=FAKE, rot=128, layout=0, n=3):
        return lib.pa_rope(q, qs, qo, qos, hq, k, ks, ko, kos, hkv, d, pos, f, rot, layout, 1.0, n,
                           None)
    assert call(n=0) == _abi.PA_OK
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(pos=None),
               dict(f=None), dict(q=ODD), dict(ko=ODD), dict(qs=504), dict(qs=516), dict(kos=248),
               dict(hq=0), dict(hkv=-1), dict(n=-1), dict(layout=2), dict(rot=-16),
               dict(pos=ctypes.c_void_p(0x10004))):
        refuse(call, _abi.PA_ERR_ARG, **kw)
    for kw in (dict(d=96), dict(rot=24), dict(hq=5000)):
        refuse(call, _abi.PA_ERR_UNSUPPORTED, **kw)
    refuse(call, _abi.PA_ERR_SHAPE, rot=144)


def test_rope_and_cache_refusals(lib):
    def call(q=FAKE, qs=512, qo=FAKE, hq=4, k=FAKE, ks=256, v=FAKE, vs=256, qw=None, kw=None,
             eps=1e-6, pos=FAKE, f=FAKE, rot=64, layout=1, kp=FAKE, vp=FAKE, desc=None, slots=FAKE,
             n=3):
        return lib.pa_rope_and_cache(q, qs, qo, 512, hq, k, ks, v, vs, qw, kw, eps, pos, f, rot,
                                     layout, 1.0, kp, vp, desc or pool(), slots, n, None)
    assert call(n=0) == _abi.PA_OK
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(kp=None), dict(vp=ODD),
               dict(slots=None), dict(qw=ODD), dict(vs=128), dict(ks=260), dict(n=-2), dict(hq=0),
               dict(qw=FAKE, eps=-1.0), dict(kw=FAKE, eps=math.nan), dict(layout=-1)):
        refuse(call, _abi.PA_ERR_ARG, **kw)
    refuse(call, _abi.PA_ERR_SHAPE, hq=3)
    refuse(call, _abi.PA_ERR_UNSUPPORTED, desc=pool(bs=32))
    refuse(call, _abi.PA_ERR_UNSUPPORTED, desc=pool(d=80))
    refuse(call, _abi.PA_ERR_UNSUPPORTED, rot=40)


def test_tree_refusals(lib):
    big = 1 << 40

    def call(q=FAKE, qs=512, cu=FAKE, total=6, max_n=5, mask=FAKE, words=1, kp=FAKE, vp=FAKE,
             desc=None, tables=FAKE, blocks=4, lens=FAKE, seqs=2, hq=4, out=FAKE, lse=None,
             ws=FAKE, ws_bytes=big):
        return lib.pa_tree_attention(q, qs, cu, total, max_n, mask, words, kp, vp, desc or pool(),
                                     tables, blocks, lens, seqs, hq, 1.0, out, lse, ws, ws_bytes,
                                     None)
    assert call(seqs=0) == _abi.PA_OK and call(total=0) == _abi.PA_OK
    for kw in (dict(q=None), dict(cu=None), dict(mask=None), dict(kp=None), dict(vp=None),
               dict(tables=None), dict(lens=None), dict(out=None), dict(q=ODD), dict(out=ODD),
               dict(qs=256), dict(qs=516), dict(max_n=0), dict(words=0), dict(max_n=65),
               dict(seqs=-1), dict(total=-1), dict(blocks=0), dict(hq=0)):
        refuse(call, _abi.PA_ERR_ARG, **kw)
    refuse(call, _abi.PA_ERR_SHAPE, hq=3)
    for kw in (dict(hq=34, qs=34 * 128), dict(desc=pool(d=96)), dict(max_n=4097, words=65),
               dict(desc=pool(nb=1 << 27))):
        refuse(call, _abi.PA_ERR_UNSUPPORTED, **kw)
    need = lib.pa_tree_workspace_size(5, 4, pool())
    for kw in (dict(ws=None), dict(ws=ODD), dict(ws_bytes=need - 1), dict(ws_bytes=0)):
        refuse(call, _abi.PA_ERR_WORKSPACE, **kw)
    assert lib.pa_tree_workspace_size(200, 4, pool()) > need > 0
    for bad in ((0, 4, pool()), (5, 0, pool()), (5, 1, pool()), (5, 40, pool())):
        assert lib.pa_tree_workspace_size(*bad) == 0


def test_mass_refusals(lib):
    def call(q=FAKE, qs=512, lse=FAKE, cu=FAKE, total=6, max_n=5, kp=FAKE, desc=None, tables=FAKE,
             blocks=4, lens=FAKE, seqs=2, hq=4, m_in=None, m_out=FAKE, stride=64):
        return lib.pa_attention_mass(q, qs, lse, cu, total, max_n, kp, desc or pool(), tables,
                                     blocks, lens, seqs, hq, 1.0, m_in, m_out, stride, None)
    assert call(seqs=0) == _abi.PA_OK
    for kw in (dict(q=None), dict(lse=None), dict(kp=None), dict(tables=None), dict(lens=None),
               dict(m_out=None), dict(q=ODD), dict(kp=ODD), dict(qs=256), dict(qs=516),
               dict(max_n=0), dict(seqs=-1), dict(total=-1), dict(blocks=0), dict(hq=0),
               dict(stride=-1), dict(cu=None), dict(cu=None, total=2)):
        refuse(call, _abi.PA_ERR_ARG, **kw)
    refuse(call, _abi.PA_ERR_SHAPE, hq=3)
    for kw in (dict(hq=34, qs=34 * 128), dict(desc=pool(d=96)), dict(max_n=(1 << 20) + 1),
               dict(desc=pool(nb=1 << 27))):
        refuse(call, _abi.PA_ERR_UNSUPPORTED, **kw)


def test_evict_refusals(lib):
    def call(mass=FAKE, stride=64, kp=FAKE, vp=FAKE, desc=None, tables=FAKE, blocks=4, lens=FAKE,
             budgets=FAKE, sink=1, recent=1, new=None, new_blocks=0, kept=FAKE, kept_stride=8,
             new_lens=ctypes.c_void_p(0x20000), m_out=ctypes.c_void_p(0x30000), out_stride=8,
             seqs=2):
        return lib.pa_evict(mass, stride, kp, vp, desc or pool(), tables, blocks, lens, budgets,
                            sink, recent, new, new_blocks, kept, kept_stride, new_lens, m_out,
                            out_stride, seqs, None)
    assert call(seqs=0) == _abi.PA_OK
    for kw in (dict(mass=None), dict(kp=None), dict(vp=ODD), dict(tables=None), dict(lens=None),
               dict(budgets=None), dict(kept=None), dict(new_lens=None), dict(m_out=None),
               dict(new_lens=FAKE), dict(sink=-1), dict(recent=-1), dict(seqs=-1), dict(blocks=0),
               dict(stride=-1), dict(kept_stride=-1), dict(new=ctypes.c_void_p(0x40000)),
               dict(new=FAKE, new_blocks=4), dict(m_out=FAKE)):
        refuse(call, _abi.PA_ERR_ARG, **kw)
    refuse(call, _abi.PA_ERR_UNSUPPORTED, desc=pool(bs=8))
    refuse(call, _abi.PA_ERR_UNSUPPORTED, blocks=(1 << 26) + 1)


def test_compact_refusals(lib):
    def call(kp=FAKE, vp=FAKE, desc=None, tables=FAKE, blocks=4, new=None, new_blocks=0, base=None,
             kept=FAKE, heads=2, stride=8, counts=FAKE, seqs=2):
        return lib.pa_compact_tokens(kp, vp, desc or pool(), tables, blocks, new, new_blocks, base,
                                     kept, heads, stride, counts, seqs, None)
    assert call(seqs=0) == _abi.PA_OK and call(stride=0) == _abi.PA_OK
    for kw in (dict(kp=None), dict(vp=None), dict(kp=ODD), dict(tables=None), dict(kept=None),
               dict(counts=None), dict(blocks=0), dict(seqs=-1), dict(stride=-1),
               dict(new=ctypes.c_void_p(0x40000)), dict(new=FAKE, new_blocks=4)):
        refuse(call, _abi.PA_ERR_ARG, **kw)
    refuse(call, _abi.PA_ERR_SHAPE, heads=3)
    refuse(call, _abi.PA_ERR_UNSUPPORTED, desc=pool(d=32))


def test_evict_refuses_a_choice_without_room(lib):
    # (the choice alone would end with its lengths still on their way: the calls after
    # it rely on the move's end)
    other = [ctypes.c_void_p(0x20000 + 0x10000 * i) for i in range(2)]
    for new, blocks in ((None, 0), (ctypes.c_void_p(0x50000), 4)):
        assert lib.pa_evict(FAKE, 64, FAKE, FAKE, pool(), FAKE, 4, FAKE, FAKE, 0, 0, new, blocks,
                            FAKE, 0, other[0], other[1], 8, 2, None) == _abi.PA_ERR_ARG


def test_compact_refuses_lists_past_its_row_numbers(lib):
    # (a turn of the move past 2^30 rows could leave an int)
    for new, blocks in ((None, 0), (ctypes.c_void_p(0x40000), 4)):
        assert lib.pa_compact_tokens(FAKE, FAKE, pool(), FAKE, 4, new, blocks, None, FAKE, 2,
                                     (1 << 30) + 1, FAKE, 2, None) == _abi.PA_ERR_UNSUPPORTED


def test_frequencies():
    f, factor = pa.pa_rope_frequencies(8)
    assert factor == 1.0 and np.allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-15)
    f4, factor = pa.pa_rope_frequencies(8, scaling=pa.PA_ROPE_SCALE_LINEAR, scale=4.0)
    assert factor == 1.0 and np.allclose(f4, f / 4, rtol=1e-15)
    # the larger base keeps the fastest pair and stretches the slowest by the scale
    fb, factor = pa.pa_rope_frequencies(64, scaling=pa.PA_ROPE_SCALE_BASE, scale=4.0)
    f64, _ = pa.pa_rope_frequencies(64)
    assert factor == 1.0 and fb[0] == 1.0 and math.isclose(fb[-1], f64[-1] / 4, rel_tol=1e-12)
    # the ramp: pairs of at least 32 turns kept, of at most 1 turn stretched
    fr, factor = pa.pa_rope_frequencies(128, scaling=pa.PA_ROPE_SCALE_RAMP, scale=16.0,
                                        original_max_position=8192)
    f0, _ = pa.pa_rope_frequencies(128)
    turns = 8192 * f0 / (2 * math.pi)
    assert math.isclose(factor, 0.1 * math.log(16) + 1, rel_tol=1e-15)
    assert np.allclose(fr[turns >= 32], f0[turns >= 32], rtol=1e-15)
    assert np.allclose(fr[turns <= 1], f0[turns <= 1] / 16, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(fr[mid] < f0[mid]) and np.all(fr[mid] > f0[mid] / 16)
    i = int(np.argmin(np.abs(turns - 16.5)))  # by hand for one pair
    w = (turns[i] - 1) / 31
    assert math.isclose(fr[i], w * f0[i] + (1 - w) * f0[i] / 16, rel_tol=1e-12)
    assert pa.pa_rope_frequencies(16, scaling=pa.PA_ROPE_SCALE_RAMP, scale=0.5,
                                  original_max_position=100)[1] == 1.0
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0),
                dict(rot_dim=8, scaling=9), dict(rot_dim=8, scaling=1, scale=0.0),
                dict(rot_dim=8, scaling=1, scale=math.nan),
                dict(rot_dim=2, scaling=2, scale=2.0), dict(rot_dim=8, scaling=3, scale=2.0),
                dict(rot_dim=8, scaling=3, scale=2.0, original_max_position=10, low_turns=5,
                     high_turns=5)):
        with pytest.raises(pa.PaError):
            pa.pa_rope_frequencies(**bad)


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pa.pa_rope(x, None, torch.zeros(2, dtype=torch.int64), torch.ones(32, dtype=torch.float64))


# ----------------------------------------------------------------------------
# Pins of the oracle
# ----------------------------------------------------------------------------
def test_oracle_rotation_is_a_complex_product():
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((5, 2, 12)), np.array([0, 1, 7, 1000, -3]), np.array([1.0, 0.1, 0.3])
    turn = 1.5 * np.exp(1j * pos[:, None, None] * f)
    z = (x[..., 0:6:2] + 1j * x[..., 1:6:2]) * turn
    got = drafting.rope(x, pos, f, True, 1.5)
    assert np.allclose(got[..., 0:6:2], z.real) and np.allclose(got[..., 1:6:2], z.imag)
    z = (x[..., :3] + 1j * x[..., 3:6]) * turn
    got = drafting.rope(x, pos, f, False, 1.5)
    assert np.allclose(got[..., :3], z.real) and np.allclose(got[..., 3:6], z.imag)
    assert np.array_equal(got[..., 6:], x[..., 6:])
    # a product of rotated rows depends on the distance of their positions alone
    a, b = rng.standard_normal((1, 1, 12)), rng.standard_normal((1, 1, 12))
    at = lambda i, j: float((drafting.rope(a, [i], np.ones(6) * 0.37, True, 1.0) *  # noqa: E731
                             drafting.rope(b, [j], np.ones(6) * 0.37, True, 1.0)).sum())
    assert math.isclose(at(5, 2), at(105, 102), rel_tol=1e-9)


def test_oracle_norm():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(drafting.head_norm(x, [1.0, 2.0], 0.0), [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])
    assert np.array_equal(drafting.head_norm(np.zeros((1, 2)), [1.0, 1.0], 1e-6), [[0.0, 0.0]])


def _batch(seed, lens, n, hq, hkv, d):
    from workloads import synth
    lay = synth.build_layout("pin", seed, lens, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                             q_lens=n, is_prefill=np.ones(len(lens), bool))
    h = synth.fill_host(lay, poison=False)
    return lay, h, np.concatenate([[0], np.cumsum(n)])


def test_oracle_tree_of_a_chain_is_causal_prefill():
    n = [3, 1, 5]
    lay, h, cu = _batch(3, [20, 1, 5], n, 4, 2, 64)
    chain = np.array([[(1 << (i + 1)) - 1] for m in n for i in range(m)], np.int64)
    got = drafting.tree_attention(h["q"], cu, chain, h["k_pool"], h["v_pool"], lay.block_tables,
                                  lay.context_lens, lay.scale)
    want = oracle.chunked_prefill(h["q"], cu, h["k_pool"], h["v_pool"], lay.block_tables,
                                  lay.context_lens, lay.scale)
    assert np.allclose(got[0], want[0], rtol=1e-12) and np.allclose(got[1], want[1], rtol=1e-12)
    # the weights of the same rows, accumulated, sum to the rows' count per head
    mass = drafting.attention_mass(h["q"], want[1], cu, h["k_pool"], lay.block_tables,
                                   lay.context_lens, lay.scale)
    for s, m in enumerate(mass):
        assert m.shape == (2, lay.context_lens[s]) and np.allclose(m.sum(1), 2 * n[s])
    # a token nobody sees changes nothing; a row that sees nothing is empty
    none = np.zeros_like(chain)
    out, lse = drafting.tree_attention(h["q"], cu, none, h["k_pool"], h["v_pool"],
                                       lay.block_tables, lay.context_lens, lay.scale)
    assert np.all(lse[3:4] == -np.inf) and not out[3:4].any()  # one token, nothing cached
    assert np.all(np.isfinite(lse[:3]))


def test_oracle_tree_branch_equals_its_own_sequence():
    # the leaf of a branch sees what it would see if its branch were all there is
    lay, h, cu = _batch(5, [24], [6], 2, 1, 64)
    parent = [-1, 0, 0, 1, 2, 3]
    rows = []
    for i, p in enumerate(parent):
        rows.append((1 << i) | (rows[p] if p >= 0 else 0))
    mask = np.array(rows, np.int64)[:, None]
    out, lse = drafting.tree_attention(h["q"], cu, mask, h["k_pool"], h["v_pool"],
                                       lay.block_tables, lay.context_lens, lay.scale)
    K, V = oracle.gather_kv(h["k_pool"], h["v_pool"], lay.block_tables[0], 24)
    branch = list(range(18)) + [18, 20, 22]  # tokens 0, 2 and 4 of the tree
    q = oracle.bf16_bits_to_f64(h["q"])
    for head in range(2):
        o, e = oracle.attend(q[4, head], oracle.bf16_bits_to_f64(K[0])[branch],
                             oracle.bf16_bits_to_f64(V[0])[branch], lay.scale)
        assert np.allclose(o, out[4, head], rtol=1e-12) and math.isclose(e, lse[4, head], rel_tol=1e-12)


def test_oracle_evict_by_hand():
    m = np.array([0.1, 9.0, 2.0, 2.0, np.nan, 2.0, 0.0, 5.0])
    choose = lambda *a: drafting.evict_choice(m, *a).tolist()  # noqa: E731
    assert choose(8, 4, 0, 0) == [1, 2, 3, 7]            # the tie goes to the lowest index
    assert choose(8, 4, 1, 1) == [0, 1, 2, 7]
    assert choose(8, 4, 3, 3) == [0, 1, 2, 7]            # the sinks come before the recent ones
    assert choose(8, 2, 5, 5) == [0, 1]
    assert choose(8, 8, 0, 0) == list(range(8)) and choose(3, 100, 1, 1) == [0, 1, 2]
    assert choose(8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]   # NaN goes first
    low = np.array([np.nan, -np.inf, -1.0])
    assert drafting.evict_choice(low, 3, 2, 0, 0).tolist() == [1, 2]
    assert choose(8, 0, 2, 2) == [] and choose(0, 5, 1, 1) == []


def test_oracle_compact():
    pool_ = np.arange(3 * 2 * 16 * 1).reshape(3, 2, 16, 1)
    got = drafting.compact(pool_, [2, 0], 4, [[0, 3, 15], [1, 2, 3]])
    assert got[2, 0, 4:7, 0].tolist() == [pool_[2, 0, 4, 0], pool_[2, 0, 7, 0], pool_[0, 0, 3, 0]]
    assert got[2, 1, 4:7, 0].tolist() == pool_[2, 1, 5:8, 0].tolist()
    assert np.array_equal(got[0], pool_[0]) and np.array_equal(got[1], pool_[1])
    far = drafting.compact(pool_, [2, 0], 0, [[17], [0]], new_table=[1])
    assert far[1, 0, 0, 0] == pool_[0, 0, 1, 0] and far[1, 1, 0, 0] == pool_[2, 1, 0, 0]


def test_mass_flags_are_checked(lib):
    def call(flags, seqs=0):
        return lib.pa_attention_mass_ex(FAKE, 512, FAKE, FAKE, 6, 5, FAKE, pool(), FAKE, 4, FAKE,
                                        seqs, 4, 1.0, None, FAKE, 64, flags, None)
    assert call(0) == call(_abi.PA_MASS_OWN_FROM_ZERO) == _abi.PA_OK
    assert call(2) == call(1 << 31) == _abi.PA_ERR_ARG
