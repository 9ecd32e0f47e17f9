"""Attention of drafted trees (``pa_tree_attention``) against float64.

Tolerances.  lse: scores of N(0, 1) inputs are sums of D products in fp32
(relative error below D * 2^-24 of sum |q k| * scale, i.e. 1e-5 at |x| of a few
units), the exponentials and the sum add a few 2^-22: 2e-5 + 1e-6 |lse|.
out: its own rounding, 2^-8 |out|; a weight enters the product within 2^-15 of
itself and carries its score's error (1e-5): 5e-5 sum_t w_t |v_t|, taken as
5e-5 max|v| (weights sum to 1)."""
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


def tree_rows(n, rng, words):
    """Ancestor masks of a random tree of ``n`` tokens."""
    rows = np.zeros((n, words * 64), bool)
    for i in range(n):
        if i and rng.random() < 0.85:
            rows[i] = rows[int(rng.integers(max(0, i - 5), i))]
        rows[i, i] = True
    return np.packbits(rows, axis=1, bitorder="little").view(np.int64)


class Batch:
    def __init__(self, seed, lens, n, hq, hkv, d, words=None, mask=None):
        rng = np.random.default_rng(seed)
        self.lay = synth.build_layout("tree", seed, lens, num_q_heads=hq, num_kv_heads=hkv,
                                      head_dim=d, q_lens=n, is_prefill=np.ones(len(lens), bool),
                                      extra_table_cols=1)
        self.h = synth.fill_host(self.lay, poison=True)
        self.n = np.asarray(n)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        words = words or max(1, -(-int(self.n.max()) // 64))
        if mask is None:
            mask = np.concatenate([tree_rows(int(x), rng, words) for x in self.n])
        self.mask = mask
        # the cache write of the drafted tokens
        from oracle import reshape_and_cache
        self.kp, self.vp = reshape_and_cache(self.h["k_pool"], self.h["v_pool"], self.h["key"],
                                             self.h["value"], self.lay.slot_mapping())

    def device(self):
        return dict(q=H.dev_bf16(self.h["q"]), cu_q_lens=H.dev_i32(self.cu),
                    max_q_len=int(self.n.max()), tree_mask=H.dev_i64(self.mask),
                    k_pool=H.dev_bf16(self.kp), v_pool=H.dev_bf16(self.vp),
                    block_tables=H.dev_i32(self.lay.block_tables),
                    context_lens=H.dev_i32(self.lay.context_lens), scale=self.lay.scale)

    def want(self):
        return drafting.tree_attention(self.h["q"], self.cu, self.mask, self.kp, self.vp,
                                       self.lay.block_tables, self.lay.context_lens,
                                       self.lay.scale)


def check(out, lse, want, vmax=6.0, rows=None):
    o, e = want
    got, gl = H.host_f64(out), lse.cpu().numpy().astype(np.float64)
    if rows is not None:
        o, e, got, gl = o[rows], e[rows], got[rows], gl[rows]
    assert np.array_equal(np.isneginf(gl), np.isneginf(e))
    live = np.isfinite(e)
    assert np.all(np.abs(gl[live] - e[live]) <= 2e-5 + 1e-6 * np.abs(e[live])), \
        np.abs(gl[live] - e[live]).max()
    bad = ~(np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + 5e-5 * vmax)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - o).max())


CASES = [  # lens, drafted tokens, hq, hkv, d
    ([1], [1], 1, 1, 64),
    ([1], [1], 16, 1, 128),
    ([17, 16, 15], [1, 16, 15], 4, 2, 128),
    ([128, 129, 127], [5, 1, 127], 2, 2, 64),
    ([300], [8], 64, 8, 128),                       # one row tile, split streams
    ([300, 260], [17, 30], 16, 2, 128),             # two row tiles
    ([513, 64, 1000], [33, 64, 48], 16, 2, 64),     # more than one pass
    ([2000, 5, 700], [16, 5, 3], 10, 2, 128),       # group 5
    ([1500], [25], 32, 32, 128),                    # groups of one
    ([130, 2049], [65, 100], 7, 1, 128),            # masks of two words, group 7
    ([4000], [2], 12, 1, 64),                       # group 12
    ([90] * 40, [7] * 40, 8, 8, 128),               # many short sequences
    ([257, 1024, 640], [129, 200, 256], 4, 4, 128),  # row tiles of 128 tokens
]


@pytest.mark.parametrize("lens,n,hq,hkv,d", CASES)
def test_tree_matches_the_definition(lens, n, hq, hkv, d):
    b = Batch(len(lens) * 100 + n[0], lens, n, hq, hkv, d)
    out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
    check(out, lse, b.want())
    assert pa().pa_get_device_error() == 0
    # lse is optional and does not change the output
    again, none = pa().pa_tree_attention(**b.device())
    assert none is None and np.array_equal(H.host_bits(again), H.host_bits(out))


def test_tree_random_sizes():
    rng = np.random.default_rng(12)
    for _ in range(12):
        hkv = int(rng.choice([1, 2, 4]))
        g = int(rng.choice([1, 2, 3, 4, 6, 8, 16]))
        s = int(rng.integers(1, 7))
        n = rng.integers(1, 40, s)
        lens = n + rng.integers(0, 900, s)
        b = Batch(int(rng.integers(1 << 30)), lens, n, hkv * g, hkv, int(rng.choice([64, 128])))
        out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
        check(out, lse, b.want())
    assert pa().pa_get_device_error() == 0


def test_a_chain_is_chunked_prefill():
    n = [40, 9, 100]
    chain = np.zeros((sum(n), 2), np.int64)
    bits = np.concatenate([np.tril(np.ones((x, 128), bool)) for x in n])
    chain = np.packbits(bits, axis=1, bitorder="little").view(np.int64)
    b = Batch(31, [700, 9, 2300], n, 16, 2, 128, mask=chain)
    dev = b.device()
    out, lse = pa().pa_tree_attention(**dev, want_lse=True)
    ref, ref_lse = pa().pa_chunked_prefill(dev["q"], dev["cu_q_lens"], max(n), dev["k_pool"],
                                           dev["v_pool"], dev["block_tables"],
                                           dev["context_lens"], b.lay.scale, want_lse=True,
                                           exact_weights=True)
    assert float((lse - ref_lse).abs().max()) <= 4e-5
    # both round the same value: they may differ by one step of bf16
    assert bool(((out.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 6e-4).all())


def test_rows_that_see_nothing():
    # no bit set, cached tokens or none; bits past the drafted tokens are ignored
    mask = np.zeros((9, 1), np.int64)
    mask[4] = 1 << 7     # past the sequence's 5 tokens
    mask[6] = 0b10       # only its sibling
    b = Batch(7, [5, 200], [5, 4], 8, 2, 128, mask=mask)
    out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
    check(out, lse, b.want())
    assert not H.host_bits(out)[:5].any() and bool((lse[:5] == -float("inf")).all())
    assert bool((lse[5:] > 0).all())


def test_empty_sequences_and_rows_behind_the_last():
    import torch
    b = Batch(9, [40, 33, 64], [3, 4, 5], 4, 4, 64)
    dev = b.device()
    # sequence 1 drafts nothing this step, and two padding rows follow the last one
    cu = np.array([0, 3, 3, 8], np.int32)
    dev["cu_q_lens"] = H.dev_i32(cu)
    rows = np.r_[0:3, 7:12, 0, 0]
    dev["q"] = dev["q"][torch.as_tensor(rows, device="cuda")].contiguous()
    dev["tree_mask"] = dev["tree_mask"][torch.as_tensor(rows, device="cuda")].contiguous()
    out = torch.full((10, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((10, 4), 5.0, device="cuda")
    pa().pa_tree_attention(**dev, out=out, lse=lse)
    o, e = b.want()
    check(out[:8], lse[:8], (o[rows[:8]], e[rows[:8]]))
    assert bool((out[8:] == 5).all()) and bool((lse[8:] == 5).all())
    assert pa().pa_get_device_error() == 0


def test_bad_values_are_left_out():
    import torch
    b = Batch(19, [150, 140, 333, 90], [6, 5, 7, 4], 8, 2, 128)
    dev = b.device()
    lens = b.lay.context_lens.copy()
    lens[1] = 3                       # fewer tokens than are drafted
    tables = b.lay.block_tables.copy()
    tables[2, 3] = b.lay.num_blocks   # its 16 tokens drop out
    tables[3, 0] = -5
    dev["context_lens"], dev["block_tables"] = H.dev_i32(lens), H.dev_i32(tables)
    out = torch.full((22, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((22, 8), 5.0, device="cuda")
    pa().pa_tree_attention(**dev, out=out, lse=lse)
    err = pa().pa_get_device_error()
    assert err == pa().PA_DEV_ERR_CONTEXT | pa().PA_DEV_ERR_BLOCK_ID
    assert bool((out[6:11] == 5).all()) and bool((lse[6:11] == 5).all())
    check(out, lse, b.want(), rows=np.r_[0:6])
    # the definition without the lost blocks' tokens
    from oracle import bf16_bits_to_f64, gather_kv, attend
    for s, r0, lost in ((2, 11, range(48, 64)), (3, 18, range(0, 16))):
        L, n = int(lens[s]), int(b.n[s])
        K, V = gather_kv(b.kp, b.vp, b.lay.block_tables[s], L)
        for i in range(n):
            see = [t for t in drafting._visible(b.mask[r0 + i], L - n, n) if t not in lost]
            for h in range(8):
                o, e = attend(bf16_bits_to_f64(b.h["q"][r0 + i, h]),
                              bf16_bits_to_f64(K[h // 4])[see], bf16_bits_to_f64(V[h // 4])[see],
                              b.lay.scale)
                assert abs(float(lse[r0 + i, h]) - e) <= 2e-5 + 1e-6 * abs(e)
                d = np.abs(H.host_f64(out[r0 + i, h]) - o)
                assert np.all(d <= 2.0 ** -8 * np.abs(o) + 3e-4)


@pytest.mark.parametrize("n,hq,hkv", [(20, 4, 4), (40, 16, 2)], ids=["split", "pair"])
def test_infinities_and_nan_of_unseen_drafted_tokens(n, hq, hkv):
    # the tokens of a rejected branch may hold anything: rows that do not see them
    # are as if they were not there; rows that see a bad V are NaN
    b = Batch(23, [260], [n], hq, hkv, 128)
    for g in range(hkv):
        t = 260 - n + 7
        blk, off = int(b.lay.block_tables[0, t // 16]), t % 16
        b.vp[blk, g, off, 3] = 0x7F80   # +inf
        t = 260 - n + 9
        blk, off = int(b.lay.block_tables[0, t // 16]), t % 16
        b.vp[blk, g, off, :] = 0x7FC0   # NaN
        b.kp[blk, g, off, :] = 0x7FC0
    out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
    sees7 = ((b.mask[:, 0] >> 7) & 1).astype(bool)
    sees9 = ((b.mask[:, 0] >> 9) & 1).astype(bool)
    clean = np.nonzero(~sees7 & ~sees9)[0]
    assert len(clean) and sees7.any() and sees9.any()
    with np.errstate(invalid="ignore"):
        want = b.want()
    check(out, lse, want, rows=clean)
    got = H.host_f64(out)
    assert np.isnan(got[sees7 | sees9]).all()
    only7 = np.nonzero(sees7 & ~sees9)[0]
    assert np.all(np.abs(lse.cpu().numpy()[only7] - want[1][only7]) <= 1e-4)


def test_extreme_scores():
    # scores of +-1e4 in one row: the maximum in use is raised again and again
    b = Batch(41, [700], [6], 4, 1, 128)
    b.h["q"] = synth.f32_to_bf16_bits(300 * np.random.default_rng(3).standard_normal(
        b.h["q"].shape).astype(np.float32))
    out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
    o, e = b.want()
    got, gl = H.host_f64(out), lse.cpu().numpy()
    # a score's fp32 error: D products of up to 300 * 4 * 4 * scale, 128 * 2^-24 of
    # the sum of their sizes (about 1e4): 0.02 at most; weights move by exp(0.02)
    assert np.all(np.abs(gl - e) <= 0.02)
    assert np.all(np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + 0.04 * 6)


def test_strided_q_negative_and_zero_scale():
    import torch
    b = Batch(43, [333, 64], [9, 20], 8, 2, 64)
    dev = b.device()
    t = int(b.cu[-1])
    wide = torch.zeros((t, 13, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = dev["q"]
    dev["q"] = wide[:, 3:11]
    for scale in (b.lay.scale, -0.2, 0.0):
        dev["scale"] = scale
        out, lse = pa().pa_tree_attention(**dev, want_lse=True)
        want = drafting.tree_attention(b.h["q"], b.cu, b.mask, b.kp, b.vp, b.lay.block_tables,
                                       b.lay.context_lens, scale)
        check(out, lse, want)


def test_graph_replay_and_two_streams():
    import torch
    b1, b2 = Batch(51, [900, 50], [12, 9], 16, 2, 128), Batch(52, [77, 2000], [30, 4], 8, 8, 64)
    d1, d2 = b1.device(), b2.device()
    want1, want2 = (pa().pa_tree_attention(**d) for d in (d1, d2))
    graphs = []
    for d in (d1, d2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, _ = pa().pa_tree_attention(**d)
        graphs.append((g, out))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (g, out) in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want1[0]) and torch.equal(graphs[1][1], want2[0])
    o1, _ = pa().pa_tree_attention(**d1, stream=s1)
    o2, _ = pa().pa_tree_attention(**d2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(o1, want1[0]) and torch.equal(o2, want2[0])


def test_bad_block_in_the_middle_of_two_row_tiles():
    # a lost block among the cached tokens: both row tiles leave its tokens out,
    # whatever lay in shared memory where its V would be
    b = Batch(61, [700, 900], [40, 33], 16, 2, 128)
    dev = b.device()
    tables = b.lay.block_tables.copy()
    tables[0, 10] = b.lay.num_blocks
    tables[1, 0] = -1
    dev["block_tables"] = H.dev_i32(tables)
    poison = H.dev_bf16(np.full_like(b.kp, synth.BF16_NAN))  # leaves NaN in the SMs
    pa().pa_tree_attention(**{**b.device(), "k_pool": poison, "v_pool": poison})
    out, lse = pa().pa_tree_attention(**dev, want_lse=True)
    assert pa().pa_get_device_error() == pa().PA_DEV_ERR_BLOCK_ID
    from oracle import bf16_bits_to_f64, gather_kv, attend
    for s, r0, lost in ((0, 0, range(160, 176)), (1, 40, range(0, 16))):
        L, n = int(b.lay.context_lens[s]), int(b.n[s])
        K, V = gather_kv(b.kp, b.vp, b.lay.block_tables[s], L)
        for i in (0, 5, n - 1):
            see = [t for t in drafting._visible(b.mask[r0 + i], L - n, n) if t not in lost]
            for h in range(16):
                o, e = attend(bf16_bits_to_f64(b.h["q"][r0 + i, h]),
                              bf16_bits_to_f64(K[h // 8])[see], bf16_bits_to_f64(V[h // 8])[see],
                              b.lay.scale)
                assert abs(float(lse[r0 + i, h]) - e) <= 2e-5 + 1e-6 * abs(e)
                d = np.abs(H.host_f64(out[r0 + i, h]) - o)
                assert np.all(d <= 2.0 ** -8 * np.abs(o) + 3e-4)


@pytest.mark.parametrize("n,hq,hkv,d", [(3, 4, 4, 128), (20, 16, 2, 64), (40, 16, 2, 128)])
def test_contexts_that_end_in_either_half_of_a_tile(n, hq, hkv, d):
    # the drafted tokens cross the halves of a tile, or the last half holds no key
    rng = np.random.default_rng(n)
    for ends in ([1, 63, 64, 65, 127, 128], [64] * 6, [1, 128] * 3, [20, 70, 64, 65, 33, 1]):
        lens = [128 * int(rng.integers(0, 5)) + e for e in ends * 2]
        lens = [L if L >= n else L + 128 for L in lens]
        b = Batch(sum(lens) + n, lens, [n] * len(lens), hq, hkv, d)
        out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
        check(out, lse, b.want())
    # one long item shared by all CTAs
    for L in (128 * 80 + 2, 128 * 80 + 64, 128 * 81):
        b = Batch(L, [L], [n], hq, hkv, d)
        out, lse = pa().pa_tree_attention(**b.device(), want_lse=True)
        check(out, lse, b.want())
    assert pa().pa_get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (32, 32, 128), (32, 8, 64)])
def test_results_are_the_same_every_time(hq, hkv, d):
    # items of one and of two row tiles, short and long ones, in turn on the same CTAs:
    # each stream of a CTA passes over what is the other's, and equal inputs give equal
    # bits however the copies arrive; two batches between which nothing waits
    import torch
    states = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        n = rng.integers(7, 64, 40)
        lens = np.maximum(n + 1, np.exp(rng.uniform(np.log(130), np.log(9000), 40)).astype(int))
        blocks = -(-lens // 16)
        nb = int(blocks.sum())
        tables = np.zeros((40, int(blocks.max())), np.int32)
        order, at = rng.permutation(nb), 0
        for s, k in enumerate(blocks):
            tables[s, :k] = order[at:at + k]
            at += k
        rand = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        total = int(n.sum())
        mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (total, 1), generator=g, device="cuda")
        states.append(dict(q=rand(total, hq, d), max_q_len=64, tree_mask=mask,
                           cu_q_lens=H.dev_i32(np.concatenate([[0], np.cumsum(n)])),
                           k_pool=rand(nb, hkv, 16, d), v_pool=rand(nb, hkv, 16, d),
                           block_tables=H.dev_i32(tables), context_lens=H.dev_i32(lens),
                           scale=d ** -0.5))
    first = [pa().pa_tree_attention(**s, want_lse=True) for s in states]
    for _ in range(60):
        got = [pa().pa_tree_attention(**s, want_lse=True) for s in states]
        for (o, e), (o0, e0) in zip(got, first):
            assert torch.equal(o, o0) and torch.equal(e, e0)
    assert pa().pa_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_runs_of_one_tile_units_between_pairs(d):
    # a dozen units of one key tile on every CTA, in which one of the two streams has
    # nothing to do, with items of two row tiles among them
    rng = np.random.default_rng(d)
    n = rng.choice([1, 4, 16, 20, 31], 220)
    lens = np.minimum(128, n + rng.integers(0, 128, 220))
    b = Batch(71 + d, lens, n, 64, 8, d)
    dev = b.device()
    first = pa().pa_tree_attention(**dev, want_lse=True)
    for _ in range(30):
        out, lse = pa().pa_tree_attention(**dev, want_lse=True)
        assert bool((out == first[0]).all()) and bool((lse == first[1]).all())
    assert pa().pa_get_device_error() == 0
    rows = int(b.cu[30])  # of the first thirty sequences
    want = drafting.tree_attention(b.h["q"][:rows], b.cu[:31], b.mask[:rows], b.kp, b.vp,
                                   b.lay.block_tables[:30], b.lay.context_lens[:30], b.lay.scale)
    check(*first, want, rows=np.arange(rows))


def test_outputs_are_rounded_both_ways_alike():
    # Outputs that differ from the 64-bit result rounded to bf16 lie one step above or
    # below it, by chance: of m of them, those towards zero exceed the others by 5 sqrt(m)
    # at most, and by what a systematic loss turns: the accumulator is cut off, by 2^-24
    # of itself on average, after each of 32 products (200 keys, 16 a time, two parts of
    # the weight), and a loss of 2^-19 crosses a border between steps of 2^-8 or more for
    # 2^-11 of the outputs at most.
    import torch
    s, n, hq, hkv, d, L = 16, 16, 64, 8, 128, 200
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda",  # noqa: E731
                                      dtype=torch.bfloat16)
    blocks = -(-L // 16)
    q, k, v = rand(s * n, hq, d), rand(s * blocks, hkv, 16, d), rand(s * blocks, hkv, 16, d)
    tables = torch.randperm(s * blocks, generator=g, device="cuda").int().view(s, blocks)
    out, _ = pa().pa_tree_attention(q, H.dev_i32(n * np.arange(s + 1)), n,
                                    torch.full((s * n, 1), -1, device="cuda"), k, v, tables,
                                    H.dev_i32([L] * s), d ** -0.5)
    rows = lambda pool: pool[tables.long()].transpose(2, 3).reshape(  # noqa: E731
        s, 16 * blocks, hkv, d)[:, :L].double()
    x = torch.einsum("sihgd,sthd->sihgt", q.double().view(s, n, hkv, hq // hkv, d), rows(k))
    p = torch.softmax(x * float(np.float32(d ** -0.5)), -1)
    want = torch.einsum("sihgt,sthd->sihgd", p, rows(v)).reshape(s * n, hq, d)
    nearest = want.to(torch.bfloat16)
    off = (out.double() - nearest.double()) * want.sign()
    low, high = int((off < 0).sum()), int((off > 0).sum())
    assert abs(low - high) <= 5 * (low + high) ** 0.5 + 2.0 ** -11 * want.numel(), (low, high)


@pytest.mark.parametrize("hq,hkv,d", [(16, 1, 64), (4, 4, 128)])
def test_the_most_drafted_tokens(hq, hkv, d):
    # 4096 of them (256 passes at group 16), any bits; some rows against 64 bits
    import torch
    n, c = 4096, 104
    L = n + c
    g = torch.Generator(device="cuda").manual_seed(hq)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda",  # noqa: E731
                                      dtype=torch.bfloat16)
    blocks = -(-L // 16)
    q, k, v = rand(n, hq, d), rand(blocks + 5, hkv, 16, d), rand(blocks + 5, hkv, 16, d)
    table = torch.randperm(blocks + 5, generator=g, device="cuda")[:blocks].int()[None]
    mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (n, 64), generator=g, device="cuda")
    out, lse = pa().pa_tree_attention(q, H.dev_i32([0, n]), n, mask, k, v, table.contiguous(),
                                      H.dev_i32([L]), d ** -0.5, want_lse=True)
    rows = torch.randperm(n, generator=g, device="cuda")[:96]
    rows[:2] = torch.tensor([0, n - 1], device="cuda")
    flat = lambda pool: pool[table[0].long()].transpose(1, 2).reshape(-1, hkv, d)[:L].double()  # noqa: E731
    x = torch.einsum("ihgd,thd->ihgt", q[rows].double().view(-1, hkv, hq // hkv, d), flat(k))
    j = torch.arange(n, device="cuda")
    see = ((mask[rows][:, j // 64] >> (j % 64)) & 1).bool()
    see = torch.cat([torch.ones((len(rows), c), dtype=torch.bool, device="cuda"), see], 1)
    x = (x * float(np.float32(d ** -0.5))).masked_fill(~see[:, None, None], -float("inf"))
    e = torch.logsumexp(x, -1)
    o = torch.einsum("ihgt,thd->ihgd", torch.exp(x - e[..., None]), flat(v))
    check(out[rows], lse[rows], (o.reshape(-1, hq, d).cpu().numpy(), e.reshape(-1, hq).cpu().numpy()))
    assert pa().pa_get_device_error() == 0
