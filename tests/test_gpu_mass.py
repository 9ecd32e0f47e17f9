"""Accumulated attention weight (``pa_attention_mass``) against float64.

Tolerance of a token's sum W of weights: a weight is off by its score's error
(sums of D products in fp32: below 1e-5 for N(0, 1) inputs), by the rounding of
lse to its own 2^-24 (1e-6 of the weight at |lse| = 16) and of the exponential
(2^-22), and the sum of at most 1000 rows by 1000 * 2^-24: 8e-5 W together, and
the last addition by 2^-24 of the result."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
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
    def __init__(self, seed, lens, n, hq, hkv, d, width=None):
        rng = np.random.default_rng(seed)
        self.lay = synth.build_layout("mass", seed, lens, num_q_heads=hq, num_kv_heads=hkv,
                                      head_dim=d, q_lens=n, is_prefill=np.ones(len(lens), bool),
                                      extra_table_cols=1)
        self.h = synth.fill_host(self.lay, poison=True)
        self.n, self.lens = np.asarray(n), np.asarray(lens)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.kp, self.vp = oracle.reshape_and_cache(self.h["k_pool"], self.h["v_pool"],
                                                    self.h["key"], self.h["value"],
                                                    self.lay.slot_mapping())
        _, lse = oracle.chunked_prefill(self.h["q"], self.cu, self.kp, self.vp,
                                        self.lay.block_tables, self.lay.context_lens,
                                        self.lay.scale)
        self.lse = lse.astype(np.float32)
        self.width = width or 16 * self.lay.block_tables.shape[1]
        self.before = rng.random((len(lens), hkv, self.width)).astype(np.float32) * 1e-2

    def device(self, cu=True):
        return dict(q=H.dev_bf16(self.h["q"]), lse=dev_f32(self.lse),
                    cu_q_lens=H.dev_i32(self.cu) if cu else None, max_q_len=int(self.n.max()),
                    k_pool=H.dev_bf16(self.kp), block_tables=H.dev_i32(self.lay.block_tables),
                    context_lens=H.dev_i32(self.lay.context_lens), scale=self.lay.scale)

    def want(self, lse=None):
        return drafting.attention_mass(self.h["q"], self.lse if lse is None else lse, self.cu,
                                       self.kp, self.lay.block_tables, self.lay.context_lens,
                                       self.lay.scale)

    def check(self, got, before=None, want=None, skip=()):
        """``before``: what was there (None: zeros); past a length it is unchanged."""
        got = got.cpu().numpy()
        want = self.want() if want is None else want
        for s, w in enumerate(want):
            if s in skip:
                continue
            L = int(self.lens[s])
            b = np.zeros_like(got[s]) if before is None else before[s]
            tot = b[:, :L].astype(np.float64) + w
            err = np.abs(got[s, :, :L] - tot)
            tol = 8e-5 * w + 2.0 ** -24 * np.abs(tot) + 1e-30
            assert np.all(err <= tol), (s, np.argwhere(err > tol)[:3], (err / np.maximum(w, 1e-30)).max())
            assert np.array_equal(got[s, :, L:], b[:, L:])


CASES = [  # lens, queries, hq, hkv, d
    ([1], [1], 1, 1, 64),
    ([1, 2, 128, 129], [1, 1, 1, 1], 16, 1, 128),
    ([700, 31, 2000], [1, 1, 1], 64, 8, 128),
    ([300, 17], [17, 17], 10, 2, 128),              # group 5, the whole context is new
    ([513, 64, 1000], [33, 64, 40], 16, 2, 64),     # several column tiles
    ([400], [400], 8, 1, 128),                      # a whole prompt, causal
    ([129, 640], [128, 130], 4, 4, 64),             # groups of one
    ([1500], [25], 32, 2, 128),                     # group 16
    ([257, 50], [200, 0], 7, 1, 128),               # group 7; a sequence with no rows
    ([60] * 40, [3] * 40, 8, 8, 64),
]


@pytest.mark.parametrize("lens,n,hq,hkv,d", CASES)
def test_mass_matches_the_definition(lens, n, hq, hkv, d):
    b = Batch(len(lens) * 31 + sum(n), lens, n, hq, hkv, d)
    dev = b.device()
    b.check(pa().pa_attention_mass(**dev))
    # added to what was there, into another tensor and in place
    before = dev_f32(b.before)
    out = before.clone()
    out += 1
    got = pa().pa_attention_mass(**dev, mass_in=before, mass=out)
    assert got is out
    tail = b.before.copy()
    for s, L in enumerate(lens):
        tail[s, :, L:] += 1
    b.check(got, tail)
    again = pa().pa_attention_mass(**dev, mass_in=before, mass=before)
    for s, L in enumerate(lens):
        assert np.array_equal(again.cpu().numpy()[s, :, :L], got.cpu().numpy()[s, :, :L])
    assert pa().pa_get_device_error() == 0


def test_mass_random_sizes():
    rng = np.random.default_rng(8)
    for _ in range(10):
        hkv, g = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 3, 4, 6, 8, 16]))
        s = int(rng.integers(1, 6))
        n = rng.integers(1, 60, s)
        lens = n + rng.integers(0, 700, s)
        b = Batch(int(rng.integers(1 << 30)), lens, n, hkv * g, hkv, int(rng.choice([64, 128])))
        b.check(pa().pa_attention_mass(**b.device()))
    assert pa().pa_get_device_error() == 0


def test_decode_form_and_its_lse():
    # a decode step through the library: its own log-sum-exp, one row a sequence;
    # the weights of a row's G heads sum to G over the context
    b = Batch(21, [900, 5, 333, 64], [1, 1, 1, 1], 16, 2, 128)
    dev = b.device(cu=False)
    _, lse = pa().pa_decode(dev["q"], dev["k_pool"], H.dev_bf16(b.vp), dev["block_tables"],
                            dev["context_lens"], b.lay.scale, want_lse=True)
    dev["lse"] = lse
    got = pa().pa_attention_mass(**dev)
    b.check(got, want=b.want(lse.cpu().numpy()))
    assert float((got.sum(2) - 8).abs().max()) < 1e-2
    both = pa().pa_attention_mass(**{**dev, "cu_q_lens": H.dev_i32(b.cu)})
    assert bool((both == got).all())


def test_empty_rows_and_contexts():
    b = Batch(23, [90, 40], [4, 2], 4, 2, 64)
    b.lse[1] = -np.inf      # a row that saw nothing adds nothing
    b.lse[5, 2] = -np.inf
    b.check(pa().pa_attention_mass(**b.device()))
    # an empty context in a decode batch: its row of mass stays
    import torch
    d = Batch(25, [33, 20, 50], [1, 1, 1], 4, 4, 64)
    dev = d.device(cu=False)
    dev["context_lens"] = H.dev_i32([33, 0, 50])
    out = torch.full((3, 4, d.width), 7.0, device="cuda")
    pa().pa_attention_mass(**dev, mass=out)
    assert bool((out[1] == 7).all()) and bool((out[0, :, 33:] == 7).all())
    keep = np.full((3, 4, d.width), 7.0, np.float32)
    keep[0, :, :33] = 0
    keep[2, :, :50] = 0
    d.check(out, keep, skip=(1,))
    assert pa().pa_get_device_error() == 0


def test_bad_values_are_left_out():
    import torch
    b = Batch(27, [150, 140, 333], [6, 5, 7], 8, 2, 128, width=340)
    dev = b.device()
    lens = b.lay.context_lens.copy()
    lens[1] = 4
    tables = b.lay.block_tables.copy()
    tables[2, 3] = -1
    dev["context_lens"], dev["block_tables"] = H.dev_i32(lens), H.dev_i32(tables)
    out = dev_f32(b.before)
    pa().pa_attention_mass(**dev, mass_in=out, mass=out)
    assert pa().pa_get_device_error() == pa().PA_DEV_ERR_CONTEXT | pa().PA_DEV_ERR_BLOCK_ID
    got = out.cpu().numpy()
    assert np.array_equal(got[1], b.before[1])
    want = b.want()
    want[2][:, 48:64] = 0
    b.check(out, b.before, want=want, skip=(1,))
    # a context longer than the rows of mass
    out = torch.zeros((3, 2, 200), device="cuda")
    pa().pa_attention_mass(**{**b.device()}, mass=out)
    assert pa().pa_get_device_error() == pa().PA_DEV_ERR_CONTEXT
    assert not bool(out[2].any()) and bool(out[0].any())


def test_strided_q_and_scales():
    import torch
    b = Batch(29, [333, 64], [9, 20], 8, 2, 64)
    dev = b.device()
    wide = torch.zeros((29, 13, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = dev["q"]
    dev["q"] = wide[:, 3:11]
    for scale in (b.lay.scale, -0.1, 0.0):
        dev["scale"] = scale
        want = drafting.attention_mass(b.h["q"], b.lse, b.cu, b.kp, b.lay.block_tables,
                                       b.lay.context_lens, scale)
        b.check(pa().pa_attention_mass(**dev), want=want)


def test_mass_in_graphs_on_two_streams():
    import torch
    b1, b2 = Batch(31, [900, 50], [12, 9], 16, 2, 128), Batch(32, [77, 2000], [1, 1], 8, 8, 64)
    devs = [b.device() for b in (b1, b2)]
    want = [pa().pa_attention_mass(**d) for d in devs]
    graphs = []
    for d in devs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = pa().pa_attention_mass(**d)
        graphs.append((g, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (g, out) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (g, out), w in zip(graphs, want):
        assert torch.equal(out, w)
    got = pa().pa_attention_mass(**devs[0], stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(got, want[0])


def test_bad_blocks_among_sequences_without_rows():
    # units whose K is passed over (no rows) let the copies run far ahead of the tiles
    # still in work: each tile's pages have to stay its own
    lens = [640, 2100, 70, 1900, 513, 129, 2048, 33] * 6
    n = [1, 0, 3, 0, 1, 0, 0, 2] * 6
    for d in (64, 128):
        b = Batch(41 + d, lens, n, 4, 1, d)
        dev = b.device()
        tables = b.lay.block_tables.copy()
        want = b.want()
        for s, L in enumerate(lens):
            if n[s] and s % 3:
                k = (5 * s) % (-(-L // 16))
                tables[s, k] = -1
                want[s][:, 16 * k:16 * k + 16] = 0
        dev["block_tables"] = H.dev_i32(tables)
        for _ in range(5):
            got = pa().pa_attention_mass(**dev)
            b.check(got, want=want)
        assert pa().pa_get_device_error() == pa().PA_DEV_ERR_BLOCK_ID


def test_a_row_that_saw_nothing_adds_nothing_whatever_it_scores():
    # lse -inf, and keys whose scores are infinite or NaN: one that only such a row sees,
    # and a whole sequence of such rows
    b = Batch(45, [90, 200, 64], [4, 3, 1], 8, 2, 64)
    b.lse[3] = -np.inf          # the last row of sequence 0
    b.lse[4:7] = -np.inf        # all of sequence 1
    kp = b.kp.copy()

    def fill(s, t, bits):
        kp[int(b.lay.block_tables[s, t // 16]), :, t % 16] = bits

    fill(0, 89, 0x7F80)         # +inf (times q of either sign)
    fill(1, 0, 0x7FC0)          # NaN
    fill(1, 77, 0x7F80)
    fill(1, 199, 0xFF80)
    dev = b.device()
    dev["k_pool"] = H.dev_bf16(kp)
    want = [np.array(w) for w in b.want()]
    got = pa().pa_attention_mass(**dev)
    assert bool((got[1] == 0).all()) and bool((got[0, :, 89] == 0).all())
    b.check(got, want=want)
    assert pa().pa_get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (4, 4, 64)])
def test_weights_of_an_accepted_branch(hq, hkv, d):
    # A tree whose rejected siblings score high: after packing, the accepted rows are a
    # chain, and their weights (with the lse the tree gave) sum to 1 a row and head.
    c = [130, 47]
    parent = [-1, 0, 0, 1, 2, 4, 4]
    branch = [0, 2, 4, 6]
    n, m = len(parent), len(branch)
    bits = []
    for i, p in enumerate(parent):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    b = Batch(47, [x + n for x in c], [n, n], hq, hkv, d)
    kp = b.kp.copy()
    for s, x in enumerate(c):
        for i in set(range(n)) - set(branch):  # aligned with every query of the group
            t = x + i
            for g in range(hkv):
                k = 8 * oracle.bf16_bits_to_f64(b.h["q"][s * n + 6, g * (hq // hkv)])
                kp[int(b.lay.block_tables[s, t // 16]), g, t % 16] = synth.f32_to_bf16_bits(
                    k.astype(np.float32))
    dk, dv = H.dev_bf16(kp), H.dev_bf16(b.vp)
    tables, scale = H.dev_i32(b.lay.block_tables), b.lay.scale
    q = H.dev_bf16(b.h["q"])
    _, lse = pa().pa_tree_attention(q, H.dev_i32(b.cu), n, H.dev_i64(np.array(bits * 2)[:, None]),
                                    dk, dv, tables, H.dev_i32([x + n for x in c]), scale,
                                    want_lse=True)
    pa().pa_compact_tokens(dk, dv, tables, H.dev_i32([[branch], [branch]]), H.dev_i32([m, m]),
                           base=H.dev_i32(c))
    import torch
    rows = torch.tensor([s * n + i for s in range(2) for i in branch], device="cuda")
    lens = [x + m for x in c]
    mass = pa().pa_attention_mass(q[rows], lse[rows], H.dev_i32([0, m, 2 * m]), m, dk, tables,
                                  H.dev_i32(lens), scale)
    want = drafting.attention_mass(b.h["q"][rows.cpu().numpy()], lse[rows].cpu().numpy(),
                                   [0, m, 2 * m], H.host_bits(dk), b.lay.block_tables,
                                   np.array(lens), scale)
    b.lens = np.array(lens)
    b.check(mass, want=want)
    # a row's weights sum to 1: each is off by its score's error and the lse's, 8e-5 together
    assert float((mass.sum(2) - m * (hq // hkv)).abs().max()) <= 1e-4 * m * (hq // hkv)
    assert pa().pa_get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (3, 3, 64)])
def test_weights_of_a_whole_prompt(hq, hkv, d):
    # every query of 4500 tokens; a token's two sums take up to 4500 * G / 2 terms each,
    # rounded after each: 2^-24 of W for every one, and 8e-5 W as above
    import torch
    n = 4500
    g = torch.Generator(device="cuda").manual_seed(d)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda",  # noqa: E731
                                      dtype=torch.bfloat16)
    blocks = -(-n // 16)
    q, k = rand(n, hq, d), rand(blocks, hkv, 16, d)
    table = torch.randperm(blocks, generator=g, device="cuda").int()[None].contiguous()
    scale = float(np.float32(d ** -0.5))
    rows = k[table[0].long()].transpose(1, 2).reshape(-1, hkv, d)[:n].double()
    later = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
    want = torch.zeros((hkv, n), dtype=torch.float64, device="cuda")
    lse = torch.empty((n, hq), device="cuda")
    for h in range(hq):
        x = (q[:, h].double() @ rows[:, h // (hq // hkv)].T * scale).masked_fill(later, -float("inf"))
        lse[:, h] = torch.logsumexp(x, -1).float()
        want[h // (hq // hkv)] += torch.exp(x - lse[:, h, None].double()).sum(0)
    got = pa().pa_attention_mass(q, lse, H.dev_i32([0, n]), n, k, table, H.dev_i32([n]), scale)
    err = (got[0, :, :n].double() - want).abs()
    assert bool((err <= (8e-5 + n * (hq // hkv) / 2 * 2.0 ** -24) * want).all())
    assert not bool(got[0, :, n:].any()) and pa().pa_get_device_error() == 0
