"""The drafting and eviction calls together, as a serving step uses them, with the
block manager handing out the blocks and float64 following every step."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from oracle import bf16_bits_to_f64, drafting
from workloads.synth import f32_to_bf16_bits

import gpu_helpers as H

pytestmark = pytest.mark.gpu

HQ, HKV, D, ROT = 16, 4, 128, 64
SCALE = 1.0 / np.sqrt(D)


def pa():
    import paged_kv_cache_454_b200 as m
    return m


def dev_f64(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Model:
    """Projections of made-up tokens: bits of q, K and V rows by token id."""

    def __init__(self, seed):
        self.rng = np.random.default_rng(seed)
        self.f = 10000.0 ** (-np.arange(0, ROT, 2) / ROT)
        self.qw, self.kw = (f32_to_bf16_bits((1 + 0.1 * self.rng.standard_normal(D)).astype(np.float32))
                            for _ in range(2))

    def rows(self, n):
        return f32_to_bf16_bits(self.rng.standard_normal((n, HQ + 2 * HKV, D)).astype(np.float32))

    def write(self, rows, positions, slots, dk, dv):
        """One pa_rope_and_cache call; returns the prepared q."""
        x = H.dev_bf16(rows)
        return pa().pa_rope_and_cache(
            x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], dk, dv, H.dev_i64(slots),
            H.dev_i64(positions), dev_f64(self.f), q_weight=H.dev_bf16(self.qw),
            k_weight=H.dev_bf16(self.kw), eps=1e-6)

    def prepared(self, rows, positions):
        """The same in float64: q, K (normed, rotated) and V."""
        x = bf16_bits_to_f64(rows)
        q = drafting.head_norm(x[:, :HQ], bf16_bits_to_f64(self.qw), 1e-6)
        k = drafting.head_norm(x[:, HQ:HQ + HKV], bf16_bits_to_f64(self.kw), 1e-6)
        return (drafting.rope(q, positions, self.f, False, 1.0),
                drafting.rope(k, positions, self.f, False, 1.0), x[:, HQ + HKV:])


def attend(q, k, v):
    """One float64 query [HQ, D] over rows [L, HKV, D]."""
    o = np.zeros((HQ, D))
    for h in range(HQ):
        o[h], _ = oracle.attend(q[h], k[:, h // (HQ // HKV)], v[:, h // (HQ // HKV)], SCALE)
    return o


def close(got, want):
    """q and K are rounded to bf16 on the way (half a step, 2^-8, each): a score of
    up to 12 moves by at most 2 * 2^-8 * sum |q k| * scale, in practice a few
    percent; the outputs are means of N(0, 1) values.  This pins the plumbing (a wrong
    token, position or page is off by 0.1 and more), the kernels' own tests the digits."""
    assert np.abs(H.host_f64(got) - want).max() < 0.06


def test_draft_verify_accept_decode():
    import torch
    m = Model(1)
    from paged_kv_cache_454_b200.kv_manager import KvManager
    mgr = KvManager(64)
    dk = torch.zeros((64, HKV, 16, D), dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros_like(dk)
    lens = [37, 200]
    hist = []  # (rows, positions) of every sequence
    for s, L in enumerate(lens):
        slots, _ = mgr.add_sequence(s, np.arange(L, dtype=np.int32))
        rows = m.rows(L)
        m.write(rows, np.arange(L), slots, dk, dv)
        hist.append([m.prepared(rows, np.arange(L))])
    # a tree of 7 tokens each: two children, and so on; positions are depths
    parent = [-1, 0, 0, 1, 1, 2, 5]
    depth = [0, 1, 1, 2, 2, 2, 3]
    bits = []
    for i, p in enumerate(parent):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    n = len(parent)
    drafts, slots = [], []
    for s, L in enumerate(lens):
        sl, pairs = mgr.append_tokens(s, np.zeros(n, np.int32))
        assert not pairs
        slots.append(sl)
        drafts.append(m.rows(n))
    pos = np.concatenate([L + np.array(depth) for L in lens])
    q = m.write(np.concatenate(drafts), pos, np.concatenate(slots), dk, dv)
    width = 16
    tables, ctx = mgr.batch([0, 1], width)
    dt, dl = H.dev_i32(tables), H.dev_i32(ctx)
    out, lse = pa().pa_tree_attention(q, H.dev_i32([0, n, 2 * n]), n,
                                      H.dev_i64(np.array(bits * 2)[:, None]), dk, dv, dt, dl,
                                      SCALE, want_lse=True)
    for s, L in enumerate(lens):
        qd, kd, vd = m.prepared(drafts[s], L + np.array(depth))
        _, k0, v0 = hist[s][0]
        for i in range(n):
            see = [j for j in range(n) if (bits[i] >> j) & 1]
            close(out[s * n + i], attend(qd[i], np.concatenate([k0, kd[see]]),
                                         np.concatenate([v0, vd[see]])))
    # the branch 0, 2, 5, 6 is accepted by sequence 0, the root alone by sequence 1
    branches = [[0, 2, 5, 6], [0]]
    kept = np.zeros((2, 1, 4), np.int32)
    for s, br in enumerate(branches):
        kept[s, 0, :len(br)] = br
    pa().pa_compact_tokens(dk, dv, dt, H.dev_i32(kept), H.dev_i32([4, 1]), base=H.dev_i32(lens))
    new_lens = [L + len(br) for L, br in zip(lens, branches)]
    # the next token, behind the accepted ones
    rows = m.rows(2)
    slot = [int(tables[s, L // 16]) * 16 + L % 16 for s, L in enumerate(new_lens)]
    q = m.write(rows, np.array(new_lens), np.array(slot), dk, dv)
    out, _ = pa().pa_decode(q, dk, dv, dt, H.dev_i32([L + 1 for L in new_lens]), SCALE)
    qn, kn, vn = m.prepared(rows, np.array(new_lens))
    for s, br in enumerate(branches):
        _, kd, vd = m.prepared(drafts[s], lens[s] + np.array(depth))
        _, k0, v0 = hist[s][0]
        close(out[s], attend(qn[s], np.concatenate([k0, kd[br], kn[s:s + 1]]),
                             np.concatenate([v0, vd[br], vn[s:s + 1]])))
    assert pa().pa_get_device_error() == 0


def test_prompt_decode_evict_decode():
    import torch
    from paged_kv_cache_454_b200.kv_manager import KvManager
    m = Model(2)
    mgr = KvManager(96)
    dk = torch.zeros((96, HKV, 16, D), dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros_like(dk)
    lens = np.array([300, 133])
    width = 24
    kv = []
    rows = [m.rows(int(L)) for L in lens]
    slots = [mgr.add_sequence(s, np.zeros(int(L), np.int32))[0] for s, L in enumerate(lens)]
    q = m.write(np.concatenate(rows), np.concatenate([np.arange(L) for L in lens]),
                np.concatenate(slots), dk, dv)
    for s, L in enumerate(lens):
        kv.append(m.prepared(rows[s], np.arange(L))[1:])
    tables, ctx = mgr.batch([0, 1], width)
    dt, dl = H.dev_i32(tables), H.dev_i32(ctx)
    cu = H.dev_i32([0, 300, 433])
    _, lse = pa().pa_chunked_prefill(q, cu, 300, dk, dv, dt, dl, SCALE, want_lse=True)
    mass = pa().pa_attention_mass(q, lse, cu, 300, dk, dt, dl, SCALE)
    # every query spreads a weight of 1 per head: G heads and L queries
    assert np.allclose(mass.sum(2).cpu().numpy(), np.repeat(lens[:, None] * 4.0, HKV, 1), rtol=1e-3)
    # two decode steps add theirs
    for _ in range(2):
        r = m.rows(2)
        sl, pairs = mgr.decode_step([0, 1], np.zeros(2, np.int32))
        assert not pairs
        qd = m.write(r, lens, sl, dk, dv)
        lens = lens + 1
        tables, ctx = mgr.batch([0, 1], width)
        dt, dl = H.dev_i32(tables), H.dev_i32(ctx)
        _, lse = pa().pa_decode(qd, dk, dv, dt, dl, SCALE, want_lse=True)
        pa().pa_attention_mass(qd, lse, None, 1, dk, dt, dl, SCALE, mass_in=mass, mass=mass)
        _, k, v = m.prepared(r, lens - 1)
        kv = [(np.concatenate([a, k[s:s + 1]]), np.concatenate([b, v[s:s + 1]]))
              for s, (a, b) in enumerate(kv)]
    assert np.allclose(mass.sum(2).cpu().numpy(), np.repeat(lens[:, None] * 4.0, HKV, 1), rtol=1e-3)
    # down to 100 tokens a head, into the blocks of two new sequences
    for s in range(2):
        mgr.add_sequence(10 + s, np.zeros(100, np.int32))
    fresh, _ = mgr.batch([10, 11], width)
    before = mass.cpu().numpy()
    kept, new_lens, _ = pa().pa_evict(mass, dk, dv, dt, dl, H.dev_i32([100, 100]), sink=4,
                                      recent=20, new_tables=H.dev_i32(fresh), max_keep=100)
    assert new_lens.tolist() == [100, 100]
    for s in range(2):
        mgr.free_sequence(s)
        for g in range(HKV):
            want = drafting.evict_choice(before[s, g], int(lens[s]), 100, 4, 20)
            assert np.array_equal(kept[s, g].cpu().numpy(), want)
    # a decode step over what is left: each head attends to its own tokens
    r = m.rows(2)
    sl, _ = mgr.decode_step([10, 11], np.zeros(2, np.int32))
    qd = m.write(r, lens, sl, dk, dv)
    tables, ctx = mgr.batch([10, 11], width)
    assert ctx.tolist() == [101, 101]
    out, _ = pa().pa_decode(qd, dk, dv, H.dev_i32(tables), H.dev_i32(ctx), SCALE)
    qn, kn, vn = m.prepared(r, lens)
    for s in range(2):
        k, v = kv[s]
        for g in range(HKV):
            idx = kept[s, g].cpu().numpy()
            for h in range(4 * g, 4 * g + 4):
                o, _ = oracle.attend(qn[s, h], np.concatenate([k[idx, g], kn[s:s + 1, g]]),
                                     np.concatenate([v[idx, g], vn[s:s + 1, g]]), SCALE)
                assert np.abs(H.host_f64(out[s, h]) - o).max() < 0.06
    assert pa().pa_get_device_error() == 0


def test_the_chain_in_one_graph():
    # cache write, tree, weights and eviction captured together and replayed
    import torch
    m = Model(3)
    dk = torch.zeros((40, HKV, 16, D), dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros_like(dk)
    tables = H.dev_i32(np.arange(20).reshape(2, 10))
    fresh = H.dev_i32(20 + np.arange(20).reshape(2, 10))
    L, n = 150, 6
    rows = m.rows(2 * L)
    slots = np.concatenate([s * 160 + np.arange(L) for s in range(2)])
    m.write(rows, np.tile(np.arange(L), 2), slots, dk, dv)
    x = H.dev_bf16(m.rows(2 * n))
    pos = H.dev_i64(np.tile(L + np.arange(n), 2))
    sl = H.dev_i64(np.concatenate([s * 160 + L + np.arange(n) for s in range(2)]))
    cu, lens = H.dev_i32([0, n, 2 * n]), H.dev_i32([L + n, L + n])
    mask = H.dev_i64(np.tile([(1 << (i + 1)) - 1 for i in range(n)], 2)[:, None])
    f, budgets = dev_f64(m.f), H.dev_i32([64, 64])

    def step():
        q = pa().pa_rope_and_cache(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], dk, dv, sl, pos, f)
        out, lse = pa().pa_tree_attention(q, cu, n, mask, dk, dv, tables, lens, SCALE, want_lse=True)
        mass = pa().pa_attention_mass(q, lse, cu, n, dk, tables, lens, SCALE)
        return (out, lse, mass) + pa().pa_evict(mass, dk, dv, tables, lens, budgets, sink=2, recent=8,
                                                new_tables=fresh, max_keep=64)

    want = [t.clone() for t in step()]
    want_k = dk[20:].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for _ in range(3):
        dk[20:].zero_()
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(dk[20:], want_k)
    assert pa().pa_get_device_error() == 0


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "fresh"])
def test_evict_again_and_again(in_place):
    # A budget of 64 tokens, two decode steps, down to the budget again: the new tokens'
    # weights start from 0, whatever an evicted token's or a draft's weight left there.
    # float64 follows the weights from what the eviction kept; tolerances of
    # tests/test_gpu_mass.py.
    import torch
    m = Model(4)
    S, width, budget = 3, 12, 64
    dk = torch.zeros((2 * S * width, HKV, 16, D), dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros_like(dk)
    own = np.arange(2 * S * width).reshape(2, S, width)
    lens = np.array([64, 150, 97])
    tables = own[0]
    m.write(m.rows(int(lens.sum())), np.concatenate([np.arange(x) for x in lens]),
            np.concatenate([tables[s, np.arange(x) // 16] * 16 + np.arange(x) % 16
                            for s, x in enumerate(lens)]), dk, dv)
    mass = torch.rand((S, HKV, 16 * width), device="cuda")
    if in_place:
        mass[:, :, 152:] = float("nan")  # of tokens not there yet
    else:
        for s, x in enumerate(lens):
            mass[s, :, x:] = 0
    for turn in range(3):
        for _ in range(2):
            dt = H.dev_i32(tables)
            slots = np.array([tables[s, x // 16] * 16 + x % 16 for s, x in enumerate(lens)])
            q = m.write(m.rows(S), lens, slots, dk, dv)
            had = mass.cpu().numpy().astype(np.float64)
            _, lse = pa().pa_decode(q, dk, dv, dt, H.dev_i32(lens + 1), SCALE, want_lse=True)
            pa().pa_attention_mass(q, lse, None, 1, dk, dt, H.dev_i32(lens + 1), SCALE, mass_in=mass,
                                   mass=mass, own_from_zero=in_place)
            want = drafting.attention_mass(H.host_bits(q), lse.cpu().numpy(), np.arange(S + 1),
                                           H.host_bits(dk), tables, lens + 1, SCALE)
            got = mass.cpu().numpy()
            for s, x in enumerate(lens):
                had[s, :, x] = 0
                total = had[s, :, :x + 1] + want[s]
                assert np.all(np.abs(got[s, :, :x + 1] - total)
                              <= 8e-5 * want[s] + 2.0 ** -24 * total + 1e-30)
            lens = lens + 1
        before = mass.cpu().numpy()
        new = None if in_place else own[(turn + 1) % 2]
        kept, nl, out = pa().pa_evict(mass, dk, dv, dt, H.dev_i32(lens), H.dev_i32([budget] * S),
                                      sink=2, recent=5, mass_out=mass if in_place else None,
                                      new_tables=None if in_place else H.dev_i32(new),
                                      max_keep=budget)
        assert nl.tolist() == [budget] * S and out.shape == mass.shape
        for s in range(S):
            for g in range(HKV):
                want = drafting.evict_choice(before[s, g], int(lens[s]), budget, 2, 5)
                assert np.array_equal(kept[s, g].cpu().numpy(), want)
                assert np.array_equal(out[s, g, :budget].cpu().numpy(), before[s, g, want])
        if not in_place:
            assert not bool(out[:, :, budget:].any())
            tables = new
        mass = out
        lens = np.full(S, budget)
    assert pa().pa_get_device_error() == 0


def test_the_block_manager_carries_drafts_and_evictions():
    # prefix caching on, one prompt for two sequences: a tree each, its accepted branch, a
    # decode step; then one sequence packed into fresh blocks, the other in place, another
    # step; at last the prompt again, whose cached blocks must still hold it
    import torch
    from paged_kv_cache_454_b200.kv_manager import KvManager
    m = Model(5)
    mgr = KvManager(80, prefix_caching=True)
    dk = torch.zeros((80, HKV, 16, D), dtype=torch.bfloat16, device="cuda")
    dv = torch.zeros_like(dk)
    P, width = 70, 8
    prompt = np.arange(1000, 1000 + P, dtype=np.int32)
    rows = m.rows(P)
    for s in range(2):
        slots, cached = mgr.add_sequence(s, prompt)
        assert cached == (0, 64)[s]
        m.write(rows, np.arange(P), slots, dk, dv)
    k0, v0 = m.prepared(rows, np.arange(P))[1:]
    bits, depth = [1, 3, 5, 0b1011], np.array([0, 1, 1, 2])
    n, branches = 4, [[0, 1, 3], [0, 2]]
    drafts, slots = [m.rows(n) for _ in range(2)], []
    for s in range(2):
        sl, pairs = mgr.append_draft(s, n)
        if pairs:
            pa().pa_copy_blocks(dk, dv, pairs)
        slots.append(sl)
    pos = np.tile(P + depth, 2)
    q = m.write(np.concatenate(drafts), pos, np.concatenate(slots), dk, dv)
    tables, ctx = mgr.batch([0, 1], width)
    assert ctx.tolist() == [P + n] * 2
    dt = H.dev_i32(tables)
    out, _ = pa().pa_tree_attention(q, H.dev_i32([0, n, 2 * n]), n,
                                    H.dev_i64(np.array(bits * 2)[:, None]), dk, dv, dt,
                                    H.dev_i32(ctx), SCALE)
    kept = np.zeros((2, 1, 3), np.int32)
    for s, br in enumerate(branches):
        kept[s, 0, :len(br)] = br
    pa().pa_compact_tokens(dk, dv, dt, H.dev_i32(kept), H.dev_i32([3, 2]), base=H.dev_i32([P, P]))
    kv = []
    for s, br in enumerate(branches):
        mgr.accept_draft(s, 2000 + 10 * s + np.array(br))
        qd, kd, vd = m.prepared(drafts[s], P + depth)
        for i in range(n):
            see = [j for j in range(n) if (bits[i] >> j) & 1]
            close(out[s * n + i], attend(qd[i], np.concatenate([k0, kd[see]]),
                                         np.concatenate([v0, vd[see]])))
        kv.append((np.concatenate([k0, kd[br]]), np.concatenate([v0, vd[br]])))
    lens = np.array([P + 3, P + 2])

    def step(ids, positions, rows_of):
        """A decode step of sequences ``ids``; ``rows_of(s, g)``: K and V rows head g of
        sequence s attends to besides its own new one."""
        r = m.rows(2)
        sl, pairs = mgr.decode_step(ids, [7, 7])
        assert not pairs
        qd = m.write(r, positions, sl, dk, dv)
        tables, ctx = mgr.batch(ids, width)
        out, lse = pa().pa_decode(qd, dk, dv, H.dev_i32(tables), H.dev_i32(ctx), SCALE,
                                  want_lse=True)
        qn, kn, vn = m.prepared(r, positions)
        for s in range(2):
            for g in range(HKV):
                k, v = rows_of(s, g)
                for h in range(4 * g, 4 * g + 4):
                    o, _ = oracle.attend(qn[s, h], np.concatenate([k, kn[s:s + 1, g]]),
                                         np.concatenate([v, vn[s:s + 1, g]]), SCALE)
                    assert np.abs(H.host_f64(out[s, h]) - o).max() < 0.06
            kv[s] = np.concatenate([kv[s][0], kn[s:s + 1]]), np.concatenate([kv[s][1], vn[s:s + 1]])
        return qd, lse, tables, ctx

    qd, lse, tables, ctx = step([0, 1], lens, lambda s, g: (kv[s][0][:, g], kv[s][1][:, g]))
    assert ctx.tolist() == [P + 4, P + 3]
    mass = pa().pa_attention_mass(qd, lse, None, 1, dk, H.dev_i32(tables), H.dev_i32(ctx), SCALE)
    # sequence 0 into fresh blocks; 1 in place, which its blocks, still the prompt's, forbid
    mgr.add_reserved(10, 40)
    fresh, _ = mgr.batch([10], width)
    kept0, _, _ = pa().pa_evict(mass[:1], dk, dv, H.dev_i32(tables[:1]), H.dev_i32(ctx[:1]),
                                H.dev_i32([40]), sink=2, recent=8, new_tables=H.dev_i32(fresh))
    from paged_kv_cache_454_b200.kv_manager import KvManagerError
    with pytest.raises(KvManagerError):
        mgr.evicted(1, 40)
    mgr.add_reserved(11, 50)
    fresh, _ = mgr.batch([11], width)
    kept1, _, mass1 = pa().pa_evict(mass[1:].contiguous(), dk, dv, H.dev_i32(tables[1:]),
                                    H.dev_i32(ctx[1:]), H.dev_i32([50]), sink=2, recent=8,
                                    new_tables=H.dev_i32(fresh))
    mgr.free_sequence(0)
    mgr.free_sequence(1)
    # the second one once more, now in place: its blocks are its own
    again, _, _ = pa().pa_evict(mass1, dk, dv, H.dev_i32(fresh), H.dev_i32([50]), H.dev_i32([30]),
                                sink=1, recent=4, max_keep=30)
    mgr.evicted(11, 30)
    idx = [kept0[0, :, :40].cpu().numpy(),
           np.take_along_axis(kept1[0, :, :50].cpu().numpy(), again[0].cpu().numpy(), 1)]
    full = list(kv)
    step([10, 11], np.array([P + 4, P + 3]),
         lambda s, g: (full[s][0][idx[s][g], g], full[s][1][idx[s][g], g]))
    assert mgr.context_len(10) == 41 and mgr.context_len(11) == 31
    # the prompt is still found, and still there
    slots, cached = mgr.add_sequence(20, prompt)
    assert cached == 64
    m.write(rows, np.arange(P), slots, dk, dv)
    r = m.rows(1)
    sl, _ = mgr.decode_step([20], [9])
    qn = m.write(r, np.array([P]), sl, dk, dv)
    tables, ctx = mgr.batch([20], width)
    out, _ = pa().pa_decode(qn, dk, dv, H.dev_i32(tables), H.dev_i32(ctx), SCALE)
    qx, kx, vx = m.prepared(r, np.array([P]))
    close(out[0], attend(qx[0], np.concatenate([k0, kx]), np.concatenate([v0, vx])))
    assert pa().pa_get_device_error() == 0


def test_blocks_past_2_to_the_31_elements():
    # a pool of 4.4 GB: the same calls on blocks at its end and on a small pool, bit by bit
    import torch
    S, L, n, hkv = 2, 200, 5, 8
    per = hkv * 16 * D
    nb = 2 ** 31 // per + 64
    need = -(-L // 16)
    far = nb - 1 - np.random.default_rng(1).permutation(60)[:4 * need // 2 * 2].reshape(2, S, -1)
    assert far.min() * per > 2 ** 31 - 64 * per and (far * per).max() > 2 ** 31
    near = np.arange(far.size).reshape(far.shape)
    big = [torch.empty((nb, hkv, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = [torch.empty((far.size, hkv, 16, D), dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    m = Model(6)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((S * L, 2 * hkv + 16, D), generator=g, device="cuda", dtype=torch.bfloat16)
    pos = H.dev_i64(np.tile(np.arange(L), S))
    cu = H.dev_i32(n * np.arange(S + 1))
    mask = H.dev_i64(np.tile([(1 << (i + 1)) - 1 for i in range(n)], S)[:, None])
    lens, f = H.dev_i32([L] * S), dev_f64(m.f)
    t = np.arange(L)
    rows = torch.tensor([s * L + L - n + i for s in range(S) for i in range(n)], device="cuda")

    def run(pools, blocks):
        k, v = pools
        ids = torch.as_tensor(blocks[1].reshape(-1), device="cuda")
        k[ids] = 0
        v[ids] = 0
        slots = np.concatenate([blocks[0, s, t // 16].astype(np.int64) * 16 + t % 16
                                for s in range(S)])
        q = pa().pa_rope_and_cache(x[:, :16], x[:, 16:16 + hkv], x[:, 16 + hkv:], k, v,
                                   H.dev_i64(slots), pos, f)[rows]
        tables, new = H.dev_i32(blocks[0]), H.dev_i32(blocks[1])
        out, lse = pa().pa_tree_attention(q, cu, n, mask, k, v, tables, lens, SCALE, want_lse=True)
        mass = pa().pa_attention_mass(q, lse, cu, n, k, tables, lens, SCALE)
        kept, _, w = pa().pa_evict(mass, k, v, tables, lens, H.dev_i32([90] * S), sink=2, recent=9,
                                   new_tables=new, max_keep=90)
        pa().pa_compact_tokens(k, v, new, H.dev_i32([[[3, 4, 9]]] * S), H.dev_i32([3] * S),
                               base=H.dev_i32([50] * S))
        return out, lse, mass[..., :L], kept, w[..., :90], k[ids], v[ids]

    for a, b in zip(run(big, far), run(small, near)):
        assert torch.equal(a, b)
    assert pa().pa_get_device_error() == 0
