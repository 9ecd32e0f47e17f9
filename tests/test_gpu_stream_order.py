"""Calls in order on one stream that pass memory on to one another: a scratch buffer
that several calls share, inputs whose memory is the next call's scratch, lengths that
the kernel before wrote.  Each order runs many times without a wait, and every result
has the bits of a run that synchronises after every call."""
from __future__ import annotations

import numpy as np
import pytest

import gpu_helpers as H

pytestmark = pytest.mark.gpu

HQ, D, S, N = 8, 128, 3, 5


def pa():
    import paged_kv_cache_454_b200 as m
    return m


class Step:
    """Few KV heads and short tables, so that the grids are small and a kernel that may
    start early finds room."""

    def __init__(self, hkv, seed):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hkv = hkv
        lens = rng.integers(300, 1500, S)
        blocks = -(-lens // 16)
        nb = int(blocks.sum()) + 4
        tables = np.zeros((S, int(blocks.max())), np.int32)
        order, at = rng.permutation(nb), 0
        for s, k in enumerate(blocks):
            tables[s, :k] = order[at:at + k]
            at += k
        rand = lambda *shape: torch.randn(shape, generator=g, device="cuda",  # noqa: E731
                                          dtype=torch.bfloat16)
        self.k, self.v = rand(nb, hkv, 16, D), rand(nb, hkv, 16, D)
        self.tables, self.lens = H.dev_i32(tables), H.dev_i32(lens)
        self.cu = H.dev_i32(N * np.arange(S + 1))
        self.qt, self.qd = rand(S * N, HQ, D), rand(S, HQ, D)
        self.mask = torch.randint(0, 2 ** N, (S * N, 1), generator=g, device="cuda")
        self.scale = D ** -0.5
        # one scratch buffer, large enough for either call
        self.scratch = torch.empty(
            max(pa().pa_tree_workspace_size(N, HQ, self.k),
                pa().pa_decode_workspace_size(S, HQ, self.k, tables.shape[1])),
            dtype=torch.uint8, device="cuda")
        self.mass = torch.zeros((S, hkv, 16 * tables.shape[1]), device="cuda")

    def tree(self, **kw):
        return pa().pa_tree_attention(self.qt, self.cu, N, self.mask, self.k, self.v, self.tables,
                                      self.lens, self.scale, want_lse=True, **kw)

    def decode(self, **kw):
        return pa().pa_decode(self.qd, self.k, self.v, self.tables, self.lens, self.scale,
                              want_lse=True, **kw)

    def weigh(self, lse):
        return pa().pa_attention_mass(self.qd, lse, None, 1, self.k, self.tables, self.lens,
                                      self.scale, mass_in=self.mass, mass=self.mass)


def runs(order, repeats):
    """The results of ``order(sync)`` with a wait after every call, and of ``repeats``
    runs of it without one, none of which waits for the other."""
    import torch
    want = order(torch.cuda.synchronize)
    got = [order(lambda: None) for _ in range(repeats)]
    torch.cuda.synchronize()
    assert pa().pa_get_device_error() == 0
    for one in got:
        for x, y in zip(one, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("hkv", [1, 8])
@pytest.mark.parametrize("shared", [True, False], ids=["one_scratch", "default"])
def test_tree_then_decode(hkv, shared):
    st = Step(hkv, 1)
    kw = {"workspace": st.scratch} if shared else {}

    def order(sync):
        res = []
        for _ in range(2):
            res += st.tree(**kw)
            sync()
            res += st.decode(**kw)
            sync()
        return res

    runs(order, 150)


@pytest.mark.parametrize("hkv", [1, 8])
def test_decode_weight_decode_on_one_scratch(hkv):
    st = Step(hkv, 2)

    def order(sync):
        st.mass.zero_()
        res = []
        for _ in range(2):
            out, lse = st.decode(workspace=st.scratch)
            sync()
            st.weigh(lse)
            sync()
            again = st.decode(workspace=st.scratch)
            sync()
            res += [out, lse, *again]
        return res + [st.mass.clone()]

    runs(order, 100)


def test_decode_after_decode_without_workspaces_of_their_own():
    st = Step(2, 3)

    def order(sync):
        res = []
        for _ in range(3):
            res += st.decode(workspace=st.scratch)
            sync()
        return res

    runs(order, 100)


def test_inputs_of_a_cache_write_become_the_workspace():
    # K and V of the step lie in the buffer that the decode then takes as its scratch
    import torch
    st = Step(2, 4)
    n = 2 * S
    rows = torch.randn((n, HQ + 2 * 2, D), device="cuda", dtype=torch.bfloat16)
    bits = rows.view(torch.uint8).flatten()
    last = (st.lens.long() - 1)
    at = torch.stack([last - 1, last], 1)
    slots = (torch.gather(st.tables.long(), 1, at // 16) * 16 + at % 16).flatten()
    pos = at.flatten().contiguous()
    freq = torch.from_numpy(pa().pa_rope_frequencies(D)[0]).cuda()
    scratch = torch.empty(max(bits.numel(), st.scratch.numel()), dtype=torch.uint8, device="cuda")

    def order(sync):
        st.k.zero_()
        scratch[:bits.numel()].copy_(bits)
        x = scratch[:bits.numel()].view(torch.bfloat16).view(n, HQ + 4, D)
        sync()
        pa().pa_rope_and_cache(x[:, :HQ], x[:, HQ:HQ + 2], x[:, HQ + 2:], st.k, st.v, slots, pos,
                               freq)
        sync()
        res = list(st.decode(workspace=scratch))
        sync()
        return res + [st.k.clone(), st.v.clone()]

    runs(order, 60)


def test_lengths_written_by_the_kernel_before():
    # directly before tree attention, weight and decode: by an elementwise kernel and by
    # an eviction
    st = Step(2, 5)
    full = st.lens.clone()
    short = full - 100
    cu = st.cu.clone()
    budgets = H.dev_i32([200] * S)

    def order(sync):
        st.mass.copy_(st.mass0)
        st.k.copy_(st.k0)
        st.v.copy_(st.v0)
        res = []
        for lens in (short, full):
            st.lens.copy_(lens)
            res += st.tree()
            sync()
            st.cu.zero_()
            sync()
            st.lens.add_(-3)
            st.cu.add_(cu)
            res += st.tree()
            sync()
            out, lse = st.decode()
            st.lens.sub_(0)
            res += [out, lse, st.weigh(lse).clone()]
            sync()
        keep = st.lens
        _, st.lens, _ = pa().pa_evict(st.mass, st.k, st.v, st.tables, st.lens, budgets, sink=2,
                                      recent=N)
        sync()
        res += st.tree()
        sync()
        res += st.decode()
        sync()
        res.append(st.lens)
        st.lens = keep
        return res

    st.mass0, st.k0, st.v0 = st.mass + 1, st.k.clone(), st.v.clone()
    runs(order, 40)
