"""Drafts and evicted caches in the block manager (``append_draft``, ``accept_draft``,
``add_reserved``, ``evicted``): hand-made scenarios that the oracle and the C++ manager
both have to pass, and random streams of all operations, op by op.  On the host."""
from __future__ import annotations

import random

import pytest

import oracle
from paged_kv_cache_454_b200.kv_manager import KvManager, KvManagerError
import test_kv_manager as both
from test_kv_manager_oracle import random_ops

MANAGERS = [pytest.param(lambda nb, bs, pc: oracle.KvManager(nb, bs, pc, 4), id="oracle"),
            pytest.param(lambda nb, bs, pc: KvManager(nb, bs, pc, 4), id="library")]
ERRORS = (oracle.KvManagerError, oracle.NoBlocks, KvManagerError)


def run(target, op):
    kind = op[0]
    if kind not in ("draft", "accept", "reserve", "evicted"):
        return both.run(target, op)

    class Calls:  # (the four under a name that the other runner knows: its error mapping)
        def free_sequence(self, _):
            if kind == "draft":
                slots, pairs = target.append_draft(op[1], op[2])
                self.res = ([int(s) for s in slots], [tuple(map(int, p)) for p in pairs])
            elif kind == "accept":
                target.accept_draft(op[1], op[2])
            elif kind == "reserve":
                target.add_reserved(op[1], op[2])
            else:
                target.evicted(op[1], op[2])

    calls = Calls()
    return both.run(calls, ("free", None)) + (getattr(calls, "res", None),)


@pytest.mark.parametrize("pc", [False, True])
@pytest.mark.parametrize("make", MANAGERS)
def test_an_accepted_branch_keeps_its_slots(make, pc):
    m = make(16, 4, pc)
    m.add_sequence(0, [1, 2, 3, 4, 5, 6])
    slots, pairs = m.append_draft(0, 9)          # blocks 0, 1 | 1, 2, 3
    assert list(slots) == [6, 7, 8, 9, 10, 11, 12, 13, 14] and not pairs
    assert m.context_len(0) == 15 and len(m.block_table(0)) == 4
    m.accept_draft(0, [7, 8, 9])
    assert m.context_len(0) == 9 and m.block_table(0) == [0, 1, 2] and m.num_free_blocks() == 13
    slots, _ = m.decode_step([0], [10])          # right behind the accepted ones
    assert list(slots) == [9]
    # all dropped, and nothing drafted
    m.append_draft(0, 5)
    m.accept_draft(0, [])
    assert m.context_len(0) == 10 and m.block_table(0) == [0, 1, 2]
    m.append_draft(0, 0)
    m.accept_draft(0, [])
    with pytest.raises(ERRORS):
        m.accept_draft(0, [1])
    assert m.context_len(0) == 10


@pytest.mark.parametrize("make", MANAGERS)
def test_only_accepted_tokens_are_cached(make):
    m = make(16, 4, True)
    m.add_sequence(0, [1, 2, 3])
    m.append_draft(0, 6)
    # (another sequence of other tokens meanwhile)
    assert m.add_sequence(1, [1, 2, 3, 0])[1] == 0
    m.accept_draft(0, [7, 8, 9, 10, 11])
    table = m.block_table(0)
    slots, cached = m.add_sequence(2, [1, 2, 3, 7, 8, 9, 10, 11, 12])
    assert cached == 8 and m.block_table(2)[:2] == table[:2] and list(slots[:8]) == [-1] * 8
    assert m.ref_count(table[0]) == 2


@pytest.mark.parametrize("make", MANAGERS)
def test_a_draft_behind_a_shared_block_is_copied(make):
    m = make(16, 4, False)
    m.add_sequence(0, [1, 2, 3, 4, 5])
    m.fork(0, 1)
    slots, pairs = m.append_draft(1, 2)
    assert [tuple(p) for p in pairs] == [(1, 2)] and list(slots) == [9, 10]
    m.accept_draft(1, [])
    assert m.block_table(0) == [0, 1] and m.block_table(1) == [0, 2]


@pytest.mark.parametrize("make", MANAGERS)
def test_what_an_open_draft_refuses(make):
    m = make(16, 4, True)
    m.add_sequence(0, list(range(8)))
    m.add_sequence(1, list(range(20, 28)))
    m.append_draft(0, 3)
    for call in (lambda: m.append_tokens(0, [1]), lambda: m.append_draft(0, 1),
                 lambda: m.decode_step([1, 0], [1, 1]), lambda: m.fork(0, 5),
                 lambda: m.share_prefix(0, 5, 1), lambda: m.share_blocks(0, 1, [0]),
                 lambda: m.share_blocks(1, 0, [0]), lambda: m.swap_out(0),
                 lambda: m.evicted(0, 4), lambda: m.accept_draft(0, [1, 2, 3, 4])):
        with pytest.raises(ERRORS):
            call()
    assert m.context_len(0) == 11 and m.context_len(1) == 8 and m.num_free_blocks() == 11
    m.free_sequence(0)
    assert m.num_free_blocks() == 14


@pytest.mark.parametrize("make", MANAGERS)
def test_reserved_sequences_share_nothing(make):
    m = make(16, 4, True)
    m.add_sequence(0, [0] * 8)
    m.add_reserved(1, 8)
    m.add_reserved(2, 7)
    tables = [set(m.block_table(s)) for s in range(3)]
    assert not tables[0] & tables[1] and not tables[1] & tables[2] and not tables[0] & tables[2]
    m.decode_step([1, 2], [0, 0])
    assert m.context_len(1) == 9 and m.context_len(2) == 8
    # nothing of them is found, not even blocks that filled up later
    m.free_sequence(0)
    for _ in range(3):
        m.decode_step([1, 2], [0, 0])
    m.fork(1, 3)
    m.decode_step([3], [0])
    slots, cached = m.add_sequence(4, [0] * 12)
    assert cached == 8 and not set(m.block_table(4)) & (tables[1] | tables[2])
    with pytest.raises(ERRORS):
        m.share_blocks(4, 1, [0])
    with pytest.raises(ERRORS):
        m.share_blocks(1, 4, [0])
    with pytest.raises(ERRORS):
        m.add_reserved(4, 1)
    with pytest.raises(ERRORS):
        m.add_reserved(5, 16 * 4)
    with pytest.raises(ERRORS):
        m.add_reserved(5, 2 ** 31 - 1)


@pytest.mark.parametrize("make", MANAGERS)
def test_evicted_blocks_leave_the_cache(make):
    m = make(16, 4, True)
    m.add_sequence(0, list(range(16)))
    table = m.block_table(0)
    m.add_sequence(1, list(range(8)) + [50] * 4)  # shares the first two blocks
    with pytest.raises(ERRORS):
        m.evicted(0, 9)                           # its first blocks are another's too
    with pytest.raises(ERRORS):
        m.evicted(0, 17)
    assert m.context_len(0) == 16
    m.free_sequence(1)                            # [50] * 4 stays cached behind the two
    m.evicted(0, 6)
    assert m.context_len(0) == 6 and m.block_table(0) == table[:2]
    assert m.num_free_blocks() == 14
    assert m.add_sequence(2, list(range(8)) + [50] * 4 + [1])[1] == 0
    slots, _ = m.append_tokens(0, [6, 7])
    assert [int(s) for s in slots] == [table[1] * 4 + 2, table[1] * 4 + 3]
    # a sequence whose kept blocks are its own, the dropped ones shared
    m.add_sequence(5, [90, 91])
    m.append_tokens(5, [92])
    m.evicted(5, 0)
    assert m.context_len(5) == 0 and m.block_table(5) == []


def drafting_ops(seed, n_ops, nb, bs, pc):
    """The streams of the manager's other tests, with drafts and evictions in between;
    ids from 10^6 on are reserved sequences."""
    rng = random.Random(1000 + seed)
    known, next_id = [], 10 ** 6
    for op in random_ops(seed, n_ops, nb, bs, pc):
        yield op
        known += [op[1]] if op[0] == "add" else [op[2]] if op[0] in ("fork", "share_prefix") else []
        if rng.random() < 0.5 and known:
            sid = rng.choice(known[-12:])
            r = rng.random()
            if r < 0.35:
                yield ("draft", sid, rng.randrange(0, 2 * bs + 2))
                if rng.random() < 0.3:  # something else while it is open
                    yield ("append", sid, [1])
                    yield ("fork", sid, next_id)
                    next_id += 1
                yield ("accept", sid, [rng.randrange(4) for _ in range(rng.randrange(0, bs + 3))])
                yield ("accept", sid, [])
            elif r < 0.55:
                yield ("evicted", sid, rng.randrange(0, 3 * bs))
            elif r < 0.75:
                yield ("reserve", next_id, rng.randrange(0, 3 * bs))
                yield ("step", [next_id], [1])
                if rng.random() < 0.7:
                    yield ("free", next_id)
                else:
                    known.append(next_id)
                next_id += 1
            elif r < 0.9:
                yield ("append", sid, [rng.randrange(4) for _ in range(rng.randrange(1, bs + 2))])
            else:
                yield ("free", sid)


@pytest.mark.parametrize("pc", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_random_streams_op_by_op(seed, pc):
    nb, bs = 90, 4
    ref, lib = oracle.KvManager(nb, bs, pc, 10), KvManager(nb, bs, pc, 10)
    done = {}
    for op in drafting_ops(seed, 800, nb, bs, pc):
        a, b = run(ref, op), run(lib, op)
        assert a == b, (op, a, b)
        if a[0] == "ok":
            done[op[0]] = done.get(op[0], 0) + 1
        both.compare_state(ref, lib, list(ref.seqs))
    assert all(done.get(k, 0) >= 3 for k in ("draft", "accept", "reserve", "evicted")), done
