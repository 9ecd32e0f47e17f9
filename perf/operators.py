"""Measured cases of the paged cache's drafting and eviction operators.

Five operators over the block-paged KV pool (bf16 ``[num_blocks, Hkv, 16, D]``):

rope          rotary positions on q and k rows (half or interleaved pairs, part of
              the head, frequencies scaled for long contexts)
norm_rope     per-head RMS norms of q and k, the rotation, and the cache write of
              K and V, in one pass
tree          attention of a tree of drafted tokens over a sequence's cache
mass          accumulated attention weight of every cached token
evict         keep a budget of tokens per KV head by accumulated weight and pack
              them into fresh blocks

``run`` computes the plain form in elementary torch operations (fp32, fp64 for
angles) where ``own`` is false, and calls ``paged_kv_cache_454_b200`` where it is
true.  Everything is written out of place, so a pass can be repeated on a state.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence being decoded: the smallest call, all latency
        {"name": "rope_one_token", "op": "rope", "tokens": 1, "hq": 64, "hkv": 8, "dim": 128,
         "rot": 128, "interleaved": False, "scaled": False, "far": 4096},
        # a prefill chunk of an odd length, a quarter of the head rotated in
        # interleaved pairs, frequencies stretched to a million positions
        {"name": "rope_partial_long", "op": "rope", "tokens": 6145, "hq": 32, "hkv": 32, "dim": 64,
         "rot": 16, "interleaved": True, "scaled": True, "far": 1000000},
        # the 128-sequence decode step of the 70B-like GQA layer
        {"name": "norm_decode128", "op": "norm_rope", "tokens": 128, "hq": 64, "hkv": 8, "dim": 128,
         "rot": 128, "interleaved": False, "scaled": False, "far": 32768, "pad": 0},
        # all new tokens of the Qwen-32B-like continuous-batching step (8 chunks
        # of 512 and 192 decode tokens), with padded rows
        {"name": "norm_mixed4288", "op": "norm_rope", "tokens": 4288, "hq": 40, "hkv": 8,
         "dim": 128, "rot": 128, "interleaved": False, "scaled": True, "far": 131072, "pad": 61},
        # a whole 32K prompt written in one step
        {"name": "norm_prompt32k", "op": "norm_rope", "tokens": 32768, "hq": 64, "hkv": 8,
         "dim": 128, "rot": 64, "interleaved": True, "scaled": False, "far": 32768, "pad": 0},
        # one user, a short chat, a tree of 16 drafted tokens
        {"name": "tree_single", "op": "tree", "seqs": 1, "hq": 64, "hkv": 8, "dim": 128,
         "lo": 1000, "hi": 1000, "nlo": 16, "nhi": 16},
        # multi-head attention (7B-like), ragged trees
        {"name": "tree_mha", "op": "tree", "seqs": 24, "hq": 32, "hkv": 32, "dim": 128,
         "lo": 129, "hi": 2048, "nlo": 3, "nhi": 25},
        # a serving batch at group 8, long and ragged contexts, trees up to 63 tokens
        {"name": "tree_batch", "op": "tree", "seqs": 48, "hq": 64, "hkv": 8, "dim": 128,
         "lo": 300, "hi": 16001, "nlo": 7, "nhi": 63},
        # weight of a decode step's token on every cached token, long contexts
        {"name": "mass_decode", "op": "mass", "seqs": 40, "hq": 64, "hkv": 8, "dim": 128,
         "lo": 1024, "hi": 16384, "nlo": 1, "nhi": 1},
        # weight of an observation window at the end of each prompt
        {"name": "mass_window", "op": "mass", "seqs": 9, "hq": 40, "hkv": 8, "dim": 128,
         "lo": 500, "hi": 4203, "nlo": 17, "nhi": 40},
        # a batch of caches of a few thousand tokens each brought down to a budget
        {"name": "evict_batch", "op": "evict", "seqs": 48, "hkv": 8, "dim": 128,
         "lo": 2000, "hi": 8192, "keep": 1531, "sink": 4, "recent": 256},
        # one long conversation: few heads, many tokens each
        {"name": "evict_long", "op": "evict", "seqs": 1, "hkv": 8, "dim": 128,
         "lo": 31337, "hi": 31337, "keep": 4096, "sink": 16, "recent": 512},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "tree", "mass", "evict"])
    dim = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    if op in ("rope", "norm_rope"):
        c = {"op": op, "tokens": _log_int(rng, 1, 12000), "hq": hq, "hkv": hkv, "dim": dim,
             "rot": rng.choice([16, 32, 48, dim, dim, dim]), "interleaved": rng.random() < 0.5,
             "scaled": rng.random() < 0.5, "far": _log_int(rng, 100, 1000000)}
        if op == "norm_rope":
            c["pad"] = rng.choice([0, 1, c["tokens"] // 10])
        return c
    lo = _log_int(rng, 70, 4000)
    hi = _log_int(rng, lo, 16000)
    seqs = max(1, min(_log_int(rng, 1, 64), 400000 // hi))
    c = {"op": op, "seqs": seqs, "hkv": hkv, "dim": dim, "lo": lo, "hi": hi}
    if op == "evict":
        c["keep"] = _log_int(rng, 16, hi)
        c["sink"] = rng.choice([0, 1, 4, 16])
        c["recent"] = rng.choice([0, 1, 33, 256])
        return c
    c["hq"] = hq
    top = 64 if hq // hkv <= 8 else 32
    c["nhi"] = 1 if op == "mass" and rng.random() < 0.5 else _log_int(rng, 1, top)
    c["nlo"] = rng.randint(1, c["nhi"])
    return c


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _frequencies(case):
    """Inverse frequencies (fp64) of the rotation and the factor on cos and sin;
    scaled: low frequencies stretched 16x, high ones kept, a ramp between."""
    rot = case["rot"]
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if not case["scaled"]:
        return f, 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * keep + f / 16.0 * (1 - keep), 0.1 * math.log(16.0) + 1.0


def _spread(case):
    """Context lengths (spread over their range's logarithm) and new-token counts
    (spread evenly): the same for every seed, which only changes their order."""
    s = case["seqs"]
    at = (np.arange(s) + 0.5) / s
    lens = np.floor(case["lo"] * (case["hi"] / case["lo"]) ** at).astype(np.int64)
    n = np.ones(s, np.int64)
    if "nlo" in case:
        n = case["nlo"] + np.floor((case["nhi"] + 1 - case["nlo"]) * at).astype(np.int64)
    if s > 1:  # the ends of the ranges are among them
        lens[0], lens[-1] = case["lo"], case["hi"]
    return lens, n


def _lengths(case, r):
    lens, n = _spread(case)
    return r.permutation(lens), r.permutation(n)


def _tables(lens, r, first, total, width):
    """Block tables over a shuffled pool; entries past a context are padding."""
    need = -(-lens // BLOCK)
    perm = r.permutation(total)[first:first + int(need.sum())]
    out = np.full((len(lens), width), 2**31 - 1, np.int32)
    for s, at in enumerate(np.concatenate([[0], np.cumsum(need)[:-1]])):
        out[s, :need[s]] = perm[at:at + need[s]]
    return out


def _tree_bits(n, r, words):
    """Each token's ancestors and itself, as bits: token i hangs on an earlier one."""
    rows = np.zeros((n, words * 64), bool)
    for i in range(n):
        if i:
            p = int(r.integers(max(0, i - 6), i)) if r.random() < 0.9 else -1
            if p >= 0:
                rows[i] = rows[p]
        rows[i, i] = True
    return np.packbits(rows, axis=1, bitorder="little").view(np.int64)


def prepare(case, seed):
    dev = torch.device("cuda")
    r = np.random.default_rng([seed, 77])
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    st = {"case": case, "op": case["op"]}
    d, hkv = case["dim"], case["hkv"]
    if case["op"] in ("rope", "norm_rope"):
        t, hq = case["tokens"], case["hq"]
        # one projection's output rows: q, k and v of a token next to each other
        qkv = normal(t, (hq + 2 * hkv), d).mul_(2.0).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        f, factor = _frequencies(case)
        st["inv_freq"], st["factor"] = put(f), factor
        st["positions"] = put(r.integers(0, case["far"], t).astype(np.int64))
        st["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        if case["op"] == "rope":
            st["k_out"] = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev)
            return st
        st["qw"] = (1 + 0.1 * normal(d)).to(torch.bfloat16)
        st["kw"] = (1 + 0.1 * normal(d)).to(torch.bfloat16)
        blocks = (t * 5) // (4 * BLOCK) + 2
        st["k_pool"] = normal(blocks, hkv, BLOCK, d).to(torch.bfloat16)
        st["v_pool"] = normal(blocks, hkv, BLOCK, d).to(torch.bfloat16)
        need = -(-t // BLOCK)
        order = r.permutation(blocks)[:need]
        slots = order[np.arange(t) // BLOCK].astype(np.int64) * BLOCK + np.arange(t) % BLOCK
        if case["pad"]:
            slots[r.choice(t, min(case["pad"], t), replace=False)] = -1
        st["slots"] = put(slots)
        return st
    lens, n = _lengths(case, r)
    width = -(-case["hi"] // BLOCK) + 1
    if case["op"] == "evict":
        kept = np.minimum(lens, case["keep"])
        used, fresh = int((-(-lens // BLOCK)).sum()), int((-(-kept // BLOCK)).sum())
        blocks = used + fresh + 3
        st["tables"] = put(_tables(lens, np.random.default_rng([seed, 6]), 0, blocks, width))
        st["new_tables"] = put(_tables(kept, np.random.default_rng([seed, 6]), used, blocks,
                                       -(-case["keep"] // BLOCK)))
        st["budgets"] = put(np.full(case["seqs"], case["keep"], np.int32))
        # accumulated weights: a few heavy tokens, a long light tail, exact ties
        # among tokens that were never looked at
        m = torch.exp(3.0 * normal(case["seqs"], hkv, case["hi"]))
        m = torch.where(torch.rand(m.shape, generator=g, device=dev) < 0.05, torch.zeros_like(m), m)
        st["mass"] = m
        st["kept"] = torch.full((case["seqs"], hkv, case["keep"]), -1, dtype=torch.int32, device=dev)
        st["mass_out"] = torch.zeros((case["seqs"], hkv, case["keep"]), device=dev)
        st["new_lens"] = torch.zeros(case["seqs"], dtype=torch.int32, device=dev)
    else:
        hq = case["hq"]
        blocks = int((-(-lens // BLOCK)).sum() * 5 // 4) + 2
        st["tables"] = put(_tables(lens, np.random.default_rng([seed, 6]), 0, blocks, width))
        cu = np.concatenate([[0], np.cumsum(n)])
        st["cu"], st["max_n"] = put(cu.astype(np.int32)), int(n.max())
        st["q"] = normal(int(cu[-1]), hq, d).to(torch.bfloat16)
        st["row_seq"] = put(np.repeat(np.arange(len(n)), n))
        st["row_pos"] = put(np.concatenate([np.arange(x) for x in n]))
        st["scale"] = 1.0 / math.sqrt(d)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((int(cu[-1]), hq), device=dev)
    st["lens"] = put(lens.astype(np.int32))
    st["host_lens"], st["host_n"] = lens, n
    st["k_pool"] = normal(blocks, hkv, BLOCK, d).to(torch.bfloat16)
    if case["op"] == "tree":
        words = -(-st["max_n"] // 64)
        st["mask"] = put(np.concatenate([_tree_bits(int(x), r, words) for x in n]))
    if case["op"] == "mass":
        # the log-sum-exp that attention over the same rows gave: scores of
        # N(0, 1) keys have variance |q|^2 / d, so it is near log(L) + |q|^2 / 2d
        qn = st["q"].float().square().sum(-1) * (0.5 / d)
        length = st["lens"].float()[st["row_seq"]]
        st["lse"] = length.log()[:, None] + qn + 0.1 * normal(*qn.shape)
        st["mass_in"] = torch.rand((case["seqs"], hkv, case["hi"]), generator=g, device=dev)
        st["mass_in"] *= 16.0 / case["hi"]  # what a few earlier steps left
        st["mass_out"] = torch.zeros_like(st["mass_in"])
    else:
        st["v_pool"] = normal(blocks, hkv, BLOCK, d).to(torch.bfloat16)
    return st


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------
def _plain_rotate(x, st):
    """Rotation of the leading ``rot`` dims of fp32 rows [T, H, D]."""
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    a = st["positions"].double()[:, None] * st["inv_freq"]
    c = (torch.cos(a) * st["factor"]).float()[:, None]
    s = (torch.sin(a) * st["factor"]).float()[:, None]
    if case["interleaved"]:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)
    else:
        x0, x1 = x[..., :half], x[..., half:rot]
        y = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def _plain_norm(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_pages(pool, st):
    """Every sequence's rows of a pool, padded: fp32 [S, Hkv, tokens, D]."""
    nb = -(-int(st["host_lens"].max()) // BLOCK)
    ids = st["tables"][:, :nb].long()
    ids = torch.where(ids < pool.shape[0], ids, torch.zeros_like(ids))
    x = pool[ids].float()  # [S, nb, Hkv, 16, D]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], nb * BLOCK, x.shape[4])


def _plain_scores(st):
    """Scaled scores [S, Hkv, G, n, tokens], and the padded rows' index [S, n]."""
    case = st["case"]
    nseq, nmax, hq, hkv = case["seqs"], st["max_n"], case["hq"], case["hkv"]
    q = torch.zeros((nseq, nmax, hq, case["dim"]), device=st["q"].device)
    q[st["row_seq"], st["row_pos"]] = st["q"].float()
    q = q.reshape(nseq, nmax, hkv, hq // hkv, -1).permute(0, 2, 3, 1, 4)
    k = _plain_pages(st["k_pool"], st)
    x = torch.matmul(q.reshape(nseq, hkv, -1, case["dim"]), k.transpose(2, 3)) * st["scale"]
    return x.reshape(nseq, hkv, hq // hkv, nmax, k.shape[2])


def _run_plain(st):
    case, op = st["case"], st["op"]
    if op == "rope":
        return {"q": _plain_rotate(st["q"].float(), st), "k": _plain_rotate(st["k"].float(), st)}
    if op == "norm_rope":
        q = _plain_rotate(_plain_norm(st["q"], st["qw"]), st)
        k = _plain_rotate(_plain_norm(st["k"], st["kw"]), st)
        ok = st["slots"] >= 0
        at = st["slots"][ok]
        st["k_pool"][at // BLOCK, :, at % BLOCK] = k[ok]
        st["v_pool"][at // BLOCK, :, at % BLOCK] = st["v"][ok]
        return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if op == "evict":
        m, lens = st["mass"], st["lens"].long()
        keep = torch.minimum(lens, st["budgets"].long())
        t = torch.arange(m.shape[2], device=m.device)
        sink = torch.clamp(keep, max=case["sink"])[:, None, None]
        recent = torch.minimum(keep, torch.clamp(keep - sink[:, 0, 0], max=case["recent"]))[:, None, None]
        ln = lens[:, None, None]
        forced = (t < sink) | ((t >= ln - recent) & (t < ln))
        rank = torch.where(forced, torch.full_like(m, float("inf")), m)
        rank = torch.where(t < ln, rank, torch.full_like(m, -float("inf")))
        order = torch.sort(rank, dim=2, descending=True, stable=True).indices
        place = torch.arange(m.shape[2], device=m.device)
        chosen = torch.where(place < keep[:, None, None], order, torch.full_like(order, m.shape[2]))
        chosen = torch.sort(chosen, dim=2).values[:, :, :case["keep"]]
        live = chosen < m.shape[2]
        src = torch.where(live, chosen, torch.zeros_like(chosen))
        kept = torch.where(live, chosen, torch.full_like(chosen, -1)).to(torch.int32)
        mass = torch.where(live, torch.gather(m, 2, src), torch.zeros_like(m[:, :, :1]))
        s, h, i = torch.nonzero(live, as_tuple=True)
        at = src[s, h, i]
        sb = st["tables"][s, at // BLOCK].long()
        db = st["new_tables"][s, i // BLOCK].long()
        st["k_pool"][db, h, i % BLOCK] = st["k_pool"][sb, h, at % BLOCK]
        st["v_pool"][db, h, i % BLOCK] = st["v_pool"][sb, h, at % BLOCK]
        return {"kept": kept, "lens": keep.to(torch.int32), "mass": mass,
                "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    x = _plain_scores(st)
    tok = torch.arange(x.shape[-1], device=x.device)
    lens = st["lens"].long()
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    rel = tok[None, :] - (lens - n)[:, None]  # [S, tokens]: index among the new tokens
    if op == "mass":
        row = torch.arange(st["max_n"], device=x.device)
        see = (rel[:, None, :] <= row[:, None]) & (row[:, None] < n[:, None, None])
        lse = torch.full((case["seqs"], st["max_n"], case["hq"]), float("inf"), device=x.device)
        lse[st["row_seq"], st["row_pos"]] = st["lse"]
        lse = lse.reshape(case["seqs"], st["max_n"], case["hkv"], -1).permute(0, 2, 3, 1)
        w = torch.exp(x - lse[..., None])
        w = torch.where(see[:, None, None], w, torch.zeros_like(w)).sum((2, 3))
        width = min(w.shape[2], st["mass_in"].shape[2])
        live = tok[:width] < lens[:, None, None]
        new = st["mass_in"][:, :, :width] + w[:, :, :width]
        st["mass_out"][:, :, :width] = torch.where(live, new, st["mass_out"][:, :, :width])
        return {"mass": st["mass_out"]}
    # tree: cached tokens are seen by all, drafted ones by the mask's bits
    words = torch.zeros((case["seqs"], st["max_n"], st["mask"].shape[1]), dtype=torch.int64,
                        device=x.device)
    words[st["row_seq"], st["row_pos"]] = st["mask"]
    bit = torch.clamp(rel, min=0, max=64 * words.shape[2] - 1)  # [S, tokens]
    word = torch.gather(words, 2, (bit // 64)[:, None, :].expand(-1, words.shape[1], -1))
    drafted = ((word >> (bit % 64)[:, None, :]) & 1).bool()
    see = ((rel < 0)[:, None, :] | drafted) & (tok < lens[:, None])[:, None, :]
    see = see[:, None, None]
    x = torch.where(see, x, torch.full_like(x, -float("inf")))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -float("inf"), torch.zeros_like(top), top))
    z = p.sum(-1, keepdim=True)
    v = _plain_pages(st["v_pool"], st)
    o = torch.matmul(p.flatten(2, 3), v).reshape(*p.shape[:4], -1)
    o = o / torch.where(z > 0, z, torch.ones_like(z))
    lse = (top + torch.log(z))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(case["seqs"], st["max_n"], case["hq"], -1)
    lse = lse.permute(0, 3, 1, 2).reshape(case["seqs"], st["max_n"], case["hq"])
    at = (st["row_seq"], st["row_pos"])
    return {"out": o[at].to(torch.bfloat16), "lse": lse[at]}


# ----------------------------------------------------------------------------
# The framework's calls
# ----------------------------------------------------------------------------
def _run_own(st):
    import paged_kv_cache_454_b200 as pa
    case, op = st["case"], st["op"]
    if op == "rope":
        q, k = pa.pa_rope(st["q"], st["k"], st["positions"], st["inv_freq"],
                          interleaved=case["interleaved"], factor=st["factor"],
                          q_out=st["q_out"], k_out=st["k_out"])
        return {"q": q, "k": k}
    if op == "norm_rope":
        q = pa.pa_rope_and_cache(st["q"], st["k"], st["v"], st["k_pool"], st["v_pool"],
                                 st["slots"], st["positions"], st["inv_freq"],
                                 interleaved=case["interleaved"], factor=st["factor"],
                                 q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
                                 q_out=st["q_out"])
        return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if op == "tree":
        out, lse = pa.pa_tree_attention(st["q"], st["cu"], st["max_n"], st["mask"], st["k_pool"],
                                        st["v_pool"], st["tables"], st["lens"], st["scale"],
                                        out=st["out"], lse=st["lse"])
        return {"out": out, "lse": lse}
    if op == "mass":
        mass = pa.pa_attention_mass(st["q"], st["lse"], st["cu"], st["max_n"], st["k_pool"],
                                    st["tables"], st["lens"], st["scale"],
                                    mass_in=st["mass_in"], mass=st["mass_out"])
        return {"mass": mass}
    kept, lens, mass = pa.pa_evict(st["mass"], st["k_pool"], st["v_pool"], st["tables"],
                                   st["lens"], st["budgets"], sink=case["sink"],
                                   recent=case["recent"], new_tables=st["new_tables"],
                                   kept=st["kept"], new_lens=st["new_lens"],
                                   mass_out=st["mass_out"])
    return {"kept": kept, "lens": lens, "mass": mass, "k_pool": st["k_pool"],
            "v_pool": st["v_pool"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    d, hkv = case["dim"], case["hkv"]
    if case["op"] in ("rope", "norm_rope"):
        t, hq, rot = case["tokens"], case["hq"], case["rot"]
        rows = hq + hkv + (hkv if case["op"] == "norm_rope" else 0)
        extra = 8 * t + 8 * (rot // 2) + ((8 * t + 4 * d) if case["op"] == "norm_rope" else 0)
        norm = 4 * d if case["op"] == "norm_rope" else 0
        return {"bytes": 2 * 2 * rows * t * d + extra, "flops": t * (hq + hkv) * (3 * rot + norm)}
    lens, n = _spread(case)
    total, rows = int(lens.sum()), int(n.sum())
    if case["op"] == "evict":
        kept = int(np.minimum(lens, case["keep"]).sum())
        return {"bytes": hkv * (4 * total + 8 * kept + 2 * 4 * d * kept) + (total + kept) / 4,
                "flops": 0.0}
    hq = case["hq"]
    # a query's products reach its whole context but for about half the new tokens
    pairs = hq * d * float((n * (lens - n / 2)).sum())
    io = 2 * rows * hq * d
    if case["op"] == "mass":
        return {"bytes": total * hkv * (2 * d + 8) + io + 4 * rows * hq + total / 4,
                "flops": 2 * pairs}
    return {"bytes": total * hkv * 4 * d + 2 * io + 4 * rows * hq + 8 * rows + total / 4,
            "flops": 4 * pairs}


# ----------------------------------------------------------------------------
# The definitions in 64 bits, one sequence (or tensor) at a time
# ----------------------------------------------------------------------------
def _exact_rotated(x, case, positions, freq, factor):
    """Each pair of fp64 rows [T, H, D] as a complex number times factor * e^(i angle)."""
    rot = case["rot"]
    turn = factor * torch.exp(1j * positions.double()[:, None, None] * freq)
    y = x.clone()
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous())
        y[..., :rot] = torch.view_as_real(z * turn).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "norm_rope"):
        q, k = st["q"].double(), st["k"].double()
        if op == "norm_rope":
            q = q / q.square().mean(-1, keepdim=True).add(1e-6).sqrt() * st["qw"].double()
            k = k / k.square().mean(-1, keepdim=True).add(1e-6).sqrt() * st["kw"].double()
        q = _exact_rotated(q, case, st["positions"], st["inv_freq"], st["factor"])
        k = _exact_rotated(k, case, st["positions"], st["inv_freq"], st["factor"])
        if op == "rope":
            return {"q": q, "k": k}
        pool = st["k_pool"].double()
        flat = pool.permute(0, 2, 1, 3).reshape(-1, case["hkv"], case["dim"])
        live = torch.nonzero(st["slots"] >= 0)[:, 0]
        flat[st["slots"][live]] = k[live]
        pool = flat.reshape(-1, BLOCK, case["hkv"], case["dim"]).permute(0, 2, 1, 3)
        return {"q": q, "k_pool": pool.contiguous(), "v_pool": None}
    if op == "evict":
        return None  # whole numbers and moved values: nothing is computed
    lens, n = st["host_lens"], st["host_n"]
    group = case["hq"] // case["hkv"]
    row = 0
    outs, lses = [], []
    mass = st["mass_out"].double() if op == "mass" else None
    for s in range(case["seqs"]):
        L, c, m = int(lens[s]), int(lens[s] - n[s]), int(n[s])
        ids = st["tables"][s, :-(-L // BLOCK)].long()
        k = st["k_pool"][ids].double().transpose(1, 2).flatten(0, 1)[:L]
        q = st["q"][row:row + m].double().unflatten(1, (case["hkv"], group))
        x = torch.einsum("ihgd,thd->ihgt", q, k) * st["scale"]
        i = torch.arange(m, device=x.device)[:, None]
        j = torch.arange(L, device=x.device)[None, :] - c
        if op == "mass":
            e = st["lse"][row:row + m].double().unflatten(1, (case["hkv"], group))
            w = torch.exp(x - e[..., None]).masked_fill((j > i)[:, None, None], 0.0)
            mass[s, :, :L] = st["mass_in"][s, :, :L].double() + w.sum((0, 2))
        else:
            v = st["v_pool"][ids].double().transpose(1, 2).flatten(0, 1)[:L]
            bits = np.unpackbits(st["mask"][row:row + m].cpu().numpy().view(np.uint8), axis=1,
                                 bitorder="little")[:, :m].astype(bool)
            see = torch.ones((m, L), dtype=torch.bool, device=x.device)
            see[:, c:] = torch.from_numpy(bits).to(x.device)
            x = x.masked_fill(~see[:, None, None], -float("inf"))
            lse = torch.logsumexp(x, -1)
            outs.append(torch.einsum("ihgt,thd->ihgd", torch.exp(x - lse[..., None]), v).flatten(1, 2))
            lses.append(lse.flatten(1))
        row += m
    if op == "mass":
        return {"mass": mass}
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
