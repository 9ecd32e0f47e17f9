"""PagedAttention over a block-paged KV pool, for NVIDIA B200 (sm_100a).

The work runs in ``libpa.so`` (hand-written CUDA, C ABI in ``include/pa.h``).
This module only marshals torch tensors (device memory, streams) into that ABI;
the function names are the C names.  There is no fallback: if the library is
missing or a tensor is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _abi
from ._abi import (PA_DEV_ERR_BLOCK_ID, PA_DEV_ERR_CONTEXT, PA_DEV_ERR_SLOT,  # noqa: F401
                   PA_DEV_ERR_TIMEOUT, PA_KERNEL_AUTO, PA_KERNEL_SIMT, PA_KERNEL_TCGEN05,
                   PA_PREFILL_EXACT_WEIGHTS, PA_ROPE_SCALE_BASE, PA_ROPE_SCALE_LINEAR,
                   PA_ROPE_SCALE_NONE, PA_ROPE_SCALE_RAMP, PaError, PoolDesc)

__all__ = [
    "pa_reshape_and_cache", "pa_copy_blocks", "pa_decode", "pa_decode_workspace_size",
    "pa_decode_noalloc",
    "pa_chunked_prefill", "pa_gather_kv", "pa_get_device_error", "pa_sample", "pa_swap_blocks",
    "pa_read_probe",
    "pa_rope", "pa_rope_and_cache", "pa_rope_frequencies",
    "pa_tree_attention", "pa_tree_workspace_size",
    "pa_attention_mass", "pa_evict", "pa_compact_tokens",
    "pool_desc", "lib",
    "PaError", "PA_KERNEL_AUTO", "PA_KERNEL_SIMT", "PA_KERNEL_TCGEN05",
    "PA_PREFILL_EXACT_WEIGHTS",
    "PA_ROPE_SCALE_NONE", "PA_ROPE_SCALE_LINEAR", "PA_ROPE_SCALE_BASE", "PA_ROPE_SCALE_RAMP",
]


def lib():
    return _abi.load()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _need_cuda(name, t, dtype=None, contiguous=True):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def pool_desc(k_pool) -> PoolDesc:
    """Descriptor of a ``[num_blocks, num_kv_heads, block_size, head_dim]`` pool."""
    nb, hkv, bs, d = k_pool.shape
    return PoolDesc(nb, hkv, bs, d)


def _check_pools(k_pool, v_pool):
    torch = _torch()
    _need_cuda("k_pool", k_pool, torch.bfloat16)
    _need_cuda("v_pool", v_pool, torch.bfloat16)
    if k_pool.dim() != 4 or k_pool.shape != v_pool.shape:
        raise ValueError("k_pool and v_pool must be [num_blocks, Hkv, block_size, D] alike")


def _row_stride(name, t):
    """Token stride (elements) of a [T, H, D] tensor whose heads are packed."""
    if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
        raise ValueError(f"{name} must be [T, H, D] with packed heads")
    return t.stride(0)


def pa_reshape_and_cache(key, value, k_pool, v_pool, slot_mapping, stream=None) -> None:
    """Write new tokens' K/V (bf16 [T, Hkv, D]) into the pools at ``slot_mapping``
    (int64 [T]; negative = skip)."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    _need_cuda("key", key, torch.bfloat16, contiguous=False)
    _need_cuda("value", value, torch.bfloat16, contiguous=False)
    _need_cuda("slot_mapping", slot_mapping, torch.int64)
    ks, vs = _row_stride("key", key), _row_stride("value", value)
    if ks != vs:
        raise ValueError("key and value must share a token stride")
    _abi.check("pa_reshape_and_cache", lib().pa_reshape_and_cache(
        _ptr(key), _ptr(value), ks, _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool),
        _ptr(slot_mapping), key.shape[0], _stream(stream)))


def pa_copy_blocks(k_pool, v_pool, pairs, stream=None) -> None:
    """Copy whole blocks src -> dst in both pools.  ``pairs``: host int64 [P, 2]."""
    _check_pools(k_pool, v_pool)
    arr = np.ascontiguousarray(np.asarray(pairs, dtype=np.int64).reshape(-1, 2))
    _abi.check("pa_copy_blocks", lib().pa_copy_blocks(
        _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool),
        arr.ctypes.data_as(ctypes.c_void_p), arr.shape[0], _stream(stream)))


def pa_decode_workspace_size(num_seqs, num_q_heads, k_pool, max_blocks_per_seq,
                             partition_tokens=0) -> int:
    return int(lib().pa_decode_workspace_size_ex(num_seqs, num_q_heads, pool_desc(k_pool),
                                                 max_blocks_per_seq, partition_tokens))


def pa_decode(q, k_pool, v_pool, block_tables, context_lens, scale, out=None, lse=None,
              workspace=None, partition_tokens=0, kernel=PA_KERNEL_AUTO, stream=None,
              want_lse=False):
    """Single-query paged attention.  ``q`` bf16 [S, Hq, D]; ``block_tables`` int32
    [S, max_blocks]; ``context_lens`` int32 [S].  Returns ``(out, lse)``; ``lse``
    is None unless given or ``want_lse``."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    _need_cuda("q", q, torch.bfloat16, contiguous=False)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    S, hq, d = q.shape
    qs = _row_stride("q", q)
    if out is None:
        out = torch.empty((S, hq, d), dtype=torch.bfloat16, device=q.device)
    _need_cuda("out", out, torch.bfloat16)
    if lse is None and want_lse:
        lse = torch.empty((S, hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_cuda("lse", lse, torch.float32)
    mb = block_tables.shape[1]
    if workspace is None:
        n = pa_decode_workspace_size(S, hq, k_pool, mb, partition_tokens)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    _need_cuda("workspace", workspace, torch.uint8)
    _abi.check("pa_decode_ex", lib().pa_decode_ex(
        _ptr(q), qs, _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool), _ptr(block_tables), mb,
        _ptr(context_lens), S, hq, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), int(partition_tokens), int(kernel), _stream(stream)))
    return out, lse


def pa_decode_noalloc(q, k_pool, v_pool, block_tables, context_lens, scale, out=None, lse=None,
                      stream=None, want_lse=False):
    """``pa_decode`` for callers that cannot allocate device memory: the split
    scratch comes from a fixed array inside the library (``_abi.PA_NOALLOC_SCRATCH_BYTES``
    per device, shared by all calls on the device, so calls must not overlap on
    the GPU).  This wrapper itself allocates ``out``/``lse`` only when they are
    not given."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    _need_cuda("q", q, torch.bfloat16, contiguous=False)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    S, hq, d = q.shape
    qs = _row_stride("q", q)
    if out is None:
        out = torch.empty((S, hq, d), dtype=torch.bfloat16, device=q.device)
    _need_cuda("out", out, torch.bfloat16)
    if lse is None and want_lse:
        lse = torch.empty((S, hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_cuda("lse", lse, torch.float32)
    _abi.check("pa_decode_noalloc", lib().pa_decode_noalloc(
        _ptr(q), qs, _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool), _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), S, hq, float(scale), _ptr(out), _ptr(lse),
        _stream(stream)))
    return out, lse


def pa_chunked_prefill(q, cu_q_lens, max_q_len, k_pool, v_pool, block_tables, context_lens,
                       scale, out=None, lse=None, stream=None, want_lse=False,
                       exact_weights=False):
    """Causal attention of each sequence's new chunk over its cached context plus
    itself.  ``q`` bf16 [total_q, Hq, D]; ``cu_q_lens`` int32 [S+1] (device).
    ``exact_weights`` asks for the weights' bf16 remainder on every key tile
    (``pa_chunked_prefill_ex`` with ``PA_PREFILL_EXACT_WEIGHTS``)."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    _need_cuda("q", q, torch.bfloat16, contiguous=False)
    _need_cuda("cu_q_lens", cu_q_lens, torch.int32)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    total_q, hq, d = q.shape
    qs = _row_stride("q", q)
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=torch.bfloat16, device=q.device)
    _need_cuda("out", out, torch.bfloat16)
    if lse is None and want_lse:
        lse = torch.empty((total_q, hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_cuda("lse", lse, torch.float32)
    S = context_lens.shape[0]
    if exact_weights:
        _abi.check("pa_chunked_prefill_ex", lib().pa_chunked_prefill_ex(
            _ptr(q), qs, _ptr(cu_q_lens), total_q, int(max_q_len), _ptr(k_pool), _ptr(v_pool),
            pool_desc(k_pool), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), S,
            hq, float(scale), _ptr(out), _ptr(lse), PA_PREFILL_EXACT_WEIGHTS, _stream(stream)))
    else:
        _abi.check("pa_chunked_prefill", lib().pa_chunked_prefill(
            _ptr(q), qs, _ptr(cu_q_lens), total_q, int(max_q_len), _ptr(k_pool), _ptr(v_pool),
            pool_desc(k_pool), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), S,
            hq, float(scale), _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


def pa_gather_kv(k_pool, v_pool, block_tables, context_lens, cu_kv_lens, max_context,
                 total_tokens, stream=None):
    """Contiguous copies ``[total_tokens, Hkv, D]`` of every sequence's K and V."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    _need_cuda("cu_kv_lens", cu_kv_lens, torch.int32)
    _, hkv, _, d = k_pool.shape
    k_out = torch.empty((total_tokens, hkv, d), dtype=torch.bfloat16, device=k_pool.device)
    v_out = torch.empty_like(k_out)
    _abi.check("pa_gather_kv", lib().pa_gather_kv(
        _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), _ptr(cu_kv_lens), context_lens.shape[0], int(max_context),
        _ptr(k_out), _ptr(v_out), _stream(stream)))
    return k_out, v_out


def pa_get_device_error(stream=None) -> int:
    """Wait for ``stream`` and return-and-clear the device error word."""
    v = ctypes.c_uint32(0)
    _abi.check("pa_get_device_error", lib().pa_get_device_error(ctypes.byref(v), _stream(stream)))
    return int(v.value)


def pa_sample(logits, temperature, top_k, top_p, uniform, out=None, stream=None):
    """Fused temperature / Top-K / Top-P sampling, one token per row of ``logits``
    (fp32 [rows, vocab], rows contiguous).  ``temperature``, ``top_p``, ``uniform``:
    fp32 [rows]; ``top_k``: int32 [rows]; all CUDA tensors.  Returns int32 [rows]."""
    torch = _torch()
    _need_cuda("logits", logits, torch.float32, contiguous=False)
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [rows, vocab] with unit stride along the vocabulary")
    rows, vocab = logits.shape
    for name, t, dt in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("uniform", uniform, torch.float32)):
        _need_cuda(name, t, dt)
        if t.shape != (rows,):
            raise ValueError(f"{name} must have shape ({rows},)")
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=logits.device)
    _need_cuda("out", out, torch.int32)
    _abi.check("pa_sample", lib().pa_sample(
        _ptr(logits), logits.stride(0), rows, vocab, _ptr(temperature), _ptr(top_k),
        _ptr(top_p), _ptr(uniform), _ptr(out), _stream(stream)))
    return out


def pa_swap_blocks(k_pool, v_pool, k_host, v_host, pairs, direction, stream=None) -> None:
    """Copy whole blocks between the device pools and page-locked host pools of
    the same block shape (``k_host``/``v_host``: pinned CPU tensors).
    ``direction``: ``_abi.PA_SWAP_OUT`` (device src -> host dst) or
    ``_abi.PA_SWAP_IN`` (host src -> device dst); ``pairs``: int64 [P, 2]."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    for name, t in (("k_host", k_host), ("v_host", v_host)):
        if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_pinned():
            raise TypeError(f"{name} must be a pinned CPU tensor")
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or t.shape[1:] != k_pool.shape[1:]:
            raise ValueError(f"{name} must be bf16 [num_host_blocks, {tuple(k_pool.shape[1:])}]")
    arr = np.ascontiguousarray(np.asarray(pairs, dtype=np.int64).reshape(-1, 2))
    _abi.check("pa_swap_blocks", lib().pa_swap_blocks(
        _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool), _ptr(k_host), _ptr(v_host),
        k_host.shape[0], arr.ctypes.data_as(ctypes.c_void_p), arr.shape[0], int(direction),
        _stream(stream)))


def pa_read_probe(k_pool, v_pool, block_tables, context_lens, num_ctas=None, out=None,
                  stream=None):
    """Read every K/V page a decode over ``block_tables`` / ``context_lens``
    reads, and nothing else (a read-bandwidth measurement).  Returns the
    per-CTA sums (int64 [num_ctas], the bits of uint64 sums modulo 2^64) of the
    pages' 32-bit words; ``num_ctas`` defaults to the SM count."""
    torch = _torch()
    _check_pools(k_pool, v_pool)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    if block_tables.dim() != 2 or block_tables.shape[0] != context_lens.shape[0]:
        raise ValueError("block_tables must be [S, max_blocks] with S = len(context_lens)")
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(k_pool.device).multi_processor_count
    if out is None:
        out = torch.empty(num_ctas, dtype=torch.int64, device=k_pool.device)
    _need_cuda("out", out, torch.int64)
    if out.numel() < num_ctas:
        raise ValueError("out holds fewer than num_ctas sums")
    _abi.check("pa_read_probe", lib().pa_read_probe(
        _ptr(k_pool), _ptr(v_pool), pool_desc(k_pool), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), context_lens.shape[0], _ptr(out), int(num_ctas), _stream(stream)))
    return out


# ----------------------------------------------------------------------------
# Drafting and eviction (include/pa_rope.h, include/pa_tree.h, include/pa_evict.h)
#
# These calls run on the device their tensors are on (whatever the current one)
# and, without a `stream`, on that device's current stream; what they allocate
# belongs to the stream they run on.
# ----------------------------------------------------------------------------
def _arg(name, t, dtype, device, shape=None, contiguous=True):
    """Check one tensor argument (``shape``: the sizes it must have).  One pass of
    cheap comparisons; the words for what is wrong are found only then."""
    try:
        if (t.dtype is dtype and t.get_device() == device.index
                and (shape is None or t.shape == shape)
                and (not contiguous or t.is_contiguous())):
            return
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dims(name, t, dims):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {list(t.shape)}")


def _rows_arg(name, t, device, shape=None):
    """A bf16 [T, H, D] tensor whose heads are packed (``shape``: the sizes it must
    have); returns its token stride."""
    _arg(name, t, _torch().bfloat16, device, shape, contiguous=False)
    if shape is None:
        _dims(name, t, 3)
        shape = t.shape
    tokens, heads, dim = shape
    if t.is_contiguous():
        return heads * dim
    stride, by_head, by_dim = t.stride()
    if (by_dim != 1 and dim > 1) or (by_head != dim and heads > 1):
        raise ValueError(f"{name} must be [T, H, D] with packed heads")
    return stride if tokens > 1 else max(stride, heads * dim)


def _empty(shape, dtype, device, stream):
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_entry_points = {}


def _run(name, device, stream, *args):
    """Call ``name`` of the library with the stream's handle as its last argument."""
    fn = _entry_points.get(name)
    if fn is None:
        fn = _entry_points[name] = getattr(_abi.load(), name)
    cuda = _torch()._C
    if stream is None:
        handle = cuda._cuda_getCurrentRawStream(device.index)
    else:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        handle = stream.cuda_stream
    if device.index == cuda._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with _torch().cuda.device(device):
            status = fn(*args, handle)
    if status:
        _abi.check(name, status)


def pa_rope_frequencies(rot_dim, base=10000.0, scaling=_abi.PA_ROPE_SCALE_NONE, scale=1.0,
                        original_max_position=0.0, low_turns=1.0, high_turns=32.0):
    """Inverse frequencies (NumPy float64 [rot_dim / 2]) and the factor that goes with
    them, for ``pa_rope``; ``scaling``: one of ``PA_ROPE_SCALE_*``."""
    out = np.empty(max(int(rot_dim), 0) // 2, np.float64)
    factor = ctypes.c_double(1.0)
    _abi.check("pa_rope_frequencies", lib().pa_rope_frequencies(
        int(rot_dim), float(base), int(scaling), float(scale), float(original_max_position),
        float(low_turns), float(high_turns), out.ctypes.data_as(ctypes.c_void_p),
        ctypes.byref(factor)))
    return out, factor.value


def pa_rope(q, k, positions, inv_freq, interleaved=False, factor=1.0, q_out=None, k_out=None,
            stream=None):
    """Rotate ``q`` (bf16 [T, Hq, D]) and ``k`` (bf16 [T, Hkv, D], or None) by their
    tokens' ``positions`` (int64 [T]) and ``inv_freq`` (float64 [rot_dim / 2]; the
    first ``rot_dim`` dims of a head are rotated).  ``q_out`` / ``k_out`` may be the
    inputs.  Returns ``(q_out, k_out)``."""
    torch = _torch()
    dev = q.device
    qs = _rows_arg("q", q, dev)
    tokens, hq, d = q.shape
    _arg("positions", positions, torch.int64, dev, (tokens,))
    _arg("inv_freq", inv_freq, torch.float64, dev)
    _dims("inv_freq", inv_freq, 1)
    if q_out is None:
        q_out = _empty((tokens, hq, d), torch.bfloat16, dev, stream)
    qos = _rows_arg("q_out", q_out, dev, (tokens, hq, d))
    hkv = ks = kos = 0
    if k is not None:
        ks = _rows_arg("k", k, dev)
        hkv = k.shape[1]
        if k.shape != (tokens, hkv, d):
            raise ValueError(f"k must be [{tokens}, Hkv, {d}], got {list(k.shape)}")
        if k_out is None:
            k_out = _empty((tokens, hkv, d), torch.bfloat16, dev, stream)
        kos = _rows_arg("k_out", k_out, dev, (tokens, hkv, d))
    elif k_out is not None:
        raise ValueError("k_out without k")
    _run("pa_rope", dev, stream, q.data_ptr(), qs, q_out.data_ptr(), qos, hq, _ptr(k), ks,
         _ptr(k_out), kos, hkv, d, positions.data_ptr(), inv_freq.data_ptr(),
         2 * inv_freq.shape[0], int(bool(interleaved)), float(factor), tokens)
    return q_out, k_out


def pa_rope_and_cache(q, key, value, k_pool, v_pool, slot_mapping, positions, inv_freq,
                      interleaved=False, factor=1.0, q_weight=None, k_weight=None, eps=1e-6,
                      q_out=None, stream=None):
    """Norm each head of ``q`` and ``key`` (where a bf16 [D] weight is given), rotate
    them as ``pa_rope`` does, write the prepared key and ``value`` into the pools at
    ``slot_mapping`` (int64 [T]; negative = skip) and return the prepared q
    (``q_out`` may be ``q``)."""
    torch = _torch()
    dev = q.device
    bf16 = torch.bfloat16
    _arg("k_pool", k_pool, bf16, dev)
    _dims("k_pool", k_pool, 4)
    _arg("v_pool", v_pool, bf16, dev, k_pool.shape)
    qs = _rows_arg("q", q, dev)
    tokens, hq, d = q.shape
    desc = pool_desc(k_pool)
    hkv = desc.num_kv_heads
    if desc.head_dim != d:
        raise ValueError(f"q has head_dim {d}, the pools {desc.head_dim}")
    ks = _rows_arg("key", key, dev, (tokens, hkv, d))
    vs = _rows_arg("value", value, dev, (tokens, hkv, d))
    _arg("slot_mapping", slot_mapping, torch.int64, dev, (tokens,))
    _arg("positions", positions, torch.int64, dev, (tokens,))
    _arg("inv_freq", inv_freq, torch.float64, dev)
    _dims("inv_freq", inv_freq, 1)
    if q_weight is not None:
        _arg("q_weight", q_weight, bf16, dev, (d,))
    if k_weight is not None:
        _arg("k_weight", k_weight, bf16, dev, (d,))
    if q_out is None:
        q_out = _empty((tokens, hq, d), bf16, dev, stream)
    qos = _rows_arg("q_out", q_out, dev, (tokens, hq, d))
    _run("pa_rope_and_cache", dev, stream, q.data_ptr(), qs, q_out.data_ptr(), qos, hq,
         key.data_ptr(), ks, value.data_ptr(), vs, _ptr(q_weight), _ptr(k_weight), float(eps),
         positions.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.shape[0],
         int(bool(interleaved)), float(factor), k_pool.data_ptr(), v_pool.data_ptr(),
         desc, slot_mapping.data_ptr(), tokens)
    return q_out


def _batch_args(k_pool, block_tables, context_lens, dev):
    """Checks shared by the calls that read a batch's cache: ``(desc, S, max_blocks)``."""
    torch = _torch()
    _arg("k_pool", k_pool, torch.bfloat16, dev)
    _dims("k_pool", k_pool, 4)
    _arg("context_lens", context_lens, torch.int32, dev)
    _dims("context_lens", context_lens, 1)
    _arg("block_tables", block_tables, torch.int32, dev)
    _dims("block_tables", block_tables, 2)
    seqs, blocks = block_tables.shape
    if context_lens.shape[0] != seqs:
        raise ValueError(f"{seqs} block tables for {context_lens.shape[0]} context lengths")
    return pool_desc(k_pool), seqs, blocks


def pa_tree_workspace_size(max_q_len, num_q_heads, k_pool) -> int:
    return int(_abi.load().pa_tree_workspace_size(int(max_q_len), int(num_q_heads),
                                                  pool_desc(k_pool)))


_tree_workspace = {}


def pa_tree_attention(q, cu_q_lens, max_q_len, tree_mask, k_pool, v_pool, block_tables,
                      context_lens, scale, out=None, lse=None, workspace=None, stream=None,
                      want_lse=False):
    """Attention of each sequence's drafted tokens (``q`` bf16 [total_q, Hq, D],
    ``cu_q_lens`` int32 [S+1] on the device) over its cached tokens and, among the
    drafted ones, those of the row's ``tree_mask`` (int64 [total_q, words], bit j of
    word j // 64 = drafted token j).  ``context_lens`` counts the drafted tokens,
    whose K and V are in the pools.  Returns ``(out, lse)``; ``lse`` is None unless
    given or ``want_lse``."""
    torch = _torch()
    dev = q.device
    qs = _rows_arg("q", q, dev)
    total_q, hq, d = q.shape
    desc, seqs, blocks = _batch_args(k_pool, block_tables, context_lens, dev)
    if desc.head_dim != d:
        raise ValueError(f"q has head_dim {d}, the pools {desc.head_dim}")
    _arg("v_pool", v_pool, torch.bfloat16, dev, k_pool.shape)
    _arg("cu_q_lens", cu_q_lens, torch.int32, dev, (seqs + 1,))
    _arg("tree_mask", tree_mask, torch.int64, dev)
    _dims("tree_mask", tree_mask, 2)
    if tree_mask.shape[0] != total_q:
        raise ValueError(f"tree_mask must have {total_q} rows, got {tree_mask.shape[0]}")
    if out is None:
        out = _empty((total_q, hq, d), torch.bfloat16, dev, stream)
    else:
        _arg("out", out, torch.bfloat16, dev, (total_q, hq, d))
    if lse is not None:
        _arg("lse", lse, torch.float32, dev, (total_q, hq))
    elif want_lse:
        lse = _empty((total_q, hq), torch.float32, dev, stream)
    if workspace is None:
        sizes = (int(max_q_len), hq, desc.num_kv_heads, d)
        n = _tree_workspace.get(sizes)  # (a function of these sizes alone)
        if n is None:
            n = _tree_workspace[sizes] = max(pa_tree_workspace_size(max_q_len, hq, k_pool), 16)
        workspace = _empty(n, torch.uint8, dev, stream)
    else:
        _arg("workspace", workspace, torch.uint8, dev)
    _run("pa_tree_attention", dev, stream, q.data_ptr(), qs, cu_q_lens.data_ptr(), total_q,
         int(max_q_len), tree_mask.data_ptr(), tree_mask.shape[1], k_pool.data_ptr(),
         v_pool.data_ptr(), desc, block_tables.data_ptr(), blocks, context_lens.data_ptr(), seqs,
         hq, float(scale), out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out, lse


def pa_attention_mass(q, lse, cu_q_lens, max_q_len, k_pool, block_tables, context_lens, scale,
                      mass_in=None, mass=None, stream=None, own_from_zero=False):
    """Add to every cached token the softmax weights that the rows of ``q`` (bf16
    [total_q, Hq, D], with the ``lse`` fp32 [total_q, Hq] their attention returned)
    gave it.  Query i of a sequence's n sees all but the last n - 1 - i tokens: of a
    tree only the accepted branch, packed by ``pa_compact_tokens``, is such a chain.
    ``cu_q_lens`` int32 [S+1] on the device, or None for a decode step (one row per
    sequence).  ``mass_in``: fp32 [S, Hkv, W] so far (None: zeros);
    ``mass``: where the sums go (may be ``mass_in``; default: a new tensor, zero
    past each sequence's length).  ``own_from_zero``: the tokens of this step start
    from 0 whatever ``mass_in`` holds for them (what an eviction in place or a rejected
    draft left); without it ``mass_in`` has to be 0 there.  Returns ``mass``."""
    torch = _torch()
    dev = q.device
    f32 = torch.float32
    qs = _rows_arg("q", q, dev)
    total_q, hq, d = q.shape
    desc, seqs, blocks = _batch_args(k_pool, block_tables, context_lens, dev)
    if desc.head_dim != d:
        raise ValueError(f"q has head_dim {d}, the pool {desc.head_dim}")
    _arg("lse", lse, f32, dev, (total_q, hq))
    if cu_q_lens is not None:
        _arg("cu_q_lens", cu_q_lens, torch.int32, dev, (seqs + 1,))
    if mass_in is not None:
        _arg("mass_in", mass_in, f32, dev)
        _dims("mass_in", mass_in, 3)
    if mass is None:
        shape = (seqs, desc.num_kv_heads,
                 blocks * desc.block_size if mass_in is None else mass_in.shape[2])
        mass = _empty(shape, f32, dev, stream)
        with torch.cuda.stream(stream):  # (None: the current one)
            mass.zero_()
    else:
        _arg("mass", mass, f32, dev)
        _dims("mass", mass, 3)
    width = mass.shape[2]
    if mass.shape != (seqs, desc.num_kv_heads, width) or (
            mass_in is not None and mass_in.shape != mass.shape):
        raise ValueError(f"mass and mass_in must be [{seqs}, {desc.num_kv_heads}, W] alike")
    _run("pa_attention_mass_ex", dev, stream, q.data_ptr(), qs, lse.data_ptr(), _ptr(cu_q_lens),
         total_q, int(max_q_len), k_pool.data_ptr(), desc, block_tables.data_ptr(), blocks,
         context_lens.data_ptr(), seqs, hq, float(scale), _ptr(mass_in), mass.data_ptr(), width,
         _abi.PA_MASS_OWN_FROM_ZERO if own_from_zero else 0)
    return mass


def pa_evict(mass, k_pool, v_pool, block_tables, context_lens, budgets, sink=0, recent=0,
             new_tables=None, kept=None, new_lens=None, mass_out=None, max_keep=None, stream=None):
    """Bring every sequence down to ``budgets`` (int32 [S]) tokens per KV head: the
    first ``sink``, the last ``recent`` and the heaviest others by ``mass`` (fp32
    [S, Hkv, W]), packed in order in place or into the blocks of ``new_tables``
    (int32 [S, blocks]).  Returns ``(kept, new_lens, mass_out)``: the kept tokens'
    indices (int32 [S, Hkv, K]), the new lengths (int32 [S]) and the kept tokens'
    weights; what is past a new length in ``kept`` and ``mass_out`` is not written.
    K comes from ``kept``, or else is ``max_keep`` (default: W), an upper bound of
    the budgets.  ``mass_out`` may be ``mass`` (evicted weights then stay behind the
    kept ones: ``own_from_zero`` of the next ``pa_attention_mass``); default: a new
    fp32 [S, Hkv, W], zero past each new length."""
    torch = _torch()
    dev = mass.device
    desc, seqs, blocks = _batch_args(k_pool, block_tables, context_lens, dev)
    _arg("v_pool", v_pool, torch.bfloat16, dev, k_pool.shape)
    _arg("mass", mass, torch.float32, dev)
    _dims("mass", mass, 3)
    hkv = desc.num_kv_heads
    width = mass.shape[2]
    if mass.shape != (seqs, hkv, width):
        raise ValueError(f"mass must be [{seqs}, {hkv}, W], got {list(mass.shape)}")
    _arg("budgets", budgets, torch.int32, dev, (seqs,))
    new_blocks = 0
    if new_tables is not None:
        _arg("new_tables", new_tables, torch.int32, dev)
        _dims("new_tables", new_tables, 2)
        if new_tables.shape[0] != seqs:
            raise ValueError(f"new_tables must have {seqs} rows, got {new_tables.shape[0]}")
        new_blocks = new_tables.shape[1]
    if kept is None:
        keep = width if max_keep is None else int(max_keep)
        kept = _empty((seqs, hkv, keep), torch.int32, dev, stream)
    else:
        _arg("kept", kept, torch.int32, dev)
        _dims("kept", kept, 3)
        keep = kept.shape[2]
        if kept.shape != (seqs, hkv, keep):
            raise ValueError(f"kept must be [{seqs}, {hkv}, K], got {list(kept.shape)}")
    if new_lens is None:
        new_lens = _empty((seqs,), torch.int32, dev, stream)
    else:
        _arg("new_lens", new_lens, torch.int32, dev, (seqs,))
    if mass_out is None:
        mass_out = _empty((seqs, hkv, width), torch.float32, dev, stream)
        with torch.cuda.stream(stream):  # (None: the current one)
            mass_out.zero_()
    else:
        _arg("mass_out", mass_out, torch.float32, dev)
        _dims("mass_out", mass_out, 3)
        if mass_out.shape[:2] != (seqs, hkv):
            raise ValueError(f"mass_out must be [{seqs}, {hkv}, K], got {list(mass_out.shape)}")
    _run("pa_evict", dev, stream, mass.data_ptr(), width, k_pool.data_ptr(), v_pool.data_ptr(),
         desc, block_tables.data_ptr(), blocks, context_lens.data_ptr(), budgets.data_ptr(),
         int(sink), int(recent), _ptr(new_tables), new_blocks, kept.data_ptr(), keep,
         new_lens.data_ptr(), mass_out.data_ptr(), mass_out.shape[2], seqs)
    return kept, new_lens, mass_out


def pa_compact_tokens(k_pool, v_pool, block_tables, kept, counts, base=None, new_tables=None,
                      stream=None) -> None:
    """Move K and V of row ``base[s] + kept[s][g][i]`` to row ``base[s] + i`` for every
    sequence, KV head and i < ``counts[s]`` (int32 [S]), in place or into the blocks of
    ``new_tables``.  ``kept``: int32 [S, Hkv, K], or [S, 1, K] for all heads alike,
    ascending in i; ``base``: int32 [S] or None (zeros)."""
    torch = _torch()
    dev = k_pool.device
    i32 = torch.int32
    _arg("counts", counts, i32, dev)
    desc, seqs, blocks = _batch_args(k_pool, block_tables, counts, dev)
    _arg("v_pool", v_pool, torch.bfloat16, dev, k_pool.shape)
    _arg("kept", kept, i32, dev)
    _dims("kept", kept, 3)
    if kept.shape[0] != seqs:
        raise ValueError(f"kept must have {seqs} rows, got {kept.shape[0]}")
    if base is not None:
        _arg("base", base, i32, dev, (seqs,))
    new_blocks = 0
    if new_tables is not None:
        _arg("new_tables", new_tables, i32, dev)
        _dims("new_tables", new_tables, 2)
        if new_tables.shape[0] != seqs:
            raise ValueError(f"new_tables must have {seqs} rows, got {new_tables.shape[0]}")
        new_blocks = new_tables.shape[1]
    _run("pa_compact_tokens", dev, stream, k_pool.data_ptr(), v_pool.data_ptr(), desc,
         block_tables.data_ptr(), blocks, _ptr(new_tables), new_blocks, _ptr(base),
         kept.data_ptr(), kept.shape[1], kept.shape[2], counts.data_ptr(), seqs)
