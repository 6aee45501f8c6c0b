"""Operators beside the decode path (``include/pkv_ops.h``): rotary positions on the
way into the cache, block-scaled E4M3 pools, and attention with capped scores, a
distance bias or a sliding window. Argument marshalling only, as the package's
other functions: a call that is in order goes through ``csrc/torch_marshal.cpp`` (about
1 us), anything else through the checks below, which say what is wrong (and make the
call themselves where the marshaller was not built).

    turns = rotary_turns(rotary_dim, base)                  # once, host
    rope_kv_append(q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache, q_out)
    rope_kv_append_fp8_block(..., k_cache, v_cache, k_scale, v_scale, q_out)
    paged_decode_attention_fp8_block(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                     context_lens, n_query_per_seq, scale, out)
    paged_decode_attention_scored(q, k_cache, v_cache, block_tables, context_lens,
                                  n_query_per_seq, scale, out, softcap=, alibi_slopes=,
                                  window=, k_scale=, v_scale=)

Block-scaled pools are uint8 ``[num_blocks, 16, Hkv, D]`` with uint8 scales
``[num_blocks, Hkv]`` (``2 ** (byte - 127)``; ``zero`` for a new pool). To copy
blocks (copy-on-write) of such a pool: ``copy_blocks(k_cache.view(torch.bfloat16),
v_cache.view(torch.bfloat16), src, dst)`` and the scale rows of the same blocks.
"""
from __future__ import annotations

import ctypes
import functools

import paged_kv_cache_101_gb300 as _pkv

_fast = None      # the C++ marshaller (csrc/torch_marshal.cpp), or False without it
_torch = None


def _load():
    """Load the marshaller and hand it the library's entry points."""
    global _fast, _torch
    _torch = _pkv._torch()
    lib = _pkv.lib()
    try:
        from . import _torch_marshal as fast
    except ImportError:
        _fast = False
        return _fast
    fast.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
        "pkv_rope_kv_append", "pkv_rope_kv_append_fp8_block", "pkv_paged_decode_attention_scored",
        "pkv_workspace_size_scored")))
    _fast = fast
    return _fast


def _here():
    """The current device and its current stream's handle."""
    dev = _torch._C._cuda_getDevice()
    return dev, _torch._C._cuda_getCurrentRawStream(dev)


_KINDS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3}


def rotary_turns(rotary_dim, base=10000.0, kind="plain", factor=1.0, original_length=1.0,
                 low=1.0, high=32.0):
    """The rotation frequencies as an int64 CPU tensor ``[rotary_dim / 2]`` (64-bit
    fixed point, see ``pkv_rotary_turns``); ``kind`` scales them for long contexts:
    ``"plain"``, ``"linear"``, ``"base"`` or ``"ramp"``."""
    torch = _pkv._torch()
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, got {kind!r}")
    out = torch.empty(max(int(rotary_dim) // 2, 1), dtype=torch.int64)
    st = _pkv.lib().pkv_rotary_turns(int(rotary_dim), float(base), _KINDS[kind], float(factor),
                                     float(original_length), float(low), float(high),
                                     out.data_ptr())
    if st != _pkv.PKV_OK:
        raise _pkv.PkvError("pkv_rotary_turns", st)
    return out


def _on_device(tensors):
    """All on the current CUDA device; returns its index."""
    torch = _pkv._torch()
    dev = torch.cuda.current_device()
    for name, t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"{name} is not on the current CUDA device (cuda:{dev})")
    return dev


def _rows(t, name, dtype):
    """[n, heads, D] with contiguous rows; the elements between two rows."""
    torch = _pkv._torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, got {tuple(t.shape)}")
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: the heads and dims of a row must be contiguous")
    return sn if n > 1 else h * d


def _rope(fn, q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache, scales, q_out,
          interleaved, rotary_scale):
    torch = _pkv._torch()
    k_stride = _rows(k_new, "k_new", torch.bfloat16)
    v_stride = _rows(v_new, "v_new", torch.bfloat16)
    check = _pkv._check
    check(positions, "positions", torch.int64, 1)
    check(turns, "turns", torch.int64, 1)
    check(slot_mapping, "slot_mapping", torch.int64, 1)
    pool = torch.uint8 if scales else torch.bfloat16
    check(k_cache, "k_cache", pool, 4)
    check(v_cache, "v_cache", pool, 4)
    NB, bs, Hkv, D = k_cache.shape
    if bs != _pkv.BLOCK_SIZE or v_cache.shape != k_cache.shape:
        raise ValueError("pools must be [num_blocks, 16, Hkv, D] and equal in shape")
    n = slot_mapping.shape[0]
    if (k_new.shape != (n, Hkv, D) or v_new.shape != k_new.shape
            or positions.shape[0] != n):
        raise ValueError("k_new/v_new must be [n_new, Hkv, D] matching the pool, with one slot and "
                         "one position per row")
    on = [("k_new", k_new), ("v_new", v_new), ("positions", positions), ("turns", turns),
          ("slot_mapping", slot_mapping), ("k_cache", k_cache), ("v_cache", v_cache)]
    if scales:
        for name, t in zip(("k_scale", "v_scale"), scales):
            check(t, name, torch.uint8, 2)
            if t.shape != (NB, Hkv):
                raise ValueError(f"{name} must be [num_blocks, Hkv]")
            on.append((name, t))
    if (q is None) != (q_out is None):
        raise ValueError("give q and q_out, or neither")
    if q is not None:
        q_stride = _rows(q, "q", torch.bfloat16)
        check(q_out, "q_out", torch.bfloat16, 3)
        Hq = q.shape[1]
        if q.shape != (n, Hq, D) or q_out.shape != q.shape:
            raise ValueError("q and q_out must be [n_new, Hq, D]")
        on += [("q", q), ("q_out", q_out)]
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    else:
        q_stride, Hq, q_ptr, out_ptr = 0, 0, None, None
    dev = _on_device(on)
    st = getattr(_pkv.lib(), fn)(
        q_ptr, q_stride, k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride,
        positions.data_ptr(), turns.data_ptr(), slot_mapping.data_ptr(), n, out_ptr,
        k_cache.data_ptr(), v_cache.data_ptr(), *[t.data_ptr() for t in scales], NB, Hq, Hkv, D,
        2 * turns.shape[0], 1 if interleaved else 0, float(rotary_scale),
        torch.cuda.current_stream(dev).cuda_stream)
    if st != _pkv.PKV_OK:
        raise _pkv.PkvError(fn, st)
    return q_out


def rope_kv_append(q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache, q_out,
                   interleaved=False, rotary_scale=1.0):
    """Rotate ``q`` ``[n, Hq, D]`` into ``q_out`` and ``k_new`` ``[n, Hkv, D]`` into its
    pool rows by ``positions`` (int64 ``[n]``); ``v_new`` goes to its rows as it is.
    ``turns``: ``rotary_turns(...)`` on the device, half as long as the rotated part of
    a head. q, k_new and v_new may be slices of one ``[n, ...]`` projection output;
    ``q`` and ``q_out`` None: keys and values only."""
    if _fast or _fast is None and _load():
        try:
            st = _fast.rope(q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache,
                            None, None, q_out, interleaved, rotary_scale, *_here())
        except RuntimeError:  # no device
            st = None
        if st == _pkv.PKV_OK:
            return q_out
    return _rope("pkv_rope_kv_append", q, k_new, v_new, positions, turns, slot_mapping, k_cache,
                 v_cache, (), q_out, interleaved, rotary_scale)


def rope_kv_append_fp8_block(q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache,
                             k_scale, v_scale, q_out, interleaved=False, rotary_scale=1.0):
    """``rope_kv_append`` into block-scaled E4M3 pools; updates ``k_scale``, ``v_scale``
    (uint8 ``[num_blocks, Hkv]``). The rows of one block follow one another."""
    if _fast or _fast is None and _load():
        try:
            st = None if k_scale is None else _fast.rope(
                q, k_new, v_new, positions, turns, slot_mapping, k_cache, v_cache, k_scale,
                v_scale, q_out, interleaved, rotary_scale, *_here())
        except RuntimeError:
            st = None
        if st == _pkv.PKV_OK:
            return q_out
    return _rope("pkv_rope_kv_append_fp8_block", q, k_new, v_new, positions, turns, slot_mapping,
                 k_cache, v_cache, (k_scale, v_scale), q_out, interleaved, rotary_scale)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(S, nq, Hq, Hkv, D, dev):
    return int(_pkv.lib().pkv_workspace_size_scored(S, nq, Hq, Hkv, D))


def workspace_size_scored(num_seqs, n_query_per_seq, num_q_heads, num_kv_heads, head_dim) -> int:
    """Bytes of workspace of the two attention calls for this geometry (0: unsupported)."""
    return int(_pkv.lib().pkv_workspace_size_scored(num_seqs, n_query_per_seq, num_q_heads,
                                                    num_kv_heads, head_dim))


_workspaces = {}


def _workspace(dev, stream, nbytes):
    """The workspace of calls that bring none: one per stream, so that calls on two
    streams never share it; under stream capture a new one, which the graph owns (two
    graphs, or a graph and later eager calls, may then run at the same time)."""
    torch = _pkv._torch()
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=f"cuda:{dev}")
    ws = _workspaces.get((dev, stream))
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=f"cuda:{dev}")
        _workspaces[(dev, stream)] = ws
    return ws


def _attend(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, n_query_per_seq,
            scale, out, softcap, alibi_slopes, window, ws):
    if _fast or _fast is None and _load():
        try:
            dev, stream = _here()
            if ws is None and not _torch.cuda.is_current_stream_capturing():
                use = _workspaces.get((dev, stream))
            else:
                use = ws
            st = _fast.attend(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                              n_query_per_seq, scale, out, softcap, alibi_slopes, window, use, dev,
                              stream)
        except RuntimeError:  # no device
            st = None
        if st == _pkv.PKV_OK:
            return out
    torch = _pkv._torch()
    check = _pkv._check
    check(q, "q", torch.bfloat16, 3)
    if (k_scale is None) != (v_scale is None):
        raise ValueError("give both scales (block-scaled E4M3 pools) or neither (bf16 pools)")
    pool = torch.bfloat16 if k_scale is None else torch.uint8
    check(k_cache, "k_cache", pool, 4)
    check(v_cache, "v_cache", pool, 4)
    check(block_tables, "block_tables", torch.int32, 2)
    check(context_lens, "context_lens", torch.int32, 1)
    if not isinstance(out, torch.Tensor) or out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be a bfloat16 or float32 tensor")
    check(out, "out", out.dtype, 3)
    NB, bs, Hkv, D = k_cache.shape
    if bs != _pkv.BLOCK_SIZE or v_cache.shape != k_cache.shape:
        raise ValueError("pools must be [num_blocks, 16, Hkv, D] and equal in shape")
    S = context_lens.shape[0]
    nq = int(n_query_per_seq)
    Hq = q.shape[1]
    if q.shape != (S * nq, Hq, D) or out.shape != q.shape or block_tables.shape[0] != S:
        raise ValueError("q/out must be [num_seqs * n_query_per_seq, Hq, D], tables [num_seqs, MB]")
    on = [("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("block_tables", block_tables),
          ("context_lens", context_lens), ("out", out)]
    ks = vs = slopes = None
    if k_scale is not None:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            check(t, name, torch.uint8, 2)
            if t.shape != (NB, Hkv):
                raise ValueError(f"{name} must be [num_blocks, Hkv]")
            on.append((name, t))
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    if alibi_slopes is not None:
        check(alibi_slopes, "alibi_slopes", torch.float32, 1)
        if alibi_slopes.shape[0] != Hq:
            raise ValueError("alibi_slopes must hold one float per query head")
        on.append(("alibi_slopes", alibi_slopes))
        slopes = alibi_slopes.data_ptr()
    if ws is not None:
        check(ws, "ws", torch.uint8, 1)
        on.append(("ws", ws))
    dev = _on_device(on)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if ws is None:
        ws = _workspace(dev, stream, _workspace_bytes(S, nq, Hq, Hkv, D, dev))
    st = _pkv.lib().pkv_paged_decode_attention_scored(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), NB, ks, vs,
        block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), S, nq, Hq, Hkv,
        D, float(scale), float(softcap), slopes, int(window), out.data_ptr(),
        _pkv.PKV_FP32 if out.dtype == torch.float32 else _pkv.PKV_BF16, ws.data_ptr(), ws.numel(),
        stream)
    if st != _pkv.PKV_OK:
        raise _pkv.PkvError("pkv_paged_decode_attention_scored", st)
    return out


def paged_decode_attention_fp8_block(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                     context_lens, n_query_per_seq, scale, out, ws=None):
    """Decode attention over block-scaled E4M3 (uint8) pools; writes ``out`` (bf16 or fp32).
    Tables no wider than the batch needs are faster where sequences are few or short."""
    if k_scale is None or v_scale is None:
        raise ValueError("k_scale and v_scale are required")
    return _attend(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   n_query_per_seq, scale, out, 0.0, None, 0, ws)


def paged_decode_attention_scored(q, k_cache, v_cache, block_tables, context_lens,
                                  n_query_per_seq, scale, out, softcap=0.0, alibi_slopes=None,
                                  window=0, k_scale=None, v_scale=None, ws=None):
    """Decode attention with scores capped at ``softcap`` (tanh), biased by
    ``alibi_slopes`` (float32 ``[Hq]``) times the distance, or limited to the last
    ``window`` positions; bf16 pools, or block-scaled E4M3 pools with both scales."""
    return _attend(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                   n_query_per_seq, scale, out, softcap, alibi_slopes, window, ws)
