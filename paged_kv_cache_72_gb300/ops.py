"""Thin torch-facing wrappers over the C ABI (argument marshalling only).

Every function takes CUDA tensors, checks dtypes and shapes, passes raw device
pointers, sizes and the current CUDA stream to libpa.so, and raises PAError on
a non-zero status.  The appends, the 4-bit cache's calls and the prefill over
quantized caches are marshalled by an extension module (csrc/pa_call.cpp), the
others here through ctypes.  Nothing is
computed here.
"""
import ctypes

import torch

from . import _lib
from ._lib import (PA_BF16, PA_DECODE_AUTO, PA_F16, PA_FP4_E2M1, PA_FP8_E4M3,
                   PA_PREFILL_QUANT_COUNTERS, PA_SWAP_IN, PA_SWAP_OUT)


class PAError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = _lib.load().pa_strerror(status)
        super().__init__("%s failed: %s (status %d)" % (what, msg.decode() if msg else "?", status))


def _check(status, what):
    if status != 0:
        raise PAError(status, what)


def _dtype_code(t):
    if t.dtype == torch.float16:
        return PA_F16
    if t.dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError("expected float16 or bfloat16, got %s" % t.dtype)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _pool_shape(k_cache, v_cache):
    _cuda(k_cache, "k_cache")
    _cuda(v_cache, "v_cache")
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must share one shape [num_blocks, B, H_kv, D]")
    return k_cache.shape


def _fp8_pools(k_cache, v_cache):
    shape = _pool_shape(k_cache, v_cache)
    if k_cache.dtype != torch.uint8:
        raise TypeError("E4M3 pools must be uint8 tensors of codes")
    return shape


def pa_fp4_pool_shape(num_blocks, block_size, num_kv_heads, head_dim):
    """Shape of a 4-bit pool, a uint8 tensor: [num_blocks, H_kv, B, 9 D / 16].  A
    block's head holds its codes [B, D / 2], then its scales
    [B / 4, D / 16, 4], in the B * 9 D / 16 bytes of that plane."""
    return (num_blocks, num_kv_heads, block_size, head_dim // 2 + head_dim // 16)


# bytes of a 4-bit row -> head_dim
_FP4_HEAD_DIM = {36: 64, 72: 128}


_CODE = {torch.float16: PA_F16, torch.bfloat16: PA_BF16}


def _block_pools(k_cache, v_cache):
    """(num_blocks, B, H_kv, D, dtype code) of pools of any element type."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != dtype:
        raise ValueError("k_cache and v_cache must share one shape [num_blocks, B, H_kv, D]")
    a, b, c, d = shape
    if dtype in _CODE:
        return a, b, c, d, _CODE[dtype]
    if dtype != torch.uint8:
        raise TypeError("expected float16, bfloat16 or uint8 pools, got %s" % dtype)
    if d in _FP4_HEAD_DIM:
        return a, c, b, _FP4_HEAD_DIM[d], PA_FP4_E2M1
    return a, b, c, d, PA_FP8_E4M3


def _fp4_pools(k_cache, v_cache):
    """(B, H_kv, D) of a pair of 4-bit pools."""
    _, B, H, D, code = _block_pools(k_cache, v_cache)
    if code != PA_FP4_E2M1:
        raise ValueError("4-bit pools must be uint8 [num_blocks, H_kv, B, 9 D / 16], D 64 or 128")
    return B, H, D


_call = None


def _calls():
    """The extension module behind the append's and the 4-bit cache's calls.  It
    checks types, shapes, layouts and devices, and raises TypeError or
    ValueError; there is no fallback."""
    global _call
    if _call is None:
        _lib.load()
        from . import _pa_call
        _call = _pa_call
    return _call


def pa_version():
    return _lib.load().pa_version()


def pa_slot_mapping(block_tables, token_seq, token_pos, block_size, num_blocks, out=None,
                    err=None):
    """int64 slots block_tables[seq][pos // B] * B + pos % B for each new token."""
    L = _lib.load()
    for t, n in ((block_tables, "block_tables"), (token_seq, "token_seq"), (token_pos, "token_pos")):
        _cuda(t, n)
        if t.dtype != torch.int32:
            raise TypeError("%s must be int32" % n)
    n_tok = token_seq.numel()
    if token_pos.numel() != n_tok:
        raise ValueError("token_seq and token_pos differ in length")
    if out is None:
        out = torch.empty(n_tok, dtype=torch.int64, device=token_seq.device)
    _check(L.pa_slot_mapping(_ptr(block_tables), block_tables.shape[1], block_tables.shape[0],
                             _ptr(token_seq), _ptr(token_pos), n_tok, int(block_size),
                             int(num_blocks), _ptr(out), _ptr(err), _stream()), "pa_slot_mapping")
    return out


def pa_cache_write(k, v, slot_mapping, k_cache, v_cache, err=None):
    """Store k[n], v[n] ([n_tok, H_kv, D]) at pool slot slot_mapping[n]."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    _cuda(k, "k")
    _cuda(v, "v")
    _cuda(slot_mapping, "slot_mapping")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    n_tok = slot_mapping.numel()
    if k.shape != (n_tok, H, D) or v.shape != (n_tok, H, D):
        raise ValueError("k, v must be [num_tokens, H_kv, D]")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype:
        raise TypeError("k, v and the pools must share a dtype")
    _check(L.pa_cache_write(_ptr(k), _ptr(v), _ptr(slot_mapping), n_tok, _ptr(k_cache),
                            _ptr(v_cache), nb, B, H, D, _dtype_code(k_cache), _ptr(err),
                            _stream()), "pa_cache_write")


def pa_cache_write_mapped(k, v, block_tables, token_seq, token_pos, k_cache, v_cache,
                          slot_mapping=None, err=None):
    """pa_slot_mapping and pa_cache_write in one launch: store k[n], v[n]
    ([n_tok, H_kv, D]) at slot block_tables[seq][pos // B] * B + pos % B of
    new token n; the int64 slots go to slot_mapping when given."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    for t, n in ((block_tables, "block_tables"), (token_seq, "token_seq"), (token_pos, "token_pos")):
        _cuda(t, n)
        if t.dtype != torch.int32:
            raise TypeError("%s must be int32" % n)
    _cuda(k, "k")
    _cuda(v, "v")
    n_tok = token_seq.numel()
    if token_pos.numel() != n_tok:
        raise ValueError("token_seq and token_pos differ in length")
    if k.shape != (n_tok, H, D) or v.shape != (n_tok, H, D):
        raise ValueError("k, v must be [num_tokens, H_kv, D]")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype:
        raise TypeError("k, v and the pools must share a dtype")
    if slot_mapping is not None:
        _cuda(slot_mapping, "slot_mapping")
        if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n_tok:
            raise ValueError("slot_mapping must be int64 [num_tokens]")
    _check(L.pa_cache_write_mapped(_ptr(k), _ptr(v), _ptr(block_tables), block_tables.shape[1],
                                   block_tables.shape[0], _ptr(token_seq), _ptr(token_pos), n_tok,
                                   _ptr(k_cache), _ptr(v_cache), nb, B, H, D,
                                   _dtype_code(k_cache), _ptr(slot_mapping), _ptr(err), _stream()),
           "pa_cache_write_mapped")
    return slot_mapping


def pa_copy_blocks(pairs, k_cache, v_cache, err=None):
    """Copy pool block src -> dst (K and V) for each row (src, dst) of pairs.

    Pools of float16 / bfloat16 elements, uint8 E4M3 codes, or 4-bit pools: uint8
    with a last dimension of 36 or 72, which no E4M3 pool has."""
    L = _lib.load()
    _pool_shape(k_cache, v_cache)
    nb, B, H, D, code = _block_pools(k_cache, v_cache)
    _cuda(pairs, "pairs")
    if pairs.dtype != torch.int32:
        raise TypeError("pairs must be int32 [n, 2]")
    n = pairs.numel() // 2
    _check(L.pa_copy_blocks(_ptr(pairs), n, _ptr(k_cache), _ptr(v_cache), nb, B, H, D,
                            code, _ptr(err), _stream()), "pa_copy_blocks")


def pa_swap_blocks(pairs, src_k, src_v, dst_k, dst_v, err=None):
    """Copy block src of the source pools to block dst of the destination
    pools for each row (src, dst) of pairs: one pool pair on the GPU, the other
    in host memory the GPU can address (pinned; or any host memory where the
    GPU reads the host's page tables).  The direction follows from which is
    which."""
    L = _lib.load()
    _cuda(pairs, "pairs")
    if pairs.dtype != torch.int32:
        raise TypeError("pairs must be int32 [n, 2]")
    if src_k.is_cuda == dst_k.is_cuda:
        raise ValueError("one pool pair must be on the GPU and the other in pinned host memory")
    dev_k, dev_v, host_k, host_v = (src_k, src_v, dst_k, dst_v) if src_k.is_cuda else \
        (dst_k, dst_v, src_k, src_v)
    for t in (host_k, host_v):
        if not t.is_contiguous():
            raise ValueError("the host pools must be contiguous")
    _pool_shape(dev_k, dev_v)
    nbd, B, H, D, code = _block_pools(dev_k, dev_v)
    if host_k.shape[1:] != dev_k.shape[1:] or host_k.dtype != dev_k.dtype or \
            host_v.shape != host_k.shape or host_v.dtype != host_k.dtype:
        raise ValueError("host and device pools must share the block shape and dtype")
    direction = PA_SWAP_OUT if src_k.is_cuda else PA_SWAP_IN
    _check(L.pa_swap_blocks(_ptr(pairs), pairs.numel() // 2, direction, _ptr(dev_k), _ptr(dev_v),
                            nbd, ctypes.c_void_p(host_k.data_ptr()),
                            ctypes.c_void_p(host_v.data_ptr()), host_k.shape[0], B, H, D, code,
                            _ptr(err), _stream()), "pa_swap_blocks")


def pa_cache_write_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, err=None):
    """Quantize k[n], v[n] ([n_tok, H_kv, D], float16 / bfloat16) to E4M3 codes
    (value / scale, round to nearest even, saturating) at pool slot
    slot_mapping[n] of the uint8 pools."""
    L = _lib.load()
    nb, B, H, D = _fp8_pools(k_cache, v_cache)
    _cuda(k, "k")
    _cuda(v, "v")
    _cuda(slot_mapping, "slot_mapping")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    n_tok = slot_mapping.numel()
    if k.shape != (n_tok, H, D) or v.shape != (n_tok, H, D) or k.dtype != v.dtype:
        raise ValueError("k, v must be [num_tokens, H_kv, D] of one dtype")
    _check(L.pa_cache_write_fp8(_ptr(k), _ptr(v), _dtype_code(k), _ptr(slot_mapping), n_tok,
                                _ptr(k_cache), _ptr(v_cache), nb, B, H, D, float(k_scale),
                                float(v_scale), _ptr(err), _stream()), "pa_cache_write_fp8")


def pa_cache_write_fp8_mapped(k, v, block_tables, token_seq, token_pos, k_cache, v_cache,
                              k_scale, v_scale, slot_mapping=None, err=None):
    """pa_slot_mapping and pa_cache_write_fp8 in one launch: E4M3 codes of
    k[n] / k_scale and v[n] / v_scale ([n_tok, H_kv, D], float16 / bfloat16)
    stored at slot block_tables[seq][pos // B] * B + pos % B of new token n;
    the int64 slots go to slot_mapping when given."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    for t, n in ((block_tables, "block_tables"), (token_seq, "token_seq"), (token_pos, "token_pos")):
        _cuda(t, n)
        if t.dtype != torch.int32:
            raise TypeError("%s must be int32" % n)
    _cuda(k, "k")
    _cuda(v, "v")
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8:
        raise TypeError("E4M3 pools are uint8 codes")
    n_tok = token_seq.numel()
    if token_pos.numel() != n_tok:
        raise ValueError("token_seq and token_pos differ in length")
    if k.shape != (n_tok, H, D) or v.shape != (n_tok, H, D) or k.dtype != v.dtype:
        raise ValueError("k, v must be [num_tokens, H_kv, D] of one dtype")
    if slot_mapping is not None:
        _cuda(slot_mapping, "slot_mapping")
        if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != n_tok:
            raise ValueError("slot_mapping must be int64 [num_tokens]")
    _check(L.pa_cache_write_fp8_mapped(_ptr(k), _ptr(v), _dtype_code(k), _ptr(block_tables),
                                       block_tables.shape[1], block_tables.shape[0],
                                       _ptr(token_seq), _ptr(token_pos), n_tok, _ptr(k_cache),
                                       _ptr(v_cache), nb, B, H, D, float(k_scale), float(v_scale),
                                       _ptr(slot_mapping), _ptr(err), _stream()),
           "pa_cache_write_fp8_mapped")
    return slot_mapping


def pa_decode_workspace_size(num_q_heads, num_kv_heads, head_dim, block_size, dtype,
                             flags=PA_DECODE_AUTO, num_ctas=0):
    L = _lib.load()
    if isinstance(dtype, torch.dtype):
        dtype = {torch.float16: PA_F16, torch.bfloat16: PA_BF16, torch.uint8: PA_FP8_E4M3}[dtype]
    n = ctypes.c_size_t(0)
    _check(L.pa_decode_workspace_size(num_q_heads, num_kv_heads, head_dim, block_size, dtype,
                                      flags, num_ctas, ctypes.byref(n)),
           "pa_decode_workspace_size")
    return n.value


def pa_decode(q, k_cache, v_cache, block_tables, seq_lens, scale, out=None, workspace=None,
              flags=PA_DECODE_AUTO, num_ctas=0, err=None):
    """Paged single-query decode attention: out [N, Hq, D]."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    _cuda(q, "q")
    _cuda(block_tables, "block_tables")
    _cuda(seq_lens, "seq_lens")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    N, Hq, Dq = q.shape
    if Dq != D or q.dtype != k_cache.dtype:
        raise ValueError("q must be [N, Hq, D] in the pool dtype")
    if block_tables.dim() != 2 or block_tables.shape[0] != N or seq_lens.numel() != N:
        raise ValueError("block_tables must be [N, stride] and seq_lens [N]")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = pa_decode_workspace_size(Hq, H, D, B, _dtype_code(q), flags, num_ctas)
        # zero-filled once; the decode leaves it ready for the next call
        workspace = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    _check(L.pa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                       block_tables.shape[1], _ptr(seq_lens), N, Hq, H, D, B, nb,
                       _dtype_code(q), float(scale), _ptr(out), _ptr(workspace),
                       workspace.numel() * workspace.element_size(), int(flags), int(num_ctas),
                       _ptr(err), _stream()), "pa_decode")
    return out


def pa_decode_window(q, k_cache, v_cache, block_tables, seq_lens, scale, window, out=None,
                     workspace=None, flags=PA_DECODE_AUTO, num_ctas=0, err=None):
    """Sliding-window decode: the query of position T - 1 attends to tokens
    [max(0, T - window), T); table entries of blocks before the window are
    never read (released blocks may be -1)."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    _cuda(q, "q")
    _cuda(block_tables, "block_tables")
    _cuda(seq_lens, "seq_lens")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    N, Hq, Dq = q.shape
    if Dq != D or q.dtype != k_cache.dtype:
        raise ValueError("q must be [N, Hq, D] in the pool dtype")
    if block_tables.dim() != 2 or block_tables.shape[0] != N or seq_lens.numel() != N:
        raise ValueError("block_tables must be [N, stride] and seq_lens [N]")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = pa_decode_workspace_size(Hq, H, D, B, _dtype_code(q), flags, num_ctas)
        workspace = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    _check(L.pa_decode_window(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                              block_tables.shape[1], _ptr(seq_lens), N, Hq, H, D, B, nb,
                              _dtype_code(q), float(scale), int(window), _ptr(out),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              int(flags), int(num_ctas), _ptr(err), _stream()),
           "pa_decode_window")
    return out


def pa_decode_fp8(q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale, v_scale, out=None,
                  workspace=None, flags=PA_DECODE_AUTO, num_ctas=0, err=None):
    """Paged decode over uint8 E4M3 pools (value = code * scale): out [N, Hq, D]
    in q's dtype."""
    L = _lib.load()
    nb, B, H, D = _fp8_pools(k_cache, v_cache)
    _cuda(q, "q")
    _cuda(block_tables, "block_tables")
    _cuda(seq_lens, "seq_lens")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    N, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q must be [N, Hq, D]")
    if block_tables.dim() != 2 or block_tables.shape[0] != N or seq_lens.numel() != N:
        raise ValueError("block_tables must be [N, stride] and seq_lens [N]")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = pa_decode_workspace_size(Hq, H, D, B, PA_FP8_E4M3, flags, num_ctas)
        # zero-filled once; the decode leaves it ready for the next call
        workspace = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    _check(L.pa_decode_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                           block_tables.shape[1], _ptr(seq_lens), N, Hq, H, D, B, nb,
                           _dtype_code(q), float(scale), float(k_scale), float(v_scale),
                           _ptr(out), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), int(flags),
                           int(num_ctas), _ptr(err), _stream()), "pa_decode_fp8")
    return out


def pa_append_rope(q, k, v, cos_sin, block_tables, token_seq, token_pos, k_cache, v_cache,
                   interleaved=False, q_norm=None, k_norm=None, eps=1e-6, k_scale=1.0,
                   v_scale=1.0, q_out=None, slot_mapping=None, err=None):
    """A step's projections into the attention in one launch: RMS norms of the
    query and key heads (when q_norm / k_norm, [D], are given), the position
    rotation, the rotated queries returned ([num_tokens, Hq, D]) and keys and
    values stored at slot block_tables[seq][pos // B] * B + pos % B.

    q [num_tokens, Hq, D] (or None), k, v [num_tokens, H_kv, D]: float16 or
    bfloat16, heads contiguous, tokens any multiple of 8 elements apart (views
    of a fused projection's output).  cos_sin: float32 [max_pos, rotary_dim],
    the row of a position holding rotary_dim / 2 cosines, then as many sines
    (None: no rotation).  Element i pairs with i + rotary_dim / 2, or 2 i with
    2 i + 1 when interleaved.  The pools are of the inputs' dtype
    [num_blocks, B, H_kv, D], uint8 E4M3 codes of that shape, or 4-bit pools
    (pa_fp4_pool_shape); k_scale and v_scale apply to the last two.  Tokens of
    sequence -1 are padding: they write nothing, and their rows of q_out keep
    what they held (zeros when q_out is made here)."""
    if q_out is None and q is not None:
        q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    status = (_call or _calls()).append_rope(
        q, k, v, cos_sin, block_tables, token_seq, token_pos, k_cache, v_cache, interleaved, q_norm,
        k_norm, eps, k_scale, v_scale, q_out, slot_mapping, err)
    if status:
        raise PAError(status, "pa_append_rope")
    return q_out


def pa_append_rope_axes(q, k, v, cos_sin, axis_of, rot_pos, block_tables, token_seq, token_pos,
                        k_cache, v_cache, interleaved=False, q_norm=None, k_norm=None, eps=1e-6,
                        k_scale=1.0, v_scale=1.0, q_out=None, slot_mapping=None, err=None):
    """pa_append_rope for tokens whose position has several axes: frequency i takes
    its angle from row rot_pos[axis_of[i], token] of cos_sin.

    axis_of: uint8 [rotary_dim / 2], the axis of every frequency; rot_pos: int32
    [num_axes, num_tokens], 1 to 4 axes, the positions that select angles.
    token_pos places the token in the cache alone.  Everything else is as for
    pa_append_rope, to which the call is equal bit for bit when every row of
    rot_pos is token_pos."""
    if q_out is None and q is not None:
        q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    status = (_call or _calls()).append_rope_axes(
        q, k, v, cos_sin, axis_of, rot_pos, block_tables, token_seq, token_pos, k_cache, v_cache,
        interleaved, q_norm, k_norm, eps, k_scale, v_scale, q_out, slot_mapping, err)
    if status:
        raise PAError(status, "pa_append_rope_axes")
    return q_out


def pa_cache_write_fp4(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, err=None):
    """Quantize k[n], v[n] ([n_tok, H_kv, D], float16 / bfloat16) to E2M1 codes
    with an E4M3 scale per 16 head_dim values (value = code * scale16 * scale)
    at pool slot slot_mapping[n] of the 4-bit pools (pa_fp4_pool_shape)."""
    status = (_call or _calls()).cache_write_fp4(k, v, slot_mapping, k_cache, v_cache, k_scale,
                                                 v_scale, err)
    if status:
        raise PAError(status, "pa_cache_write_fp4")


def pa_cache_write_fp4_mapped(k, v, block_tables, token_seq, token_pos, k_cache, v_cache,
                              k_scale, v_scale, slot_mapping=None, err=None):
    """Slot mapping and pa_cache_write_fp4 in one launch: new token n goes to
    slot block_tables[seq][pos // B] * B + pos % B; the int64 slots go to
    slot_mapping when given.  Tokens of sequence -1 are padding (slot -1)."""
    status = (_call or _calls()).cache_write_fp4_mapped(k, v, block_tables, token_seq, token_pos,
                                                        k_cache, v_cache, k_scale, v_scale,
                                                        slot_mapping, err)
    if status:
        raise PAError(status, "pa_cache_write_fp4_mapped")
    return slot_mapping


def pa_cache_read_fp4(slot_mapping, k_cache, v_cache, k_scale, v_scale, dtype=torch.bfloat16,
                      k_out=None, v_out=None, err=None):
    """The rows at pool slots slot_mapping[n] of 4-bit pools as 16-bit values
    (k, v), each [n, H_kv, D].  Rows of negative slots keep what the outputs
    held (zeros when the outputs are made here)."""
    if (k_out is None) != (v_out is None):
        raise ValueError("give both of k_out and v_out, or neither")
    if k_out is None:
        _, H, D = _fp4_pools(k_cache, v_cache)
        k_out = torch.zeros((slot_mapping.numel(), H, D), dtype=dtype, device=k_cache.device)
        v_out = torch.zeros_like(k_out)
    status = (_call or _calls()).cache_read_fp4(slot_mapping, k_cache, v_cache, k_scale, v_scale,
                                                k_out, v_out, err)
    if status:
        raise PAError(status, "pa_cache_read_fp4")
    return k_out, v_out


def pa_decode_fp4(q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale, v_scale, window=0,
                  out=None, workspace=None, flags=PA_DECODE_AUTO, num_ctas=0, err=None):
    """Paged decode over 4-bit pools (value = code * scale16 * scale): out
    [N, Hq, D] in q's dtype.  window >= 1: the query of position T - 1 attends
    to tokens [max(0, T - window), T); 0: to all of them."""
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        B, H, D = _fp4_pools(k_cache, v_cache)
        nbytes = pa_decode_workspace_size(q.shape[1], H, D, B, PA_FP4_E2M1, flags, num_ctas)
        # zero-filled once; the decode leaves it ready for the next call
        workspace = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    status = (_call or _calls()).decode_fp4(q, k_cache, v_cache, block_tables, seq_lens, scale,
                                            k_scale, v_scale, window, out, workspace, flags,
                                            num_ctas, err)
    if status:
        raise PAError(status, "pa_decode_fp4")
    return out


def pa_prefill(q, k_cache, v_cache, block_tables, seq_lens, query_start, scale, out=None,
               workspace=None, err=None):
    """Multi-query paged attention (chunked prefill, decode tokens allowed):
    q [total_q, Hq, D]; sequence i's new tokens are rows [query_start[i],
    query_start[i+1]), already written at the end of its seq_lens[i] tokens."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    for t, n in ((q, "q"), (block_tables, "block_tables"), (seq_lens, "seq_lens"),
                 (query_start, "query_start")):
        _cuda(t, n)
    for t, n in ((block_tables, "block_tables"), (seq_lens, "seq_lens"),
                 (query_start, "query_start")):
        if t.dtype != torch.int32:
            raise TypeError("%s must be int32" % n)
    total, Hq, Dq = q.shape
    N = seq_lens.numel()
    if Dq != D or q.dtype != k_cache.dtype:
        raise ValueError("q must be [total_q, Hq, D] in the pool dtype")
    if query_start.numel() != N + 1 or block_tables.dim() != 2 or block_tables.shape[0] != N:
        raise ValueError("query_start must be [N + 1] and block_tables [N, stride]")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(L.pa_prefill_workspace_size(ctypes.byref(n)), "pa_prefill_workspace_size")
        workspace = torch.zeros(n.value, dtype=torch.uint8, device=q.device)
    _check(L.pa_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                        block_tables.shape[1], _ptr(seq_lens), _ptr(query_start), N, total, Hq, H,
                        D, B, nb, _dtype_code(q), float(scale), _ptr(out), _ptr(workspace),
                        workspace.numel(), _ptr(err), _stream()), "pa_prefill")
    return out


def pa_prefill_quant_workspace_size(num_q_heads, num_kv_heads, head_dim):
    """Bytes of workspace that pa_prefill_fp8 and pa_prefill_fp4 need for this
    shape on the current device; the first PA_PREFILL_QUANT_COUNTERS of them
    must be zero before its first use."""
    n = ctypes.c_size_t(0)
    _check(_lib.load().pa_prefill_quant_workspace_size(num_q_heads, num_kv_heads, head_dim,
                                                       ctypes.byref(n)),
           "pa_prefill_quant_workspace_size")
    return n.value


def _quant_workspace(num_q_heads, num_kv_heads, head_dim, device):
    ws = torch.empty(pa_prefill_quant_workspace_size(num_q_heads, num_kv_heads, head_dim),
                     dtype=torch.uint8, device=device)
    ws[:PA_PREFILL_QUANT_COUNTERS].zero_()
    return ws


def pa_prefill_fp8(q, k_cache, v_cache, block_tables, seq_lens, query_start, scale, k_scale,
                   v_scale, window=0, out=None, workspace=None, err=None):
    """Multi-query paged attention (chunks of new tokens, single tokens allowed)
    over uint8 E4M3 pools [num_blocks, B, H_kv, D] (value = code * scale): q
    [total_q, Hq, D]; sequence i's new tokens are rows [query_start[i],
    query_start[i+1]), already written at the end of its seq_lens[i] tokens.
    window >= 1: position p attends to tokens [max(0, p - window + 1), p]; 0: to
    [0, p].  Rows of no sequence keep what out held (zeros when it is made
    here)."""
    if out is None:
        out = torch.zeros_like(q)
    if workspace is None:
        _, _, H, D = _fp8_pools(k_cache, v_cache)
        workspace = _quant_workspace(q.shape[1], H, D, q.device)
    status = (_call or _calls()).prefill_fp8(q, k_cache, v_cache, block_tables, seq_lens,
                                             query_start, scale, k_scale, v_scale, window, out,
                                             workspace, err)
    if status:
        raise PAError(status, "pa_prefill_fp8")
    return out


def pa_prefill_fp4(q, k_cache, v_cache, block_tables, seq_lens, query_start, scale, k_scale,
                   v_scale, window=0, out=None, workspace=None, err=None):
    """pa_prefill_fp8 over 4-bit pools (pa_fp4_pool_shape; value = code * scale16 *
    scale)."""
    if out is None:
        out = torch.zeros_like(q)
    if workspace is None:
        _, H, D = _fp4_pools(k_cache, v_cache)
        workspace = _quant_workspace(q.shape[1], H, D, q.device)
    status = (_call or _calls()).prefill_fp4(q, k_cache, v_cache, block_tables, seq_lens,
                                             query_start, scale, k_scale, v_scale, window, out,
                                             workspace, err)
    if status:
        raise PAError(status, "pa_prefill_fp4")
    return out


def pa_prefill_kernel(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_seqs):
    """Which kernel pa_prefill runs for this shape on the current device:
    PA_PREFILL_TENSOR_CORE or PA_PREFILL_WARP_MMA."""
    L = _lib.load()
    kind = ctypes.c_int32(-1)
    _check(L.pa_prefill_kernel(num_q_heads, num_kv_heads, head_dim, block_size, dtype, num_seqs,
                               ctypes.byref(kind)), "pa_prefill_kernel")
    return kind.value


def pa_gather_kv(k_cache, v_cache, block_tables, seq_lens, out_offsets, total_rows,
                 flags=PA_DECODE_AUTO, err=None):
    """Contiguous copies [total_rows, H_kv, D] of every sequence's K and V."""
    L = _lib.load()
    nb, B, H, D = _pool_shape(k_cache, v_cache)
    N = seq_lens.numel()
    k_out = torch.empty((total_rows, H, D), dtype=k_cache.dtype, device=k_cache.device)
    v_out = torch.empty_like(k_out)
    _check(L.pa_gather_kv(_ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                          _ptr(seq_lens), _ptr(out_offsets), N, H, D, B, nb,
                          _dtype_code(k_cache), int(flags), _ptr(k_out), _ptr(v_out), _ptr(err),
                          _stream()), "pa_gather_kv")
    return k_out, v_out


def pa_get_error(err):
    """Synchronize the current stream, return and clear the device error bits."""
    L = _lib.load()
    flags = ctypes.c_int32(0)
    rc = L.pa_get_error(_ptr(err), _stream(), ctypes.byref(flags))
    if rc not in (0, _lib.PA_ERR_DEVICE_INDEX):
        raise PAError(rc, "pa_get_error")
    return flags.value
