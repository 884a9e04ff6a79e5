"""Binding of the serving operators: decode with row statistics, attention mass, eviction, rotary
cache write and draft verification.

Like _lib.py this is argument marshalling only, of the same C entry points (include/q8kv.h). The
checks and the call sit in a compiled module (binding/q8kv_torch.cpp): a serving loop makes
these calls once per layer and step, often on a few sequences, where the host's time per
call counts as much as the kernel's.

Tensors must be contiguous, of the type and shape each function names, and on one CUDA device;
the call runs there, on that device's current stream unless ``stream`` is given. A tensor that
does not fit raises ValueError (or TypeError), a refusal of the library Q8KVError.
"""
from __future__ import annotations

import ctypes
import operator
import threading

from . import _lib
from . import build as _build
from ._lib import Q8KVError

_lock = threading.Lock()
_native = None


def native():
    """The compiled module, bound to the loaded library (both built first when missing or older
    than their sources)."""
    global _native
    L = _lib.lib()
    with _lock:
        if _native is None:
            _build.build_binding()
            from . import _q8kv_torch as module

            entry = lambda name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value
            module.bind(entry("q8kv_decode_attn_lse"), entry("q8kv_attn_mass"),
                        entry("q8kv_evict"), entry("q8kv_rope_cache_write"),
                        entry("q8kv_verify_draft"))
            _native = module
    return _native


def q8kv_decode_attn_lse(out, lse, q, k_blocks, v_blocks, kscale, vscale, block_table, seq_lens,
                         scale, workspace=None, stream=None):
    """q8kv_decode_attn_multi (q, out [B][n_queries][Hq][D]) that also writes the log-sum-exp of
    every row to lse [B][n_queries][Hq] (-inf for a row that sees no token). ``workspace``: a
    CUDA tensor of q8kv_workspace_bytes(B, n_queries * Hq, Hk, D) bytes, or None for the
    library-managed one."""
    status = (_native or native()).decode_attn_lse(out, lse, q, k_blocks, v_blocks, kscale, vscale,
                                                   block_table, seq_lens, scale, workspace, stream)
    if status:
        raise Q8KVError(status, "q8kv_decode_attn_lse")
    return out


def q8kv_attn_mass(mass, q, lse, k_blocks, kscale, block_table, seq_lens, scale, decay=1.0,
                   stream=None):
    """mass[b][kv][t] = decay * mass[b][kv][t] + sum over the head's query rows of
    exp(score - lse): mass fp32 [B][Hk][max_blocks * block_size], q [B][n_queries][Hq][D], lse
    [B][n_queries][Hq] as q8kv_decode_attn_lse left it."""
    status = (_native or native()).attn_mass(mass, q, lse, k_blocks, kscale, block_table, seq_lens,
                                             scale, decay, stream)
    if status:
        raise Q8KVError(status, "q8kv_attn_mass")
    return mass


def q8kv_evict(k_blocks, v_blocks, kscale, vscale, new_mass, kept, new_lens, mass, block_table,
               seq_lens, new_block_table, sink=0, recent=0, stream=None):
    """Keep kept.shape[2] tokens per (sequence, KV head) -- the first ``sink``, the last
    ``recent``, the heaviest others -- and move their rows, in order, to the blocks of
    new_block_table. Writes new_mass fp32 [B][Hk][new_max_blocks * block_size], kept int32
    [B][Hk][keep] (old positions, then -1) and new_lens int32 [B]."""
    status = (_native or native()).evict(k_blocks, v_blocks, kscale, vscale, new_mass, kept,
                                         new_lens, mass, block_table, seq_lens, new_block_table,
                                         sink, recent, stream)
    if status:
        raise Q8KVError(status, "q8kv_evict")


def q8kv_rope_cache_write(q_out, k_blocks, v_blocks, kscale, vscale, q_new, k_new, v_new,
                          slot_mapping, positions, cos_sin, pair_axis=None, adjacent=False,
                          stream=None):
    """Rotate q_new [n][Hq][D] into q_out (fp32) and k_new [n][Hk][D], and write the rotated keys
    and v_new to the q8 cache at slot_mapping (int64 [n], negative = padding). q_new, k_new
    and v_new: one of float32, float16, bfloat16, token dimension strided (k_new and v_new
    alike). positions int32 [n_axes][n]; cos_sin fp32 [max_position][rotary_dim], cosines then
    sines; pair_axis: the axis of each of the rotary_dim / 2 pairs (a host sequence or bytes),
    None for one axis; adjacent: pairs (2p, 2p + 1) instead of (p, p + rotary_dim / 2)."""
    if pair_axis is not None:
        # bytes() of a count is that many zeros, and of an array its memory: only what holds one
        # axis per entry goes there as it is
        if not isinstance(pair_axis, (bytes, bytearray, list, tuple)):
            try:
                pair_axis = [operator.index(axis) for axis in pair_axis]
            except TypeError:
                raise TypeError("pair_axis must be a sequence of integers") from None
        pair_axis = bytes(pair_axis)
    status = (_native or native()).rope_cache_write(q_out, k_blocks, v_blocks, kscale, vscale,
                                                    q_new, k_new, v_new, slot_mapping, positions,
                                                    cos_sin, pair_axis, adjacent, stream)
    if status:
        raise Q8KVError(status, "q8kv_rope_cache_write")
    return q_out


def q8kv_verify_draft(n_accepted, tokens, target_probs, draft_probs, draft_tokens, uniforms,
                      n_drafts=None, stream=None):
    """Speculative sampling's accept test and draw: target_probs [B][n + 1][vocab], draft_probs
    [B][n][vocab] of the same type (float32, float16, bfloat16; None for drafts without
    probabilities), draft_tokens int32 [B][n], uniforms fp32 [B][n + 1] (the last one draws),
    n_drafts int32 [B] or None. Writes n_accepted int32 [B] and tokens int32 [B][n + 1]: the
    accepted drafts, the drawn token, then -1. Rows of probabilities may be evenly strided."""
    status = (_native or native()).verify_draft(n_accepted, tokens, target_probs, draft_probs,
                                                draft_tokens, uniforms, n_drafts, stream)
    if status:
        raise Q8KVError(status, "q8kv_verify_draft")
    return tokens
