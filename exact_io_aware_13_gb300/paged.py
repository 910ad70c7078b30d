"""The paged cache: writing new tokens (bf16 or e4m3), reading them back, and attention of
ragged chunks of new tokens over it, on the C ABI (include/attn.h states layouts, scales and
bad-input rules; csrc/binding.cpp checks the tensors). Decode over the cache is
attention.decode_paged.

A call's rows are packed: offsets int32 [B + 1] cuts them into sequences, and sequence b's
rows are its newest tokens, row i of n at position seq_lens[b] - n + i. An e4m3 cache is two
uint8 tensors of codes plus kv_exp uint8 [pages, Hkv, page_size, 2], the biased exponents of
each token's K and V scale; passing kv_exp selects it. Wrong tensors raise ValueError, a
refusal of the library AttnError. stream (default: the current one) may be another stream of
the device: the call waits for nothing on the current one, and the tensors that it makes are
memory of that stream.
"""
from __future__ import annotations

from typing import Optional

from . import _lib
from .attention import MASK_NONE, SCORE_NONE, _num_sms

CACHE_BF16, CACHE_E4M3 = 0, 1


def cache_write(k, v, k_cache, v_cache, page_table, offsets, seq_lens, *, kv_exp=None,
                stream=None) -> None:
    """Write the new tokens' K and V rows (bf16 [T, Hkv, d], any token and head stride that
    is a multiple of 8) into the cache: as they are, or with kv_exp as e4m3 codes under the
    smallest power-of-two scale that holds each row."""
    status = _lib.binding().cache_write(k, v, k_cache, v_cache, page_table, offsets, seq_lens,
                                        kv_exp, stream)
    if status is not None:
        _lib.check(status, "attn_cache_write")


def cache_read_into(k_cache, v_cache, page_table, offsets, seq_lens, k, v, *, kv_exp=None,
                    stream=None) -> None:
    """Read the newest tokens of each sequence into k and v (bf16 [T, Hkv, d], contiguous);
    rows behind offsets[B] keep what they held."""
    if k is None or v is None:
        raise ValueError("k and v must be tensors")
    status = _lib.binding().cache_read(k_cache, v_cache, page_table, offsets, seq_lens, kv_exp,
                                       stream, k, v, None)
    if status is not None:
        _lib.check(status, "attn_cache_read")


def cache_read(k_cache, v_cache, page_table, offsets, seq_lens, n_tokens: int, *, kv_exp=None,
               stream=None):
    """Allocating form of cache_read_into for n_tokens = offsets[B] rows: (k, v)."""
    out = _lib.binding().cache_read(k_cache, v_cache, page_table, offsets, seq_lens, kv_exp,
                                    stream, None, None, n_tokens)
    if out.__class__ is int:
        _lib.check(out, "attn_cache_read")
    return out


def prefill_split_keys(cache_kind: int, B: int, T: int, Hq: int, Hkv: int, max_new: int,
                       max_seq_len: int, total_kv_tokens: int,
                       num_sms: Optional[int] = None) -> int:
    """The library's split size for a prefill_paged call (keys per chunk)."""
    return int(_lib.load().attn_prefill_split_keys(
        int(cache_kind), int(B), int(T), int(Hq), int(Hkv), int(max_new), int(max_seq_len),
        int(total_kv_tokens), _num_sms() if num_sms is None else int(num_sms)))


def prefill_workspace_size(T: int, Hq: int, d: int, max_seq_len: int, split_keys: int) -> int:
    return int(_lib.load().attn_prefill_workspace_size(int(T), int(Hq), int(d), int(max_seq_len),
                                                       int(split_keys)))


def prefill_paged_into(q, k_cache, v_cache, page_table, offsets, seq_lens, o, lse, workspace, *,
                       max_new: int, max_seq_len: int, split_keys: int, scale: float,
                       kv_exp=None, mask_kind: int = MASK_NONE, window: int = 0,
                       score_kind: int = SCORE_NONE, softcap: float = 0.0, stream=None) -> None:
    """attn_prefill_paged on caller-owned tensors: q bf16 [T, Hq, d] (any token and head
    stride that is a multiple of 8), o bf16 [T, Hq, d] and lse fp32 [T, Hq] contiguous. Rows
    behind offsets[B] keep what they held."""
    if o is None or lse is None:
        raise ValueError("o and lse must be tensors")
    status = _lib.binding().prefill(q, k_cache, v_cache, page_table, offsets, seq_lens, kv_exp,
                                    stream, o, lse, workspace, max_new, max_seq_len, split_keys,
                                    None, scale, mask_kind, window, score_kind, softcap)
    if status is not None:
        _lib.check(status, "attn_prefill_paged")


def prefill_paged(q, k_cache, v_cache, page_table, offsets, seq_lens, *, kv_exp=None,
                  max_new: Optional[int] = None, max_seq_len: Optional[int] = None,
                  split_keys: Optional[int] = None, total_kv_tokens: Optional[int] = None,
                  scale: Optional[float] = None, mask_kind: int = MASK_NONE, window: int = 0,
                  score_kind: int = SCORE_NONE, softcap: float = 0.0, stream=None):
    """Allocating form of prefill_paged_into: (o, lse) of the chunks' rows. max_new (the
    longest chunk) defaults to T, max_seq_len to the page table's capacity, split_keys to
    the library's choice (total_kv_tokens, the sum of seq_lens when the caller knows it,
    lets it weigh long sequences against short ones)."""
    out = _lib.binding().prefill(q, k_cache, v_cache, page_table, offsets, seq_lens, kv_exp,
                                 stream, None, None, None, max_new, max_seq_len, split_keys,
                                 total_kv_tokens, scale, mask_kind, window, score_kind, softcap)
    if out.__class__ is int:
        _lib.check(out, "attn_prefill_paged")
    return out
