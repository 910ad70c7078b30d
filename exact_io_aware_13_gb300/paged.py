"""The paged cache: writing new tokens (bf16 or e4m3), reading them back, and attention of
ragged chunks of new tokens over it. Argument checks and marshalling for the C ABI
(include/attn.h states layouts, scales and bad-input rules); decode over the cache is
attention.decode_paged.

A call's rows are packed: offsets int32 [B + 1] cuts them into sequences, and sequence b's
rows are its newest tokens, row i of n at position seq_lens[b] - n + i. An e4m3 cache is two
uint8 tensors of codes plus kv_exp uint8 [pages, Hkv, page_size, 2], the biased exponents of
each token's K and V scale; passing kv_exp selects it.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .attention import (MASK_NONE, SCORE_NONE, _BF16, _F32, _I32, _U8, _check_call,
                        _current_device, _mask_score_params, _ptr, _stream, _workspace_bytes,
                        prefill_split_keys, prefill_workspace_size)

CACHE_BF16, CACHE_E4M3 = 0, 1


def _cache(k_cache, v_cache, page_table, kv_exp, offsets, seq_lens, *more):
    """Checks of the cache and the batch (and of `more`, (tensor, dtype, name) triples of
    contiguous tensors); the cache description and B."""
    kind = _BF16 if kv_exp is None else _U8
    _check_call(((k_cache, kind, "k_cache"), (v_cache, kind, "v_cache"), (kv_exp, _U8, "kv_exp"),
                 (page_table, _I32, "page_table"), (offsets, _I32, "offsets"),
                 (seq_lens, _I32, "seq_lens"), *more))
    shape, table_shape, B = k_cache.shape, page_table.shape, seq_lens.numel()
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [pages, Hkv, page_size, d]")
    pages, Hkv, page_size, d = shape
    if kv_exp is not None and kv_exp.shape != (pages, Hkv, page_size, 2):
        raise ValueError(f"kv_exp must have shape {(pages, Hkv, page_size, 2)}, got "
                         f"{tuple(kv_exp.shape)}")
    if seq_lens.dim() != 1 or offsets.shape != (B + 1,):
        raise ValueError("offsets must be [B + 1] and seq_lens [B]")
    if len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError("page_table must be [B, max_pages]")
    return _lib.PagedCache(k_cache.data_ptr(), v_cache.data_ptr(),
                           None if kv_exp is None else kv_exp.data_ptr(), page_table.data_ptr(),
                           CACHE_BF16 if kv_exp is None else CACHE_E4M3, pages, Hkv, page_size, d,
                           table_shape[1]), B


def _rows(t, H: int, d: int, name: str):
    """Pointer and element strides of packed rows [T, H, d], d contiguous."""
    if not t.is_cuda or t.get_device() != _current_device():
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.dtype != _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != H or shape[2] != d:
        raise ValueError(f"{name} must be [T, {H}, {d}], got {tuple(shape)}")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must be contiguous along d")
    return t.data_ptr(), token if shape[0] > 1 else 0, head if H > 1 else 0


def cache_write(k, v, k_cache, v_cache, page_table, offsets, seq_lens, *, kv_exp=None,
                stream=None) -> None:
    """Write the new tokens' K and V rows (bf16 [T, Hkv, d], any token and head stride that
    is a multiple of 8) into the cache: as they are, or with kv_exp as e4m3 codes under the
    smallest power-of-two scale that holds each row."""
    cache, B = _cache(k_cache, v_cache, page_table, kv_exp, offsets, seq_lens)
    kp, kt, kh = _rows(k, cache.Hkv, cache.d, "k")
    vp, vt, vh = _rows(v, cache.Hkv, cache.d, "v")
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v disagree on the number of tokens")
    _lib.check(_lib.load().attn_cache_write(cache, kp, kt, kh, vp, vt, vh, offsets.data_ptr(),
                                            seq_lens.data_ptr(), B, T, _stream(stream)),
               "attn_cache_write")


def cache_read_into(k_cache, v_cache, page_table, offsets, seq_lens, k, v, *, kv_exp=None,
                    stream=None) -> None:
    """Read the newest tokens of each sequence into k and v (bf16 [T, Hkv, d], contiguous);
    rows behind offsets[B] keep what they held."""
    cache, B = _cache(k_cache, v_cache, page_table, kv_exp, offsets, seq_lens, (k, _BF16, "k"),
                      (v, _BF16, "v"))
    shape = k.shape
    if len(shape) != 3 or shape[1:] != (cache.Hkv, cache.d) or v.shape != shape:
        raise ValueError(f"k and v must be [T, {cache.Hkv}, {cache.d}]")
    _lib.check(_lib.load().attn_cache_read(cache, k.data_ptr(), v.data_ptr(), offsets.data_ptr(),
                                           seq_lens.data_ptr(), B, shape[0], _stream(stream)),
               "attn_cache_read")


def cache_read(k_cache, v_cache, page_table, offsets, seq_lens, n_tokens: int, *, kv_exp=None,
               stream=None):
    """Allocating wrapper of cache_read_into for n_tokens = offsets[B] rows: (k, v)."""
    _, Hkv, _, d = k_cache.shape
    shape, device = (int(n_tokens), Hkv, d), k_cache.device
    k = torch.empty(shape, dtype=_BF16, device=device)
    v = torch.empty(shape, dtype=_BF16, device=device)
    cache_read_into(k_cache, v_cache, page_table, offsets, seq_lens, k, v, kv_exp=kv_exp,
                    stream=stream)
    return k, v


def _prefill_launch(cache, B, q_rows, T, Hq, offsets, seq_lens, o, lse, workspace, ws_bytes,
                    max_new, max_seq_len, split_keys, scale, mask_kind, window, score_kind,
                    softcap, stream) -> None:
    mp, sp, _keep = _mask_score_params(window, softcap)
    _lib.check(_lib.load().attn_prefill_paged(
        cache, *q_rows, o.data_ptr(), lse.data_ptr(), offsets.data_ptr(), seq_lens.data_ptr(), B, T,
        Hq, int(max_new), int(max_seq_len), int(split_keys), scale, mask_kind, mp, score_kind, sp,
        _ptr(workspace), ws_bytes, _stream(stream)), "attn_prefill_paged")


def prefill_paged_into(q, k_cache, v_cache, page_table, offsets, seq_lens, o, lse, workspace, *,
                       max_new: int, max_seq_len: int, split_keys: int, scale: float,
                       kv_exp=None, mask_kind: int = MASK_NONE, window: int = 0,
                       score_kind: int = SCORE_NONE, softcap: float = 0.0, stream=None) -> None:
    """attn_prefill_paged on caller-owned tensors: q bf16 [T, Hq, d] (any token and head
    stride that is a multiple of 8), o bf16 [T, Hq, d] and lse fp32 [T, Hq] contiguous. Rows
    behind offsets[B] keep what they held."""
    cache, B = _cache(k_cache, v_cache, page_table, kv_exp, offsets, seq_lens, (o, _BF16, "o"),
                      (lse, _F32, "lse"))
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [T, Hq, d]")
    q_rows = _rows(q, shape[1], cache.d, "q")
    if o.shape != shape or lse.shape != shape[:2]:
        raise ValueError("o must be [T, Hq, d] and lse [T, Hq]")
    _prefill_launch(cache, B, q_rows, shape[0], shape[1], offsets, seq_lens, o, lse, workspace,
                    _workspace_bytes(workspace), max_new, max_seq_len, split_keys, scale,
                    mask_kind, window, score_kind, softcap, stream)


def prefill_paged(q, k_cache, v_cache, page_table, offsets, seq_lens, *, kv_exp=None,
                  max_new: Optional[int] = None, max_seq_len: Optional[int] = None,
                  split_keys: Optional[int] = None, total_kv_tokens: Optional[int] = None,
                  scale: Optional[float] = None, mask_kind: int = MASK_NONE, window: int = 0,
                  score_kind: int = SCORE_NONE, softcap: float = 0.0, stream=None):
    """Allocating form of prefill_paged_into: (o, lse) of the chunks' rows. max_new (the
    longest chunk) defaults to T, max_seq_len to the page table's capacity, split_keys to
    the library's choice (total_kv_tokens, the sum of seq_lens when the caller knows it,
    lets it weigh long sequences against short ones)."""
    cache, B = _cache(k_cache, v_cache, page_table, kv_exp, offsets, seq_lens)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [T, Hq, d]")
    T, Hq, d = shape
    q_rows = _rows(q, Hq, cache.d, "q")
    if max_seq_len is None:
        max_seq_len = cache.max_pages_per_seq * cache.page_size
    if max_new is None:
        max_new = T
    if split_keys is None:
        split_keys = prefill_split_keys(cache.kind, B, T, Hq, cache.Hkv, max_new, max_seq_len,
                                        total_kv_tokens or B * max_seq_len)
    if scale is None:
        scale = float(d) ** -0.5
    device = q.device
    o = torch.empty(shape, dtype=_BF16, device=device)
    lse = torch.empty((T, Hq), dtype=_F32, device=device)
    nbytes = prefill_workspace_size(T, Hq, d, max_seq_len, split_keys)
    ws = torch.empty((nbytes,), dtype=_U8, device=device) if nbytes else None
    _prefill_launch(cache, B, q_rows, T, Hq, offsets, seq_lens, o, lse, ws, nbytes, max_new,
                    max_seq_len, split_keys, scale, mask_kind, window, score_kind, softcap, stream)
    return o, lse
