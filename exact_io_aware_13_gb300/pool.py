"""Which sequence holds which page of a paged cache, on the device: fork, resize, compact and copy,
and the verification of drafted tokens, whose result says how far the cache is rolled back. On
the C ABI (include/attn.h states the rules in full; csrc/binding.cpp checks the tensors).

Three int32 tensors hold the state and are changed in place: page_table [B, max_pages], seq_lens
[B] and page_refs [pages], the number of table entries that hold each page (0: free). A decode
loop with drafted tokens runs without a host round trip:

    missing = cache_resize(k_cache, v_cache, table, lens, refs, lens + n_new)
    rows = offsets * (missing == 0)                        # no rows where the pool is full
    cache_write(...); o, _ = prefill_paged(...)            # of rows: score the drafts
    accepted, token, kept = verify_drafts(probs, tokens, rows, u, u2, draft=q, seq_lens=lens)
    cache_resize(k_cache, v_cache, table, lens, refs, kept)  # roll back

Without `rows`, or a look at `missing`, the calls behind a refused cache_resize take the last cached
tokens for the new ones: they are overwritten, in shared pages too, and rolled back.

Wrong tensors raise ValueError, a refusal of the library AttnError. workspace (default: made for
the call) is a tensor of the bytes that the call's size function gives, 256-byte aligned, not
shared with a concurrent call. stream (default: the current one) may be another stream of the
device: the call waits for nothing on the current one, and the tensors that it makes are memory
of that stream.
"""
from __future__ import annotations

from . import _lib


def fork_workspace_size(B: int, max_pages: int) -> int:
    return int(_lib.load().attn_fork_workspace_size(int(B), int(max_pages)))


def resize_workspace_size(B: int, max_pages: int, num_pages: int) -> int:
    return int(_lib.load().attn_resize_workspace_size(int(B), int(max_pages), int(num_pages)))


def compact_workspace_size(num_pages: int) -> int:
    return int(_lib.load().attn_compact_workspace_size(int(num_pages)))


def copy_workspace_size(num_pages_to: int, n: int) -> int:
    return int(_lib.load().attn_copy_workspace_size(int(num_pages_to), int(n)))


def cache_fork(page_table, seq_lens, page_refs, parents, *, page_size: int, workspace=None,
               stream=None) -> None:
    """Row i takes over what row parents[i] held (int32 [B]; negative: row i becomes empty, i:
    it stays). Rows with one parent share its pages, the partly filled last one too:
    cache_resize copies that one before one of them writes into it."""
    status = _lib.binding().cache_fork(page_table, seq_lens, page_refs, parents, page_size,
                                       workspace, stream)
    if status is not None:
        _lib.check(status, "attn_cache_fork")


def cache_resize_into(k_cache, v_cache, page_table, seq_lens, page_refs, new_lens, missing,
                      workspace, *, kv_exp=None, window: int = 0, stream=None) -> None:
    """cache_resize with the caller's missing (int32 [1]) and workspace."""
    if missing is None:
        raise ValueError("missing must be a tensor")
    out = _lib.binding().cache_resize(k_cache, v_cache, page_table, seq_lens, page_refs, new_lens,
                                      kv_exp, window, stream, missing, workspace)
    if out.__class__ is int:
        _lib.check(out, "attn_cache_resize")


def cache_resize(k_cache, v_cache, page_table, seq_lens, page_refs, new_lens, *, kv_exp=None,
                 window: int = 0, stream=None):
    """Take every row to new_lens[b] tokens (int32 [B]): pages for new tokens (a partly filled
    page that others hold too is copied first), pages behind the new length given back, and with
    a sliding window of `window` tokens (0: none) those that it has passed. Returns how many
    free pages lack (int32 [1]); if that is not 0 nothing has changed, seq_lens neither, and the
    new tokens must not be written (see the loop above)."""
    out = _lib.binding().cache_resize(k_cache, v_cache, page_table, seq_lens, page_refs, new_lens,
                                      kv_exp, window, stream, None, None)
    if out.__class__ is int:
        _lib.check(out, "attn_cache_resize")
    return out


def cache_compact_into(k_cache, v_cache, page_table, seq_lens, page_refs, used, page_map, workspace,
                       *, kv_exp=None, stream=None) -> None:
    """cache_compact with the caller's used (int32 [1]), page_map (int32 [pages]) and workspace."""
    if used is None or page_map is None:
        raise ValueError("used and page_map must be tensors")
    out = _lib.binding().cache_compact(k_cache, v_cache, page_table, seq_lens, page_refs, kv_exp,
                                       stream, used, page_map, workspace)
    if out.__class__ is int:
        _lib.check(out, "attn_cache_compact")


def cache_compact(k_cache, v_cache, page_table, seq_lens, page_refs, *, kv_exp=None, stream=None):
    """Move the used pages to the front of the pool. Returns (used, page_map): their number
    (int32 [1]; the pages from there on are free) and each page's new index (int32 [pages], -1
    for a free one)."""
    out = _lib.binding().cache_compact(k_cache, v_cache, page_table, seq_lens, page_refs, kv_exp,
                                       stream, None, None, None)
    if out.__class__ is int:
        _lib.check(out, "attn_cache_compact")
    return out


def cache_copy(k_cache, v_cache, k_to, v_to, src_pages, dst_pages, *, kv_exp=None, kv_exp_to=None,
               workspace=None, stream=None) -> None:
    """Copy page src_pages[i] of one pool to page dst_pages[i] of another (int32 [n]); an entry
    with a negative page is skipped. Both pools may be the same one if no destination is
    another entry's source."""
    status = _lib.binding().cache_copy(k_cache, v_cache, k_to, v_to, src_pages, dst_pages, kv_exp,
                                       kv_exp_to, workspace, stream)
    if status is not None:
        _lib.check(status, "attn_cache_copy")


def verify_drafts_into(target, tokens, offsets, accept_u, sample_u, accepted, next_tokens, *,
                       draft=None, seq_lens=None, kept_lens=None, stream=None) -> None:
    """verify_drafts with the caller's outputs (int32 [B] each; kept_lens with seq_lens)."""
    if accepted is None or next_tokens is None or (seq_lens is not None and kept_lens is None):
        raise ValueError("accepted, next_tokens and, with seq_lens, kept_lens must be tensors")
    out = _lib.binding().verify_drafts(target, tokens, offsets, accept_u, sample_u, draft, seq_lens,
                                       stream, accepted, next_tokens, kept_lens)
    if out.__class__ is int:
        _lib.check(out, "attn_verify_drafts")


def verify_drafts(target, tokens, offsets, accept_u, sample_u, *, draft=None, seq_lens=None,
                  stream=None):
    """Which drafted tokens stay, and the token that follows them, from given uniform random
    numbers. target and draft (fp32, bf16 or fp16 [T, V], contiguous along V) are the
    probabilities of the token after each packed row of the scored chunks; tokens int32 [T], a
    sequence's first row being the token before its drafts; without draft the tokens count as
    drawn with certainty. Rows may be padded; target and draft alike, or their loads take elements
    one by one. Returns (accepted, next_tokens), int32 [B], and with seq_lens the
    lengths that cache_resize rolls back to."""
    out = _lib.binding().verify_drafts(target, tokens, offsets, accept_u, sample_u, draft, seq_lens,
                                       stream, None, None, None)
    if out.__class__ is int:
        _lib.check(out, "attn_verify_drafts")
    return out
