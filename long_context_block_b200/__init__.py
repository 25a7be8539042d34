"""MISA indexer hot path for NVIDIA B200 (sm_100a).

Kernels live in libmisa_b200.so (C ABI in include/misa.h); this package is a thin
binding plus compositions of the entry points:

  misa_indexer  -- pool keys, route heads, routed score + top-k   (Eqs. 4, 7-10)
  misa_dagger   -- misa_indexer with k' candidates, then the all-head re-rank (Eqs. 11-12)
  hisa_indexer  -- the HISA-style token-axis block filter the pages contrast MISA with
  misa_sparse_attention -- an indexer's selection and the attention over it, from a paged
                   key-value cache (misa_paged_*, misa_pages_*)

Reference: "MISA: Mixture of Indexer Sparse Attention for Long-Context LLM
Inference" (picx.dev summary page, Methodology sections 1-2).
"""

from ._binding import (  # noqa: F401
    HEAD_DIM,
    LIB_PATH,
    MisaError,
    declared_symbols,
    dsa_score_topk,
    hisa_block_filter_topk,
    library,
    misa_check_device_status,
    misa_dagger_rerank,
    misa_paged_append,
    misa_paged_attention,
    misa_pages_compact,
    misa_pages_fork,
    misa_pages_resize,
    misa_pool_keys,
    misa_pool_keys_range,
    misa_route_heads,
    misa_score_rows,
    misa_score_topk,
    misa_score_topk_noalloc,
    misa_testing_paged_attention_wait_expiry,
    misa_testing_score_rows_wait_expiry,
    misa_testing_score_rows_timed,
    misa_testing_score_simt,
    misa_workspace_size,
    workspace,
)


def misa_indexer(q, w, k, pos, B: int, h: int, topk: int, return_vals: bool = True,
                 k_pool=None):
    """MISA for a batch of queries: Eq. (4) pooling (skipped when k_pool is given),
    Eqs. (7)-(8) routing, Eqs. (9)-(10) routed scoring and top-k.

    Returns (idx, vals, heads)."""
    if k_pool is None:
        k_pool = misa_pool_keys(k, B)
    heads = misa_route_heads(q, w, k, k_pool, pos, B, h)
    idx, vals = misa_score_topk(q, w, k, heads, pos, topk, return_vals=True)
    return (idx, vals, heads) if return_vals else (idx, None, heads)


def misa_dagger(q, w, k, pos, B: int, h: int, topk: int, kprime: int, k_pool=None):
    """MISA-dagger: routed coarse top-k' (Eq. 11), then the all-head re-rank to top-k
    (Eq. 12).  Returns (idx, vals, cand, heads)."""
    if k_pool is None:
        k_pool = misa_pool_keys(k, B)
    heads = misa_route_heads(q, w, k, k_pool, pos, B, h)
    cand = misa_score_topk(q, w, k, heads, pos, kprime, return_vals=False)
    idx, vals = misa_dagger_rerank(q, w, k, pos, cand, topk)
    return idx, vals, cand, heads


def hisa_indexer(q, w, k, pos, B: int, m: int, topk: int, k_pool=None):
    """HISA-style block filter: pool with B (skipped when k_pool is given), keep each
    query's top-m blocks by head-summed affinity, top-k of the all-head scores of their
    tokens.  Returns (idx, vals, blocks)."""
    if k_pool is None:
        k_pool = misa_pool_keys(k, B)
    return hisa_block_filter_topk(q, w, k, k_pool, pos, B, m, topk, return_blocks=True)


def misa_sparse_attention(qi, w, ki, pos, B: int, h: int, topk: int, q, k_cache, v_cache,
                          page_table, k_new=None, v_new=None, k_pool=None,
                          kprime: int | None = None, scale: float | None = None):
    """One step of sparse attention: the step's keys and values (k_new / v_new, when given) into
    their pages, misa_indexer's tokens of every query (misa_dagger's with kprime), and attention
    over them.  qi, w, ki: the indexer's queries, head weights and keys (the step's included); q:
    the attention's queries; pos: the positions of both, -1 for padded rows, which append nothing,
    select nothing (idx -1) and get out 0.  ki is dense, [nseq, L, 128]: a caller that forks pages
    reorders its rows too.  The indexer's workspace is one per device: calls on several streams must
    not overlap.  Returns (out, idx, heads)."""
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new come together")
    if k_new is not None:
        misa_paged_append(k_new, v_new, pos, page_table, k_cache, v_cache)
    if kprime is None:
        idx, _, heads = misa_indexer(qi, w, ki, pos, B, h, topk, return_vals=False, k_pool=k_pool)
    else:
        idx, _, _, heads = misa_dagger(qi, w, ki, pos, B, h, topk, kprime, k_pool=k_pool)
    out = misa_paged_attention(q, k_cache, v_cache, page_table, pos, idx=idx, scale=scale)
    return out, idx, heads
