"""Softmax attention and its paged key-value cache, on torch tensors in device
memory: the layers of a stack that stand beside the recurrent ones of mixer.py.

Every value is computed by the kernels behind ``include/gdr.h``, which documents
shapes, dtypes and errors; the marshalling is compiled (``csrc/gdr_torch.cpp``).
"""
from __future__ import annotations

from .mixer import _t


def attn_fwd(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, window=0, scale=None, output_lse=True, o=None,
             lse=None):
    """Softmax attention: q ``[B, Tq, Hq, d]``, k and v ``[B, Tk, Hk, d]`` (rows
    may be slices of a wider projection), Hq a multiple of Hk, ``cu_seqlens``
    int32 ``[N+1]`` (B == 1), ``cu_seqlens_k`` likewise where the keys have
    other lengths.  Causal: the last query of a sequence is beside its last key,
    and with ``window`` a query sees that many keys at most.  ``scale`` None:
    ``d ** -0.5``.  Returns ``(o, lse)``: lse fp32 ``[B, Tq, Hq]`` (None unless
    ``output_lse``) is what the gradient needs."""
    return _t.attn_fwd(q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale, output_lse, o, lse)


def attn_bwd(q, k, v, o, lse, do, cu_seqlens=None, cu_seqlens_k=None, causal=True, window=0, scale=None, dq=None, dk=None,
             dv=None):
    """Gradients of ``attn_fwd`` given its ``(o, lse)`` and do ``[B, Tq, Hq, d]``:
    ``(dq, dk, dv)`` in q's dtype, dk and dv summed over each key head's group."""
    return _t.attn_bwd(q, k, v, o, lse, do, cu_seqlens, cu_seqlens_k, causal, window, scale, dq, dk, dv)


def attn_paged_step(q, k_pages, v_pages, block_table, lens, window=0, scale=None, o=None):
    """Attention of one new token per sequence, q ``[N, Hq, d]``, over the
    ``lens`` (int32 ``[N]``) keys in the pages ``block_table`` (int32 ``[N, M]``)
    names of k_pages and v_pages ``[P, page, Hk, d]``.  Returns o ``[N, Hq, d]``."""
    return _t.attn_paged_step(q, k_pages, v_pages, block_table, lens, window, scale, o)


def page_plan(past, new, free_pages, block_table, page, tokens, cu_seqlens=None, lens=None, positions=None, slots=None,
              used=None):
    """Where the next tokens of N requests go: past and new int32 ``[N]`` count
    the tokens each has and gets, ``tokens`` (on the host) is at least their sum;
    block_table int32 ``[N, M]`` is updated in place with pages from free_pages.
    Returns ``(cu_seqlens, lens, positions, slots, used)``: offsets ``[N+1]``,
    past + new ``[N]``, place in the request and row in the pages ``[1, tokens]``
    (-1: no page; given ones may be ``[tokens]``), and ``[2]`` the tokens and pages
    taken."""
    return _t.page_plan(past, new, free_pages, block_table, page, tokens, cu_seqlens, lens, positions, slots, used)


def page_store(k, v, slots, k_pages, v_pages):
    """Copies k and v ``[B, T, Hk, d]`` to the rows ``slots`` (int32 ``[B, T]``
    or ``[B * T]``) of k_pages and v_pages ``[P, page, Hk, d]``; a negative slot stores nothing."""
    _t.page_store(k, v, slots, k_pages, v_pages)
