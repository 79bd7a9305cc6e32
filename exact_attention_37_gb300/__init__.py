"""Exact scaled-dot-product attention for GB300 (sm_103a): fused forward with online
softmax and a key-block-parallel backward, behind a small C ABI.

    import exact_attention_37_gb300 as fa
    o, lse = fa.forward(q, k, v, causal=True)          # q: [B, H, N_q, d], k, v: [B, H_kv, N_k, d]
    dq, dk, dv = fa.backward(q, k, v, o, lse, dout, causal=True)

H_kv may be smaller than H (grouped-query / multi-query attention) and N_k may
differ from N_q (the causal mask is then aligned at the bottom right).

    rule = fa.ScoreRule(causal=True, cap=50.0, q_doc=ids, k_doc=ids)   # capped scores, packed documents
    o, lse = fa.forward_rule(q, k, v, rule)
    dq, dk, dv = fa.backward_rule(q, k, v, o, lse, dout, rule)

    cache = fa.KV4Cache.empty(pages, H_kv, 64, 128, torch.bfloat16)    # a paged cache in 4 bits
    fa.kv4_append(cache, k_new, v_new, page_table, start)
    o, lse = fa.kv4_attend(q_new, cache, page_table, lengths, cap=50.0)

    freqs = fa.rotary_freqs(128)                                       # rotary positions, either direction
    q, k = fa.rotary(q, k, positions, freqs)
    dq, dk = fa.rotary_backward(dq, dk, positions, freqs)

    pages = fa.KV4Pages.empty(B, max_pages, num_pages)                 # a step of a server that drafts trees of tokens
    count, lengths, slots, positions = fa.kv4_plan(pages, 64, start, count, N, parents=parents)
    fa.kv4_append(cache, k, v, pages.table, start, count)
    o, lse = fa.kv4_attend_tree(q, cache, pages.table, lengths, parents, count)
    fa.kv4_keep(cache, pages.table, start, path, kept)                 # the accepted branch

``forward``/``backward`` allocate their outputs with torch and call the C ABI;
``fa_fwd``/``fa_bwd`` take caller-owned outputs.  All compute runs in the
library's CUDA kernels; there is no CPU fallback.
"""
from __future__ import annotations

import math

from ._lib import (  # noqa: F401
    FA_BF16,
    FA_FP16,
    FaError,
    KV4Cache,
    KV4Pages,
    ScoreRule,
    fa_bwd,
    fa_bwd_rule,
    fa_bwd_rule_workspace_size,
    fa_profile_begin,
    fa_profile_end,
    fa_bwd_workspace_size,
    fa_check_device_status,
    fa_fwd,
    fa_fwd_bwd_host,
    fa_fwd_host,
    fa_fwd_rule,
    fa_fwd_rule_workspace_size,
    fa_cta_head_group,
    fa_host_chunk_plan,
    fa_host_scratch_size,
    fa_kv4_append,
    fa_kv4_attend,
    fa_kv4_attend_tree,
    fa_kv4_attend_tree_workspace_size,
    fa_kv4_attend_workspace_size,
    fa_kv4_keep,
    fa_kv4_plan,
    fa_kv4_read,
    fa_kv4_row,
    fa_kv4_tree_many_rows,
    fa_rotary,
    fa_rotary_turns,
    fa_status_string,
    fa_version,
    load,
    native,
)

__all__ = ["forward", "backward", "fa_fwd", "fa_bwd", "fa_bwd_workspace_size", "fa_check_device_status",
           "fa_fwd_host", "fa_fwd_bwd_host", "fa_host_scratch_size", "fa_host_chunk_plan", "fa_cta_head_group",
           "FaError", "load", "ScoreRule", "forward_rule", "backward_rule", "fa_fwd_rule", "fa_bwd_rule",
           "fa_fwd_rule_workspace_size", "fa_bwd_rule_workspace_size", "KV4Cache", "kv4_append", "kv4_read",
           "kv4_attend", "fa_kv4_append", "fa_kv4_read", "fa_kv4_attend", "fa_kv4_attend_workspace_size",
           "fa_kv4_row", "fa_kv4_tree_many_rows", "KV4Pages", "kv4_plan", "kv4_attend_tree", "kv4_keep", "rotary", "rotary_backward", "rotary_freqs",
           "fa_kv4_plan", "fa_kv4_attend_tree", "fa_kv4_attend_tree_workspace_size", "fa_kv4_keep", "fa_rotary",
           "fa_rotary_turns"]


def _default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def forward(q, k, v, scale: float | None = None, causal: bool = False, stream=None):
    """Returns (O, L): O like q, L fp32 [B, H, N]."""
    import torch

    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, _default_scale(d) if scale is None else scale, causal, stream)
    return o, lse


def backward(q, k, v, o, lse, dout, scale: float | None = None, causal: bool = False, stream=None, workspace=None):
    """Returns (dQ, dK, dV) like q, k, v.  ``workspace`` (uint8 CUDA tensor) is allocated if not given."""
    import torch

    B, H, N, d = q.shape
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(max(1, fa_bwd_workspace_size(B, H, N, d)), dtype=torch.uint8, device=q.device)
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, _default_scale(d) if scale is None else scale, causal,
           stream)
    return dq, dk, dv


def _result(where: str, r):
    """Outputs of a native call, or the exception for the status it returned."""
    if r.__class__ is int:
        raise FaError(where, r)
    return r


def _on(stream, x, *read):
    """Makes ``stream`` current: outputs and workspaces are allocated for it, so that memory
    that a call drops is reused in that stream's order.  It has to be one of the device that
    ``x`` is on: another device's would be current there and not used.  What the call reads
    (``x`` and ``read``) may be dropped by the caller as soon as it returns: its memory is not
    reused before ``stream`` is done with it."""
    import torch

    if stream.device != getattr(x, "device", None):
        raise ValueError("the stream must be one of the tensors' device")
    for t in (x, *read):
        if isinstance(t, torch.Tensor) and t.device == stream.device:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _arrays(rule):
    return rule.slopes, rule.q_doc, rule.k_doc, rule.prefix


def forward_rule(q, k, v, rule: ScoreRule, scale: float | None = None, stream=None):
    """Forward pass with a score rule (cap, distance bias, documents, prefix, causal mask).
    Returns (O, L): O like q, L fp32 [B, H, N_q], -inf for rows that see nothing.  scale: 1/sqrt(d) if None."""
    if stream is not None:
        with _on(stream, q, k, v, *_arrays(rule)):
            return forward_rule(q, k, v, rule, scale)
    return _result("fa_fwd_rule", native().forward_rule(q, k, v, rule.causal, rule.cap, rule.slopes, rule.q_doc, rule.k_doc,
                                                        rule.prefix, scale))


def backward_rule(q, k, v, o, lse, dout, rule: ScoreRule, scale: float | None = None, stream=None, workspace=None):
    """Gradients (dQ, dK, dV) like q, k, v of the forward pass with the same rule."""
    if stream is not None:
        with _on(stream, q, k, v, o, lse, dout, workspace, *_arrays(rule)):
            return backward_rule(q, k, v, o, lse, dout, rule, scale, None, workspace)
    return _result("fa_bwd_rule", native().backward_rule(q, k, v, o, lse, dout, rule.causal, rule.cap, rule.slopes, rule.q_doc,
                                                         rule.k_doc, rule.prefix, scale, workspace))


def kv4_append(cache: KV4Cache, k, v, page_table, start, count=None, stream=None):
    """Stores rows k, v [B, H_kv, N, d] as tokens start[b] + i (i < count[b]) of the cache's sequences."""
    if stream is not None:
        with _on(stream, cache, *cache.pools, k, v, page_table, start, count):
            return kv4_append(cache, k, v, page_table, start, count)
    _result("fa_kv4_append", native().kv4_append(*cache.pools, k, v, page_table, start, count))


def kv4_read(cache: KV4Cache, page_table, start, N: int, lengths, stream=None):
    """(k, v) [B, H_kv, N, d]: the values of tokens start[b] .. start[b] + N - 1, zeros from lengths[b] on."""
    if stream is not None:
        with _on(stream, cache, *cache.pools, page_table, start, lengths):
            return kv4_read(cache, page_table, start, N, lengths)
    return _result("fa_kv4_read", native().kv4_read(*cache.pools, page_table, start, N, lengths))


def kv4_attend(q, cache: KV4Cache, page_table, lengths, scale: float | None = None, causal: bool = True,
               cap: float = 0.0, slopes=None, stream=None, workspace=None):
    """(O, L) of each sequence's last N_q tokens q [B, H, N_q, d] over its lengths[b] cached tokens.  Many causal rows
    are faster as a chain of drafted ones (kv4_attend_tree with parents -1, 0, 1, ..) where fa_kv4_tree_many_rows says so."""
    if stream is not None:
        with _on(stream, cache, *cache.pools, q, page_table, lengths, slopes, workspace):
            return kv4_attend(q, cache, page_table, lengths, scale, causal, cap, slopes, None, workspace)
    return _result("fa_kv4_attend", native().kv4_attend(q, *cache.pools, page_table, lengths, scale, causal, cap, slopes,
                                                        workspace))


def kv4_attend_tree(q, cache: KV4Cache, page_table, lengths, parents, count=None, scale: float | None = None, cap: float = 0.0,
                    slopes=None, stream=None, workspace=None):
    """(O, L) of a tree of drafted tokens q [B, H, N_q, d], the last count[b] (None: N_q) of each sequence's
    lengths[b] cached tokens: each sees the tokens in front of the draft, its ancestors and itself.  parents [B, N_q]
    int32: the drafted token that each one follows, -1 for the cached ones."""
    if stream is not None:
        with _on(stream, cache, *cache.pools, q, page_table, lengths, parents, count, slopes, workspace):
            return kv4_attend_tree(q, cache, page_table, lengths, parents, count, scale, cap, slopes, None, workspace)
    return _result("fa_kv4_attend_tree", native().kv4_attend_tree(q, *cache.pools, page_table, lengths, parents, count, scale, cap,
                                                                  slopes, workspace))


def kv4_keep(cache: KV4Cache, page_table, start, path, kept, stream=None):
    """Tokens start[b] + path[b, j] of the cache become tokens start[b] + j, for j < kept[b]: the accepted
    branch of a draft moves together.  path [B, N] int32, N <= 128."""
    if stream is not None:
        with _on(stream, cache, *cache.pools, page_table, start, path, kept):
            return kv4_keep(cache, page_table, start, path, kept)
    _result("fa_kv4_keep", native().kv4_keep(*cache.pools, page_table, start, path, kept))


def kv4_plan(pages: KV4Pages, page_size: int, start, count, N: int, parents=None, stream=None):
    """Pages for count[b] <= N tokens behind start[b] of every sequence, from (and back to) the free ones of ``pages``,
    which it changes.  Returns (count, lengths, slots, positions): count [B], 0 for sequences that got no room; lengths
    [B] = start + count; the new tokens' rows in the pool and their positions [B, N], -1 behind count.  With the
    parents of drafted tokens, positions go by depth.  start = count = 0 ends a sequence."""
    if stream is not None:
        with _on(stream, pages, *pages.arrays, start, count, parents):
            return kv4_plan(pages, page_size, start, count, N, parents)
    return _result("fa_kv4_plan", native().kv4_plan(*pages.arrays, page_size, start, count, N, parents))


def rotary(q, k, positions, freqs, interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """(q, k) with channels in pairs turned by positions[b, n] * freqs[i] radians: q [B, H, N, d], k [B, H_kv, N, d]
    (or None) with any strides, positions [B, N] int32 (None: 0 .. N - 1), freqs [dims / 2] float64 (rotary_freqs).
    Pairs are channels (i, i + dims / 2), or (2 i, 2 i + 1) if interleaved; channels from dims on are copied, the
    others multiplied by ``amplitude`` too.  out: (q, k) to write, which may be the inputs; contiguous if None."""
    if stream is not None:
        with _on(stream, q, k, positions, freqs, *(out or ())):
            return rotary(q, k, positions, freqs, interleaved, amplitude, out)
    out_q, out_k = out or (None, None)
    return _result("fa_rotary", native().rotary(q, k, positions, freqs, interleaved, False, amplitude, out_q, out_k))


def rotary_backward(dq, dk, positions, freqs, interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """Gradients of ``rotary``'s inputs from those of its outputs, with the same other arguments."""
    if stream is not None:
        with _on(stream, dq, dk, positions, freqs, *(out or ())):
            return rotary_backward(dq, dk, positions, freqs, interleaved, amplitude, out)
    out_q, out_k = out or (None, None)
    return _result("fa_rotary", native().rotary(dq, dk, positions, freqs, interleaved, True, amplitude, out_q, out_k))


def rotary_freqs(dims: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0, trained: int = 8192,
                 low: float = 1.0, high: float = 4.0, device="cuda"):
    """freqs [dims / 2] of ``rotary``: base^(-2 i / dims) radians a position, for contexts ``factor`` times the
    ``trained`` positions scaled by

      "linear"  all divided by factor
      "ntk"     base times factor^(dims / (dims - 2)): the slowest divided by factor, the fastest as they were
      "bands"   pairs with at most ``low`` turns in the trained positions divided by factor, with at least ``high`` as
                they were, in between a mixture by their turns
    """
    import torch

    if dims < 16 or dims % 16:
        raise ValueError("dims must be a multiple of 16")
    if scaling not in (None, "linear", "ntk", "bands"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'bands'")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base and factor must be finite and above 0")
    if scaling == "bands" and not (trained > 0 and low < high):
        raise ValueError("bands need trained positions and low < high")
    if scaling == "ntk":
        base = base * factor ** (dims / (dims - 2))
    out = []
    for i in range(dims // 2):
        f = base ** (-2.0 * i / dims)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            keep = min(1.0, max(0.0, (trained * f / (2.0 * math.pi) - low) / (high - low)))
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device=device)
