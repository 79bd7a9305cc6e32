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
    fa_kv4_attend_workspace_size,
    fa_kv4_read,
    fa_kv4_row,
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
           "fa_kv4_row"]


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
    """(O, L) of each sequence's last N_q tokens q [B, H, N_q, d] over its lengths[b] cached tokens."""
    if stream is not None:
        with _on(stream, cache, *cache.pools, q, page_table, lengths, slopes, workspace):
            return kv4_attend(q, cache, page_table, lengths, scale, causal, cap, slopes, None, workspace)
    return _result("fa_kv4_attend", native().kv4_attend(q, *cache.pools, page_table, lengths, scale, causal, cap, slopes,
                                                        workspace))
