"""The 4-bit cache without a GPU: the token lookup, what the calls refuse, and the format's
definition."""
import ctypes
import types

import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from exact_attention_37_gb300 import _lib
from exact_attention_37_gb300 import build as fabuild
from oracle import kv4


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return _lib.load()


@pytest.mark.parametrize("page_size", [16, 64, 1024])
def test_lookup_of_tokens_and_of_bad_pages(lib, page_size):
    pages = [3, 0, 7, -1, 8, 2 ** 31 - 1, -2 ** 31]
    row = lambda pos: fa.fa_kv4_row(pages, page_size, 8, pos)  # noqa: E731
    assert row(0) == 3 * page_size and row(page_size - 1) == 4 * page_size - 1
    assert row(page_size) == 0 and row(3 * page_size - 1) == 8 * page_size - 1
    for bad in (-1, -2 ** 40, 3 * page_size, 4 * page_size, 5 * page_size, 6 * page_size + 5, 7 * page_size, 2 ** 40):
        assert row(bad) == -1
    assert fa.fa_kv4_row([], 64, 8, 0) == -1
    assert fa.fa_kv4_row([0], 24, 8, 0) == -1


def cache_struct(**over):
    a = dict(k_codes=256, k_params=256, v_codes=256, v_params=256, num_pages=4, page_size=16, H_kv=2, d=64, dtype=1)
    a.update(over)
    return _lib.KV4CacheStruct(*a.values())


BAD_CACHES = [(dict(d=96), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=2048), 2), (dict(dtype=5), 1),
              (dict(H_kv=0), 1), (dict(num_pages=-1), 1), (dict(k_codes=0), 1), (dict(v_params=264), 3)]


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, over, code):
    vp, c = ctypes.c_void_p, cache_struct(**over)
    p = vp(256)
    assert lib.fa_kv4_append(ctypes.byref(c), p, p, p, 3, p, None, 2, 5, None) == code
    assert lib.fa_kv4_read(ctypes.byref(c), p, 3, p, p, p, p, 2, 5, None) == code
    assert lib.fa_kv4_attend(p, ctypes.byref(c), p, 3, p, p, p, 1, 0.0, None, p, 1 << 30, 2, 4, 1, 0.1, None) == code


def test_bad_arguments_are_refused(lib):
    vp = ctypes.c_void_p
    c, p, z = ctypes.byref(cache_struct()), vp(256), vp(0)
    assert lib.fa_kv4_append(None, p, p, p, 3, p, None, 2, 5, None) == 1
    assert lib.fa_kv4_append(c, z, p, p, 3, p, None, 2, 5, None) == 1
    assert lib.fa_kv4_append(c, p, p, z, 3, p, None, 2, 5, None) == 1
    assert lib.fa_kv4_append(c, p, p, p, 3, z, None, 2, 5, None) == 1
    assert lib.fa_kv4_append(c, vp(264), p, p, 3, p, None, 2, 5, None) == 3
    assert lib.fa_kv4_append(c, p, p, p, 3, vp(258), None, 2, 5, None) == 3
    assert lib.fa_kv4_append(c, p, p, p, 1 << 27, p, None, 2, 5, None) == 2  # 2^31 tokens a sequence
    assert lib.fa_kv4_append(c, p, p, p, 3, p, None, -2, 5, None) == 1
    assert lib.fa_kv4_append(c, z, z, z, 3, z, None, 0, 5, None) == 0        # nothing to store
    assert lib.fa_kv4_read(c, p, 3, p, z, p, p, 2, 5, None) == 1
    assert lib.fa_kv4_read(c, p, 3, p, p, p, p, 2, 0, None) == 0
    at = lambda **o: lib.fa_kv4_attend(*[{**dict(q=p, c=c, t=p, m=3, l=p, o=p, s=p, causal=1, cap=0.0, sl=z, ws=p, b=1 << 30, B=2,  # noqa: E731
                                                H=4, N=1, scale=0.1, st=None), **o}[k] for k in
                                         ("q", "c", "t", "m", "l", "o", "s", "causal", "cap", "sl", "ws", "b", "B", "H", "N",
                                          "scale", "st")])
    assert at(H=3) == 1
    assert at(cap=-1.0) == 1 and at(cap=float("nan")) == 1 and at(scale=0.0) == 1
    assert at(sl=vp(258)) == 3
    assert at(ws=z) == 4 and at(b=100) == 4 and at(ws=vp(256 + 16)) == 3
    assert at(B=4097) == 2
    assert at(q=z) == 1 and at(l=z) == 1
    assert at(N=0) == 0 and at(B=0) == 0
    assert lib.fa_kv4_attend_workspace_size(2, 4, 2, 1, 64) > 0
    assert lib.fa_kv4_attend_workspace_size(2, 3, 2, 1, 64) == 0
    assert lib.fa_kv4_attend_workspace_size(0, 4, 2, 1, 64) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_workspace_does_not_grow_with_the_rows(lib, d):
    """It holds what stretches leave of the units they cut, two a CTA, not a place for each unit."""
    size = lambda B, Nq: lib.fa_kv4_attend_workspace_size(B, 32, 8, Nq, d)  # noqa: E731
    assert size(1, 64) == size(4096, 64) == size(4, 4096) == size(1, 1 << 20) <= 22 << 20
    assert 0 < size(1, 1) == size(4096, 1) <= size(1, 64)


def rule_struct(**over):
    a = dict(causal=1, cap=0.0, slopes=0, q_doc=0, k_doc=0, prefix=0)
    a.update(over)
    return _lib.ScoreRuleStruct(*a.values())


def test_bad_rules_are_refused(lib):
    vp, p = ctypes.c_void_p, ctypes.c_void_p(256)

    def fwd(rule, ws=p, size=1 << 30, B=1, N=8, d=64):
        return lib.fa_fwd_rule(p, p, p, p, p, rule and ctypes.byref(rule), ws, size, B, 2, 1, N, N, d, 0.1, 1, None)

    def bwd(rule, ws=p, size=1 << 30, N=8):
        return lib.fa_bwd_rule(*([p] * 9), rule and ctypes.byref(rule), ws, size, 1, 2, 1, N, N, 64, 0.1, 1, None)

    for call in (fwd, bwd):
        assert call(None) == 1
        for cap in (-1.0, float("nan"), float("inf"), 1e-40):
            assert call(rule_struct(cap=cap)) == 1
        assert call(rule_struct(q_doc=256)) == 1 and call(rule_struct(k_doc=256)) == 1
        assert call(rule_struct(slopes=258)) == 3 and call(rule_struct(prefix=257)) == 3
        assert call(rule_struct(q_doc=256, k_doc=256), ws=vp(0)) == 4
        assert call(rule_struct(q_doc=256, k_doc=256), size=64) == 4
        assert call(rule_struct(q_doc=256, k_doc=256), ws=vp(272)) == 3
    assert bwd(rule_struct(), ws=vp(0)) == 4  # the row vectors
    assert fwd(rule_struct(), d=80) == 2
    assert fwd(rule_struct(), N=0) == 0 and fwd(rule_struct(), B=0) == 0
    assert lib.fa_fwd_rule_workspace_size(1, 2, 300, 300, 64, 0) == 0
    assert lib.fa_fwd_rule_workspace_size(1, 2, 300, 300, 64, 1) > 0
    assert lib.fa_bwd_rule_workspace_size(1, 2, 300, 300, 64, 0) == lib.fa_bwd_workspace_size(1, 2, 300, 64)
    assert lib.fa_bwd_rule_workspace_size(1, 2, 300, 300, 96, 1) == 0


def test_ids_of_a_side_without_rows_may_be_null(lib):
    """An empty array has no address."""
    p = ctypes.c_void_p(256)

    def call(name, rule, B, Nq, Nk, H=2):
        ptrs = [p] * (5 if name == "fa_fwd_rule" else 9)
        return getattr(lib, name)(*ptrs, ctypes.byref(rule), p, 1 << 30, B, H, 1, Nq, Nk, 64, 0.1, 1, None)

    q, k = rule_struct(q_doc=256), rule_struct(k_doc=256)
    assert call("fa_fwd_rule", k, 2, 0, 30) == 0 and call("fa_fwd_rule", k, 2, 0, 0) == 0
    assert call("fa_fwd_rule", k, 0, 8, 30) == 0 and call("fa_fwd_rule", q, 0, 8, 30) == 0
    assert call("fa_bwd_rule", k, 2, 0, 0) == 0 and call("fa_bwd_rule", q, 0, 8, 8) == 0
    assert call("fa_fwd_rule", q, 2, 0, 30) == 1 and call("fa_fwd_rule", k, 2, 8, 30) == 1
    assert call("fa_fwd_rule", q, 2, 8, 0, H=0) == 0 and call("fa_fwd_rule", q, 2, 8, 0) == 2


def test_python_checks_before_the_library():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.float16)
    for call in (lambda: fa.forward_rule(q, q, q, fa.ScoreRule()),
                 lambda: fa.backward_rule(q, q, q, q, q, q, fa.ScoreRule()),
                 lambda: fa.KV4Cache.empty(2, 2, 16, 64, torch.float16, device="cpu")):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):
            call()
    with pytest.raises(TypeError):
        fa.KV4Cache.empty(2, 2, 16, 64, torch.float32, device="cpu")


def test_caller_owned_cache_calls_check_what_the_allocating_ones_check():
    """Arrays that have to be there, and a cache without heads (tensors of no device stand in
    for a device's)."""
    t = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = lambda H: types.SimpleNamespace(dev=-1, dtype=torch.float16, H_kv=H, d=64)  # noqa: E731
    k, q, lse = t(2, 2, 3, 64), t(2, 4, 1, 64), torch.zeros(2, 4, 1)
    for call in (lambda: fa.fa_kv4_append(cache(2), k, k, i(2, 3), None), lambda: fa.fa_kv4_append(cache(2), k, k, i(2, 3), None, i(2)),
                 lambda: fa.fa_kv4_append(cache(2), k, k, i(2, 3), i(2), i(3)), lambda: fa.fa_kv4_append(cache(3), k, k, i(2, 3), i(2)),
                 lambda: fa.fa_kv4_read(cache(2), i(2, 3), None, i(2), k, k), lambda: fa.fa_kv4_read(cache(2), i(2, 3), i(2), None, k, k),
                 lambda: fa.fa_kv4_attend(q, cache(2), i(2, 3), None, q, lse, None, 0.1),
                 lambda: fa.fa_kv4_attend(q, cache(0), i(2, 3), i(2), q, lse, None, 0.1),
                 lambda: fa.fa_kv4_attend(q, cache(3), i(2, 3), i(2), q, lse, None, 0.1),
                 lambda: fa.fa_kv4_attend(q, cache(2), i(2, 3), i(2), q, lse[:, :3], None, 0.1),
                 lambda: fa.fa_kv4_attend(q[0], cache(2), i(2, 3), i(2), q[0], lse[0], None, 0.1)):
        with pytest.raises(ValueError):
            call()


def test_a_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), device_index=1, cuda_stream=77)
    x = types.SimpleNamespace(device=torch.device("cuda", 0), pools=())
    rule = fa.ScoreRule()
    for call in (lambda: fa.forward_rule(x, x, x, rule, stream=stream),
                 lambda: fa.backward_rule(x, x, x, x, x, x, rule, stream=stream),
                 lambda: fa.kv4_append(x, x, x, x, x, stream=stream), lambda: fa.kv4_read(x, x, x, 1, x, stream=stream),
                 lambda: fa.kv4_attend(x, x, x, x, stream=stream), lambda: _lib._raw_stream(stream, 0)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert _lib._raw_stream(stream, 1) == 77


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_format_is_within_half_a_step(dtype):
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(50, 128, generator=g) * torch.exp(2 * torch.randn(50, 1, generator=g)) + 3).to(dtype)
    x[0] = 0
    x[1] = 1.5
    codes, scale, low = kv4.store(x)
    assert codes.min() >= 0 and codes.max() == 15
    v = kv4.values(codes, scale, low, dtype)
    step = np.repeat(scale, 32, -1)
    eps = torch.finfo(dtype).eps
    # half a step, the scale's own rounding over 15 steps (eps / 2 each), and the value's rounding
    assert (np.abs(v - x.double().numpy()) <= step * (0.5 + 15 * eps) + np.abs(v) * eps / 2 + 1e-6).all()
    assert (v[0] == 0).all() and (v[1] == 1.5).all()
