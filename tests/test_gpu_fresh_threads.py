"""Calls that are the first of their thread: nothing on it has made the device's context current."""
import threading

import pytest
import torch

import exact_attention_37_gb300 as fa

from .test_gpu_kv4_tree import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def in_a_new_thread(f):
    err = []

    def work():
        try:
            f()
        except Exception as e:  # noqa: BLE001
            err.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not err, err
    torch.cuda.synchronize()


def test_forward_and_backward_first():
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(1, 4, 300, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    o, lse = fa.forward(q, k, v, scale=0.125, causal=True)
    grads = fa.backward(q, k, v, o, lse, do, scale=0.125, causal=True)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    in_a_new_thread(lambda: fa.fa_fwd(q, k, v, o2, lse2, 0.125, True))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    out = [torch.empty_like(x) for x in grads]
    ws = torch.empty(fa.fa_bwd_workspace_size(1, 4, 300, 64), dtype=torch.uint8, device="cuda")
    in_a_new_thread(lambda: fa.fa_bwd(q, k, v, o, do, lse, *out, ws, 0.125, True))
    assert all(torch.equal(x, y) for x, y in zip(grads, out))
    rule = fa.ScoreRule(causal=True, cap=20.0)
    want = fa.forward_rule(q, k, v, rule, scale=0.125)
    ws = torch.empty(max(256, fa.fa_fwd_rule_workspace_size(1, 4, 300, 300, 64, False)), dtype=torch.uint8, device="cuda")
    in_a_new_thread(lambda: fa.fa_fwd_rule(q, k, v, o2, lse2, rule, ws, 0.125))
    assert torch.equal(want[0], o2) and torch.equal(want[1], lse2)
    fa.fa_check_device_status()


@pytest.mark.parametrize("room", [900, 30000])
def test_calls_of_a_drafting_server_first(room):
    s, t = Step(seed=5, N=19, room=room), Step(seed=5, N=19, room=room)
    s.admit(), t.admit()
    want = s.draft()
    B, H, Hkv, N, d, page = t.shape
    par, count, _ = t.t
    out_count, lens = torch.empty_like(count), torch.empty_like(count)
    slots, pos = torch.empty(B, N, dtype=torch.int64, device="cuda"), torch.empty(B, N, dtype=torch.int32, device="cuda")
    q, k, o, lse = torch.empty_like(t.q), torch.empty_like(t.k), torch.empty_like(t.q), torch.empty(B, H, N, device="cuda")
    ws = torch.empty(fa.fa_kv4_attend_tree_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8, device="cuda")
    in_a_new_thread(lambda: fa.fa_kv4_plan(t.pages, page, t.length, count, par, out_count, lens, slots, pos))
    in_a_new_thread(lambda: fa.fa_rotary(t.q, t.k, pos, t.freqs, q, k))
    in_a_new_thread(lambda: fa.fa_kv4_append(t.cache, k, t.v, t.pages.table, t.length, out_count))
    in_a_new_thread(lambda: fa.fa_kv4_attend_tree(q, t.cache, t.pages.table, lens, par, out_count, o, lse, ws, d ** -0.5))
    in_a_new_thread(lambda: fa.fa_kv4_keep(t.cache, t.pages.table, t.length, t.path, t.kept))
    for x, y in zip((q, k, o, lse, slots, pos, *t.cache.pools), (*want, *s.cache.pools)):
        assert torch.equal(x, y)
    fa.fa_check_device_status()
