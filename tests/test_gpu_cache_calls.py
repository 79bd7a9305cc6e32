"""How the cache's calls may be made: in the checked build, from several threads, through the
caller-owned forms; what both forms refuse; and what the measurement hook records of the calls
with a score rule."""
import ctypes
import threading

import pytest
import torch

import exact_attention_37_gb300 as fa
from exact_attention_37_gb300 import _lib

from . import rules

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Rows of a batch, an empty cache for them, and the calls of a step through either form."""

    def __init__(self, B, H, Hkv, Nq, n, d, dtype, seed=0, page=32, room=None):
        g = torch.Generator().manual_seed(seed)
        per, used = -(-(room or n) // page), -(-n // page)
        self.cache = fa.KV4Cache.empty(B * used, Hkv, page, d, dtype)
        for x in self.cache.pools:
            x.zero_()
        self.table = torch.full((B, per), -1, dtype=torch.int32)
        self.table[:, :used] = torch.randperm(B * used, generator=g).view(B, used)
        self.table = self.table.cuda()
        self.k, self.v = (torch.randn(B, Hkv, n, d, generator=g).to(dtype).cuda() for _ in range(2))
        self.q = torch.randn(B, H, Nq, d, generator=g).to(dtype).cuda()
        self.lens = i32([max(0, n - 11 * b) for b in range(B)])
        self.start = torch.zeros_like(self.lens)
        self.slopes = rules.slopes(H)
        self.shape = (B, H, Hkv, Nq, n, d)

    def native(self):
        fa.kv4_append(self.cache, self.k, self.v, self.table, self.start, self.lens)
        k, v = fa.kv4_read(self.cache, self.table, self.start, self.shape[4], self.lens)
        return k, v, *fa.kv4_attend(self.q, self.cache, self.table, self.lens, cap=8.0, slopes=self.slopes)

    def owned(self, stream=None):
        B, H, Hkv, Nq, n, d = self.shape
        k, v, o, lse = torch.empty_like(self.k), torch.empty_like(self.v), torch.empty_like(self.q), torch.empty(B, H, Nq, device="cuda")
        ws = torch.empty(fa.fa_kv4_attend_workspace_size(B, H, Hkv, Nq, d), dtype=torch.uint8, device="cuda")
        fa.fa_kv4_append(self.cache, self.k, self.v, self.table, self.start, self.lens, stream=stream)
        fa.fa_kv4_read(self.cache, self.table, self.start, self.lens, k, v, stream=stream)
        fa.fa_kv4_attend(self.q, self.cache, self.table, self.lens, o, lse, ws, d ** -0.5, True, 8.0, self.slopes, stream=stream)
        return k, v, o, lse


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


CASES = [  # B, H, Hkv, Nq, n, room: a CTA a unit, clusters, stretches with a small grid and with a full one
    (3, 4, 2, 1, 90, None), (2, 8, 2, 3, 700, None), (1, 4, 1, 2, 700, 8000), (2, 16, 4, 1, 700, 30000)]


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16), (128, torch.bfloat16), (256, torch.bfloat16)])
@pytest.mark.parametrize("B,H,Hkv,Nq,n,room", CASES)
def test_checked_build_runs_the_cache_calls_clean(B, H, Hkv, Nq, n, room, d, dtype):
    """Every device-side check silent, and the results those of the release build."""
    from exact_attention_37_gb300 import build

    lib = _lib.open_library(build.build(debug=True))
    c = Case(B, H, Hkv, Nq, n, d, dtype, room=room)
    want = c.native()
    pools = [x.clone() for x in c.cache.pools]
    for x in c.cache.pools:
        x.zero_()
    k, v, o, lse = (torch.empty_like(x) for x in want)
    ws = torch.empty(lib.fa_kv4_attend_workspace_size(B, H, Hkv, Nq, d), dtype=torch.uint8, device="cuda")
    s, p, room = c.cache.struct(), lambda t: t.data_ptr(), c.table.shape[1]
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    at = ctypes.addressof(s)
    assert lib.fa_kv4_append(at, p(c.k), p(c.v), p(c.table), room, p(c.start), p(c.lens), B, n, st) == 0
    assert lib.fa_kv4_read(at, p(c.table), room, p(c.start), p(c.lens), p(k), p(v), B, n, st) == 0
    assert lib.fa_kv4_attend(p(c.q), at, p(c.table), room, p(c.lens), p(o), p(lse), 1, 8.0, p(c.slopes), p(ws), ws.numel(), B, H, Nq,
                             d ** -0.5, st) == 0
    assert lib.fa_check_device_status(st) == 0
    assert same((k, v, o, lse), want) and same(c.cache.pools, pools)
    assert same(c.owned(), want)
    fa.fa_check_device_status()


def test_cache_calls_from_several_threads():
    """Caches of their own, streams of their own, batches of every launch form at once."""
    cases = [Case(*x[:5], 128, torch.bfloat16, seed=i, room=x[5]) for i, x in enumerate(CASES)]
    want = [c.native() for c in cases]
    torch.cuda.synchronize()
    got, err = [None] * 8, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            c = cases[i % 4] if i < 4 else Case(*CASES[i % 4][:5], 128, torch.bfloat16, seed=i % 4, room=CASES[i % 4][5])
            torch.cuda.current_stream().synchronize()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[i] = c.native() if i < 4 else c.owned(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            err.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not err, err
    for i in range(8):
        assert same(got[i], want[i % 4])
    fa.fa_check_device_status()


def test_both_forms_refuse_the_same_calls():
    """The allocating calls check in the native module, the caller-owned ones in the binding."""
    c = Case(2, 4, 2, 1, 40, 64, torch.bfloat16)
    o, lse = torch.empty_like(c.q), torch.empty(2, 4, 1, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    good = dict(q=c.q, k=c.k, v=c.v, table=c.table, start=c.start, lens=c.lens, slopes=None)

    def forms(**over):
        a = {**good, **over}
        return {"append": (lambda: fa.kv4_append(c.cache, a["k"], a["v"], a["table"], a["start"], a["lens"]),
                           lambda: fa.fa_kv4_append(c.cache, a["k"], a["v"], a["table"], a["start"], a["lens"])),
                "read": (lambda: fa.kv4_read(c.cache, a["table"], a["start"], 40, a["lens"]),
                         lambda: fa.fa_kv4_read(c.cache, a["table"], a["start"], a["lens"], torch.empty_like(c.k), torch.empty_like(c.v))),
                "attend": (lambda: fa.kv4_attend(a["q"], c.cache, a["table"], a["lens"], slopes=a["slopes"], workspace=ws),
                           lambda: fa.fa_kv4_attend(a["q"], c.cache, a["table"], a["lens"], o, lse, ws, 0.1, slopes=a["slopes"]))}

    for pair in forms().values():
        for call in pair:
            call()
    bad = {"append": [dict(k=c.k.half()), dict(v=c.v[:, :, :39]), dict(k=c.k[0]), dict(k=c.k.cpu()), dict(v=c.v.transpose(1, 2)),
                      dict(start=None), dict(start=c.start.long()), dict(lens=c.lens[:1]), dict(table=c.table[:1]), dict(table=c.table.float()),
                      dict(table=c.table[0]), dict(table=c.table.t().contiguous().t())],
           "read": [dict(start=None), dict(lens=None), dict(start=c.start.cpu()), dict(lens=c.lens.long()), dict(table=c.table[:1])],
           "attend": [dict(q=c.q.half()), dict(q=c.q[:, :3].contiguous()), dict(q=c.q[0]), dict(q=c.q.cpu()), dict(lens=None), dict(lens=c.lens[:1]),
                      dict(slopes=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(4)), dict(table=c.table.long())]}
    for name, overs in bad.items():
        for over in overs:
            for form in forms(**over)[name]:
                with pytest.raises((ValueError, TypeError)):
                    form()
    q, k, v, do = rules.problem(1, "bf16", 1, 4, 2, 40, 40, 64)
    ids = torch.zeros(1, 40, dtype=torch.int32, device="cuda")
    o, lse = fa.forward_rule(q, k, v, fa.ScoreRule())
    grads = [torch.empty_like(x) for x in (q, k, v)]
    for x in ((q.half(), k, v), (q, k.half(), v), (q, k, v[:, :, :39]), (q[0], k, v), (q, k[:, :1, :, :32], v[:, :1, :, :32]),
              (q[:, :3].contiguous(), k, v), (q.transpose(2, 3), k, v), (q, k.cpu(), v), (q.float(), k, v)):
        for form in (lambda: fa.forward_rule(*x, fa.ScoreRule()), lambda: fa.fa_fwd_rule(*x, o, lse, fa.ScoreRule(), None, 0.1),
                     lambda: fa.backward_rule(*x, o, lse, do, fa.ScoreRule()),
                     lambda: fa.fa_bwd_rule(*x, o, do, lse, *grads, fa.ScoreRule(), ws, 0.1)):
            with pytest.raises((ValueError, TypeError)):
                form()
    for r in (fa.ScoreRule(q_doc=ids), fa.ScoreRule(k_doc=ids), fa.ScoreRule(q_doc=ids, k_doc=ids[:, :39]),
              fa.ScoreRule(q_doc=ids.long(), k_doc=ids.long()), fa.ScoreRule(prefix=ids[0]), fa.ScoreRule(slopes=torch.zeros(4).cuda().half())):
        for form in (lambda: fa.forward_rule(q, k, v, r), lambda: fa.fa_fwd_rule(q, k, v, o, lse, r, ws, 0.1),
                     lambda: fa.backward_rule(q, k, v, o, lse, do, r), lambda: fa.fa_bwd_rule(q, k, v, o, do, lse, *grads, r, ws, 0.1)):
            with pytest.raises((ValueError, TypeError)):
                form()
    fa.fa_check_device_status()


@pytest.mark.parametrize("d,kinds", [(64, ["fwd", "bwd_kv", "bwd_q"]), (256, ["fwd", "bwd_fused"])])
@pytest.mark.parametrize("docs", [False, True])
def test_the_measurement_hook_records_rule_calls_too(d, kinds, docs):
    q, k, v, do = rules.problem(1, "bf16", 1, 4, 2, 300, 300, d)
    ids = rules.packed_ids([[120, 180]]) if docs else None
    rule = fa.ScoreRule(causal=True, q_doc=ids, k_doc=ids)
    want = fa.forward_rule(q, k, v, rule)
    want = (*want, *fa.backward_rule(q, k, v, *want, do, rule))
    fa.fa_profile_begin(8)
    got = fa.forward_rule(q, k, v, rule)
    got = (*got, *fa.backward_rule(q, k, v, *got, do, rule))
    recorded = fa.fa_profile_end()
    assert [n for n, _ in recorded] == kinds and all(0 < ms < 1000 for _, ms in recorded)
    assert same(got, want)


def test_inputs_that_the_caller_drops_while_another_stream_works():
    """Temporaries handed to a call on a stream that is busy: nothing else gets their memory
    before the call has read them."""
    c = Case(2, 4, 2, 1, 700, 128, torch.bfloat16)
    x = rules.problem(1, "bf16", 1, 4, 2, 512, 512, 128)
    ids = rules.packed_ids([[200, 312]])
    rule = lambda: fa.ScoreRule(causal=True, slopes=rules.slopes(4), q_doc=ids.clone(), k_doc=ids.clone())  # noqa: E731

    def calls(stream, wait):
        def done(r):
            if wait:
                torch.cuda.synchronize()
            return r

        out = [done(fa.kv4_attend(c.q * 2, c.cache, c.table.clone(), c.lens - 1, slopes=rules.slopes(4), stream=stream))]
        out.append(done(fa.forward_rule(x[0] * 2, x[1] * 1, x[2] * 1, rule(), stream=stream)))
        o, lse = (t.clone() for t in ref)
        out.append(done(fa.backward_rule(x[0] * 2, x[1] * 1, x[2] * 1, o, lse, x[3] * 1, rule(), stream=stream)))
        del o, lse
        out.append(done(fa.kv4_read(c.cache, c.table.clone(), c.start + 3, 50, c.lens - 1, stream=stream)))
        return out

    c.native()
    ref = fa.forward_rule(x[0] * 2, x[1], x[2], rule())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    want = calls(s, True)
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = calls(s, False)  # (the temporaries are made by the other stream at once, and done long before)
        for like in (c.q, c.table, c.lens, x[0], x[1], x[2], ids, ref[1]):  # whatever was dropped would be handed out here
            for _ in range(6):
                torch.empty_like(like).fill_(1)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    fa.fa_check_device_status()


def test_the_stream_argument_inside_a_capture():
    c = Case(2, 4, 2, 1, 700, 128, torch.bfloat16)
    x = rules.problem(2, "bf16", 1, 4, 2, 300, 300, 64)
    rule = fa.ScoreRule(causal=True, cap=9.0)
    other = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        q = c.q * 2
        other.wait_stream(main)
        a = fa.kv4_attend(q, c.cache, c.table, c.lens, stream=other)
        del q
        o, lse = fa.forward_rule(*x[:3], rule)  # on the capturing stream, beside it
        main.wait_stream(other)
        return (*a, o, lse)

    c.native()
    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    fa.fa_check_device_status()
