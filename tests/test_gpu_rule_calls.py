"""How the rule and cache calls may be made: captured and replayed, on other streams and
from several threads, through the caller-owned forms, in the checked build, on empty and
on very large problems; and what they refuse."""
import ctypes
import threading

import pytest
import torch

import exact_attention_37_gb300 as fa
from exact_attention_37_gb300 import _lib
from oracle import rules as oracle

from . import rules

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def packed_rule(B, H, N, cap=20.0, pad=9, bias=True, prefix=True):
    ids = rules.packed_ids([[N // 3, 1, N - N // 3 - 1 - pad]] * B, pad)
    return fa.ScoreRule(causal=True, cap=cap, slopes=rules.slopes(H) if bias else None, q_doc=ids, k_doc=ids,
                        prefix=torch.full((B,), 40, dtype=torch.int32, device="cuda") if prefix else None)


def step(q, k, v, do, rule):
    o, lse = fa.forward_rule(q, k, v, rule)
    return (o, lse, *fa.backward_rule(q, k, v, o, lse, do, rule))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def cache_problem(seed=0, B=3, H=8, Hkv=2, Nq=2, page=32, d=128, n=900, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    per = -(-n // page)
    cache = fa.KV4Cache.empty(B * per, Hkv, page, d, dtype)
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    k, v = (torch.randn(B, Hkv, n, d, generator=g).to(dtype).cuda() for _ in range(2))
    q = torch.randn(B, H, Nq, d, generator=g).to(dtype).cuda()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.kv4_append(cache, k, v, table, zero)
    return cache, table, q, k, v


@pytest.mark.parametrize("d", [64, 128, 256])
def test_repeated_calls_are_bitwise_equal(d):
    x = rules.problem(d, "bf16", 2, 8, 2, 700, 700, d, gain=2.0)
    rule = packed_rule(2, 8, 700)
    a = step(*x, rule)
    for _ in range(3):
        assert same(a, step(*x, rule))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("docs", [True, False])
def test_captured_steps_replay_on_new_inputs(d, docs):
    B, H, N = 2, 4, 400
    x = rules.problem(d, "fp16", B, H, 2, N, N, d)
    rule = packed_rule(B, H, N) if docs else fa.ScoreRule(causal=True, cap=30.0, slopes=rules.slopes(H))
    step(*x, rule)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*x, rule)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*x, rule)
    for seed in (1, 2):
        y = rules.problem(100 * seed + d, "fp16", B, H, 2, N, N, d)
        for dst, src in zip(x, y):
            dst.copy_(src)
        if docs:  # other documents in the captured arrays too
            ids = rules.packed_ids([[N - 50 * seed, 50 * seed - 5]] * B, 5)
            rule.q_doc.copy_(ids)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, step(*y, rule))
    fa.fa_check_device_status()


def test_captured_decoding_follows_lengths_on_the_device():
    cache, table, q, k, v = cache_problem()
    B = q.shape[0]
    lengths = torch.tensor([500, 3, 0], dtype=torch.int32, device="cuda")
    one = lambda x, at: torch.stack([x[b, :, at[b]:at[b] + 1] for b in range(B)]).contiguous()  # noqa: E731
    kn, vn = one(k, [0, 1, 2]), one(v, [0, 1, 2])

    def decode():
        fa.kv4_append(cache, kn, vn, table, lengths)
        return fa.kv4_attend(q, cache, table, lengths + 1, cap=5.0)

    decode()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = decode()
    for lens in ([500, 3, 0], [899, 0, 128], [1, 31, 640]):
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        assert same(got, decode())
    fa.fa_check_device_status()


def test_other_streams():
    """The stream argument: work and memory belong to that stream."""
    x = rules.problem(1, "bf16", 2, 8, 8, 900, 900, 128)
    rule = packed_rule(2, 8, 900)
    ref = step(*x, rule)
    cache, table, q, _, _ = cache_problem()
    lens = torch.tensor([900, 17, 400], dtype=torch.int32, device="cuda")
    ref4 = fa.kv4_attend(q, cache, table, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:  # no waiting between them: two calls at once
        o, lse = fa.forward_rule(*x[:3], rule, stream=s)
        got.append(((o, lse, *fa.backward_rule(*x[:3], o, lse, x[3], rule, stream=s)),
                    fa.kv4_attend(q, cache, table, lens, stream=s), fa.kv4_read(cache, table, lens * 0, 30, lens, stream=s)))
    torch.cuda.synchronize()
    for a, b, c in got:
        assert same(a, ref) and same(b, ref4) and same(c, fa.kv4_read(cache, table, lens * 0, 30, lens))


def test_calls_from_several_threads():
    xs = [rules.problem(n, "bf16", 1, 4, 2, 600, 600, 64) for n in range(4)]
    rule = packed_rule(1, 4, 600)
    ref = [step(*x, rule) for x in xs]
    torch.cuda.synchronize()
    out, err = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    out[i] = step(*xs[i], rule)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            err.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not err
    for a, b in zip(out, ref):
        assert same(a, b)


@pytest.mark.parametrize("heads,tokens", [(1, 4200), (4, 20000)])  # 32- and 64-token tiles
def test_caches_of_different_batches_from_several_threads(heads, tokens):
    """One kernel instance of the two-launch form, batches whose shared memory differs: the C
    call runs without the interpreter's lock, so the calls overlap.  Most calls find their
    lengths 0 and are short; the last of each thread does its work."""
    lib, d, results, codes = fa.load(), 128, [], []
    calls, want = [], []
    for B in (1, 7 if heads == 1 else 300):
        cache, table, q, _, _ = cache_problem(B=1, H=heads, Hkv=heads, Nq=1, n=tokens, page=1024, d=d)
        table, q = table.expand(B, -1).contiguous(), q.expand(B, -1, -1, -1).contiguous()
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        lens[:5] = torch.tensor([tokens - 3 * b for b in range(min(B, 5))], dtype=torch.int32)
        calls.append((cache, table, q, lens))
        want.append(fa.kv4_attend(q, cache, table, lens))
    torch.cuda.synchronize()

    def work(i):
        cache, table, q, lens = calls[i % 2]
        B, H, N, _ = q.shape
        ws = torch.empty(fa.fa_kv4_attend_workspace_size(B, H, cache.H_kv, N, d), dtype=torch.uint8, device="cuda")
        o, lse, none, s = torch.empty_like(q), torch.empty(B, H, N, device="cuda"), torch.zeros_like(lens), torch.cuda.Stream()
        torch.cuda.current_stream().synchronize()
        c = cache.struct()
        args = lambda n: (q.data_ptr(), ctypes.addressof(c), table.data_ptr(), table.shape[1], n.data_ptr(), o.data_ptr(),  # noqa: E731
                          lse.data_ptr(), 1, 0.0, None, ws.data_ptr(), ws.numel(), B, H, N, d ** -0.5, s.cuda_stream)
        short, last = args(none), args(lens)
        codes.extend(lib.fa_kv4_attend(*short) for _ in range(600))
        codes.append(lib.fa_kv4_attend(*last))
        s.synchronize()
        results.append((i % 2, (o, lse)))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert len(results) == 6 and not any(codes), sum(c != 0 for c in codes)
    for i, got in results:
        assert same(got, want[i])
    fa.fa_check_device_status()


def test_caller_owned_forms_are_the_same_calls():
    q, k, v, do = rules.problem(2, "fp16", 2, 6, 3, 333, 333, 128)
    rule = packed_rule(2, 6, 333)
    ref = step(q, k, v, do, rule)
    B, H, N, d = q.shape
    sizes = (B, H, N, k.shape[2], d, True)
    ws = torch.empty(fa.fa_fwd_rule_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    wb = torch.empty(fa.fa_bwd_rule_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa.fa_fwd_rule(q, k, v, o, lse, rule, ws, d ** -0.5)
    fa.fa_bwd_rule(q, k, v, o, do, lse, dq, dk, dv, rule, wb, d ** -0.5)
    assert same(ref, (o, lse, dq, dk, dv))
    assert same(ref[2:], fa.backward_rule(q, k, v, o, lse, do, rule, workspace=wb))
    cache, table, q, k, v = cache_problem()
    lens = torch.tensor([900, 17, 400], dtype=torch.int32, device="cuda")
    start = torch.tensor([3, 0, 7], dtype=torch.int32, device="cuda")
    fa.fa_kv4_append(cache, k, v, table, start * 0)
    ok, ov = torch.empty_like(k[:, :, :50]).contiguous(), torch.empty_like(k[:, :, :50]).contiguous()
    fa.fa_kv4_read(cache, table, start, lens, ok, ov)
    assert same((ok, ov), fa.kv4_read(cache, table, start, 50, lens))
    B, H, N, d = q.shape
    w4 = torch.empty(fa.fa_kv4_attend_workspace_size(B, H, cache.H_kv, N, d), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    fa.fa_kv4_attend(q, cache, table, lens, o, lse, w4, d ** -0.5, True, 3.0)
    assert same((o, lse), fa.kv4_attend(q, cache, table, lens, cap=3.0))
    assert same((o, lse), fa.kv4_attend(q, cache, table, lens, cap=3.0, workspace=w4))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_tensors_at_sixteen_byte_addresses(d):
    """16-byte alignment is what the calls ask for: tensors that begin 16 bytes into a buffer."""
    x = rules.problem(d, "bf16", 1, 4, 2, 300, 300, d)
    rule = packed_rule(1, 4, 300)
    ref = step(*x, rule)

    def off(t):
        buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = buf[8:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    q, k, v, do = (off(t) for t in x)
    o, lse = fa.forward_rule(q, k, v, rule)
    assert same(ref, (o, lse, *fa.backward_rule(q, k, v, off(o), lse, do, rule)))
    cache, table, q, k, v = cache_problem(d=d)
    lens = torch.tensor([900, 17, 400], dtype=torch.int32, device="cuda")
    a = fa.kv4_attend(q, cache, table, lens)
    fa.kv4_append(cache, off(k), off(v), table, lens * 0)
    assert same(a, fa.kv4_attend(off(q), cache, table, lens))


def test_two_sequences_may_read_the_same_pages():
    cache, table, q, _, _ = cache_problem(B=2, n=300)
    shared = table[:1].expand(2, -1).contiguous()
    lens = torch.tensor([300, 170], dtype=torch.int32, device="cuda")
    o, lse = fa.kv4_attend(q, cache, shared, lens)
    for b in range(2):
        a = fa.kv4_attend(q[b:b + 1].contiguous(), cache, table[:1].contiguous(), lens[b:b + 1].contiguous())
        # alone and in a batch the work is cut differently: the sums' order differs
        assert float((o[b] - a[0][0]).abs().max()) <= 2.0 ** -7 * float(o[b].abs().max())
        assert float((lse[b] - a[1][0]).abs().max()) <= 3e-5 * max(1.0, float(lse[b].abs().max()))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_empty_problems(d):
    rule = fa.ScoreRule(causal=True, cap=5.0)
    t = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    o, lse = fa.forward_rule(t(2, 4, 0, d), t(2, 2, 30, d), t(2, 2, 30, d), rule)
    assert o.numel() == 0 and lse.numel() == 0
    dq, dk, dv = fa.backward_rule(t(2, 4, 0, d), t(2, 2, 30, d), t(2, 2, 30, d), o, lse, o, rule)
    assert dq.numel() == 0 and bool((dk == 0).all()) and bool((dv == 0).all())
    assert fa.forward_rule(t(0, 4, 8, d), t(0, 2, 8, d), t(0, 2, 8, d), rule)[0].numel() == 0
    with pytest.raises(fa.FaError) as e:  # queries without a key set
        fa.forward_rule(t(1, 4, 8, d), t(1, 2, 0, d), t(1, 2, 0, d), rule)
    assert e.value.code == 2
    cache = fa.KV4Cache.empty(0, 2, 16, d, torch.bfloat16)
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    o, lse = fa.kv4_attend(t(2, 4, 1, d), cache, none, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
    fa.fa_check_device_status()


def test_wrong_arguments_are_refused():
    q, k, v, do = rules.problem(1, "bf16", 1, 4, 2, 40, 40, 64)
    rule = fa.ScoreRule(causal=True)
    ids = torch.zeros(1, 40, dtype=torch.int32, device="cuda")
    bad_rules = [fa.ScoreRule(q_doc=ids), fa.ScoreRule(q_doc=ids.long(), k_doc=ids), fa.ScoreRule(q_doc=ids.cpu(), k_doc=ids),
                 fa.ScoreRule(q_doc=ids[:, :39], k_doc=ids), fa.ScoreRule(slopes=torch.zeros(3, device="cuda")),
                 fa.ScoreRule(slopes=torch.zeros(8, device="cuda")[::2]), fa.ScoreRule(prefix=ids[0])]
    o, lse = fa.forward_rule(q, k, v, rule)
    for r in bad_rules:
        with pytest.raises(ValueError):
            fa.forward_rule(q, k, v, r)
        with pytest.raises(ValueError):
            fa.backward_rule(q, k, v, o, lse, do, r)
        with pytest.raises(ValueError):
            fa.fa_fwd_rule(q, k, v, o, lse, r, None, 0.1)
    for cap in (-1.0, float("nan")):
        with pytest.raises(fa.FaError):
            fa.forward_rule(q, k, v, fa.ScoreRule(cap=cap))
    for bad in ((q.cpu(), k, v), (q.float(), k, v), (q, k.half(), v), (q, k, v[:, :, :39]), (q.transpose(1, 2), k, v), (q[0], k, v),
                (q, k[:, :, :, :32], v[:, :, :, :32]), (q[:, :3].contiguous(), k, v)):
        with pytest.raises((ValueError, TypeError)):
            fa.forward_rule(*bad, rule)
    for bad in ((o.float(), lse, do), (o, lse.half(), do), (o, lse, do[:, :, :39]), (o, lse.cpu(), do)):
        with pytest.raises((ValueError, TypeError)):
            fa.backward_rule(q, k, v, *bad, rule)
    with pytest.raises(fa.FaError) as e:
        fa.backward_rule(q, k, v, o, lse, do, rule, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4
    cache, table, q4, k4, v4 = cache_problem()
    lens = torch.tensor([900, 17, 400], dtype=torch.int32, device="cuda")
    for call in (lambda: fa.kv4_attend(q4, cache, table.long(), lens), lambda: fa.kv4_attend(q4, cache, table, lens.cpu()),
                 lambda: fa.kv4_attend(q4, cache, table[:2], lens), lambda: fa.kv4_attend(q4.half(), cache, table, lens),
                 lambda: fa.kv4_attend(q4[:, :3].contiguous(), cache, table, lens), lambda: fa.kv4_attend(q4, cache, table, None),
                 lambda: fa.kv4_append(cache, k4.half(), v4, table, lens), lambda: fa.kv4_append(cache, k4, v4, table, None),
                 lambda: fa.kv4_append(cache, k4, v4[:, :, :5], table, lens), lambda: fa.kv4_read(cache, table, lens, -1, lens),
                 lambda: fa.KV4Cache(cache.k_codes, cache.v_codes, cache.k_params, cache.v_params),
                 lambda: fa.KV4Cache(cache.k_codes[:, :, :, ::2], cache.k_params, cache.v_codes, cache.v_params)):
        with pytest.raises((ValueError, TypeError)):
            call()
    fa.fa_check_device_status()


# ------------------------------------------------------------------ the checked build


@pytest.fixture(scope="module")
def dlib():
    from exact_attention_37_gb300 import build

    return _lib.open_library(build.build(debug=True))


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("heads", [4, 160])
@pytest.mark.parametrize("kind", ["mask", "capbias", "packed", "mixed", "none"])
def test_checked_build_runs_clean(dlib, d, dtype, heads, kind):
    """Every device-side check (copies' boxes, tensor-memory columns, each barrier's phases)
    silent, and the results those of the release build."""
    B, H, Hkv, N = 1, heads, heads // 2, 300
    q, k, v, do = rules.problem(d, dtype, B, H, Hkv, N, N, d)
    ids = {"packed": rules.packed_ids([[100, 3, 150]], 47), "none": torch.full((1, N), -1, dtype=torch.int32, device="cuda"),
           "mixed": torch.randint(-1, 3, (1, N), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()}.get(kind)
    capped = kind in ("capbias", "packed")
    rule = fa.ScoreRule(causal=kind != "mixed", cap=9.0 if capped else 0.0, slopes=rules.slopes(H) if capped else None,
                        q_doc=ids, k_doc=ids)
    ref = step(q, k, v, do, rule)
    r = rule.struct(0, B, H, N, N)
    docs = int(ids is not None)
    ws = torch.empty(max(256, dlib.fa_bwd_rule_workspace_size(B, H, N, N, d, docs)), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    scale = d ** -0.5
    code = 1 if dtype == "bf16" else 0
    p = [t.data_ptr() for t in (q, k, v, o, lse, do, dq, dk, dv)]
    assert dlib.fa_fwd_rule(p[0], p[1], p[2], p[3], p[4], ctypes.addressof(r), ws.data_ptr(), ws.numel(), B, H, Hkv, N, N, d,
                            scale, code, st) == 0
    assert dlib.fa_bwd_rule(p[0], p[1], p[2], p[3], p[5], p[4], p[6], p[7], p[8], ctypes.addressof(r), ws.data_ptr(),
                            ws.numel(), B, H, Hkv, N, N, d, scale, code, st) == 0
    got = dlib.fa_check_device_status(st)
    rec = (ctypes.c_uint32 * 4)()
    dlib.fa_last_device_error_detail(rec)
    assert got == 0, [int(x) for x in rec]
    assert same(ref, (o, lse, dq, dk, dv))


# ------------------------------------------------------------------ sizes past 32 bits


def test_tensors_past_two_to_the_31_elements():
    """Heads on both sides of element 2^31, with documents and a cap, forward and backward:
    the same as those heads alone, and as the definition."""
    B, H, N, d = 3, 44, 256 * 127, 64  # 2.75e9 elements, 44 * 127 * 256 rows a batch entry
    g = torch.Generator(device="cuda").manual_seed(0)
    q, do = (torch.randn(B, H, N, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(B, H, N, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ids = (torch.arange(N, device="cuda") // 333).to(torch.int32).expand(B, N).contiguous()
    rule = fa.ScoreRule(causal=True, cap=15.0, q_doc=ids, k_doc=ids)
    out = step(q, k, v, do, rule)
    fa.fa_check_device_status()
    for b, h in ((0, 0), (2, 14), (2, 15), (2, 43)):  # element 2^31 lies in head (2, 15)
        one = [x[b:b + 1, h:h + 1].contiguous() for x in (q, k, v, do)]
        r1 = fa.ScoreRule(causal=True, cap=15.0, q_doc=ids[:1].contiguous(), k_doc=ids[:1].contiguous())
        alone = step(*one, r1)
        for x, y, n in zip(out, alone, ("O", "L", "dQ", "dK", "dV")):
            # one head takes other blocks of rows a CTA, so O's sums may differ in order
            x, y = x[b, h].float(), y[0, 0].float()
            assert float((x - y).abs().max()) <= 2.0 ** -7 * max(1.0, float(y.abs().max())), n
        last = slice(N - 700, N)
        ro, rl, a, s = oracle.forward(*[x[:, :, last] for x in one[:3]], rules.f32(d ** -0.5), causal=True, cap=15.0,
                                      q_doc=ids[:1, last], k_doc=ids[:1, last])
        tail = slice(400, 700)  # rows whose document begins inside the slice
        u = rules.U[torch.bfloat16]
        rules.within(out[0][b:b + 1, h:h + 1, last][:, :, tail], ro[:, :, tail],
                     (u * (a + ro.abs()) + rules.E * a + rules.S[torch.bfloat16] * (s + 1))[:, :, tail], "O")
        rules.check_l(out[1][b:b + 1, h:h + 1, last][:, :, tail], rl[:, :, tail])


def test_a_pool_past_four_gigabytes():
    """Pages whose bytes lie behind 2^32: stored, read back and attended over."""
    d, Hkv, page = 256, 8, 1024
    pages = 4500  # 1 MB of codes a page for keys and for values each
    cache = fa.KV4Cache.empty(pages, Hkv, page, d, torch.float16)
    table = torch.tensor([[pages - 1, 0], [4100, pages - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(0)
    n = 1500
    k, v = (torch.randn(2, Hkv, n, d, generator=g).half().cuda() for _ in range(2))
    zero, lens = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([n, n], dtype=torch.int32, device="cuda")
    fa.kv4_append(cache, k, v, table, zero)
    small = fa.KV4Cache.empty(4, Hkv, page, d, torch.float16)
    t2 = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    fa.kv4_append(small, k, v, t2, zero)
    assert same(fa.kv4_read(cache, table, zero, n, lens), fa.kv4_read(small, t2, zero, n, lens))
    q = torch.randn(2, 16, 2, d, generator=g).half().cuda()
    assert same(fa.kv4_attend(q, cache, table, lens), fa.kv4_attend(q, small, t2, lens))
    fa.fa_check_device_status()


@pytest.mark.parametrize("N", [150, 1100])
def test_calls_that_overlap_give_what_calls_one_by_one_give(N):
    """A call may start while the one ahead of it in the stream ends: each takes what the one
    before has just written, through the same buffers."""
    B, H, Hkv, d, t = 1, 4, 2, 64, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda h: torch.randn(B, h, N, d, generator=g, device="cuda").to(t)  # noqa: E731
    q0, k0, v0, do = r(H), r(Hkv), r(Hkv), r(H)
    ids = (torch.arange(N, device="cuda", dtype=torch.int32) // 70)[None].contiguous()
    pages = -(-N // 16)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    start, lengths = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (0, N))
    kinds = [fa.ScoreRule(causal=True, cap=5.0), fa.ScoreRule(causal=True, q_doc=ids, k_doc=ids), fa.ScoreRule(slopes=rules.slopes(H))]

    def chain(wait):
        def done(x):
            if wait:
                torch.cuda.synchronize()
            return x

        q, k, v = q0.clone(), k0.clone(), v0.clone()
        cache = fa.KV4Cache.empty(pages, Hkv, 16, d, t)
        o, lse = torch.empty_like(q), torch.empty((B, H, N), device="cuda")
        ws = torch.empty(fa.fa_fwd_rule_workspace_size(B, H, N, N, d, True), dtype=torch.uint8, device="cuda")
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        out = []
        for i in range(12):
            rule = kinds[i % 3]
            done(fa.fa_fwd_rule(q, k, v, o, lse, rule, ws, 0.125))
            dq, dk, dv = done(fa.backward_rule(q, k, v, o, lse, do, rule, scale=0.125))
            done(fa.fa_kv4_append(cache, dk, dv, table, start))
            done(fa.fa_kv4_read(cache, table, start, lengths, kr, vr))
            qa, la = done(fa.kv4_attend(o[:, :, -3:].contiguous(), cache, table, lengths, scale=0.125))
            done(fa.fa_fwd_rule(dq, kr, vr, q, lse, kinds[(i + 1) % 3], ws, 0.125))
            k, v = kr, vr
            kr, vr = torch.empty_like(k), torch.empty_like(v)
            out += [dq, qa, la, lse.clone()]
        torch.cuda.synchronize()
        fa.fa_check_device_status()
        return out

    want = chain(True)
    for _ in range(3):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


def test_captured_calls_behind_copies_fills_and_other_streams():
    """What is ahead of a call in a graph need not be a kernel, nor be one thing."""
    B, H, N, d, t = 1, 2, 200, 64, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    host = [torch.randn(B, H, N, d, generator=g).to(t).pin_memory() for _ in range(3)]
    q, k, v = (torch.zeros(B, H, N, d, dtype=t, device="cuda") for _ in range(3))
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    start, lengths = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (0, N))
    cache = fa.KV4Cache.empty(4, H, 64, d, t)
    rule = fa.ScoreRule(causal=True, cap=9.0)
    other = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        for x, h in zip((q, k, v), host):
            x.copy_(h, non_blocking=True)
        o, lse = fa.forward_rule(q, k, v, rule)              # behind a copy
        other.wait_stream(main)
        with torch.cuda.stream(other):
            for x in cache.pools:
                x.zero_()
            fa.kv4_append(cache, k, v, table, start)         # behind a fill, on a stream that was forked
        grads = fa.backward_rule(q, k, v, o, lse, q, rule)
        main.wait_stream(other)
        a, la = fa.kv4_attend(q[:, :, -2:].contiguous(), cache, table, lengths, cap=9.0)  # behind both streams
        kr, vr = fa.kv4_read(cache, table, start, N, lengths)
        return [o, lse, *grads, a, la, kr, vr]

    want = [x.clone() for x in work()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        for x in (q, k, v, *cache.pools):
            x.zero_()
        for x in got:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        fa.fa_check_device_status()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_gradients_of_calls_in_a_row_through_the_same_buffers(d):
    """Every kernel of a backward pass starts while the one ahead ends.  L, D, the ids and the
    block lists lie where another problem's lay a call before, O, L and the ids' source too:
    each call takes its own."""
    B, H, Hkv, N, scale = 1, 8, 2, 900, d ** -0.5
    xs = [rules.problem(40 + i, "bf16", B, H, Hkv, N, N, d) for i in range(3)]
    docs = [rules.packed_ids([x], 30) for x in ([400, 470], [7] * 100 + [170], [870])]
    docs[1] = docs[1].flip(1).contiguous()  # ids in no order
    ids, o, lse = torch.empty_like(docs[0]), torch.empty_like(xs[0][0]), torch.empty(B, H, N, device="cuda")
    rule = fa.ScoreRule(causal=True, cap=10.0, q_doc=ids, k_doc=ids)
    ws = torch.empty(max(f(B, H, N, N, d, True) for f in (fa.fa_fwd_rule_workspace_size, fa.fa_bwd_rule_workspace_size)),
                     dtype=torch.uint8, device="cuda")

    def run(wait):
        out = []
        for i in (0, 1, 2, 1, 0, 2) * 3:
            q, k, v, do = xs[i]
            ids.copy_(docs[i])
            fa.fa_fwd_rule(q, k, v, o, lse, rule, ws, scale)
            grads = [torch.empty_like(x) for x in (q, k, v)]
            fa.fa_bwd_rule(q, k, v, o, do, lse, *grads, rule, ws, scale)
            if wait:
                torch.cuda.synchronize()
            out += [o.clone(), lse.clone(), *grads]
        torch.cuda.synchronize()
        fa.fa_check_device_status()
        return out

    want = run(True)
    for _ in range(3):
        assert same(run(False), want)


# caches that take stretches and a join, not a cluster: a grid that lets its neighbours in the
# stream overlap, with 32-token tiles, and a full one with 64-token tiles
@pytest.mark.parametrize("H,Hkv,n", [(4, 1, 8000), (16, 4, 16000)])
def test_captured_decoding_over_stretches_follows_lengths_on_the_device(H, Hkv, n):
    cache, table, q, k, v = cache_problem(B=2, H=H, Hkv=Hkv, Nq=1, n=n, page=64)
    lengths = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
    kn, vn = (torch.randn(2, Hkv, 1, 128, generator=torch.Generator().manual_seed(i)).to(k.dtype).cuda() for i in (1, 2))

    def decode():  # two steps: a join ahead of an append, and parts where the step before left its own
        a = fa.kv4_attend(q, cache, table, lengths, cap=5.0)
        fa.kv4_append(cache, kn, vn, table, lengths)
        return *a, *fa.kv4_attend(q, cache, table, lengths + 1, cap=5.0)

    decode()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = decode()
    for lens in ([n - 1, 0], [0, 77], [n // 2, n - 1], [3, 2], [0, 0], [517, 6000]):
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        for x in out:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        assert same(got, decode())
        for b in range(2):  # each sequence alone: other stretches, so other orders of the sums
            a = fa.kv4_attend(q[b:b + 1].contiguous(), cache, table[b:b + 1].contiguous(), lengths[b:b + 1] + 1, cap=5.0)
            assert float((got[2][b] - a[0][0]).abs().max()) <= 2.0 ** -7 * float(a[0].abs().max())
            assert float((got[3][b] - a[1][0]).abs().max()) <= 3e-5 * max(1.0, float(a[1].abs().max()))
    fa.fa_check_device_status()


@pytest.mark.parametrize("H,Hkv,n", [(4, 1, 8000), (16, 4, 16000)])
def test_cache_calls_that_overlap_over_stretches(H, Hkv, n):
    """Lengths, queries, pages and the workspace change from call to call, without waits and with."""
    d = 128
    cache, table, q0, k, v = cache_problem(B=2, H=H, Hkv=Hkv, Nq=1, n=n, page=64)
    rows = [[n, 17], [0, n - 5], [4000, 4000], [1, 0], [n - 1, n]]
    lens = torch.tensor(rows, dtype=torch.int32, device="cuda")
    start = torch.tensor([[max(0, x - 3) for x in r] for r in rows], dtype=torch.int32, device="cuda")
    pools = [x.clone() for x in cache.pools]
    now, at = torch.empty_like(lens[0]), torch.empty_like(lens[0])
    ws = torch.empty(fa.fa_kv4_attend_workspace_size(2, H, Hkv, 1, d), dtype=torch.uint8, device="cuda")

    def chain(wait):
        for x, y in zip(cache.pools, pools):
            x.copy_(y)
        out, q = [], q0.clone()
        for i in range(20):
            now.copy_(lens[i % 5])
            at.copy_(start[i % 5])
            o, lse = fa.kv4_attend(q, cache, table, now, workspace=ws)
            new = o[:, :Hkv].contiguous()
            fa.kv4_append(cache, new, new, table, at)
            o2, lse2 = fa.kv4_attend(q, cache, table, now, cap=3.0, workspace=ws)
            q = (q0 + o2).contiguous()
            if wait:
                torch.cuda.synchronize()
            out += [o, lse, o2, lse2]
        torch.cuda.synchronize()
        fa.fa_check_device_status()
        return out

    want = chain(True)
    for _ in range(3):
        assert same(chain(False), want)


@pytest.mark.parametrize("Nk", [0, 30])
def test_document_ids_of_empty_problems(Nk):
    t = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    ids = lambda n: torch.zeros(2, n, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = t(2, 4, 0, 64), t(2, 2, Nk, 64), t(2, 2, Nk, 64)
    rule = fa.ScoreRule(causal=True, q_doc=ids(0), k_doc=ids(Nk), prefix=ids(1)[:, 0].contiguous())
    o, lse = fa.forward_rule(q, k, v, rule)
    assert o.shape == q.shape and lse.shape == (2, 4, 0)
    fa.fa_fwd_rule(q, k, v, o, lse, rule, None, 0.1)
    dq, dk, dv = fa.backward_rule(q, k, v, o, lse, o, rule)
    assert dq.numel() == 0 and bool((dk == 0).all()) and bool((dv == 0).all())
    dk.fill_(1), dv.fill_(1)
    fa.fa_bwd_rule(q, k, v, o, o, lse, dq, dk, dv, rule, None, 0.1)
    assert bool((dk == 0).all()) and bool((dv == 0).all())
