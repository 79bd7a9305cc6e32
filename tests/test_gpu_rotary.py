"""Rotary positions on the GPU against their definition.

Bound of an element (u = finfo.eps / 2, s half of fp16's smallest step): u |y| + s for the one rounding,
and (2^-20 + 2^-22) amplitude (|x1| + |x2|) for cosine and sine (the fast ones are within 2^-21.1 on half a
turn either way; their argument, rounded twice in fp32, within 2 pi 2^-24 = 2^-21.3; together under 2^-20)
and the three fp32 roundings of a product and the sum."""
import numpy as np
import pytest
import torch

import exact_attention_37_gb300 as fa
from oracle import drafts

from .drafts import bounds, i32

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from exact_attention_37_gb300 import build

    build.build()
    fa.load()


def close(got, x, positions, freqs, t, interleaved=False, amplitude=1.0, backward=False):
    y, size = drafts.rotary(x.double().cpu().numpy(), positions, freqs.cpu().numpy(), interleaved, amplitude, backward)
    u, s = bounds()[t]
    off = np.abs(got.double().cpu().numpy() - y)
    trig = (2.0 ** -20 + 2.0 ** -22) * abs(amplitude) * size
    over = off / ((1 + u) * trig + np.where(size > 0, u * np.abs(y) + s, 0) + 1e-300)
    turned = 2 * freqs.shape[0]
    assert over[..., :turned].max(initial=0) <= 1, f"{over[..., :turned].max():.3g} of the bound"
    assert (off[..., turned:] == 0).all()


def make(B, H, Hkv, N, d, t, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, H, N, d, generator=g).to(t).cuda(), torch.randn(B, Hkv, N, d, generator=g).to(t).cuda()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hkv,N,d,dims", [(1, 1, 1, 1, 64, 64), (3, 5, 1, 7, 64, 16), (2, 4, 2, 33, 128, 128), (1, 7, 7, 65, 128, 48),
                                              (2, 6, 3, 17, 256, 256), (1, 3, 1, 31, 256, 64), (5, 8, 8, 1, 128, 128), (2, 9, 3, 130, 64, 32)])
def test_forward_and_backward(B, H, Hkv, N, d, dims, interleaved, dtype):
    t = TYPES[dtype]
    q, k = make(B, H, Hkv, N, d, t)
    rng = np.random.default_rng(N)
    pos = rng.integers(-1000, 200000, (B, N))
    f = fa.rotary_freqs(dims, base=500000.0)
    for backward in (False, True):
        call = fa.rotary_backward if backward else fa.rotary
        q0, k0 = q.clone(), k.clone()
        a, b = call(q, k, i32(pos), f, interleaved=interleaved, amplitude=1.25)
        assert torch.equal(q, q0) and torch.equal(k, k0) and a.is_contiguous() and b.is_contiguous()
        close(a, q, pos, f, t, interleaved, 1.25, backward)
        close(b, k, pos, f, t, interleaved, 1.25, backward)


def test_far_positions_and_odd_frequencies():
    t = torch.bfloat16
    pos = np.array([[0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7]])
    q, k = make(1, 2, 1, 7, 64, t)
    f = torch.tensor([1.0, 6.283185307179586, -0.5, 1e-9, 0.0, 1e4, 3.0, 1e-30], dtype=torch.float64, device="cuda")
    a, b = fa.rotary(q, k, i32(pos), f)
    close(a, q, pos, f, t)
    close(b, k, pos, f, t)


def test_positions_count_up_by_default_and_keys_may_be_absent():
    q, k = make(2, 4, 2, 40, 128, torch.float16)
    f = fa.rotary_freqs(128)
    pos = np.tile(np.arange(40), (2, 1))
    a, b = fa.rotary(q, k, None, f)
    c, d = fa.rotary(q, k, i32(pos), f)
    assert torch.equal(a, c) and torch.equal(b, d)
    e, none = fa.rotary(q, None, None, f)
    assert none is None and torch.equal(e, a)
    close(a, q, pos, f, torch.float16)


@pytest.mark.parametrize("dims", [128, 32])
def test_joint_projection_in_and_out(dims):
    """Strided rows: parts of a joint projection, its gradient, and the rows themselves."""
    B, N, H, Hkv, d = 2, 37, 6, 2, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, N, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    f, pos = fa.rotary_freqs(dims), i32(np.tile(np.arange(5, 5 + N), (B, 1)))
    want = fa.rotary(q.contiguous(), k.contiguous(), pos, f)
    got = fa.rotary(q, k, pos, f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].is_contiguous()
    room = torch.full_like(x, 3.0)
    out = room[:, :, :H].transpose(1, 2), room[:, :, H:H + Hkv].transpose(1, 2)
    r = fa.rotary(q, k, pos, f, out=out)
    assert r[0].data_ptr() == room.data_ptr() and torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert bool((room[:, :, H + Hkv:] == 3).all())
    v = x[:, :, H + Hkv:].clone()
    fa.rotary(q, k, pos, f, out=(q, k))  # in place
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, H + Hkv:], v)
    # rows that all batch entries share are read with a stride of 0
    one = torch.randn(1, 3, N, d, generator=g).to(torch.bfloat16).cuda()
    many = one.expand(B, -1, -1, -1)
    assert torch.equal(fa.rotary(many, None, pos, f)[0], fa.rotary(many.contiguous(), None, pos, f)[0])


def test_gradient_is_the_formulas_and_that_of_differences():
    """sum(y g) changes by the gradient's product with a change of x: y is linear in x."""
    B, H, N, d = 1, 2, 9, 64
    q, g = make(B, H, H, N, d, torch.float16)
    f, pos = fa.rotary_freqs(32), i32([list(range(100, 100 + N))])
    for inter in (False, True):
        dq, _ = fa.rotary_backward(g, None, pos, f, interleaved=inter)
        y = lambda x: fa.rotary(x, None, pos, f, interleaved=inter)[0].double()  # noqa: E731
        e = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(torch.float16).cuda()
        plus, minus = (q + e), (q - e)
        step = (plus.double() - minus.double())
        lhs = ((y(plus) - y(minus)) * g.double()).sum().item()
        rhs = (step * dq.double()).sum().item()
        # every y is rounded once, and every dq
        room = 2.0 ** -11 * ((y(plus).abs() + y(minus).abs()) * g.double().abs() + step.abs() * dq.double().abs()).sum().item()
        assert abs(lhs - rhs) <= 1.01 * room


def test_empty_sizes_and_refusals():
    f = fa.rotary_freqs(64)
    for shape in ((0, 2, 3, 64), (1, 0, 3, 64), (1, 2, 0, 64)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        a, b = fa.rotary(x, x, None, f)
        assert a.shape == x.shape and b.shape == x.shape
    q, k = make(1, 2, 2, 8, 64, torch.bfloat16)
    pos = i32([list(range(8))])
    bad = [lambda: fa.rotary(q, k.half(), pos, f), lambda: fa.rotary(q, k[:, :, :4], pos, f), lambda: fa.rotary(q, k, pos.long(), f),
           lambda: fa.rotary(q, k, pos[:, :4], f), lambda: fa.rotary(q, k, pos, f.float()), lambda: fa.rotary(q, k, pos, f.cpu()),
           lambda: fa.rotary(q.transpose(2, 3).contiguous().transpose(2, 3), k, pos, f), lambda: fa.rotary(q, k, pos, f, out=(q[:, :1], k)),
           lambda: fa.rotary(q, None, pos, f, out=(q, k)), lambda: fa.rotary(q.float(), k.float(), pos, f), lambda: fa.rotary(q[0], k[0], pos, f)]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    wide = torch.zeros(1, 2, 8, 68, dtype=torch.bfloat16, device="cuda")
    for call, code in ((lambda: fa.rotary(q, k, pos, fa.rotary_freqs(80)), 2), (lambda: fa.rotary(q, k, pos, f[:5]), 2),
                       (lambda: fa.rotary(wide[..., :64], None, pos, f), 3), (lambda: fa.rotary(wide[..., 4:], None, pos, f), 3),
                       (lambda: fa.rotary(q, k, pos, f, amplitude=float("nan")), 1),
                       (lambda: fa.rotary(q, k, pos, f, out=(q[:, :1].expand(-1, 2, -1, -1), k)), 1)):
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.code == code
    fa.fa_check_device_status()


def test_caller_owned_form_streams_and_capture():
    q, k = make(2, 4, 2, 300, 128, torch.bfloat16)
    f, pos = fa.rotary_freqs(96), i32(np.tile(np.arange(300), (2, 1)))
    want = fa.rotary(q, k, pos, f, interleaved=True)
    a, b = torch.empty_like(q), torch.empty_like(k)
    fa.fa_rotary(q, k, pos, f, a, b, interleaved=True)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c, d = fa.rotary(q, k, pos, f, interleaved=True, stream=s)
    s.synchronize()
    assert torch.equal(c, want[0]) and torch.equal(d, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = fa.rotary(q, k, pos, f, interleaved=True)
        z = fa.rotary_backward(*y, pos, f, interleaved=True)
    q.copy_(torch.randn_like(q))
    k.copy_(torch.randn_like(k))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    w = fa.rotary(q, k, pos, f, interleaved=True)
    x = fa.rotary_backward(*w, pos, f, interleaved=True)
    assert all(torch.equal(m, n) for m, n in zip((*y, *z), (*w, *x)))


def test_rows_past_2_31_elements():
    B, H, N, d = 1, 2, 4200000, 256
    q = torch.zeros(B, H, N, d, dtype=torch.bfloat16, device="cuda")
    at = N - 5
    row = torch.randn(d).to(torch.bfloat16).cuda()
    q[0, 1, at] = row
    f = fa.rotary_freqs(256)
    fa.rotary(q, None, None, f, out=(q, None))
    close(q[:, 1:, at:at + 1], row.view(1, 1, 1, d), np.array([[at]]), f, torch.bfloat16)
    assert not bool(q[0, 0, -1].any())
