"""Rotary positions and norms against the formula in 64 bits.

Tolerances.  With u = 2^-24 (half a step of fp32): an angle's sine and cosine are
off by at most 4 u each (their argument is at most pi / 4 and rounded to fp32, the
functions themselves are good to 2 u, the factor's product adds one), a product
and a sum add 2 u of what they combine; so a rotated element is off by at most
8 u (|a| + |b|) * magnitude.  A norm multiplies by a root good to (D / 2 + 4) u
relative -- D / 32 + 6 partial sums in the worst order stay far below that -- and
by a weight: (D / 2 + 8) u more.  bf16 outputs add 2^-8 of the result, fp32 ones u."""
import math

import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ver():
    v = sv.Verifier(1, 0, 1)
    yield v
    v.close()


def reference(x, positions, f, weight, eps, interleaved):
    """(value, tolerance before the last rounding) in 64 bits."""
    y = x.double()
    D, r = y.shape[-1], f.rotary_dim
    tol = torch.zeros_like(y)
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
        tol = (D / 2 + 8) * U * y.abs()
    inv = torch.tensor(f.inverse, dtype=torch.float64, device=x.device)
    t = positions.double()[:, None] * inv
    c, s = (torch.cos(t) * f.magnitude)[:, None], (torch.sin(t) * f.magnitude)[:, None]
    i = torch.arange(r // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    out, err = y.clone(), tol.clone()
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    e = 8 * U * (y[..., a].abs() + y[..., b].abs()) * abs(f.magnitude) + (tol[..., a] + tol[..., b]) * abs(f.magnitude)
    err[..., a], err[..., b] = e, e
    return out, err


def check(got, x, positions, f, weight=None, eps=1e-6, interleaved=False):
    want, err = reference(x, positions, f, weight, eps, interleaved)
    half_step = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    live = (positions >= 0)[:, None, None].expand_as(want)
    # (the last rounding is of the computed value, at most half a step of it, and of bf16's smallest step)
    bad = ((got.double() - want).abs() > err + half_step * (want.abs() + err) + 2.0 ** -126) & live
    assert not bool(bad.any()), float(((got.double() - want).abs() - err)[live].max())


def inputs(T, hq, hk, D, dtype, seed, far=100000, padded=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, hq + 2 * hk, D, generator=gen, device="cuda") * 3).to(dtype)
    pos = torch.randint(0, far, (T,), generator=gen, device="cuda").to(torch.int32)
    pos[torch.rand(T, generator=gen, device="cuda") < padded] = -1
    w = (1 + 0.3 * torch.randn(2, D, generator=gen, device="cuda")).to(dtype)
    return x[:, :hq], x[:, hq:hq + hk], pos, w


SHAPES = [  # tokens, query heads, key heads, head size, rotated part
    (1, 1, 1, 64, 64), (20, 32, 8, 128, 128), (333, 4, 1, 128, 64), (77, 8, 2, 256, 64), (1000, 3, 3, 80, 20),
    (50, 2, 1, 80, 80), (9, 5, 2, 96, 96), (64, 1, 0, 128, 32), (17, 0, 2, 64, 16), (5, 2, 2, 512, 512), (31, 2, 1, 7, 6),
    (40, 3, 1, 1, 0), (12, 4, 2, 128, 0), (3000, 16, 2, 64, 64), (6, 4, 4, 384, 96), (8, 70, 70, 32, 32),
]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hq,hk,D,r", SHAPES)
def test_against_the_formula(ver, T, hq, hk, D, r, dtype, interleaved, norm):
    q, key, pos, w = inputs(T, hq, hk, D, dtype, T + D)
    f = sv.RotaryFrequencies(r, base=10000.0, device="cuda")
    qw, kw = (w[0], w[1]) if norm else (None, None)
    qo = torch.full((T, hq, D), 7.0, dtype=dtype, device="cuda")
    ko = torch.full((T, hk, D), 7.0, dtype=dtype, device="cuda")
    ver.rotate(q=q if hq else None, key=key if hk else None, positions=pos, frequencies=f, q_out=qo if hq else None,
               key_out=ko if hk else None, q_weight=qw, key_weight=kw, interleaved=interleaved)
    check(qo, q, pos, f, qw, interleaved=interleaved)
    check(ko, key, pos, f, kw, interleaved=interleaved)
    idle = pos < 0
    assert bool((qo[idle] == 7.0).all()) and bool((ko[idle] == 7.0).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_is_the_same(ver, dtype, norm):
    q, key, pos, w = inputs(100, 8, 2, 128, dtype, 3)
    f = sv.RotaryFrequencies(128)
    kw = dict(q_weight=w[0], key_weight=w[1]) if norm else {}
    qo, ko = q.clone(), key.clone()
    ver.rotate(q=q, key=key, positions=pos, frequencies=f, q_out=qo, key_out=ko, **kw)
    a, b = ver.rotate(q=q, key=key, positions=pos, frequencies=f, **kw)
    assert a is q and b is key and torch.equal(a, qo) and torch.equal(b, ko)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_and_unaligned_rows(ver, dtype, interleaved):
    q, key, pos, w = inputs(70, 6, 2, 128, dtype, 4)
    f = sv.RotaryFrequencies(64)
    odd = torch.zeros(6, 70, 131, dtype=dtype, device="cuda").permute(1, 0, 2)[..., 3:]
    odd.copy_(q)
    ko = torch.zeros(70, 5, 130, dtype=dtype, device="cuda")
    ko[:, 1::2, 1:129] = key
    ww = torch.zeros(257, dtype=dtype, device="cuda")[1:].view(2, 128)
    ww.copy_(w)
    a, b = ver.rotate(q=odd, key=key, positions=pos, frequencies=f, q_out=odd, key_out=ko[:, 1::2, 1:129],
                      q_weight=ww[0], key_weight=ww[1], interleaved=interleaved)
    check(a, q, pos, f, w[0], interleaved=interleaved)
    check(b, key, pos, f, w[1], interleaved=interleaved)
    idle = pos < 0
    assert torch.equal(a[idle], q[idle]) and torch.equal(b[idle], key[idle])  # (what was there)
    assert bool((ko[:, 0::2] == 0).all()) and bool((ko[..., 0] == 0).all())


def test_far_positions_lose_nothing(ver):
    """Up to the largest position, where a product in fp32 would be off by many turns."""
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    x = torch.randn(6, 4, 128, generator=torch.Generator().manual_seed(6)).cuda()
    f = sv.RotaryFrequencies(128, base=1e6)
    out, _ = ver.rotate(q=x, positions=pos, frequencies=f, q_out=torch.empty_like(x))
    # the formula by whole numbers: the fraction of a turn, from the turns of a position to 2^-64
    words = [int(t) % (1 << 64) for t in f.turns.tolist()]
    for k, p in enumerate(pos.tolist()):
        t = torch.tensor([((w * p) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for w in words], dtype=torch.float64).cuda()
        a, b = x[k, :, :64].double(), x[k, :, 64:].double()
        want = torch.cat([a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()], -1)
        assert bool(((out[k].double() - want).abs() <= 9 * U * torch.cat([a.abs() + b.abs()] * 2, -1)).all())


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
                                dict(base=500000.0, scaling="yarn", factor=16.0, trained_len=32768),
                                dict(inverse=[0.5 ** i for i in range(32)], magnitude=1.25), dict(magnitude=-0.5)])
def test_scaled_frequencies(ver, kw):
    q, key, pos, w = inputs(40, 4, 2, 64, torch.float32, 5, far=1 << 20)
    f = sv.RotaryFrequencies(64, **kw)
    a, b = ver.rotate(q=q, key=key, positions=pos, frequencies=f, q_out=q.clone(), key_out=key.clone())
    check(a, q, pos, f)
    check(b, key, pos, f)


def test_turning_keeps_what_attention_sees(ver):
    """Products of queries and keys depend on the distance of their positions alone."""
    gen = torch.Generator().manual_seed(7)
    q, k = torch.randn(1, 1, 128, generator=gen).cuda(), torch.randn(1, 1, 128, generator=gen).cuda()
    f = sv.RotaryFrequencies(128)
    dots = []
    for at in (5, 1000, 99999):
        pos = torch.tensor([at], dtype=torch.int32, device="cuda")
        a, b = ver.rotate(q=q, key=k, positions=pos, frequencies=f, q_out=torch.empty_like(q), key_out=torch.empty_like(k))
        c, _ = ver.rotate(q=q, positions=pos - 3, frequencies=f, q_out=torch.empty_like(q))
        dots.append((float((a * b).sum()), float((c * b).sum())))
    # a pair's two products are off by 32 u of (|qa| + |qb|)(|ka| + |kb|), their sums by 256 u more, on both sides
    pairs = [t[0, 0, :64].abs() + t[0, 0, 64:].abs() for t in (q, k)]
    for x in dots[1:]:
        assert all(abs(u - v) <= 576 * U * float((pairs[0] * pairs[1]).sum()) for u, v in zip(x, dots[0]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norms_of_zero_small_and_infinite_rows(ver, dtype):
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(8)).cuda()
    x[0] = 0
    x[1] *= 1e-4
    x[2] *= 1e12
    x = x.to(dtype)
    x[3, 0, 5] = float("nan")
    x[4, 1, 3] = float("inf")
    w = torch.ones(64, dtype=dtype, device="cuda")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    f = sv.RotaryFrequencies(64)
    out, _ = ver.rotate(q=x, positions=pos, frequencies=f, q_weight=w, eps=1e-5, q_out=torch.empty_like(x))
    clean = [0, 1, 2, 5]
    check(out[clean], x[clean], pos[clean], f, w, 1e-5)
    assert bool((out[0] == 0).all()) and bool(torch.isnan(out[3, 0]).all()) and not bool(torch.isnan(out[3, 1]).any())
    assert bool(torch.isnan(out[4, 1, 3])) and not bool(torch.isnan(out[4, 0]).any())


def test_on_another_stream_and_in_a_graph(ver):
    q, key, pos, w = inputs(50, 8, 2, 128, torch.bfloat16, 9)
    f = sv.RotaryFrequencies(128)
    qo, ko = q.clone(), key.clone()
    want = ver.rotate(q=q, key=key, positions=pos, frequencies=f, q_out=q.clone(), key_out=key.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ver.rotate(q=q, key=key, positions=pos, frequencies=f, q_out=qo, key_out=ko, stream=side)
    side.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ver.rotate(q=q, key=key, positions=pos, frequencies=f, q_out=qo, key_out=ko)
    pos.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    check(qo, q, pos, f)
    check(ko, key, pos, f)


def test_no_tokens_and_no_heads(ver):
    f = sv.RotaryFrequencies(64)
    none = torch.empty(0, 4, 64, device="cuda")
    ver.rotate(q=none, positions=torch.empty(0, dtype=torch.int32, device="cuda"), frequencies=f)
    ver.rotate(q=torch.empty(5, 0, 64, device="cuda"), positions=torch.zeros(5, dtype=torch.int32, device="cuda"),
               frequencies=f)
    torch.cuda.synchronize()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,r,at", [(128, 64, 100), (128, 64, 64), (80, 20, 33), (128, 0, 5), (64, 32, 63)])
def test_an_infinity_in_what_stays_stays_alone(ver, D, r, at, dtype, interleaved):
    q, key, pos, _ = inputs(30, 4, 1, D, dtype, at)
    q[:, 1, at], q[:, 2, at] = math.inf, math.nan
    f = sv.RotaryFrequencies(r)
    qo = torch.empty_like(q)
    ver.rotate(q=q, positions=pos, frequencies=f, q_out=qo, interleaved=interleaved)
    live = pos >= 0
    assert bool((qo[live, 1, at] == math.inf).all()) and bool(qo[live, 2, at].isnan().all())
    clean, want = q.clone(), qo.clone()
    clean[:, 1:3, at] = want[:, 1:3, at] = 0
    check(want, clean, pos, f, interleaved=interleaved)
