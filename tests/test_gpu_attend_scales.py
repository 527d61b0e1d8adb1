"""Attention over caches whose scales kv_write would not have written: byte x
stands for x * scale whatever the scale is.  A value scale of 0 makes a zero
value, whose key still counts in lse and in the weights' sum; a negative one
turns a value round; one that is no number makes the outputs of the rows that
see the key NaN, and leaves their lse alone; one below 2^-64, the writer's
smallest, counts as 0.

Tolerances are those of test_gpu_attend.py.  In the term for 16-bit weights
that underflow, the largest product of a weight and its value's scale counts
each scale as 2^-64 at least."""
import math

import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend import make, run, verifier

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -64


def shared_prefix(gammas, *, kv_heads=2, group=4, dim=128, block=16, uniform=True, **_):
    """The shortest prefix that a call of these sizes computes once for all requests.  (One that every request reads for
    itself needs the workspace of a call without a prefix.)"""
    N, G = len(gammas), max(gammas)
    rows = sum(gammas) + N
    assert rows * group >= 96

    def size(prefix, most):
        return sv.spec_verify_attend_workspace_size(verifier().handle, num_reqs=N, max_spec_len=G,
                                                    num_q_heads=kv_heads * group, num_kv_heads=kv_heads, head_dim=dim,
                                                    max_seq_len=most, shared_prefix_len=prefix, num_tokens=rows)

    for prefix in range(128 // block * block, 1 << 16, block):
        if size(prefix, prefix + 4096) != size(0, prefix + 4096):
            return prefix
    raise AssertionError("no prefix is shared")


def shared(gammas, own, **kw):
    """A call with a prefix that is shared; `own`: tokens behind it (before its end if negative; None: no tokens at all)."""
    prefix = shared_prefix(gammas, **kw)
    return make(gammas, [0 if n is None else prefix + n for n in own], prefix=prefix, **kw)


FORMS = {
    "few rows": lambda seed, **kw: make([3, 1], [400, 90], seed=seed, **kw),
    "many requests": lambda seed, **kw: make([1] * 30, [20 + 11 * i for i in range(30)], seed=seed, **kw),
    "prefix, few rows": lambda seed, **kw: make([1, 0], [2500, 2421], prefix=2400, group=2, seed=seed, **kw),
    "prefix, many rows": lambda seed, **kw: shared([4] * 40, [10 + i for i in range(40)], uniform=True, seed=seed, **kw),
}


def reference(c):
    """(out, lse, tolerance of out, tolerance of lse), in 64 bits; NaN in out where a value that a row sees is none."""
    cache, grp = c["cache"], c["group"]
    h, d, b = cache.num_kv_heads, cache.head_dim, cache.block_size
    rows = c["q"].shape[0]
    out = torch.zeros(rows, h, grp, d, dtype=torch.float64, device="cuda")
    lse = torch.full((rows, h, grp), -math.inf, dtype=torch.float64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for i, (g, n) in enumerate(zip(c["gammas"], c["lens"])):
        if n > 0:
            t = torch.arange(n, device="cuda")
            page, off = c["table"][i].long()[t // b], t % b

            def side(data, scale):
                raw = (data if data.dtype == torch.int8 else data.view(torch.uint8))[page, :, off]
                x = raw.double() if data.dtype == torch.int8 else raw.view(torch.float8_e4m3fn).double()
                return x.permute(1, 0, 2), scale[page, :, off].double().t()[..., None]  # [h, n, d], [h, n, 1]

            (kb, ks), (vb, vs) = side(cache.k, cache.k_scale), side(cache.v, cache.v_scale)
            k = kb * ks
            odd = ~torch.isfinite(vs)
            vs = torch.where(odd | (vs.abs() < LEAST), torch.zeros_like(vs), vs)
            v = vb * vs
            q = c["q"][at:at + g + 1].double().reshape(g + 1, h, grp, d).permute(1, 0, 2, 3).reshape(h, -1, d)
            a = torch.matmul(q, k.transpose(1, 2)) * c["scale"]
            big = (torch.matmul(q.abs(), k.abs().transpose(1, 2)) * abs(c["scale"])).amax(-1)
            pos = n - (g + 1) + torch.arange(g + 1, device="cuda").repeat_interleave(grp)
            see = t[None, :] <= pos[:, None]
            a = a.masked_fill(~see, -math.inf)
            z = torch.logsumexp(a, -1)
            p = torch.exp(a - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o, e = torch.matmul(p, v), 2.0 ** -24 * (d + 32) * big
            w = (2 * e + 2.0 ** -20 + 2.0 ** -11)[..., None] * torch.matmul(p, v.abs()) + 2.0 ** -8 * o.abs()
            most = (p * vs.abs().clamp_min(LEAST).transpose(1, 2)).amax(-1, keepdim=True)
            w = w + 2.0 ** -25 * most * torch.matmul(see.double().expand(h, -1, -1), vb.abs() * (vs != 0))
            o = torch.where(torch.matmul(see.double().expand(h, -1, -1), odd.double()) > 0, math.nan, o)
            y = e + 2.0 ** -20 * (1 + torch.where(torch.isinf(z), torch.zeros_like(z), z).abs())
            for dst, src in ((out, o), (tol, w)):
                dst[at:at + g + 1] = src.reshape(h, g + 1, grp, d).permute(1, 0, 2, 3)
            for dst, src in ((lse, z), (ltol, y)):
                dst[at:at + g + 1] = src.reshape(h, g + 1, grp).permute(1, 0, 2)
        at += g + 1
    return out.reshape(rows, -1, d), lse.reshape(rows, -1), tol.reshape(rows, -1, d), ltol.reshape(rows, -1)


def check(c, status=0, **kw):
    out, lse, got = run(c, **kw)
    ref, rlse, tol, ltol = reference(c)
    assert got == status
    assert torch.equal(torch.isinf(lse), torch.isinf(rlse)) and not bool(torch.isnan(lse).any())
    live = ~torch.isinf(rlse)
    assert bool(((lse.double() - rlse).abs() <= ltol)[live].all())
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    number = ~torch.isnan(ref)
    assert bool((out.double() - ref).abs().le(tol)[number].all())
    return out, lse


def some(c, share, seed=5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(c["cache"].v_scale.shape, generator=gen, device="cuda") < share


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("share", [0.02, 0.5, 1.0])
@pytest.mark.parametrize("form", FORMS)
def test_value_scales_of_zero(form, share, fmt):
    c = FORMS[form](1, fmt=fmt)
    c["cache"].v_scale[some(c, share)] = 0.0
    check(c)


@pytest.mark.parametrize("form", FORMS)
def test_a_zero_value_scale_at_the_row_s_best_key(form):
    """Its weight is nearly all of the sum: out is next to nothing, lse that key's score."""
    c = FORMS[form](2)
    c["q"] = c["q"] * 20
    zero = some(c, 0.02)
    c["cache"].v_scale[zero] = 0.0
    c["cache"].k_scale[zero] *= 4
    check(c)


@pytest.mark.parametrize("form", FORMS)
def test_negative_value_scales(form):
    c = FORMS[form](3)
    c["cache"].v_scale[some(c, 0.4)] *= -1
    check(c)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS)
def test_value_scales_that_are_no_numbers(form, value):
    """Out of the rows that see one is NaN (for its head only); lse, and the other rows, are what they were."""
    c = FORMS[form](4)
    cache, b = c["cache"], c["cache"].block_size
    for i, back in ((0, 1), (len(c["lens"]) - 1, 2)):  # seen by the last row of a request, and by the last two
        k = c["lens"][i] - back
        cache.v_scale[int(c["table"][i, k // b]), 1, k % b] = value
    out, _ = check(c)
    assert bool(torch.isnan(out).any()) and not bool(torch.isnan(out).all())
    # and a key of the prefix, or of one request's first page
    k = 5
    cache.v_scale[int(c["table"][0, k // b]), 0, k % b] = value
    check(c)


@pytest.mark.parametrize("form", FORMS)
def test_value_scales_below_the_writer_s_smallest(form):
    c = FORMS[form](6)
    for size, share in ((2.0 ** -70, 0.3), (2.0 ** -100, 0.2), (2.0 ** -140, 0.2)):
        c["cache"].v_scale[some(c, share, seed=int(-math.log2(size)))] = size
    check(c)
    c["cache"].v_scale.fill_(2.0 ** -66)
    check(c)


@pytest.mark.parametrize("form", FORMS)
def test_zero_rows_before_large_ones(form):
    """The first value rows are zeros as the writer leaves them (scale 2^-64), the later ones near 2^36."""
    c = FORMS[form](7)
    b = c["cache"].block_size
    c["cache"].v_scale.mul_(2.0 ** 36)
    for t in range(160):
        if t < min(c["lens"]) or c["prefix"]:
            page, off = int(c["table"][0, t // b]), t % b
            c["cache"].v_scale[page, :, off] = LEAST
            c["cache"].v[page, :, off] = 0
    check(c)


@pytest.mark.parametrize("form", FORMS)
def test_tiny_queries_and_huge_keys(form):
    """Key scales up to the stated 2^96 (with the call's own), queries as small as makes the scores ordinary ones."""
    c = FORMS[form](8)
    c["q"] = (c["q"].float() * 2.0 ** -97).to(torch.bfloat16)
    k = c["cache"].k_scale
    k.mul_(2.0 ** 97)
    most = 2.0 ** 95 / c["scale"]
    k.clamp_(max=most)
    k[some(c, 0.01)] = most
    check(c)
