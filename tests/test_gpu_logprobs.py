"""Log-probabilities of committed tokens against the definition in 64 bits.

Ids and ranks have to be equal.  Tolerances, from the arithmetic: with d =
(x - max) / T in fp32, exp d is off by (3 |d| + 4) 2^-24 relative; a sum of
positive terms over chains of at most 700 additions adds 700 * 2^-24.  So the
normaliser, relative, and lse - max, absolute, are off by at most z = 2^-24 *
(3 E|d| + 704), log-probabilities by z + 2^-22 |d|, and the entropy (lse - max
minus the mean of d) by z + (z + 2^-22) E|d|."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv

pytestmark = pytest.mark.gpu

VER = {}


def verifier(flags=0):
    if flags not in VER:
        VER[flags] = sv.Verifier(1 << 16, sv.SV_MAX_SPEC_LEN, 1 << 19, flags=flags)
    return VER[flags]


def make(N, G, V, dtype, *, ragged=False, pad=0, shift=0, temps=None, seed=0, spread=2.5, levels=None):
    gen = torch.Generator().manual_seed(seed)
    gam = torch.randint(0, G + 1, (N,), generator=gen) if ragged else torch.full((N,), G)
    rows = int(gam.sum()) + N
    x = spread * torch.randn(rows, V, generator=gen)
    if levels:  # a few distinct values: ties everywhere
        x = (x * levels / spread).round() / levels
    flat = torch.zeros(rows * (V + pad) + shift, dtype=dtype, device="cuda")
    logits = flat[shift:].view(rows, V + pad)[:, :V]
    logits.copy_(x)
    com = (torch.rand(N, generator=gen) * (gam + 1)).long()  # accepted drafts
    tok = torch.randint(0, V, (N, G + 1), generator=gen, dtype=torch.int32)
    tok[torch.arange(G + 1)[None, :] > com[:, None]] = -1
    t = None
    if temps:
        t = torch.tensor([temps[i % len(temps)] for i in range(N)], dtype=torch.float32)
    return dict(logits=logits, tokens=tok, gam=gam, G=G, temperature=t,
                cu=gam.cumsum(0).to(torch.int32) if ragged else None)


def run(c, K, flags=0, stream=None):
    N, cols = c["tokens"].shape
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(logprobs=torch.full((N, cols), 777.0, device="cuda"), entropy=torch.full((N, cols), 777.0, device="cuda"),
              ranks=torch.full((N, cols), 777, dtype=torch.int32, device="cuda"),
              top_ids=torch.full((N, cols, K), 777, dtype=torch.int32, device="cuda"),
              top_logprobs=torch.full((N, cols, K), 777.0, device="cuda"))
    r = verifier(flags).logprobs(logits=c["logits"], out_tokens=c["tokens"].cuda(),
                                 cu_num_draft_tokens=None if c["cu"] is None else c["cu"].cuda(),
                                 temperature=None if c["temperature"] is None else c["temperature"].cuda(),
                                 num_top=K, status=status, stream=stream, **kw)
    torch.cuda.synchronize()
    return [t.cpu() for t in (r.logprobs, r.ranks, r.entropy, r.top_ids, r.top_logprobs)], int(status.item())


def check(c, K, **kw):
    (logp, ranks, ent, ids, tlp), status = run(c, K, **kw)
    assert status == 0
    x_all = c["logits"].cpu().double()
    first = 0
    for i in range(len(c["gam"])):
        T = 1.0 if c["temperature"] is None else float(c["temperature"][i]) or 1.0
        for m in range(c["G"] + 1):
            tok = int(c["tokens"][i, m])
            if tok < 0:
                assert logp[i, m] == 0 and ent[i, m] == 0 and ranks[i, m] == -1
                assert bool((ids[i, m] == -1).all()) and bool((tlp[i, m] == 0).all())
                continue
            raw = x_all[first + m]
            d = (raw - raw.max()) / T
            p = torch.softmax(d, 0)
            live = p > 0
            mean = float((p * d.abs())[live].sum())
            z = 2.0 ** -24 * (3 * mean + 704)
            lse = float(torch.logsumexp(d, 0))
            want = d - lse
            if torch.isinf(want[tok]):
                assert logp[i, m] == -float("inf")
            else:
                assert abs(float(logp[i, m]) - float(want[tok])) <= z + 2.0 ** -22 * abs(float(d[tok]))
            assert abs(float(ent[i, m]) - (lse + mean)) <= z + (z + 2.0 ** -22) * mean
            assert int(ranks[i, m]) == 1 + int((raw > raw[tok]).sum())
            if K:
                order = torch.sort(raw, descending=True, stable=True).indices[:K]
                assert torch.equal(ids[i, m].long(), order)
                got, exact = tlp[i, m].double(), want[order]
                assert torch.equal(torch.isinf(got), torch.isinf(exact))
                fin = ~torch.isinf(exact)
                assert bool(((got - exact).abs() <= z + 2.0 ** -22 * d[order].abs())[fin].all())
        first += int(c["gam"][i]) + 1


CASES = {
    "one entry": (dict(N=2, G=0, V=1, dtype=torch.float32), 1),
    "seven entries, all of them": (dict(N=3, G=2, V=7, dtype=torch.bfloat16), 7),
    "small, no alternatives": (dict(N=4, G=4, V=1000, dtype=torch.bfloat16), 0),
    "odd size, odd stride": (dict(N=5, G=3, V=3001, dtype=torch.bfloat16, ragged=True, pad=2, shift=3), 20),
    "odd size, fp32": (dict(N=5, G=3, V=4099, dtype=torch.float32, ragged=True, pad=1, shift=1), 32),
    "ties everywhere": (dict(N=6, G=1, V=5000, dtype=torch.bfloat16, levels=2), 32),
    "ties everywhere, fp32": (dict(N=6, G=1, V=5000, dtype=torch.float32, levels=2), 31),
    "temperatures": (dict(N=6, G=2, V=2000, dtype=torch.float32, temps=[0.0, 0.3, 1.0, 3.0]), 5),
    "temperatures, bf16": (dict(N=6, G=2, V=2000, dtype=torch.bfloat16, temps=[0.0, 0.3, 1.0, 3.0], ragged=True), 5),
    "one long row": (dict(N=1, G=0, V=151936, dtype=torch.bfloat16), 20),
    "one long row, fp32": (dict(N=1, G=0, V=262145, dtype=torch.float32), 20),
    "one long row, unaligned": (dict(N=1, G=1, V=128257, dtype=torch.bfloat16, shift=1, pad=1), 20),
    "a few long rows": (dict(N=9, G=4, V=128256, dtype=torch.bfloat16, ragged=True), 8),
    "many rows": (dict(N=700, G=0, V=900, dtype=torch.float32), 3),
    "many longer rows": (dict(N=400, G=0, V=20001, dtype=torch.bfloat16, pad=7), 11),
    "a wide range": (dict(N=3, G=1, V=6000, dtype=torch.float32, spread=300.0), 6),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    kw, K = CASES[name]
    check(make(seed=len(name), **kw), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_entries(dtype):
    """-inf and the type's lowest value among the logits, in blocks and alone, and a row with one finite entry."""
    c = make(4, 0, 5003, dtype, seed=20)
    c["logits"][0, 100:4000] = -float("inf")
    c["logits"][1, :] = -float("inf")
    c["logits"][1, 4242] = 1.5
    c["logits"][2, ::2] = torch.finfo(dtype).min
    c["logits"][3, 1:] = torch.finfo(dtype).min
    c["tokens"][0, 0] = 200  # a masked token: log-probability -inf
    c["tokens"][1, 0] = 4242
    check(c, 9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows_and_signed_zeros(dtype):
    c = make(3, 0, 3000, dtype, seed=21)
    c["logits"][0] = -2.0
    c["logits"][1] = 0.0
    c["logits"][1, ::3] = -0.0  # equal to +0: the lowest index first
    c["logits"][2] = torch.finfo(dtype).max
    check(c, 32)


def test_bad_rows_and_parameters():
    bits, nan = sv.DATA_STATUS_BITS, float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        clean = make(5, 0, 2000, dtype, seed=22)
        want, _ = run(clean, 4)

        def damaged(change, bit, bad):
            c = dict(clean, logits=clean["logits"].clone(), tokens=clean["tokens"].clone(),
                     temperature=torch.ones(5), cu=None)
            change(c)
            got, status = run(c, 4)
            assert status == bits[bit]
            assert torch.isnan(got[0][bad]).all() and torch.isnan(got[2][bad]).all() and torch.isnan(got[4][bad]).all()
            assert (got[1][bad] == -1).all() and (got[3][bad] == -1).all()
            for a, b in zip(got, want):
                a[bad] = b[bad]
                assert torch.equal(a, b)

        damaged(lambda c: c["logits"].__setitem__((1, 1999), nan), "BAD_VALUES", 1)
        damaged(lambda c: c["logits"].__setitem__((4, 0), float("inf")), "BAD_VALUES", 4)
        damaged(lambda c: c["logits"].__setitem__((2, slice(None)), -float("inf")), "BAD_VALUES", 2)
        damaged(lambda c: c["tokens"].__setitem__((0, 0), 2000), "BAD_DRAFT_ID", 0)
        damaged(lambda c: c["tokens"].__setitem__((0, 0), -2), "BAD_DRAFT_ID", 0)
        for t in (-1.0, nan, float("inf"), 1e-40):
            damaged(lambda c: c["temperature"].__setitem__(3, t), "BAD_PARAM", 3)


def test_bad_ranges():
    c = make(4, 3, 500, torch.float32, ragged=True, seed=23)
    want, _ = run(c, 2)
    c["cu"] = c["cu"].clone()
    c["cu"][3] = 100
    got, status = run(c, 2)
    assert status == sv.DATA_STATUS_BITS["BAD_CU"]
    for a, b in zip(got, want):
        assert torch.equal(a[:3], b[:3])
    assert (got[0][3] == 0).all() and (got[1][3] == -1).all() and (got[3][3] == -1).all()


def test_rejected_rows_are_not_read():
    c = make(6, 4, 3000, torch.bfloat16, seed=24)
    want, _ = run(c, 5)
    for i in range(6):
        for m in range(5):
            if c["tokens"][i, m] < 0:
                c["logits"][i * 5 + m] = float("nan")
    got, status = run(c, 5)
    assert status == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N,G,V,dtype", [(40, 3, 30000, torch.bfloat16), (2, 1, 151936, torch.float32)])
def test_repeats_and_launch_modes_are_bitwise_equal(N, G, V, dtype):
    c = make(N, G, V, dtype, seed=25)
    want, _ = run(c, 20)
    for flags in (0, sv.SV_FLAG_SERIAL_LAUNCH):
        got, _ = run(c, 20, flags=flags)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = run(c, 20, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_after_a_verification():
    """out_tokens as spec_verify_run leaves them, read in stream order."""
    N, G, V = 8, 4, 2000
    gen = torch.Generator().manual_seed(26)
    target = 2.5 * torch.randn(N * (G + 1), V, generator=gen)
    draft = target.view(N, G + 1, V)[:, :G].reshape(-1, V) + 0.5 * torch.randn(N * G, V, generator=gen)
    ids = draft.argmax(-1).to(torch.int32).cuda()
    target = target.to(torch.bfloat16).cuda()
    ver = verifier()
    res = ver.verify(entry="logits", draft_ids=ids, target=target, draft=draft.to(torch.bfloat16).cuda(),
                     max_spec_len=G, num_reqs=N, seed=3)
    r = ver.logprobs(logits=target, out_tokens=res.out_tokens, num_top=4)
    torch.cuda.synchronize()
    tok = res.out_tokens.cpu()
    assert torch.equal(r.ranks.cpu() >= 1, tok >= 0)
    check(dict(logits=target, tokens=tok, gam=torch.full((N,), G), G=G, temperature=None, cu=None), 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [3, 20])
def test_most_blocks_masked(dtype, K):
    c = make(320, 0, 40000, dtype, seed=29)
    c["logits"][:, 9:39990] = -float("inf")  # 19 entries left, in the first and the last block
    c["tokens"][c["tokens"] >= 0] = 7
    check(c, K)


# Rows, or their shares in a cluster, with fewer 2 KB blocks than alternatives: parts of blocks decide.
FEW = {
    "one block": (dict(N=5, G=1, V=1000, dtype=torch.bfloat16), 32),
    "less than one block": (dict(N=3, G=0, V=40, dtype=torch.float32), 32),
    "fewer lanes than alternatives": (dict(N=3, G=0, V=100, dtype=torch.bfloat16, shift=5), 32),
    "eight blocks and one entry": (dict(N=400, G=0, V=8193, dtype=torch.bfloat16), 9),
    "nine blocks, four lanes a part": (dict(N=400, G=0, V=9215, dtype=torch.bfloat16, pad=1), 32),
    "blocks one short": (dict(N=350, G=0, V=31 * 512, dtype=torch.float32, shift=3, pad=1), 32),
    "as many blocks as alternatives": (dict(N=350, G=0, V=32 * 512, dtype=torch.float32), 32),
    "shares of a cluster": (dict(N=2, G=1, V=92471, dtype=torch.bfloat16, pad=8, temps=[0.7]), 32),
    "shares of a cluster, fp32": (dict(N=2, G=1, V=50001, dtype=torch.float32, pad=3), 31),
    "ties": (dict(N=350, G=0, V=7001, dtype=torch.bfloat16, levels=8), 32),
    "ties in shares": (dict(N=2, G=0, V=60001, dtype=torch.float32, levels=16), 32),
}


@pytest.mark.parametrize("name", FEW)
def test_few_blocks(name):
    kw, K = FEW[name]
    check(make(seed=100 + len(name), **kw), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_blocks_with_masked_entries(dtype):
    c = make(4, 1, 6000, dtype, seed=31)
    c["logits"][:, 20:5990] = -float("inf")  # 30 entries left, fewer than alternatives
    c["tokens"][c["tokens"] >= 0] = 7
    check(c, 32)
