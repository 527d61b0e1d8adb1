"""Cases of the operators around a verification step: the paged 8-bit KV cache
(written, read back), the verify tokens' attention over it with a prefix
shared by the batch, and the log-probabilities of the committed tokens.

With ``own`` false ``run`` computes an operator in plain torch operations (32
bits, rounded once at the end); with ``own`` true it calls this package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"int8": 127.0, "e4m3": 448.0}
MIN_SCALE = 2.0 ** -64  # the cache's smallest scale: a zero row still has a positive one


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _store(name, tokens, kv_heads, dim, block, fmt, dtype, nhd=False, rolled=0, lens=1):
    return dict(name=name, op="store", tokens=tokens, kv_heads=kv_heads, dim=dim, block=block, fmt=fmt, dtype=dtype,
                nhd=nhd, rolled=rolled, lens=lens)


def _fetch(name, tokens, kv_heads, dim, block, fmt, dtype, nhd=False, lens=1):
    return dict(name=name, op="fetch", tokens=tokens, kv_heads=kv_heads, dim=dim, block=block, fmt=fmt, dtype=dtype,
                nhd=nhd, lens=lens)


def _attend(name, reqs, spec, ragged, prefix, least, most, q_heads, kv_heads, dim, block, fmt, nhd=False, lens=1):
    return dict(name=name, op="attend", reqs=reqs, spec=spec, ragged=ragged, prefix=prefix, least=least, most=most,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, block=block, fmt=fmt, nhd=nhd, lens=lens)


def _logprobs(name, reqs, spec, ragged, vocab, top, dtype, warm=False, pad=0, lens=1):
    return dict(name=name, op="logprobs", reqs=reqs, spec=spec, ragged=ragged, vocab=vocab, top=top, dtype=dtype,
                warm=warm, pad=pad, lens=lens)


def listed():
    return [
        # the verify tokens of a small batch (4 requests, gamma 4) written and read back: a call whose latency counts
        _store("store_step_small", 20, 8, 128, 16, "int8", "bf16"),
        # one step of the full batch (512 requests, gamma 7), a third of the slots rolled back to -1
        _store("store_step_full", 4096, 8, 128, 16, "e4m3", "bf16", rolled=33),
        # a long prompt filled at once, fp32 rows, token-major pages of an odd size
        _store("store_prompt", 50001, 4, 64, 24, "int8", "f32", nhd=True),
        # pages gathered for one request that moves elsewhere
        _fetch("fetch_request", 1023, 8, 64, 16, "e4m3", "f32"),
        # many requests' pages gathered back to bf16
        _fetch("fetch_batch", 131072, 8, 128, 32, "int8", "bf16"),
        # one request, one token, a thousand cached tokens: the single-token form
        _attend("attend_single", 1, 0, False, 0, 1000, 1000, 32, 8, 128, 16, "int8"),
        # a system prompt shared by 64 requests that verify 4 drafts each
        _attend("attend_shared", 64, 4, False, 8192, 5, 1024, 32, 8, 128, 16, "int8"),
        # 256 ragged requests (gamma 0..8) with long private histories and no common prefix
        _attend("attend_private", 256, 8, True, 0, 0, 8192, 32, 8, 128, 16, "e4m3"),
        # the full batch over a long shared context, few own tokens each
        _attend("attend_shared_full", 512, 7, False, 16384, 8, 256, 32, 8, 128, 32, "e4m3"),
        # committed tokens of a small batch with five alternatives
        _logprobs("logprobs_small", 4, 4, False, 32000, 5, "bf16"),
        # committed tokens of a ragged batch, fp32 rows of an odd stride, temperatures
        _logprobs("logprobs_ragged", 256, 8, True, 128256, 8, "f32", warm=True, pad=1),
        # committed tokens of the full batch with twenty alternatives
        _logprobs("logprobs_full", 512, 7, False, 151936, 20, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "fetch", "attend", "attend", "logprobs"])
    fmt = rng.choice(["int8", "e4m3"])
    dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 24, 32, 64])
    nhd = rng.random() < 0.3
    lens = rng.randrange(1 << 20)
    if op in ("store", "fetch"):
        heads = rng.choice([1, 2, 3, 4, 8])
        tokens = _spread(rng, 1, 131072 * 1024 // (heads * 128))
        tokens = min(tokens, 131072)
        dtype = rng.choice(["bf16", "f32"])
        if op == "store":
            c = _store("", tokens, heads, dim, block, fmt, dtype, nhd, rng.choice([0, 20, 60]), lens)
        else:
            c = _fetch("", tokens, heads, dim, block, fmt, dtype, nhd, lens)
    elif op == "attend":
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8])
        spec = rng.choice([0, 1, 3, 4, 7])
        reqs = _spread(rng, 1, 256)
        prefix = block * rng.choice([0, 0, _spread(rng, 1, 8192 // block)])
        rows = reqs * (spec + 1) * group * kv_heads
        most = _spread(rng, spec + 1, 8192)
        # keep the scores of a drawn case within those of the largest listed one
        most = max(spec + 1, min(most, (1 << 30) // (rows * 4), (1 << 20) // reqs))
        c = _attend("", reqs, spec, rng.random() < 0.5, prefix, rng.choice([0, min(most, spec + 1)]), most,
                    kv_heads * group, kv_heads, dim, block, fmt, nhd, lens)
    else:
        reqs = _spread(rng, 1, 256)
        c = _logprobs("", reqs, rng.choice([0, 1, 4, 7]), rng.random() < 0.5, _spread(rng, 1000, 151936),
                      rng.choice([0, 1, 5, 20, 32]), rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                      rng.choice([0, 1, 8]), lens)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# a case's lengths (the same for every seed)
# ----------------------------------------------------------------------------
def _gammas(case):
    rng = random.Random(case["lens"])
    if not case["ragged"]:
        return [case["spec"]] * case["reqs"]
    return [rng.randint(0, case["spec"]) for _ in range(case["reqs"])]


def _committed(case):
    rng = random.Random(case["lens"] + 1)
    return [1 + sum(rng.random() < 0.6 for _ in range(g)) for g in _gammas(case)]


def _owned(case):
    """Private tokens of every request (0: an idle place of the batch); the verify tokens are among them."""
    rng = random.Random(case["lens"] + 2)
    out = []
    for g in _gammas(case):
        n = rng.randint(case["least"], case["most"])
        out.append(0 if n == 0 and case["prefix"] == 0 else max(n, g + 1))
    return out


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _quantise(x, fmt):
    """(bytes, scale) of x [..., D] in fp32."""
    most = x.abs().amax(-1)
    # (a divisor on the device: a true division, where a Python number would be multiplied by its reciprocal)
    scale = (most / most.new_full((), QMAX[fmt])).clamp_min(MIN_SCALE)
    y = x / scale[..., None]
    if fmt == "int8":
        return y.round().clamp(-127, 127).to(torch.int8), scale
    return y.to(torch.float8_e4m3fn), scale


def _bytes(t):
    return t if t.dtype == torch.int8 else t.view(torch.uint8)


def _values(raw, fmt):
    """fp32 numbers of gathered cache bytes."""
    return raw.float() if fmt == "int8" else raw.view(torch.float8_e4m3fn).float()


def _fill(gen, case, blocks):
    """One side (K or V) of a cache of `blocks` pages [blocks, heads, block, D] with its scales."""
    h, b, d = case["kv_heads"], case["block"], case["dim"]
    shape = (blocks, b, h, d) if case["nhd"] else (blocks, h, b, d)
    # activations have a few channels that are larger than the rest
    chan = torch.exp(0.5 * _randn(gen, d))
    data = torch.empty(shape, dtype=torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(shape[:-1], device=DEV)
    step = max(1, (1 << 28) // (h * b * d))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        q, s = _quantise(_randn(gen, n, *shape[1:]) * chan, case["fmt"])
        _bytes(data)[i:i + n] = _bytes(q)
        scale[i:i + n] = s
    return (data.permute(0, 2, 1, 3), scale.permute(0, 2, 1)) if case["nhd"] else (data, scale)


def _empty(case, blocks):
    h, b, d = case["kv_heads"], case["block"], case["dim"]
    shape = (blocks, b, h, d) if case["nhd"] else (blocks, h, b, d)
    data = torch.zeros(shape, dtype=torch.uint8, device=DEV)
    data = data.view(torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn)
    scale = torch.ones(shape[:-1], device=DEV)
    return (data.permute(0, 2, 1, 3), scale.permute(0, 2, 1)) if case["nhd"] else (data, scale)


def _handle(reqs, spec, vocab):
    """The verifier handle that the program keeps (only the package's own calls use one)."""
    if not own:
        return None
    import speculative_decoding_token_rejection_gb300 as sv
    return sv.Verifier(reqs, spec, vocab)


def _cache(s):
    """The package's description of the cache, kept beside the handle."""
    if not own:
        return None
    import speculative_decoding_token_rejection_gb300 as sv
    return sv.KVCache(k=s["k"], v=s["v"], k_scale=s["ks"], v_scale=s["vs"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("store", "fetch"):
        T, h, d, b = case["tokens"], case["kv_heads"], case["dim"], case["block"]
        blocks = -(-T // b) + 3
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        slots = torch.randperm(blocks - 1, generator=gen, device=DEV)[:-(-T // b)]
        slots = (slots[:, None] * b + torch.arange(b, device=DEV)).reshape(-1)[:T].contiguous()
        if op == "store":
            # key and value are slices of the projection's output, whose rows hold the query heads as well
            qkv = _randn(gen, T, 4 * h, d) * torch.exp(0.5 * _randn(gen, d))
            qkv = qkv.to(dt)
            s["key"], s["value"] = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
            gone = torch.rand(T, generator=gen, device=DEV) * 100 < case["rolled"]
            slots = torch.where(gone, torch.full_like(slots, -1), slots)
            s["k"], s["ks"] = _empty(case, blocks)
            s["v"], s["vs"] = _empty(case, blocks)
        else:
            s["k"], s["ks"] = _fill(gen, case, blocks)
            s["v"], s["vs"] = _fill(gen, case, blocks)
        s["slots"] = slots
        s["key_out"] = torch.empty(T, h, d, dtype=dt, device=DEV)
        s["value_out"] = torch.empty(T, h, d, dtype=dt, device=DEV)
        s["handle"], s["cache"] = _handle(1, 0, 1), _cache(s)
    elif op == "attend":
        N, b, h, hq, d = case["reqs"], case["block"], case["kv_heads"], case["q_heads"], case["dim"]
        gam, own_len = _gammas(case), _owned(case)
        need = [-(-n // b) for n in own_len]
        pre = case["prefix"] // b
        blocks = pre + sum(need) + 1
        width = pre + max(max(need), 1)
        order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros(N, width, dtype=torch.int32)
        place = torch.arange(blocks, dtype=torch.int32)
        at = pre
        for i in range(N):  # rows of logical page numbers, mapped to shuffled pages below
            table[i, :pre] = place[:pre]
            table[i, pre:pre + need[i]] = place[at:at + need[i]]
            at += need[i]
        s["table"] = order[table.to(DEV).long()].contiguous()
        s["seq_lens"] = torch.tensor([case["prefix"] + n for n in own_len], dtype=torch.int32, device=DEV)
        s["max_seq_len"] = case["prefix"] + max(case["most"], case["spec"] + 1)
        s["cu"] = torch.tensor(gam, device=DEV).cumsum(0).to(torch.int32) if case["ragged"] else None
        rows = sum(gam) + N
        qkv = _randn(gen, rows, hq + 2 * h, d).to(torch.bfloat16)
        s["q"] = qkv[:, :hq]
        s["k"], s["ks"] = _fill(gen, case, blocks)
        s["v"], s["vs"] = _fill(gen, case, blocks)
        s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(rows, hq, device=DEV)
        s["handle"], s["cache"] = _handle(N, case["spec"], 1), _cache(s)
        s["workspace"] = None
        if own:
            s["workspace"] = s["handle"].attend_workspace(num_reqs=N, max_spec_len=case["spec"], num_q_heads=hq,
                                                          num_kv_heads=h, head_dim=d, max_seq_len=s["max_seq_len"],
                                                          shared_prefix_len=case["prefix"], num_tokens=rows)
    else:
        N, G, V, K = case["reqs"], case["spec"], case["vocab"], case["top"]
        gam, com = _gammas(case), _committed(case)
        rows = sum(gam) + N
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = torch.empty(rows, V + case["pad"], dtype=dt, device=DEV)
        step = max(1, (1 << 28) // V)
        for i in range(0, rows, step):
            n = min(step, rows - i)
            wide[i:i + n, :V] = 2.5 * _randn(gen, n, V)
        s["logits"] = wide[:, :V]
        s["cu"] = torch.tensor(gam, device=DEV).cumsum(0).to(torch.int32) if case["ragged"] else None
        # most committed tokens are likely ones: the best of a few places of the row
        first = torch.tensor([sum(gam[:i]) + i for i in range(N)], device=DEV)
        col = torch.arange(G + 1, device=DEV)
        at = (first[:, None] + col).clamp_max(rows - 1)
        cand = torch.randint(0, V, (N, G + 1, 64), generator=gen, device=DEV)
        best = s["logits"][at[..., None], cand].float().argmax(-1, keepdim=True)
        tok = cand.gather(-1, best)[..., 0].to(torch.int32)
        s["tokens"] = torch.where(col < torch.tensor(com, device=DEV)[:, None], tok, torch.full_like(tok, -1))
        s["temperature"] = None
        if case["warm"]:
            s["temperature"] = 0.5 + torch.rand(N, generator=gen, device=DEV)
        s["handle"] = _handle(N, G, V)
        s["logprobs"] = torch.empty(N, G + 1, device=DEV)
        s["entropy"] = torch.empty(N, G + 1, device=DEV)
        s["ranks"] = torch.empty(N, G + 1, dtype=torch.int32, device=DEV)
        s["top_ids"] = torch.empty(N, G + 1, K, dtype=torch.int32, device=DEV)
        s["top_logprobs"] = torch.empty(N, G + 1, K, device=DEV)
    return s


# ----------------------------------------------------------------------------
# a pass
# ----------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "store":
        _plain_write(state, case)
        return _plain_read(state, case)
    if case["op"] == "fetch":
        return _plain_read(state, case)
    if case["op"] == "attend":
        return _plain_attend(state, case)
    return _plain_logprobs(state, case)


def _run_own(s, case):
    op, ver = case["op"], s["handle"]
    if op == "logprobs":
        ver.logprobs(logits=s["logits"], out_tokens=s["tokens"], cu_num_draft_tokens=s["cu"],
                     temperature=s["temperature"], num_top=case["top"], logprobs=s["logprobs"], ranks=s["ranks"],
                     entropy=s["entropy"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
        return {k: s[k] for k in ("logprobs", "ranks", "entropy", "top_ids", "top_logprobs")}
    cache = s["cache"]
    if op == "attend":
        ver.attend(q=s["q"], cache=cache, block_tables=s["table"], seq_lens=s["seq_lens"],
                   max_seq_len=s["max_seq_len"], max_spec_len=case["spec"], cu_num_draft_tokens=s["cu"],
                   shared_prefix_len=case["prefix"], scale=case["dim"] ** -0.5, out=s["out"], lse=s["lse"],
                   workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "store":
        ver.kv_write(cache=cache, key=s["key"], value=s["value"], slot_mapping=s["slots"])
    ver.kv_read(cache=cache, slot_mapping=s["slots"], key_out=s["key_out"], value_out=s["value_out"])
    return {"key": s["key_out"], "value": s["value_out"]}


def _places(s, case, positions):
    """(page, offset in it) of slots; -1 gives page 0."""
    p = positions.clamp_min(0)
    return p // case["block"], p % case["block"]


def _plain_write(s, case):
    # tokens whose slot was rolled back land on the last page, which no request uses
    keep = s["slots"] >= 0
    page, off = _places(s, case, s["slots"])
    page = torch.where(keep, page, torch.full_like(page, s["k"].shape[0] - 1))[:, None]
    head = torch.arange(case["kv_heads"], device=DEV)[None, :]
    for x, data, scale in ((s["key"], s["k"], s["ks"]), (s["value"], s["v"], s["vs"])):
        q, sc = _quantise(x.float(), case["fmt"])
        _bytes(data).index_put_((page, head, off[:, None]), _bytes(q))
        scale.index_put_((page, head, off[:, None]), sc)


def _plain_read(s, case):
    page, off = _places(s, case, s["slots"])
    keep = (s["slots"] >= 0)[:, None, None]

    def one(data, scale):
        x = _values(_bytes(data)[page, :, off], case["fmt"]) * scale[page, :, off][..., None]
        return torch.where(keep, x, torch.zeros_like(x)).to(s["key_out"].dtype)

    return {"key": one(s["k"], s["ks"]), "value": one(s["v"], s["vs"])}


def _padded_rows(s, n, spec, rows):
    """Rows [n, spec + 1] of flattened requests (clamped), and which of them are real."""
    col = torch.arange(spec + 1, device=DEV)
    if s["cu"] is None:
        at = torch.arange(n, device=DEV)[:, None] * (spec + 1) + col
        return at, torch.ones_like(at, dtype=torch.bool)
    cu = s["cu"].long()
    g = torch.diff(cu, prepend=cu.new_zeros(1))
    at = (cu - g + torch.arange(n, device=DEV))[:, None] + col
    return at.clamp_max(rows - 1), col <= g[:, None]


def _plain_attend(s, case):
    N, G, b, P = case["reqs"], case["spec"], case["block"], case["prefix"]
    h, d = case["kv_heads"], case["dim"]
    grp = case["q_heads"] // h
    rows = s["q"].shape[0]
    at, real = _padded_rows(s, N, G, rows)
    g1 = real.sum(1)
    q = s["q"][at].float().reshape(N, G + 1, h, grp, d)
    pos = s["seq_lens"].long()[:, None] - g1[:, None] + torch.arange(G + 1, device=DEV)

    def gather(data, scale, page, off):
        x = _values(_bytes(data)[page, :, off], case["fmt"])
        return x * scale[page, :, off][..., None]

    # private keys, padded to the longest request
    t = P + torch.arange(s["max_seq_len"] - P, device=DEV)
    live = t[None, :] < s["seq_lens"][:, None]
    page = s["table"].long()[:, (t // b).clamp_max(s["table"].shape[1] - 1)]
    off = (t % b).expand_as(page)
    k = gather(s["k"], s["ks"], page, off)
    score = torch.einsum("ntkgd,nskd->ntkgs", q, k) * d ** -0.5
    del k
    see = live[:, None, :] & (t <= pos[..., None])
    score = torch.where(see[:, :, None, None], score, -math.inf)
    if P:
        # the prefix's keys are the same for every request
        tp = torch.arange(P, device=DEV)
        pp, po = s["table"].long()[0, tp // b], tp % b
        kp = gather(s["k"], s["ks"], pp, po)
        sp = torch.einsum("ntkgd,skd->ntkgs", q, kp) * d ** -0.5
        sp = torch.where((tp <= pos[..., None])[:, :, None, None], sp, -math.inf)
        score = torch.cat([sp, score], -1)
        del sp, kp
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    del score
    total = w.sum(-1, keepdim=True)
    lse = torch.log(total)[..., 0] + torch.where(torch.isinf(top), torch.zeros_like(top), top)[..., 0]
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    v = gather(s["v"], s["vs"], page, off)
    o = torch.einsum("ntkgs,nskd->ntkgd", w[..., P:], v)
    del v
    if P:
        o = o + torch.einsum("ntkgs,skd->ntkgd", w[..., :P], gather(s["v"], s["vs"], pp, po))
    # back to flattened rows: padded rows go to a spare one behind the end
    to = torch.where(real, at, torch.full_like(at, rows)).reshape(-1)
    out = o.new_zeros(rows + 1, h * grp, d)
    out[to] = o.reshape(-1, h * grp, d)
    flat = lse.new_zeros(rows + 1, h * grp)
    flat[to] = lse.reshape(-1, h * grp)
    return {"out": out[:rows].to(torch.bfloat16), "lse": flat[:rows]}


def _plain_logprobs(s, case):
    N, G, V, K = case["reqs"], case["spec"], case["vocab"], case["top"]
    rows = s["logits"].shape[0]
    at, _ = _padded_rows(s, N, G, rows)
    tok = s["tokens"]
    keep = tok >= 0
    raw = s["logits"][at].float()
    x = raw if s["temperature"] is None else raw / s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    ent = lse[..., 0] - (e * x).sum(-1) / total[..., 0]
    del e
    ids = tok.clamp_min(0).long()[..., None]
    mine = x.gather(-1, ids)
    logp = (mine - lse)[..., 0]
    rank = 1 + (raw > raw.gather(-1, ids)).sum(-1).to(torch.int32)
    # one whole number per entry, ordered by value and, among equal values, by the lower index
    bits = (raw + 0.0).view(torch.int32).long()
    del raw
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    code = bits * (1 << 31) + ((1 << 31) - 1 - torch.arange(V, device=DEV))
    del bits
    best = code.topk(K, -1).values
    del code
    tid = (1 << 31) - 1 - best % (1 << 31)
    tlp = x.gather(-1, tid) - lse
    k3 = keep[..., None]
    return {"logprobs": torch.where(keep, logp, torch.zeros_like(logp)),
            "ranks": torch.where(keep, rank, torch.full_like(rank, -1)),
            "entropy": torch.where(keep, ent, torch.zeros_like(ent)),
            "top_ids": torch.where(k3, tid, torch.full_like(tid, -1)).to(torch.int32),
            "top_logprobs": torch.where(k3, tlp, torch.zeros_like(tlp))}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("store", "fetch"):
        n = case["tokens"] * case["kv_heads"] * 2
        elem = 2 if case["dtype"] == "bf16" else 4
        kept = 1.0 - case.get("rolled", 0) / 100.0
        cache = kept * n * (case["dim"] + 4)
        rows = n * case["dim"] * elem
        if op == "store":  # rows that are written, the cache written and read, rows out, slots twice
            return {"bytes": int(kept * rows + 2 * cache + rows + 16 * case["tokens"]),
                    "flops": int(5 * kept * n * case["dim"])}
        return {"bytes": int(cache + rows + 8 * case["tokens"]), "flops": int(n * case["dim"])}
    if op == "attend":
        gam, priv = _gammas(case), _owned(case)
        P, d, hq, h = case["prefix"], case["dim"], case["q_heads"], case["kv_heads"]
        rows = sum(gam) + len(gam)
        tokens = P + sum(priv)
        pairs = 0
        for g, n in zip(gam, priv):
            for j in range(g + 1):
                pairs += max(0, P + n - g + j)
        return {"bytes": tokens * h * (2 * d + 8) + rows * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    com = sum(_committed(case))
    elem = 2 if case["dtype"] == "bf16" else 4
    places = case["reqs"] * (case["spec"] + 1)
    return {"bytes": com * case["vocab"] * elem + places * (16 + 8 * case["top"]), "flops": 6 * com * case["vocab"]}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("store", "fetch"):
        return _exact_cache(s, case)
    if case["op"] == "attend":
        return _exact_attend(s, case)
    return _exact_logprobs(s, case)


def _exact_cache(s, case):
    slots, b, q = s["slots"], case["block"], QMAX[case["fmt"]]
    keep = slots >= 0
    out = {}
    for name, x, data, scale in (("key", s.get("key"), s["k"], s["ks"]), ("value", s.get("value"), s["v"], s["vs"])):
        y = torch.zeros(s["key_out"].shape, dtype=torch.float64, device=DEV)
        if case["op"] == "store":
            x64 = x[keep].double()
            step = (x64.abs().amax(-1, keepdim=True) / q).clamp_min(MIN_SCALE)
            z = x64 / step
            if case["fmt"] == "int8":
                z = torch.round(z)
            else:  # 4 significant bits, steps of 2^-9 below 2^-6
                exp = torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6)))
                grid = torch.exp2(exp - 3)
                z = torch.round(z / grid) * grid
            y[keep] = z * step
        else:
            page, off = slots // b, slots % b
            flat = data.permute(0, 2, 1, 3)[page, off] if data.dtype == torch.int8 else \
                data.view(torch.uint8).permute(0, 2, 1, 3)[page, off].view(torch.float8_e4m3fn)
            y = flat.double() * scale.permute(0, 2, 1)[page, off].double()[..., None]
        out[name] = y
    return out


def _exact_attend(s, case):
    gam, b = _gammas(case), case["block"]
    h, d = case["kv_heads"], case["dim"]
    grp = case["q_heads"] // h
    rows = s["q"].shape[0]
    out = torch.zeros(rows, h, grp, d, dtype=torch.float64, device=DEV)
    lse = torch.full((rows, h, grp), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for i, (g, L) in enumerate(zip(gam, s["seq_lens"].tolist())):
        if L > 0:
            t = torch.arange(L, device=DEV)
            page, off = s["table"][i].long()[t // b], t % b

            def side(data, scale):
                raw = (data if data.dtype == torch.int8 else data.view(torch.uint8)).permute(0, 2, 1, 3)[page, off]
                raw = raw if data.dtype == torch.int8 else raw.view(torch.float8_e4m3fn)
                x = raw.double() * scale.permute(0, 2, 1)[page, off].double()[..., None]
                return x.permute(1, 0, 2)  # [h, L, d]

            k, v = side(s["k"], s["ks"]), side(s["v"], s["vs"])
            qi = s["q"][at:at + g + 1].double().reshape(g + 1, h, grp, d).permute(1, 0, 2, 3).reshape(h, -1, d)
            a = torch.matmul(qi, k.transpose(1, 2)) / math.sqrt(d)
            pos = L - (g + 1) + torch.arange(g + 1, device=DEV).repeat_interleave(grp)
            a = a.masked_fill(t[None, :] > pos[:, None], -math.inf)
            z = torch.logsumexp(a, -1)
            p = torch.exp(a - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o = torch.matmul(p, v)
            out[at:at + g + 1] = o.reshape(h, g + 1, grp, d).permute(1, 0, 2, 3)
            lse[at:at + g + 1] = z.reshape(h, g + 1, grp).permute(1, 0, 2)
        at += g + 1
    return {"out": out.reshape(rows, h * grp, d), "lse": lse.reshape(rows, h * grp)}


def _exact_logprobs(s, case):
    N, G, K = case["reqs"], case["spec"], case["top"]
    gam, com = _gammas(case), _committed(case)
    logp = torch.zeros(N, G + 1, dtype=torch.float64, device=DEV)
    ent = torch.zeros(N, G + 1, dtype=torch.float64, device=DEV)
    tlp = torch.zeros(N, G + 1, K, dtype=torch.float64, device=DEV)
    first = 0
    for i in range(N):
        n = com[i]
        x = s["logits"][first:first + n].double()
        if s["temperature"] is not None:
            x = x / s["temperature"][i].double()
        lp = torch.log_softmax(x, -1)
        logp[i, :n] = lp.gather(1, s["tokens"][i, :n].long()[:, None])[:, 0]
        ent[i, :n] = -(lp.exp() * lp).sum(-1)
        tlp[i, :n] = lp.topk(K, -1).values
        first += gam[i] + 1
    return {"logprobs": logp, "ranks": None, "entropy": ent, "top_ids": None, "top_logprobs": tlp}
