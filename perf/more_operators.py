"""Cases of the operators that lead up to a verification step over a 4-bit cache:
block tables and slot maps built from request lengths, rotary positions (with
norms of queries and keys), the paged 4-bit KV cache written and read back, and
the verify tokens' attention over it.

With ``own`` false ``run`` computes an operator in plain torch operations (32
bits, angles in 64, rounded once at the end); with ``own`` true it calls this
package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"e2m1": 6.0, "int4": 7.0}
GROUP = 16  # elements that share an e4m3 scale
GROUP_MAX = 448.0
MIN_SCALE = 2.0 ** -64  # the cache's smallest row scale: a zero row still has a positive one
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _plan(name, reqs, least, most, fresh, past, block, pad, done, lens=1):
    return dict(name=name, op="plan", reqs=reqs, least=least, most=most, fresh=fresh, past=past, block=block, pad=pad,
                done=done, lens=lens)


def _rotate(name, tokens, q_heads, kv_heads, dim, rotary, pairs, norm, scaling, far, dtype, padded=0):
    return dict(name=name, op="rotate", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim, rotary=rotary,
                pairs=pairs, norm=norm, scaling=scaling, far=far, dtype=dtype, padded=padded)


def _store(name, tokens, kv_heads, dim, block, fmt, dtype, nhd=False, rolled=0):
    return dict(name=name, op="store", tokens=tokens, kv_heads=kv_heads, dim=dim, block=block, fmt=fmt, dtype=dtype,
                nhd=nhd, rolled=rolled)


def _fetch(name, tokens, kv_heads, dim, block, fmt, dtype, nhd=False):
    return dict(name=name, op="fetch", tokens=tokens, kv_heads=kv_heads, dim=dim, block=block, fmt=fmt, dtype=dtype,
                nhd=nhd)


def _attend(name, reqs, spec, ragged, prefix, least, most, q_heads, kv_heads, dim, block, fmt, nhd=False, lens=1):
    return dict(name=name, op="attend", reqs=reqs, spec=spec, ragged=ragged, prefix=prefix, least=least, most=most,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, block=block, fmt=fmt, nhd=nhd, lens=lens)


def listed():
    return [
        # the verify tokens of a small batch (4 requests, gamma 4): a call whose latency counts
        _plan("plan_step_small", 4, 5, 5, False, 1000, 16, 0, 0),
        # one step of the full batch (gamma 0..7), rows padded to a captured graph's size, a tenth of the requests done
        _plan("plan_step_full", 512, 1, 8, False, 16384, 16, 333, 10),
        # prompts that arrive together, nothing cached yet
        _plan("plan_prompts", 64, 300, 32768, True, 0, 32, 0, 0),
        # queries and keys of a small batch's verify tokens
        _rotate("rotate_small", 20, 32, 8, 128, 128, "half", False, "none", 8192, "bf16"),
        # the full batch with norms of each head, positions far beyond the trained length
        _rotate("rotate_norm_full", 4096, 32, 8, 128, 128, "half", True, "yarn", 1 << 20, "bf16", 5),
        # a long prompt, fp32 rows, half of each head rotated, neighbouring elements paired
        _rotate("rotate_prompt", 50001, 8, 2, 128, 64, "interleaved", False, "linear", 131072, "f32"),
        # one step of the full batch, a third of the slots rolled back to -1, written and read back
        _store("store4_step_full", 4096, 8, 128, 16, "e2m1", "bf16", rolled=33),
        # many requests' pages gathered back to bf16
        _fetch("fetch4_batch", 131072, 8, 128, 32, "int4", "bf16"),
        # one request, one token, a thousand cached tokens: the single-token form
        _attend("attend4_single", 1, 0, False, 0, 1000, 1000, 32, 8, 128, 16, "e2m1"),
        # 256 ragged requests (gamma 0..8) with long private histories and no common prefix
        _attend("attend4_private", 256, 8, True, 0, 0, 8192, 32, 8, 128, 16, "e2m1"),
        # few requests with very long contexts, eight query heads to a kv head, eight verify tokens
        _attend("attend4_long", 6, 7, False, 0, 60001, 131072, 64, 8, 128, 32, "int4"),
        # a system prompt shared by 64 requests that verify 4 drafts each
        _attend("attend4_shared", 64, 4, False, 8192, 5, 1024, 32, 8, 128, 16, "e2m1"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rotate", "store", "fetch", "attend", "attend", "attend"])
    fmt = rng.choice(["e2m1", "int4"])
    dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 24, 32, 64])
    nhd = rng.random() < 0.3
    lens = rng.randrange(1 << 20)
    if op == "plan":
        reqs = _spread(rng, 1, 2048)
        most = _spread(rng, 1, min(32768, (1 << 21) // reqs))
        c = _plan("", reqs, rng.choice([0, 1, most]), most, rng.random() < 0.3, _spread(rng, 1, 32768), block,
                  rng.choice([0, 0, 7, 500]), rng.choice([0, 0, 15]), lens)
    elif op == "rotate":
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 3, 4, 8])
        dim = rng.choice([64, 80, 128, 256])
        tokens = _spread(rng, 1, 50001 * 10 * 128 // ((q_heads + kv_heads) * dim))
        c = _rotate("", tokens, q_heads, kv_heads, dim, rng.choice([dim, dim, dim // 2, dim // 4]),
                    rng.choice(["half", "half", "interleaved"]), rng.random() < 0.5,
                    rng.choice(["none", "linear", "ntk", "yarn"]), _spread(rng, 1, 1 << 22),
                    rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 0, 20]))
    elif op in ("store", "fetch"):
        heads = rng.choice([1, 2, 3, 4, 8])
        tokens = min(131072, _spread(rng, 1, 131072 * 1024 // (heads * 128)))
        dtype = rng.choice(["bf16", "f32"])
        if op == "store":
            c = _store("", tokens, heads, dim, block, fmt, dtype, nhd, rng.choice([0, 20, 60]))
        else:
            c = _fetch("", tokens, heads, dim, block, fmt, dtype, nhd)
    else:
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8])
        spec = rng.choice([0, 1, 3, 4, 7])
        reqs = _spread(rng, 1, 256)
        prefix = block * rng.choice([0, 0, 0, _spread(rng, 1, 8192 // block)])
        rows = reqs * (spec + 1) * group * kv_heads
        most = _spread(rng, spec + 1, 131072)
        # keep the scores of a drawn case within those of the largest listed one
        most = max(spec + 1, min(most, (1 << 30) // (rows * 4), (1 << 20) // reqs))
        c = _attend("", reqs, spec, rng.random() < 0.5, prefix, rng.choice([0, min(most, spec + 1), most // 2]), most,
                    kv_heads * group, kv_heads, dim, block, fmt, nhd, lens)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# a case's lengths (the same for every seed)
# ----------------------------------------------------------------------------
def _plan_lengths(case):
    """(new tokens, computed tokens, pages held) of every request; -1 computed tokens: it is done, its rows are idle."""
    rng = random.Random(case["lens"])
    new, past, held = [], [], []
    for _ in range(case["reqs"]):
        new.append(_spread(rng, max(1, case["least"]), case["most"]) if case["least"] else rng.randint(0, case["most"]))
        past.append(0 if case["fresh"] else rng.randint(0, case["past"]))
        # (a step whose drafts were rejected may have left a page more than the tokens need)
        held.append(0 if case["fresh"] else -(-past[-1] // case["block"]) + (rng.random() < 0.2))
        if rng.random() * 100 < case["done"]:
            past[-1] = -1
    return new, past, held


def _gammas(case):
    rng = random.Random(case["lens"])
    if not case["ragged"]:
        return [case["spec"]] * case["reqs"]
    return [rng.randint(0, case["spec"]) for _ in range(case["reqs"])]


def _owned(case):
    """Private tokens of every request (0: an idle place of the batch); the verify tokens are among them."""
    rng = random.Random(case["lens"] + 2)
    out = []
    for g in _gammas(case):
        n = rng.randint(case["least"], case["most"])
        out.append(0 if n == 0 and case["prefix"] == 0 else max(n, g + 1))
    return out


def _scaling(case):
    """Arguments of the frequencies: what a model's configuration says."""
    return {"none": dict(base=10000.0), "linear": dict(base=10000.0, scaling="linear", factor=8.0),
            "ntk": dict(base=10000.0, scaling="ntk", factor=4.0),
            "yarn": dict(base=500000.0, scaling="yarn", factor=16.0, trained_len=32768)}[case["scaling"]]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _e2m1_code(z):
    """Codes 0 .. 7 of |z| rounded to the numbers of E2M1, ties to the even code."""
    a = z.abs().clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    v = (a / step).round() * step  # (a number that rounds up to the next range lies on both grids)
    return torch.where(v < 2, 2 * v, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)


def _quantise(x, fmt):
    """(bytes of two elements each, group scales, row scale) of x [..., D] in fp32."""
    top = x.abs().amax(-1)
    # (divisors on the device: true divisions, where a Python number would be multiplied by its reciprocal)
    scale = (top / top.new_full((), QMAX[fmt] * GROUP_MAX)).clamp_min(MIN_SCALE)
    y = x.unflatten(-1, (-1, GROUP))
    group = (y.abs().amax(-1) / (scale * QMAX[fmt])[..., None]).clamp_max(GROUP_MAX).to(torch.float8_e4m3fn)
    unit = (group.float() * scale[..., None])[..., None]
    z = torch.where(unit > 0, y / unit, torch.zeros_like(y)).flatten(-2)
    if fmt == "int4":
        code = z.round().clamp(-7, 7).to(torch.int8).view(torch.uint8) & 15
    else:
        code = _e2m1_code(z) | (z < 0).to(torch.uint8) << 3
    return code[..., 0::2] | code[..., 1::2] << 4, group, scale


def _numbers(raw, group, fmt):
    """fp32 numbers of gathered bytes [..., D/2] and group scales [..., D/16], without the row scale (exact)."""
    code = torch.stack([raw & 15, raw >> 4], -1).flatten(-2).long()
    if fmt == "int4":
        x = ((code ^ 8) - 8).float()
    else:
        x = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=raw.device)[code]
    return (x.unflatten(-1, (-1, GROUP)) * group.float()[..., None]).flatten(-2)


def _sides(s):
    return {"k": (s["k"], s["kg"], s["ks"]), "v": (s["v"], s["vg"], s["vs"])}


def _new_side(case, blocks):
    """(bytes, group scales, row scales) of one side [blocks, heads, block, ...], zeros; and its memory's order."""
    h, b, d = case["kv_heads"], case["block"], case["dim"]
    lead = (blocks, b, h) if case["nhd"] else (blocks, h, b)
    data = torch.zeros(*lead, d // 2, dtype=torch.uint8, device=DEV)
    group = torch.zeros(*lead, d // GROUP, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    return data, group, torch.ones(lead, device=DEV)


def _view(case, side):
    data, group, scale = side
    if case["nhd"]:
        return data.permute(0, 2, 1, 3), group.permute(0, 2, 1, 3), scale.permute(0, 2, 1)
    return side


def _fill(gen, case, blocks):
    side = data, group, scale = _new_side(case, blocks)
    # activations have a few channels that are larger than the rest
    chan = torch.exp(0.5 * _randn(gen, case["dim"]))
    step = max(1, (1 << 27) // (data[0].numel() * 2))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        q, g, sc = _quantise(_randn(gen, n, *data.shape[1:-1], case["dim"]) * chan, case["fmt"])
        data[i:i + n], scale[i:i + n] = q, sc
        group.view(torch.uint8)[i:i + n] = g.view(torch.uint8)
    return _view(case, side)


def _handle(reqs, spec):
    """The verifier handle that the program keeps (only the package's own calls use one)."""
    if not own:
        return None
    import speculative_decoding_token_rejection_gb300 as sv
    return sv.Verifier(reqs, spec, 1)


def _cache(s, case):
    """The package's description of the cache, kept beside the handle."""
    if not own:
        return None
    import speculative_decoding_token_rejection_gb300 as sv
    return sv.KVCache4(k=s["k"], v=s["v"], k_group=s["kg"], v_group=s["vg"], k_scale=s["ks"], v_scale=s["vs"],
                       format=case["fmt"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "plan":
        return _prepare_plan(s, case, gen)
    if op == "rotate":
        return _prepare_rotate(s, case, gen)
    if op == "attend":
        return _prepare_attend(s, case, gen)
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
        s["k"], s["kg"], s["ks"] = _view(case, _new_side(case, blocks))
        s["v"], s["vg"], s["vs"] = _view(case, _new_side(case, blocks))
    else:
        s["k"], s["kg"], s["ks"] = _fill(gen, case, blocks)
        s["v"], s["vg"], s["vs"] = _fill(gen, case, blocks)
    s["slots"] = slots
    s["key_out"] = torch.empty(T, h, d, dtype=dt, device=DEV)
    s["value_out"] = torch.empty(T, h, d, dtype=dt, device=DEV)
    s["handle"], s["cache"] = _handle(1, 0), _cache(s, case)
    return s


def _prepare_plan(s, case, gen):
    N, b = case["reqs"], case["block"]
    new, past, held = _plan_lengths(case)
    need = [-(-(p + n) // b) if p >= 0 else 0 for n, p in zip(new, past)]
    width = max(max(need), max(held), 1)
    spare = sum(max(0, a - h) for a, h in zip(need, held)) + 5
    blocks = sum(held) + spare
    order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=DEV)
    s["new"], s["past"], s["held"] = (torch.tensor(x, **i32) for x in (new, past, held))
    col = torch.arange(width, device=DEV)
    first = s["held"].long().cumsum(0) - s["held"]
    used = col < s["held"][:, None]
    s["table"] = torch.where(used, order[(first[:, None] + col).clamp_max(blocks - 1)], torch.full((), -1, **i32))
    # the free pages stand in a ring, from a place that differs from run to run
    at = torch.randint(0, 1 << 40, (1,), generator=gen, device=DEV)
    s["ring"] = torch.full((blocks,), -1, **i32)
    s["ring"][(at + torch.arange(spare, device=DEV)) % blocks] = order[blocks - spare:]
    s["range"] = torch.cat([at, at + spare])
    s["rows"] = sum(new) + case["pad"]
    s["positions"] = torch.empty(s["rows"], **i32)
    s["slots"] = torch.empty(s["rows"], dtype=torch.int64, device=DEV)
    s["seq_lens"], s["held_out"] = torch.empty(N, **i32), torch.empty(N, **i32)
    s["range_out"] = torch.empty(2, dtype=torch.int64, device=DEV)
    s["handle"], s["workspace"] = _handle(N, 0), None
    if own:
        s["workspace"] = s["handle"].plan_workspace(num_reqs=N)
    return s


def _prepare_rotate(s, case, gen):
    T, hq, h, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = (_randn(gen, T, hq + 2 * h, d) * torch.exp(0.5 * _randn(gen, d))).to(dt)
    s["q"], s["key"] = qkv[:, :hq], qkv[:, hq:hq + h]
    pos = torch.randint(0, case["far"], (T,), generator=gen, device=DEV).to(torch.int32)
    gone = torch.rand(T, generator=gen, device=DEV) * 100 < case["padded"]
    s["positions"] = torch.where(gone, torch.full_like(pos, -1), pos)
    s["q_weight"] = s["key_weight"] = None
    if case["norm"]:
        s["q_weight"] = (1 + 0.2 * _randn(gen, d)).to(dt)
        s["key_weight"] = (1 + 0.2 * _randn(gen, d)).to(dt)
    s["q_out"] = torch.zeros(T, hq, d, dtype=dt, device=DEV)
    s["key_out"] = torch.zeros(T, h, d, dtype=dt, device=DEV)
    s["handle"] = _handle(1, 0)
    if own:
        import speculative_decoding_token_rejection_gb300 as sv
        s["frequencies"] = sv.RotaryFrequencies(case["rotary"], device=DEV, **_scaling(case))
    else:
        inv, s["magnitude"] = _frequencies(case)
        s["inv"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
    return s


def _prepare_attend(s, case, gen):
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
    s["q"] = _randn(gen, rows, hq + 2 * h, d).to(torch.bfloat16)[:, :hq]
    s["k"], s["kg"], s["ks"] = _fill(gen, case, blocks)
    s["v"], s["vg"], s["vs"] = _fill(gen, case, blocks)
    s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(rows, hq, device=DEV)
    s["handle"], s["cache"] = _handle(N, case["spec"]), _cache(s, case)
    s["workspace"] = None
    if own:
        s["workspace"] = s["handle"].attend_workspace(cache=s["cache"], num_reqs=N, max_spec_len=case["spec"],
                                                      num_q_heads=hq, max_seq_len=s["max_seq_len"],
                                                      shared_prefix_len=case["prefix"], num_tokens=rows)
    return s


# ----------------------------------------------------------------------------
# a pass
# ----------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "plan":
        return _plain_plan(state, case)
    if case["op"] == "rotate":
        return _plain_rotate(state, case)
    if case["op"] == "attend":
        return _plain_attend(state, case)
    if case["op"] == "store":
        _plain_write(state, case)
    return _plain_read(state, case)


def _run_own(s, case):
    op, ver = case["op"], s["handle"]
    if op == "plan":
        ver.plan_step(num_new_tokens=s["new"], num_computed_tokens=s["past"], block_tables=s["table"],
                      held_pages=s["held"], free_pages=s["ring"], free_range=s["range"], block_size=case["block"],
                      num_rows=s["rows"], positions=s["positions"], slot_mapping=s["slots"], seq_lens=s["seq_lens"],
                      held_pages_out=s["held_out"], free_range_out=s["range_out"], workspace=s["workspace"])
        return _plan_outputs(s)
    if op == "rotate":
        ver.rotate(q=s["q"], key=s["key"], positions=s["positions"], frequencies=s["frequencies"],
                   interleaved=case["pairs"] == "interleaved", q_weight=s["q_weight"], key_weight=s["key_weight"],
                   eps=1e-6, q_out=s["q_out"], key_out=s["key_out"])
        return {"q": s["q_out"], "key": s["key_out"]}
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


def _plan_outputs(s):
    return {"positions": s["positions"], "slot_mapping": s["slots"], "seq_lens": s["seq_lens"],
            "held_pages": s["held_out"], "free_range": s["range_out"], "free_pages": s["ring"],
            "block_tables": s["table"]}


def _plain_plan(s, case):
    b, R = case["block"], s["rows"]
    n, past, held = s["new"].long(), s["past"].long(), s["held"].long()
    N, width = s["table"].shape
    done = past < 0
    last = n.cumsum(0)
    first = last - n
    # pages that are missing are taken from the ring's head, in the requests' order
    total = (past + n + b - 1) // b
    ok = ~done & (total <= width) & (last <= R)
    want = torch.where(ok, (total - held).clamp_min(0), torch.zeros_like(n))
    upto = want.cumsum(0)
    ok = ok & ((want == 0) | (upto <= s["range"][1] - s["range"][0]))
    take = torch.where(ok, want, torch.zeros_like(want))
    col = torch.arange(width, device=DEV)
    fresh = (col >= held[:, None]) & (col < (held + take)[:, None])
    at = (s["range"][0] + (upto - want - held)[:, None] + col) % s["ring"].numel()
    s["table"].copy_(torch.where(fresh, s["ring"][at], s["table"]))
    # pages of requests that are done go to its tail
    back = torch.where(done, held, torch.zeros_like(held))
    at = (s["range"][1] + (back.cumsum(0) - back)[:, None] + col) % s["ring"].numel()
    gone = col < back[:, None]
    spare = s["ring"].numel()
    ring = torch.cat([s["ring"], s["ring"].new_zeros(1)])
    ring[torch.where(gone, at, torch.full_like(at, spare))] = s["table"]
    s["ring"].copy_(ring[:spare])
    s["held_out"].copy_(torch.where(done, torch.zeros_like(held), held + take))
    s["range_out"].copy_(s["range"] + torch.stack([take.sum(), back.sum()]))
    s["seq_lens"].copy_(torch.where(ok, past + n, torch.zeros_like(n)))
    # every row's request, its position and slot
    row = torch.arange(R, device=DEV)
    i = torch.searchsorted(last, row, right=True)
    live = i < N
    i = i.clamp_max(N - 1)
    live = live & ok[i]
    pos = torch.where(live, past[i] + row - first[i], torch.full_like(row, -1))
    page = s["table"][i, pos.clamp_min(0) // b].long()
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, page * b + pos % b, torch.full_like(row, -1)))
    return _plan_outputs(s)


def _frequencies(case):
    """Radians per position of every pair, and the factor of the rotated elements."""
    a, d = _scaling(case), case["rotary"]
    base, factor = a["base"], a.get("factor", 1.0)
    if a.get("scaling") == "ntk":
        base *= factor ** (d / (d - 2))
    inv = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if a.get("scaling") == "linear":
        return [f / factor for f in inv], 1.0
    if a.get("scaling") != "yarn":
        return inv, 1.0

    # pairs that turn more than 32 times over the trained length are kept, those that turn less than once are stretched
    def pair_of(turns):
        return d * math.log(a["trained_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), d - 1)
    out = []
    for i, f in enumerate(inv):
        ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(f / factor * ramp + f * (1.0 - ramp))
    return out, 0.1 * math.log(factor) + 1.0


def _plain_rotate(s, case):
    keep = (s["positions"] >= 0)[:, None, None]
    angle = s["positions"].double()[:, None] * s["inv"]
    cos = (torch.cos(angle) * s["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * s["magnitude"]).float()[:, None]
    r = case["rotary"]

    def one(x, weight, out):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6) * weight.float()
        if case["pairs"] == "half":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out.copy_(torch.where(keep, torch.cat([turned, y[..., r:]], -1).to(out.dtype), out))
        return out

    return {"q": one(s["q"], s["q_weight"], s["q_out"]), "key": one(s["key"], s["key_weight"], s["key_out"])}


def _places(case, positions):
    """(page, offset in it) of slots; -1 gives page 0."""
    p = positions.clamp_min(0)
    return p // case["block"], p % case["block"]


def _plain_write(s, case):
    # tokens whose slot was rolled back land on the last page, which no request uses
    keep = s["slots"] >= 0
    page, off = _places(case, s["slots"])
    page = torch.where(keep, page, torch.full_like(page, s["k"].shape[0] - 1))[:, None]
    at = (page, torch.arange(case["kv_heads"], device=DEV)[None, :], off[:, None])
    for x, (data, group, scale) in zip((s["key"], s["value"]), _sides(s).values()):
        q, g, sc = _quantise(x.float(), case["fmt"])
        data.index_put_(at, q)
        group.view(torch.uint8).index_put_(at, g.view(torch.uint8))
        scale.index_put_(at, sc)


def _gather(side, case, page, off):
    """fp32 values [..., heads, D] of gathered cache rows."""
    data, group, scale = side
    x = _numbers(data[page, :, off], group.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn), case["fmt"])
    return x * scale[page, :, off][..., None]


def _plain_read(s, case):
    page, off = _places(case, s["slots"])
    keep = (s["slots"] >= 0)[:, None, None]

    def one(side):
        x = _gather(side, case, page, off)
        return torch.where(keep, x, torch.zeros_like(x)).to(s["key_out"].dtype)

    sides = _sides(s)
    return {"key": one(sides["k"]), "value": one(sides["v"])}


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
    sides = _sides(s)
    at, real = _padded_rows(s, N, G, rows)
    g1 = real.sum(1)
    q = s["q"][at].float().reshape(N, G + 1, h, grp, d)
    pos = s["seq_lens"].long()[:, None] - g1[:, None] + torch.arange(G + 1, device=DEV)

    # private keys, padded to the longest request
    t = P + torch.arange(s["max_seq_len"] - P, device=DEV)
    live = t[None, :] < s["seq_lens"][:, None]
    page = s["table"].long()[:, (t // b).clamp_max(s["table"].shape[1] - 1)]
    off = (t % b).expand_as(page)

    def private(side):  # (a request at a time: the gathered bytes' whole numbers are wide)
        x = torch.empty(*page.shape, h, d, device=DEV)
        for i in range(N):
            x[i] = _gather(side, case, page[i], off[i])
        return x

    k = private(sides["k"])
    score = torch.einsum("ntkgd,nskd->ntkgs", q, k) * d ** -0.5
    del k
    see = live[:, None, :] & (t <= pos[..., None])
    score = torch.where(see[:, :, None, None], score, -math.inf)
    if P:
        # the prefix's keys are the same for every request
        tp = torch.arange(P, device=DEV)
        pp, po = s["table"].long()[0, tp // b], tp % b
        sp = torch.einsum("ntkgd,skd->ntkgs", q, _gather(sides["k"], case, pp, po)) * d ** -0.5
        sp = torch.where((tp <= pos[..., None])[:, :, None, None], sp, -math.inf)
        score = torch.cat([sp, score], -1)
        del sp
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    del score
    total = w.sum(-1, keepdim=True)
    lse = torch.log(total)[..., 0] + torch.where(torch.isinf(top), torch.zeros_like(top), top)[..., 0]
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    o = torch.einsum("ntkgs,nskd->ntkgd", w[..., P:], private(sides["v"]))
    if P:
        o = o + torch.einsum("ntkgs,skd->ntkgd", w[..., :P], _gather(sides["v"], case, pp, po))
    # back to flattened rows: padded rows go to a spare one behind the end
    to = torch.where(real, at, torch.full_like(at, rows)).reshape(-1)
    out = o.new_zeros(rows + 1, h * grp, d)
    out[to] = o.reshape(-1, h * grp, d)
    flat = lse.new_zeros(rows + 1, h * grp)
    flat[to] = lse.reshape(-1, h * grp)
    return {"out": out[:rows].to(torch.bfloat16), "lse": flat[:rows]}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        new, past, held = _plan_lengths(case)
        rows = sum(new)
        moved = touched = 0
        for n, p, h in zip(new, past, held):
            need = -(-(p + n) // case["block"])
            moved += h if p < 0 else max(0, need - h)
            touched += 0 if n == 0 or p < 0 else need - p // case["block"]  # pages that rows lie in
        return {"bytes": 12 * (rows + case["pad"]) + 8 * moved + 4 * touched + 20 * case["reqs"] + 32,
                "flops": 4 * (rows + case["pad"])}
    if op == "rotate":
        heads = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        elem = 2 if case["dtype"] == "bf16" else 4
        kept = 1.0 - case["padded"] / 100.0
        return {"bytes": int(kept * heads * case["dim"] * 2 * elem) + 4 * case["tokens"] + 4 * case["rotary"],
                "flops": int(kept * heads * (3 * case["rotary"] + (4 * case["dim"] if case["norm"] else 0)))}
    if op in ("store", "fetch"):
        n = case["tokens"] * case["kv_heads"] * 2
        elem = 2 if case["dtype"] == "bf16" else 4
        kept = 1.0 - case.get("rolled", 0) / 100.0
        cache = kept * n * (case["dim"] // 2 + case["dim"] // GROUP + 4)
        rows = n * case["dim"] * elem
        if op == "store":  # rows that are written, the cache written and read, rows out, slots twice
            return {"bytes": int(kept * rows + 2 * cache + rows + 16 * case["tokens"]),
                    "flops": int(6 * kept * n * case["dim"])}
        return {"bytes": int(cache + rows + 8 * case["tokens"]), "flops": int(2 * n * case["dim"])}
    gam, priv = _gammas(case), _owned(case)
    P, d, hq, h = case["prefix"], case["dim"], case["q_heads"], case["kv_heads"]
    rows = sum(gam) + len(gam)
    tokens = P + sum(priv)
    pairs = 0
    for g, n in zip(gam, priv):
        for j in range(g + 1):
            pairs += max(0, P + n - g + j)
    return {"bytes": tokens * h * (d + 2 * (d // GROUP) + 8) + rows * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s, case)
    if case["op"] == "rotate":
        return _exact_rotate(s, case)
    if case["op"] == "attend":
        return _exact_attend(s, case)
    return _exact_cache(s, case)


def _exact_plan(s, case):
    """A request at a time, as a scheduler on the host keeps its books."""
    b = case["block"]
    new, past, held = (s[k].tolist() for k in ("new", "past", "held"))
    table, ring = s["table"].cpu(), s["ring"].tolist()
    head, tail = s["range"].tolist()
    begin, end = head, tail
    R, C = s["rows"], len(ring)
    positions, slots = torch.full((R,), -1, dtype=torch.int32), torch.full((R,), -1, dtype=torch.int64)
    seq, kept = [], []
    row = wanted = 0
    for i, (n, p, h) in enumerate(zip(new, past, held)):
        if p < 0:
            for x in table[i, :h].tolist():
                ring[end % C] = x
                end += 1
            seq.append(0)
            kept.append(0)
            row += n
            continue
        need = -(-(p + n) // b)
        good = need <= table.shape[1] and row + n <= R
        if good and need > h:
            wanted += need - h
            good = wanted <= tail - head
        if good and need > h:
            table[i, h:need] = torch.tensor([ring[(begin + x) % C] for x in range(need - h)], dtype=torch.int32)
            begin += need - h
            h = need
        if good:
            t = torch.arange(p, p + n)
            positions[row:row + n] = t.to(torch.int32)
            slots[row:row + n] = table[i, t // b].long() * b + t % b
        seq.append(p + n if good else 0)
        kept.append(h)
        row += n
    i32 = dict(dtype=torch.int32, device=DEV)
    return {"positions": positions.to(DEV), "slot_mapping": slots.to(DEV), "seq_lens": torch.tensor(seq, **i32),
            "held_pages": torch.tensor(kept, **i32), "free_range": torch.tensor([begin, end], device=DEV),
            "free_pages": torch.tensor(ring, **i32), "block_tables": table.to(DEV)}


def _exact_rotate(s, case):
    inv, magnitude = _frequencies(case)
    pos = s["positions"].double()
    live = pos >= 0
    out = {}
    for name, x, weight in (("q", s["q"], s["q_weight"]), ("key", s["key"], s["key_weight"])):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.double()
        z = y.clone()
        for i, f in enumerate(inv):
            a, b = (i, i + case["rotary"] // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
            turn = torch.polar(torch.full_like(pos, magnitude), pos * f)[:, None] * torch.complex(y[..., a], y[..., b])
            z[..., a], z[..., b] = turn.real, turn.imag
        out[name] = torch.where(live[:, None, None], z, torch.zeros_like(z))
    return out


def _exact_values(side, case, page, off):
    """Values [tokens, heads, D] of cache rows in 64 bits, looked up code by code."""
    data, group, scale = side
    pairs = data[page, :, off].to(torch.int16)
    code = torch.zeros(*pairs.shape[:-1], case["dim"], dtype=torch.int16, device=DEV)
    code[..., 0::2], code[..., 1::2] = pairs % 16, pairs // 16
    if case["fmt"] == "int4":
        x = torch.where(code > 7, code - 16, code).double()
    else:
        size = code % 8  # exponent and one bit of mantissa; the smallest numbers have no leading one
        e, m = (size // 2).double(), (size % 2).double()
        x = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2) * torch.where(code > 7, -1.0, 1.0)
    g = group.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).double()
    return x * g.repeat_interleave(GROUP, -1) * scale[page, :, off].double()[..., None]


def _exact_cache(s, case):
    slots, b, q = s["slots"], case["block"], QMAX[case["fmt"]]
    keep = slots >= 0
    out = {}
    for name, x, side in zip(("key", "value"), (s.get("key"), s.get("value")), _sides(s).values()):
        y = torch.zeros(s["key_out"].shape, dtype=torch.float64, device=DEV)
        if case["op"] == "fetch":
            y[keep] = _exact_values(side, case, slots[keep] // b, slots[keep] % b)
        else:
            # the scales and the quotients are fp32 numbers by definition
            x64 = x[keep].double()
            row = (x64.abs().amax(-1) / (q * 448)).float().double().clamp_min(MIN_SCALE)[..., None]
            parts = []
            for i in range(0, case["dim"], GROUP):
                part = x64[..., i:i + GROUP]
                want = (part.abs().amax(-1, keepdim=True) / (q * row).float().double()).float().double()
                grid = torch.exp2(torch.floor(torch.log2(want.clamp_min(2.0 ** -6))) - 3)  # 4 significant bits
                g = (torch.round(want / grid) * grid).clamp_max(448.0)
                z = (part / (g * row).float().double().clamp_min(1e-300)).float().double() * (g > 0)
                if case["fmt"] == "int4":
                    z = torch.round(z)
                else:  # 2 significant bits, steps of 1/2 below 1
                    grid = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(1.0))) - 1)
                    z = torch.round(z / grid) * grid
                parts.append(z.clamp(-q, q) * g * row)
            y[keep] = torch.cat(parts, -1)
        out[name] = y
    return out


def _exact_attend(s, case):
    gam, b = _gammas(case), case["block"]
    h, d = case["kv_heads"], case["dim"]
    grp = case["q_heads"] // h
    rows = s["q"].shape[0]
    out = torch.zeros(rows, h, grp, d, dtype=torch.float64, device=DEV)
    lse = torch.full((rows, h, grp), -math.inf, dtype=torch.float64, device=DEV)
    sides = _sides(s)
    at = 0
    for i, (g, L) in enumerate(zip(gam, s["seq_lens"].tolist())):
        if L > 0:
            t = torch.arange(L, device=DEV)
            page, off = s["table"][i].long()[t // b], t % b
            k, v = (_exact_values(sides[x], case, page, off).permute(1, 0, 2) for x in "kv")
            qi = s["q"][at:at + g + 1].double().reshape(g + 1, h, grp, d).permute(1, 0, 2, 3).reshape(h, -1, d)
            a = torch.matmul(qi, k.transpose(1, 2)) / math.sqrt(d)
            pos = L - (g + 1) + torch.arange(g + 1, device=DEV).repeat_interleave(grp)
            a = a.masked_fill(t[None, :] > pos[:, None], -math.inf)
            z = torch.logsumexp(a, -1)
            p = torch.exp(a - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            out[at:at + g + 1] = torch.matmul(p, v).reshape(h, g + 1, grp, d).permute(1, 0, 2, 3)
            lse[at:at + g + 1] = z.reshape(h, g + 1, grp).permute(1, 0, 2)
        at += g + 1
    return {"out": out.reshape(rows, h * grp, d), "lse": lse.reshape(rows, h * grp)}
