"""A step's calls one after another, as a server makes them: pages, positions and
slots from plan_step, queries and keys through rotate, keys and values through
the 4-bit cache, attention over it -- each compared with what the books and the
formulas make of the outputs of the one before it."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
import test_gpu_attend4 as attend4
import test_gpu_kv4_cache as cache4
import test_gpu_plan as plan
import test_gpu_rotate as rotate
from test_gpu_example import example

pytestmark = pytest.mark.gpu


class Server:
    """N requests' device state, and one step of it."""

    def __init__(self, N, heads, group, dim, block, width, fmt, seed, shared=0):
        self.shared = shared  # pages of a prefix at the head of every table
        self.N, self.heads, self.group, self.dim, self.block, self.width = N, heads, group, dim, block, width
        self.ver = sv.Verifier(N, 63, 8)
        self.cache = cache4.make_cache4(N * width, heads, block, dim, fmt)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tables, self.held = torch.zeros(N, width, **i32), torch.zeros(N, **i32)
        gen = torch.Generator().manual_seed(seed)
        pages = torch.randperm(N * width, generator=gen).to(torch.int32).cuda()
        self.free = pages[shared:].contiguous()
        self.tables[:, :shared] = pages[:shared]
        self.held += shared
        self.span = torch.tensor([0, N * width - shared], device="cuda")
        self.computed = torch.zeros(N, **i32)
        if shared:
            rows = torch.randn(2, shared * block, heads, dim, generator=gen).cuda()
            slots = (pages[:shared, None].long() * block + torch.arange(block, device="cuda")).flatten()
            self.ver.kv_write(cache=self.cache, key=rows[0], value=rows[1], slot_mapping=slots)
        self.new = torch.zeros(N, **i32)
        self.status = torch.zeros(1, **i32)
        self.frequencies = sv.RotaryFrequencies(dim, scaling="yarn", factor=4.0, trained_len=64)
        self.norms = (1 + 0.3 * torch.randn(2, dim, generator=gen)).cuda().to(torch.bfloat16)

    def step(self, qkv, rows, most, cu, stream=None):
        """(plan, rotated queries, rotated keys, values, attention)."""
        hq = self.heads * self.group
        q, key, value = qkv[:, :hq], qkv[:, hq:hq + self.heads], qkv[:, hq + self.heads:]
        p = self.ver.plan_step(num_new_tokens=self.new, num_computed_tokens=self.computed, block_tables=self.tables,
                               held_pages=self.held, free_pages=self.free, free_range=self.span, num_rows=rows,
                               block_size=self.block, num_shared_pages=self.shared, cu_num_draft_tokens=cu,
                               status=self.status, stream=stream)
        q, key = self.ver.rotate(q=q, key=key, positions=p.positions, frequencies=self.frequencies, q_weight=self.norms[0],
                                 key_weight=self.norms[1], stream=stream)
        self.ver.kv_write(cache=self.cache, key=key, value=value, slot_mapping=p.slot_mapping, status=self.status,
                          stream=stream)
        out = self.ver.attend(q=q, cache=self.cache, block_tables=self.tables, seq_lens=p.seq_lens,
                              max_seq_len=self.width * self.block, max_spec_len=most, scale=self.dim ** -0.5,
                              shared_prefix_len=self.shared * self.block, cu_num_draft_tokens=cu, status=self.status,
                              stream=stream)
        return p, q, key, value, out


@pytest.mark.parametrize("kw", [dict(N=5, heads=2, group=4, dim=128, block=16, width=12, fmt="e2m1"),
                                dict(N=40, heads=1, group=3, dim=64, block=7, width=20, fmt="int4"),
                                dict(N=30, heads=2, group=2, dim=64, block=64, width=260, fmt="e2m1", shared=257)])
def test_steps_against_books_and_formulas(kw):
    """Prompts, verify steps, rollbacks, a request that ends and one that takes its place."""
    s = Server(seed=1, **kw)
    N, block = s.N, s.block
    gen = torch.Generator().manual_seed(2)
    begin = s.shared * block
    new, past = torch.randint(1, 60, (N,), generator=gen).tolist(), [begin] * N
    for step in range(5):
        rows, most = sum(new), max(new) - 1
        s.new.copy_(torch.tensor(new))
        s.computed.copy_(torch.tensor(past))
        want, bits = plan.books(dict(new=new, past=past, held=s.held.tolist(), block=block, table=s.tables.cpu(),
                                     ring=s.free.tolist(), range=s.span.tolist(), rows=rows, shared=s.shared))
        assert bits == 0
        qkv = (2 * torch.randn(rows, s.heads * (s.group + 2), s.dim, generator=gen)).cuda().to(torch.bfloat16)
        given = qkv.clone()
        cu = torch.zeros(N, dtype=torch.int32, device="cuda")
        p, q, key, value, out = s.step(qkv, rows, most, cu)
        assert int(s.status.item()) == 0
        # the books
        for name, got in (("positions", p.positions), ("slots", p.slot_mapping), ("table", s.tables)):
            assert torch.equal(got.cpu(), want[name]), name
        assert (p.seq_lens.tolist(), s.held.tolist(), s.span.tolist(), s.free.tolist(), cu.tolist()) == (
            want["seq"], want["kept"], want["range"], want["ring"], want["cu"])
        # positions
        hq = s.heads * s.group
        rotate.check(q, given[:, :hq], p.positions, s.frequencies, s.norms[0])
        rotate.check(key, given[:, hq:hq + s.heads], p.positions, s.frequencies, s.norms[1])
        # the cache holds what those rows are quantised to
        live = p.slot_mapping >= 0
        read = s.ver.kv_read(cache=s.cache, slot_mapping=p.slot_mapping[live], dtype=torch.float32)
        for x, got in zip((key, value), read):
            codes, group, scale = cache4.quantise4(x[live].float(), kw["fmt"])
            assert torch.equal(got.cpu(), cache4.values4(codes, group, scale, kw["fmt"]))
        # attention over it
        ref, _, tol, _ = attend4.reference(dict(cache=s.cache, group=s.group, q=q, gammas=[n - 1 for n in new],
                                                lens=want["seq"], table=s.tables, scale=s.dim ** -0.5))
        assert bool(((out.double() - ref).abs() <= tol).all())
        # drafts are rejected, a request ends, another begins
        for i in range(N):
            if past[i] < 0:
                past[i], new[i] = begin, 1 + (7 * i + step) % 30
            else:
                past[i] = want["seq"][i] - (int(torch.randint(0, 4, (1,), generator=gen)) % new[i] if step else 0)
                new[i] = 1 + int(torch.randint(0, 6, (1,), generator=gen))
                if (i + step) % 5 == 0:
                    past[i], new[i] = -1, 1
    s.ver.close()


def test_a_captured_step_goes_on():
    """A whole step in one graph, replayed: the same as calls on a stream of their own."""
    kw = dict(N=6, heads=2, group=4, dim=64, block=8, width=10, fmt="e2m1", seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    inputs = torch.randn(6, 30, 12, 64, generator=gen, device="cuda").to(torch.bfloat16)
    cu = torch.arange(1, 7, device="cuda", dtype=torch.int32) * 4
    wants, side = [], torch.cuda.Stream()
    a = Server(**kw)
    a.new.fill_(5)
    side.wait_stream(torch.cuda.current_stream())
    for x in inputs:
        x = x.clone()
        torch.cuda.synchronize()
        p, *_, out = a.step(x, 30, 4, cu.clone(), stream=side)
        side.synchronize()
        wants.append(out.clone())
        a.computed.copy_(p.seq_lens)
    b = Server(**kw)
    b.new.fill_(5)
    x, got_cu, graph = inputs[0].clone(), cu.clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        p, *_, out = b.step(x, 30, 4, got_cu)
        b.computed.copy_(p.seq_lens)
    for given, want in zip(inputs, wants):
        x.copy_(given)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(got_cu, cu)
    assert b.computed.tolist() == [30] * 6 and int(b.status.item()) == int(a.status.item()) == 0
    a.ver.close()
    b.ver.close()


@pytest.mark.parametrize("kw", [dict(), dict(places=20, requests=50, gamma=4, prompt=200, dim=128, block=32, fmt="int4",
                                             q_heads=16, kv_heads=4, new_tokens=30)])
def test_the_example_serves_everyone(kw):
    serve = example().serve
    texts, held, (head, tail), free = result = serve(say=lambda line: None, **kw)
    least, surplus = kw.get("new_tokens", 20), kw.get("gamma", 3)
    assert len(texts) == kw.get("requests", 10) and all(least <= len(t) <= least + surplus for t in texts)
    # every page is back, once
    assert held == [0] * kw.get("places", 4) and tail - head == len(free)
    assert sorted(free[x % len(free)] for x in range(head, tail)) == list(range(len(free)))
    assert serve(say=lambda line: None, **kw) == result
