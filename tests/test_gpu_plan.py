"""Block tables, positions and slots of a step against a scheduler's books kept
on the host, a request at a time: whole numbers, equal to the last one."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv

pytestmark = pytest.mark.gpu

BITS = sv.DATA_STATUS_BITS


@pytest.fixture(scope="module")
def ver():
    v = sv.Verifier(1 << 17, 8, 8)
    yield v
    v.close()


def books(c):
    """(outputs, status) of a state dict of lists and CPU tensors."""
    b, R, C = c["block"], c["rows"], len(c["ring"])
    table, ring = c["table"].clone(), list(c["ring"])
    width, shared = table.shape[1], c.get("shared", 0)
    head, tail = c["range"]
    pool = head >= 0 and head <= tail and tail - head <= C
    status = 0 if pool else BITS["BAD_PARAM"]
    begin, end = head, tail
    positions, slots = torch.full((R,), -1, dtype=torch.int32), torch.full((R,), -1, dtype=torch.int64)
    seq, kept, cu = [], [], []
    row = wanted = 0
    for i, (n, p, h) in enumerate(zip(c["new"], c["past"], c["held"])):
        good = p >= 0
        if n < 0 or not 0 <= h <= width:
            good = False
            status |= BITS["BAD_PARAM"]
        n = max(n, 0)
        row += n
        cu.append(min(row - (i + 1), 2 ** 31 - 1))
        need = -(-(p + n) // b)
        if good and (need > width or p + n > 2 ** 31 - 1 or h * b < p or h < shared):
            good = False
            status |= BITS["BAD_PARAM"]
        if good and row > R:
            good = False
            status |= BITS["BAD_CU"]
        if good and need > h:
            wanted += need - h
            if not pool or wanted > tail - head:
                good = False
                status |= BITS["NO_PAGES"]
        if p < 0 and pool and shared < h <= width:
            for x in table[i, shared:h].tolist():
                ring[end % C] = x
                end += 1
            h = shared
        if good and need > h:
            table[i, h:need] = torch.tensor([c["ring"][(begin + x) % C] for x in range(need - h)], dtype=torch.int32)
            begin += need - h
            h = need
        if good and n:
            t = torch.arange(p, p + n)
            positions[row - n:row] = t.to(torch.int32)
            slots[row - n:row] = table[i, t // b].long() * b + t % b
        seq.append(p + n if good else 0)
        kept.append(h)
    return dict(positions=positions, slots=slots, seq=seq, kept=kept, range=[begin, end], ring=ring, table=table,
                cu=cu), status


def state(new, past, *, block=16, held=None, spare=50, at=0, pad=0, rows=None, width=None, seed=0, capacity=None):
    gen = torch.Generator().manual_seed(seed)
    held = [-(-max(p, 0) // block) for p in past] if held is None else held
    need = [-(-(max(p, 0) + max(n, 0)) // block) for n, p in zip(new, past)]
    width = max(need + held + [1]) if width is None else width
    total = sum(max(h, 0) for h in held) + spare
    capacity = total if capacity is None else capacity
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    x = 0
    for i, h in enumerate(held):
        h = min(max(h, 0), width)
        table[i, :h] = order[x:x + h]
        x += h
    ring = torch.full((capacity,), -1, dtype=torch.int32)
    for k in range(spare):
        ring[(at + k) % capacity] = order[total - spare + k]
    rows = sum(max(n, 0) for n in new) + pad if rows is None else rows
    return dict(new=new, past=past, held=held, block=block, table=table, ring=ring.tolist(), range=[at, at + spare],
                rows=rows)


def call(ver, c, in_place=False, stream=None, wide=0):
    """The kernels on the state; outputs like books'."""
    t32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    N = len(c["new"])
    full = torch.full((N, c["table"].shape[1] + wide), -9, dtype=torch.int32, device="cuda")
    table = full[:, :c["table"].shape[1]]
    table.copy_(c["table"])
    new, past, held, ring = t32(c["new"]), t32(c["past"]), t32(c["held"]), t32(c["ring"])
    span = torch.tensor(c["range"], device="cuda")
    outs = {} if in_place else dict(held_pages_out=torch.full_like(held, 77), free_range_out=torch.zeros_like(span))
    if in_place:
        outs["seq_lens"] = past
    cu, status = torch.full_like(held, 77), torch.zeros(1, dtype=torch.int32, device="cuda")
    positions = torch.full((c["rows"],), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((c["rows"],), 77, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    if "shared" in c:
        outs["num_shared_pages"] = c["shared"]
    r = ver.plan_step(num_new_tokens=new, num_computed_tokens=past, block_tables=table, held_pages=held,
                      free_pages=ring, free_range=span, block_size=c["block"], num_rows=c["rows"], positions=positions,
                      slot_mapping=slots, cu_num_draft_tokens=cu, status=status, stream=stream, **outs)
    torch.cuda.synchronize()
    assert wide == 0 or bool((full[:, c["table"].shape[1]:] == -9).all())
    if not in_place:
        assert held.tolist() == c["held"] and span.tolist() == c["range"] and past.tolist() == c["past"]
    return dict(positions=positions.cpu(), slots=slots.cpu(), seq=r.seq_lens.tolist(), kept=r.held_pages.tolist(),
                range=r.free_range.tolist(), ring=ring.tolist(), table=table.cpu(), cu=cu.tolist()), int(status)


def check(ver, c, status=0, **kw):
    want, bits = books(c)
    got, got_bits = call(ver, c, **kw)
    assert bits == status and got_bits == status
    for name, x in want.items():
        assert torch.equal(got[name], x) if isinstance(x, torch.Tensor) else got[name] == x, name
    return got


def rand(seed, N, most, past, done=0.1):
    gen = torch.Generator().manual_seed(seed)
    new = torch.randint(0, most + 1, (N,), generator=gen).tolist()
    old = torch.randint(0, past + 1, (N,), generator=gen).tolist()
    gone = (torch.rand(N, generator=gen) < done).tolist()
    held_extra = torch.randint(0, 2, (N,), generator=gen).tolist()
    return new, [-1 if g else p for p, g in zip(old, gone)], old, held_extra


@pytest.mark.parametrize("N,most,past,block", [(1, 1, 0, 16), (1, 5, 1000, 16), (3, 40, 100, 1), (33, 8, 700, 7),
                                               (512, 8, 3000, 16), (1024, 3, 50, 16), (1025, 9, 333, 24),
                                               (2500, 2, 90, 32), (7, 9000, 100, 16), (64, 3000, 0, 32),
                                               (5000, 8, 200, 64)])
def test_against_the_books(ver, N, most, past, block):
    new, computed, old, extra = rand(N + block, N, most, past)
    held = [-(-p // block) + e for p, e in zip(old, extra)]
    spare = sum(max(0, -(-(p + n) // block) - h) for n, p, h in zip(new, old, held)) + 3
    c = state(new, computed, block=block, held=held, spare=spare, at=(1 << 40) + 12345, pad=N % 5, seed=N)
    check(ver, c)
    check(ver, c, in_place=True, wide=3)


@pytest.mark.parametrize("pad", [0, 1, 4095, 20000])
def test_idle_rows_behind_the_last_request(ver, pad):
    check(ver, state([3, 0, 5], [14, 30, -1], pad=pad))
    check(ver, state([0, 0], [0, 16], pad=pad))


def test_no_requests_and_no_rows(ver):
    check(ver, state([], [], pad=5))
    check(ver, state([], [], pad=5000))
    check(ver, state([0, 0], [5, -1]))
    check(ver, state([], []))


def test_everyone_is_done(ver):
    check(ver, state([1] * 40, [-1] * 40, held=[i for i in range(40)], spare=2, at=7, pad=3))


def test_pages_run_out(ver):
    """Requests are served in order; one that wants nothing is not refused."""
    c = state([20, 40, 1, 20, 16], [16, 0, 3, 0, 0], spare=4, pad=2)
    got = check(ver, c, BITS["NO_PAGES"])  # wants 2, 3, 0, 2, 1 of 4
    assert got["seq"] == [36, 0, 4, 0, 0]
    check(ver, state([20] * 2000, [0] * 2000, spare=1001), BITS["NO_PAGES"])
    check(ver, state([20], [0], spare=0, capacity=3), BITS["NO_PAGES"])


def test_the_last_free_page(ver):
    got = check(ver, state([16, 16], [0, 16], spare=2, at=5))
    assert got["range"] == [7, 7]


def test_rows_that_do_not_fit(ver):
    for rows in (0, 1, 9, 10, 11):
        check(ver, state([4, 6, 0, 3], [0, 5, 2, 1], rows=rows), BITS["BAD_CU"])


def test_bad_requests_take_nothing(ver):
    bad = BITS["BAD_PARAM"]
    check(ver, state([4, -3, 5], [0, 20, 3]), bad)
    check(ver, state([4, 3, 5], [0, 20, 3], held=[0, 1, 1]), bad)  # fewer pages than its computed tokens fill
    check(ver, state([4, 3, 5], [0, 20, 3], held=[0, -1, 1]), bad)
    check(ver, state([4, 3, 5], [0, 20, 3], held=[0, 9, 1], width=5), bad)
    check(ver, state([4, 300, 5], [0, 20, 3], width=5), bad)
    # (its rows count: those of the one behind it do not fit)
    check(ver, state([4, 2 ** 31 - 1, 5], [0, 20, 3], width=5, rows=20), bad | BITS["BAD_CU"])
    check(ver, state([4, 1, 5], [0, -1, 3], held=[0, -4, 1]), bad)


@pytest.mark.parametrize("span", [[-1, 4], [5, 4], [0, 51]])
def test_a_bad_range_gives_and_takes_nothing(ver, span):
    c = state([4, 3, 5, 1], [0, 20, 3, -1], held=[0, 2, 1, 3], capacity=50, spare=44)
    c["range"] = span
    got, status = call(ver, c)
    assert status & BITS["BAD_PARAM"] and got["kept"] == c["held"] and got["range"] == span
    assert got["ring"] == c["ring"] and torch.equal(got["table"], c["table"])
    assert got["seq"] == [0, 23, 8, 0]


def test_steps_follow_one_another(ver):
    """Verify steps with rollbacks and finished requests, the outputs of one the inputs of the next; no page is ever lost
    or held twice."""
    gen = torch.Generator().manual_seed(5)
    N, block, blocks, width = 40, 8, 400, 30
    c = dict(new=[20] * N, past=[0] * N, held=[0] * N, block=block, table=torch.full((N, width), -1, dtype=torch.int32),
             ring=torch.randperm(blocks, generator=gen).to(torch.int32).tolist(), range=[0, blocks], rows=0)
    for step in range(25):
        c["rows"] = sum(c["new"]) + 2
        got, status = call(ver, c)
        want, bits = books(c)
        assert status == bits and all(torch.equal(got[k], x) if isinstance(x, torch.Tensor) else got[k] == x
                                      for k, x in want.items())
        c["held"], c["range"], c["ring"], c["table"] = got["kept"], got["range"], got["ring"], got["table"]
        free = [c["ring"][x % blocks] for x in range(*c["range"])]
        owned = [x for i in range(N) for x in c["table"][i, :c["held"][i]].tolist()]
        assert sorted(free + owned) == list(range(blocks))
        used = got["slots"][got["slots"] >= 0]
        assert len(set(used.tolist())) == len(used)
        for i in range(N):
            if got["seq"][i]:
                c["past"][i] = got["seq"][i] - int(torch.randint(0, max(1, c["new"][i]), (1,), generator=gen))
            else:
                c["past"][i] = 0 if c["past"][i] < 0 else c["past"][i]
            if float(torch.rand(1, generator=gen)) < 0.1 or c["past"][i] > width * block - 8:
                c["past"][i] = -1
            c["new"][i] = 20 if c["past"][i] == 0 else int(torch.randint(1, 7, (1,), generator=gen))


def test_serial_launch_and_another_stream(ver):
    c = state([5, 9, 1, 700, 5000], [0, 20, 31, 7, -1], pad=300, spare=500)
    other = sv.Verifier(8, 8, 8, flags=sv.SV_FLAG_SERIAL_LAUNCH)
    want = check(ver, c)
    side = torch.cuda.Stream()
    for got in (call(other, c)[0], call(ver, c, stream=side)[0]):
        for name, x in want.items():
            assert torch.equal(got[name], x) if isinstance(x, torch.Tensor) else got[name] == x
    other.close()


def test_in_a_graph(ver):
    """A captured step, replayed: the state goes on by itself."""
    N, block = 6, 4
    i32 = dict(dtype=torch.int32, device="cuda")
    table, held = torch.full((N, 20), -1, **i32), torch.zeros(N, **i32)
    ring, span = torch.arange(80, **i32), torch.tensor([0, 80], device="cuda")
    seq, new = torch.zeros(N, **i32), torch.full((N,), 5, **i32)
    positions, slots = torch.zeros(40, **i32), torch.zeros(40, dtype=torch.int64, device="cuda")
    ws = ver.plan_workspace(num_reqs=N)
    ws.fill_(0xFF)

    def step():
        ver.plan_step(num_new_tokens=new, num_computed_tokens=seq, block_tables=table, held_pages=held, free_pages=ring,
                      free_range=span, block_size=block, num_rows=40, positions=positions, slot_mapping=slots,
                      seq_lens=seq, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        assert seq.tolist() == [5 * k] * N and held.tolist() == [-(-5 * k // block)] * N
        assert span.tolist() == [sum(held.tolist()), 80]
        assert positions.tolist() == list(range(5 * k - 5, 5 * k)) * N + [-1] * 10
        t = positions[:30].long().view(N, 5)
        assert torch.equal(slots[:30].view(N, 5), table.long().gather(1, t // block) * block + t % block)


def test_small_workspace(ver):
    c = state([5], [0])
    with pytest.raises(sv.SpecVerifyError) as ei:
        t = torch.zeros(1, dtype=torch.int32, device="cuda")
        ver.plan_step(num_new_tokens=t, num_computed_tokens=t, block_tables=c["table"].cuda(), held_pages=t,
                      free_pages=t, free_range=torch.zeros(2, dtype=torch.int64, device="cuda"), block_size=16,
                      num_rows=0, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert ei.value.code == sv.SV_ERR_CAPACITY


@pytest.mark.parametrize("N", [5, 60, 700])
def test_pages_that_all_share_stay(ver, N):
    """A prefix of three pages at the head of every table: done requests give back only what is their own."""
    new, past, *_ = rand(N, N, 9, 400, done=0.3)
    past = [p if p < 0 else p + 48 for p in past]
    held = [3 + i % 7 if p < 0 else -(-p // 16) for i, p in enumerate(past)]
    c = state(new, past, held=held, pad=7, spare=N + 5)
    c["table"][:, :3] = torch.tensor([9000, 9001, 9002], dtype=torch.int32)
    c["shared"] = 3
    check(ver, c)
    check(ver, c, in_place=True)
    c["held"][0], c["past"][0] = 2, 20  # (a live request that does not hold them)
    check(ver, c, BITS["BAD_PARAM"])
    c["held"][0], c["past"][0] = 2, -1  # (an idle place need not)
    check(ver, c)
