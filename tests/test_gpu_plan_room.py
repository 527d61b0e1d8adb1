"""plan_step with books that are wrong: pages that come back to a ring that has no
place for them.  What is free stays, and so do the tables of requests that take
pages in the same call."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_plan import BITS, call, ver  # noqa: F401 (ver is a fixture)

pytestmark = pytest.mark.gpu


def step(idle, width, at):
    """Ten places, seven of them free: done requests that hold 2, 2, 0 and 1 pages, one that takes 3, and `idle` more."""
    ring = [-1] * 10
    for k in range(7):
        ring[(at + k) % 10] = 100 + k
    table = torch.full((5 + idle, width), -1, dtype=torch.int32)
    table[0, :2], table[1, :2], table[3, :1] = torch.tensor([1, 2]), torch.tensor([3, 4]), 5
    return dict(new=[0, 0, 0, 0, 40] + [0] * idle, past=[-1, -1, -1, -1, 0] + [-1] * idle, held=[2, 2, 0, 1, 0] + [0] * idle,
                block=16, table=table, ring=ring, range=[at, at + 7], rows=40)


@pytest.mark.parametrize("idle, width", [(0, 4), (1500, 4), (700, 40), (3000, 40)])
@pytest.mark.parametrize("at", [0, 4, (1 << 40) + 3])
def test_pages_that_have_no_place_stay(ver, idle, width, at):  # noqa: F811
    c = step(idle, width, at)
    got, status = call(ver, c)
    assert status == BITS["BAD_PARAM"]
    # the first request's two pages find places; with the second's there would be four for three, and so on
    assert got["kept"][:5] == [0, 2, 0, 1, 3] and not any(got["kept"][5:])
    assert got["range"] == [at + 3, at + 9]
    assert [got["ring"][(at + k) % 10] for k in range(9)] == [100 + k for k in range(7)] + [1, 2]
    assert got["ring"][(at + 9) % 10] == -1
    assert got["table"][4, :3].tolist() == [100, 101, 102]
    assert got["slots"].tolist() == [(100 + t // 16) * 16 + t % 16 for t in range(40)]
    # the same again with books in order: they go back once there is room
    for name, x in (("held", "kept"), ("range", "range"), ("ring", "ring"), ("table", "table")):
        c[name] = got[x]
    c["new"][4], c["past"][4] = 0, 40
    got, status = call(ver, c)
    assert status == 0 and got["kept"][:5] == [0, 0, 0, 0, 3] and got["range"] == [at + 3, at + 12]
    assert [got["ring"][(at + 3 + k) % 10] for k in range(9)] == [103, 104, 105, 106, 1, 2, 3, 4, 5]


def test_a_ring_that_is_full(ver):  # noqa: F811
    c = step(0, 4, 2)
    c["ring"], c["range"] = list(range(100, 110)), [2, 12]
    got, status = call(ver, c, in_place=True)
    assert status == BITS["BAD_PARAM"] and got["kept"] == [2, 2, 0, 1, 3] and got["range"] == [5, 12]
    assert got["ring"] == c["ring"] and got["table"][4, :3].tolist() == [102, 103, 104]
