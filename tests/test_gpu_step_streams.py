"""Outputs and workspaces that the calls of a step allocate for themselves: on
another stream they come from that stream's memory pool."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend4 import make, run, verifier
from test_gpu_call_streams import call_stream, pool_of
from test_gpu_kv4_cache import make_cache4

pytestmark = pytest.mark.gpu


def test_attend(call_stream, monkeypatch):
    given, stream = call_stream
    c = make([3, 1, 0], [9000, 90, 17], seed=15)  # cut into chunks: a workspace is needed
    want = run(c)[0]
    made = []
    original = sv.Verifier.attend_workspace
    monkeypatch.setattr(sv.Verifier, "attend_workspace",
                        lambda self, **kw: made.append(original(self, **kw)) or made[-1])
    torch.cuda.synchronize()
    out = verifier().attend(q=c["q"], cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=9000,
                            max_spec_len=3, scale=c["scale"], cu_num_draft_tokens=c["cu"], stream=given)
    stream.synchronize()
    assert torch.equal(out, want)
    assert made[0].numel() > 16
    assert pool_of(made[0]) == pool_of(out) == stream.cuda_stream


def test_kv_read(call_stream):
    given, stream = call_stream
    cache = make_cache4(4, 2, 16, 128, "int4")
    cache.k.fill_(0x33)
    cache.k_group.copy_(torch.ones(cache.k_group.shape))
    torch.cuda.synchronize()
    key, value = verifier().kv_read(cache=cache, slot_mapping=torch.arange(40, device="cuda"), stream=given)
    torch.cuda.synchronize()
    assert bool((key == 3).all()) and bool((value == 0).all())
    assert pool_of(key) == pool_of(value) == stream.cuda_stream


def test_plan_step(call_stream, monkeypatch):
    given, stream = call_stream
    i32 = dict(dtype=torch.int32, device="cuda")
    made = []
    original = sv.Verifier.plan_workspace
    monkeypatch.setattr(sv.Verifier, "plan_workspace", lambda self, **kw: made.append(original(self, **kw)) or made[-1])
    new, computed = torch.full((3,), 5, **i32), torch.zeros(3, **i32)
    tables, held, free = torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.arange(12, **i32)
    span = torch.tensor([0, 12], device="cuda")
    torch.cuda.synchronize()
    p = verifier().plan_step(num_new_tokens=new, num_computed_tokens=computed, block_tables=tables, held_pages=held,
                             free_pages=free, free_range=span, block_size=4, num_rows=16, stream=given)
    stream.synchronize()
    assert p.positions.tolist() == [0, 1, 2, 3, 4] * 3 + [-1]
    assert p.slot_mapping.tolist() == [*range(5), *range(8, 13), *range(16, 21), -1]
    for t in (made[0], p.positions, p.slot_mapping, p.seq_lens):
        assert pool_of(t) == stream.cuda_stream
