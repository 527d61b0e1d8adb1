"""Outputs and scratch that a call allocates for itself.  On another stream they come
from that stream's memory pool: what is handed out there is neither still in
use on another stream nor given away while the call runs."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend import make, run, verifier
from test_gpu_kv_cache import make_cache
from test_gpu_logprobs import make as make_rows

pytestmark = pytest.mark.gpu


def pool_of(t):
    """The stream whose pool the tensor's memory is from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.fixture(params=["stream", "integer", "default as integer"])
def call_stream(request):
    """(what is passed, the stream it stands for); another stream is current meanwhile."""
    if request.param == "default as integer":
        with torch.cuda.stream(torch.cuda.Stream()):
            yield 0, torch.cuda.default_stream()
        return
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    yield (s if request.param == "stream" else s.cuda_stream), s


def test_attend(call_stream, monkeypatch):
    given, stream = call_stream
    c = make([3, 1, 0], [3000, 90, 17], seed=15)  # cut into chunks: a workspace is needed
    want = run(c)[0]
    made = []
    original = sv.Verifier.attend_workspace
    monkeypatch.setattr(sv.Verifier, "attend_workspace",
                        lambda self, **kw: made.append(original(self, **kw)) or made[-1])
    torch.cuda.synchronize()
    out = verifier().attend(q=c["q"], cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=3000,
                            max_spec_len=3, scale=c["scale"], cu_num_draft_tokens=c["cu"], stream=given)
    stream.synchronize()
    assert torch.equal(out, want)
    assert made[0].numel() > 16
    assert pool_of(made[0]) == pool_of(out) == stream.cuda_stream


def test_kv_read(call_stream):
    given, stream = call_stream
    cache = make_cache(4, 2, 16, 128, "int8")
    cache.k.fill_(3)
    torch.cuda.synchronize()
    key, value = verifier().kv_read(cache=cache, slot_mapping=torch.arange(40, device="cuda"), stream=given)
    torch.cuda.synchronize()
    assert bool((key == 3).all()) and bool((value == 0).all())
    assert pool_of(key) == pool_of(value) == stream.cuda_stream


def test_logprobs(call_stream):
    given, stream = call_stream
    c = make_rows(3, 2, 500, torch.float32)
    ver, tokens = sv.Verifier(8, 4, 1000), c["tokens"].cuda()
    want = ver.logprobs(logits=c["logits"], out_tokens=tokens, num_top=4)
    torch.cuda.synchronize()
    got = ver.logprobs(logits=c["logits"], out_tokens=tokens, num_top=4, stream=given)
    stream.synchronize()
    for name in ("logprobs", "ranks", "entropy", "top_ids", "top_logprobs"):
        assert torch.equal(getattr(got, name), getattr(want, name))
        assert pool_of(getattr(got, name)) == stream.cuda_stream
    ver.close()


def test_the_workspace_goes_by_what_the_tables_hold(monkeypatch):
    """max_seq_len is an upper bound: the workspace of a call's own is that of the lengths its block tables allow."""
    c = make([3, 1, 0], [3000, 90, 17], seed=15)
    made = []
    original = sv.Verifier.attend_workspace

    def small(self, **kw):
        assert kw["max_seq_len"] <= 3008
        made.append(original(self, **kw))
        return made[-1]

    monkeypatch.setattr(sv.Verifier, "attend_workspace", small)
    outs = [verifier().attend(q=c["q"], cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"], max_seq_len=most,
                              max_spec_len=3, scale=c["scale"], cu_num_draft_tokens=c["cu"]) for most in (3000, 3008, 1 << 30)]
    assert made[1].numel() == made[2].numel()
    assert torch.equal(outs[1], outs[2])
    assert torch.equal(outs[0], run(c)[0])
