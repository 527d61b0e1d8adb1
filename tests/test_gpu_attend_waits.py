"""Waits of the shared prefix's kernel that run out, without faulting a GPU: the
call flag SV_TEST_EXPIRE_PRODUCT_WAIT makes each CTA's products give up at
their first wait for a tile's weights, with the other roles' copies, waits and
products under way.  The status word says so whichever role gave up, the rows
are NaN rather than what the workspace held, and the next call is an ordinary
one."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend import run, verifier
from test_gpu_attend_scales import make, shared_prefix

pytestmark = pytest.mark.gpu

SIZES = {  # longer: keys more than the shortest prefix that is shared; segments of a few key tiles, of many, and several
    "few tiles": (dict(gammas=[4] * 40, uniform=True), 0),
    "many tiles": (dict(gammas=[4] * 40, uniform=True), 16384),
    "many heads": (dict(gammas=[3] * 300, uniform=True, kv_heads=8, group=2, dim=64, fmt="e4m3"), 800),
}


@pytest.mark.parametrize("flags", [0, sv.SV_FLAG_SERIAL_LAUNCH])
@pytest.mark.parametrize("name", SIZES)
def test_an_expired_wait_is_reported_and_gives_nan(name, flags):
    kw, longer = SIZES[name]
    prefix = shared_prefix(**kw) + longer
    N = len(kw["gammas"])
    c = make(lens=[prefix + 5 + i % 50 for i in range(N)], prefix=prefix, seed=5, **kw)
    ver, cache = verifier(flags), c["cache"]
    rows, hq = c["q"].shape[:2]
    ws = ver.attend_workspace(num_reqs=N, max_spec_len=c["G"], num_q_heads=hq, num_kv_heads=cache.num_kv_heads,
                              head_dim=cache.head_dim, max_seq_len=max(c["lens"]), shared_prefix_len=prefix, num_tokens=rows)
    ws.zero_()  # left-overs that would pass for a result
    want, want_lse, status = run(c, flags=flags, workspace=ws)
    assert status == 0
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.spec_verify_attend(ver.handle, q=c["q"], cache=cache, block_tables=c["table"], seq_lens=c["seq_lens"],
                          max_seq_len=max(c["lens"]), max_spec_len=c["G"], scale=c["scale"], out=out, lse=lse,
                          cu_num_draft_tokens=c["cu"], shared_prefix_len=prefix, workspace=ws, status=bits,
                          test_flags=sv.SV_TEST_EXPIRE_PRODUCT_WAIT)
    torch.cuda.synchronize()
    assert int(bits.item()) == sv.DATA_STATUS_BITS["COPY_TIMEOUT"]
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    got = run(c, flags=flags, workspace=ws)
    assert got[2] == 0 and torch.equal(got[0], want) and torch.equal(got[1], want_lse)


def test_a_call_without_such_waits_ignores_the_flag():
    c = make([2, 0, 5], [300, 20, 900], seed=20)
    want = run(c)
    out = torch.zeros_like(want[0])
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    ver = verifier()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    sv.spec_verify_attend(ver.handle, q=c["q"], cache=c["cache"], block_tables=c["table"], seq_lens=c["seq_lens"],
                          max_seq_len=900, max_spec_len=5, scale=c["scale"], out=out, cu_num_draft_tokens=c["cu"],
                          workspace=ws, status=bits, test_flags=sv.SV_TEST_EXPIRE_PRODUCT_WAIT)
    assert int(bits.item()) == 0 and torch.equal(out, want[0])
