"""Waits of the 4-bit cache's attention that run out, without faulting a GPU: the
call flag SV_TEST_EXPIRE_PRODUCT_WAIT makes a product's first wait give up.  The
status word says so, the rows are NaN rather than what the workspace held, and
the next call is an ordinary one."""
import pytest
import torch

import speculative_decoding_token_rejection_gb300 as sv
from test_gpu_attend4 import make, run, verifier

pytestmark = pytest.mark.gpu

CASES = {
    "one chunk": dict(gammas=[2, 0, 5], lens=[300, 20, 90]),
    "chunks": dict(gammas=[3, 3], lens=[30000, 17000], dim=64, fmt="int4"),
    "many rows": dict(gammas=[8] * 4, lens=[700, 900, 128, 9], group=8, uniform=True),
    "shared prefix": dict(gammas=[4] * 40, lens=[2330 + i for i in range(40)], prefix=2240, uniform=True),
    "shared prefix, many heads": dict(gammas=[3] * 300, lens=[2600] * 300, prefix=2560, uniform=True, kv_heads=8, group=2,
                                      dim=64, fmt="int4"),
}


@pytest.mark.parametrize("flags", [0, sv.SV_FLAG_SERIAL_LAUNCH])
@pytest.mark.parametrize("name", CASES)
def test_an_expired_wait_is_reported_and_gives_nan(name, flags):
    c = make(seed=5, **CASES[name])
    ver, cache, N = verifier(flags), c["cache"], len(c["gammas"])
    rows, hq = c["q"].shape[:2]
    ws = ver.attend_workspace(cache=cache, num_reqs=N, max_spec_len=c["G"], num_q_heads=hq, max_seq_len=max(c["lens"]),
                              shared_prefix_len=c["prefix"], num_tokens=rows)
    ws.zero_()  # left-overs that would pass for a result
    want, want_lse, status = run(c, flags=flags, workspace=ws)
    assert status == 0
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.spec_verify_attend(ver.handle, q=c["q"], cache=cache, block_tables=c["table"], seq_lens=c["seq_lens"],
                          max_seq_len=max(c["lens"]), max_spec_len=c["G"], scale=c["scale"], out=out, lse=lse,
                          cu_num_draft_tokens=c["cu"], shared_prefix_len=c["prefix"], workspace=ws, status=bits,
                          test_flags=sv.SV_TEST_EXPIRE_PRODUCT_WAIT)
    torch.cuda.synchronize()
    assert int(bits.item()) == sv.DATA_STATUS_BITS["COPY_TIMEOUT"]
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    got = run(c, flags=flags, workspace=ws)
    assert got[2] == 0 and torch.equal(got[0], want) and torch.equal(got[1], want_lse)
