"""The example of a whole verification step: its calls work together, its
bookkeeping adds up, and a run repeats itself."""
import importlib.util

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("verify_step", ROOT / "examples" / "verify_step.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [dict(), dict(requests=60, gamma=3, prompt=256, q_heads=8, kv_heads=1, dim=128, block=32,
                                             steps=3, fmt=torch.float8_e4m3fn)])
def test_the_step_runs_and_adds_up(kw):
    run = example().run
    texts, logprobs, computed = run(say=lambda line: None, **kw)
    prompt = kw.get("prompt", 64)
    for text, lp, n in zip(texts, logprobs, computed):
        # every committed token but the last one of a step has its key in the cache by the end of it
        assert n == prompt + len(text) and len(lp) == len(text)
        assert all(x <= 0 for x in lp)
    steps = kw.get("steps", 4)
    assert sum(len(t) for t in texts) > steps * len(texts)  # some drafts were accepted
    assert run(say=lambda line: None, **kw) == (texts, logprobs, computed)


def test_a_step_that_shares_its_prompt():
    """At these sizes the prompt goes through the kernels that compute it once for the batch."""
    import speculative_decoding_token_rejection_gb300 as sv
    module = example()
    kw = module.SHARED
    N, G, prompt = kw["requests"], 4, kw["prompt"]
    ver = sv.Verifier(N, G, 2000)

    def size(prefix):
        return sv.spec_verify_attend_workspace_size(ver.handle, num_reqs=N, max_spec_len=G, num_q_heads=kw["q_heads"],
                                                    num_kv_heads=kw["kv_heads"], head_dim=64, max_seq_len=prompt + 64,
                                                    shared_prefix_len=prefix, num_tokens=N * (G + 1))

    assert size(prompt) != size(0)
    texts, logprobs, computed = module.run(steps=2, say=lambda line: None, **kw)
    assert all(n == prompt + len(text) and len(lp) == len(text) for text, lp, n in zip(texts, logprobs, computed))
    assert sum(len(t) for t in texts) > 2 * N
    assert module.run(steps=2, say=lambda line: None, **kw) == (texts, logprobs, computed)
    ver.close()
