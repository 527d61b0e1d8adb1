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
