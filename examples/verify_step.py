"""One verification step of a small model, with every call the library has for it.

A batch of requests shares a system prompt.  A step takes each request's drafts:

1. their keys and values (and the last committed token's) are quantised into
   the paged cache at slot_mapping                              kv_write
2. the verify tokens attend to the cache, the shared prompt's pages read
   once for the whole batch                                     attend
3. the model's head gives target logits                         (torch)
4. drafts are accepted or replaced, the slots of rejected ones
   become -1 and num_computed_tokens is taken back              verify
5. the committed tokens' log-probabilities, with alternatives   logprobs
6. the accepted tokens' cache rows are read back, as a server does that moves a
   request                                                      kv_read

The model is one attention layer with random weights; its drafts come from a
noisy copy of its own head, so some are accepted.  Run it on a GPU:

    python examples/verify_step.py
"""
import pathlib
import sys

import torch

ROOT = pathlib.Path(__file__).resolve().parents[1]
if str(ROOT) not in sys.path:
    sys.path.insert(0, str(ROOT))

import speculative_decoding_token_rejection_gb300 as sv  # noqa: E402


class Model:
    """One attention layer: embedding, projections, head."""

    def __init__(self, vocab, q_heads, kv_heads, dim, gen, device):
        def weight(*shape):
            return torch.randn(*shape, generator=gen, device=device).to(torch.bfloat16) * shape[-1] ** -0.5

        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.embed = weight(vocab, q_heads * dim) * (q_heads * dim) ** 0.5
        self.qkv = weight((q_heads + 2 * kv_heads) * dim, q_heads * dim)
        self.head = weight(vocab, q_heads * dim) * 12

    def project(self, tokens):
        """(q, key, value) of tokens: slices of one product."""
        x = (self.embed[tokens] @ self.qkv.t()).view(len(tokens), self.q_heads + 2 * self.kv_heads, self.dim)
        a, b = self.q_heads, self.q_heads + self.kv_heads
        return x[:, :a], x[:, a:b], x[:, b:]

    def logits(self, attended):
        return attended.flatten(1) @ self.head.t()


def run(requests=8, gamma=4, prompt=64, steps=4, vocab=2000, q_heads=8, kv_heads=2, dim=64, block=16, fmt=torch.int8,
        seed=0, device="cuda", say=print):
    device = torch.device(device, torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    model = Model(vocab, q_heads, kv_heads, dim, gen, device)
    N, G = requests, gamma
    ver = sv.Verifier(N, G, vocab, device=device.index)

    # a cache with the prompt's pages and a few of its own for every request
    pages = -(-(steps * (G + 1) + G + 1) // block)
    blocks = prompt // block + N * pages
    shape = (blocks, kv_heads, block, dim)
    cache = sv.KVCache(k=torch.zeros(shape, dtype=torch.uint8, device=device).view(fmt),
                       v=torch.zeros(shape, dtype=torch.uint8, device=device).view(fmt),
                       k_scale=torch.ones(shape[:3], device=device), v_scale=torch.ones(shape[:3], device=device))
    own = prompt // block + torch.arange(N * pages, device=device, dtype=torch.int32).view(N, pages)
    tables = torch.cat([torch.arange(prompt // block, device=device, dtype=torch.int32).expand(N, -1), own], 1).contiguous()
    prompt_tokens = torch.randint(0, vocab, (prompt,), generator=gen, device=device)
    _, key, value = model.project(prompt_tokens)
    ver.kv_write(cache=cache, key=key, value=value, slot_mapping=torch.arange(prompt, device=device))

    most = prompt + pages * block
    workspace = ver.attend_workspace(num_reqs=N, max_spec_len=G, num_q_heads=q_heads, num_kv_heads=kv_heads, head_dim=dim,
                                     max_seq_len=most, shared_prefix_len=prompt, num_tokens=N * (G + 1))
    computed = torch.full((N,), prompt, dtype=torch.int32, device=device)  # tokens whose keys are in the cache
    last = torch.randint(0, vocab, (N,), generator=gen, device=device)
    texts, logprobs = [[] for _ in range(N)], [[] for _ in range(N)]
    status = torch.zeros(1, dtype=torch.int32, device=device)
    column = torch.arange(G + 1, device=device)
    for step in range(steps):
        def forward(tokens):
            """Target logits of each request's last token and drafts [N * (G + 1), V], and the tokens' slots."""
            q, key, value = model.project(tokens.reshape(-1))
            position = computed[:, None].long() + column
            slots = tables.long().gather(1, position // block) * block + position % block
            slots = slots.reshape(-1).contiguous()
            ver.kv_write(cache=cache, key=key, value=value, slot_mapping=slots, status=status)
            attended = ver.attend(q=q, cache=cache, block_tables=tables, seq_lens=computed + G + 1, max_seq_len=most,
                                  max_spec_len=G, shared_prefix_len=prompt, scale=dim ** -0.5, workspace=workspace,
                                  status=status)
            return model.logits(attended), slots

        # drafts: token by token from the model itself with noise on its logits
        tokens = torch.zeros(N, G + 1, dtype=torch.long, device=device)
        tokens[:, 0] = last
        draft = torch.empty(N, G, vocab, dtype=torch.bfloat16, device=device)
        for j in range(G):
            noisy = forward(tokens)[0].view(N, G + 1, vocab)[:, j].float()
            noisy = noisy + 0.5 * torch.randn(noisy.shape, generator=gen, device=device)
            draft[:, j] = noisy.to(torch.bfloat16)
            tokens[:, j + 1] = draft[:, j].float().argmax(-1)
        # the step itself
        target, slots = forward(tokens)
        computed += G + 1
        result = ver.verify(entry="logits", draft_ids=tokens[:, 1:].reshape(-1).to(torch.int32).contiguous(), target=target,
                            draft=draft.view(N * G, vocab), max_spec_len=G, num_reqs=N, seed=seed, offset=step,
                            num_computed_tokens=computed, slot_mapping=slots, status=status)
        lp = ver.logprobs(logits=target, out_tokens=result.out_tokens, num_top=5, status=status)
        # rejected drafts' slots are -1 now: they read back as zeros
        kept, _ = ver.kv_read(cache=cache, slot_mapping=slots, status=status)
        rows = kept.view(N, G + 1, -1).abs().amax(-1) > 0
        accepted = result.num_accepted
        assert torch.equal(rows.sum(1).to(torch.int32), accepted + 1)
        for i in range(N):
            n = int(accepted[i]) + 1
            texts[i] += result.out_tokens[i, :n].tolist()
            logprobs[i] += lp.logprobs[i, :n].tolist()
        last = result.out_tokens.gather(1, accepted[:, None].long())[:, 0].long()
        say(f"step {step}: accepted {accepted.tolist()}, mean log-probability "
            f"{float(lp.logprobs[result.out_tokens >= 0].mean()):.2f}, status {int(status.item())}")
    assert int(status.item()) == 0
    ver.close()
    return texts, logprobs, computed.tolist()


# Sizes at which attention computes the prompt once for the batch (in smaller calls every request reads it for itself).
SHARED = dict(requests=512, prompt=768, q_heads=8, kv_heads=8)

if __name__ == "__main__":
    run()
