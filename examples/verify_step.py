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

serve() does such steps for requests that come and go, over a 4-bit cache whose
pages they take and give back: before the keys are written,

0. every request's missing pages are taken from the free ones, those of requests
   that are done go back, and rows get their positions and slots    plan_step
   queries and keys get a norm of each head and turn to their
   positions                                                        rotate

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


def serve(places=4, requests=10, gamma=3, prompt=60, new_tokens=20, vocab=1000, q_heads=8, kv_heads=2, dim=64, block=16,
          fmt="e2m1", seed=0, device="cuda", say=print):
    """Requests with prompts of up to `prompt` tokens, of which `places` run at once; each gets `new_tokens` and a step's
    surplus.  Returns their texts and what the cache's books say at the end."""
    device = torch.device(device, torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    model = Model(vocab, q_heads, kv_heads, dim, gen, device)
    N, G = places, gamma
    longest = prompt + new_tokens + 2 * (G + 1)
    ver = sv.Verifier(N, max(G, prompt - 1), vocab, device=device.index)
    frequencies = sv.RotaryFrequencies(dim, device=device)
    norms = torch.rand(2, dim, generator=gen, device=device).add_(0.5).to(torch.bfloat16)

    def i32(*shape, fill=0):
        return torch.full(shape, fill, dtype=torch.int32, device=device)

    # a cache of as many pages as the places may need, all of them free
    width = -(-longest // block)
    lead = (N * width, kv_heads, block)
    sides = {x: torch.zeros(*lead, dim // 2, dtype=torch.uint8, device=device) for x in "kv"}
    groups = {x + "_group": torch.zeros(*lead, dim // 16, device=device).to(torch.float8_e4m3fn) for x in "kv"}
    scales = {x + "_scale": torch.zeros(lead, device=device) for x in "kv"}
    cache = sv.KVCache4(**sides, **groups, **scales, format=fmt)
    tables, held, computed = i32(N, width), i32(N), i32(N, fill=-1)
    free, span = torch.arange(N * width, dtype=torch.int32, device=device), torch.tensor([0, N * width], device=device)
    workspace = ver.plan_workspace(num_reqs=N)
    status = i32(1)

    waiting = [torch.randint(0, vocab, (int(n),), generator=gen, device=device) for n in
               torch.randint(1, prompt + 1, (requests,), generator=gen, device=device)]
    texts, running = [[] for _ in waiting], [None] * N  # the request in each place
    coming = list(range(requests))
    last = torch.zeros(N, dtype=torch.long, device=device)

    def prepare(new):
        """The plan of a step of new[i] tokens a request, and a function of the tokens to the rows' target logits."""
        cu = i32(N)
        most = max(new) - 1
        plan = ver.plan_step(num_new_tokens=torch.tensor(new, dtype=torch.int32, device=device),
                             num_computed_tokens=computed, block_tables=tables, held_pages=held, free_pages=free,
                             free_range=span, block_size=block, num_rows=sum(new), cu_num_draft_tokens=cu,
                             workspace=workspace, status=status)

        def forward(tokens):
            q, key, value = model.project(tokens)
            ver.rotate(q=q, key=key, positions=plan.positions, frequencies=frequencies, q_weight=norms[0],
                       key_weight=norms[1])
            ver.kv_write(cache=cache, key=key, value=value, slot_mapping=plan.slot_mapping, status=status)
            return model.logits(ver.attend(q=q, cache=cache, block_tables=tables, seq_lens=plan.seq_lens,
                                           max_seq_len=width * block, max_spec_len=most, scale=dim ** -0.5,
                                           cu_num_draft_tokens=cu, status=status))
        return plan, forward

    step = 0
    while coming or any(x is not None for x in running):
        new = [1] * N
        arriving = [i for i in range(N) if running[i] is None][:len(coming)]
        if arriving:  # prompts of requests that come; the others go on by a token
            for i in arriving:
                running[i] = coming.pop(0)
                new[i], computed[i] = len(waiting[running[i]]), 0
            tokens = torch.cat([waiting[running[i]] if i in arriving else last[i:i + 1] for i in range(N)])
            plan, forward = prepare(new)
            target = forward(tokens)[torch.tensor(new, device=device).cumsum(0) - 1]
            drafts = dict(draft_ids=i32(0), draft=target[:0], max_spec_len=0)
            slots = None
        else:
            new = [G + 1] * N
            tokens = torch.zeros(N, G + 1, dtype=torch.long, device=device)
            tokens[:, 0] = last
            draft = torch.empty(N, G, vocab, dtype=torch.bfloat16, device=device)
            plan, forward = prepare(new)
            for j in range(G):
                noisy = forward(tokens.view(-1)).view(N, G + 1, vocab)[:, j].float()
                noisy = noisy + 0.5 * torch.randn(noisy.shape, generator=gen, device=device)
                draft[:, j] = noisy.to(torch.bfloat16)
                tokens[:, j + 1] = draft[:, j].float().argmax(-1)
            target = forward(tokens.view(-1))
            drafts = dict(draft_ids=tokens[:, 1:].reshape(-1).to(torch.int32).contiguous(), draft=draft.view(N * G, vocab),
                          max_spec_len=G)
            slots = plan.slot_mapping
        live = plan.seq_lens > 0
        after = torch.where(live, plan.seq_lens, computed)
        result = ver.verify(entry="logits", target=target.contiguous(), num_reqs=N, seed=seed, offset=step, status=status,
                            num_computed_tokens=after, slot_mapping=slots, **drafts)
        computed.copy_(torch.where(live, after, computed))
        last = result.out_tokens.gather(1, result.num_accepted[:, None].long())[:, 0].long()
        accepted = result.num_accepted.tolist()
        for i, request in enumerate(running):
            if request is None:
                continue
            texts[request] += result.out_tokens[i, :accepted[i] + 1].tolist()
            if len(texts[request]) >= new_tokens:  # its pages go back in the next step, or to the next request here
                running[i], computed[i] = None, -1
        say(f"step {step}: {'prompts' if arriving else 'drafts'}, running {running}, free pages {int(span[1] - span[0])}")
        step += 1
    # the last ones' pages
    ver.plan_step(num_new_tokens=i32(N), num_computed_tokens=computed, block_tables=tables, held_pages=held, free_pages=free,
                  free_range=span, block_size=block, num_rows=0, workspace=workspace, status=status)
    assert int(status.item()) == 0
    ver.close()
    return texts, held.tolist(), span.tolist(), free.tolist()


# Sizes at which attention computes the prompt once for the batch (in smaller calls every request reads it for itself).
SHARED = dict(requests=512, prompt=768, q_heads=8, kv_heads=8)

if __name__ == "__main__":
    run()
    serve()
