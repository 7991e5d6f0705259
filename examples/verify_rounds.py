"""Speculative rounds from end to end: append, attend, accept, commit.

A toy target of one attention layer decodes several requests behind one shared
prompt.  Each round verifies k drafts per request:

  1. ``AttnPlan.append`` normalises and rotates the rows' heads and writes their
     keys and values after the request's committed tokens;
  2. ``AttnPlan.attend`` lets every row see the prompt, the committed tokens and
     the round's rows up to itself;
  3. ``Plan.run`` accepts the leading drafts that match the target's argmax and
     writes the records of the tokens that were emitted;
  4. the committed lengths grow by the accepted drafts and one more.  Rejected
     tokens stay in the cache, past the length: nothing reads them there, and
     the next round writes over them.

The batch has a slot without a request, as a captured batch has: its rows go
through every call, its length stays negative, and its old page table, which
names pages that other requests hold by now, is not written through.

The drafts are what followed the same token the last time, so they are accepted
as soon as the decoding repeats itself.

With ``kv_bits=4`` the cache is held in 4 bits (``append4``, ``attend4``), and
``AttnPlan.reserve`` lays each round out on the device: a request takes pages from a
queue of free ones as it grows, and the rows' positions follow from its length.  A
request that gets none sits the round out.
The toy's logits then move by what 4 bits lose.  Run it on a GB300:

    python examples/verify_rounds.py [--kv-bits 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import logprob_epilogue_gb300 as lpe  # noqa: E402

EPS = 1e-6


class Target:
    """The toy target's weights, and its plain form in 64 bits."""

    def __init__(self, vocab=2048, hidden=256, q_heads=8, kv_heads=2, head_dim=64, positions=1024, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.vocab, self.q_heads, self.kv_heads, self.head_dim = vocab, q_heads, kv_heads, head_dim

        def weight(n, m):
            return (torch.randn(n, m, generator=g, device=device) * n ** -0.5).bfloat16()
        self.embed = torch.randn(vocab, hidden, generator=g, device=device).bfloat16()
        self.qkv = weight(hidden, (q_heads + 2 * kv_heads) * head_dim)
        self.out = weight(q_heads * head_dim, hidden)
        self.head = weight(hidden, vocab)
        self.q_norm, self.k_norm = ((1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).bfloat16() for _ in range(2))
        angle = torch.arange(positions, device=device)[:, None] * 10000.0 ** (-torch.arange(0, head_dim, 2, device=device) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

    def heads(self, tokens):
        """q, k and v of the tokens' rows: views of one product."""
        x = self.embed[tokens]
        y, d, n, m = x @ self.qkv, self.head_dim, self.q_heads, self.kv_heads
        return x, *(y[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, n), (n, n + m), (n + m, n + 2 * m)))

    def logits(self, x, attended):
        return ((x + attended.flatten(1) @ self.out) @ self.head).contiguous()

    def plain_logits(self, tokens):
        """Logits after every token of one sequence, all of it in 64 bits."""
        x, q, k, v = (t.double() for t in self.heads(tokens))
        half, pos = self.head_dim // 2, torch.arange(len(tokens), device=tokens.device)

        def rotate(t, weight):
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * weight.double()
            cos, sin = self.cos_sin[pos].double().unsqueeze(1).split(half, -1)
            a, b = t[..., :half], t[..., half:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        q, k = rotate(q, self.q_norm), rotate(k, self.k_norm)
        share = self.q_heads // self.kv_heads
        s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(share, 1)) * self.head_dim ** -0.5
        s = s.masked_fill(pos[None, :] > pos[:, None], float("-inf")).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", s, v.repeat_interleave(share, 1))
        return (x + o.flatten(1) @ self.out.double()) @ self.head.double()


def decode(target, prompt, firsts, rounds=24, drafts=3, page=16, idle=1, kv_bits=16, free=None):
    """Decodes from each of ``firsts`` behind ``prompt``, with ``idle`` slots of the batch free: the emitted tokens of each
    request, the rounds' accepted drafts (-1: the request sat out), and the slots' committed lengths.  ``free``: pages that 4
    bits find in the queue (as many as all slots need unless given)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    requests, groups, rows_of, m = len(firsts), len(firsts) + idle, drafts + 1, len(prompt)
    rows, prompt_pages = groups * rows_of, -(-m // page)
    max_pages = max(prompt_pages, -(-(rounds * rows_of) // page) + 1)
    num_pages = groups * max_pages + prompt_pages
    four, shape = kv_bits == 4, (num_pages, target.kv_heads, page)
    if four:
        names = {"k_cache": (2, torch.uint8), "v_cache": (2, torch.uint8), "k_scales": (16, torch.float8_e4m3fn), "v_scales": (16, torch.float8_e4m3fn)}
    else:
        names = {"k_cache": (1, torch.bfloat16), "v_cache": (1, torch.bfloat16)}
    caches = {name: torch.zeros(*shape, target.head_dim // lanes, dtype=dtype, device=dev) for name, (lanes, dtype) in names.items()}
    tables = i32(torch.arange(groups * max_pages).view(groups, max_pages))
    tables[requests:] = tables[0].clone()  # what a request that has left held belongs to another now
    prompt_table = i32([[groups * max_pages + i for i in range(prompt_pages)]])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    attention = lpe.AttnPlan(max_rows=rows, max_groups=groups, q_heads=target.q_heads, kv_heads=target.kv_heads,
                             head_dim=target.head_dim, page_size=page, num_pages=num_pages, max_pages=max_pages,
                             max_group_rows=rows_of, max_prefixes=1, max_prefix_pages=prompt_pages, device=dev.index,
                             kv_bits=kv_bits)
    epilogue = lpe.Plan(max_rows=rows, max_groups=groups, k_max=drafts, V=target.vocab, V_padded=target.vocab, dtype="bf16",
                        device=dev.index)
    common = dict(status=status, **caches)
    rope = dict(cos_sin=target.cos_sin, q_weight=target.q_norm, k_weight=target.k_norm, eps=EPS)

    # the prompt's keys and values, once for all requests
    filler = lpe.AttnPlan(max_rows=m, max_groups=1, q_heads=target.q_heads, kv_heads=target.kv_heads, head_dim=target.head_dim,
                          page_size=page, num_pages=num_pages, max_pages=prompt_pages, device=dev.index, kv_bits=kv_bits)
    _, _, k, v = target.heads(torch.as_tensor(prompt, device=dev))
    fill, append, attend = ((filler.append4, attention.append4, attention.attend4) if four else
                            (filler.append, attention.append, attention.attend))
    fill(k=k, v=v, group_indptr=i32([0, m]), lens=i32([0]), block_tables=prompt_table, positions=i32(range(m)), **rope, **common)

    indptr, lens = i32([g * rows_of for g in range(groups + 1)]), i32([0] * requests + [-1] * idle)
    if four:  # all pages but the prompt's are free, and nobody holds any
        tables, held, queue = i32([[-1] * max_pages] * groups), i32([0] * groups), torch.tensor([0, groups * max_pages if free is None else free], device=dev)
        layout = dict(counts=i32([rows_of] * groups), starts=i32([m] * groups), held=held, held_out=held, queue=queue, queue_out=queue,
                      free_pages=i32(range(groups * max_pages)), block_tables=tables, group_indptr=indptr, status=status,
                      round_lens=i32([0] * groups), positions=i32([0] * rows))
    epilogue_io = dict(group_indptr=indptr, sampled_tokens=i32([-1] * groups), requested=i32([1] * groups), top_k=i32([5] * groups),
                       token_ids=i32([[-1] * lpe.MAX_IDS] * groups), id_counts=i32([0] * groups),
                       records=i32([[0] * lpe.RECORD_WORDS] * rows), accepted=i32([0] * groups), emitted_tokens=i32([0] * rows),
                       status=torch.zeros(1, dtype=torch.int32, device=dev))
    q_out, out = (torch.empty(rows, target.q_heads, target.head_dim, dtype=torch.bfloat16, device=dev) for _ in range(2))
    emitted, followed, accepted_of = [[t] for t in firsts], {}, []
    for _ in range(rounds):
        block = []
        for g in range(requests):
            block.append(emitted[g][-1])
            for _ in range(drafts):
                block.append(followed.get(block[-1], 0))
        block += [0] * (idle * rows_of)
        tokens = torch.tensor(block, device=dev)
        x, q, k, v = target.heads(tokens)
        if four:
            attention.reserve(lens=lens, **layout)
            positions, round_lens = layout["positions"], layout["round_lens"]
        else:
            positions, round_lens = (m + lens.clamp(min=0)[:, None] + torch.arange(rows_of, dtype=torch.int32, device=dev)).flatten(), lens
        append(q=q, k=k, v=v, q_out=q_out, group_indptr=indptr, lens=round_lens, block_tables=tables, positions=positions, **rope, **common)
        attend(q=q_out, out=out, group_indptr=indptr, lens=round_lens, block_tables=tables, prefix_indptr=i32([0, groups]),
               prefix_lens=i32([m]), prefix_tables=prompt_table, **common)
        draft_tokens = i32([block[r + 1] if (r + 1) % rows_of else -1 for r in range(rows)])
        epilogue.bind(logits=target.logits(x, out), draft_tokens=draft_tokens, **epilogue_io)
        epilogue.run()
        took_part = torch.where(round_lens < 0, -1, epilogue_io["accepted"])
        lens += took_part + 1
        accepted, new = took_part[:requests].tolist(), epilogue_io["emitted_tokens"].view(groups, rows_of).tolist()
        for g, a in enumerate(accepted):
            for t in new[g][:a + 1]:
                followed[emitted[g][-1]] = t
                emitted[g].append(t)
        accepted_of.append(accepted)
    for name, word in (("attention", status), ("epilogue", epilogue_io["status"])):
        if int(word) & ~lpe.STATUS_NO_PAGES:
            raise RuntimeError(f"{name}: status {int(word):#x}")
    for plan in (attention, filler, epilogue):
        plan.close()
    return emitted, accepted_of, lens.tolist()


def shortfall(target, prompt, emitted):
    """How far an emitted token's logit lies below the largest of the plain form, at most."""
    worst = 0.0
    for e in emitted:
        logits = target.plain_logits(torch.tensor(prompt + e[:-1], device="cuda"))[len(prompt):]
        chosen = logits.gather(1, torch.tensor(e[1:], device="cuda")[:, None])[:, 0]
        worst = max(worst, float((logits.max(1).values - chosen).max()))
    return worst


def main(kv_bits=16):
    if not torch.cuda.is_available():
        raise SystemExit("this example needs a CUDA device")
    target = Target()
    prompt = torch.randint(0, target.vocab, (100,), generator=torch.Generator().manual_seed(1)).tolist()
    emitted, accepted, _ = decode(target, prompt, firsts=list(range(8)), kv_bits=kv_bits)
    tokens = sum(len(e) - 1 for e in emitted)
    print(f"{len(emitted)} requests, {len(accepted)} rounds: {tokens} tokens, {sum(map(sum, accepted))} of them accepted drafts")
    worst = shortfall(target, prompt, emitted)
    print(f"an emitted token's logit lies at most {worst:.3f} below the largest of the plain form in 64 bits")
    return emitted, accepted, worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description="Speculative rounds of a toy target.")
    parser.add_argument("--kv-bits", type=int, choices=(4, 16), default=16, help="bits of a cached key or value")
    main(parser.parse_args().kv_bits)
