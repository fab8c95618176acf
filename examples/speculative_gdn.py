"""Speculative decoding with gated-delta-rule layers over state slots.

A small draft model proposes K tokens a step, the target model reads all of them in one
multi-token call that keeps the state after each, verify_drafts decides how many stand and
which token follows, and both models go back to the state after the last accepted token:

    prefill -> [draft: decode_step, snapshot] x K+1 -> decode_multi -> verify_drafts -> restore

The weights are random; the generated tokens have the target model's distribution all the
same.  Run:  python examples/speculative_gdn.py [--tokens 64] [--batch 32] [--draft 4]
"""
import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rwkv_wkv_gb300 import GdnPool  # noqa: E402


class Model:
    """An embedding, gated-delta-rule layers with residuals, and an output projection."""

    def __init__(self, seed, layers, k_heads, v_heads, width, vocab, embedding=None):
        gen = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[-2] ** -0.5).to(torch.bfloat16)

        self.k_heads, self.v_heads, self.vocab = k_heads, v_heads, vocab
        self.sizes = [k_heads * 64, k_heads * 64, v_heads * 64, v_heads, v_heads]
        own = weight(vocab, 1, width)[:, 0]  # drawn in any case: a seed names the other weights too
        self.embedding = own if embedding is None else embedding
        self.wide = [weight(width, sum(self.sizes)) for _ in range(layers)]
        self.back = [weight(v_heads * 64, width) for _ in range(layers)]
        self.head = weight(width, vocab)

    def pool(self, slots, snapshots):
        return GdnPool(len(self.wide), self.k_heads, self.v_heads, slots, n_snapshots=snapshots, head_k=64, head_v=64,
                       out_dtype="bf16")

    def probs(self, tokens, call):
        """Next-token probabilities after each of `tokens`; call(layer, q, k, v, g, beta) is the
        pool's call for rows of tokens' shape."""
        x = self.embedding[tokens.long()]
        for layer, (wide, back) in enumerate(zip(self.wide, self.back)):
            q, k, v, a, b = (F.rms_norm(x, x.shape[-1:]) @ wide).split(self.sizes, -1)
            q, k, v = (y.unflatten(-1, (-1, 64)) for y in (q, k, v))
            o = call(layer, q, k, v, -F.softplus(a.float() - 2), torch.sigmoid(b.float()))
            x = x + F.rms_norm(o, o.shape[-1:]).flatten(-2) @ back
        return torch.softmax((F.rms_norm(x, x.shape[-1:]) @ self.head).float(), -1)


def generate(target, draft, prompts, n_new, n_draft, seed=0):
    """Continue each prompt (a list of token lists) by at least n_new tokens.  Returns the
    tokens, the mean number of accepted drafts a step, and the target's states, which have read
    everything but each row's last token."""
    n, vocab, dev = len(prompts), target.vocab, "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    norm = {"l2norm_eps": 1e-6}

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    # all but the last token of each prompt
    lens = [len(p) - 1 for p in prompts]
    cu = i32([0] + lens).cumsum(0, dtype=torch.int32)
    packed = i32([t for p in prompts for t in p[:-1]])
    last = i32([p[-1] for p in prompts])
    rows = [list(p) for p in prompts]
    accepted_sum = steps = 0
    with target.pool(n, n * (n_draft + 1)) as tp, draft.pool(n, n * (n_draft + 1)) as dp:
        ids = i32(tp.create(n))
        assert dp.create(n) == ids.tolist()
        # one snapshot for the state after each of [last, drafts]; the same numbers in both pools
        snaps = i32(tp.snapshot_alloc(n * (n_draft + 1))).view(n, n_draft + 1)
        assert dp.snapshot_alloc(n * (n_draft + 1)) == snaps.flatten().tolist()
        if len(packed):
            for m, pool in ((target, tp), (draft, dp)):
                m.probs(packed, lambda layer, *x: pool.prefill(layer, ids, cu, *x, max_seqlen=max(lens), **norm))
        while min(len(r) - len(p) for r, p in zip(rows, prompts)) < n_new:
            # the draft model: K tokens, one after the other
            fed, q = [last], []
            for j in range(n_draft + 1):
                p = draft.probs(fed[j], lambda layer, *x: dp.decode_step(layer, ids, *x, **norm))
                dp.snapshot(ids, snaps[:, j].contiguous())
                if j < n_draft:
                    noise = torch.empty(n, vocab, device=dev).exponential_(generator=gen)
                    q.append(p)
                    fed.append((p / noise).argmax(-1).int())
            fed = torch.stack(fed, 1)
            # the target model reads them all, keeping the state after each
            p = target.probs(fed, lambda layer, *x: tp.decode_multi(layer, ids, *x, step_snap_ids=snaps, **norm))
            accepted, tokens, resume = tp.verify_drafts(
                fed[:, 1:].contiguous(), p, torch.stack(q, 1),
                torch.rand(n, n_draft, generator=gen, device=dev),
                torch.empty(n, vocab, device=dev).exponential_(generator=gen), step_snap_ids=snaps)
            # both go on from the last accepted token's state
            tp.restore(resume, ids)
            dp.restore(resume, ids)
            last = tokens.gather(1, accepted.long()[:, None])[:, 0]
            for row, new, m in zip(rows, tokens.tolist(), accepted.tolist()):
                row += new[:m + 1]
                accepted_sum += m
            steps += 1
        for pool in (tp, dp):
            assert pool.device_status() == 0
        states = tp.states.clone()
    return rows, accepted_sum / max(1, steps * n), states


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64, help="new tokens for each prompt")
    ap.add_argument("--batch", type=int, default=32, help="prompts")
    ap.add_argument("--draft", type=int, default=4, help="drafted tokens a step")
    args = ap.parse_args()
    if args.tokens < 1 or args.batch < 1 or args.draft < 1:
        ap.error("--tokens, --batch and --draft must be at least 1")
    target = Model(1, 4, 8, 16, 512, 1000)
    draft = Model(2, 1, 2, 4, 512, 1000, target.embedding)
    draft.head = target.head
    prompts = [[(7 * i + j) % 1000 for j in range(20 + i % 50)] for i in range(args.batch)]
    generate(target, draft, prompts, 2, args.draft)  # warm-up
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rows, accepted, _ = generate(target, draft, prompts, args.tokens, args.draft)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    new = sum(len(r) - len(p) for r, p in zip(rows, prompts))
    print(f"{new} tokens for {args.batch} prompts in {dt * 1e3:.1f} ms, {accepted:.2f} of {args.draft} drafts accepted a step")
    print("first prompt goes on with", rows[0][len(prompts[0]):][:16])


if __name__ == "__main__":
    main()
