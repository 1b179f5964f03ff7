"""Speculative decoding's verify step on the library's operators: a small decoder with random weights drafts nothing
itself, but checks blocks of drafted tokens against a 4-bit key/value cache.

    python examples/verify_step.py                 # 4 sequences, blocks of 16, a few steps, one captured graph

A layer is: projection to queries, keys and values (``gemm_w4a16``), rotation and the cache's new rows
(``kv4_append``), attention over the cache (``kv4_attention``), output projection, MLP (``mlp``).  The logits of the
block's rows (``gemm_w8a16``) go to ``token_logprobs``: a drafted token that is the first of the row's top ids is what
greedy decoding would have chosen (a rank of 0 is not enough: bf16 logits often tie, and greedy decoding takes the lowest
id), so the longest prefix of such tokens is kept.  Lengths, page tables and tokens are device tensors, so one
captured graph serves every step; a sequence's rejected tokens are simply overwritten by the next block.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_weight_only_wq_gb300 as wq  # noqa: E402


def _norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Verifier:
    """``layers`` decoder layers of random weights, and the cache of ``seqs`` sequences of up to ``max_len`` tokens."""

    def __init__(self, layers=2, hidden=2560, Hq=32, Hkv=8, D=128, inner=9728, vocab=32000, seqs=4, max_len=1024,
                 page_size=64, group=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(K, N, bits):
            return wq.pack_symmetric(torch.randn(K, N, generator=g, device="cuda") / K ** 0.5, bits)

        self.Hq, self.Hkv, self.D, self.vocab, self.seqs = Hq, Hkv, D, vocab, seqs
        self.embed = torch.randn(vocab, hidden, generator=g, device="cuda", dtype=torch.bfloat16)
        self.layers = [dict(qkv=weight(hidden, (Hq + 2 * Hkv) * D, 4), out=weight(Hq * D, hidden, 4),
                            up=weight(hidden, inner, 4), down=weight(inner, hidden, 4)) for _ in range(layers)]
        self.head = weight(hidden, vocab, 8)
        self.qkv_width, self.hidden = (Hq + 2 * Hkv) * D, hidden
        pages = -(-max_len // page_size)
        self.caches = [wq.kv4_cache(seqs * pages, Hkv, D, page_size, group) for _ in range(layers)]
        # any pages in any order: here a permutation, as a server's free list would give them
        self.table = torch.randperm(seqs * pages, generator=g, device="cuda").int().view(seqs, pages)
        self.rope = wq.rope_table(pages * page_size, D)
        self.workspace = wq.kv4_workspace(Hq, self.caches[0])

    def batch(self, q_len, kv_len):
        """The batch of ``q_len`` new tokens a sequence (a list), ``kv_len`` (int32, device) cached ones with them."""
        cu = torch.tensor([0] + q_len, dtype=torch.int32).cumsum(0).int().cuda()
        return wq.kv4_batch(self.table, cu, kv_len, sum(q_len), max(q_len))

    def logits(self, tokens, batch):
        """Logits [T, vocab] of the rows of ``tokens`` (int64 [T]), which go into the cache on the way."""
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        x = self.embed[tokens]
        for w, cache in zip(self.layers, self.caches):
            qkv = wq.gemm_w4a16(_norm(x), *w["qkv"], self.qkv_width).view(-1, Hq + 2 * Hkv, D)
            q = wq.kv4_append(cache, batch, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], Q=qkv[:, :Hq], rope=self.rope)
            a = wq.kv4_attention(q, cache, batch, workspace=self.workspace)
            x = x + wq.gemm_w4a16(a.view(-1, Hq * D), *w["out"], self.hidden)
            x = x + wq.mlp(_norm(x), *w["up"], *w["down"], 4, act="silu")[1]
        return wq.gemm_w8a16(_norm(x), *self.head, self.vocab)

    def verify(self, tokens, batch, block, k=4):
        """One step over blocks of ``block`` tokens a sequence: row i predicts token i + 1 of its block.  Returns the
        tokens kept of each block (the first one is given), the drafted tokens' log probabilities and the rows'
        alternatives: (kept [seqs], logprob [seqs, block - 1], top ids [T, k])."""
        logits = self.logits(tokens, batch)
        drafted = tokens.view(-1, block).roll(-1, 1).flatten()  # (a block's last row has no drafted successor)
        logprob, _, _, top, _ = wq.token_logprobs(logits, drafted, k)
        right = (top[:, 0] == drafted).view(-1, block)[:, :-1].int()
        return 1 + right.cumprod(1).sum(1), logprob.view(-1, block)[:, :-1], top


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--block", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    B, block, v = a.seqs, a.block, Verifier(seqs=a.seqs)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [a.prompt + 17 * b for b in range(B)]
    kv_len = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    tokens = torch.randint(v.vocab, (sum(prompts),), generator=g, device="cuda")
    ends = torch.tensor(prompts, device="cuda").cumsum(0) - 1
    last = v.logits(tokens, v.batch(prompts, kv_len))[ends].argmax(-1)  # the prompts go in; the first new tokens come out

    # the step that is captured: block tokens a sequence, lengths in `kv_len`
    step_tokens = torch.zeros(B * block, dtype=torch.int64, device="cuda")
    batch = v.batch([block] * B, kv_len)
    kv_len += block
    kept, logprob, top = v.verify(step_tokens, batch, block)  # warm-up; its rows are overwritten below
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, logprob, top = v.verify(step_tokens, batch, block)
    for step in range(a.steps):
        # a stand-in for the drafter: what this model itself says (asked once), with one wrong token in each block
        draft = torch.randint(v.vocab, (B, block), generator=g, device="cuda")
        draft[:, 0] = last
        for i in range(min(step, block - 1)):
            step_tokens.copy_(draft.flatten())
            graph.replay()
            draft[:, i + 1] = top.view(B, block, -1)[:, i, 0]
        step_tokens.copy_(draft.flatten())
        a0, a1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a0.record()
        graph.replay()
        a1.record()
        torch.cuda.synchronize()
        n = kept.long()
        last = top.view(B, block, -1)[torch.arange(B, device="cuda"), n - 1, 0].long()  # the target's own next token
        print(f"step {step}: kept {n.tolist()} of {block}, drafted tokens' mean log probability "
              f"{logprob.mean().item():.2f}, {a0.elapsed_time(a1) * 1e3:.0f} us")
        kv_len += n.int()  # the kept tokens stay; the next block follows them
    status = wq.wq_last_device_error()
    if status != wq.WQ_OK:
        raise SystemExit(wq.status_string(status))


if __name__ == "__main__":
    main()
