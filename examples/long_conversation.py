"""A decoder layer's attention block with rotary positions and capped scores, and
a cache that is kept within a budget.

    python examples/long_conversation.py

Prompts of different lengths go through the quantized projections; their queries
and keys are turned by their positions while keys and values are written into a
paged cache, and the whole prompts attend to themselves in one call.  Then tokens
are generated one at a time: turn and write, attention over the cache with capped
scores, and what every cached token got of it, all captured in one HIP graph that
is replayed for every step.  From time to time every sequence is brought back to
its budget: the tokens that gathered most move to other pages, the old ones are
free again.  At the end the block's last output is compared with the same
computation in binary32 on the dequantized weights and the cache read back.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import group_wise_affine_aq_amd as aq  # noqa: E402


class Block:
    """Projections with packed weights (4 bits, groups of 64) around a paged cache."""

    def __init__(self, sequences, budget, hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_size=16,
                 cache_bits=8, cache_group=32, softcap=20.0, room=64, dtype=torch.float16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.softcap = q_heads, kv_heads, head_dim, softcap
        self.page_size, self.packing, self.dtype, self.budget = page_size, (cache_group, cache_bits), dtype, budget

        def packed(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device="cuda") * cols ** -0.5
            return aq.aq_quantize(w, 64, 4)

        self.w_qkv = packed((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = packed(hidden, q_heads * head_dim)
        # the model's frequencies, stretched for contexts four times as long as it was trained on
        self.freqs, self.factor = aq.aq_rope_frequencies(head_dim, 10000.0, "by_index", 4.0, 2048, 1, 32)
        # pages for the longest sequences, and as many again to move into
        self.per = -(-(budget + room) // page_size)
        pages = 2 * sequences * self.per
        shape = (pages, kv_heads, page_size)
        self.cache = []
        for _ in range(2):  # K, V
            if cache_bits == 16:
                self.cache += [torch.zeros(shape + (head_dim,), dtype=dtype, device="cuda"), None, None]
            else:
                groups = shape + (head_dim // cache_group,)
                self.cache += [torch.zeros(shape + (head_dim * cache_bits // 32,), dtype=torch.int32, device="cuda"),
                               torch.zeros(groups, dtype=torch.float16, device="cuda"),
                               torch.zeros(groups, dtype=torch.float16, device="cuda")]
        order = torch.randperm(pages, generator=gen, device="cuda").int().view(2, sequences, self.per)
        self.table, self.free = order[0].clone(), order[1].clone()
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device="cuda")    # tokens in the cache
        self.positions = torch.zeros(sequences, dtype=torch.int32, device="cuda")  # tokens of the conversation
        self.weights = torch.zeros((sequences, self.per * page_size), device="cuda")
        self.workspace = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")

    def project(self, x):
        """x [T, hidden] -> q [T, q_heads, head_dim], k and v [T, kv_heads, head_dim], parts of
        one projection's rows."""
        rows = aq.aq_quantized_matmul(x, *self.w_qkv, 64, 4)
        d = self.head_dim
        q, k, v = rows.split([self.q_heads * d, self.kv_heads * d, self.kv_heads * d], dim=1)
        return q.unflatten(1, (-1, d)), k.unflatten(1, (-1, d)), v.unflatten(1, (-1, d))

    def slots(self, sequence, places):
        """Cache slots of places in sequences (both int64)."""
        page = self.table[sequence, places // self.page_size].long()
        return page * self.page_size + places % self.page_size

    def prompts(self, x, lengths):
        """x: all prompts' rows one after the other -> their outputs."""
        starts = torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32, device="cuda")
        n = torch.tensor(lengths, device="cuda")
        who = torch.arange(len(lengths), device="cuda").repeat_interleave(n)
        places = torch.arange(len(x), device="cuda") - starts[who]
        q, k, v = self.project(x)
        turned = torch.empty((len(x), self.kv_heads, self.head_dim), dtype=x.dtype, device="cuda")
        q = aq.aq_rope_append(q, k, v, places.int(), self.freqs, self.slots(who, places), *self.cache,
                              *self.packing, factor=self.factor, k_out=turned)
        out = aq.aq_prompt_attention(q, turned, v, starts, starts, softcap=self.softcap, workspace=self.workspace)
        self.lengths.copy_(n)
        self.positions.copy_(n)
        return aq.aq_quantized_matmul(out.flatten(1), *self.w_out, 64, 4)

    def step(self, x):
        """x [sequences, hidden]: a new token of each -> [sequences, hidden]."""
        every = torch.arange(len(x), device="cuda")
        q, k, v = self.project(x)
        q = aq.aq_rope_append(q, k, v, self.positions, self.freqs, self.slots(every, self.lengths.long()),
                              *self.cache, *self.packing, factor=self.factor)
        self.lengths += 1
        self.positions += 1
        out, lse = aq.aq_paged_attention_masked(q, *self.cache, self.table, self.lengths, *self.packing,
                                                softcap=self.softcap, return_lse=True, workspace=self.workspace)
        aq.aq_kv_weigh(q, lse, *self.cache, self.table, self.lengths, self.weights, *self.packing,
                       softcap=self.softcap)
        return aq.aq_quantized_matmul(out.flatten(1), *self.w_out, 64, 4)

    def evict(self):
        """Every sequence back to its budget: the first tokens, the last quarter and what gathered most."""
        kept, _, weights = aq.aq_kv_evict(self.weights, self.lengths, self.table, self.free, *self.cache, *self.packing,
                                          keep=self.budget, sinks=4, recent=self.budget // 4, new_lengths=self.lengths)
        self.weights.zero_()
        self.weights[:, :self.budget] = weights
        old = self.table.clone()
        self.table.copy_(self.free)
        self.free.copy_(old)
        return kept


def reference(block, x):
    """step() on the cache as it stands, in binary32."""
    dense = [aq.aq_dequantize(*w, 64, 4, out_dtype=torch.float32) for w in (block.w_qkv, block.w_out)]
    d, group = block.head_dim, block.q_heads // block.kv_heads
    q = (x.float() @ dense[0][:block.q_heads * d].T).to(block.dtype).float().view(len(x), block.q_heads, d)
    angles = (block.positions.double()[:, None] - 1) * block.freqs.double()
    cos, sin = ((f(angles) * block.factor).float()[:, None] for f in (torch.cos, torch.sin))
    a, b = q.split(d // 2, dim=-1)
    q = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1).to(block.dtype).float()
    out = torch.zeros_like(q)
    for s, n in enumerate(block.lengths.tolist()):
        places = torch.arange(n, device="cuda")
        k, v = aq.aq_kv_read(block.slots(torch.full_like(places, s), places), *block.cache, *block.packing,
                             out_dtype=torch.float32)
        for h in range(block.q_heads):
            score = q[s, h] @ k[:, h // group].T * d ** -0.5
            score = block.softcap * torch.tanh(score / block.softcap)
            out[s, h] = torch.softmax(score, -1) @ v[:, h // group]
    return out.flatten(1) @ dense[1].T


def converse(prompts=(100, 37, 70), budget=64, steps=40, every=12, seed=0, **more):
    """Prompts of random rows, then `steps` tokens of each sequence, back to the budget after every
    so many -> (largest difference from the reference in units of its largest value, block, how many
    tokens were evicted)."""
    hidden = 512
    block = Block(len(prompts), budget, hidden, room=max(0, max(prompts) - budget) + steps, **more)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)

    def rows(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(block.dtype)

    block.prompts(rows(sum(prompts), hidden), list(prompts))
    x = rows(len(prompts), hidden)
    block.step(x)  # (what is made once is made now)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    lengths, positions, weights = block.lengths.clone(), block.positions.clone(), block.weights.clone()
    with torch.cuda.graph(graph, stream=stream):
        y = block.step(x)
    torch.cuda.synchronize()
    # (capturing does not run: the sequences stand where they stood)
    assert torch.equal(lengths, block.lengths) and torch.equal(positions, block.positions)
    assert torch.equal(weights, block.weights)
    evicted = 0
    for i in range(steps - 1):
        if i % every == every - 1:
            before = block.lengths.sum()
            block.evict()
            evicted += int(before - block.lengths.sum())
        x.copy_(rows(len(prompts), hidden))
        graph.replay()
    torch.cuda.synchronize()
    ref = reference(block, x)
    return float((y.float() - ref).abs().max() / ref.abs().max()), block, evicted


def main() -> int:
    if not torch.cuda.is_available():
        print("this example needs an MI355X")
        return 1
    for bits in (4, 8, 16):
        off, block, evicted = converse(cache_bits=bits)
        print(f"{bits}-bit cache, {evicted} tokens evicted, lengths {block.lengths.tolist()} of "
              f"{block.positions.tolist()}: largest difference from binary32 {off:.2e} of the largest value")
    return 0


if __name__ == "__main__":
    sys.exit(main())
