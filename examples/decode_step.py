"""A decoder layer's attention block on packed weights and a packed cache.

    python examples/decode_step.py

Several sequences of different lengths share one paged key-value cache.  Their
prompts go through the quantized projections and are written into the cache
(quantized as they are written); then tokens are generated one at a time, or
several at once as when drafted tokens are checked: the projections of the new
tokens, their rows appended to the cache, attention over it, and the output
projection, all captured in one HIP graph that is replayed for every step while
the sequences grow.  At the end the block's last output is compared with the
same computation in binary32 on the dequantized weights and the cache read
back.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import group_wise_affine_aq_amd as aq  # noqa: E402


class AttentionBlock:
    """Projections with packed weights (4 bits, groups of 64) around a paged cache."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, pages=64, page_size=16,
                 cache_bits=8, cache_group=32, dtype=torch.float16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.page_size, self.bits, self.group, self.dtype = page_size, cache_bits, cache_group, dtype

        def packed(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device="cuda") * cols ** -0.5
            return aq.aq_quantize(w, 64, 4)

        self.w_qkv = packed((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = packed(hidden, q_heads * head_dim)
        shape = (pages, kv_heads, page_size)
        self.cache = []
        for _ in range(2):  # K, V
            if cache_bits == 16:
                self.cache += [torch.zeros(shape + (head_dim,), dtype=dtype, device="cuda"), None, None]
            else:
                groups = shape + (head_dim // cache_group,)
                self.cache += [torch.zeros(shape + (head_dim * cache_bits // 32,),
                                           dtype=torch.int32, device="cuda"),
                               torch.zeros(groups, dtype=torch.float16, device="cuda"),
                               torch.zeros(groups, dtype=torch.float16, device="cuda")]
        self.workspace = None

    def project(self, x):
        """x [T, hidden] -> q [T, q_heads, head_dim], k and v [T, kv_heads, head_dim], parts of
        one projection's rows."""
        rows = aq.aq_quantized_matmul(x, *self.w_qkv, 64, 4)
        d = self.head_dim
        q, k, v = rows.split([self.q_heads * d, self.kv_heads * d, self.kv_heads * d], dim=1)
        return q.unflatten(1, (-1, d)), k.unflatten(1, (-1, d)), v.unflatten(1, (-1, d))

    def append(self, k, v, slots):
        aq.aq_kv_append(k, v, slots, *self.cache, self.group, self.bits)

    def slots(self, table, sequence, positions):
        """Cache slots of the positions of a sequence (both int64 [T])."""
        page = table[sequence, positions // self.page_size].long()
        return page * self.page_size + positions % self.page_size

    def step(self, x, slots, table, lengths):
        """x [B, L, hidden]: the newest L tokens of every sequence -> [B, L, hidden]."""
        B, L, hidden = x.shape
        q, k, v = self.project(x.view(B * L, hidden))
        self.append(k, v, slots)
        if self.workspace is None:  # zeroed once, kept for every step
            need = aq.aq_paged_attention_workspace(B, L, self.q_heads, self.kv_heads, self.head_dim)
            self.workspace = torch.zeros(need, dtype=torch.uint8, device="cuda")
        out = aq.aq_paged_attention(q.unflatten(0, (B, L)), *self.cache, table, lengths, self.group,
                                    self.bits, workspace=self.workspace)
        return aq.aq_quantized_matmul(out.view(B * L, -1), *self.w_out, 64, 4).view(B, L, hidden)


def reference(block, x, table, lengths):
    """step() on the cache as it stands, in binary32, sequence by sequence."""
    B, L, hidden = x.shape
    dense = [aq.aq_dequantize(*w, 64, 4, out_dtype=torch.float32) for w in (block.w_qkv, block.w_out)]
    d, group = block.head_dim, block.q_heads // block.kv_heads
    q = (x.float() @ dense[0][:block.q_heads * d].T).to(block.dtype).float()
    q = q.view(B, L, block.q_heads, d)
    out = torch.zeros_like(q)
    for b, n in enumerate(lengths.tolist()):
        positions = torch.arange(n, device="cuda")
        k, v = aq.aq_kv_read(block.slots(table, torch.full_like(positions, b), positions),
                             *block.cache, block.group, block.bits, out_dtype=torch.float32)
        for h in range(block.q_heads):
            score = q[b, :, h] @ k[:, h // group].T * d ** -0.5
            hidden_from = positions[None] > n - L + torch.arange(L, device="cuda")[:, None]
            out[b, :, h] = torch.softmax(score.masked_fill(hidden_from, -torch.inf), -1) @ v[:, h // group]
    return (out.view(B, L, -1) @ dense[1].T).view(B, L, hidden)


def generate(prompts=(37, 5, 90), steps=6, tokens=1, seed=0, **block_args):
    """Prompts of random rows, then `steps` steps of `tokens` new random rows per sequence.
    -> (largest difference from the reference in units of its largest value, block)."""
    hidden = 512
    need = max(prompts) + steps * tokens
    page_size = block_args.get("page_size", 16)
    per = -(-need // page_size)
    B = len(prompts)
    block = AttentionBlock(hidden=hidden, pages=B * per, **block_args)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    # every sequence's pages, scattered over the cache
    table = torch.randperm(B * per, generator=gen, device="cuda").int().view(B, per)

    def rows(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(block.dtype)

    for b, n in enumerate(prompts):
        _, k, v = block.project(rows(n, hidden))
        positions = torch.arange(n, device="cuda")
        block.append(k, v, block.slots(table, torch.full_like(positions, b), positions))

    # one step, captured once and replayed while the lengths grow
    x = torch.zeros((B, tokens, hidden), dtype=block.dtype, device="cuda")
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B * tokens, dtype=torch.int64, device="cuda")
    who = torch.arange(B, device="cuda").repeat_interleave(tokens)

    def load():
        positions = (lengths[:, None] + torch.arange(tokens, device="cuda")).view(-1).long()
        slots.copy_(block.slots(table, who, positions))
        x.copy_(rows(B, tokens, hidden))
        lengths.add_(tokens)

    load()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        block.step(x, slots, table, lengths)  # (allocates the workspace)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            y = block.step(x, slots, table, lengths)
    torch.cuda.synchronize()
    for i in range(steps):
        if i:
            load()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
    ref = reference(block, x, table, lengths)
    return float((y.float() - ref).abs().max() / ref.abs().max()), block


def main() -> int:
    if not torch.cuda.is_available():
        print("this example needs an MI355X")
        return 1
    for tokens in (1, 3):
        for bits in (4, 8, 16):
            off, block = generate(tokens=tokens, cache_bits=bits)
            stored = sum(t.numel() * t.element_size() for t in block.cache if t is not None)
            print(f"{tokens} token(s) a step, {bits}-bit cache ({stored} bytes): largest difference "
                  f"from binary32 {off:.2e} of the largest value")
    return 0


if __name__ == "__main__":
    sys.exit(main())
