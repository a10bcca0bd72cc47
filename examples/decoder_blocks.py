"""Serving with the library's operators: two decoder blocks, prompts and decode steps in one loop.

Each step places the new tokens in pages (``KvStep``); each block then projects
q, k and v (a plain matrix product), appends k and v to its NVFP4 cache,
attends over it (``Kv4Cache``), adds the residual and norms for the MoE layer
(``block_norm``), runs it (``Nvfp4MoeLayer``) and adds and norms again.
Weights are random: the text is noise, the data flow is a server's.

    python examples/decoder_blocks.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from nvfp4_mixture_experts_moe_gb300 import Kv4Cache, KvStep, Nvfp4MoeLayer, block_norm  # noqa: E402

HIDDEN, INTER, EXPERTS, TOP_K, VOCAB, LAYERS = 512, 256, 16, 4, 1000, 2
Q_HEADS, KV_HEADS, DIM = 8, 2, 64
PAGE, MAX_PAGES, NUM_PAGES = 16, 20, 64
EPS = 1e-6


def rotate(x, positions):
    """Rotary position embedding of ``[tokens, heads, DIM]``, halves paired."""
    freq = 10000.0 ** (-torch.arange(0, DIM // 2, device=x.device) / (DIM // 2))
    angle = positions[:, None].float() * freq
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1).to(x.dtype)


class Block:
    """One decoder block and its cache."""

    def __init__(self, seed, max_tokens, batch):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).to(torch.bfloat16)
        self.w_qkv = weight((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.w_o = weight(HIDDEN, Q_HEADS * DIM)
        self.norm_moe = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        # keys and values of normed rows stay within about 6
        self.cache = Kv4Cache(NUM_PAGES, PAGE, KV_HEADS, DIM, k_gs=2688 / 6, v_gs=2688 / 6)
        self.attn_ws = self.cache.attention_workspace(max_tokens, batch, Q_HEADS, max_tokens, MAX_PAGES)
        self.moe = Nvfp4MoeLayer(T=max_tokens, H=HIDDEN, I=INTER, E=EXPERTS, k=TOP_K)
        for e in range(EXPERTS + 1):
            self.moe.set_expert(e, weight(INTER, HIDDEN), weight(INTER, HIDDEN), weight(HIDDEN, INTER))
        self.moe.set_router(weight(EXPERTS, HIDDEN))
        self.moe_ws = self.moe.workspace()

    def attend(self, h, x, step, table, max_q):
        """Attention half: residual stream ``h`` and its normed rows ``x`` to the same for the MoE layer."""
        n = x.shape[0]
        qkv = (x @ self.w_qkv.t()).view(n, Q_HEADS + 2 * KV_HEADS, DIM)
        positions = step.positions[:n]
        q = rotate(qkv[:, :Q_HEADS], positions)
        k = rotate(qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], positions)
        self.cache.append(k, qkv[:, Q_HEADS + KV_HEADS:], step.slots[:n])
        o, _ = self.cache.attention(q, step.cu_q, step.kv_len, table, max_q=max_q, ws=self.attn_ws)
        return block_norm(o.view(n, -1) @ self.w_o.t(), h, w_pre=self.norm_moe, eps=EPS)

    def __call__(self, h, x, step, table, max_q, next_norm):
        h, x = self.attend(h, x, step, table, max_q)
        return block_norm(self.moe.forward(x, ws=self.moe_ws), h, w_pre=next_norm, eps=EPS)


class Server:
    """``batch`` request slots over shared pages."""

    def __init__(self, batch, max_tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.max_tokens = batch, max_tokens
        self.embedding = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        self.head = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        self.norm = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.blocks = [Block(seed + 1 + i, max_tokens, batch) for i in range(LAYERS)]
        self.tables = KvStep(batch, max_tokens, PAGE, MAX_PAGES)
        self.block_table = torch.zeros(batch, MAX_PAGES, dtype=torch.int32, device="cuda")
        self.free_pages = torch.arange(NUM_PAGES, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), NUM_PAGES, dtype=torch.int32, device="cuda")
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, tokens, new):
        """Feeds ``new[b]`` tokens of each request (``tokens``: all of them in order); the next token of each, -1 for one
        that was fed nothing."""
        counts = torch.tensor(new, dtype=torch.int32, device="cuda")
        s = self.tables.run(self.length, counts, self.block_table, self.free_pages, self.free_count)
        h, x = block_norm(None, self.embedding[tokens], w_pre=self.norm, eps=EPS)
        for block in self.blocks:
            h, x = block(h, x, s, self.block_table, max(new), self.norm)
        self.length.copy_(s.kv_len)
        self.free_count.copy_(s.free_count)
        last = s.cu_q[1:].long() - 1
        return torch.where(counts > 0, (x[last] @ self.head.t()).argmax(dim=-1), -1)

    def finish(self, request):
        """Puts a request's pages back on the stack; its slot is empty then."""
        pages, count = -(-int(self.length[request]) // PAGE), int(self.free_count)
        self.free_pages[count:count + pages] = self.block_table[request, :pages]
        self.free_count += pages
        self.length[request] = 0


def main():
    prompts = [70, 9, 130]
    server = Server(len(prompts), max_tokens=256)
    tokens = torch.randint(0, VOCAB, (sum(prompts),), generator=torch.Generator().manual_seed(1)).cuda()
    token = server.step(tokens, prompts)                       # the prompts in one step
    text = [token]
    for _ in range(12):                                        # then one token of each request at a time
        token = server.step(token, [1] * len(prompts))
        text.append(token)
    refused = int(server.tables.status)
    for b, row in enumerate(torch.stack(text, dim=1).tolist()):
        print(f"request {b}: {prompts[b]} prompt tokens, then {row}")
    held = NUM_PAGES - int(server.free_count)
    for b in range(len(prompts)):
        server.finish(b)
    print(f"{held} pages held, {int(server.free_count)} of {NUM_PAGES} free at the end, status {refused}")
    return refused


if __name__ == "__main__":
    sys.exit(main())
