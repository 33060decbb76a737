"""A prompt and decode steps through the 4-bit cache, as a server would run them.

Random weights, INT4 linears and operators of this package only:

    qkv linear -> norm, rotation and append of k and v -> attention over the
    cache -> output linear, for each layer; vocabulary linear -> sampling

The prompts of all requests are one step; then every replay of one captured
CUDA graph gives each request its next token (lengths, block tables and tokens
stay on the device).

    python examples/decode_kv4.py [--layers 2] [--requests 4] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_w4a16_gemv_gb300 as w4  # noqa: E402


class Linear:
    """INT4 weights [N, K], group 128, FP16 scale and zero point."""

    def __init__(self, N, K, g):
        self.qw = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
        self.s = torch.full((N, K // 128), 0.2 * K ** -0.5, dtype=torch.float16, device="cuda")
        self.z = torch.full((N, K // 128), 7.5, dtype=torch.float16, device="cuda")

    def __call__(self, x):
        if x.shape[0] == 1:
            return w4.w4a16_gemv(x[0], self.qw, self.s, self.z)[None]
        return w4.w4a16_gemm(x, self.qw, self.s, self.z)


class Model:
    def __init__(self, layers, hidden, Hq, Hkv, D, vocab, max_positions, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda").to(torch.bfloat16)
        self.qkv = [Linear((Hq + 2 * Hkv) * D, hidden, g) for _ in range(layers)]
        self.out = [Linear(hidden, Hq * D, g) for _ in range(layers)]
        self.norm = [(torch.ones(D, dtype=torch.bfloat16, device="cuda"),) * 2 for _ in range(layers)]
        self.vocab = Linear(vocab, hidden, g)
        angle = torch.arange(max_positions)[:, None] * 10000.0 ** (-torch.arange(D // 2) * 2.0 / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


class Server:
    """Requests with their caches, one per layer, over shared block tables."""

    def __init__(self, model, requests, max_len, block_size=16):
        m, self.model, self.bs = model, model, block_size
        most = -(-max_len // block_size)
        self.caches = [w4.kv4_cache(requests * most, m.Hkv, block_size, m.D) for _ in m.qkv]
        self.scratch = w4.kv4_attention_scratch(m.Hq, m.Hkv, m.D)
        self.block_table = torch.full((requests, most), -1, dtype=torch.int32, device="cuda")
        self.free = torch.arange(requests * most, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def step(self, tokens, new_lens, max_new, draw):
        """The new tokens of every request in; the logits of each one's last
        token, and the next token that `draw` (sampling settings) gives."""
        m, T = self.model, tokens.numel()
        plan = w4.kv4_plan(self.ctx, new_lens, self.block_table, self.free, self.bs, num_tokens=T)
        x = m.embedding[tokens]
        for cache, qkv, out, (qn, kn) in zip(self.caches, m.qkv, m.out, m.norm):
            row = qkv(torch.nn.functional.rms_norm(x, x.shape[1:]))
            q, k, v = (t.unflatten(1, (-1, m.D)) for t in row.split([m.Hq * m.D, m.Hkv * m.D, m.Hkv * m.D], 1))
            q = w4.kv4_append(k, v, cache, plan.slots, q=q, q_weight=qn, k_weight=kn, cos_sin=m.cos_sin,
                              positions=plan.positions)
            a = w4.kv4_attention(q, cache, self.block_table, plan.seq_lens, plan.cu_new, self.scratch, max_new=max_new)
            x = x + out(a.flatten(1))
        last = x[plan.cu_new[1:].long() - 1]
        logits = m.vocab(torch.nn.functional.rms_norm(last, last.shape[1:]))
        # the step's tokens and blocks are taken
        self.ctx.copy_(plan.seq_lens)
        at = torch.arange(self.free.numel(), device="cuda") + plan.taken
        self.free.copy_(torch.where(at < self.free.numel(), self.free[at.clamp(max=self.free.numel() - 1)], -1))
        return logits, w4.w4a16_sample(logits, **draw)


def generate(model, prompts, steps, draw, u, graph=True, block_size=16):
    """Tokens [steps + 1, requests] after the prompts (lists of token ids), with
    the uniform numbers u [steps + 1, requests]."""
    B = len(prompts)
    s = Server(model, B, max(map(len, prompts)) + steps + 1, block_size)
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    ids = torch.tensor(sum(prompts, []), device="cuda")
    _, tokens = s.step(ids, lens, max(map(len, prompts)), dict(draw, u=u[0]))
    got = [tokens.clone()]
    ones, now = torch.ones_like(lens), u[1].clone()
    settings = dict(draw, u=now)
    if graph and steps:
        keep = [t.clone() for t in (s.ctx, s.free, s.block_table)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):       # once outside the graph; its append is repeated by the first replay
            s.step(tokens, ones, 1, settings)
        torch.cuda.current_stream().wait_stream(side)
        for t, was in zip((s.ctx, s.free, s.block_table), keep):
            t.copy_(was)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tokens.copy_(s.step(tokens, ones, 1, settings)[1])
    for i in range(1, steps + 1):
        now.copy_(u[i])
        if graph:
            g.replay()
        else:
            tokens.copy_(s.step(tokens, ones, 1, settings)[1])
        got.append(tokens.clone())
    return torch.stack(got)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=3840)
    ap.add_argument("--vocab", type=int, default=262144)
    a = ap.parse_args(argv)
    model = Model(a.layers, a.hidden, 16, 8, 256, a.vocab, 4096)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, a.vocab, (int(n),), generator=g).tolist()
               for n in torch.randint(1, 200, (a.requests,), generator=g)]
    u = torch.rand(a.steps + 1, a.requests, generator=g).cuda()
    full = lambda v, **kw: torch.full((a.requests,), v, device="cuda", **kw)
    draw = dict(temperature=full(0.8), top_k=full(50, dtype=torch.int32), top_p=full(0.95))
    tokens = generate(model, prompts, a.steps, draw, u)
    torch.cuda.synchronize()
    if w4.w4a16_check_device_error():
        raise RuntimeError(w4.w4a16_last_error_string())
    for b, p in enumerate(prompts):
        print("request %d: %d tokens of prompt, then %s" % (b, len(p), tokens[:, b].tolist()))
    return tokens


if __name__ == "__main__":
    main()
