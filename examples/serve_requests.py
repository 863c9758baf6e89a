"""A small model served from the paged pool, step by step.

Every step builds its block tables, slots and positions on the GPU from the
requests' lengths (paged_tables_build), rotates and appends each layer's q, k
and v (paged_rope_append, rotary positions scaled for a longer context, pairs
interleaved, part of the head), attends with capped scores over alternating
whole and windowed layers (paged_gqa_prefill_scored for the prompts,
paged_gqa_decode_scored for one token a request) and scores the next tokens
with their log-probabilities, entropy and alternatives (token_logprobs). The
weights are random; nothing is read from the GPU until the end.

    python examples/serve_requests.py [--steps 8]
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import paged_kv_decode_rope_gb300 as pkv  # noqa: E402


@dataclasses.dataclass
class Config:
    layers: int = 4
    q_heads: int = 8
    kv_heads: int = 2
    vocab: int = 5003
    context: int = 512
    rot_dim: int = 32
    softcap: float = 20.0
    window: int = 48  # of every second layer
    top: int = 5

    @property
    def width(self) -> int:
        return self.q_heads * pkv.HEAD_DIM


class Model:
    """Embedding, `layers` attention layers with residuals, tied logits."""

    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.cfg = cfg
        self.embed = (torch.randn(cfg.vocab, cfg.width, generator=g, device=device)).to(torch.bfloat16)
        heads = cfg.q_heads + 2 * cfg.kv_heads
        self.qkv = [weight(heads * pkv.HEAD_DIM, cfg.width) for _ in range(cfg.layers)]
        self.out = [weight(cfg.width, cfg.width) for _ in range(cfg.layers)]
        # rotary positions for four times the context that the frequencies were made for
        self.freqs, self.magnitude = pkv.rope_frequencies(10000.0, cfg.rot_dim, "banded", 4.0,
                                                          original_context=cfg.context // 4)

    def project(self, layer: int, x: torch.Tensor):
        """q, k, v: slices of one projection's output, as paged_rope_append takes them."""
        cfg = self.cfg
        qkv = (norm(x) @ self.qkv[layer].T).view(x.shape[0], -1, pkv.HEAD_DIM)
        return qkv.split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], dim=1)

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        return norm(x) @ self.embed.T


def norm(x: torch.Tensor) -> torch.Tensor:
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Server:
    """The pool, the block tables and one step after another of a fixed batch of requests."""

    def __init__(self, model: Model, batch: int, pages: int, max_tokens: int, device="cuda"):
        cfg = model.cfg
        self.model, self.batch = model, batch
        i32 = dict(dtype=torch.int32, device=device)
        self.storage = torch.zeros(pages * pkv.kv_pool_page_bytes(cfg.kv_heads), dtype=torch.uint8, device=device)
        self.pool = pkv.kv_pool_create(self.storage, cfg.kv_heads)
        self.blocks = -(-cfg.context // pkv.PAGE_SIZE)
        self.tables = torch.full((cfg.layers, batch, self.blocks), -1, **i32)
        self.free = torch.randperm(pages, device=device).to(torch.int32)
        # lengths and the next free entry, before and after a step in turns: a step captured into a graph reads
        # and writes the same words every time
        self.all_lens = [torch.zeros(batch, **i32), torch.zeros(batch, **i32)]
        self.heads = [torch.zeros(1, **i32), torch.zeros(1, **i32)]
        self.rope = pkv.alloc_rope_table(cfg.context, device)
        pkv.paged_rope_table_build_freqs(model.freqs, cfg.context, self.rope, model.magnitude)
        self.decode_ws = pkv.alloc_decode_workspace(batch, cfg.q_heads, cfg.kv_heads, self.blocks, device=device)
        self.prefill_ws = pkv.alloc_prefill_workspace(max_tokens, batch, self.blocks, device=device)
        self.logprobs_ws = pkv.alloc_logprobs_workspace(batch, cfg.vocab, cfg.top, device=device)
        self.steps = 0

    def step(self, tokens: torch.Tensor, new_tokens: torch.Tensor, one_each: bool) -> dict:
        """Feed new_tokens[b] tokens of every request (tokens: all of them, one
        after the other); returns the next token of each with its scoring."""
        cfg, model = self.model.cfg, self.model
        dev, total = tokens.device, tokens.shape[0]
        i32 = dict(dtype=torch.int32, device=dev)
        cu = torch.empty(self.batch + 1, **i32)
        positions, slots = torch.empty(total, **i32), torch.empty(cfg.layers, total, **i32)
        now, then = self.steps % 2, (self.steps + 1) % 2
        lens_before, lens = self.all_lens[now], self.all_lens[then]
        pkv.paged_tables_build(self.pool, lens_before, new_tokens, self.free, self.heads[now], self.heads[then],
                               self.tables, cu, lens, positions, slots)
        x = model.embed[tokens.long()]
        q_rot = torch.empty(total, cfg.q_heads, pkv.HEAD_DIM, dtype=torch.float32, device=dev)
        attended = torch.empty(total, cfg.q_heads, pkv.HEAD_DIM, dtype=torch.bfloat16, device=dev)
        for layer in range(cfg.layers):
            q, k, v = model.project(layer, x)
            pkv.paged_rope_append(self.pool, q, k, v, q_rot, slots[layer], positions, self.rope, rot_dim=cfg.rot_dim,
                                  interleaved=True)
            scoring = dict(softcap=cfg.softcap, window=cfg.window if layer % 2 else 0)
            if one_each:
                pkv.paged_gqa_decode_scored(self.pool, q_rot, attended, self.tables[layer], lens, pkv.HEAD_DIM ** -0.5,
                                            self.decode_ws, **scoring)
            else:
                pkv.paged_gqa_prefill_scored(self.pool, q_rot, attended, self.tables[layer], cu, lens_before,
                                             pkv.HEAD_DIM ** -0.5, self.prefill_ws, **scoring)
            x = x + attended.view(total, -1) @ model.out[layer].T
        logits = model.logits(x[cu[1:].long() - 1])
        out = dict(top_ids=torch.empty(self.batch, cfg.top, **i32), logits=logits)
        for name, shape in (("top_logprobs", (self.batch, cfg.top)), ("entropy", (self.batch,))):
            out[name] = torch.empty(*shape, dtype=torch.float32, device=dev)
        pkv.token_logprobs(logits, None, None, out["entropy"], out["top_ids"], out["top_logprobs"], self.logprobs_ws)
        self.steps += 1
        return out

    def error_bits(self) -> int:
        return pkv.pkv_get_error(self.pool)

    def close(self) -> None:
        self.pool.close()


def generate(model: Model, prompts: list[list[int]], steps: int) -> tuple[torch.Tensor, list[dict]]:
    """Greedy tokens [steps][batch] after the prompts, and every step's scoring."""
    cfg = model.cfg
    flat = [t for p in prompts for t in p]
    need = cfg.layers * sum(-(-(len(p) + steps) // pkv.PAGE_SIZE) for p in prompts)
    server = Server(model, len(prompts), need, len(flat))
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = [server.step(torch.tensor(flat, **i32), torch.tensor([len(p) for p in prompts], **i32), one_each=False)]
    one = torch.ones(len(prompts), **i32)
    for _ in range(steps - 1):
        outs.append(server.step(outs[-1]["top_ids"][:, 0].contiguous(), one, one_each=True))
    bits = server.error_bits()  # the first time the host looks at the GPU
    server.close()
    if bits:
        raise RuntimeError(f"the pool's error word is {bits:#x}")
    return torch.stack([o["top_ids"][:, 0] for o in outs]), outs


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    cfg = Config()
    model = Model(cfg)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, cfg.vocab, (n,), generator=g).tolist() for n in (5, 130, 33, 64, 1)]
    tokens, outs = generate(model, prompts, args.steps)
    for b, prompt in enumerate(prompts):
        print(f"request {b}: prompt of {len(prompt)} tokens, then {tokens[:, b].tolist()}")
    last = outs[-1]
    for b in range(len(prompts)):
        alternatives = ", ".join(f"{i} {v:.2f}" for i, v in zip(last["top_ids"][b].tolist(), last["top_logprobs"][b].tolist()))
        print(f"  last step, request {b}: entropy {float(last['entropy'][b]):.2f}, alternatives {alternatives}")


if __name__ == "__main__":
    main()
