"""Speculative decoding through one layer: paged 8-bit cache, tree attention, resident-expert routed MoE.

    python examples/tree_decode.py [--steps N]

Synthetic weights and hidden states (the tiny layer of ``synth``). Each lane's prompt is written and attended in one
chunk; then every step drafts a token tree a lane, runs the layer for all nodes at once, accepts a path (here: drawn
at random), keeps its rows in the cache and goes on from there. At the end the kept rows are read back.
"""
from __future__ import annotations

import argparse
import os
import random
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import resident_expert_routed_gb300 as moe
import synth
from resident_expert_routed_gb300.decode import DecodeLayer, LanePages, Step
from resident_expert_routed_gb300.layer import LayerBuffers

HEADS, KV_HEADS, HEAD_DIM, PAGE = 8, 2, 64, 16


def build(lanes: int, max_tokens: int, n_pages: int, seed: int = 0, norms=None) -> DecodeLayer:
    cfg = synth.TINY
    bias = synth.router_bias(cfg.seed, cfg.E, cfg.sigma)
    resident = synth.resident_set(cfg, bias)
    slot_of = synth.slot_table(cfg, resident, cfg.resident)
    owner = np.full(cfg.resident, -1, np.int32)                          # expert of each slot of the arena
    owner[slot_of[resident]] = resident
    rec = synth.slot_record(cfg.d, cfg.ffn)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    slots = torch.zeros(cfg.resident * rec["slot_bytes"], dtype=torch.uint8, device="cuda")
    synth.fill_slots_device(slots, cfg.d, cfg.ffn, cfg.seed, cfg.E, dev(owner))
    arena = moe.Arena(slots, rec["slot_bytes"], cfg.resident, cfg.d, cfg.ffn, rec["off_gu_codes"], rec["off_gu_scales"],
                      rec["off_dn_codes"], rec["off_dn_scales"])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda *shape: (torch.randn(shape, generator=gen, device="cuda") * shape[1] ** -0.5).bfloat16()  # noqa: E731
    moe_args = (dev(synth.router_weights(cfg.seed, cfg.E, cfg.d)), dev(bias), dev(slot_of), arena,
                torch.zeros((1, cfg.E), dtype=torch.int64, device="cuda"), torch.zeros((1, cfg.E), device="cuda"), 0)
    return DecodeLayer(w((HEADS + 2 * KV_HEADS) * HEAD_DIM, cfg.d), w(cfg.d, HEADS * HEAD_DIM),
                       moe.KvCache.empty(n_pages, KV_HEADS, PAGE, HEAD_DIM), HEADS, lanes, max_tokens, moe_args,
                       LayerBuffers(max_tokens, cfg.k, cfg.E, cfg.d, cfg.ffn, cfg.resident), norms)


def draft(rng: random.Random, n: int) -> list[int]:
    """Parents of a random tree of n nodes under one root (the token decided last)."""
    return [-1] + [rng.randrange(max(0, i - 3), i) for i in range(1, n)]


def accept(rng: random.Random, parents: list[int]) -> list[int]:
    """A path from the root to a random node."""
    node, path = rng.randrange(len(parents)), []
    while node >= 0:
        path.append(node)
        node = parents[node]
    return path[::-1]


def main(steps: int = 8, lanes: int = 3, seed: int = 0):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    prompts = [5 + 17 * b for b in range(lanes)]
    layer = build(lanes, max(sum(prompts), 24 * lanes), 64)
    pages = LanePages(lanes, 64, PAGE, 16)
    d = layer.w_qkv.shape[1]
    hidden = torch.randn((sum(prompts), d), generator=gen, device="cuda").bfloat16()
    tables = Step(pages, [list(range(-1, n - 1)) for n in prompts])
    layer.step(hidden, tables, tree=False)
    for b, n in enumerate(prompts):
        pages.advance(b, n)
    for step in range(steps):
        # the last lane waits every third step
        parents = [[] if b == lanes - 1 and step % 3 == 2 else draft(rng, rng.randint(1, 16)) for b in range(lanes)]
        tables = Step(pages, parents)
        hidden = torch.randn((tables.n_nodes, d), generator=gen, device="cuda").bfloat16()
        out = layer.step(hidden, tables)
        paths = [accept(rng, p) if p else [] for p in parents]
        width = max(1, max(map(len, paths)))
        path = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        layer.keep(tables, path, torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"))
        for b, p in enumerate(paths):
            pages.advance(b, len(p))
        print(f"step {step}: nodes {tables.counts}, kept {[len(p) for p in paths]}, |output| {out.float().norm().item():.2f}")
    cu = torch.tensor([sum(pages.rows[:b]) for b in range(lanes + 1)], dtype=torch.int32, device="cuda")
    k, v = (torch.empty((sum(pages.rows), KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_kv_read(layer.cache, pages.table.cuda(), None, cu, k, v)
    st, bits = moe.moe_device_status()
    assert st == moe.MOE_OK, f"device status {st} bits {bits:#x}"
    print(f"rows kept {pages.rows}, read back |k| {k.float().norm().item():.2f} |v| {v.float().norm().item():.2f}")
    return layer, pages, k, v


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    main(ap.parse_args().steps)
