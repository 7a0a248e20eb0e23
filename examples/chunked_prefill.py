"""Prompts in chunks beside lanes that decode, through one layer: pages planned on the device, head norms with rotary
positions, attention of each lane's chunk over the paged 8-bit cache, resident-expert routed MoE.

    python examples/chunked_prefill.py [--steps N]

Synthetic weights and hidden states (the tiny layer of ``synth``). Every step has room for so many tokens: lanes that decode
take one each, the others share what is left for the next part of their prompts. A lane that has decoded enough is done: its
pages go back, and it begins a new prompt.
"""
from __future__ import annotations

import argparse
import os
import random
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import resident_expert_routed_gb300 as moe
from examples.tree_decode import HEAD_DIM, PAGE, build
from resident_expert_routed_gb300.decode import DevicePages, HeadNorms
from resident_expert_routed_gb300.rotary import rotary_frequencies, rotary_turns


def schedule(left: list[int], decode: list[int], budget: int) -> list[int]:
    """New tokens of each lane: one of a lane that decodes, then prompts in the lanes' order as far as the budget goes."""
    new = [1 if not l and d else 0 for l, d in zip(left, decode)]
    room = budget - sum(new)
    for b, l in enumerate(left):
        if l and room > 0:
            new[b] = min(l, room)
            room -= new[b]
    return new


def main(steps: int = 24, lanes: int = 4, budget: int = 64, n_pages: int = 64, seed: int = 0):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    weight = lambda: 1 + 0.1 * torch.randn(HEAD_DIM, generator=gen, device="cuda")  # noqa: E731
    norms = HeadNorms(rotary_turns(rotary_frequencies(HEAD_DIM, stretch=4.0, rule="ramp")), weight(), weight())
    layer = build(lanes, budget, n_pages, seed, norms)
    pages = DevicePages(lanes, n_pages, PAGE, 16, budget)
    d = layer.w_qkv.shape[1]
    left = [rng.randint(5, 150) for _ in range(lanes)]          # of the prompts
    decode = [rng.randint(2, 8) for _ in range(lanes)]          # tokens still to be decoded
    rows, finished = [0] * lanes, 0                             # what the host knows without asking the device
    for step in range(steps):
        new = schedule(left, decode, budget)
        ends = [b for b in range(lanes) if not left[b] and not decode[b]]
        pages.plan(torch.tensor([-1 if b in ends else n for b, n in enumerate(new)], dtype=torch.int32).pin_memory().cuda(non_blocking=True))
        hidden = torch.randn((sum(new), d), generator=gen, device="cuda").bfloat16()
        out = layer.chunk(hidden, pages)
        pages.advance()
        for b in range(lanes):
            if b in ends:
                finished += 1
                rows[b], left[b], decode[b] = 0, rng.randint(5, 150), rng.randint(2, 8)
                continue
            rows[b] += new[b]
            if left[b]:
                left[b] -= new[b]
            else:
                decode[b] -= new[b]
        print(f"step {step}: new tokens {new}, done {ends}, rows {rows}, |output| {out.float().norm().item():.2f}")
    assert pages.rows.tolist() == rows
    held = sum(-(-r // PAGE) for r in rows)
    assert pages.n_free.item() == n_pages - held
    st, bits = moe.moe_device_status()
    assert st == moe.MOE_OK, f"device status {st} bits {bits:#x}"
    print(f"{finished} lanes finished; {held} pages held, {pages.n_free.item()} free")
    return layer, pages


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=24)
    main(ap.parse_args().steps)
