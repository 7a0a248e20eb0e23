"""One layer of a served model: attention over the paged 8-bit cache, then the routed-MoE layer step.

``LanePages`` keeps, on the host, which pages of a cache each lane holds; ``DevicePages`` keeps the same on the device
(``moe_page_plan``), so that a batch of new tokens is planned without the host's lists. ``DecodeLayer`` is a layer's
weights and buffers; ``step`` runs it for the tree nodes (or single tokens) of all lanes: the projection of queries, keys
and values (a plain library product), ``moe_qk_rotate`` where the layer has norms or rotary positions, ``moe_kv_write``,
``moe_tree_attention``, the output projection and ``layer_step``. ``chunk`` runs it for a chunk of new tokens of every lane
(a prompt, the next part of one, a single token), with ``moe_chunk_attention``. ``keep`` moves the rows of each lane's
accepted path together once the nodes have been checked. No arithmetic of the cache, the attention or the experts is done
here.
"""
from __future__ import annotations

import copy
from dataclasses import dataclass

import torch

from . import (KvCache, moe_chunk_attention, moe_chunk_attention_workspace_bytes, moe_kv_keep, moe_kv_write, moe_page_plan,
               moe_qk_rotate, moe_tree_attention, moe_tree_attention_workspace_bytes)
from .layer import LayerBuffers, layer_step


class LanePages:
    """Pages of a cache by lane: a free list and one table row a lane (host bookkeeping).

    ``table`` int32 [lanes, width] (pinned when a GPU is there), -1 past a lane's pages; ``rows[b]`` are the rows the
    lane has kept. Every layer's cache uses the same table."""

    def __init__(self, lanes: int, n_pages: int, page_size: int, width: int):
        self.page_size, self.width = page_size, width
        self.free = list(range(n_pages))[::-1]
        self.pages = [[] for _ in range(lanes)]
        self.rows = [0] * lanes
        self.table = torch.full((lanes, width), -1, dtype=torch.int32)
        if torch.cuda.is_available():
            self.table = self.table.pin_memory()

    def reserve(self, lane: int, rows: int) -> None:
        """Make room for `rows` more rows after those the lane has kept."""
        need = -(-(self.rows[lane] + rows) // self.page_size)
        if need > self.width:
            raise ValueError(f"lane {lane}: {need} pages, the table holds {self.width}")
        have = self.pages[lane]
        if need - len(have) > len(self.free):
            raise MemoryError("no free pages")
        while len(have) < need:
            self.table[lane, len(have)] = self.free[-1]
            have.append(self.free.pop())

    def slots(self, lane: int, n: int) -> list[int]:
        """Cache rows (page * page_size + row) of the next n rows of a lane."""
        at = range(self.rows[lane], self.rows[lane] + n)
        return [self.pages[lane][i // self.page_size] * self.page_size + i % self.page_size for i in at]

    def advance(self, lane: int, rows: int) -> None:
        """The lane has kept `rows` more rows; pages that were reserved for the others stay with it."""
        self.rows[lane] += rows

    def release(self, lane: int) -> None:
        """The lane is done: its pages are free."""
        self.free += self.pages[lane][::-1]
        self.pages[lane], self.rows[lane] = [], 0
        self.table[lane] = -1


class DevicePages:
    """Pages of a cache by lane, kept on the device: the state and the outputs of ``moe_page_plan``.

    ``plan`` gives every lane room for its new tokens; ``kv_len``, ``cu``, ``positions``, ``slots`` and ``idle`` (of `max_tokens`
    tokens; idle: past the last token, or of a lane that was not served) then belong to that batch, and ``advance`` keeps its rows.
    ``table`` int32 [lanes, width]; every layer's cache uses the same one. Nothing here waits for the device."""

    def __init__(self, lanes: int, n_pages: int, page_size: int, width: int, max_tokens: int, device="cuda"):
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.page_size = page_size
        self.rows, self.held, self.kv_len, self.cu = i32(lanes), i32(lanes), i32(lanes), i32(lanes + 1)
        self.table = torch.full((lanes, width), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)       # page 0 on top
        self.n_free = torch.full((1,), n_pages, dtype=torch.int32, device=device)
        self.positions = i32(max_tokens)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        self.idle = torch.ones(max_tokens, dtype=torch.bool, device=device)

    def plan(self, n_new: torch.Tensor) -> None:
        """n_new int32 [lanes] on the device: new tokens of each lane; 0: it waits; below 0: it is done, and its pages are free.
        A lane that cannot be served (no pages, no place) gets kv_len 0 and no slots, and the device status says so."""
        moe_page_plan(n_new, self.rows, self.held, self.table, self.free, self.n_free, self.page_size, self.kv_len, self.cu,
                      self.positions, self.slots)
        torch.lt(self.slots, 0, out=self.idle)

    def advance(self) -> None:
        """The rows of the batch planned last are kept (those of lanes that were not served stay as they were)."""
        self.rows.copy_(torch.maximum(self.rows, self.kv_len))


@dataclass
class HeadNorms:
    """What ``moe_qk_rotate`` does with a layer's queries and keys: `turns` (``rotary.rotary_turns``) of its positions; weights
    fp32 [head_dim] of the norms, or None."""
    turns: torch.Tensor
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    eps: float = 1e-6
    interleaved: bool = False
    magnitude: float = 1.0


def tree_mask(parents: list[int]) -> list[int]:
    """Ancestor bits of each node (its own among them) from the parents' indices, -1 for a root."""
    bits: list[int] = []
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError("a node's parent comes before it")
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


class Step:
    """Device tables of one step of all lanes: `parents[b]` are the drafted nodes of lane b (empty: the lane waits)."""

    def __init__(self, pages: LanePages, parents: list[list[int]], device="cuda"):
        counts = [len(p) for p in parents]
        for b, n in enumerate(counts):
            pages.reserve(b, n)
        self.counts, self.n_nodes, self.max_nodes = counts, sum(counts), max(1, max(counts))
        words = -(-self.max_nodes // 32)
        trees = [tree_mask(p) for p in parents]
        mask = [[(bits >> 32 * w & 0xFFFFFFFF) - ((bits >> 32 * w & 0x80000000) << 1) for w in range(words)]
                for tree in trees for bits in tree]
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        dev = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=device)  # noqa: E731
        self.table = pages.table.to(device, copy=True)       # (complete on return: the host's table may change at once)
        # a node's place in its lane's text: behind the prefix, as deep as it stands in the tree
        places = [r + bits.bit_count() - 1 for r, tree in zip(pages.rows, trees) for bits in tree]
        lens = [r + n for r, n in zip(pages.rows, counts)]
        self.prefix, self.kv_len, self.positions = dev(pages.rows + lens + places).split([len(lens), len(lens), len(places)])
        self.cu = dev(cu)
        self.slots = dev([s for b, n in enumerate(counts) for s in pages.slots(b, n)], torch.int64)
        self.mask = dev(mask).view(-1, words)


def _first_rows(buf: LayerBuffers, n: int) -> LayerBuffers:
    """The buffers of a batch of n tokens inside those of a larger one (the demand update takes its tokens from them)."""
    b = copy.copy(buf)
    b.T = n
    for name in ("want_e", "want_s", "sel_e", "sel_slot", "sel_w", "out"):
        setattr(b, name, getattr(buf, name)[:n])
    return b


class DecodeLayer:
    """Weights, cache and buffers of one layer: grouped-query attention, then the routed experts of `moe_args`.

    w_qkv bf16 [(n_q_heads + 2 * n_kv_heads) * head_dim, d], w_out bf16 [d, n_q_heads * head_dim]; moe_args: (w_router,
    bias, slot_of, arena, demand, miss_max, layer) as for ``layer_step``; buf: its LayerBuffers, for at least
    `max_tokens` tokens; norms: the norms and rotary positions of its queries and keys, or None.
    """

    def __init__(self, w_qkv: torch.Tensor, w_out: torch.Tensor, cache: KvCache, n_q_heads: int, lanes: int, max_tokens: int,
                 moe_args: tuple, buf: LayerBuffers, norms: HeadNorms | None = None):
        self.w_qkv, self.w_out, self.cache, self.moe_args, self.buf = w_qkv, w_out, cache, moe_args, buf
        self.heads, self.scale, self.norms, self.lanes = n_q_heads, cache.head_dim ** -0.5, norms, lanes
        self.chunk_workspace = None          # of the first chunk on
        self.out = torch.zeros((max_tokens, n_q_heads, cache.head_dim), dtype=torch.bfloat16, device=w_qkv.device)
        self.workspace = torch.empty(moe_tree_attention_workspace_bytes(max_tokens, n_q_heads, cache.n_kv_heads, cache.head_dim, lanes),
                                     dtype=torch.uint8, device=w_qkv.device)

    def step(self, hidden: torch.Tensor, tables: Step, tree: bool = True) -> torch.Tensor:
        """hidden bf16 [n_nodes, d] of the step's nodes, lane by lane; returns the layer's bf16 output. tree = False:
        each lane's nodes are a chain (a chunk of its prompt)."""
        n = tables.n_nodes
        if n == 0:                           # every lane waits
            return torch.empty_like(hidden)
        q = self._write(hidden, tables.positions, tables.slots)
        out = self.out[:n]
        moe_tree_attention(q, self.cache, tables.table, tables.kv_len, tables.cu, tables.max_nodes, tables.mask if tree else None,
                           self.scale, out, self.workspace)
        return self._experts(hidden, out)

    def chunk(self, hidden: torch.Tensor, pages: DevicePages) -> torch.Tensor:
        """hidden bf16 [n, d] of the new tokens that `pages` has planned last, lane by lane; returns the layer's bf16 output.
        It may have rows behind them (a batch of one size, for a captured graph): what comes out there means nothing, nor what
        comes out for lanes that were not served, whose tokens attend to nothing; neither is counted as demand."""
        n, H, D = hidden.shape[0], self.cache.n_kv_heads, self.cache.head_dim
        if n > min(self.out.shape[0], pages.slots.shape[0]):
            raise ValueError(f"{n} tokens: the layer has places for {self.out.shape[0]}, the plan for {pages.slots.shape[0]}")
        if n == 0:
            return torch.empty_like(hidden)
        if self.chunk_workspace is None:
            size = moe_chunk_attention_workspace_bytes(self.out.shape[0], self.heads, H, D, self.lanes)
            self.chunk_workspace = torch.empty(size, dtype=torch.uint8, device=hidden.device)
        q = self._write(hidden, pages.positions[:n], pages.slots[:n])
        out = self.out[:n]
        moe_chunk_attention(q, self.cache, pages.table, pages.kv_len, pages.cu, self.scale, out, self.chunk_workspace)
        return self._experts(hidden, out, pages.idle[:n])

    def _write(self, hidden: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
        """Queries of the tokens; their keys and values are in the cache."""
        n, H, D = hidden.shape[0], self.cache.n_kv_heads, self.cache.head_dim
        qkv = hidden @ self.w_qkv.T
        q, k, v = (x.view(n, -1, D) for x in qkv.split([self.heads * D, H * D, H * D], 1))
        if self.norms is not None:
            c = self.norms
            moe_qk_rotate(q, k, positions, c.turns, q, k, q_weight=c.q_weight, k_weight=c.k_weight, eps=c.eps, interleaved=c.interleaved,
                          magnitude=c.magnitude)
        moe_kv_write(k, v, slots, self.cache)
        return q

    def _experts(self, hidden: torch.Tensor, out: torch.Tensor, idle: torch.Tensor | None = None) -> torch.Tensor:
        n = hidden.shape[0]
        x = hidden + out.view(n, -1) @ self.w_out.T
        w_router, bias, slot_of, arena, demand, miss_max, layer = self.moe_args
        y = layer_step(x, w_router, bias, slot_of, arena, demand, miss_max, layer, _first_rows(self.buf, n), idle=idle)
        return (x + y).to(torch.bfloat16)

    def keep(self, tables: Step, path: torch.Tensor, n_keep: torch.Tensor) -> None:
        """Keep the accepted nodes path[b, :n_keep[b]] (ascending) of every lane in this layer's cache."""
        moe_kv_keep(self.cache, tables.table, tables.prefix, path, n_keep)
