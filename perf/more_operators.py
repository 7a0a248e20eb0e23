"""Cases and plain forms of what a chunk of new tokens needs in front of the routed experts.

A server takes prompts in chunks: a batch holds so many new tokens of each of
its lanes (a whole prompt, the next part of a long one, one token of a lane that
decodes). Before the experts run, each layer turns the projection's output into
queries, keys and values, and attends over the lanes' cache rows. Three
operators stand there beside the paged 8-bit key/value cache:

  plan       from the lanes' numbers of new tokens, on the GPU: pages from a free
             stack into the page table (and back from lanes that are done), and
             each token's position and cache slot
  rotate     queries and keys of each head normed and turned by their token's
             position, in one pass
  attention  the new tokens of every lane over the lane's cache rows up to their
             own

Cache: codes [pages, kv heads, page rows, dim], scales [pages, kv heads, page
rows]. Row i of a lane is row i % page of page table[lane, i // page]; table
entries past a lane's rows hold -1.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BASE = 10000.0                 # of the rotary frequencies
LIMIT_FLOPS = 1.13e12          # of the largest listed attention
LIMIT_SCORES = 2.3e9           # its scores, lanes padded to the longest
LIMIT_BYTES = 3.4e8            # of the largest rotation


def listed():
    return [
        # two lanes decode one token each: the plan of such a step
        {"name": "plan_step", "op": "plan", "lanes": 2, "chunk": 1, "length": 8191, "page": 64, "busy": 1.0, "short": False},
        # 256 lanes, most of them decoding, some done, some waiting
        {"name": "plan_lanes", "op": "plan", "lanes": 256, "chunk": 9, "length": 4097, "page": 16, "busy": 0.8, "short": False},
        # a prefill batch of 48 uneven chunks; the pool runs out of pages before its last lanes
        {"name": "plan_chunks", "op": "plan", "lanes": 48, "chunk": 2048, "length": 16384, "page": 32, "busy": 1.0, "short": True},
        # two decoded tokens
        {"name": "rotate_step", "op": "rotate", "tokens": 2, "q_heads": 32, "kv_heads": 8, "dim": 128, "turned": 128,
         "type": "bf16", "norm": True, "interleaved": False, "length": 8192, "stretch": 1.0},
        # 833 tokens of a mixed batch; a quarter of each head turned, pairs side by side, positions stretched for a long context
        {"name": "rotate_mixed", "op": "rotate", "tokens": 833, "q_heads": 20, "kv_heads": 5, "dim": 64, "turned": 16,
         "type": "fp16", "norm": False, "interleaved": True, "length": 131072, "stretch": 8.0},
        # a chunk of 8192 tokens, the largest batch of the benchmark's prefill
        {"name": "rotate_chunk", "op": "rotate", "tokens": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128, "turned": 128,
         "type": "bf16", "norm": True, "interleaved": False, "length": 131072, "stretch": 4.0},
        # one short prompt: latency
        {"name": "attn_short", "op": "attention", "lanes": 1, "chunk": 300, "length": 0, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "ragged": False, "single": 0.0, "lse": True},
        # a whole prompt of 8192 tokens in one chunk
        {"name": "attn_prompt", "op": "attention", "lanes": 1, "chunk": 8192, "length": 0, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "ragged": False, "single": 0.0, "lse": False},
        # prompts of different lengths packed into one batch, a key head for each query head
        {"name": "attn_packed", "op": "attention", "lanes": 24, "chunk": 1531, "length": 0, "q_heads": 16, "kv_heads": 16, "dim": 64,
         "page": 16, "ragged": True, "single": 0.0, "lse": False},
        # the next 1024 tokens of a long prompt
        {"name": "attn_long", "op": "attention", "lanes": 1, "chunk": 1024, "length": 65536, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "ragged": False, "single": 0.0, "lse": False},
        # a mixed batch: two lanes in three decode one token, the others take a chunk, all over prefixes of different lengths
        {"name": "attn_mixed", "op": "attention", "lanes": 33, "chunk": 333, "length": 4095, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 32, "ragged": True, "single": 0.67, "lse": True},
        # wide heads
        {"name": "attn_wide", "op": "attention", "lanes": 3, "chunk": 1025, "length": 7000, "q_heads": 20, "kv_heads": 4, "dim": 256,
         "page": 128, "ragged": True, "single": 0.0, "lse": True},
    ]


def draw(rng):
    def log(a, b):
        return int(min(b, max(a, round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))

    while True:
        op = rng.choice(["plan", "rotate", "attention", "attention"])
        if op == "plan":
            c = {"op": op, "lanes": log(1, 512), "chunk": log(1, 8192), "length": log(1, 65536), "page": rng.choice([16, 32, 64, 128]),
                 "busy": rng.choice([1.0, 0.5, 0.8]), "short": rng.random() < 0.3}
            if c["lanes"] * c["chunk"] > 98304 or c["lanes"] * (c["length"] + c["chunk"]) // c["page"] > 1 << 20:
                continue
            return c
        c = {"op": op, "dim": rng.choice([64, 128, 128, 256]), "kv_heads": rng.choice([1, 2, 3, 4, 5, 8, 16])}
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 8, 16])
        if c["q_heads"] > 128:
            continue
        if op == "rotate":
            c |= {"tokens": log(1, 8192), "turned": c["dim"] // rng.choice([1, 1, 2, 4]), "type": rng.choice(sorted(TYPES)),
                  "norm": rng.random() < 0.6, "interleaved": rng.random() < 0.4, "length": log(1, 1 << 20),
                  "stretch": rng.choice([1.0, 1.0, 2.5, 32.0])}
            if work(c)["bytes"] <= LIMIT_BYTES:
                return c
            continue
        c |= {"lanes": log(1, 64), "chunk": log(1, 8192), "length": rng.choice([0, log(1, 131072)]), "page": rng.choice([16, 32, 64, 128]),
              "ragged": rng.random() < 0.6, "single": rng.choice([0.0, 0.0, 0.5, 0.8]), "lse": rng.random() < 0.5}
        scores = c["lanes"] * c["chunk"] * c["q_heads"] * (c["chunk"] + c["length"])
        if work(c)["flops"] <= LIMIT_FLOPS and scores <= LIMIT_SCORES and c["lanes"] * (c["length"] + c["chunk"]) * c["kv_heads"] * c["dim"] < 1 << 30:
            return c


# ------------------------------------------------------------------ what a case's lanes hold (by the case alone)

def _spread(n, k):
    """n fractions in [0, 1), evenly spread, the first of them 0."""
    return [(i * k) % 1.0 for i in range(n)]


def _lanes(case):
    """(prefix rows, new tokens) of each lane."""
    n, chunk, length = case["lanes"], case["chunk"], case["length"]
    if case["op"] == "plan":
        new = [max(1, chunk - int(chunk * f)) for f in _spread(n, 0.4142135624)]
        for i, f in enumerate(_spread(n, 0.7320508076)):
            if i and f >= case["busy"]:
                new[i] = -1 if (i * 13) % 3 == 0 else 0          # done, or waiting
        return [length - int(length * f) for f in _spread(n, 0.6180339887)], new
    if not case["ragged"]:
        lens, new = [length] * n, [chunk] * n
    else:
        lens = [length - int(length * f) for f in _spread(n, 0.6180339887)]
        new = [chunk - int(chunk * f * f) for f in _spread(n, 0.4142135624)]
        if n > 4:
            new[3] = 0                                           # a lane that waits
    new = [1 if i and f < case["single"] and x else x for i, (f, x) in enumerate(zip(_spread(n, 0.7320508076), new))]
    return lens, new


def work(case):
    if case["op"] == "plan":
        rows, new = _lanes(case)
        tokens = sum(max(0, n) for n in new)
        # per lane: new, rows, held, kv_len, cu; per token: its position and slot; a new page: the stack's entry and the table's
        grown = sum(-(-(r + max(0, n)) // case["page"]) - -(-r // case["page"]) for r, n in zip(rows, new))
        gone = sum(-(-r // case["page"]) for r, n in zip(rows, new) if n < 0)
        return {"bytes": 20 * case["lanes"] + 12 * tokens + 8 * grown + 12 * gone, "flops": 0}
    if case["op"] == "rotate":
        heads, size = case["q_heads"] + case["kv_heads"], TYPES[case["type"]].itemsize
        return {"bytes": case["tokens"] * (heads * case["dim"] * size * 2 + 4), "flops": 0}
    H, D, Q = case["kv_heads"], case["dim"], case["q_heads"]
    lens, new = _lanes(case)
    seen = sum(l + n for l, n in zip(lens, new) if n)
    b = seen * 2 * H * (D + 1) + sum(new) * Q * (D * 2 * 2 + (4 if case["lse"] else 0))
    return {"bytes": b, "flops": sum(4 * D * Q * (n * l + n * (n + 1) // 2) for l, n in zip(lens, new))}


# ------------------------------------------------------------------ inputs

def _values(codes, scales):
    """The values that codes and scales stand for, in 32 bits."""
    s = torch.ldexp(torch.ones((), device=codes.device), scales.to(torch.int32) - 127)
    return codes.view(torch.float8_e4m3fn).float() * s.unsqueeze(-1)


def _cache(gen, pages, H, page, D):
    """A pool of pages with rows in it, as a running server's has: a power of two for each vector, e4m3 codes."""
    got = []
    for key in (True, False):
        codes = torch.empty((pages, H, page, D), dtype=torch.uint8, device="cuda")
        scales = torch.empty((pages, H, page), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (H * page * D))
        for p in range(0, pages, step):
            x = torch.randn(codes[p:p + step].shape, generator=gen, device="cuda")
            if key:                          # a few channels of the keys are much larger than the rest
                x[..., 3::32] *= 6.0
            else:                            # the rows of the values differ in size
                x *= torch.exp(torch.randn(x.shape[:-1], generator=gen, device="cuda")).unsqueeze(-1)
            m, e = torch.frexp(x.abs().amax(-1))
            e = e - 9 + (m > 0.875).to(e.dtype)
            codes[p:p + step] = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
            scales[p:p + step] = (e + 127).to(torch.uint8)
        got += [codes, scales]
    return {"k_codes": got[0], "k_scales": got[1], "v_codes": got[2], "v_scales": got[3]}


def _table(rng, rows, page, width=None, spare=3):
    """A page table for lanes of so many rows, pages in no order; the pool's size; the pages that are left."""
    need = [-(-r // page) for r in rows]
    pages = sum(need) + spare
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(rows), width or max(1, max(need))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, pages, ids[at:]


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _frequencies(case):
    """Radians a position of each turned pair, in 64 bits; a stretched context divides the slow ones (they turn less than
    once in 4096 positions) and leaves the fast ones, with a ramp between (from 32 turns to one)."""
    n = case["turned"] // 2
    f = BASE ** (-np.arange(n, dtype=np.float64) * 2 / case["turned"])
    turns = 4096 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0.0, 1.0)
    return f * keep + f / case["stretch"] * (1 - keep)


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "rotate":
        T, Q, H, D, kind = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
        # queries, keys and values come as one projection's output
        qkv = torch.randn((T, (Q + 2 * H) * D), generator=gen, device="cuda").to(kind)
        s["q"], s["k"] = qkv[:, :Q * D].view(T, Q, D), qkv[:, Q * D:(Q + H) * D].view(T, H, D)
        s["q_out"] = torch.empty((T, Q, D), dtype=kind, device="cuda")
        s["k_out"] = torch.empty((T, H, D), dtype=kind, device="cuda")
        s["positions"] = _dev(rng.randint(0, case["length"], T).astype(np.int32))
        f = _frequencies(case)
        s["frequencies"] = _dev(f)
        # the same as whole numbers of 2^-64 turns
        s["turns"] = _dev(np.array([int(round(x / (2 * math.pi) * 2 ** 64)) for x in f.tolist()], dtype=np.uint64).view(np.int64))
        s["weights"] = [(1 + 0.2 * torch.randn(D, generator=gen, device="cuda")) if case["norm"] else None for _ in range(2)]
        s["eps"] = 1e-6
        s["interleaved"] = case["interleaved"]
        s["magnitude"] = 0.1 * math.log(case["stretch"]) + 1.0
        return s
    page = case["page"]
    s["page"] = page
    rows, new = _lanes(case)
    order = rng.permutation(len(rows))
    rows, new = [rows[i] for i in order], [new[i] for i in order]
    if op == "plan":
        grown = sum(-(-(r + max(0, n)) // page) - -(-r // page) for r, n in zip(rows, new))
        width = max(-(-(r + max(0, n)) // page) for r, n in zip(rows, new)) + 1
        gone = sum(-(-r // page) for r, n in zip(rows, new) if n < 0)
        spare = max(0, grown * 3 // 4 - gone) if case["short"] else grown + 5
        table, pages, left = _table(rng, rows, page, width, spare)
        free = np.full(pages, -1, np.int32)
        free[:len(left)] = left
        s |= {"table": _dev(table), "free": _dev(free), "n_free": _dev(np.array([len(left)], np.int32)), "rows": _dev(np.array(rows, np.int32)),
              "held": _dev(np.array([-(-r // page) for r in rows], np.int32)), "new": _dev(np.array(new, np.int32))}
        tokens = sum(max(0, n) for n in new)
        T = tokens + tokens // 8 + 1         # the batch's room; places past the last token are told apart
        s |= {"kv_len": torch.empty(len(rows), dtype=torch.int32, device="cuda"), "cu": torch.empty(len(rows) + 1, dtype=torch.int32, device="cuda"),
              "positions": torch.empty(T, dtype=torch.int32, device="cuda"), "slots": torch.empty(T, dtype=torch.int64, device="cuda")}
        return s
    H, Q, D = case["kv_heads"], case["q_heads"], case["dim"]
    table, pages, _ = _table(rng, [a + b for a, b in zip(rows, new)], page)
    s |= _cache(gen, pages, H, page, D)
    N = sum(new)
    s |= {"table": _dev(table), "rows": rows, "new": new, "scale": D ** -0.5}
    s["cu"] = _dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    s["kv_len"] = _dev(np.array([a + b for a, b in zip(rows, new)], np.int32))
    s["q"] = torch.randn((N, (Q + 2 * H) * D), generator=gen, device="cuda").bfloat16()[:, :Q * D].view(N, Q, D)
    s["out"] = torch.empty((N, Q, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((N, Q), dtype=torch.float32, device="cuda") if case["lse"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else {"plan": _plan, "rotate": _rotate, "attention": _attention}[s["op"]](s)


def _planned(s):
    return {x: s[x] for x in ("table", "free", "n_free", "rows", "held", "kv_len", "cu", "positions", "slots")}


def _run_own(s):
    import resident_expert_routed_gb300 as moe

    if s["op"] == "plan":
        moe.moe_page_plan(s["new"], s["rows"], s["held"], s["table"], s["free"], s["n_free"], s["page"], s["kv_len"], s["cu"], s["positions"], s["slots"])
        return _planned(s)
    if s["op"] == "rotate":
        moe.moe_qk_rotate(s["q"], s["k"], s["positions"], s["turns"], s["q_out"], s["k_out"], q_weight=s["weights"][0], k_weight=s["weights"][1],
                          eps=s["eps"], interleaved=s["interleaved"], magnitude=s["magnitude"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cache = moe.KvCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    if "workspace" not in s:                 # a user keeps one for all layers and steps
        n = moe.moe_chunk_attention_workspace_bytes(s["q"].shape[0], s["q"].shape[1], cache.n_kv_heads, cache.head_dim, len(s["rows"]))
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_chunk_attention(s["q"], cache, s["table"], s["kv_len"], s["cu"], s["scale"], s["out"], s["workspace"], lse=s["lse"])
    return {"out": s["out"]} | ({"lse": s["lse"]} if s["lse"] is not None else {})


def _plan(s):
    page, new, rows, held, table, free, n_free = (s[x] for x in ("page", "new", "rows", "held", "table", "free", "n_free"))
    (B, W), n, T = table.shape, free.numel(), s["slots"].numel()
    col, dev = torch.arange(W, device="cuda"), table.device
    # pages of lanes that are done go to the stack's top, in the lanes' order
    done = new < 0
    back = done.unsqueeze(1) & (col < held.unsqueeze(1))
    at = torch.where(back, n_free + torch.cumsum(back.view(-1), 0).view(B, W) - 1, n)
    stack = torch.cat([free, torch.zeros(1, dtype=torch.int32, device=dev)])
    stack.scatter_(0, at.view(-1).long(), table.view(-1))
    free.copy_(stack[:n])
    there = n_free + back.sum()
    table.masked_fill_(done.unsqueeze(1), -1)
    rows.masked_fill_(done, 0)
    held.masked_fill_(done, 0)
    # a lane gets its pages where all lanes' up to it are there and its rows and tokens fit
    more = new.clamp(min=0)
    last = torch.cumsum(more, 0)
    pages = (rows + more + page - 1) // page
    fits = (pages <= W) & (last <= T)
    need = torch.where(fits & (more > 0), (pages - held).clamp(min=0), torch.zeros_like(held))
    upto = torch.cumsum(need, 0)
    ok = (more == 0) | (fits & ((upto <= there) | (need == 0)))
    need = torch.where(ok, need, torch.zeros_like(need))
    # the i-th page from the stack's top; lanes that get none stand behind those that do
    i = col - held.unsqueeze(1)
    gets = (i >= 0) & (i < need.unsqueeze(1))
    at = torch.where(gets, there - 1 - ((upto - need).unsqueeze(1) + i), 0).clamp(0, n - 1)
    table.copy_(torch.where(gets, free[at.long()], table))
    held.add_(need.to(torch.int32))
    n_free.copy_(there - need.sum())
    s["kv_len"].copy_(torch.where(ok, rows + more, torch.zeros_like(rows)))
    s["cu"][0] = 0
    s["cu"][1:] = last.clamp(max=T)
    t = torch.arange(T, device=dev)
    lane = torch.searchsorted(s["cu"][1:], t, right=True)
    on, lane = lane < B, lane.clamp(max=B - 1)
    pos = torch.where(on, rows[lane] + t - s["cu"][lane], 0)
    s["positions"].copy_(pos)
    on &= ok[lane]
    where = table[lane, (pos // page).clamp(max=W - 1)].long()
    s["slots"].copy_(torch.where(on, where * page + pos % page, -1))
    return _planned(s)


def _rotate(s):
    # angles of far positions: 32 bits would lose them
    angle = s["positions"].double().unsqueeze(1) * s["frequencies"]
    cos, sin = ((f(angle) * s["magnitude"]).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    got = {}
    for name, weight in zip("qk", s["weights"]):
        x = s[name].float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight
        n = 2 * s["frequencies"].numel()
        turned = x[..., :n]
        a, b = (turned[..., 0::2], turned[..., 1::2]) if s["interleaved"] else (turned[..., :n // 2], turned[..., n // 2:])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        got[name] = s[name + "_out"].copy_(torch.cat([turned, x[..., n:]], -1))
    return got


def _attention(s):
    page, q, (N, Q, D) = s["page"], s["q"], s["q"].shape
    B, H = s["table"].shape[0], s["k_codes"].shape[1]
    most, n = max(a + b for a, b in zip(s["rows"], s["new"])), max(s["new"])
    pos = torch.arange(most, device="cuda")
    where = s["table"][:, pos // page].long().clamp(min=0)
    keys, values = (_values(s[x + "_codes"][where, :, pos % page], s[x + "_scales"][where, :, pos % page]) for x in "kv")    # [B, L, H, D]
    row = torch.arange(N, device="cuda", dtype=torch.int32)
    lane = torch.searchsorted(s["cu"], row, right=True) - 1
    i = (row - s["cu"][lane]).long()
    padded = torch.zeros((B, n, Q, D), device="cuda")
    padded[lane, i] = q.float()
    x = padded.view(B, n, H, Q // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, Q // H * n, D)
    score = torch.matmul(x, keys.permute(0, 2, 3, 1)).view(B, H, Q // H, n, most)
    score *= s["scale"]
    total = s["kv_len"].long()
    prefix = total - (s["cu"][1:] - s["cu"][:-1])
    own_row = prefix.unsqueeze(1) + torch.arange(n, device="cuda")                                                            # [B, n]
    hidden = pos > own_row.unsqueeze(2)
    score.masked_fill_(hidden.view(B, 1, 1, n, most), float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    whole = p.sum(-1, keepdim=True)
    # rows behind a lane's last hold another lane's, or anything
    values = torch.where((pos < total.unsqueeze(1))[:, :, None, None], values, torch.zeros_like(values))
    o = torch.matmul(p.view(B, H, Q // H * n, most), values.permute(0, 2, 1, 3)).view(B, H, Q // H, n, D) / whole
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, n, Q, D)[lane, i])
    got = {"out": s["out"]}
    if s["lse"] is not None:
        s["lse"].copy_((top + torch.log(whole)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, Q)[lane, i])
        got["lse"] = s["lse"]
    return got


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":                    # whole numbers: one lane after the other
        page, T = s["page"], s["slots"].numel()
        new, rows, held, free, n = (s[x].tolist() for x in ("new", "rows", "held", "free", "n_free"))
        table, n = s["table"].cpu().numpy().copy(), n[0]
        for b, k in enumerate(new):
            if k < 0:
                free[n:n + held[b]] = table[b, :held[b]].tolist()
                n += held[b]
                table[b], rows[b], held[b] = -1, 0, 0
        kv_len, cu, positions, slots, asked, there = [], [0], [0] * T, [-1] * T, 0, n
        for b, k in enumerate(new):
            k, first = max(k, 0), cu[-1]
            cu.append(min(T, sum(max(x, 0) for x in new[:b + 1])))
            want = -(-(rows[b] + k) // page)
            need = max(0, want - held[b]) if k and want <= table.shape[1] and first + k <= T else 0
            asked += need
            fine = k == 0 or (want <= table.shape[1] and first + k <= T and (need == 0 or asked <= there))
            for i in range(need if fine else 0):
                n -= 1
                table[b, held[b] + i] = free[n]
            held[b] += need if fine else 0
            kv_len.append(rows[b] + k if fine else 0)
            for t in range(first, cu[-1]):
                at = rows[b] + t - first
                positions[t] = at
                slots[t] = int(table[b, at // page]) * page + at % page if fine else -1
        kinds = {"slots": np.int64}
        got = {"table": table, "free": free, "n_free": [n], "rows": rows, "held": held, "kv_len": kv_len, "cu": cu, "positions": positions, "slots": slots}
        return {x: np.array(v, kinds.get(x, np.int32)) for x, v in got.items()}
    if s["op"] == "rotate":
        got, n = {}, case["turned"]
        angle = s["positions"].double()[:, None] * s["frequencies"]
        turn = torch.polar(torch.full_like(angle, s["magnitude"]), angle)[:, None]
        for name, weight in zip("qk", s["weights"]):
            x = s[name].double()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * weight.double()
            y = x.clone()
            first, second = (slice(0, n, 2), slice(1, n, 2)) if case["interleaved"] else (slice(0, n // 2), slice(n // 2, n))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            y[..., first], y[..., second] = z.real, z.imag
            got[name] = y
        return got
    (N, Q, D), H, page, at = s["q"].shape, s["k_codes"].shape[1], s["page"], 0
    out = torch.zeros((N, Q, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((N, Q), dtype=torch.float64, device="cuda")
    for b, (length, n) in enumerate(zip(s["rows"], s["new"])):
        if not n:
            continue
        ids = s["table"][b, :-(-(length + n) // page)].long()
        for h in range(H):
            k, v = (s[x + "_codes"][ids, h].view(torch.float8_e4m3fn).double().reshape(-1, D) *
                    torch.exp2(s[x + "_scales"][ids, h].double() - 127).reshape(-1, 1) for x in "kv")
            for j in range(h * (Q // H), (h + 1) * (Q // H)):
                for first in range(0, n, 1024):
                    m = min(n, first + 1024) - first
                    rows = slice(at + first, at + first + m)
                    seen = length + first + m
                    z = s["q"][rows, j].double() @ k[:seen].T * s["scale"]
                    z[torch.arange(seen, device="cuda") > length + first + torch.arange(m, device="cuda")[:, None]] = -math.inf
                    lse[rows, j] = torch.logsumexp(z, -1)
                    out[rows, j] = torch.softmax(z, -1) @ v[:seen]
        at += n
    return {"out": out} | ({"lse": lse} if s["lse"] is not None else {})
