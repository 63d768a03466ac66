"""Cases of the tree-verification and cache-eviction operators.

Five operators work on one paged KV cache. A drafter proposes a tree of
tokens (``mask``: parents to ancestor bits), one attention call verifies every
node over the cache (``tree``), and the accepted path's rows become the cache
(``commit``). The attention weight that each cached token has drawn is summed
over the steps (``weights``), and the tokens that drew least leave the cache
when it outgrows its budget (``evict``).

``run`` computes a case in its plain form, elementary torch operations in 32
bits, or, with ``own`` set, by the framework's calls.
"""
import math

import torch

own = False

BLOCK = 16          # tokens per block of the pool
DIM = 128           # head dimension
TILE = 2112         # bytes of an 8-bit (block, KV head) tile: 16 x 128 codes, 16 fp32 scales
SCALE = 1.0 / math.sqrt(DIM)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the drafter's tree of a handful of interactive requests
        {"name": "mask_small", "op": "mask", "seqs": 4, "nodes_lo": 8, "nodes_hi": 8},
        # a full serving batch, each request with a tree of its own size
        {"name": "mask_batch", "op": "mask", "seqs": 256, "nodes_lo": 20, "nodes_hi": 64},
        # four chats just begun, seven drafted tokens each: the call's latency is all there is
        {"name": "tree_first", "op": "tree", "seqs": 4, "ctx_lo": 128, "ctx_hi": 384,
         "nodes_lo": 7, "nodes_hi": 7, "hq": 16, "hkv": 8},
        # the verify half of a mixed batch, trees of 17 to 33 nodes over contexts up to 8192
        {"name": "tree_batch", "op": "tree", "seqs": 48, "ctx_lo": 256, "ctx_hi": 8192,
         "nodes_lo": 17, "nodes_hi": 33, "hq": 16, "hkv": 8},
        # long documents with wide trees and four query heads to a KV head
        {"name": "tree_long", "op": "tree", "seqs": 8, "ctx_lo": 30011, "ctx_hi": 32768,
         "nodes_lo": 64, "nodes_hi": 64, "hq": 16, "hkv": 4},
        # the accepted tokens of the four chats
        {"name": "commit_first", "op": "commit", "seqs": 4, "ctx_lo": 128, "ctx_hi": 384,
         "nodes_lo": 7, "nodes_hi": 7, "path_hi": 4, "hkv": 8, "format": "bf16"},
        # a full serving batch over an 8-bit pool, up to nine tokens accepted
        {"name": "commit_batch", "op": "commit", "seqs": 256, "ctx_lo": 100, "ctx_hi": 1500,
         "nodes_lo": 20, "nodes_hi": 64, "path_hi": 9, "hkv": 8, "format": "int8"},
        # one decode step of a ragged continuous batch, weights summed on
        {"name": "weights_step", "op": "weights", "seqs": 256, "ctx_lo": 1, "ctx_hi": 4096,
         "q_lo": 1, "q_hi": 1, "hq": 16, "hkv": 8, "format": "bf16", "add": True},
        # the same for long documents over an FP8 pool
        {"name": "weights_long", "op": "weights", "seqs": 8, "ctx_lo": 30011, "ctx_hi": 32768,
         "q_lo": 1, "q_hi": 1, "hq": 16, "hkv": 8, "format": "fp8", "add": True},
        # prompts just prefilled, scored by their last 64 queries before the first eviction
        {"name": "weights_window", "op": "weights", "seqs": 16, "ctx_lo": 1000, "ctx_hi": 8192,
         "q_lo": 64, "q_hi": 64, "hq": 16, "hkv": 8, "format": "bf16", "add": False},
        # a serving batch that has grown a few blocks over its budget
        {"name": "evict_step", "op": "evict", "seqs": 32, "ctx_lo": 1030, "ctx_hi": 1153,
         "budget": 1024, "sinks": 4, "recent": 256, "hkv": 8, "format": "bf16"},
        # long prompts cut to an eighth after their prefill, over an int8 pool
        {"name": "evict_prompt", "op": "evict", "seqs": 8, "ctx_lo": 30011, "ctx_hi": 32768,
         "budget": 4096, "sinks": 16, "recent": 1000, "hkv": 8, "format": "int8"},
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    case = _draw(rng)
    # at most the largest listed work of its kind
    most = {"mask": (2e5, 0), "tree": (8.4e8, 1.3e11), "commit": (5.4e6, 0),
            "weights": (2.8e8, 1.9e10), "evict": (2.7e8, 0)}[case["op"]]
    while case["seqs"] > 1 and (work(case)["bytes"] > most[0] or work(case)["flops"] > most[1]):
        case["seqs"] = max(1, case["seqs"] * 3 // 4)
    return case


def _draw(rng):
    op = rng.choice(["mask", "tree", "tree", "tree", "commit", "weights", "weights", "weights",
                     "evict", "evict"])
    fmt = rng.choice(["bf16", "int8", "fp8"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 2, 3, 4, 8])
    if op == "mask":
        hi = _log(rng, 8, 400)
        return {"op": op, "seqs": _log(rng, 1, 256 if hi <= 64 else 32),
                "nodes_lo": rng.randint(4, hi), "nodes_hi": hi}
    if op == "commit":
        nodes = _log(rng, 1, 128)
        ctx = max(nodes, _log(rng, 16, 4096))
        return {"op": op, "seqs": _log(rng, 1, 256), "ctx_lo": rng.randint(max(nodes, ctx // 4), ctx),
                "ctx_hi": ctx, "nodes_lo": rng.randint(1, nodes), "nodes_hi": nodes,
                "path_hi": rng.randint(1, min(nodes, 16)), "hkv": hkv, "format": fmt}
    ctx = _log(rng, 64, 32768)
    seqs = _log(rng, 1, 128)
    lo = rng.randint(max(2, ctx // 8), ctx)
    if op == "tree":
        nodes = min(ctx, _log(rng, 1, 128))
        return {"op": op, "seqs": seqs, "ctx_lo": max(nodes, lo), "ctx_hi": ctx,
                "nodes_lo": rng.randint(1, nodes), "nodes_hi": nodes, "hq": hkv * group,
                "hkv": hkv}
    if op == "weights":
        q = rng.choice([1, min(ctx, _log(rng, 2, 512))])
        q = max(1, min(q, int(1.5e8 // (group * hkv * ctx))))  # for the plain form's score matrix
        return {"op": op, "seqs": seqs, "ctx_lo": max(q, lo), "ctx_hi": ctx,
                "q_lo": rng.randint(1, q), "q_hi": q, "hq": hkv * group, "hkv": hkv,
                "format": fmt, "add": rng.random() < 0.5}
    budget = rng.randint(max(2, ctx // 8), ctx)
    sinks = rng.randint(0, min(8, budget // 2))
    return {"op": op, "seqs": seqs, "ctx_lo": lo, "ctx_hi": ctx, "budget": budget,
            "sinks": sinks, "recent": rng.randint(0, (budget - sinks) // 2), "hkv": hkv,
            "format": fmt}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _lengths(g, lo, hi, n, log=False):
    """n lengths spread evenly over lo .. hi (over their logarithm: log), in
    random order. Another seed has the same lengths in another order."""
    at = [(i + 0.5) / n for i in range(n)]
    if log:
        got = [int(min(hi, max(lo, math.exp(u * math.log(hi + 1))))) for u in at]
    else:
        got = [int(min(hi, lo + u * (hi - lo + 1))) for u in at]
    order = torch.randperm(n, generator=g, device="cuda")
    return torch.tensor(got, device="cuda")[order]


def _randn(g, shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _pool(g, blocks, hkv, fmt, heavy=0.0, gain=1.0):
    """One pool array in the framework's layout. A share of `heavy` of the rows
    are `gain` times as long as the others."""
    if fmt == "bf16":
        x = _randn(g, (blocks, hkv, BLOCK, DIM))
        if heavy:
            x *= torch.where(torch.rand((blocks, hkv, BLOCK, 1), generator=g, device="cuda") < heavy,
                             gain, 1.0).to(x.dtype)
        return x
    tile = torch.empty((blocks, hkv, TILE), dtype=torch.uint8, device="cuda")
    rows = blocks * hkv * BLOCK
    scales = 2.5 + torch.rand((rows,), generator=g, device="cuda")  # largest magnitude of a row
    if heavy:
        scales *= torch.where(torch.rand((rows,), generator=g, device="cuda") < heavy, gain, 1.0)
    x = _randn(g, (rows, DIM)).float().clamp_(-2.5, 2.5).div_(2.5)
    if fmt == "int8":
        codes = (x * 127).round_().to(torch.int8).view(torch.uint8)
        scales = scales / 127
    else:
        codes = (x * 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scales = scales / 448
    tile[..., :BLOCK * DIM] = codes.reshape(blocks, hkv, BLOCK * DIM)
    tile[..., BLOCK * DIM:] = scales.view(torch.uint8).reshape(blocks, hkv, BLOCK * 4)
    return tile


def _offsets(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)


def _parents(g, cu, total):
    """A random tree for each sequence: a node's parent is an earlier node of
    its window, or -1 where it follows the cached context directly."""
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    j = at - cu[seq]
    u = torch.rand((total,), generator=g, device="cuda", dtype=torch.float64)
    return ((u * (j + 1)).floor().to(torch.int64).clamp(max=j) - 1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, seqs = case["op"], case["seqs"]
    s = {"op": op}
    if op in ("mask", "tree", "commit"):
        nodes = _lengths(g, case["nodes_lo"], case["nodes_hi"], seqs)
    elif op == "weights":
        nodes = _lengths(g, case["q_lo"], case["q_hi"], seqs)
    else:
        nodes = None
    if nodes is not None:
        s["q_max"] = int(nodes.max())
        s["cu"] = _offsets(nodes)
        s["total"] = int(nodes.sum())
    if op in ("mask", "tree"):
        s["parents"] = _parents(g, s["cu"], s["total"])
        s["mask"] = torch.zeros((s["total"], (s["q_max"] + 31) // 32), dtype=torch.int32,
                                device="cuda")
        s["depths"] = torch.zeros((s["total"],), dtype=torch.int32, device="cuda")
    if op == "mask":
        return s
    # a shuffled pool, some of it held by others
    # (the lengths of a continuous batch are log-uniform)
    lens = _lengths(g, case["ctx_lo"], case["ctx_hi"], seqs, log=case["ctx_lo"] == 1)
    per = (lens + BLOCK - 1) // BLOCK
    width = int(per.max())
    need = int(per.sum())
    blocks = need + need // 10 + 1
    ids = torch.randperm(blocks, generator=g, device="cuda")
    col = torch.arange(width, device="cuda")
    flat = (per.cumsum(0) - per)[:, None] + col
    used = col < per[:, None]
    s["tables"] = torch.where(used, ids[flat.clamp(max=blocks - 1)], -1).to(torch.int32).contiguous()
    s["lens"] = lens.to(torch.int32)
    s["new_lens"] = torch.zeros_like(s["lens"])
    hkv = case["hkv"]
    fmt = case.get("format", "bf16")
    s["format"] = fmt
    if op == "tree":
        # outlier keys in one row of a hundred
        s["k"] = _pool(g, blocks, hkv, fmt, 0.01, 8.0)
        s["v"] = _pool(g, blocks, hkv, fmt)
        s["q"] = _randn(g, (s["total"], case["hq"], DIM))
        s["mask"].copy_(_plain_mask(s)[0])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((s["total"], case["hq"]), dtype=torch.float32, device="cuda")
    elif op == "commit":
        s["k"], s["v"] = _pool(g, blocks, hkv, fmt), _pool(g, blocks, hkv, fmt)
        # a path of increasing nodes of the window, of one node up to path_hi
        p = case["path_hi"]
        n = torch.minimum(_ints(g, 1, p, seqs), nodes)
        key = torch.rand((seqs, s["q_max"]), generator=g, device="cuda")
        key = torch.where(torch.arange(s["q_max"], device="cuda") < nodes[:, None], key, 2.0)
        some = key.argsort(1)[:, :p]  # distinct nodes in random order
        some = torch.where(torch.arange(some.shape[1], device="cuda") < n[:, None], some, 1 << 20)
        some = torch.nn.functional.pad(some.sort(1).values, (0, p - some.shape[1]), value=1 << 20)
        s["path"] = torch.where(some < (1 << 20), some, -1).to(torch.int32).contiguous()
        s["path_lens"] = n.to(torch.int32)
    elif op == "weights":
        # keys that draw more than the others, as the heavy hitters of a text
        s["k"] = _pool(g, blocks, hkv, fmt, 0.02, 2.5)
        s["q"] = _randn(g, (s["total"], case["hq"], DIM))
        # what some sixteen earlier steps have left
        s["weights"] = torch.rand((seqs, hkv, width * BLOCK), generator=g, device="cuda")
        s["weights"] *= (32 * case["hq"] / hkv / lens)[:, None, None]
        s["add"] = bool(case["add"])
        z, sees = _scores(s)
        z = torch.where(sees, z, -math.inf)
        _, inside, at = _window(s)
        lse = torch.logsumexp(z, -1).permute(0, 3, 1, 2)       # [S, L, Hkv, G]
        s["lse"] = lse[inside].reshape(s["total"], case["hq"]).contiguous()
    else:
        s["k"], s["v"] = _pool(g, blocks, hkv, fmt), _pool(g, blocks, hkv, fmt)
        u = torch.rand((seqs, hkv, width * BLOCK), generator=g, device="cuda")
        # a heavy tail, and one token in ten that nothing has looked at
        s["weights"] = torch.where(u < 0.1, 0.0, 0.02 / (1.0001 - u)).float()
        s["budget"] = case["budget"]
        s["budgets"] = torch.full((seqs,), case["budget"], dtype=torch.int32, device="cuda")
        s["sinks"], s["recent"] = case["sinks"], case["recent"]
        s["kept"] = torch.zeros((seqs, hkv, case["budget"]), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _window(s):
    """Query rows of a ragged batch as [S, L]: index into the rows, and which are real."""
    cu = s["cu"].to(torch.int64)
    n = cu[1:] - cu[:-1]
    j = torch.arange(s["q_max"], device="cuda")
    inside = j < n[:, None]
    return n, inside, torch.where(inside, cu[:-1, None] + j, 0)


def _rows(x, tables, fmt):
    """The cached rows of every sequence in 32 bits: [S, Hkv, positions, D]."""
    S, width = tables.shape
    t = x[tables.clamp(min=0).to(torch.int64)]
    if fmt == "bf16":
        r = t.float()
    else:
        codes = t[..., :BLOCK * DIM].contiguous()
        codes = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
        scales = t[..., BLOCK * DIM:].contiguous().view(torch.float32)
        r = codes.reshape(*scales.shape, DIM) * scales[..., None]
    return r.permute(0, 2, 1, 3, 4).reshape(S, r.shape[2], width * BLOCK, DIM)


def _plain_mask(s):
    """Ancestors from the parents: with P the parent matrix of a window,
    (I - P)^-1 = I + P + P^2 + ... has a one for a node and each of its ancestors."""
    n, inside, at = _window(s)
    L = s["q_max"]
    parent = torch.where(inside, s["parents"][at].to(torch.int64), -1)
    link = (parent[..., None] == torch.arange(L, device="cuda")).double()
    eye = torch.eye(L, device="cuda", dtype=torch.float64).expand_as(link)
    seen = torch.linalg.solve_triangular(eye - link, eye, upper=False, unitriangular=True) > 0.5
    depths = seen.sum(-1) - 1
    words = (L + 31) // 32
    bits = torch.nn.functional.pad(seen, (0, words * 32 - L)).reshape(*seen.shape[:2], words, 32)
    word = (bits.to(torch.int64) << torch.arange(32, device="cuda")).sum(-1)
    word = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    return word[inside], depths[inside].to(torch.int32)


def _scores(s):
    """Scaled scores [S, Hkv, G, L, positions] of a window's queries, and what a causal window sees."""
    n, inside, at = _window(s)
    k = _rows(s["k"], s["tables"], s["format"])
    S, hkv, C, _ = k.shape
    q = s["q"][at].float()                                     # [S, L, Hq, D]
    G, L = q.shape[2] // hkv, q.shape[1]
    q = q.reshape(S, L, hkv, G, DIM).permute(0, 2, 3, 1, 4).reshape(S, hkv, G * L, DIM)
    z = (torch.matmul(q, k.transpose(-1, -2)) * SCALE).reshape(S, hkv, G, L, C)
    c = s["lens"].to(torch.int64)
    last = (c - n)[:, None] + torch.arange(L, device="cuda")   # [S, L]
    sees = (torch.arange(C, device="cuda") <= last[..., None]) & inside[..., None]
    return z, sees[:, None, None]


def _plain_tree(s):
    n, inside, at = _window(s)
    z, _ = _scores(s)
    S, hkv, G, L, C = z.shape
    c = s["lens"].to(torch.int64)
    p = torch.arange(C, device="cuda")
    i = p - (c - n)[:, None]                                   # key's place in the window
    word = s["mask"][at].to(torch.int64)                       # [S, L, words]
    w = (i // 32).clamp(0, word.shape[-1] - 1)
    got = torch.gather(word, 2, w[:, None].expand(S, L, C)) >> (i % 32)[:, None]
    sees = torch.where((i < 0)[:, None], True, (got & 1) == 1)
    sees = (sees & (p < c[:, None])[:, None])[:, None, None]
    z = torch.where(sees, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    v = _rows(s["v"], s["tables"], s["format"])
    v = torch.where((p < c[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(e.reshape(S, hkv, G * L, C), v).reshape(S, hkv, G, L, DIM)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
    return {"out": o[inside].reshape(s["q"].shape).to(torch.bfloat16),
            "lse": lse[inside].reshape(s["q"].shape[:2])}


def _move(x, s, src, dst):
    """Rows src of every (sequence, KV head) to dst, both [S, Hkv, n]. Where they
    are equal nothing changes."""
    heads = torch.arange(src.shape[1], device="cuda")[None, :, None]
    t = s["tables"].to(torch.int64)
    seqs = torch.arange(src.shape[0], device="cuda")[:, None, None]
    if s["format"] == "bf16":
        x[t[seqs, dst // BLOCK], heads, dst % BLOCK] = x[t[seqs, src // BLOCK], heads, src % BLOCK]
        return
    codes = x[..., :BLOCK * DIM].unflatten(-1, (BLOCK, DIM))
    scales = x[..., BLOCK * DIM:].unflatten(-1, (BLOCK, 4))
    codes[t[seqs, dst // BLOCK], heads, dst % BLOCK] = \
        codes[t[seqs, src // BLOCK], heads, src % BLOCK]
    scales[t[seqs, dst // BLOCK], heads, dst % BLOCK] = \
        scales[t[seqs, src // BLOCK], heads, src % BLOCK]


def _plain_commit(s):
    c = s["lens"].to(torch.int64)[:, None]
    cu = s["cu"].to(torch.int64)
    p0 = c - (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(s["path"].shape[1], device="cuda")
    real = i < s["path_lens"][:, None]
    src = torch.where(real, p0 + s["path"], p0)
    dst = torch.where(real, p0 + i, p0)
    # what is not on the path writes the row that the path's first node gets
    src = torch.where(real, src, p0 + s["path"][:, :1])
    hkv = s["k"].shape[1]
    src, dst = (x[:, None].expand(-1, hkv, -1) for x in (src, dst))
    _move(s["k"], s, src, dst)
    _move(s["v"], s, src, dst)
    s["new_lens"].copy_((p0[:, 0] + s["path_lens"]).to(torch.int32))
    return {"k": s["k"], "v": s["v"], "new_lens": s["new_lens"]}


def _plain_weights(s):
    n, inside, at = _window(s)
    z, sees = _scores(s)
    S, hkv, G, L, C = z.shape
    lse = s["lse"][at].reshape(S, L, hkv, G).permute(0, 2, 3, 1)[..., None]
    drawn = torch.where(sees, torch.exp(z - lse), 0.0).sum((2, 3))  # [S, Hkv, positions]
    c = s["lens"].to(torch.int64)
    p = torch.arange(C, device="cuda")
    old = (p < (c - n)[:, None])[:, None]
    if s["add"]:
        drawn = torch.where(old, s["weights"] + drawn, drawn)
    s["weights"].copy_(torch.where((p < c[:, None])[:, None], drawn, s["weights"]))
    return s["weights"]


def _plain_evict(s):
    w = s["weights"]
    S, hkv, C = w.shape
    c = s["lens"].to(torch.int64)[:, None, None]
    budget = s["budgets"].to(torch.int64)[:, None, None]
    p = torch.arange(C, device="cuda")
    held = (p < s["sinks"]) | (p >= c - s["recent"])
    key = torch.where(p < c, torch.where(held, math.inf, w), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, p.expand_as(order))
    keep = (rank < budget) & (p < c)
    n = torch.minimum(c, budget)
    kept = torch.where(keep, p, C).sort(-1).values
    i = torch.arange(s["budget"], device="cuda")
    kept = torch.nn.functional.pad(kept, (0, max(0, s["budget"] - C)), value=C)[..., :s["budget"]]
    real = i < n
    src = torch.where(real, kept, torch.minimum(i, c - 1))
    dst = torch.where(real, i, torch.minimum(i, c - 1)).expand_as(src)
    _move(s["k"], s, src, dst)
    _move(s["v"], s, src, dst)
    w.scatter_(-1, dst, torch.gather(w, -1, src))
    s["kept"].copy_(torch.where(real, kept, -1))
    s["new_lens"].copy_(n[:, 0, 0])
    return {"k": s["k"], "v": s["v"], "weights": w, "kept": s["kept"], "new_lens": s["new_lens"]}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _call(s):
    """The prepared call on a state's buffers, as a serving loop keeps it."""
    from paged_kv_decode_18_gb300 import binding as B
    op = s["op"]
    if op == "mask":
        return B.prepare_tree_mask(s["parents"], s["cu"], s["q_max"], s["mask"], s["depths"])
    if op == "tree":
        shape = B.shape_of(s["q"], s["k"], s["tables"])
        room = B.workspace(B.pa_decode_tree_workspace_size(shape, s["total"], s["q_max"]))
        return B.prepare_decode_tree(s["q"], s["k"], s["v"], s["tables"], s["lens"], s["cu"],
                                     s["mask"], s["q_max"], SCALE, s["out"], s["lse"],
                                     workspace=room)
    if op == "commit":
        return B.prepare_commit_path(s["k"], s["v"], s["tables"], s["lens"], s["cu"], s["path"],
                                     s["path_lens"], s["new_lens"])
    if op == "weights":
        kind = {"bf16": B.PA_KV_BF16, "int8": B.PA_KV_INT8, "fp8": B.PA_KV_FP8}[s["format"]]
        return B.prepare_accumulate_weights(s["q"], s["k"], s["lse"], s["tables"], s["lens"],
                                            SCALE, s["weights"], cu_seqlens_q=s["cu"],
                                            max_q_len=s["q_max"], accumulate=s["add"],
                                            kv_format=kind)
    return B.prepare_evict(s["k"], s["v"], s["tables"], s["lens"], s["weights"], s["budgets"],
                           s["sinks"], s["recent"], s["kept"], s["new_lens"])


def _own(s):
    if "call" not in s:
        s["call"] = _call(s)
    s["call"]()
    op = s["op"]
    if op == "mask":
        return s["mask"], s["depths"]
    if op == "tree":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "commit":
        return {"k": s["k"], "v": s["v"], "new_lens": s["new_lens"]}
    if op == "weights":
        return s["weights"]
    return {"k": s["k"], "v": s["v"], "weights": s["weights"], "kept": s["kept"],
            "new_lens": s["new_lens"]}


def run(state):
    if own:
        return _own(state)
    return {"mask": _plain_mask, "tree": _plain_tree, "commit": _plain_commit,
            "weights": _plain_weights, "evict": _plain_evict}[state["op"]](state)


# ---------------------------------------------------------------------------
# floors and exact results
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations for the middle of the case's ranges."""
    op, S = case["op"], case["seqs"]
    row = {"bf16": 256, "int8": 132, "fp8": 132}[case.get("format", "bf16")]
    if op == "mask":
        nodes = (case["nodes_lo"] + case["nodes_hi"]) / 2
        words = (case["nodes_hi"] + 31) // 32
        return {"bytes": S * nodes * (4 + 4 * words + 4) + 4 * (S + 1), "flops": 0}
    ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
    if case["ctx_lo"] == 1:
        ctx = case["ctx_hi"] / math.log(case["ctx_hi"] + 1)
    hkv, table = case["hkv"], S * (ctx / BLOCK * 4 + 4)
    if op == "tree":
        rows = S * (case["nodes_lo"] + case["nodes_hi"]) / 2 * case["hq"]
        words = (case["nodes_hi"] + 31) // 32
        return {"bytes": S * ctx * hkv * 2 * row + rows * (4 * DIM + 4 + 4 * words / case["hq"])
                + table, "flops": 4 * DIM * rows * ctx}
    if op == "commit":
        moved = S * hkv * (1 + min(case["path_hi"], case["nodes_hi"])) / 2
        return {"bytes": moved * 2 * 2 * row + S * (16 + 4 * case["path_hi"]), "flops": 0}
    if op == "weights":
        rows = S * (case["q_lo"] + case["q_hi"]) / 2 * case["hq"]
        return {"bytes": S * ctx * hkv * (row + (8 if case["add"] else 4))
                + rows * (2 * DIM + 4) + table, "flops": 2 * DIM * rows * ctx}
    n = min(ctx, case["budget"])
    moved = max(0, n - case["sinks"]) if ctx > case["budget"] else 0
    return {"bytes": S * hkv * (ctx * 4 + n * 4 + moved * (2 * 2 * row + 4)) + table, "flops": 0}


def exact(case, seed):
    """Attention and its weights by their definition in 64 bits, a sequence and
    a KV head at a time. The other operators move and order values: they
    compute none."""
    if case["op"] not in ("tree", "weights"):
        return None
    s = prepare(case, seed)
    fmt, lens, cu = s["format"], s["lens"].tolist(), s["cu"].tolist()
    hq, hkv = case["hq"], case["hkv"]
    G = hq // hkv

    def cached(pool, b, h, c):
        ids = s["tables"][b, :(c + BLOCK - 1) // BLOCK].long()
        t = pool[ids, h]
        if fmt == "bf16":
            return t.double().reshape(-1, DIM)[:c]
        code = t[:, :BLOCK * DIM].contiguous()
        code = code.view(torch.int8).double() if fmt == "int8" \
            else code.view(torch.float8_e4m3fn).float().double()
        scale = t[:, BLOCK * DIM:].contiguous().view(torch.float32).double()
        return (code.reshape(-1, BLOCK, DIM) * scale.reshape(-1, BLOCK, 1)).reshape(-1, DIM)[:c]

    if case["op"] == "tree":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    else:
        w = s["weights"].double()
    for b, c in enumerate(lens):
        a, e = cu[b], cu[b + 1]
        L = e - a
        if case["op"] == "tree":
            # follow the parents of every node
            sees = torch.zeros((L, L), dtype=torch.bool)
            for j, parent in enumerate(s["parents"][a:e].tolist()):
                if parent >= 0:
                    sees[j] = sees[parent]
                sees[j, j] = True
        else:
            sees = torch.ones((L, L), dtype=torch.bool).tril()
        hidden = torch.cat([torch.zeros((L, c - L), dtype=torch.bool), ~sees], 1).cuda()
        for h in range(hkv):
            k = cached(s["k"], b, h, c)
            q = s["q"][a:e, h * G:(h + 1) * G].double().transpose(0, 1)  # [G, L, D]
            z = (q @ k.T) / math.sqrt(DIM)
            z.masked_fill_(hidden, -math.inf)
            if case["op"] == "tree":
                out[a:e, h * G:(h + 1) * G] = \
                    (torch.softmax(z, -1) @ cached(s["v"], b, h, c)).transpose(0, 1)
                lse[a:e, h * G:(h + 1) * G] = torch.logsumexp(z, -1).T
            else:
                got = s["lse"][a:e, h * G:(h + 1) * G].double().T[..., None]
                drawn = torch.exp(z - got).sum((0, 1))
                if case["add"]:
                    drawn[:c - L] += w[b, h, :c - L]
                w[b, h, :c] = drawn
    return {"out": out, "lse": lse} if case["op"] == "tree" else w
