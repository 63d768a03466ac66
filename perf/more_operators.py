"""Cases of the rotary-position and differential-attention operators.

Four operators of one attention layer over a paged KV cache. Queries are
rotated by their positions (``rotate``); a step's keys are rotated and join
the cache with their values, the queries rotated in the same call
(``append``); keys already cached are turned to new positions when what was
before them has left the cache (``move``); and differential attention reads
the cache: the difference of two softmax maps over pairs of KV heads, with a
norm over each head's output (``diff``).

``run`` computes a case in its plain form, elementary torch operations in 32
bits (angles in 64), or, with ``own`` set, by the framework's calls.
"""
import math

import torch

own = False

BLOCK = 16          # tokens per block of the pool
DIM = 128           # head dimension
TILE = 2112         # bytes of an 8-bit (block, KV head) tile: 16 x 128 codes, 16 fp32 scales
SCALE = 1.0 / math.sqrt(DIM)
EPS = 1e-5          # of the norm after differential attention
GAIN = 0.8          # factor behind that norm


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the queries of four chats in a layer that reads another layer's keys: latency is all there is
        {"name": "rotate_first", "op": "rotate", "seqs": 4, "new_lo": 1, "new_hi": 1, "ctx": 384,
         "hq": 16, "rot": 128, "pairs": "half", "scaling": "none", "turn": "on"},
        # long prompts, half of each head rotated, pairs side by side, frequencies scaled in bands
        {"name": "rotate_prompt", "op": "rotate", "seqs": 4, "new_lo": 4011, "new_hi": 4096,
         "ctx": 32768, "hq": 16, "rot": 64, "pairs": "side", "scaling": "bands", "turn": "on"},
        # one decode step of the four chats
        {"name": "append_first", "op": "append", "seqs": 4, "new_lo": 1, "new_hi": 1, "ctx": 384,
         "hq": 16, "hkv": 8, "format": "bf16", "rot": 128, "pairs": "half", "scaling": "none"},
        # one decode step of a full batch, far positions of a context stretched by a ramp
        {"name": "append_step", "op": "append", "seqs": 256, "new_lo": 1, "new_hi": 1,
         "ctx": 131072, "hq": 16, "hkv": 8, "format": "bf16", "rot": 128, "pairs": "half",
         "scaling": "ramp"},
        # prompts entering the cache
        {"name": "append_prompt", "op": "append", "seqs": 4, "new_lo": 2011, "new_hi": 4096,
         "ctx": 4096, "hq": 16, "hkv": 8, "format": "bf16", "rot": 128, "pairs": "half",
         "scaling": "none"},
        # chunks of prompts entering an FP8 cache
        {"name": "append_chunks", "op": "append", "seqs": 16, "new_lo": 500, "new_hi": 512,
         "ctx": 32768, "hq": 16, "hkv": 8, "format": "fp8", "rot": 128, "pairs": "half",
         "scaling": "linear"},
        # a serving batch whose caches were just cut to 1024 positions a head
        {"name": "move_step", "op": "move", "seqs": 32, "ctx_lo": 1024, "ctx_hi": 1024, "by": "kept",
         "first": 4, "hkv": 8, "format": "bf16", "rot": 128, "pairs": "half", "scaling": "none"},
        # long documents whose oldest part left the cache, behind sixteen positions that stay
        {"name": "move_long", "op": "move", "seqs": 8, "ctx_lo": 24011, "ctx_hi": 28672,
         "by": "shift", "first": 16, "hkv": 8, "format": "bf16", "rot": 128, "pairs": "half",
         "scaling": "none"},
        # one decode step of the four chats
        {"name": "diff_first", "op": "diff", "seqs": 4, "ctx_lo": 128, "ctx_hi": 384, "q_lo": 1,
         "q_hi": 1, "hq": 16, "hkv": 8, "norm": True},
        # one decode step of a ragged continuous batch
        {"name": "diff_step", "op": "diff", "seqs": 256, "ctx_lo": 1, "ctx_hi": 4096, "q_lo": 1,
         "q_hi": 1, "hq": 16, "hkv": 8, "norm": True},
        # long documents, four query heads to a KV head
        {"name": "diff_long", "op": "diff", "seqs": 8, "ctx_lo": 30011, "ctx_hi": 32768, "q_lo": 1,
         "q_hi": 1, "hq": 16, "hkv": 4, "norm": True},
        # chunks of prompts over what is cached of them
        {"name": "diff_chunk", "op": "diff", "seqs": 4, "ctx_lo": 2048, "ctx_hi": 8192, "q_lo": 512,
         "q_hi": 512, "hq": 16, "hkv": 8, "norm": True},
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    case = _draw(rng)
    # at most the largest listed work of its kind
    most = {"rotate": (1.3e8, 1e9), "append": (1.9e8, 1e9), "move": (8.6e8, 1e10),
            "diff": (5.2e8, 1.2e11)}[case["op"]]
    while case["seqs"] > 1 and (work(case)["bytes"] > most[0] or work(case)["flops"] > most[1]):
        case["seqs"] = max(1, case["seqs"] * 3 // 4)
    return case


def _draw(rng):
    op = rng.choice(["rotate", "rotate", "append", "append", "append", "move", "move", "diff",
                     "diff", "diff"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 2, 3, 4, 8])
    ctx = _log(rng, 64, 32768)
    # how a model lays its pairs out, and how many of a head's dimensions it rotates
    turns = {"rot": rng.choice([128, 128, 128, 64, 96, 32, 2 * rng.randint(1, 64)]),
             "pairs": rng.choice(["half", "half", "side"]),
             "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"])}
    if op == "diff":
        hkv = rng.choice([2, 2, 4, 8])
        seqs = _log(rng, 1, 128)
        q = rng.choice([1, min(ctx, _log(rng, 2, 512))])
        q = max(1, min(q, int(1.5e8 // (group * hkv * ctx))))  # for the plain form's score matrix
        return {"op": op, "seqs": seqs, "ctx_lo": max(q, rng.randint(max(2, ctx // 8), ctx)),
                "ctx_hi": ctx, "q_lo": rng.randint(1, q), "q_hi": q, "hq": hkv * group, "hkv": hkv,
                "norm": rng.random() < 0.8}
    if op == "move":
        by = rng.choice(["kept", "shift"])
        return {"op": op, "seqs": _log(rng, 1, 64), "ctx_lo": rng.randint(max(2, ctx // 8), ctx),
                "ctx_hi": ctx, "by": by, "first": rng.randint(0, 16), "hkv": hkv,
                "format": rng.choice(["bf16", "bf16", "int8", "fp8"]), **turns}
    new = rng.choice([1, _log(rng, 2, 4096)])
    case = {"op": op, "seqs": _log(rng, 1, 256), "new_lo": rng.randint(1, new), "new_hi": new,
            "ctx": max(new, _log(rng, 64, 131072)), "hq": hkv * group, **turns}
    if op == "rotate":
        return {**case, "turn": rng.choice(["on", "on", "back"])}
    return {**case, "hkv": hkv, "format": rng.choice(["bf16", "bf16", "int8", "fp8"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

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


def _scaling(case):
    """How far and by what rule the case's frequencies are stretched: name,
    factor, length the model was trained at, and two numbers of turns over that
    length between which the rule changes."""
    return {"none": ("none", 1.0, 8192, 1.0, 1.0), "linear": ("linear", 4.0, 8192, 1.0, 1.0),
            "base": ("base", 4.0, 8192, 1.0, 1.0), "bands": ("bands", 8.0, 8192, 1.0, 4.0),
            "ramp": ("ramp", 4.0, 32768, 1.0, 32.0)}[case["scaling"]]


def _base(case):
    return {"none": 10000.0, "linear": 10000.0, "base": 10000.0, "bands": 500000.0,
            "ramp": 1000000.0}[case["scaling"]]


def _tables(g, per, most):
    """Block tables of sequences with `per` blocks each in a shuffled pool of at
    least `most` blocks, some of it held by others."""
    width = int(per.max())
    blocks = most + most // 10 + 1
    ids = torch.randperm(blocks, generator=g, device="cuda")
    col = torch.arange(width, device="cuda")
    flat = (per.cumsum(0) - per)[:, None] + col
    used = col < per[:, None]
    return torch.where(used, ids[flat.clamp(max=blocks - 1)], -1).to(torch.int32).contiguous(), blocks


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, seqs = case["op"], case["seqs"]
    s = {"op": op, "case": dict(case)}
    if op in ("rotate", "append"):
        n = _lengths(g, case["new_lo"], case["new_hi"], seqs)
        end = torch.maximum(n, _lengths(g, 1, case["ctx"], seqs, log=True))
        total = int(n.sum())
        seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), n)
        j = torch.arange(total, device="cuda") - (n.cumsum(0) - n)[seq]
        at = (end - n)[seq] + j                                   # a token's position
        s["positions"] = at.to(torch.int32)
        hkv = case.get("hkv", 0)
        # what a fused projection leaves: q, k and v of a token side by side
        mixed = _randn(g, (total, case["hq"] + 2 * max(hkv, 1), DIM))
        s["q"] = mixed[:, :case["hq"]]
        s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        if op == "append":
            s["k"], s["v"] = mixed[:, case["hq"]:case["hq"] + hkv], mixed[:, case["hq"] + hkv:]
            # the blocks that hold the new tokens, from the block of the first of them on
            lead = (end - n) % BLOCK
            per = (lead + n + BLOCK - 1) // BLOCK
            table, blocks = _tables(g, per, int(((n + 2 * BLOCK - 2) // BLOCK).sum()))
            place = lead[seq] + j
            s["slots"] = table[seq, place // BLOCK].to(torch.int64) * BLOCK + place % BLOCK
            s["format"] = case["format"]
            s["k_pool"] = _pool(g, blocks, hkv, case["format"])
            s["v_pool"] = _pool(g, blocks, hkv, case["format"])
        return s
    # the lengths of a continuous batch are log-uniform
    lens = _lengths(g, case["ctx_lo"], case["ctx_hi"], seqs, log=case["ctx_lo"] == 1)
    per = (lens + BLOCK - 1) // BLOCK
    s["tables"], blocks = _tables(g, per, int(per.sum()))
    s["lens"] = lens.to(torch.int32)
    hkv = case["hkv"]
    if op == "move":
        s["format"] = case["format"]
        s["k_pool"] = _pool(g, blocks, hkv, case["format"])
        most = int(lens.max())
        if case["by"] == "kept":
            # positions that an eviction left: the first stay, of the others one in nine is gone
            gone = torch.rand((seqs, hkv, most), generator=g, device="cuda") < 1 / 8
            gone &= torch.arange(most, device="cuda") >= case["first"]
            i = torch.arange(most, device="cuda")
            kept = i + gone.to(torch.int64).cumsum(-1)
            s["kept"] = torch.where(i < lens[:, None, None], kept, -1).to(torch.int32)
        else:
            gone = torch.randint(1, 4096, (seqs,), generator=g, device="cuda")
            s["shifts"] = (-gone).to(torch.int32)
        return s
    new = torch.minimum(_lengths(g, case["q_lo"], case["q_hi"], seqs), lens)
    s["q_max"] = int(new.max())
    s["cu"] = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32)
    s["total"] = int(new.sum())
    # outlier keys in one row of a hundred
    s["k_pool"] = _pool(g, blocks, hkv, "bf16", 0.01, 8.0)
    s["v_pool"] = _pool(g, blocks, hkv, "bf16")
    s["q"] = _randn(g, (s["total"], case["hq"], DIM))
    heads = case["hq"] // 2
    s["lambdas"] = 0.2 + 0.6 * torch.rand((heads,), generator=g, device="cuda")
    s["weight"] = None
    if case["norm"]:
        s["weight"] = 1 + 0.1 * torch.randn((2 * DIM,), generator=g, device="cuda")
    s["out"] = torch.empty((s["total"], heads, 2 * DIM), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((s["total"], case["hq"]), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _theta(case):
    """Radians per position of every pair, in 64 bits, and the factor on cosine and sine."""
    r, base = case["rot"], _base(case)
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    kind, factor, length, low, high = _scaling(case)
    if kind == "base":
        base = base * factor ** (r / max(r - 2, 1))
    theta = base ** (-2 * i / r)
    if kind == "linear":
        return theta / factor, 1.0
    if kind == "bands":
        share = ((length * theta / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return theta * share + theta / factor * (1 - share), 1.0
    if kind == "ramp":
        def pair_with(turns):
            return r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
        a = min(max(math.floor(pair_with(high)), 0), r - 1)
        b = min(max(math.ceil(pair_with(low)), 0), r - 1)
        share = ((i - a) / max(b - a, 1e-3)).clamp(0, 1)
        return theta * (1 - share) + theta / factor * share, 0.1 * math.log(factor) + 1
    return theta, 1.0


def _turned(x, positions, case, sign=1.0, magnitude=True):
    """Rows x [..., D] in 32 bits, turned by positions [...] (broadcast over x's leading axes)."""
    theta, m = _theta(case)
    angle = positions.double()[..., None] * theta
    m = m if magnitude else 1.0
    c, sn = (m * torch.cos(angle)).float(), (sign * m * torch.sin(angle)).float()
    r = case["rot"]
    if case["pairs"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    else:
        a, b = x[..., :r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _codes(x, fmt):
    """Rows in 8 bits, one fp32 scale a row."""
    most = 127.0 if fmt == "int8" else 448.0
    amax = x.abs().amax(-1, keepdim=True)
    y = torch.where(amax > 0, x * (most / amax), torch.zeros_like(x)).clamp(-most, most)
    y = y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return y.view(torch.uint8), amax / most


def _write(pool, slots, x, fmt):
    b, i = slots // BLOCK, slots % BLOCK
    if fmt == "bf16":
        pool[b, :, i] = x.to(torch.bfloat16)
        return
    codes, scales = _codes(x, fmt)
    pool[..., :BLOCK * DIM].unflatten(-1, (BLOCK, DIM))[b, :, i] = codes
    pool[..., BLOCK * DIM:].unflatten(-1, (BLOCK, 4))[b, :, i] = scales.contiguous().view(torch.uint8)


def _values(tiles, fmt):
    """What 8-bit tiles [..., TILE] stand for: [..., BLOCK, D]."""
    codes = tiles[..., :BLOCK * DIM].contiguous()
    codes = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
    scales = tiles[..., BLOCK * DIM:].contiguous().view(torch.float32)
    return codes.unflatten(-1, (BLOCK, DIM)) * scales[..., None]


def _held(pool, s):
    """A pool after the call: the bf16 pool itself, or the values of an 8-bit one."""
    if s["format"] == "bf16":
        return pool
    return _values(pool, s["format"]).to(torch.bfloat16)


def _plain_rotate(s):
    case = s["case"]
    sign = 1.0 if case["turn"] == "on" else -1.0
    s["q_out"].copy_(_turned(s["q"].float(), s["positions"][:, None], case, sign))
    return s["q_out"]


def _plain_append(s):
    at, case, fmt = s["positions"][:, None], s["case"], s["format"]
    s["q_out"].copy_(_turned(s["q"].float(), at, case))
    _write(s["k_pool"], s["slots"], _turned(s["k"].float(), at, case), fmt)
    _write(s["v_pool"], s["slots"], s["v"].float(), fmt)
    return {"q": s["q_out"], "k": _held(s["k_pool"], s), "v": _held(s["v_pool"], s)}


def _plain_move(s):
    case, fmt, pool = s["case"], s["format"], s["k_pool"]
    S, hkv = s["tables"].shape[0], pool.shape[1]
    most = s["tables"].shape[1] * BLOCK
    i = torch.arange(most, device="cuda")
    inside = i < s["lens"][:, None]
    if case["by"] == "kept":
        kept = torch.nn.functional.pad(s["kept"], (0, most - s["kept"].shape[-1]), value=-1)
        by = torch.where(kept >= 0, i - kept, 0)                  # [S, Hkv, positions]
    else:
        by = torch.where(i >= case["first"], s["shifts"][:, None], 0)[:, None].expand(S, hkv, most)
    by = torch.where(inside[:, None], by, 0)
    by = by.unflatten(-1, (-1, BLOCK)).transpose(1, 2)            # [S, blocks, Hkv, BLOCK]
    held = s["tables"] >= 0
    ids, by = s["tables"][held].to(torch.int64), by[held]
    if fmt == "bf16":
        x = pool[ids]
        y = _turned(x.float(), by, case, magnitude=False).to(torch.bfloat16)
        pool[ids] = torch.where((by != 0)[..., None], y, x)
        return pool
    x = pool[ids]
    codes, scales = _codes(_turned(_values(x, fmt), by, case, magnitude=False), fmt)
    turned = (by != 0)[..., None]
    old = x[..., :BLOCK * DIM].unflatten(-1, (BLOCK, DIM))
    olds = x[..., BLOCK * DIM:].unflatten(-1, (BLOCK, 4))
    x[..., :BLOCK * DIM] = torch.where(turned, codes, old).flatten(-2)
    x[..., BLOCK * DIM:] = torch.where(turned, scales.contiguous().view(torch.uint8), olds).flatten(-2)
    pool[ids] = x
    return _held(pool, s)


def _rows(x, tables):
    """The cached rows of every sequence in 32 bits: [S, Hkv, positions, D]."""
    t = x[tables.clamp(min=0).to(torch.int64)].transpose(1, 2)
    return t.flatten(2, 3).float()


def _plain_diff(s):
    case = s["case"]
    hq, hkv = case["hq"], case["hkv"]
    G, P = hq // hkv, hkv // 2
    cu = s["cu"].to(torch.int64)
    n = cu[1:] - cu[:-1]
    L = s["q_max"]
    j = torch.arange(L, device="cuda")
    inside = j < n[:, None]
    at = torch.where(inside, cu[:-1, None] + j, 0)
    k = _rows(s["k_pool"], s["tables"])
    S, _, C, _ = k.shape
    q = s["q"][at].float().reshape(S, L, hkv, G, DIM).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q.reshape(S, hkv, G * L, DIM), k.transpose(-1, -2)).mul_(SCALE)
    del k
    z = z.reshape(S, hkv, G, L, C)
    c = s["lens"].to(torch.int64)
    last = (c - n)[:, None] + j                                    # [S, L]
    p = torch.arange(C, device="cuda")
    z.masked_fill_((p > last[..., None])[:, None, None], -math.inf)
    z.masked_fill_((p >= c[:, None])[:, None, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    v = _rows(s["v_pool"], s["tables"]).reshape(S, P, 2, C, DIM)
    v = v.transpose(2, 3).reshape(S, P, 1, C, 2 * DIM)
    # both maps of a pair of heads over the pair's values
    o = torch.matmul(e.reshape(S, P, 2, G * L, C), v).reshape(S, hkv, G, L, 2 * DIM) / total
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(S, L, hq)
    o = o.reshape(S, P, 2, G, L, 2 * DIM)
    lam = s["lambdas"].reshape(P, G, 1, 1)
    d = o[:, :, 0] - lam * o[:, :, 1]                              # [S, P, G, L, 2 D]
    if s["weight"] is not None:
        d = d / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    d = (GAIN * d).permute(0, 3, 1, 2, 4).reshape(S, L, hq // 2, 2 * DIM)
    return {"out": d[inside].to(torch.bfloat16), "lse": lse[inside]}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _rotation(case):
    from paged_kv_decode_18_gb300 import binding as B
    kind, factor, length, low, high = _scaling(case)
    return B.make_rotation(case["rot"], interleaved=case["pairs"] == "side", base=_base(case),
                           scaling=kind, factor=factor, original_len=length, low=low, high=high)


def _call(s):
    """The prepared call on a state's buffers, as a serving loop keeps it."""
    from paged_kv_decode_18_gb300 import binding as B
    op, case = s["op"], s["case"]
    kind = {"bf16": B.PA_KV_BF16, "int8": B.PA_KV_INT8, "fp8": B.PA_KV_FP8}[s.get("format", "bf16")]
    if op == "rotate":
        return B.prepare_rotate(s["q"], s["positions"], _rotation(case), s["q_out"],
                                transpose=case["turn"] == "back")
    if op == "append":
        return B.prepare_rotate_and_cache(s["k"], s["v"], s["positions"], s["slots"],
                                          _rotation(case), s["k_pool"], s["v_pool"], q=s["q"],
                                          q_out=s["q_out"], kv_format=kind)
    if op == "move":
        return B.prepare_rotate_cached(s["k_pool"], s["tables"], s["lens"], _rotation(case),
                                       kept=s.get("kept"), shifts=s.get("shifts"),
                                       first=case["first"] if "shifts" in s else 0, kv_format=kind)
    cu, most = (s["cu"], s["q_max"]) if s["q_max"] > 1 else (None, 1)
    shape = B.shape_of(s["q"], s["k_pool"], s["tables"])
    room = B.workspace(B.pa_decode_diff_workspace_size(shape, s["total"], most))
    return B.prepare_decode_diff(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], SCALE,
                                 s["lambdas"], s["out"], s["lse"], cu_seqlens_q=cu, max_q_len=most,
                                 norm_weight=s["weight"], norm_eps=EPS, out_scale=GAIN,
                                 workspace=room)


def _own(s):
    if "call" not in s:
        s["call"] = _call(s)
    s["call"]()
    op = s["op"]
    if op == "rotate":
        return s["q_out"]
    if op == "append":
        return {"q": s["q_out"], "k": _held(s["k_pool"], s), "v": _held(s["v_pool"], s)}
    if op == "move":
        return _held(s["k_pool"], s)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "append": _plain_append, "move": _plain_move,
            "diff": _plain_diff}[state["op"]](state)


# ---------------------------------------------------------------------------
# floors and exact results
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations for the middle of the case's ranges."""
    op, S = case["op"], case["seqs"]
    row = {"bf16": 256, "int8": 132, "fp8": 132}[case.get("format", "bf16")]
    turn = 3 * case.get("rot", 0)                                 # operations of a rotated row
    if op in ("rotate", "append"):
        T = S * (case["new_lo"] + case["new_hi"]) / 2
        hkv = case.get("hkv", 0)
        return {"bytes": T * (case["hq"] * 512 + 2 * hkv * (256 + row) + 4 + (8 if hkv else 0)),
                "flops": T * (case["hq"] + hkv) * turn}
    ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
    if case["ctx_lo"] == 1:
        ctx = case["ctx_hi"] / math.log(case["ctx_hi"] + 1)
    hkv, table = case["hkv"], S * (ctx / BLOCK * 4 + 4)
    if op == "move":
        moved = S * hkv * max(0, ctx - case["first"])
        return {"bytes": moved * (2 * row + (4 if case["by"] == "kept" else 0)) + table,
                "flops": moved * turn}
    q = (case["q_lo"] + case["q_hi"]) / 2
    rows = S * q * case["hq"]
    return {"bytes": S * ctx * hkv * 2 * 256 + rows * (4 * DIM + 4) + table,
            "flops": (2 * DIM + 4 * DIM) * rows * (ctx - (q - 1) / 2)}


def _exact_rows(x, positions, case, sign, magnitude=True):
    """Rows [n, D] turned pair by pair, as complex numbers, in 64 bits."""
    theta, m = _theta(case)
    angle = positions.double()[:, None] * theta
    spin = torch.polar(torch.full_like(angle, m if magnitude else 1.0), sign * angle)
    r, y = case["rot"], x.double().clone()
    first = torch.arange(0, r // 2, device="cuda") if case["pairs"] == "half" \
        else torch.arange(0, r, 2, device="cuda")
    second = first + (r // 2 if case["pairs"] == "half" else 1)
    z = torch.complex(y[:, first], y[:, second]) * spin
    y[:, first], y[:, second] = z.real.clone(), z.imag.clone()
    return y


def _exact_held(y, fmt):
    """What rows [n, D] stand for once they are held in the pool's format."""
    if fmt == "bf16":
        return y
    most = 127.0 if fmt == "int8" else 448.0
    scale = y.abs().amax(1, keepdim=True) / most
    x = torch.where(scale > 0, y / scale, 0.0)
    if fmt == "int8":
        return torch.round(x) * scale
    # the nearest of E4M3's numbers, ties to the even one: steps of 2^(e - 3), 2^-9 at least
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step * scale


def exact(case, seed):
    """The operators by their definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        y = _exact_rows(s["q"].reshape(-1, DIM), s["positions"].repeat_interleave(case["hq"]), case,
                        1 if case["turn"] == "on" else -1)
        return y.reshape(s["q"].shape)
    if op in ("append", "move"):
        fmt, hkv = s["format"], case["hkv"]

        def whole(pool):
            return pool.double() if fmt == "bf16" else _values(pool, fmt).double()

    if op == "append":
        k, v, slots = whole(s["k_pool"]), whole(s["v_pool"]), s["slots"]
        at = s["positions"]
        y = _exact_rows(s["k"].reshape(-1, DIM), at.repeat_interleave(hkv), case, 1)
        k[slots // BLOCK, :, slots % BLOCK] = _exact_held(y, fmt).reshape(-1, hkv, DIM)
        v[slots // BLOCK, :, slots % BLOCK] = \
            _exact_held(s["v"].double().reshape(-1, DIM), fmt).reshape(-1, hkv, DIM)
        q = _exact_rows(s["q"].reshape(-1, DIM), at.repeat_interleave(case["hq"]), case, 1)
        return {"q": q.reshape(s["q"].shape), "k": k, "v": v}
    lens = s["lens"].tolist()
    if op == "move":
        k = whole(s["k_pool"])
        for b, c in enumerate(lens):
            i = torch.arange(c, device="cuda")
            ids = s["tables"][b, i // BLOCK].long()
            for h in range(hkv):
                if case["by"] == "kept":
                    by = i - s["kept"][b, h, :c]
                else:
                    by = torch.where(i >= case["first"], s["shifts"][b], 0)
                turn = torch.nonzero(by)[:, 0]
                y = _exact_rows(k[ids[turn], h, i[turn] % BLOCK], by[turn], case, 1, magnitude=False)
                k[ids[turn], h, i[turn] % BLOCK] = _exact_held(y, fmt)
        return k
    hq, hkv, cu = case["hq"], case["hkv"], s["cu"].tolist()
    G = hq // hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, c in enumerate(lens):
        a, e = cu[b], cu[b + 1]
        ids = s["tables"][b, :(c + BLOCK - 1) // BLOCK].long()
        hidden = torch.ones((e - a, c), dtype=torch.bool, device="cuda").tril(c - (e - a)).logical_not()
        for p in range(hkv // 2):
            v = torch.cat([s["v_pool"][ids, h].reshape(-1, DIM)[:c] for h in (2 * p, 2 * p + 1)], 1)
            o = []
            for h in (2 * p, 2 * p + 1):
                k = s["k_pool"][ids, h].reshape(-1, DIM)[:c].double()
                q = s["q"][a:e, h * G:(h + 1) * G].double().transpose(0, 1)
                z = (q @ k.T / math.sqrt(DIM)).masked_fill(hidden, -math.inf)
                o.append(torch.softmax(z, -1) @ v.double())
                lse[a:e, h * G:(h + 1) * G] = torch.logsumexp(z, -1).T
            d = o[0] - s["lambdas"][p * G:(p + 1) * G].double()[:, None, None] * o[1]
            if s["weight"] is not None:
                d = d * torch.rsqrt(d.pow(2).sum(-1, keepdim=True) / (2 * DIM) + EPS)
                d = d * s["weight"].double()
            out[a:e, p * G:(p + 1) * G] = GAIN * d.transpose(0, 1)
    return {"out": out, "lse": lse}
