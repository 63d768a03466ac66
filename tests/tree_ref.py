"""Plain 64-bit forms of the tree-verification and eviction operators, written
from their definitions with loops, and the tolerances that the kernels'
roundings give. They share nothing with the library."""
import math

import numpy as np
import torch

BLOCK, DIM = 16, 128
U32 = 2.0 ** -24   # half a step of fp32
UBF = 2.0 ** -8    # half a step of bf16 (finfo.eps / 2)


def tree_mask(parents, cu, words):
    """Ancestor rows as int32 words and depths, a node at a time."""
    parents, cu = np.asarray(parents), np.asarray(cu)
    mask = np.zeros((len(parents), words), np.uint32)
    depths = np.zeros(len(parents), np.int32)
    for a, b in zip(cu[:-1], cu[1:]):
        for j in range(b - a):
            x, depth = j, -1
            while x >= 0:
                mask[a + j, x // 32] |= np.uint32(1 << (x % 32))
                x, depth = int(parents[a + x]), depth + 1
            depths[a + j] = depth
    return mask.view(np.int32), depths


def random_parents(g, lens):
    """Parents of random trees, several of them with more than one root."""
    got = []
    for n in lens:
        for j in range(n):
            got.append(int(torch.randint(-1, j, (1,), generator=g)) if j else -1)
    return torch.tensor(got, dtype=torch.int32)


def bits_to_bool(mask_row, n):
    w = np.asarray(mask_row).view(np.uint32)
    return torch.tensor([bool((int(w[i // 32]) >> (i % 32)) & 1) if i // 32 < len(w) else False
                         for i in range(n)])


def cached(pool, table, c, h):
    """Rows 0 .. c-1 of one KV head from a bf16 pool [NB, Hkv, 16, D], fp64."""
    ids = table[:(c + BLOCK - 1) // BLOCK].long()
    return pool[ids, h].reshape(-1, DIM)[:c].double()


def tree_attention(q, k_pool, v_pool, tables, lens, cu, mask, scale):
    """out, lse in 64 bits; and per output how far the kernel's roundings can
    take it: a score by the fp32 sum of 128 exact products (A = scale sum |q k|),
    so each softmax weight by that much of itself, the weight again by half a
    bf16 step, and the output by half a bf16 step; the lse by its scores."""
    q = q.double()
    Tq, Hq, _ = q.shape
    Hkv = k_pool.shape[1]
    G = Hq // Hkv
    out = torch.zeros(Tq, Hq, DIM, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((Tq, Hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros_like(lse)
    for s in range(len(lens)):
        a, b, c = int(cu[s]), int(cu[s + 1]), int(lens[s])
        L = b - a
        if L == 0:
            continue
        sees = torch.ones(L, c, dtype=torch.bool)
        for j in range(L):
            sees[j, c - L:] = bits_to_bool(mask[a + j], L)
        for h in range(Hkv):
            k, v = cached(k_pool, tables[s], c, h), cached(v_pool, tables[s], c, h)
            for g in range(G):
                for j in range(L):
                    see = sees[j]
                    if not see.any():
                        continue
                    kk, vv = k[see], v[see]
                    x = q[a + j, h * G + g]
                    z = scale * (kk @ x)
                    A = scale * (kk.abs() @ x.abs())
                    m = z.max()
                    p = torch.exp(z - m)
                    tot = p.sum()
                    o = (p[:, None] * vv).sum(0) / tot
                    ez = 136 * U32 * A.max() + 2.0 ** -21
                    spread = (p[:, None] * vv.abs()).sum(0) / tot
                    out[a + j, h * G + g] = o
                    tol[a + j, h * G + g] = (UBF * (1 + UBF) * (o.abs() + spread)
                                             + 4 * ez * spread + 2.0 ** -30)
                    lse[a + j, h * G + g] = m + torch.log(tot)
                    ltol[a + j, h * G + g] = 2 * ez + 4 * U32 * abs(float(m + torch.log(tot)))
    return out, lse, tol, ltol


def assert_tree_close(out, lse, ref, what=""):
    o, l, tol, ltol = ref
    got = out.cpu().double()
    fine = torch.isfinite(o)
    assert torch.equal(torch.isnan(got), torch.isnan(o)), f"{what}: NaNs differ"
    assert torch.equal(got[~fine & ~torch.isnan(o)], o[~fine & ~torch.isnan(o)]), what
    d = (got - o).abs()[fine]
    over = d - tol[fine]
    assert not fine.any() or over.max() <= 0, f"{what}: out off by {d.max():.3e}"
    if lse is not None:
        gl = lse.cpu().double()
        inf = torch.isinf(l)
        assert torch.equal(torch.isinf(gl), inf), f"{what}: empty rows differ"
        dl = (gl - l).abs()[~inf]
        assert dl.numel() == 0 or (dl - ltol[~inf]).max() <= 0, f"{what}: lse off {dl.max():.3e}"


def accumulate(q, rows_of, lse, lens, cu, scale, weights, add, Hkv):
    """The new weights in 64 bits, and how far the kernel's roundings can take
    them: each term by its score's and exponent's, the sum by half an fp32 step
    an addition."""
    q, lse = q.double(), lse.double()
    G = q.shape[1] // Hkv
    w = weights.double().clone()
    tol = torch.zeros_like(w)
    for s in range(len(lens)):
        a, b, c = int(cu[s]), int(cu[s + 1]), int(lens[s])
        L = b - a
        if c == 0:
            continue
        for h in range(Hkv):
            k = rows_of(s, h)
            tot, err, n = torch.zeros(c, dtype=torch.float64), torch.zeros(c, dtype=torch.float64), 1
            for j in range(L):
                last = c - L + j
                for g in range(G):
                    l = float(lse[a + j, h * G + g])
                    if l == -math.inf:
                        continue
                    x = q[a + j, h * G + g]
                    z = scale * (k[:last + 1] @ x)
                    A = scale * (k[:last + 1].abs() @ x.abs())
                    p = torch.exp(z - l)
                    tot[:last + 1] += p
                    err[:last + 1] += p * (140 * U32 * A + 8 * U32 * (z.abs() + abs(l))
                                           + 2.0 ** -20)
                    n += 1
            old = torch.zeros(c, dtype=torch.float64)
            if add:
                old[:c - L] = w[s, h, :c - L]
            w[s, h, :c] = old + tot
            tol[s, h, :c] = 2 * err + n * U32 * tot + 2 * U32 * (old.abs() + tot) + 1e-37
    return w, tol


def evict_positions(row, c, budget, sinks, recent):
    """Old positions that stay, by the definition, one at a time."""
    if c <= budget:
        return list(range(c))

    def key(p):
        x = float(row[p])
        return (1, 0.0) if math.isnan(x) else (0, -(x + 0.0))
    middle = sorted(range(sinks, c - recent), key=lambda p: (*key(p), p))
    best = middle[:budget - sinks - recent]
    return sorted(list(range(sinks)) + best + list(range(c - recent, c)))
