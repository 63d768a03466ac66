"""Differential attention in 64 bits, written from its definition, and how far
the kernels' roundings can take a result. It shares nothing with the library."""
import math

import torch

BLOCK, DIM = 16, 128
U32 = 2.0 ** -24   # half a step of fp32
UBF = 2.0 ** -8    # half a step of bf16 (finfo.eps / 2)


def rows_of(pool, table, c, h):
    ids = table[:(c + BLOCK - 1) // BLOCK].long()
    return pool[ids, h].reshape(-1, DIM)[:c].double()


def attend(q, kc, vc, tables, lens, cu, scale, lambdas, weight=None, eps=0.0, gain=1.0,
           causal=True):
    """out [T, Hq/2, 256], lse [T, Hq], and bounds of what the kernels may differ
    by, all in 64 bits on the CPU:
      a score: 128 exact products summed in fp32, its scaling, and the base-2
        exponential's argument and result (2^-22 of it): dz;
      a map's result: each weight by e^(2 dz) - 1 (its own and the sum's), half a step of
        bf16, and the fp32 sums: times sum p |v|;
      the difference: both maps' errors; its root mean square: at most the root
        mean square of those; the output: half a step of bf16."""
    q, kc, vc = q.cpu(), kc.cpu(), vc.cpu()
    T, hq, _ = q.shape
    hkv = kc.shape[1]
    G = hq // hkv
    out = torch.zeros(T, hq // 2, 2 * DIM, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros_like(lse)
    for s, c in enumerate(lens):
        a, e = int(cu[s]), int(cu[s + 1])
        L = e - a
        if L == 0 or c == 0:
            continue
        see = torch.ones(L, c, dtype=torch.bool)
        if causal:
            see = see.tril(c - L)
        for p in range(hkv // 2):
            v = torch.cat([rows_of(vc, tables[s], c, 2 * p + i) for i in (0, 1)], 1)
            k = [rows_of(kc, tables[s], c, 2 * p + i) for i in (0, 1)]
            for g in range(G):
                a_i, e_i = [], []
                for i in (0, 1):
                    h = (2 * p + i) * G + g
                    x = q[a:e, h].double()
                    z = torch.where(see, scale * (x @ k[i].T), -math.inf)
                    size = torch.where(see, scale * (x.abs() @ k[i].abs().T), 0.0).amax(-1)
                    dz = (128 + 4) * U32 * size + 2.0 ** -21
                    m = torch.logsumexp(z, -1)
                    w = torch.exp(z - m[:, None])
                    got, mass = w @ v, w @ v.abs()
                    a_i.append(got)
                    # (the sum over c weights in fp32: c 2^-24 at most)
                    e_i.append((torch.expm1(2 * dz) + UBF + (c + 64) * U32)[:, None] * mass)
                    lse[a:e, h] = m
                    ltol[a:e, h] = 2 * dz + (c + 64) * U32 + 4 * U32 * m.abs()
                lam = float(lambdas[p * G + g])
                d = a_i[0] - lam * a_i[1]
                ed = e_i[0] + abs(lam) * e_i[1] + 4 * U32 * (a_i[0].abs() + abs(lam) * a_i[1].abs())
                if weight is None:
                    y, ey = gain * d, abs(gain) * ed
                else:
                    w = weight.double().cpu()
                    rms = torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
                    off = torch.sqrt(ed.square().mean(-1, keepdim=True))
                    low = (rms - off).clamp(min=math.sqrt(eps) if eps else 1e-30)
                    y = gain * w * d / rms
                    ey = abs(gain) * w.abs() * ((d.abs() + ed) / low - d.abs() / rms)
                    ey = ey + 2.0 ** -20 * y.abs()
                out[a:e, p * G + g] = y
                tol[a:e, p * G + g] = ey + UBF * (y.abs() + ey) + 2.0 ** -126
    return out, lse, tol, ltol
