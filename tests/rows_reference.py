"""Plain definitions in 64 bits of the rows' permutation, weighted sum, gated activation and dropout (host tensors)."""
import math

import numpy as np
import torch

U32 = 1 << 32


def philox(counter, key):
    """Philox 4x32 with ten rounds (Salmon et al., SC 2011), one block, in Python's whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        x, y = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(y >> 32) ^ c[1] ^ k[0], y % U32, (x >> 32) ^ c[3] ^ k[1], x % U32]
        k = [(k[0] + 0x9E3779B9) % U32, (k[1] + 0xBB67AE85) % U32]
    return c


def philox_blocks(blocks, rows, key, offset):
    """The words of blocks x rows [rows, blocks, 4] as uint64."""
    u = np.uint64
    b, r = np.meshgrid(np.arange(blocks, dtype=u), np.asarray(rows, dtype=u))
    c = [b, r, np.full_like(b, offset % U32), np.full_like(b, offset // U32)]
    k = [key % U32, key // U32]
    low = u(U32 - 1)
    for _ in range(10):
        x, y = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(y >> u(32)) ^ c[1] ^ u(k[0]), y & low, (x >> u(32)) ^ c[3] ^ u(k[1]), x & low]
        k = [(k[0] + 0x9E3779B9) % U32, (k[1] + 0xBB67AE85) % U32]
    return np.stack(c, -1)


def factors(rows, cols, p, rng):
    """What dropout multiplies each element of [rows, cols] with; rows: a number, or the rows' numbers."""
    rows = np.arange(rows) if isinstance(rows, int) else np.asarray(rows)
    cut = int(np.float32(p).astype(np.float64) * 65536 + 0.5)
    if cut == 0:
        return torch.ones(len(rows), cols, dtype=torch.float64)
    seed, offset = (int(v) % (1 << 64) for v in rng)
    w = philox_blocks(-(-cols // 8), rows, seed, offset)
    half = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(len(rows), -1)[:, :cols]
    scale = 65536.0 / (65536 - cut) if cut < 65536 else 0.0
    return torch.from_numpy((half >= cut).astype(np.float64) * scale)


def sort(idx, E, block):
    """(ids, rows in use, pair_row) of the sorted layout, one expert after another."""
    T, k = idx.shape
    flat = idx.reshape(-1).tolist()
    ids, pair_row = [], [-1] * len(flat)
    mine = {}
    for i, e in enumerate(flat):
        if 0 <= e < E:
            mine.setdefault(e, []).append(i)
    for e in sorted(mine):
        for i in mine[e]:
            pair_row[i] = len(ids)
            ids.append(i)
        ids += [T * k] * (-len(ids) % block)
    return ids, len(ids), torch.tensor(pair_row, dtype=torch.int64).view(T, k)


def permute(x, ids, n, n_rows, topk):
    """rows [n_rows, H]: the first n by ids, NaN behind (to be left alone)."""
    T, H = x.shape
    rows = torch.full((n_rows, H), math.nan, dtype=torch.float64)
    for r in range(n):
        rows[r] = x[ids[r] // topk].double() if 0 <= ids[r] < T * topk else 0.0
    return rows


def gathered(rows, pair_row):
    """[T, topk, H], zeros for pairs without a row."""
    T, k = pair_row.shape
    out = torch.zeros(T, k, rows.shape[1], dtype=torch.float64)
    has = pair_row >= 0
    out[has] = rows[pair_row[has].long()].double()
    return out


def act(g, kind):
    """(act(g), act'(g)) in 64 bits; kind 0: SiLU, 1: GELU."""
    if kind == 0:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
