"""Plain implementation of the 4-bit rows, for the tests: numpy, one rule after the other as the format states them."""
from __future__ import annotations

import numpy as np

MAGS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
ROW_BYTES = {"fp4_288": 288, "fp4_416": 416}


def code_of(z):
    """Number of the nearest magnitude (ties: the even number) of z >= 0, 64 bits."""
    d = np.abs(np.asarray(z)[..., None] - MAGS)
    near = d == d.min(-1, keepdims=True)
    first = near.argmax(-1)
    both = near.sum(-1) > 1
    return np.where(both & (first % 2 == 1), first + 1, first)


def encode(x, k_pe_bits=None):
    """Rows [n, 288 or 416] uint8 of latents x [n, 512] (values of BF16 numbers) and RoPE bits [n, 64] uint16."""
    x = np.asarray(x, dtype=np.float32)
    n = x.shape[0]
    out = np.zeros((n, 288 if k_pe_bits is None else 416), np.uint8)
    with np.errstate(all="ignore"):
        for r in range(n):
            words, exps, scales = np.zeros(64, np.uint64), np.zeros(32, np.uint8), np.zeros(4, np.float32)
            for g in range(4):
                v = x[r, 128 * g:128 * g + 128]
                if not np.isfinite(v).all():
                    scales[g] = np.nan
                    s = np.float32(0)
                else:
                    s = scales[g] = np.float32(np.abs(v).max()) / np.float32(384)
                for b in range(8):
                    u = v[16 * b:16 * b + 16]
                    y = np.zeros(16, np.float32) if s == 0 else u / s
                    e = 0
                    while e < 11 and np.abs(y).max() > 7 * 2.0 ** (e - 5):
                        e += 1
                    exps[8 * g + b] = e
                    code = code_of(np.minimum(np.abs(y.astype(np.float64)) * 2.0 ** (5 - e), 6.0))
                    neg = np.signbit(u)
                    for d in range(16):
                        w, i = 16 * g + 2 * b + d // 8, d % 8
                        sign_at = 8 * i + 7 if i < 4 else 8 * (i - 4) + 3
                        words[w] |= np.uint64(int(code[d]) << 4 * i | int(neg[d]) << sign_at)
            out[r, :256] = words.astype("<u4").view(np.uint8)
            out[r, 256:272] = scales.view(np.uint8)
            out[r, 272:288] = exps[0::2] | exps[1::2] << 4
    if k_pe_bits is not None:
        out[:, 288:] = np.ascontiguousarray(k_pe_bits).astype("<u2").view(np.uint8).reshape(n, 128)
    return out


def decode(rows):
    """(codes times 2^(e - 5) [n, 512], scales [n, 4]) in 64 bits."""
    rows = np.asarray(rows)
    n = rows.shape[0]
    words = np.ascontiguousarray(rows[:, :256]).view("<u4").astype(np.int64)
    val = np.zeros((n, 64, 8))
    for i in range(8):
        sign_at = 8 * i + 7 if i < 4 else 8 * (i - 4) + 3
        val[:, :, i] = MAGS[words >> 4 * i & 7] * (1 - 2 * (words >> sign_at & 1))
    exps = np.stack([rows[:, 272:288] & 15, rows[:, 272:288] >> 4], -1).reshape(n, 32).astype(np.int64)
    val = val.reshape(n, 32, 16) * 2.0 ** (exps[..., None] - 5)
    return val.reshape(n, 512), np.ascontiguousarray(rows[:, 256:272]).view("<f4").astype(np.float64)


def expand(rows):
    """The 528- (656-) byte rows of the same values, as a CPU uint8 tensor."""
    import torch
    rows = np.asarray(rows)
    code, _ = decode(rows)
    e4m3 = torch.from_numpy(code).to(torch.float8_e4m3fn)
    assert (e4m3.double() == torch.from_numpy(code)).all()       # nothing is rounded
    parts = [e4m3.view(torch.uint8), torch.from_numpy(np.ascontiguousarray(rows[:, 256:272]))]
    if rows.shape[1] == 416:
        parts.append(torch.from_numpy(np.ascontiguousarray(rows[:, 288:])))
    return torch.cat(parts, 1)


def make_pool(rows, layout, gen, amp=1.0):
    """Random 4-bit rows as a CPU uint8 tensor: every code, exponents a few steps apart, a magnitude for each row."""
    import torch
    pool = torch.randint(0, 256, (rows, ROW_BYTES[layout]), generator=gen, dtype=torch.uint8)
    e = torch.randint(6, 12, (rows, 16, 2), generator=gen)
    pool[:, 272:288] = (e[..., 0] | e[..., 1] << 4).to(torch.uint8)
    s = amp * (0.1 + 3.9 * torch.rand(rows, 1, generator=gen)) * (0.5 + torch.rand(rows, 4, generator=gen)) / 100.0
    pool[:, 256:272] = s.view(torch.uint8)
    if layout == "fp4_416":
        pool[:, 288:] = torch.randn(rows, 64, generator=gen).to(torch.bfloat16).view(torch.uint8)
    return pool
