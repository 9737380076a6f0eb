"""Plain 64-bit implementations of the dense serving operators, for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

ROW_BYTES = {"raw512": 512, "scaled528": 528, "rope656": 656}
KEY_DIMS = {"raw512": 512, "scaled528": 512, "rope656": 576}


def pages_of(n, page):
    return -(-n // page)


# ------------------------------------------------------------- page tables

def extend(seq, new, table, page, free, count, T):
    """Lists in, the call's outputs as a dict of lists (table: a copy)."""
    table = [list(r) for r in table]
    room = len(table[0]) * page
    err = 0
    total = sum(new)
    want = sum(pages_of(s + n, page) - pages_of(s, page) for s, n in zip(seq, new) if s >= 0 and n >= 0)
    if any(s < 0 or n < 0 or s + n > room for s, n in zip(seq, new)) or total > T or not 0 <= count <= len(free):
        err = 16
    elif want > count:
        err = 32
    out = dict(page_table=table, slots=[-1] * T, positions=[0] * T, token_seq=[-1] * T, cu_q=[0] * (len(seq) + 1),
               kv_lens=list(seq), free_count=count, err=err)
    if err:
        return out
    k = t = 0
    for b, (s, n) in enumerate(zip(seq, new)):
        for p in range(pages_of(s, page), pages_of(s + n, page)):
            table[b][p] = free[count - 1 - k]
            if table[b][p] < 0:
                out["err"] |= 2
            k += 1
        for i in range(n):
            pos = s + i
            pg = table[b][pos // page]
            out["slots"][t] = pg * page + pos % page if pg >= 0 else -1
            if pg < 0:
                out["err"] |= 2
            out["positions"][t], out["token_seq"][t] = pos, b
            t += 1
        out["cu_q"][b + 1] = t
        out["kv_lens"][b] = s + n
    out["free_count"] = count - k
    return out


def release(finished, seq, table, page, free, count):
    room = len(table[0]) * page
    back = [(b, p) for b, f in enumerate(finished) if f and seq[b] > 0 for p in range(pages_of(seq[b], page))]
    out = dict(free_pages=list(free), free_count=count, seq_lens=list(seq), err=0)
    if any(s < 0 or s > room for s in seq) or not 0 <= count <= len(free):
        out["err"] = 16
    elif count + len(back) > len(free):
        out["err"] = 32
    if out["err"]:
        return out
    if any(table[b][p] < 0 for b, p in back):
        out["err"] = 2
    for k, (b, p) in enumerate(back):
        out["free_pages"][count + k] = table[b][p]
    out["free_count"] = count + len(back)
    out["seq_lens"] = [0 if f else s for f, s in zip(finished, seq)]
    return out


# ------------------------------------------------------------------- rotary

def turned(x, positions, axis, inv_freq, interleaved, mscale=1.0):
    """x [T, ..., 64] float64 turned; positions [A, T] ints."""
    T = x.shape[0]
    out = np.array(x, dtype=np.float64)
    for i in range(32):
        ang = np.array([math.fmod(int(p) * inv_freq[i], 2 * math.pi) for p in positions[axis[i]]])
        c, s = mscale * np.cos(ang), mscale * np.sin(ang)
        shape = (T,) + (1,) * (x.ndim - 2)
        c, s = c.reshape(shape), s.reshape(shape)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        a, b = x[..., ia], x[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


# ---------------------------------------------------------------- attention

def make_pool(rows, layout, gen, amp=1.0):
    """Random pool bytes [rows, R] on the CPU, as the writers leave them."""
    pool = torch.empty(rows, ROW_BYTES[layout], dtype=torch.uint8)
    x = torch.randn(rows, 512, generator=gen) * amp
    if layout == "raw512":
        pool[:] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return pool
    x = (x * (0.1 + 3.9 * torch.rand(rows, 1, generator=gen))).view(rows, 4, 128)
    s = x.abs().amax(-1, keepdim=True) / 448.0
    pool[:, :512] = torch.where(s > 0, x / s, torch.zeros(())).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, 512)
    pool[:, 512:528] = s.reshape(rows, 4).contiguous().view(torch.uint8)
    if layout == "rope656":
        pool[:, 528:] = torch.randn(rows, 64, generator=gen).to(torch.bfloat16).view(torch.uint8)
    return pool


def dequant(rows, layout):
    """(keys, values) of pool rows in float64."""
    v = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double()
    if layout != "raw512":
        s = rows[:, 512:528].contiguous().view(torch.float32).double()
        v = v * s.repeat_interleave(128, dim=1)
    k = v if layout != "rope656" else torch.cat([v, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
    return k, v


def chunk_attn(q, pool, layout, table, page, cu, kv_lens, sm_scale, causal=True):
    """(O, LSE, bound of O's error, bound of LSE's) in float64, CPU tensors; rows of no request NaN.

    The bounds count, per output: the BF16 rounding of O (2^-8 |O|); the two E4M3 terms of each softmax weight
    (2^-4 of 2^-4 of it, and FP32 sums of exponentials: 2^-8 + 2^-12 of sum_j w_j |v_j|; E4M3's smallest step: see
    below); scores in FP32 sums of up to 576 exact
    products (2^-17 of sum_d |q_d k_jd|, and once again for the queries' two E4M3 terms), which enter O through
    the weights and LSE directly.

    E4M3's smallest step.  With S_j the power of two above row j's largest scale (1 for raw rows), the operand of group g is
    P = 2^(s_j + log2 S_j - M) (s_jg / S_j) c_g, c_g >= 1.  Its two terms leave at most half of lo's smallest step: 2^-10
    where M is at most max_j (s_j + log2 S_j) - 4, or 2^-14 where lo is kept 16 times larger and M is at most that
    maximum.  P multiplies the row's byte b_jd, and l = sum_j 2^(s_j - M) = 2^(s_J - M) / w_J for the row J of the maximum,
    so O is off by at most (2^-14 / l) sum_j |b_jd| <= 2^-14 max_j (w_j S_j) sum_j |b_jd|, and S_j <= 2 x the largest scale:
    2^-13 max_j (w_j max_g s_jg) sum_j |b_jd|."""
    T, H, _ = q.shape
    q = q.double()
    o = torch.full((T, H, 512), math.nan, dtype=torch.float64)
    lse = torch.full((T, H), math.nan, dtype=torch.float64)
    otol, ltol = torch.full_like(o, math.nan), torch.full_like(lse, math.nan)
    err = 0
    for b in range(len(kv_lens)):
        t0, t1, kv = int(cu[b]), int(cu[b + 1]), int(kv_lens[b])
        if not 0 <= t0 <= t1 <= T:
            err |= 16
            continue
        if not 0 <= kv <= table.shape[1] * page:
            err |= 16
            kv = max(0, min(kv, table.shape[1] * page))
        n = t1 - t0
        if n == 0:
            continue
        j = torch.arange(kv)
        pg = table[b].long()[j // page]
        row = pg * page + j % page
        ok = (pg >= 0) & (row < pool.shape[0])
        last = kv if not causal else max(0, kv)
        if not bool(ok[:last].all()):
            err |= 2
        rows = pool[torch.where(ok, row, 0)]
        k, v = dequant(rows, layout)
        codes = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double().abs()
        big = torch.ones(kv, dtype=torch.float64)
        if layout != "raw512":
            big = rows[:, 512:528].contiguous().view(torch.float32).double().abs().amax(1)
        for i in range(n):
            see = ok & (j < (kv - n + i + 1 if causal else kv))
            kk, vv = k[see], v[see]
            qi = q[t0 + i]
            if kk.shape[0] == 0:
                o[t0 + i], lse[t0 + i], otol[t0 + i], ltol[t0 + i] = 0.0, -math.inf, 0.0, 0.0
                continue
            s = qi @ kk.T * sm_scale
            z = torch.logsumexp(s, -1)
            w = (s - z[:, None]).exp()
            o[t0 + i], lse[t0 + i] = w @ vv, z
            mag = (qi.abs() @ kk.abs().T * abs(sm_scale)).amax(-1) * 2.0 ** -16 + 2.0 ** -18
            absv = w @ vv.abs()
            step = 2.0 ** -13 * (w * big[see]).amax(-1)[:, None] * codes[see].sum(0)
            otol[t0 + i] = (2.0 ** -8 * o[t0 + i].abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * mag[:, None]) * absv
                            + step)
            ltol[t0 + i] = mag + z.abs() * 2.0 ** -22
    return o, lse, otol, ltol, err
