"""Cases of the operators around shared prefixes and 4-bit rows of the paged MLA cache.

A long prefix (a system prompt, a document) is written to the cache once and
serves every request that begins with it:

* ``write_read``: new rows are quantised to 4 bits as they are written
  (``dsa_kv_write_fp4``), and the requests' rows are read back in token order
  as BF16 (``dsa_kv_read``);
* ``read``: cached rows of a layout are read back as BF16 (``dsa_kv_read``);
* ``prefix_attn``: a batch whose requests begin with common rows attends to
  those once for all and to its own rows request by request;
* ``chunk_attn``: the dense attention of new tokens over 4-bit rows;
* ``release_own``: finished requests return their pages, but for those of the
  prefix that they share with others.

``run`` computes them in plain torch operations, or, where ``own`` is set,
through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

ROW_BYTES = {"raw512": 512, "scaled528": 528, "rope656": 656, "fp4_288": 288, "fp4_416": 416}
KEY_DIMS = {"raw512": 512, "scaled528": 512, "rope656": 576, "fp4_288": 512, "fp4_416": 576}
LAYOUTS = list(ROW_BYTES)
SM_SCALE = 1.0 / math.sqrt(576.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 tokens writes its rows and reads them back: latency
        dict(name="write_decode", op="write_read", layout="fp4_416", B=64, rows=1, page=64),
        # the rows of 16 documents on their way into the prefix cache, and back for a layer that attends in BF16
        dict(name="write_documents", op="write_read", layout="fp4_416", B=16, rows=4095, page=64),
        # the context of one request, read back before a chunk of its prompt attends without absorbed projections
        dict(name="read_context", op="read", layout="rope656", B=1, rows=8192, page=64),
        # ragged contexts of a batch of chunks, 4-bit rows, short pages
        dict(name="read_batch", op="read", layout="fp4_416", B=48, rows=4001, page=16),
        # four requests behind a short prompt: the latency of a call
        dict(name="prefix_few", op="prefix_attn", layout="raw512", B=4, G=1, H=16, new=1, prefix=1024, ctx=60, page=64),
        # a decode batch behind one document
        dict(name="prefix_batch", op="prefix_attn", layout="raw512", B=64, G=1, H=16, new=1, prefix=8192, ctx=500, page=64),
        # a decode batch of four system prompts with drafted tokens, 656-byte rows
        dict(name="prefix_drafts", op="prefix_attn", layout="rope656", B=96, G=4, H=8, new=2, prefix=6000, ctx=800, page=64),
        # an eighth of the heads, a very long document held in 4 bits, many requests
        dict(name="prefix_long_fp4", op="prefix_attn", layout="fp4_416", B=128, G=1, H=8, new=1, prefix=32768, ctx=1000, page=64),
        # a decode batch of ragged contexts over 4-bit rows
        dict(name="decode_fp4", op="chunk_attn", layout="fp4_288", B=64, H=16, new=1, ctx=8192, page=64),
        # a chunk of a prompt over a context held in 4 bits
        dict(name="chunk_fp4", op="chunk_attn", layout="fp4_416", B=1, H=32, new=2048, ctx=8192, page=64),
        # some requests of a batch behind one document finish
        dict(name="release_some", op="release_own", B=64, ctx=8192, shared=4096, page=64, finished=0.1),
        # a large batch behind one document is dropped at once
        dict(name="release_all", op="release_own", B=512, ctx=16384, shared=8192, page=16, finished=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write_read", "read", "prefix_attn", "prefix_attn", "prefix_attn", "chunk_attn", "release_own"])
    page = rng.choice([1, 16, 64, 256])
    if op == "write_read":
        B = _log_int(rng, 1, 256)
        return dict(op=op, layout=rng.choice(["fp4_288", "fp4_416"]), B=B, rows=_log_int(rng, 1, max(1, 60000 // B)), page=page)
    if op == "read":
        B = _log_int(rng, 1, 256)
        return dict(op=op, layout=rng.choice(LAYOUTS), B=B, rows=_log_int(rng, 1, max(1, 120000 // B)), page=page)
    if op == "prefix_attn":
        B = _log_int(rng, 2, 128)
        H = rng.choice([4, 8, 16, 32, 128])
        new = 1 if rng.random() < 0.6 else rng.randint(2, 5)
        most = max(200, min(32768, 60000000 // (B * H * new)))
        return dict(op=op, layout=rng.choice(LAYOUTS), B=B, G=rng.randint(1, min(B, 6)), H=H, new=new,
                    prefix=_log_int(rng, 50, most), ctx=_log_int(rng, 1, 1000), page=page)
    if op == "chunk_attn":
        layout = rng.choice(["fp4_288", "fp4_416"])
        if rng.random() < 0.5:
            B = _log_int(rng, 1, 96)
            return dict(op=op, layout=layout, B=B, H=rng.choice([8, 16, 32, 64]), new=1, ctx=_log_int(rng, 1, 300000 // B),
                        page=page)
        return dict(op=op, layout=layout, B=rng.randint(1, 3), H=rng.choice([8, 16]), new=_log_int(rng, 2, 1000),
                    ctx=_log_int(rng, 1, 6000), page=page)
    ctx = _log_int(rng, 2, 16384)
    return dict(op=op, B=_log_int(rng, 1, 512), ctx=ctx, shared=_log_int(rng, 1, ctx), page=rng.choice([16, 64, 256]),
                finished=rng.choice([0.1, 0.5, 1.0]))


def _ragged(case, what, most, least):
    """A length for each request: the first of full size, the others ragged."""
    r = random.Random("%s/%s/%s/%s" % (what, case["B"], most, least))
    return [most if i == 0 or most <= least else r.randint(least, most) for i in range(case["B"])]


def _group_cu(case):
    r = random.Random("groups/%s/%s" % (case["B"], case["G"]))
    return [0] + sorted(r.sample(range(1, case["B"]), case["G"] - 1)) + [case["B"]]


def _lengths(case):
    """(new tokens, rows of its own before them, rows of its prefix) of each request."""
    new = _ragged(case, "new", case["new"], 1)
    ctx = _ragged(case, "ctx", case["ctx"], max(1, case["ctx"] // 4))
    pre = [0] * case["B"]
    if case["op"] == "prefix_attn":
        cu = _group_cu(case)
        r = random.Random("prefix/%s/%s" % (case["G"], case["prefix"]))
        for g in range(case["G"]):
            p = case["prefix"] if g == 0 else r.randint(max(1, case["prefix"] // 2), case["prefix"])
            p = max(1, p // case["page"]) * case["page"]            # whole pages are shared
            pre[cu[g]:cu[g + 1]] = [p] * (cu[g + 1] - cu[g])
    return new, ctx, pre


def _finished(case):
    r = random.Random("finished/%s/%s" % (case["B"], case["finished"]))
    return [i == 0 or r.random() < case["finished"] for i in range(case["B"])]


def _pages(n, page):
    return -(-n // page)


def work(case):
    if case["op"] in ("write_read", "read"):
        n, wide, R = sum(_ragged(case, "rows", case["rows"], 1)), KEY_DIMS[case["layout"]] * 2, ROW_BYTES[case["layout"]]
        table = 4 * sum(_pages(r, case["page"]) for r in _ragged(case, "rows", case["rows"], 1)) + 4 * case["B"]
        if case["op"] == "read":
            return {"bytes": n * (R + wide) + table, "flops": n * 512}
        return {"bytes": n * (wide + 8 + R + wide) + table, "flops": n * 512 * 4}
    if case["op"] == "release_own":
        lens, _, own_pages = _release_lens(case)
        back = sum(p for p, f in zip(own_pages, _finished(case)) if f)
        return {"bytes": 13 * case["B"] + 8 * back, "flops": case["B"] * 3 + back}
    new, ctx, pre = _lengths(case)
    T, kd, H = sum(new), KEY_DIMS[case["layout"]], case["H"]
    rows = sum(n + c for n, c in zip(new, ctx))
    if case["op"] == "prefix_attn":
        cu = _group_cu(case)
        rows += sum(pre[cu[g]] for g in range(case["G"]))           # each prefix once
    pairs = sum(n * (c + p) + n * (n + 1) // 2 for n, c, p in zip(new, ctx, pre))
    return {"bytes": T * H * (2 * kd + 1024 + 4) + rows * ROW_BYTES[case["layout"]] + 4 * _pages(rows, case["page"])
            + 8 * case["B"], "flops": 2 * H * (kd + 512) * pairs}


def _release_lens(case):
    """(tokens, shared pages, pages of its own) of each request."""
    shared = max(1, case["shared"] // case["page"])
    lens = _ragged(case, "release", max(case["ctx"], shared * case["page"]), shared * case["page"])
    return lens, [shared] * case["B"], [_pages(n, case["page"]) - shared for n in lens]


# -------------------------------------------------------------- 4-bit rows
#
# Bytes [0, 256): 32 blocks of 16 dims, two little-endian 32-bit words each; dim i of a word's 8 has its magnitude code
# in bits 4 i .. 4 i + 2 (0, 0.5, 1, 1.5, 2, 3, 4, 6) and its sign in bit 8 i + 7 (i < 4) or 8 (i - 4) + 3.  [256, 272):
# FP32 scales of the four 128-dim groups, the group's largest magnitude / 384.  [272, 288): a nibble e for each block,
# low one first: its codes stand for code 2^(e - 5) scale, e the smallest of 0 .. 11 for which the block's largest
# x / scale is at most 7 2^(e - 5).  Codes are rounded to nearest, ties to the even code.  [288, 416): RoPE dims.

POWERS = [2.0 ** (e - 5) for e in range(16)]


def _fp4_rows(x, k_pe):
    """The rows of latents x [n, 512] (and k_pe [n, 64] BF16) as bytes."""
    n = x.shape[0]
    x = x.float().view(n, 4, 128)
    s = (x.abs().amax(-1, keepdim=True).double() / 384.0).float()
    y = torch.where(s > 0, x / s, 0.0).view(n, 32, 16)
    top = y.abs().amax(-1)
    e = torch.zeros(n, 32, dtype=torch.int32, device=x.device)
    for k in range(11):
        e += (top > 7.0 * 2.0 ** (k - 5)).int()
    mag = y.abs() / torch.tensor(POWERS, device=x.device)[e.long()][..., None]
    code = ((mag > 0.25).int() + (mag >= 0.75).int() + (mag > 1.25).int() + (mag >= 1.75).int() + (mag > 2.5).int()
            + (mag >= 3.5).int() + (mag > 5.0).int()).view(n, 64, 8)
    neg = (y < 0).int().view(n, 64, 8)
    out = torch.empty(n, 288 if k_pe is None else 416, dtype=torch.uint8, device=x.device)
    w = torch.zeros(n, 64, 4, dtype=torch.int32, device=x.device)              # bytes of a word
    for b in range(4):
        w[..., b] = (code[..., 2 * b] | code[..., 2 * b + 1] << 4 | neg[..., b] << 7 | neg[..., b + 4] << 3)
    out[:, :256] = w.view(n, 256).to(torch.uint8)
    out[:, 256:272] = s.view(n, 4).contiguous().view(torch.uint8)
    out[:, 272:288] = (e[:, 0::2] | e[:, 1::2] << 4).to(torch.uint8)
    if k_pe is not None:
        out[:, 288:] = k_pe.contiguous().view(torch.uint8)
    return out


def _rows_value(rows, layout):
    """(keys, latents) of pool rows [n, R] in 32 bits."""
    n, dev = rows.shape[0], rows.device
    if layout.startswith("fp4"):
        b = rows[:, :256].int().view(n, 64, 4)
        code = torch.stack([b & 7, b >> 4 & 7], -1).view(n, 64, 8)
        neg = torch.cat([b >> 7 & 1, b >> 3 & 1], -1)
        mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=dev)[code] * (1.0 - 2.0 * neg)
        e = rows[:, 272:288].int()
        e = torch.stack([e & 15, e >> 4], -1).view(n, 32, 1)
        lat = (mag.view(n, 32, 16) * torch.tensor(POWERS, device=dev)[e.long()]).view(n, 4, 128)
        lat = (lat * rows[:, 256:272].contiguous().view(torch.float32)[..., None]).view(n, 512)
        pe = rows[:, 288:]
    else:
        lat = rows[:, :512].contiguous().view(torch.float8_e4m3fn).float()
        if layout != "raw512":
            lat = (lat.view(n, 4, 128) * rows[:, 512:528].contiguous().view(torch.float32)[..., None]).view(n, 512)
        pe = rows[:, 528:]
    return (torch.cat([lat, pe.contiguous().view(torch.bfloat16).float()], -1) if KEY_DIMS[layout] == 576 else lat), lat


# ------------------------------------------------------------------ inputs

def _random_pool(rows, layout, gen):
    """A pool of cached rows: latents of one magnitude a row, written as the cache writes them."""
    dev = "cuda"
    out = torch.empty(rows, ROW_BYTES[layout], dtype=torch.uint8, device=dev)
    for r0 in range(0, rows, 65536):
        n = min(65536, rows - r0)
        x = torch.randn(n, 512, generator=gen, device=dev)
        part = out[r0:r0 + n]
        if layout == "raw512":
            part[:] = x.mul_(0.5).to(torch.float8_e4m3fn).view(torch.uint8)
            continue
        x = x * torch.empty(n, 1, device=dev).uniform_(0.1, 4.0, generator=gen)
        pe = None
        if KEY_DIMS[layout] == 576:
            pe = torch.randn(n, 64, generator=gen, device=dev).to(torch.bfloat16)
        if layout.startswith("fp4"):
            part[:] = _fp4_rows(x.to(torch.bfloat16), pe)
            continue
        s = x.view(n, 4, 128).abs().amax(-1, keepdim=True) / 448.0
        part[:, :512] = (x.view(n, 4, 128) / s).to(torch.float8_e4m3fn).view(torch.uint8).view(n, 512)
        part[:, 512:528] = s.view(n, 4).contiguous().view(torch.uint8)
        if pe is not None:
            part[:, 528:] = pe.view(torch.uint8)
    return out


def _table(need, gen, first=None):
    """A page table of need[b] pages a request, in no order, and the pages in all; first[b]: the request whose row
    begins b's row (its first `count` pages), or None."""
    dev = "cuda"
    fresh = [n - (first[b][1] if first and first[b] else 0) for b, n in enumerate(need)]
    n_pages = sum(fresh) + 5
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    host = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        k = 0
        if first and first[b]:
            k = first[b][1]
            host[b, :k] = host[first[b][0], :k]
        host[b, k:n] = perm[at:at + n - k]
        at += n - k
    return host, n_pages, perm[at:]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)
    st = dict(case=case, op=case["op"])
    page, B = case["page"], case["B"]
    if case["op"] in ("write_read", "read"):
        layout = case["layout"]
        lens = _ragged(case, "rows", case["rows"], 1)
        n = sum(lens)
        st["page_table"], n_pages, _ = _table([_pages(r, page) for r in lens], gen)
        st["cu_rows"] = torch.tensor(np.cumsum([0] + lens), **i32)
        st["out"] = torch.zeros(n, KEY_DIMS[layout], dtype=torch.bfloat16, device=dev)
        if case["op"] == "read":
            st["pool"] = _random_pool(n_pages * page, layout, gen)
            return st
        mult = torch.empty(n, 1, device=dev).uniform_(0.1, 8.0, generator=gen)
        st["kv_c"] = (torch.randn(n, 512, generator=gen, device=dev) * mult).to(torch.bfloat16)
        st["k_pe"] = torch.randn(n, 64, generator=gen, device=dev).to(torch.bfloat16) if KEY_DIMS[layout] == 576 else None
        st["pool"] = torch.zeros(n_pages * page, ROW_BYTES[layout], dtype=torch.uint8, device=dev)
        st["slots"] = _row_of(st)
        return st
    if case["op"] == "release_own":
        lens, shared, own_pages = _release_lens(case)
        st["page_table"], n_pages, rest = _table([_pages(n, page) for n in lens], gen,
                                                 [None if b == 0 else (0, shared[b]) for b in range(B)])
        st["seq_lens"] = torch.tensor(lens, **i32)
        st["shared_pages"] = torch.tensor(shared, **i32)
        st["finished"] = torch.tensor(_finished(case), device=dev)
        st["free_pages"] = torch.full((n_pages,), -1, **i32)
        st["free_pages"][:rest.shape[0]] = rest
        st["free_count"] = torch.tensor([rest.shape[0]], **i32)
        st["free_count_out"], st["seq_lens_out"] = torch.zeros(1, **i32), torch.zeros(B, **i32)
        return st
    new, ctx, pre = _lengths(case)
    kv = [n + c + p for n, c, p in zip(new, ctx, pre)]
    T, H, layout = sum(new), case["H"], case["layout"]
    first = None
    if case["op"] == "prefix_attn":
        cu = _group_cu(case)
        first = [None] * B
        for g in range(case["G"]):
            for b in range(cu[g] + 1, cu[g + 1]):
                first[b] = (cu[g], pre[b] // page)
        st["group_cu"] = torch.tensor(cu, **i32)
        st["prefix_lens"] = torch.tensor([pre[cu[g]] for g in range(case["G"])], **i32)
    st["page_table"], n_pages, _ = _table([_pages(k, page) for k in kv], gen, first)
    st["pool"] = _random_pool(n_pages * page, layout, gen)
    st["q"] = torch.randn(T, H, KEY_DIMS[layout], generator=gen, device=dev).to(torch.bfloat16)
    st["cu_q"] = torch.tensor(np.cumsum([0] + new), **i32)
    st["kv_lens"] = torch.tensor(kv, **i32)
    st["o"] = torch.zeros(T, H, 512, dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.zeros(T, H, dtype=torch.float32, device=dev)
    if own:
        from sparse_mla_attention_page_gb300 import binding
        make = binding.prefix_workspace_for if case["op"] == "prefix_attn" else binding.chunk_workspace_for
        st["ws"] = make(T, H, B, layout)
    return st


def _row_of(st):
    """Pool row of every row of the requests, in token order."""
    cu, page = st["cu_rows"].long(), st["case"]["page"]
    i = torch.arange(st["out"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True)
    j = i - cu[b]
    return st["page_table"].long()[b, j // page] * page + j % page


# -------------------------------------------------------------- plain forms

def _plain_write_read(st):
    layout = st["case"]["layout"]
    st["pool"][st["slots"]] = _fp4_rows(st["kv_c"], st["k_pe"])
    return _plain_read(st)


def _plain_read(st):
    return dict(out=_rows_value(st["pool"][_row_of(st)], st["case"]["layout"])[0].to(torch.bfloat16))


def _plain_attn(st):
    """Softmax over a request's prefix rows, if its group has any, and its own rows."""
    q, pool, table = st["q"], st["pool"], st["page_table"].long()
    case, layout = st["case"], st["case"]["layout"]
    T, H, kd = q.shape
    B, page = case["B"], case["page"]
    new, ctx, pre = _lengths(case)
    n_max, own_max = max(new), max(n + c for n, c in zip(new, ctx))
    cu, kv, p0 = st["cu_q"].long(), st["kv_lens"].long(), torch.tensor(pre, device=q.device)
    n = cu[1:] - cu[:-1]
    tok = torch.arange(n_max, device=q.device)
    live = tok[None] < n[:, None]
    at = torch.where(live, cu[:-1, None] + tok[None], T)
    qp = torch.cat([q.float(), q.new_zeros(1, H, kd, dtype=torch.float32)])[at].view(B, n_max * H, kd)
    j = torch.arange(own_max, device=q.device)
    pos = p0[:, None] + j[None]                                  # of the request's own rows
    there = pos < kv[:, None]
    pos = torch.where(there, pos, 0)
    row = torch.where(there, table.gather(1, pos // page) * page + pos % page, 0)
    key, lat = (x.view(B, own_max, -1) for x in _rows_value(pool[row.view(-1)], layout))
    s = torch.bmm(qp, key.transpose(1, 2)).mul_(SM_SCALE).view(B, n_max, H, own_max)
    seen = kv[:, None] - p0[:, None] - n[:, None] + tok[None] + 1
    s = torch.where((j[None, None] < seen[..., None])[:, :, None], s, -math.inf).view(B, n_max * H, own_max)
    m = s.amax(-1, keepdim=True)
    parts = []                                                   # (requests, scores over the prefix, its latents)
    if case["op"] == "prefix_attn":
        gcu = _group_cu(case)
        for g in range(case["G"]):
            b0, b1, p = gcu[g], gcu[g + 1], pre[gcu[g]]
            i = torch.arange(p, device=q.device)
            pk, pv = _rows_value(pool[table[b0, i // page] * page + i % page], layout)
            sp = (qp[b0:b1].reshape(-1, kd) @ pk.t()).mul_(SM_SCALE).view(b1 - b0, n_max * H, p)
            parts.append((b0, b1, sp, pv))
            m[b0:b1] = torch.maximum(m[b0:b1], sp.amax(-1, keepdim=True))
    w = (s - m).exp_()
    l = w.sum(-1, keepdim=True)
    o = torch.bmm(w, lat)
    for b0, b1, sp, pv in parts:
        sp = (sp - m[b0:b1]).exp_()
        l[b0:b1] += sp.sum(-1, keepdim=True)
        o[b0:b1] += (sp.view(-1, sp.shape[-1]) @ pv).view(b1 - b0, -1, 512)
    o_out = torch.zeros(T + 1, H, 512, dtype=torch.bfloat16, device=q.device)
    lse_out = torch.zeros(T + 1, H, dtype=torch.float32, device=q.device)
    o_out[at] = (o / l).view(B, n_max, H, 512).to(torch.bfloat16)
    lse_out[at] = (m + l.log()).view(B, n_max, H)
    return dict(o=o_out[:T], lse=lse_out[:T])


def _plain_release(st):
    page = st["case"]["page"]
    seq, table, free, shared = st["seq_lens"].long(), st["page_table"], st["free_pages"], st["shared_pages"].long()
    held = (seq + page - 1) // page
    back = torch.where(st["finished"], (held - shared).clamp(min=0), 0)
    ends = back.cumsum(0)
    count = st["free_count"].long()
    p = torch.arange(table.shape[1], device=table.device)
    mine = (p[None] >= shared[:, None]) & (p[None] < (shared + back)[:, None])
    at = torch.where(mine, count + (ends - back - shared)[:, None] + p[None], free.shape[0])
    free = torch.cat([free, free.new_zeros(1)]).scatter(0, at.view(-1), table.view(-1))[:-1]
    return dict(free_pages=free, free_count=(count + ends[-1]).to(torch.int32),
                seq_lens=torch.where(st["finished"], 0, st["seq_lens"]))


def run(st):
    if own:
        from sparse_mla_attention_page_gb300 import binding
        case = st["case"]
        if st["op"] == "write_read":
            binding.dsa_kv_write_fp4(st["kv_c"], st["slots"], st["pool"], k_pe=st["k_pe"])
        if st["op"] in ("write_read", "read"):
            binding.dsa_kv_read(st["pool"], case["layout"], st["page_table"], case["page"], st["cu_rows"], st["out"])
            return dict(out=st["out"])
        if st["op"] == "prefix_attn":
            binding.dsa_prefix_attn(st["q"], st["pool"], case["layout"], st["page_table"], case["page"], st["cu_q"],
                                    st["kv_lens"], st["group_cu"], st["prefix_lens"], SM_SCALE, st["o"], st["lse"], st["ws"])
            return dict(o=st["o"], lse=st["lse"])
        if st["op"] == "chunk_attn":
            binding.dsa_chunk_attn(st["q"], st["pool"], case["layout"], st["page_table"], case["page"], st["cu_q"],
                                   st["kv_lens"], SM_SCALE, st["o"], st["lse"], st["ws"])
            return dict(o=st["o"], lse=st["lse"])
        binding.dsa_pages_release_own(st["finished"], st["shared_pages"], st["seq_lens"], st["page_table"], case["page"],
                                      st["free_pages"], st["free_count"], st["free_count_out"], st["seq_lens_out"])
        return dict(free_pages=st["free_pages"], free_count=st["free_count_out"], seq_lens=st["seq_lens_out"])
    return {"write_read": _plain_write_read, "read": _plain_read, "prefix_attn": _plain_attn, "chunk_attn": _plain_attn,
            "release_own": _plain_release}[st["op"]](st)


# -------------------------------------------------------------------- exact

def _e4m3_values():
    """The value of each E4M3 code, from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    v = []
    for code in range(256):
        e, f = code >> 3 & 15, code & 7
        mag = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        v.append(math.nan if code & 127 == 127 else -mag if code & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _e2m1(code):
    """The value of a 3-bit magnitude: 2 exponent bits of bias 1, one mantissa bit."""
    return code / 2.0 if code < 2 else math.ldexp(2 + (code & 1), (code >> 1) - 2)


def _exact_rows(rows, layout):
    """(keys, latents) of pool rows in 64 bits."""
    n = rows.shape[0]
    if not layout.startswith("fp4"):
        lat = _e4m3_values()[rows[:, :512].long()]
        if layout != "raw512":
            lat = lat * rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        pe = rows[:, 528:]
    else:
        # each byte pairs two codes, dims 2 b and 2 b + 1 of a word; their signs lie elsewhere in the word
        pair = torch.tensor([[_e2m1(b & 7), _e2m1(b >> 4 & 7)] for b in range(256)], dtype=torch.float64, device="cuda")
        mag = pair[rows[:, :256].long()].view(n, 512)
        word = rows[:, :256].contiguous().view(torch.int32).long().view(n, 64, 1)
        bit = torch.tensor([7, 15, 23, 31, 3, 11, 19, 27], device="cuda")
        mag = torch.where((word >> bit & 1).view(n, 512) == 1, -mag, mag)
        nib = rows[:, 272:288].long()
        power = torch.zeros(n, 32, dtype=torch.float64, device="cuda")
        power[:, 0::2], power[:, 1::2] = (nib % 16).double() - 5, (nib // 16).double() - 5
        lat = mag * torch.exp2(power).repeat_interleave(16, 1)
        lat = lat * rows[:, 256:272].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        pe = rows[:, 288:]
    return (torch.cat([lat, pe.contiguous().view(torch.bfloat16).double()], 1) if KEY_DIMS[layout] == 576 else lat), lat


def _request_rows(st, b, first, count):
    page = st["case"]["page"]
    pages = st["page_table"][b, first // page:_pages(first + count, page)].long()
    rows = st["pool"].view(-1, page, st["pool"].shape[1])[pages].flatten(0, 1)
    return rows[first % page:first % page + count]


def _exact_write_read(case, seed):
    st = prepare(case, seed)
    x = st["kv_c"].double().view(-1, 4, 128)
    n = x.shape[0]
    scale = (x.abs().amax(-1) / 384.0).float()
    y = (x.float() / scale[..., None]).double().view(n, 32, 16)      # the row format divides in 32 bits
    top = y.abs().amax(-1)
    tops = torch.tensor([math.ldexp(7.0, k) for k in range(-5, 6)], dtype=torch.float64, device="cuda")
    unit = torch.tensor([math.ldexp(1.0, k) for k in range(-5, 7)], dtype=torch.float64, device="cuda")
    unit = unit[torch.searchsorted(tops, top.contiguous())][..., None]
    z = (y.abs() / unit).clamp(max=6.0)
    values = torch.tensor([_e2m1(c) for c in range(8)], dtype=torch.float64, device="cuda")
    hi = torch.searchsorted(values, z.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dl, dh = z - values[lo], values[hi] - z
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    lat = (values[code] * y.sign() * unit).view(n, 4, 128) * scale.double()[..., None]
    out = lat.view(n, 512)
    if st["k_pe"] is not None:
        out = torch.cat([out, st["k_pe"].double()], 1)
    return dict(out=out)


def _exact_read(case, seed):
    st = prepare(case, seed)
    lens = _ragged(case, "rows", case["rows"], 1)
    return dict(out=torch.cat([_exact_rows(_request_rows(st, b, 0, lens[b]), case["layout"])[0] for b in range(case["B"])]))


def _exact_attn(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    new, ctx, pre = _lengths(case)
    T, H = sum(new), case["H"]
    o = torch.zeros(T, H, 512, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["B"]):
        kv = new[b] + ctx[b] + pre[b]
        k, v = _exact_rows(_request_rows(st, b, 0, kv), case["layout"])
        step = max(1, int(4e8 // (H * kv)))
        for i in range(0, new[b], step):
            i1 = min(new[b], i + step)
            logits = torch.einsum("thd,kd->thk", st["q"][t0 + i:t0 + i1].double(), k) * SM_SCALE
            hidden = torch.arange(kv, device="cuda")[None] > (kv - new[b] + torch.arange(i, i1, device="cuda"))[:, None]
            logits.masked_fill_(hidden[:, None], -math.inf)
            z = torch.logsumexp(logits, -1)
            lse[t0 + i:t0 + i1] = z
            o[t0 + i:t0 + i1] = torch.einsum("thk,kd->thd", logits.sub_(z[..., None]).exp_(), v)
        t0 += new[b]
    return dict(o=o, lse=lse)


def exact(case, seed):
    if case["op"] == "write_read":
        return _exact_write_read(case, seed)
    if case["op"] == "read":
        return _exact_read(case, seed)
    if case["op"] in ("prefix_attn", "chunk_attn"):
        return _exact_attn(case, seed)
    return None
