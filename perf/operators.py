"""Cases of the dense serving operators around the paged FP8 MLA cache.

Four operators, as one engine step uses them: pages are handed to requests and
the slot map of the step's tokens is built (``pages_extend``), finished
requests return theirs (``pages_release``), queries and new KV rows get their
rotary positions and the rows are written to the 656-byte pool
(``rope_qkv656``), and the step's new tokens attend to everything their request
holds in the cache (``chunk_attn``).

``run`` computes them in plain torch operations, or, where ``own`` is set,
through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

ROW_BYTES = {"raw512": 512, "scaled528": 528, "rope656": 656}
KEY_DIMS = {"raw512": 512, "scaled528": 512, "rope656": 576}
SM_SCALE = 1.0 / math.sqrt(576.0)
THETA = 10000.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one request, one token, a short context: the latency of a single call
        dict(name="decode_one", op="chunk_attn", layout="raw512", B=1, H=16, new=1, ctx=100, page=64),
        # a decode batch of ragged contexts over raw rows
        dict(name="decode_batch_raw", op="chunk_attn", layout="raw512", B=64, H=16, new=1, ctx=8192, page=64),
        # two tokens a request (a drafted token is verified), all 128 heads on one GPU, 656-byte rows
        dict(name="verify_rope", op="chunk_attn", layout="rope656", B=32, H=128, new=2, ctx=4096, page=64),
        # a single request with a long history: one row of queries, the cache read by the whole GPU
        dict(name="decode_long_scaled", op="chunk_attn", layout="scaled528", B=1, H=32, new=1, ctx=131071, page=64),
        # a chunk of a long prompt over the context already in the cache
        dict(name="chunk_rope", op="chunk_attn", layout="rope656", B=1, H=32, new=4096, ctx=8192, page=64),
        # whole prompts of several requests, ragged, nothing in the cache before them
        dict(name="prompts_raw", op="chunk_attn", layout="raw512", B=5, H=16, new=2047, ctx=0, page=16),
        # the slot map of a decode step: one token for each of 64 requests
        dict(name="extend_decode", op="pages_extend", B=64, new=1, ctx=8192, page=64),
        # a prefill step: 256 ragged prompts, some of them continued
        dict(name="extend_prompts", op="pages_extend", B=256, new=512, ctx=2048, page=16),
        # a few of a decode batch's requests finish
        dict(name="release_some", op="pages_release", B=64, ctx=8192, page=64, finished=0.1),
        # a large batch is dropped at once
        dict(name="release_all", op="pages_release", B=512, ctx=16384, page=16, finished=1.0),
        # a decode step of 64 tokens: text positions, pairs half the width apart
        dict(name="rope_decode", op="rope_qkv656", T=64, H=16, image=False, interleaved=False, pool=131072),
        # a prefill chunk that holds an image: time, height and width positions, adjacent pairs
        dict(name="rope_chunk", op="rope_qkv656", T=4096, H=32, image=True, interleaved=True, pool=16384),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk_attn", "chunk_attn", "chunk_attn", "pages_extend", "pages_release", "rope_qkv656"])
    if op == "chunk_attn":
        layout = rng.choice(["raw512", "scaled528", "rope656"])
        H = rng.choice([8, 16, 32, 64, 128])
        page = rng.choice([1, 16, 64, 256])
        kind = rng.choice(["decode", "verify", "chunk", "prompts"])
        if kind == "decode":
            B = _log_int(rng, 1, 96)
            return dict(op=op, layout=layout, B=B, H=H, new=1, ctx=_log_int(rng, 1, min(131071, 600000 // B)), page=page)
        if kind == "verify":
            B = _log_int(rng, 1, 48)
            return dict(op=op, layout=layout, B=B, H=H, new=rng.randint(2, 8), ctx=_log_int(rng, 1, 8192), page=page)
        if kind == "chunk":
            new = _log_int(rng, 16, 4096)
            return dict(op=op, layout=layout, B=rng.randint(1, 2), H=min(H, 32 if new <= 1024 else 16), new=new,
                        ctx=_log_int(rng, 1, 8192), page=page)
        return dict(op=op, layout=layout, B=_log_int(rng, 1, 8), H=min(H, 16), new=_log_int(rng, 3, 2000), ctx=0, page=page)
    if op == "pages_extend":
        B = _log_int(rng, 1, 1024)
        return dict(op=op, B=B, new=_log_int(rng, 1, min(4096, 130000 // B)), ctx=_log_int(rng, 1, 16384),
                    page=rng.choice([1, 16, 64, 256]))
    if op == "pages_release":
        return dict(op=op, B=_log_int(rng, 1, 512), ctx=_log_int(rng, 1, 16384), page=rng.choice([16, 64, 256]),
                    finished=rng.choice([0.1, 0.5, 1.0]))
    return dict(op=op, T=_log_int(rng, 1, 4096), H=rng.choice([8, 16, 32]), image=rng.random() < 0.5,
                interleaved=rng.random() < 0.5, pool=16384)


def _lengths(case):
    """(new tokens, tokens cached before) of each request: the first of full size, the others ragged."""
    r = random.Random("%s/%s/%s/%s" % (case["op"], case["B"], case.get("new"), case["ctx"]))
    new = [case.get("new", 0) if i == 0 or case.get("new", 0) <= 1 else r.randint(1, case["new"]) for i in range(case["B"])]
    ctx = [case["ctx"] if i == 0 or case["ctx"] <= 1 else r.randint(case["ctx"] // 4, case["ctx"]) for i in range(case["B"])]
    return new, ctx


def _finished(case):
    r = random.Random("finished/%s/%s" % (case["B"], case["finished"]))
    return [i == 0 or r.random() < case["finished"] for i in range(case["B"])]


def _pages(n, page):
    return -(-n // page)


def work(case):
    if case["op"] == "chunk_attn":
        new, ctx = _lengths(case)
        T, kd, H = sum(new), KEY_DIMS[case["layout"]], case["H"]
        kv = [n + c for n, c in zip(new, ctx)]
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
        return {"bytes": T * H * (2 * kd + 1024 + 4) + sum(kv) * ROW_BYTES[case["layout"]]
                + 4 * sum(_pages(k, case["page"]) for k in kv) + 8 * case["B"],
                "flops": 2 * H * (kd + 512) * pairs}
    if case["op"] == "pages_extend":
        new, ctx = _lengths(case)
        taken = sum(_pages(n + c, case["page"]) - _pages(c, case["page"]) for n, c in zip(new, ctx))
        return {"bytes": 16 * case["B"] + 8 * taken + 4 * case["B"] + 16 * _token_rows(case), "flops": sum(new) * 4}
    if case["op"] == "pages_release":
        _, ctx = _lengths(case)
        back = sum(_pages(c, case["page"]) for c, f in zip(ctx, _finished(case)) if f)
        return {"bytes": 9 * case["B"] + 8 * back, "flops": case["B"] * 2 + back}
    T, H = case["T"], case["H"]
    return {"bytes": T * (H * 2304 + 1152 + 656 + 8 + 12), "flops": T * (H + 1) * 192 + T * 1536}


def _token_rows(case):
    """Rows of the step's token buffers: the tokens, rounded up as captured steps keep them."""
    return _pages(sum(_lengths(case)[0]), 64) * 64


# ------------------------------------------------------------------ inputs

def _rows_e4m3(rows, layout, gen):
    """A pool of cached rows: latents of one magnitude a row, written as the cache writes them."""
    dev = "cuda"
    out = torch.empty(rows, ROW_BYTES[layout], dtype=torch.uint8, device=dev)
    x = torch.randn(rows, 512, generator=gen, device=dev)
    if layout == "raw512":
        out[:] = x.mul_(0.5).to(torch.float8_e4m3fn).view(torch.uint8)
        return out
    x = (x * torch.empty(rows, 1, device=dev).uniform_(0.1, 4.0, generator=gen)).view(rows, 4, 128)
    s = x.abs().amax(-1, keepdim=True) / 448.0
    out[:, :512] = (x / s).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, 512)
    out[:, 512:528] = s.view(rows, 4).contiguous().view(torch.uint8)
    if layout == "rope656":
        out[:, 528:] = torch.randn(rows, 64, generator=gen, device=dev).to(torch.bfloat16).view(torch.uint8)
    return out


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)
    st = dict(case=case, op=case["op"])
    if case["op"] == "rope_qkv656":
        T, H = case["T"], case["H"]
        st["q_nope"] = torch.randn(T, H, 512, generator=gen, device=dev).to(torch.bfloat16)
        st["q_pe"] = torch.randn(T, H, 192, generator=gen, device=dev).to(torch.bfloat16)[:, :, 128:]   # the projection's last 64
        mult = torch.empty(T, 1, device=dev).uniform_(0.1, 8.0, generator=gen)
        st["kv_c"] = (torch.randn(T, 512, generator=gen, device=dev) * mult).to(torch.bfloat16)
        st["k_pe"] = torch.randn(T, 64, generator=gen, device=dev).to(torch.bfloat16)
        start = torch.randint(0, 100000, (1,), generator=gen, device=dev)
        t = torch.arange(T, device=dev)
        if case["image"]:      # 64 x 48 patches a frame: one time step, rows, columns
            st["positions"] = torch.stack([start + t // 3000, start + t % 3000 // 48, start + t % 48]).to(torch.int32)
        else:
            st["positions"] = (start + t)[None].expand(3, T).to(torch.int32).contiguous()
        st["sections"], st["theta"] = (8, 12, 12), THETA
        slots = torch.randperm(case["pool"], generator=gen, device=dev)[:T]
        slots[torch.rand(T, generator=gen, device=dev) < 0.02] = -1      # padding rows of a captured step
        st["slots"] = slots
        st["pool"] = torch.zeros(case["pool"], 656, dtype=torch.uint8, device=dev)
        st["q_out"] = torch.zeros(T, H, 576, dtype=torch.bfloat16, device=dev)
        if own:
            from sparse_mla_attention_page_gb300 import binding
            st["rope"] = binding.rope_spec(st["theta"], st["sections"], case["interleaved"])
        return st
    new, ctx = _lengths(case)
    page, B = case["page"], case["B"]
    st["seq_lens"] = torch.tensor(ctx, **i32)
    if case["op"] == "chunk_attn":
        kv = [n + c for n, c in zip(new, ctx)]
        T, H, layout = sum(new), case["H"], case["layout"]
        need = [_pages(k, page) for k in kv]
        n_pages = sum(need) + 7
        perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        p = torch.arange(max(need), device=dev)
        first = torch.tensor(np.cumsum([0] + need[:-1]), device=dev)[:, None]
        held = p[None] < torch.tensor(need, device=dev)[:, None]
        st["page_table"] = torch.where(held, perm[torch.where(held, first + p, 0)], -1)
        st["pool"] = _rows_e4m3(n_pages * page, layout, gen)
        st["q"] = torch.randn(T, H, KEY_DIMS[layout], generator=gen, device=dev).to(torch.bfloat16)
        st["cu_q"] = torch.tensor(np.cumsum([0] + new), **i32)
        st["kv_lens"] = torch.tensor(kv, **i32)
        st["max_new"], st["max_kv"] = max(new), max(kv)
        st["o"] = torch.zeros(T, H, 512, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(T, H, dtype=torch.float32, device=dev)
        if own:
            from sparse_mla_attention_page_gb300 import binding
            st["ws"] = binding.chunk_workspace_for(T, H, B, layout)
        return st
    held = [_pages(c, page) for c in ctx]
    most = max(_pages(n + c, page) for n, c in zip(new, ctx))
    n_pages = sum(_pages(n + c, page) for n, c in zip(new, ctx)) + 5
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    p = torch.arange(most, device=dev)
    first = torch.tensor(np.cumsum([0] + held[:-1]), device=dev)[:, None]
    mine = p[None] < torch.tensor(held, device=dev)[:, None]
    st["page_table"] = torch.where(mine, perm[torch.where(mine, first + p, 0)], -1)
    st["free_pages"] = torch.full((n_pages,), -1, **i32)
    st["free_pages"][:n_pages - sum(held)] = perm[sum(held):]
    st["free_count"] = torch.tensor([n_pages - sum(held)], **i32)
    st["free_count_out"] = torch.zeros(1, **i32)
    if case["op"] == "pages_release":
        st["finished"] = torch.tensor(_finished(case), device=dev)
        st["seq_lens_out"] = torch.zeros(B, **i32)
        return st
    rows = _token_rows(case)
    st["new_lens"] = torch.tensor(new, **i32)
    st["slots"] = torch.zeros(rows, dtype=torch.int64, device=dev)
    st["positions"], st["token_seq"] = torch.zeros(rows, **i32), torch.zeros(rows, **i32)
    st["cu_q"], st["kv_lens"] = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    return st


# -------------------------------------------------------------- plain forms

def _plain_chunk_attn(st):
    q, pool, table = st["q"], st["pool"], st["page_table"].long()
    case = st["case"]
    T, H, kd = q.shape
    B, page, n_max, kv_max = case["B"], case["page"], st["max_new"], st["max_kv"]
    cu, kv = st["cu_q"].long(), st["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    tok = torch.arange(n_max, device=q.device)
    live = tok[None] < n[:, None]
    at = torch.where(live, cu[:-1, None] + tok[None], T)
    qp = torch.cat([q.float(), q.new_zeros(1, H, kd, dtype=torch.float32)])[at].view(B, n_max * H, kd)
    j = torch.arange(kv_max, device=q.device)
    there = j[None] < kv[:, None]
    row = torch.where(there, table[:, j // page] * page + (j % page)[None], 0)
    rows = pool[row]
    lat = rows[..., :512].contiguous().view(torch.float8_e4m3fn).float()
    if kd != 512 or rows.shape[-1] == 528:
        scale = rows[..., 512:528].contiguous().view(torch.float32)
        lat = lat * scale.repeat_interleave(128, dim=-1)
    key = lat
    if kd == 576:
        key = torch.cat([lat, rows[..., 528:].contiguous().view(torch.bfloat16).float()], dim=-1)
    s = torch.bmm(qp, key.transpose(1, 2)).mul_(SM_SCALE).view(B, n_max, H, kv_max)
    seen = kv[:, None] - n[:, None] + tok[None] + 1              # keys each token may look at
    s = torch.where((j[None, None] < seen[..., None])[:, :, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = (s - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, n_max * H, kv_max), lat).view(B, n_max, H, 512) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log())[..., 0]
    o_out = torch.zeros(T + 1, H, 512, dtype=torch.bfloat16, device=q.device)
    lse_out = torch.zeros(T + 1, H, dtype=torch.float32, device=q.device)
    o_out[at] = o.to(torch.bfloat16)
    lse_out[at] = lse
    return dict(o=o_out[:T], lse=lse_out[:T])


def _plain_extend(st):
    page = st["case"]["page"]
    seq, new, table = st["seq_lens"].long(), st["new_lens"].long(), st["page_table"]
    have, need = (seq + page - 1) // page, (seq + new + page - 1) // page
    taken = (need - have).cumsum(0)
    first = taken - (need - have)
    p = torch.arange(table.shape[1], device=table.device)
    fresh = (p[None] >= have[:, None]) & (p[None] < need[:, None])
    rank = torch.where(fresh, first[:, None] + p[None] - have[:, None], 0)
    count = st["free_count"].long()
    table = torch.where(fresh, st["free_pages"][(count - 1 - rank).clamp(min=0)], table)
    ends = new.cumsum(0)
    t = torch.arange(st["slots"].shape[0], device=table.device)
    live = t < ends[-1]
    req = torch.searchsorted(ends, t, right=True).clamp(max=seq.shape[0] - 1)
    pos = torch.where(live, seq[req] + t - (ends - new)[req], 0)
    slot = table[req, pos // page].long() * page + pos % page
    i32 = torch.int32
    return dict(page_table=table, free_count=(count - taken[-1]).to(i32), slots=torch.where(live, slot, -1),
                positions=pos.to(i32), token_seq=torch.where(live, req, -1).to(i32),
                cu_q=torch.cat([ends.new_zeros(1), ends]).to(i32), kv_lens=(seq + new).to(i32))


def _plain_release(st):
    page = st["case"]["page"]
    seq, table, free = st["seq_lens"].long(), st["page_table"], st["free_pages"]
    back = torch.where(st["finished"], (seq + page - 1) // page, 0)
    ends = back.cumsum(0)
    count = st["free_count"].long()
    p = torch.arange(table.shape[1], device=table.device)
    at = torch.where(p[None] < back[:, None], count + (ends - back)[:, None] + p[None], free.shape[0])
    free = torch.cat([free, free.new_zeros(1)]).scatter(0, at.view(-1), table.view(-1))[:-1]
    return dict(free_pages=free, free_count=(count + ends[-1]).to(torch.int32),
                seq_lens=torch.where(st["finished"], 0, st["seq_lens"]))


def _turn(x, cos, sin, interleaved):
    """x [..., 64] turned by its 32 pairs' angles."""
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    c, d = a * cos - b * sin, b * cos + a * sin
    return (torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)).to(torch.bfloat16)


def _rope_outputs(st):
    pool = st["pool"]
    return dict(q=st["q_out"], latent=pool[:, :512].view(torch.float8_e4m3fn), scales=pool[:, 512:528].view(torch.float32),
                k_pe=pool[:, 528:].view(torch.bfloat16))


def _plain_rope(st):
    pair = torch.arange(32, device="cuda")
    axis = torch.tensor(st["sections"], device="cuda").cumsum(0)
    axis = torch.searchsorted(axis, pair, right=True)
    freq = st["theta"] ** (-pair.double() / 32)
    angle = st["positions"].double()[axis].t() * freq            # [T, 32]
    cos, sin = angle.cos().float(), angle.sin().float()
    inter = st["case"]["interleaved"]
    st["q_out"][..., :512] = st["q_nope"]
    st["q_out"][..., 512:] = _turn(st["q_pe"], cos[:, None], sin[:, None], inter)
    T = st["kv_c"].shape[0]
    x = st["kv_c"].float().view(T, 4, 128)
    s = x.abs().amax(-1, keepdim=True) / 448.0
    rows = torch.cat([torch.where(s > 0, x / s, 0.0).to(torch.float8_e4m3fn).view(torch.uint8).view(T, 512),
                      s.view(T, 4).view(torch.uint8),
                      _turn(st["k_pe"], cos, sin, inter).view(torch.uint8)], dim=1)
    put = st["slots"] >= 0
    st["pool"][st["slots"][put]] = rows[put]
    return _rope_outputs(st)


def run(st):
    if own:
        from sparse_mla_attention_page_gb300 import binding
        if st["op"] == "chunk_attn":
            binding.dsa_chunk_attn(st["q"], st["pool"], st["case"]["layout"], st["page_table"], st["case"]["page"],
                                   st["cu_q"], st["kv_lens"], SM_SCALE, st["o"], st["lse"], st["ws"])
            return dict(o=st["o"], lse=st["lse"])
        if st["op"] == "pages_extend":
            binding.dsa_pages_extend(st["seq_lens"], st["new_lens"], st["page_table"], st["case"]["page"],
                                     st["free_pages"], st["free_count"], st["free_count_out"], st["slots"],
                                     st["positions"], st["token_seq"], st["cu_q"], st["kv_lens"])
            return dict(page_table=st["page_table"], free_count=st["free_count_out"], slots=st["slots"],
                        positions=st["positions"], token_seq=st["token_seq"], cu_q=st["cu_q"], kv_lens=st["kv_lens"])
        if st["op"] == "pages_release":
            binding.dsa_pages_release(st["finished"], st["seq_lens"], st["page_table"], st["case"]["page"],
                                      st["free_pages"], st["free_count"], st["free_count_out"], st["seq_lens_out"])
            return dict(free_pages=st["free_pages"], free_count=st["free_count_out"], seq_lens=st["seq_lens_out"])
        binding.dsa_rope_qkv656(st["q_nope"], st["q_pe"], st["q_out"], st["kv_c"], st["k_pe"], st["slots"], st["pool"],
                                st["positions"], st["rope"])
        return _rope_outputs(st)
    return {"chunk_attn": _plain_chunk_attn, "pages_extend": _plain_extend, "pages_release": _plain_release,
            "rope_qkv656": _plain_rope}[st["op"]](st)


# -------------------------------------------------------------------- exact

def _e4m3_values():
    """The value of each E4M3 code, from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    v = []
    for code in range(256):
        e, f = code >> 3 & 15, code & 7
        mag = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        v.append(math.nan if code & 127 == 127 else -mag if code & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_chunk_attn(case, seed):
    st = prepare(case, seed)
    new, ctx = _lengths(case)
    if work(case)["flops"] > 8e12:
        return None
    codes, page, H = _e4m3_values(), case["page"], case["H"]
    T = sum(new)
    o = torch.zeros(T, H, 512, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["B"]):
        kv = new[b] + ctx[b]
        pages = st["page_table"][b, :_pages(kv, page)].long()
        rows = st["pool"].view(-1, page, st["pool"].shape[1])[pages].flatten(0, 1)[:kv]
        v = codes[rows[:, :512].long()]
        if case["layout"] != "raw512":
            v = (v.view(kv, 4, 128) * rows[:, 512:528].contiguous().view(torch.float32).double()[..., None]).view(kv, 512)
        k = v if case["layout"] != "rope656" else torch.cat([v, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
        step = max(1, int(4e8 // (H * kv)))
        for i in range(0, new[b], step):
            i1 = min(new[b], i + step)
            logits = torch.einsum("thd,kd->thk", st["q"][t0 + i:t0 + i1].double(), k) * SM_SCALE
            hidden = torch.arange(kv, device="cuda")[None] > (ctx[b] + torch.arange(i, i1, device="cuda"))[:, None]
            logits.masked_fill_(hidden[:, None], -math.inf)
            z = torch.logsumexp(logits, -1)
            lse[t0 + i:t0 + i1] = z
            o[t0 + i:t0 + i1] = torch.einsum("thk,kd->thd", logits.sub_(z[..., None]).exp_(), v)
        t0 += new[b]
    return dict(o=o, lse=lse)


def _exact_rope(case, seed):
    st = prepare(case, seed)
    T, inter = case["T"], case["interleaved"]
    pair_axis = [0] * 8 + [1] * 12 + [2] * 12
    z = torch.empty(T, 32, dtype=torch.complex128, device="cuda")
    for i in range(32):
        z[:, i] = torch.polar(torch.ones(T, dtype=torch.float64, device="cuda"),
                              st["positions"][pair_axis[i]].double() * math.pow(THETA, -2.0 * i / 64.0))

    def turned(x):
        x = x.double()
        pairs = x.unflatten(-1, (32, 2)) if inter else x.unflatten(-1, (2, 32)).transpose(-1, -2)
        w = torch.view_as_complex(pairs.contiguous())
        w = torch.view_as_real(w * (z if x.dim() == 2 else z[:, None]))
        return w.flatten(-2) if inter else w.transpose(-1, -2).flatten(-2)

    q = torch.cat([st["q_nope"].double(), turned(st["q_pe"])], -1)
    x = st["kv_c"].double().view(T, 4, 128)
    scale = (x.abs().amax(-1) / 448.0).float()
    y = (x.float() / scale[..., None]).double().view(T, 512)     # the row format divides in 32 bits
    values = _e4m3_values()[:127]                                # 0 .. 448, rising with the code
    hi = torch.searchsorted(values, y.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = y.abs() - values[lo], values[hi] - y.abs()
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    latent = torch.zeros(case["pool"], 512, dtype=torch.float64, device="cuda")
    scales = torch.zeros(case["pool"], 4, dtype=torch.float64, device="cuda")
    k_pe = torch.zeros(case["pool"], 64, dtype=torch.float64, device="cuda")
    put = st["slots"] >= 0
    at = st["slots"][put]
    latent[at] = (values[code] * y.sign())[put]
    scales[at] = (x.abs().amax(-1) / 448.0)[put]
    k_pe[at] = turned(st["k_pe"])[put]
    return dict(q=q, latent=latent, scales=scales, k_pe=k_pe)


def exact(case, seed):
    if case["op"] == "chunk_attn":
        return _exact_chunk_attn(case, seed)
    if case["op"] == "rope_qkv656":
        return _exact_rope(case, seed)
    return None
