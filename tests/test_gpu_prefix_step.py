"""Engine steps behind a shared prefix held in 4 bits: the prefix written once, requests that begin with it, their tokens
written and attended, rows read back, pages returned."""
import math

import numpy as np
import pytest
import torch

import dense_ref as ref
import fp4_ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(576.0)
I32 = dict(dtype=torch.int32, device="cuda")
BF = torch.bfloat16


@pytest.mark.parametrize("captured", [False, True])
def test_prefix_attach_decode_release(captured):
    """Row 0 of the page table is the prefix cache's, rows 1 .. B are requests.  Every step's attention is checked with the
    formula in 64 bits over the rows as the steps wrote them."""
    B, H, page, T, P = 24, 8, 16, 96, 6656 + 16
    g = torch.Generator().manual_seed(0)
    n_pages = P // page + 200
    table = torch.full((B + 1, P // page + 8), -1, **I32)
    free, count = torch.randperm(n_pages, generator=g).to(torch.int32).cuda(), torch.tensor([n_pages], **I32)
    err = torch.zeros(1, **I32)
    pool = torch.full((n_pages * page, 416), 0xFF, dtype=torch.uint8, device="cuda")      # nothing written yet: NaN
    rnd = (lambda *s: torch.randn(*s, generator=g).to(BF).cuda())

    # the document, written once
    seq = torch.zeros(1, **I32)
    slots, pos, ts = torch.zeros(P, dtype=torch.int64, device="cuda"), torch.zeros(P, **I32), torch.zeros(P, **I32)
    cu1 = torch.zeros(2, **I32)
    binding.dsa_pages_extend(seq, torch.tensor([P], **I32), table[:1], page, free, count, count, slots, pos, ts, cu1, seq, err_flag=err)
    doc_c, doc_pe = rnd(P, 512), rnd(P, 64)
    binding.dsa_kv_write_fp4(doc_c, slots, pool, k_pe=doc_pe, err_flag=err)
    doc = np.concatenate([fp4_ref.encode(doc_c[i:i + 512].float().cpu().numpy(), doc_pe[i:i + 512].view(torch.int16).cpu().numpy().view(np.uint16))
                          for i in range(0, P, 512)])
    back = torch.zeros(P, 576, dtype=BF, device="cuda")
    binding.dsa_kv_read(pool, "fp4_416", table[:1], page, cu1, back, err_flag=err)
    code, s = fp4_ref.decode(doc)
    want = (torch.from_numpy(code.astype(np.float32)) * torch.from_numpy(s.astype(np.float32)).repeat_interleave(128, 1)).to(BF)
    assert torch.equal(back[:, :512].cpu(), want) and torch.equal(back[:, 512:], doc_pe)

    # requests that begin with it
    mine = table[1:]
    mine[:, :P // page] = table[0, :P // page]
    shared = torch.full((B,), P // page, **I32)
    seq = torch.full((B,), P, **I32)
    slots, pos, ts = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, **I32), torch.zeros(T, **I32)
    cu, new = torch.zeros(B + 1, **I32), torch.zeros(B, **I32)
    gcu, plens = torch.tensor([0, B], **I32), torch.tensor([P], **I32)
    q, kv_c, k_pe = torch.zeros(T, H, 576, dtype=BF, device="cuda"), torch.zeros(T, 512, dtype=BF, device="cuda"), torch.zeros(T, 64, dtype=BF, device="cuda")
    o, lse = torch.zeros(T, H, 512, dtype=BF, device="cuda"), torch.zeros(T, H, device="cuda")
    ws = binding.prefix_workspace_for(T, H, B, "fp4_416")

    def step():
        binding.dsa_pages_extend(seq, new, mine, page, free, count, count, slots, pos, ts, cu, seq, err_flag=err)
        binding.dsa_kv_write_fp4(kv_c, slots, pool, k_pe=k_pe, err_flag=err)
        binding.dsa_prefix_attn(q, pool, "fp4_416", mine, page, cu, seq, gcu, plens, SCALE, o, lse, ws, err_flag=err)

    run = step
    if captured:
        step()                                               # (no new tokens: nothing changes)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    rows = [[] for _ in range(B)]                            # each request's own rows, as bytes
    r = np.random.default_rng(1)
    for k in range(4):
        n = r.integers(1, 5, B)
        n[r.integers(0, B, 3)] = 0
        if k == 2:
            n[:] = 1
        new.copy_(torch.from_numpy(n.astype(np.int32)))
        q.copy_(rnd(T, H, 576)), kv_c.copy_(rnd(T, 512)), k_pe.copy_(rnd(T, 64))
        o.fill_(7.0), lse.fill_(7.0)
        run()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        at = np.concatenate([[0], n.cumsum()])
        m = int(at[-1])
        enc = fp4_ref.encode(kv_c[:m].float().cpu().numpy(), k_pe[:m].view(torch.int16).cpu().numpy().view(np.uint16))
        for b in range(B):
            rows[b] += list(enc[at[b]:at[b + 1]])
        assert cu.tolist() == at.tolist() and seq.tolist() == [P + len(x) for x in rows]
        assert (o[m:] == 7.0).all() and (lse[m:] == 7.0).all()
        for b in (0, 1, 7, B - 1):                           # a few requests against the formula
            if n[b] == 0:
                continue
            wide = fp4_ref.expand(np.concatenate([doc, np.array(rows[b])]))
            kv = wide.shape[0]
            qb = q[at[b]:at[b + 1]].cpu()
            ro, rl, otol, ltol, _ = ref.chunk_attn(qb, wide, "rope656", torch.zeros(1, 1, dtype=torch.int32), kv,
                                                   [0, int(n[b])], [kv], SCALE)
            assert ((o[at[b]:at[b + 1]].cpu().double() - ro).abs() <= otol).all()
            assert ((lse[at[b]:at[b + 1]].cpu().double() - rl).abs() <= ltol).all()
    # the requests' own rows back, from behind the prefix
    lens = [len(x) for x in rows]
    cu_own = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), **I32)
    out = torch.zeros(sum(lens), 576, dtype=BF, device="cuda")
    binding.dsa_kv_read(pool, "fp4_416", mine, page, cu_own, out, starts=torch.full((B,), P, **I32), err_flag=err)
    code, s = fp4_ref.decode(np.concatenate([np.array(x) for x in rows]))
    want = (torch.from_numpy(code.astype(np.float32)) * torch.from_numpy(s.astype(np.float32)).repeat_interleave(128, 1)).to(BF)
    assert torch.equal(out[:, :512].cpu(), want)
    # a third finish: their own pages come back, the document's stay
    done = torch.arange(B, device="cuda") % 3 == 0
    before = int(count.item())
    own_pages = [mine[b, P // page:ref.pages_of(P + lens[b], page)].tolist() for b in range(B)]
    binding.dsa_pages_release_own(done, shared, seq, mine, page, free, count, count, seq, err_flag=err)
    torch.cuda.synchronize()
    want = [p for b in range(0, B, 3) for p in own_pages[b]]
    assert int(err.item()) == 0 and int(count.item()) == before + len(want)
    assert free[before:before + len(want)].tolist() == want
    assert seq.tolist() == [0 if b % 3 == 0 else P + lens[b] for b in range(B)]
    held = table[0, :P // page].tolist() + [p for b in range(B) if b % 3 for p in own_pages[b]]
    assert sorted(held + free[:int(count.item())].tolist()) == list(range(n_pages))
