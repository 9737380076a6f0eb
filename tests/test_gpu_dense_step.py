"""Engine steps of the dense operators together: pages, rotary and rows, attention, pages back."""
import math

import numpy as np
import pytest
import torch

import dense_ref as ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(576.0)
I32 = dict(dtype=torch.int32, device="cuda")


def test_prompt_decode_release():
    """Two prompts, three decode steps, a release and a new request in the freed slot; every step's attention is
    checked against the formula over the rows the earlier steps wrote."""
    B, H, page, T = 3, 16, 16, 160
    g = torch.Generator().manual_seed(0)
    table = torch.full((B, 12), -1, **I32)
    free, count = torch.randperm(30, generator=g).to(torch.int32).cuda(), torch.tensor([30], **I32)
    seq = torch.zeros(B, **I32)
    pool = torch.full((30 * page, 656), 0xFF, dtype=torch.uint8, device="cuda")     # nothing written yet: NaN
    slots, pos = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, **I32)
    ts, cu, err = torch.zeros(T, **I32), torch.zeros(B + 1, **I32), torch.zeros(1, **I32)
    spec = binding.rope_spec(10000.0, (8, 12, 12), True)
    ws = binding.chunk_workspace_for(T, H, B, "rope656")
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(T, H, device="cuda")
    sent = [[] for _ in range(B)]                            # each request's (latent, RoPE) rows, turned in 64 bits
    length = [0] * B
    for new, done in (([100, 37, 0], None), ([1, 1, 0], None), ([1, 1, 20], None), ([1, 1, 1], [False, True, False]),
                      ([1, 50, 4], None)):
        n = sum(new)
        rnd = (lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16))
        q_nope, q_pe, kv_c, k_pe = rnd(T, H, 512), rnd(T, H, 64), rnd(T, 512), rnd(T, 64)
        binding.dsa_pages_extend(seq, torch.tensor(new, **I32), table, page, free, count, count, slots, pos, ts, cu, seq,
                                 err_flag=err)
        binding.dsa_rope_qkv656(q_nope.cuda(), q_pe.cuda(), q, kv_c.cuda(), k_pe.cuda(), slots, pool,
                                pos[None].expand(3, -1), spec, err_flag=err)
        binding.dsa_chunk_attn(q, pool, "rope656", table, page, cu, seq, SCALE, o, lse, ws, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        positions = np.concatenate([np.arange(l, l + m) for l, m in zip(length, new)])
        assert pos[:n].tolist() == positions.tolist()
        turn = (lambda x: ref.turned(x[:n].double().numpy(), positions[None], [0] * 32, list(spec.inv_freq), True))
        qt = torch.cat([q_nope[:n].double(), torch.from_numpy(turn(q_pe))], -1)
        kt = torch.from_numpy(turn(k_pe))
        t = 0
        for b, m in enumerate(new):
            for i in range(m):
                sent[b].append((kv_c[t + i].double(), kt[t + i]))
                lat = torch.stack([r[0] for r in sent[b]])
                k = torch.cat([lat, torch.stack([r[1] for r in sent[b]])], 1)
                s = qt[t + i] @ k.T * SCALE
                w = s.softmax(-1)
                # rows in E4M3 (half a step 2^-4 of a value, smallest 2^-10 of amax / 448) shift scores and values
                dk = lat.abs() * 2.0 ** -4 + lat.abs().amax(1, keepdim=True) * 2.0 ** -18
                ds = (qt[t + i].abs()[:, :512] @ dk.T * SCALE + qt[t + i].abs() @ k.abs().T * SCALE * 2.0 ** -7).amax(-1, keepdim=True)
                bound = w @ dk + torch.expm1(2 * ds) * (w @ lat.abs()) + 2.0 ** -6
                assert ((o[t + i].cpu().double() - w @ lat).abs() <= bound).all()
                assert ((lse[t + i].cpu().double() - torch.logsumexp(s, -1)).abs() <= ds[:, 0] + 1e-4).all()
            t += m
            length[b] += m
        if done:
            binding.dsa_pages_release(torch.tensor(done, device="cuda"), seq, table, page, free, count, count, seq, err_flag=err)
            for b, d in enumerate(done):
                if d:
                    sent[b], length[b] = [], 0
            assert seq.tolist() == length
    held = sum(ref.pages_of(l, page) for l in length)
    assert int(count.item()) == 30 - held
    pages = [int(p) for b in range(B) for p in table[b, :ref.pages_of(length[b], page)].tolist()]
    assert sorted(pages + free[:30 - held].tolist()) == list(range(30))


@pytest.mark.parametrize("new,ctx,H", [([1] * 24, [500] * 24, 16), ([700, 300], [100, 2000], 32), ([1], [3], 8)])
def test_attention_directly_behind_the_rotary_writer(new, ctx, H):
    """Attention queued right behind the writer of its queries and rows, over buffers that earlier calls still use:
    eagerly and captured, the same bits as with a synchronisation in between."""
    page, B, T = 64, len(new), sum(new)
    g = torch.Generator(device="cuda").manual_seed(5)
    need = [ref.pages_of(a + b, page) for a, b in zip(new, ctx)]
    table = torch.full((B, max(need)), -1, **I32)
    at, cu, slots = 0, [0], []
    for b in range(B):
        table[b, :need[b]] = torch.arange(at, at + need[b])
        slots += [at * page + ctx[b] + i for i in range(new[b])]
        at += need[b]
        cu.append(cu[-1] + new[b])
    cu, kv = torch.tensor(cu, **I32), torch.tensor([a + b for a, b in zip(new, ctx)], **I32)
    slots = torch.tensor(slots, device="cuda")
    rnd = (lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16))
    pool = torch.zeros(at * page, 656, dtype=torch.uint8, device="cuda")
    binding.dsa_kv_write_rope656(rnd(at * page, 576), torch.arange(at * page, device="cuda"), pool)
    spec = binding.rope_spec()
    steps = [(rnd(T, H, 512), rnd(T, H, 64), rnd(T, 512), rnd(T, 64),
              torch.randint(0, 10 ** 6, (1, T), generator=g, device="cuda", dtype=torch.int32)) for _ in range(6)]
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16, device="cuda")
    ws = binding.chunk_workspace_for(T, H, B, "rope656")
    outs = [(torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")) for _ in steps]

    def step(i, wait=False):
        q_nope, q_pe, kv_c, k_pe, pos = steps[i]
        binding.dsa_rope_qkv656(q_nope, q_pe, q, kv_c, k_pe, slots, pool, pos, spec)
        if wait:
            torch.cuda.synchronize()
        binding.dsa_chunk_attn(q, pool, "rope656", table, page, cu, kv, SCALE, *outs[i], ws)

    def results():
        torch.cuda.synchronize()
        r = [(o.clone(), lse.clone()) for o, lse in outs]
        for o, lse in outs:
            o.zero_()
            lse.zero_()
        return r

    for i in range(6):
        step(i, wait=True)
        torch.cuda.synchronize()
    want = results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(6):
            step(i)
    for k in range(6):
        if k % 2:
            graph.replay()
        else:
            for i in range(6):
                step(i)
        for (o, lse), (wo, wl) in zip(results(), want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
