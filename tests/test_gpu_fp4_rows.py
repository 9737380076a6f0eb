"""The writer of 4-bit rows and the reader by request, against the format's rules one by one."""
import numpy as np
import pytest
import torch

import dense_ref as ref
import fp4_ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
I32 = dict(dtype=torch.int32, device="cuda")
LAYOUTS = ["raw512", "scaled528", "rope656", "fp4_288", "fp4_416"]
WIDTH = {"raw512": 512, "scaled528": 512, "rope656": 576, "fp4_288": 512, "fp4_416": 576}


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def write(x, slots, rows, k_pe=None, fill=0x5A):
    pool = torch.full((rows, 288 if k_pe is None else 416), fill, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, **I32)
    binding.dsa_kv_write_fp4(x, slots, pool, k_pe=k_pe, err_flag=err)
    torch.cuda.synchronize()
    return pool.cpu().numpy(), int(err.item())


def check_rows(x, k_pe=None, extra=3, seed=0):
    """Rows scattered over a pool: bytes as the rules give them, the other rows untouched."""
    n = x.shape[0]
    slots = torch.from_numpy(np.random.default_rng(seed).permutation(n + extra)[:n].copy()).cuda()
    pool, err = write(x, slots, n + extra, k_pe)
    assert err == 0
    want = np.full_like(pool, 0x5A)
    want[slots.cpu().numpy()] = fp4_ref.encode(x.float().cpu().numpy(), None if k_pe is None else bits(k_pe))
    bad = np.argwhere(pool != want)
    assert bad.size == 0, f"{len(bad)} bytes differ, the first at row, byte {bad[0]}"


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 200])
def test_rows_of_any_number(n, rope):
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(n, 512, generator=g) * (0.01 + 8 * torch.rand(n, 1, generator=g))).to(BF)
    check_rows(x.cuda(), torch.randn(n, 64, generator=g).to(BF).cuda() if rope else None)


def test_more_rows_than_one_wave():
    """Every warp makes several passes: compared with the same rows written a few hundred at a time."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 30011
    x = torch.randn(n, 512, generator=g, device="cuda").to(BF)
    pe = torch.randn(n, 64, generator=g, device="cuda").to(BF)
    one = torch.zeros(n, 416, dtype=torch.uint8, device="cuda")
    binding.dsa_kv_write_fp4(x, torch.arange(n, device="cuda"), one, k_pe=pe)
    few = torch.zeros_like(one)
    for i in range(0, n, 500):
        m = min(500, n - i)
        binding.dsa_kv_write_fp4(x[i:i + m], torch.arange(i, i + m, device="cuda"), few, k_pe=pe[i:i + m])
    assert torch.equal(one, few)
    assert np.array_equal(one[-40:].cpu().numpy(), fp4_ref.encode(x[-40:].float().cpu().numpy(), bits(pe[-40:])))


def test_ties_and_borders():
    """Values at and next to the borders of codes and of block exponents, in each block's place, both signs."""
    z = [0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5, 7, 7.5]
    rng = np.random.default_rng(0)
    rows = []
    for e in range(12):
        for _ in range(3):
            row = rng.choice(z, (4, 128)) * 2.0 ** (e - 5) * rng.choice([-1.0, 1.0], (4, 128))
            row[:, 0] = 384.0                          # the group's largest: scale 1 (3 times a power of two, exact in BF16)
            row = np.where(np.abs(row) > 384, 384, row)
            rows.append(row.reshape(512))
    x = torch.from_numpy(np.array(rows)).to(BF)
    assert (x.double().numpy() == np.array(rows)).all()
    check_rows(x.cuda())
    near = x.view(torch.int16) + torch.from_numpy(rng.integers(-1, 2, x.shape).astype(np.int16))
    near = torch.where(x == 0, x.view(torch.int16), near).view(BF)      # one BF16 step to either side
    check_rows(near.cuda())
    check_rows((x.double() * 3).to(BF).cuda())
    check_rows((x.double() / 7).to(BF).cuda())


def test_every_bf16_number():
    """Every finite BF16 pattern beside every magnitude of its group; signs of zero; numbers below FP32's normal range."""
    b = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(b.view(np.int16)).view(BF)
    x = x[torch.isfinite(x)].reshape(-1)
    x = torch.cat([x, x[:(-x.numel()) % 512]]).view(-1, 512)
    check_rows(x.cuda())
    perm = torch.from_numpy(np.random.default_rng(1).permutation(x.numel()))
    check_rows(x.reshape(-1)[perm].view(-1, 512).cuda())
    zero = torch.zeros(3, 512, dtype=BF)
    zero[1] = -0.0
    zero[2, :130] = 1e-40
    check_rows(zero.cuda())


def test_nan_and_infinity():
    """A group that holds one gets scale NaN, reads as NaN; the others are as they would be without it."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn(6, 512, generator=g).to(BF)
    x[0, 5], x[1, 300], x[2, 511], x[3, 128] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[4, 64:192] = float("nan")
    pool, err = write(x.cuda(), torch.arange(6).cuda(), 6)
    assert err == 0
    want = fp4_ref.encode(x.float().numpy())
    sv, ws = pool[:, 256:272].copy().view("<f4"), want[:, 256:272].copy().view("<f4")
    assert np.array_equal(np.isnan(sv), np.isnan(ws)) and np.isnan(sv).sum() == 6
    ok = ~np.isnan(ws)
    assert np.array_equal(sv[ok], ws[ok])
    assert np.array_equal(pool[:, :256].reshape(6, 4, 64)[ok], want[:, :256].reshape(6, 4, 64)[ok])
    out = torch.zeros(6, 512, dtype=BF, device="cuda")
    binding.dsa_kv_read(torch.from_numpy(pool).cuda(), "fp4_288", torch.zeros(1, 1, **I32), 6, torch.tensor([0, 6], **I32), out)
    assert np.array_equal(out.isnan().view(6, 4, 128).all(-1).cpu().numpy(), ~ok)
    assert np.array_equal(out.isnan().view(6, 4, 128).any(-1).cpu().numpy(), ~ok)


def test_slots_and_strides():
    """Skipped and out-of-range slots; rows that are parts of wider ones, at an odd vector offset."""
    g = torch.Generator().manual_seed(8)
    wide = torch.randn(9, 1000, generator=g).to(BF).cuda()
    x, pe = wide[:, 8:520], wide[:, 522:586]
    slots = torch.tensor([4, -1, 0, 11, 7, -5, 12, 2, 1 << 40]).cuda()
    pool, err = write(x, slots, 11, pe)
    assert err == binding.DSA_DEV_ERR_SLOT_RANGE
    want = np.full((11, 416), 0x5A, np.uint8)
    rows = fp4_ref.encode(x.float().cpu().numpy(), bits(pe))
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < 11:
            want[s] = rows[i]
    assert np.array_equal(pool, want)
    one = wide[:1].expand(9, 1000)                     # the same row for every slot
    pool, err = write(one[:, 8:520], torch.arange(9).cuda(), 9, one[:, 522:586])
    assert err == 0 and (pool == pool[0]).all()


def test_expands_to_e4m3():
    """Every code under every exponent is a value of E4M3's normal numbers, or zero."""
    v = {float(m) * 2.0 ** (e - 5) for m in fp4_ref.MAGS for e in range(12)} - {0.0}
    t = torch.tensor(sorted(v), dtype=torch.float64)
    assert (t.to(torch.float8_e4m3fn).double() == t).all() and t.min() >= 2.0 ** -6 and t.max() == 384


# ------------------------------------------------------------------- reader

def random_pool(rows, layout, g):
    if not layout.startswith("fp4"):
        return ref.make_pool(rows, layout, g)
    pool = torch.randint(0, 256, (rows, 288 if layout == "fp4_288" else 416), generator=g, dtype=torch.uint8)
    pool[:, 256:272] = (0.01 + torch.rand(rows, 4, generator=g)).view(torch.uint8)
    e = torch.randint(0, 12, (rows, 16, 2), generator=g)
    pool[:, 272:288] = (e[..., 0] | e[..., 1] << 4).to(torch.uint8)
    if layout == "fp4_416":
        pool[:, 288:] = torch.randn(rows, 64, generator=g).to(BF).view(torch.uint8)
    return pool


def expected(pool, layout):
    """BF16 rows: the FP32 product rounded once, then the RoPE bits."""
    if layout.startswith("fp4"):
        code, s = fp4_ref.decode(pool.numpy())
        lat = torch.from_numpy(code.astype(np.float32)) * torch.from_numpy(s.astype(np.float32)).repeat_interleave(128, 1)
        pe = pool[:, 288:]
    else:
        lat = pool[:, :512].contiguous().view(torch.float8_e4m3fn).float()
        if layout != "raw512":
            lat = lat * pool[:, 512:528].contiguous().view(torch.float32).repeat_interleave(128, 1)
        pe = pool[:, 528:]
    out = lat.to(BF)
    return torch.cat([out, pe.contiguous().view(BF)], 1) if WIDTH[layout] == 576 else out


def check_read(lens, layout, page, starts=None, lead=0, tail=0, stride=None, seed=0, damage=None):
    """damage(table, cu): changes either before the call; the rows it concerns are expected untouched."""
    g = torch.Generator().manual_seed(seed)
    st = [0] * len(lens) if starts is None else starts
    need = [ref.pages_of(n + s, page) for n, s in zip(lens, st)]
    n_pages = sum(need) + 2
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    pool = random_pool(n_pages * page, layout, g)
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    cu = torch.tensor(cu, dtype=torch.int32)
    n, w = int(cu[-1]) + tail, WIDTH[layout]
    want = torch.full((n, w), 3.0, dtype=BF)
    skip, err_want = damage(table) if damage else (set(), 0)
    rows = expected(pool, layout)
    for b, m in enumerate(lens):
        for i in range(m):
            j = st[b] + i
            if (b, j) not in skip:
                want[int(cu[b]) + i] = rows[int(table[b, j // page]) * page + j % page]
    buf = torch.full((n, stride or w), 3.0, dtype=BF, device="cuda")
    err = torch.zeros(1, **I32)
    binding.dsa_kv_read(pool.cuda(), layout, table.cuda(), page, cu.cuda(), buf[:, :w],
                        starts=None if starts is None else torch.tensor(starts, **I32), err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    assert np.array_equal(bits(buf[:, :w]), bits(want))
    assert (buf[:, w:] == 3.0).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 3, 16, 64, 256])
def test_read_page_sizes(layout, page):
    check_read([70, 1, 0, 33, 128], layout, page, seed=page)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lens", [[1], [0, 1, 0], [3] * 70, [1] * 300, [0] * 40 + [5, 0, 9]])
def test_read_lengths(layout, lens):
    check_read(lens, layout, 16, seed=len(lens))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_read_parts(layout):
    """From a key on, into rows of a wider buffer, between rows of no request."""
    check_read([40, 17, 0, 64], layout, 16, starts=[5, 100, 3, 16], lead=7, tail=30, stride=600, seed=3)


def test_read_more_rows_than_one_wave():
    check_read([20000, 1, 17000, 9], "fp4_288", 64, seed=4)


def test_read_thousands_of_requests():
    """More offsets than lie in shared memory."""
    check_read([1, 0, 2, 0] * 700, "raw512", 4, seed=5)


@pytest.mark.parametrize("layout", ["rope656", "fp4_416"])
def test_read_bad_pages(layout):
    def damage(table):
        table[0, 1], table[2, 0] = -3, 1 << 20
        return {(0, j) for j in range(16, 32)} | {(2, j) for j in range(16)}, binding.DSA_DEV_ERR_PAGE_RANGE
    check_read([50, 20, 30], layout, 16, seed=6, damage=damage)


def test_read_starts_out_of_range():
    def damage(table):
        return {(0, j) for j in range(-2, 8)} | {(2, j) for j in range(0, 300)}, binding.DSA_DEV_ERR_LENGTH
    g = torch.Generator().manual_seed(9)
    pool = random_pool(64, "raw512", g)
    table = torch.zeros(3, 4, **I32)
    out = torch.full((30, 512), 3.0, dtype=BF, device="cuda")
    err = torch.zeros(1, **I32)
    binding.dsa_kv_read(pool.cuda(), "raw512", table, 16, torch.tensor([0, 10, 20, 30], **I32), out,
                        starts=torch.tensor([-2, 0, 60], **I32), err_flag=err)
    assert int(err.item()) == binding.DSA_DEV_ERR_LENGTH
    assert (out[:10] == 3).all() and (out[24:] == 3).all()      # a negative start; keys behind the row's 64
    assert np.array_equal(bits(out[10:20]), bits(expected(pool, "raw512")[:10]))
    assert np.array_equal(bits(out[20:24]), bits(expected(pool, "raw512")[12:16]))


@pytest.mark.parametrize("cu", [[0, 20, 10, 30], [-5, 10, 20, 30], [0, 10, 20, 31], [9, 3, 1, 0]])
def test_read_offsets_out_of_order(cu):
    """Flagged; nothing outside the buffer is written."""
    pool = random_pool(64, "raw512", torch.Generator().manual_seed(9))
    buf = torch.full((50, 512), 3.0, dtype=BF, device="cuda")
    err = torch.zeros(1, **I32)
    binding.dsa_kv_read(pool.cuda(), "raw512", torch.zeros(3, 4, **I32), 16, torch.tensor(cu, **I32), buf[10:40], err_flag=err)
    assert int(err.item()) == binding.DSA_DEV_ERR_LENGTH
    assert (buf[:10] == 3).all() and (buf[40:] == 3).all()


def test_written_and_read_back_in_a_graph():
    """Behind the writer on the same stream, captured and replayed over new rows and lengths; on a side stream."""
    g = torch.Generator(device="cuda").manual_seed(11)
    B, page, T = 3, 16, 90
    table = torch.arange(B * 3, **I32).view(B, 3)
    x, pe = torch.zeros(T, 512, dtype=BF, device="cuda"), torch.zeros(T, 64, dtype=BF, device="cuda")
    slots, cu = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(B + 1, **I32)
    pool = torch.zeros(B * 3 * page, 416, dtype=torch.uint8, device="cuda")
    out = torch.zeros(T, 576, dtype=BF, device="cuda")

    def step():
        binding.dsa_kv_write_fp4(x, slots, pool, k_pe=pe)
        binding.dsa_kv_read(pool, "fp4_416", table, page, cu, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([40, 1, 33], [48, 0, 1], [2, 40, 48]):
        x.copy_(torch.randn(T, 512, generator=g, device="cuda"))
        pe.copy_(torch.randn(T, 64, generator=g, device="cuda"))
        s = [b * 3 * page + i for b, n in enumerate(lens) for i in range(n)]
        slots.copy_(torch.tensor(s + [-1] * (T - len(s))))
        cu.copy_(torch.tensor([0, lens[0], lens[0] + lens[1], sum(lens)]))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(lens)
        rows = torch.from_numpy(fp4_ref.encode(x[:n].float().cpu().numpy(), bits(pe[:n])))
        assert np.array_equal(bits(out[:n]), bits(expected(rows, "fp4_416"))) and (out[n:] == 3.0).all()


def test_rows_behind_32_bits():
    """A pool of more than 2^31 bytes: rows written, read and attended at its end as in a small one."""
    n, page, kv = 5_400_000, 64, 300
    big = torch.empty(n, 416, dtype=torch.uint8, device="cuda")
    small = torch.zeros(8 * page, 416, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    x, pe = torch.randn(kv, 512, generator=g, device="cuda").to(BF), torch.randn(kv, 64, generator=g, device="cuda").to(BF)
    q = torch.randn(2, 16, 576, generator=g, device="cuda").to(BF)
    cu, lens = torch.tensor([0, 2], **I32), torch.tensor([kv], **I32)
    outs = []
    for pool, first in ((big, n // page - 8), (small, 0)):
        table = (first + torch.arange(7, -1, -1, **I32))[None].contiguous()
        j = torch.arange(kv, device="cuda")
        slots = table[0].long()[j // page] * page + j % page
        binding.dsa_kv_write_fp4(x, slots, pool, k_pe=pe)
        out = torch.zeros(kv, 576, dtype=BF, device="cuda")
        binding.dsa_kv_read(pool, "fp4_416", table, page, torch.tensor([0, kv], **I32), out)
        o, lse = torch.zeros(2, 16, 512, dtype=BF, device="cuda"), torch.zeros(2, 16, device="cuda")
        binding.dsa_chunk_attn(q, pool, "fp4_416", table, page, cu, lens, 0.04, o, lse, binding.chunk_workspace_for(2, 16, 1, "fp4_416"))
        big_call = torch.zeros(600, 16, 512, dtype=BF, device="cuda")          # (whose rows are expanded first)
        binding.dsa_chunk_attn(q[:1].expand(600, 16, 576).contiguous(), pool, "fp4_416", table, page, torch.tensor([0, 600], **I32),
                               lens, 0.04, big_call, torch.zeros(600, 16, device="cuda"),
                               binding.chunk_workspace_for(600, 16, 1, "fp4_416"), causal=False)
        outs.append((out, o, lse, big_call))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and (a != 0).any()


def test_binding_refusals():
    x, pool = torch.zeros(4, 512, dtype=BF, device="cuda"), torch.zeros(8, 288, dtype=torch.uint8, device="cuda")
    slots, out = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, 512, dtype=BF, device="cuda")
    pe = torch.zeros(4, 64, dtype=BF, device="cuda")
    table, cu = torch.zeros(1, 2, **I32), torch.tensor([0, 4], **I32)
    bad = (TypeError, ValueError, binding.DsaError)
    for kw in (dict(kv_c=x.float()), dict(kv_c=x[:3]), dict(kv_c=x.cpu()), dict(slots=slots.int()), dict(pool=pool[:, :272]),
               dict(pool=torch.zeros(8, 416, dtype=torch.uint8, device="cuda")), dict(k_pe=pe), dict(k_pe=pe[:, :32]),
               dict(kv_c=torch.zeros(4, 513, dtype=BF, device="cuda")[:, 1:]),
               dict(kv_c=torch.zeros(512, 4, dtype=BF, device="cuda").t())):
        with pytest.raises(bad):
            binding.dsa_kv_write_fp4(**dict(dict(kv_c=x, slots=slots, pool=pool), **kw))
    base = dict(pool=pool, layout="fp4_288", page_table=table, page_size=4, cu_rows=cu, out=out)
    for kw in (dict(layout="raw512"), dict(layout=3), dict(out=out[:, :500]), dict(out=out.float()), dict(cu_rows=cu[:1]),
               dict(cu_rows=cu.long()), dict(page_table=table.cpu()), dict(page_size=0), dict(starts=cu), dict(err_flag=slots),
               dict(out=torch.zeros(4, 513, dtype=BF, device="cuda")[:, :512])):
        with pytest.raises(bad):
            binding.dsa_kv_read(**dict(base, **kw))
    binding.dsa_kv_read(**base)
    binding.dsa_kv_write_fp4(x[:0], slots[:0], pool)
    binding.dsa_kv_read(**dict(base, out=out[:0]))
