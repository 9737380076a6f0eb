"""Dense attention of new tokens over the paged pool against the formula in 64 bits."""
import math
import random

import pytest
import torch

import dense_ref as ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
LAYOUTS = ["raw512", "scaled528", "rope656"]
SCALE = 1 / math.sqrt(576.0)
BF = torch.bfloat16


def make(new, ctx, H, layout, page=64, seed=0, qamp=1.0, amp=1.0, lead=0, tail=0):
    """Requests of new[b] tokens after ctx[b] cached ones; `lead` and `tail` query rows belong to none."""
    g = torch.Generator().manual_seed(seed)
    kv = [n + c for n, c in zip(new, ctx)]
    need = [ref.pages_of(max(k, 0), page) for k in kv]
    n_pages = sum(need) + 3
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(new), max(need + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    T = lead + sum(new) + tail
    cu = [lead]
    for n in new:
        cu.append(cu[-1] + n)
    q = (torch.randn(T, H, ref.KEY_DIMS[layout], generator=g) * qamp).to(BF)
    return dict(q=q, pool=ref.make_pool(n_pages * page, layout, g, amp), layout=layout, table=table, page=page,
                cu=torch.tensor(cu, dtype=torch.int32), kv=torch.tensor(kv, dtype=torch.int32), causal=True)


def run(w, stream=None, ws=None):
    T, H, _ = w["q"].shape
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    o = torch.full((T, H, 512), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = binding.chunk_workspace_for(T, H, w["table"].shape[0], w["layout"])
    ws.fill_(0xFF)                                        # what it held before has no effect
    torch.cuda.synchronize()
    binding.dsa_chunk_attn(d["q"], d["pool"], w["layout"], d["table"], w["page"], d["cu"], d["kv"], SCALE, o, lse, ws,
                           causal=w["causal"], err_flag=err, stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), int(err.item())


def check(w, err_want=0, **kw):
    whole_o, whole_lse, err = run(w, **kw)
    o, lse = whole_o, whole_lse
    ro, rl, otol, ltol, rerr = ref.chunk_attn(w["q"], w["pool"], w["layout"], w["table"], w["page"], w["cu"], w["kv"],
                                              SCALE, w["causal"])
    assert err == err_want == rerr
    out = torch.isnan(rl)                                  # rows of no request
    assert (o[out] == 7.0).all() and (lse[out] == 7.0).all()
    o, lse, ro, rl, otol, ltol = (x[~out] for x in (o, lse, ro, rl, otol, ltol))
    none = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), none) and (o[none] == 0).all()
    d = (o.double() - ro).abs() - otol
    assert torch.isfinite(o).all() and (d <= 0).all(), f"O off by {d.max():.3e} beyond the bound at {torch.nonzero(d > 0)[:3].tolist()}"
    d = ((lse.double() - rl).abs() - ltol)[~none]
    assert d.numel() == 0 or (d <= 0).all(), f"LSE off by {d.max():.3e} beyond the bound"
    return whole_o, whole_lse


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H", [1, 8, 16, 20, 32, 64, 128])
def test_single_tokens(layout, H):
    """Decode: one token a request, contexts around the tile's 128 keys and none at all."""
    check(make([1] * 9, [0, 1, 63, 126, 127, 128, 129, 255, 700], H, layout, seed=H))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256, 1000])
def test_page_sizes(layout, page):
    check(make([1, 5, 40], [300, 77, 130], 8, layout, page=page, seed=page))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("new,ctx", [([2], [0]), ([130], [0]), ([7, 1, 33, 0, 64], [0, 500, 10, 20, 129]), ([200], [301])])
@pytest.mark.parametrize("H", [3, 16])
def test_chunks(layout, new, ctx, H):
    """Prompts, chunks and single tokens in one batch; a request without new tokens."""
    check(make(new, ctx, H, layout, seed=sum(new) + H))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_all_heads_of_a_chunk(layout):
    check(make([9, 2], [400, 130], 128, layout, seed=2))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H", [16, 128])
def test_long_context_few_rows(layout, H):
    """One request spread over every SM."""
    check(make([1], [40000], H, layout, seed=3))
    check(make([3, 1], [20011, 9], H, layout, seed=4))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_more_work_than_sms(layout):
    """Many groups of query rows of unequal length: ranges begin and end inside requests."""
    r = random.Random(5)
    check(make([r.randint(1, 90) for _ in range(24)], [r.randint(0, 400) for _ in range(24)], 16, layout, seed=5))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_not_causal(layout):
    w = make([5, 130, 1], [60, 3, 300], 8, layout, seed=6)
    w["causal"] = False
    check(w)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("qamp,amp", [(40.0, 1.0), (1e-3, 1.0), (1.0, 20.0), (0.05, 100.0), (1.0, 1e-3)])
def test_amplitudes(layout, qamp, amp):
    """Peaked and flat softmax, large and small rows."""
    if layout == "raw512" and amp < 0.01:
        amp = 0.05
    check(make([1, 20], [900, 150], 16, layout, seed=7, qamp=qamp, amp=amp))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rising_scores(layout):
    """Keys whose scores rise along the sequence: the running maximum moves in every tile."""
    w = make([1, 3], [1500, 1300], 16, layout, seed=8)
    w["q"][:] = w["q"][:1, :1]
    base = w["q"][0, 0, :512].float()
    rows = torch.arange(w["kv"][0].item())
    slot = w["table"][0].long()[rows // 64] * 64 + rows % 64
    x = base[None] * (rows[:, None] / 500.0)
    if layout == "raw512":
        w["pool"][slot] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x = x.view(-1, 4, 128)
        s = x.abs().amax(-1, keepdim=True) / 448.0
        w["pool"][slot, :512] = torch.where(s > 0, x / s, torch.zeros(())).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 512)
        w["pool"][slot, 512:528] = s.reshape(-1, 4).contiguous().view(torch.uint8)
    check(w)


@pytest.mark.parametrize("layout", ["scaled528", "rope656"])
def test_zero_and_uneven_scales(layout):
    """All-zero rows, zero groups, groups of very different scales."""
    w = make([2, 40], [300, 200], 16, layout, seed=9)
    s = w["pool"][:, 512:528].contiguous().view(torch.float32)
    g = torch.Generator().manual_seed(1)
    s *= 2.0 ** torch.randint(-30, 4, s.shape, generator=g).float()
    s[::5] = 0
    s[::3, 1] = 0
    w["pool"][:, 512:528] = s.view(torch.uint8)
    check(w)


@pytest.mark.parametrize("layout", ["scaled528", "rope656"])
def test_groups_of_very_different_size(layout):
    """A 128-dim group that is 2^12 times smaller than the others in every row (and one that gets larger along the
    sequence) keeps its own precision: its bound counts the group's own rows, lifted by the power of two that all of
    them have in common."""
    w = make([2, 40], [900, 200], 16, layout, seed=23)
    s = w["pool"][:, 512:528].contiguous().view(torch.float32)
    s[:, 1] *= 2.0 ** -12
    j = torch.arange(int(w["kv"][0]))
    slot = w["table"][0].long()[j // 64] * 64 + j % 64
    s[slot, 3] *= 2.0 ** -(12 - j * 12 // j.numel()).float()
    w["pool"][:, 512:528] = s.view(torch.uint8)
    o, _ = check(w)
    # group 1 alone: every row's scale there is within 2^6 of every other's, so the lifted operand resolves at least
    # 2^-14 2^6 of the group's largest row; with the two terms and the BF16 rounding, per unit of the group's RMS:
    ro, _, _, _, _ = ref.chunk_attn(w["q"], w["pool"], layout, w["table"], 64, w["cu"], w["kv"], SCALE)
    g, rg = o.double()[:, :, 128:256], ro[:, :, 128:256]
    assert (g - rg).norm() <= 2.0 ** -7 * rg.norm()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_huge_and_tiny_queries(layout):
    """Finite BF16 queries at both ends of the type's range."""
    w = make([3], [200], 8, layout, seed=24)
    w["q"][0] = (w["q"][0].float() * 1e-36).to(BF)
    w["q"][1, :4] = 0
    w["pool"][:] = w["pool"][:1]                       # equal keys: any finite score gives the same weights
    w["q"][2, 0] = 0
    w["q"][2, 0, 0] = torch.finfo(BF).max
    check(w)


@pytest.mark.parametrize("layout", ["raw512", "rope656"])
@pytest.mark.parametrize("H", [160, 1024])
def test_many_heads(layout, H):
    check(make([2, 1], [30, 150], H, layout, seed=25))


def test_thousands_of_requests():
    """More requests, and more units, than the planning block has threads."""
    r = random.Random(26)
    check(make([r.randint(0, 2) for _ in range(2500)], [r.randint(0, 3) for _ in range(2500)], 3, "rope656", page=16, seed=26))


def test_overlapping_ranges_do_no_harm():
    """Query ranges that overlap beyond the work list's room are reported; nothing is computed, nothing breaks."""
    w = make([30] * 40, [5] * 40, 16, "raw512", page=16, seed=27)
    w["cu"] = torch.tensor([0, 1200] * 20 + [0], dtype=torch.int32)
    o, lse, err = run(w)
    assert err == 16 and (o == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("page", [16, 32, 64, 96, 256])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_both_row_loads_agree(layout, page):
    """Pages of a multiple of 32 rows come by TMA, others row by row: the same bits."""
    a = make([1, 40, 3], [300, 77, 130], 16, layout, page=page, seed=28)
    want = run(a)
    # the same rows as pages of one row
    table = torch.full((3, a["table"].shape[1] * page), -1, dtype=torch.int32)
    for b in range(3):
        j = torch.arange(int(a["kv"][b]))
        table[b, :j.numel()] = (a["table"][b].long()[j // page] * page + j % page).to(torch.int32)
    got = run(dict(a, table=table, page=1))
    assert got[2] == want[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_share_a_workspace():
    """Captured calls of different batches, replayed in turn on one stream with one workspace."""
    a, b = make([1, 30], [3000, 10], 16, "rope656", seed=29), make([40, 2], [900, 50], 16, "rope656", seed=30)
    want = [run(a), run(b)]
    ws = binding.chunk_workspace_for(42, 16, 2, "rope656")
    graphs, outs, keep = [], [], []
    for w in (a, b):
        d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
        T, H = d["q"].shape[:2]
        o, lse = torch.zeros(T, H, 512, dtype=BF, device="cuda"), torch.zeros(T, H, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.dsa_chunk_attn(d["q"], d["pool"], "rope656", d["table"], 64, d["cu"], d["kv"], SCALE, o, lse, ws)
        graphs.append(g)
        outs.append((o, lse))
        keep.append(d)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, lse), (wo, wl, _) in zip(outs, want):
        assert torch.equal(o.cpu(), wo) and torch.equal(lse.cpu(), wl)


@pytest.mark.parametrize("page", [64, 1])
def test_wait_that_runs_out(page):
    """With a limit of 0 the first wait that is not complete at once gives up: the call returns, the flag says so, and
    the next call is right."""
    w = make([1, 40], [700, 90], 16, "rope656", page=page, seed=31)
    want = run(w)
    old = binding.dsa_set_wait_limit_ns(0)
    try:
        _, _, err = run(w)
    finally:
        binding.dsa_set_wait_limit_ns(old)
    assert err & binding.DSA_DEV_ERR_TIMEOUT
    got = run(w)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rows_of_no_request_are_left(layout):
    check(make([3, 1, 17], [40, 200, 0], 8, layout, seed=10, lead=4, tail=9))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_queries_before_the_first_key(layout):
    """More new tokens than the request holds: the first see nothing."""
    w = make([10, 3, 1], [0, 0, 200], 8, layout, seed=11)
    w["kv"][0], w["kv"][1] = 4, 0
    check(w)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page,rows", [(64, 5), (64, 100), (256, 300), (16, 37), (7, 30)])
def test_pool_that_ends_inside_a_page(layout, page, rows):
    """Keys inside the pool's last, partial page count; those behind the pool's end are masked and reported."""
    w = make([1, 20], [rows - 1, 0], 16, layout, page=page, seed=32)
    w["pool"] = w["pool"][:rows].contiguous()
    ids = torch.arange(ref.pages_of(rows, page), dtype=torch.int32)
    w["table"] = ids.repeat(2, 1).contiguous()
    w["kv"] = torch.tensor([rows, min(rows, 20)], dtype=torch.int32)
    check(w)
    if rows % page:
        w["kv"][0] = min(rows + 1, ids.numel() * page)
        check(w, err_want=2)


@pytest.mark.parametrize("T,B", [(17, 1), (33, 2), (31, 16), (64, 4)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_rows_around_a_group(layout, T, B):
    """One head: query rows around the sizes of a group, more and fewer than an average request has."""
    r = random.Random(T)
    cut = sorted(r.sample(range(1, T), B - 1)) if B > 1 else []
    new = [b - a for a, b in zip([0] + cut, cut + [T])]
    check(make(new, [r.randint(0, 200) for _ in new], 1, layout, page=8, seed=33))


@pytest.mark.parametrize("tiles", [1, 3, 4])
@pytest.mark.parametrize("B", [3, 150, 154])
def test_groups_of_few_tiles(B, tiles):
    """Row groups of so many 128-key tiles each: whole to an SM, or spread, on either side of the number of SMs."""
    r = random.Random(35)
    kv = [128 * tiles - r.randint(0, 1) * r.randint(0, 127) for _ in range(B)]
    kv[0] = 128 * tiles
    check(make([1] * B, [k - 1 for k in kv], 4, "rope656", page=32, seed=35))


def test_most_requests():
    """DSA_MAX_REQUESTS requests of a token each."""
    B = 16384
    w = make([1] * B, [0] * B, 1, "raw512", page=1, seed=34)
    check(w)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_bad_pages_are_masked(layout):
    w = make([1, 30, 1], [200, 100, 64], 16, layout, seed=12)
    w["table"][0, 1] = -1
    w["table"][1, 0] = 10 ** 6
    w["table"][2, 0] = 2 ** 31 - 1
    w["table"][2, 1] = -5
    check(w, err_want=2)


@pytest.mark.parametrize("layout", ["raw512", "rope656"])
def test_bad_lengths(layout):
    w = make([2, 3, 4], [100, 100, 100], 8, layout, seed=13, tail=2)
    w["kv"][1] = -4
    check(w, err_want=16)
    w["kv"][1] = 10 ** 9
    o, lse, err = run(w)
    assert err & 16 and torch.isfinite(lse[:2]).all() and torch.isfinite(lse[5:9]).all()
    w["kv"][1] = 103
    w["cu"] = torch.tensor([0, 2, 1, 40], dtype=torch.int32)      # descending, then beyond T
    check(w, err_want=16)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_hidden_rows_may_hold_anything(layout):
    """NaN and infinities in rows that a query does not see: rows past the end of the last page, later tokens of
    the same chunk, pages of nobody."""
    w = make([1, 6, 70], [70, 190, 0], 16, layout, seed=14)
    want_o, want_l = check(w)
    used = torch.zeros(w["pool"].shape[0], dtype=torch.bool)
    for b in range(3):
        j = torch.arange(int(w["kv"][b]))
        used[w["table"][b].long()[j // 64] * 64 + j % 64] = True
    w["pool"][~used] = 0xFF
    o, lse, _ = run(w)
    assert torch.equal(o, want_o) and torch.equal(lse, want_l)
    # the last two tokens of request 2 hold NaN bytes (and NaN scales and RoPE dims); the one before an infinite scale
    slots = [int(w["table"][2, p // 64]) * 64 + p % 64 for p in (67, 68, 69)]
    if layout != "raw512":
        w["pool"][slots[0], 512:528] = torch.full((4,), math.inf).view(torch.uint8)
    w["pool"][slots[1:]] = 0x7F
    o, lse, _ = run(w)
    last = 7 + (67 if layout != "raw512" else 68)
    ok = [t for t in range(last)]
    assert torch.equal(o[ok], want_o[ok]) and torch.equal(lse[ok], want_l[ok])
    assert torch.isnan(o[last:]).all() and torch.isnan(lse[last:]).all()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_nan_and_inf_queries_stay_in_their_rows(layout):
    w = make([1, 40], [300, 100], 16, layout, seed=15)
    want_o, want_l = check(w)
    w["q"][0, 3, 5] = float("nan")
    w["q"][20, 9, 100] = float("inf")
    w["q"][30, 0, -1] = float("nan")
    o, lse, _ = run(w)
    for t, h in ((0, 3), (20, 9), (30, 0)):
        assert torch.isnan(o[t, h]).all() and torch.isnan(lse[t, h])
        o[t, h], lse[t, h] = want_o[t, h], want_l[t, h]
    assert torch.equal(o, want_o) and torch.equal(lse, want_l)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_deterministic_and_batch_independent(layout):
    """The same call gives the same bits; zero queries average the rows."""
    w = make([1, 30, 5], [500, 10, 900], 16, layout, seed=16)
    a, b = run(w), run(w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    w["q"].zero_()
    o, lse = check(w)
    seen = torch.cat([torch.arange(int(w["kv"][i]) - int(w["cu"][i + 1] - w["cu"][i]), int(w["kv"][i])) + 1 for i in range(3)])
    assert torch.allclose(lse.double(), seen.double().log()[:, None].expand(-1, 16), rtol=2e-6, atol=2e-6)


def test_shared_pages():
    """Two requests whose first pages are the same (a shared prefix)."""
    w = make([4, 9], [200, 260], 16, "rope656", seed=17)
    w["table"][1, :3] = w["table"][0, :3]
    check(w)


def test_far_rows_of_a_large_pool():
    """Row offsets beyond 2^31 bytes."""
    rows, layout = (2 ** 32 + 2 ** 28) // 656, "rope656"
    rows -= rows % 64
    w = make([1, 3], [100, 130], 16, layout, seed=18)
    small = w["pool"]
    n = small.shape[0] // 64
    pool = torch.zeros(rows, 656, dtype=torch.uint8, device="cuda")
    far = rows // 64 - n
    pool[far * 64:] = small.cuda()
    o1, l1, _ = run(w)
    w2 = dict(w, pool=pool, table=torch.where(w["table"] >= 0, w["table"] + far, -1).to(torch.int32))
    o2, l2, err = run(w2)
    assert err == 0 and torch.equal(o1, o2) and torch.equal(l1, l2)


def test_other_stream_and_captured_lengths():
    """A captured call follows the lengths, offsets and pages that it finds when it is replayed."""
    w = make([4, 60, 9], [200, 30, 500], 16, "rope656", seed=19)
    want = run(w)
    got = run(w, stream=torch.cuda.Stream())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    T, H = w["q"].shape[:2]
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    o = torch.zeros(T, H, 512, dtype=BF, device="cuda")
    lse = torch.zeros(T, H, device="cuda")
    ws = binding.chunk_workspace_for(T, H, 3, "rope656")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.dsa_chunk_attn(d["q"], d["pool"], "rope656", d["table"], 64, d["cu"], d["kv"], SCALE, o, lse, ws)
    for cu, kv in (([0, 4, 64, 73], [204, 90, 509]), ([0, 70, 71, 73], [100, 55, 300]), ([0, 0, 1, 1], [3, 90, 0])):
        w["cu"], w["kv"] = torch.tensor(cu, dtype=torch.int32), torch.tensor(kv, dtype=torch.int32)
        d["cu"].copy_(w["cu"])
        d["kv"].copy_(w["kv"])
        o.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want = run(w)
        assert torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    a, b = make([1, 30], [5000, 10], 16, "raw512", seed=20), make([40], [900], 16, "scaled528", seed=21)
    wa, wb = run(a), run(b)
    da = {k: v.cuda() for k, v in a.items() if isinstance(v, torch.Tensor)}
    db = {k: v.cuda() for k, v in b.items() if isinstance(v, torch.Tensor)}
    outs = []
    for d in (da, db):
        T, H = d["q"].shape[:2]
        outs.append((torch.zeros(T, H, 512, dtype=BF, device="cuda"), torch.zeros(T, H, device="cuda")))
    ws = [binding.chunk_workspace_for(31, 16, 2, "raw512"), binding.chunk_workspace_for(40, 16, 1, "scaled528")]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (d, lay) in enumerate(((da, "raw512"), (db, "scaled528"))):
            binding.dsa_chunk_attn(d["q"], d["pool"], lay, d["table"], 64, d["cu"], d["kv"], SCALE, *outs[i], ws[i],
                                   stream=s[i])
    torch.cuda.synchronize()
    for (o, l), want in zip(outs, (wa, wb)):
        assert torch.equal(o.cpu(), want[0]) and torch.equal(l.cpu(), want[1])


def test_agrees_with_the_sparse_kernel():
    """A top-k list of every key gives the sparse decode's result."""
    w = make([1] * 4, [127, 255, 383, 511], 16, "rope656", seed=22)
    o, lse, _ = run(w)
    K = 512
    topk = torch.full((4, K), -1, dtype=torch.int32)
    for b in range(4):
        topk[b, :int(w["kv"][b])] = torch.arange(int(w["kv"][b]))
    so, sl = torch.empty(4, 16, 512, dtype=BF, device="cuda"), torch.empty(4, 16, device="cuda")
    binding.dsa_sparse_attn_decode(w["q"].cuda(), w["pool"].cuda(), "rope656", topk.cuda(), SCALE, so, sl,
                                   binding.workspace_for(4, 16, K), page_table=w["table"].cuda(), page_size=64,
                                   token_seq=torch.arange(4, dtype=torch.int32).cuda())
    assert (so.cpu().float() - o.float()).abs().max() < 2.0 ** -6 * o.float().abs().max()
    assert (sl.cpu() - lse).abs().max() < 1e-4


@pytest.mark.parametrize("page", [64, 16])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_wait_that_runs_out_between_units(layout, page):
    """Waits that run out while every SM works through several requests' row groups: nothing is written outside the
    requests' rows and the workspace, a call whose flag is clear is right, and the next call is."""
    r = random.Random(36)
    w = make([r.randint(10, 80) for _ in range(24)], [r.randint(0, 400) for _ in range(24)], 16, layout, page=page,
             seed=36, lead=5, tail=7)
    T, H, _ = w["q"].shape
    n = binding.dsa_chunk_attn_workspace_bytes(T, H, 24, layout)
    room = torch.empty(n + 2 * 65536, dtype=torch.uint8, device="cuda")
    ws, guards = room[65536:65536 + n], (room[:65536], room[65536 + n:])
    want = run(w, ws=ws)
    assert want[2] == 0
    mine = torch.zeros(T, dtype=torch.bool)
    mine[5:T - 7] = True
    for limit in (0, 300, 1000, 3000, 10000, 30000):
        for g in guards:
            g.fill_(0xA5)
        old = binding.dsa_set_wait_limit_ns(limit)
        try:
            o, lse, err = run(w, ws=ws)
        finally:
            binding.dsa_set_wait_limit_ns(old)
        assert err in (0, binding.DSA_DEV_ERR_TIMEOUT) and (limit or err)
        assert (o[~mine] == 7.0).all() and (lse[~mine] == 7.0).all() and all(bool((g == 0xA5).all()) for g in guards)
        if err == 0:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        o, lse, err = run(w, ws=ws)
        assert err == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_call_right_behind_one_that_gave_up():
    """A call that gave up leaves no copy of its own in flight: calls queued directly behind it, which take over its
    shared memory, are right."""
    w = make([30, 1, 50, 9] * 6, [300, 700, 20, 130] * 6, 16, "rope656", seed=37)
    want = run(w)
    T, H, _ = w["q"].shape
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    ws = binding.chunk_workspace_for(T, H, 24, "rope656")
    errs = torch.zeros(12, dtype=torch.int32, device="cuda")
    outs = [(torch.zeros(T, H, 512, dtype=BF, device="cuda"), torch.zeros(T, H, device="cuda")) for _ in range(12)]
    limit = binding.dsa_set_wait_limit_ns(0)
    try:
        for i, (o, lse) in enumerate(outs):
            binding.dsa_set_wait_limit_ns(limit if i % 2 else (0, 500, 2000)[i // 2 % 3])
            binding.dsa_chunk_attn(d["q"], d["pool"], "rope656", d["table"], 64, d["cu"], d["kv"], SCALE, o, lse, ws,
                                   err_flag=errs[i:i + 1])
    finally:
        binding.dsa_set_wait_limit_ns(limit)
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        if i % 2:
            assert int(errs[i]) == 0 and torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_largest_entries_side_by_side(layout):
    """Entries of BF16's largest value next to each other are finite: the row is scored."""
    w = make([3, 1], [200, 300], 8, layout, seed=38)
    w["pool"][:] = w["pool"][:1]                       # equal keys: any finite score gives the same weights
    w["q"][:, ::2] = 0
    big = torch.finfo(BF).max
    for at, h in ((0, 0), (10, 2), (255, 4), (510, 6)):
        w["q"][:, h, at:at + 2] = torch.tensor([big, -big if at == 10 else big], dtype=BF)
    check(w)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_infinite_rope_dims_score_nan(value):
    """A query with an infinite RoPE dim scores NaN also where every product has the same sign (all scores -inf)."""
    w = make([1, 6, 1], [0, 2, 300], 16, "rope656", seed=39)
    w["pool"][:, 528:] = torch.ones(w["pool"].shape[0], 64).to(BF).view(torch.uint8)
    want_o, want_l = check(w)
    hit = [(t, h) for t in (0, 1, 6, 7) for h in (0, 9)]
    for t, h in hit:
        w["q"][t, h, 512 + (5 * t + h) % 64] = value
    o, lse, _ = run(w)
    for t, h in hit:
        assert torch.isnan(o[t, h]).all() and torch.isnan(lse[t, h]), (t, h)
        o[t, h], lse[t, h] = want_o[t, h], want_l[t, h]
    assert torch.equal(o, want_o) and torch.equal(lse, want_l)


def scaled_by(w, layout, e):
    """Queries times 2^-e and rows (scales and RoPE dims) times 2^e: the same scores."""
    w["q"] = (w["q"].double() * 2.0 ** -e).to(BF)
    s = w["pool"][:, 512:528].contiguous().view(torch.float32) * 2.0 ** e
    w["pool"][:, 512:528] = s.view(torch.uint8)
    if layout == "rope656":
        pe = (w["pool"][:, 528:].contiguous().view(BF).double() * 2.0 ** e).to(BF)
        w["pool"][:, 528:] = pe.view(torch.uint8)
    return w


@pytest.mark.parametrize("layout", ["scaled528", "rope656"])
@pytest.mark.parametrize("e", [-40, 40, 60, 80, 95])
def test_small_queries_over_large_rows(layout, e):
    """The queries' power of two reaches every magnitude that finite scores leave room for."""
    check(scaled_by(make([1, 20], [300, 150], 16, layout, seed=40), layout, e))


@pytest.mark.parametrize("big", [20, 60, 100])
def test_large_rope_dims_of_a_query(big):
    """RoPE dims of a query far above its latent dims, over rows whose RoPE dims are as much smaller."""
    w = make([1, 20], [300, 150], 16, "rope656", seed=41)
    w["q"][:, :, 512:] = (w["q"][:, :, 512:].double() * 2.0 ** big).to(BF)
    pe = (w["pool"][:, 528:].contiguous().view(BF).double() * 2.0 ** -big).to(BF)
    w["pool"][:, 528:] = pe.view(torch.uint8)
    check(w)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("scale", [0.0, -0.03, 1.0])
def test_other_score_scales(layout, scale, monkeypatch):
    """No scale, a negative one, one that peaks the softmax."""
    monkeypatch.setitem(globals(), "SCALE", scale)
    check(make([1, 20], [700, 150], 16, layout, seed=42))


@pytest.mark.parametrize("layout", ["scaled528", "rope656"])
def test_negative_scales(layout):
    w = make([1, 20], [700, 150], 16, layout, seed=43)
    s = w["pool"][:, 512:528].contiguous().view(torch.float32)
    s[::3] *= -1
    s[:, 2] *= -1
    w["pool"][:, 512:528] = s.view(torch.uint8)
    check(w)
