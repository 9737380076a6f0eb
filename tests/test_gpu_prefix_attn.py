"""Attention of requests that begin with common rows, against the formula in 64 bits.

Where the rows of a group are meant to be shared, the entries of the shared tiles' pages are taken out of every page-table
row but the first's, so that a right result without an error flag shows that they were read once, through that one."""
import math
import random

import pytest
import torch

import dense_ref as ref
import fp4_ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
LAYOUTS = ["raw512", "scaled528", "rope656", "fp4_288", "fp4_416"]
WIDE = {"fp4_288": "scaled528", "fp4_416": "rope656"}
SCALE = 1 / math.sqrt(576.0)
BF = torch.bfloat16


def make(groups, H, layout, page=64, seed=0, alone=((), ()), lead=0, tail=0, qamp=1.0, causal=True, copies=False):
    """groups: (prefix, [(new, own context), ...]) each; alone: requests (new, context) in front of and behind the groups.
    A prefix may end inside a page: each request then holds its own copy of that page's rows (copies: of every row)."""
    g = torch.Generator().manual_seed(seed)
    reqs = [(n, c, 0, None) for n, c in alone[0]]
    gcu, plens = [len(reqs)], []
    for gi, (p, members) in enumerate(groups):
        reqs += [(n, c, p, gi) for n, c in members]
        gcu.append(len(reqs))
        plens.append(p)
    reqs += [(n, c, 0, None) for n, c in alone[1]]
    kv = [p + c + n for n, c, p, _ in reqs]
    need = [ref.pages_of(k, page) for k in kv]
    n_pages = sum(need) + 3
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    pool = (fp4_ref.make_pool if layout in WIDE else ref.make_pool)(n_pages * page, layout, g)
    table = torch.full((len(reqs), max(need + [1]) + 1), -1, dtype=torch.int32)
    at, first = 0, {}
    for b, (n, c, p, gi) in enumerate(reqs):
        whole = 0
        if gi in first and not copies:
            whole = p // page
            table[b, :whole] = table[first[gi], :whole]
        table[b, whole:need[b]] = ids[at:at + need[b] - whole]
        at += need[b] - whole
        if gi is not None and gi not in first:
            first[gi] = b
        elif gi is not None:
            j = torch.arange(whole * page, p)
            src, dst = (table[x].long()[j // page] * page + j % page for x in (first[gi], b))
            pool[dst] = pool[src]
    T = lead + sum(r[0] for r in reqs) + tail
    cu = [lead]
    for r in reqs:
        cu.append(cu[-1] + r[0])
    q = (torch.randn(T, H, ref.KEY_DIMS[WIDE.get(layout, layout)], generator=g) * qamp).to(BF)
    i32 = (lambda x: torch.tensor(x, dtype=torch.int32))
    return dict(q=q, pool=pool, layout=layout, table=table, page=page, cu=i32(cu), kv=i32(kv), gcu=i32(gcu), plens=i32(plens),
                causal=causal)


def enough(H, news, sms=152):
    """Keys of a prefix that pays for news[b] new tokens of the group's requests: packing their rows saves a unit's tiles
    as often as units get fewer, and is more than enough at four tiles a CTA, beside what a packed unit costs (below three tiles)."""
    units, packed = sum(-(-n * H // 32) for n in news), -(-sum(news) * H // 32)
    return 128 * -(-(4 * sms + 3 * packed) // (units - packed))


def hide_shared(w, keys):
    """Takes the first keys[g] keys' whole pages out of the rows of every request of group g but the first."""
    t = w["table"].clone()
    for g, k in enumerate(keys):
        t[int(w["gcu"][g]) + 1:int(w["gcu"][g + 1]), :k // w["page"]] = -1
    return t


def run(w, stream=None, ws=None, table=None, fn="prefix"):
    T, H, _ = w["q"].shape
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    if table is not None:
        d["table"] = table.cuda()
    o = torch.full((T, H, 512), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = binding.prefix_workspace_for(T, H, d["table"].shape[0], w["layout"])
    ws.fill_(0xFF)                                        # what it held before has no effect
    torch.cuda.synchronize()
    common = (d["q"], d["pool"], w["layout"], d["table"], w["page"], d["cu"], d["kv"])
    if fn == "chunk":
        binding.dsa_chunk_attn(*common, SCALE, o, lse, ws, causal=w["causal"], err_flag=err, stream=stream)
    else:
        binding.dsa_prefix_attn(*common, d["gcu"], d["plens"], SCALE, o, lse, ws, causal=w["causal"], err_flag=err, stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), int(err.item())


def check(w, err_want=0, hidden=None, only=None, **kw):
    """hidden: shared keys of each group, or None; only: requests that are compared (None: all)."""
    whole_o, whole_lse, err = run(w, table=None if hidden is None else hide_shared(w, hidden), **kw)
    o, lse = whole_o, whole_lse
    cu = w["cu"]
    wide = fp4_ref.expand(w["pool"].numpy()) if w["layout"] in WIDE else w["pool"]
    table, kv, q = w["table"], w["kv"], w["q"]
    if only is not None:
        rows = torch.cat([torch.arange(int(cu[b]), int(cu[b + 1])) for b in only])
        n = [int(cu[b + 1] - cu[b]) for b in only]
        cu = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32)
        table, kv, q, o, lse = table[list(only)], kv[list(only)], q[rows], o[rows], lse[rows]
    ro, rl, otol, ltol, _ = ref.chunk_attn(q, wide, WIDE.get(w["layout"], w["layout"]), table, w["page"], cu, kv, SCALE, w["causal"])
    assert err == err_want
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


ONE = [(1, c) for c in (0, 1, 60, 127, 128, 129, 300, 5, 9, 200, 31, 2, 70, 400, 33, 8)]
MIXED = [(1, 3), (2, 200), (1, 0), (3, 50), (1, 129), (1, 9), (2, 0), (1, 64), (1, 300), (2, 5), (1, 1), (1, 90)]


def common(H, members=ONE):
    return enough(H, [m[0] for m in members])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H", [1, 4, 8, 16, 20])
def test_single_tokens(layout, H):
    """Requests of one token: their rows are packed."""
    w = make([(common(H), ONE)], H, layout, seed=H)
    check(w, hidden=[common(H)])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H", [32, 64, 128])
def test_heads_that_fill_the_tiles(layout, H):
    """Nothing to save: the same work as without groups, the same bits."""
    w = make([(640, ONE[:4])], H, layout, seed=H)
    o, lse = check(w)
    o2, lse2, err = run(w, fn="chunk")
    assert err == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("more", [-1, 0, 1, 63, 127])
def test_prefix_lengths(layout, more):
    """Prefixes that end inside a tile, and inside a page; one that is a key too short to pay; hardly any."""
    p = common(8, MIXED) + more
    check(make([(p, MIXED)], 8, layout, seed=p), hidden=[p // 128 * 128] if more >= 0 else None)
    check(make([(1 + more // 2, MIXED[:5])], 8, layout, seed=p) if more > 0 else make([(500, MIXED[:5])], 8, layout, seed=p))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("p", [100, 130, 256, 400, 1000])
def test_short_prefixes_in_a_wide_table(layout, p):
    """The page table has room for a prefix that pays: a short one is shared too, from two tiles on (16 units' tiles against
    four packed units' and their cost, below three tiles each)."""
    w = make([(p, ONE)], 8, layout, seed=p)
    w["table"] = torch.cat([w["table"], torch.full((len(ONE), common(8) // w["page"]), -1, dtype=torch.int32)], 1)
    check(w, hidden=[p // 128 * 128] if p >= 256 else None)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 3, 16, 48, 256, 1000])
def test_page_sizes(layout, page):
    p = common(8, MIXED)
    w = make([(p + 60, MIXED)], 8, layout, page=page, seed=page)
    check(w, hidden=[p])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_groups_and_requests_alone(layout):
    """Groups of several sizes, one of a single request, an empty one; requests of none in front and behind; rows of no
    request; requests without new tokens, a group that begins with one."""
    groups = [(8000, MIXED), (300, [(2, 10)]), (200, []), (6000, [(0, 5), (1, 70), (1, 3), (0, 0), (3, 200)] + ONE)]
    w = make(groups, 8, layout, page=16, seed=3, alone=([(1, 50), (40, 0)], [(0, 7), (2, 400), (1, 0)]), lead=3, tail=5)
    w["table"][int(w["gcu"][3])] = -1                      # of the request without new tokens: nothing is read through it
    check(w)


@pytest.mark.parametrize("layout", ["raw512", "fp4_416"])
def test_chunks_behind_a_prefix(layout):
    """Drafted tokens and chunks: rows of a request over several tiles, and over two tiles of the packed rows."""
    m = [(n, c) for n, c in zip((5, 3, 7, 1, 6, 2, 5, 3, 9, 1, 8, 4), (0, 90, 4, 300, 128, 1, 2, 60, 11, 0, 31, 200))]
    check(make([(common(5, m), m)], 5, layout, seed=4), hidden=[common(5, m)])
    m = [(12, 10), (23, 0), (21, 77), (13, 5), (2, 0), (34, 1), (1, 0), (12, 3)]
    check(make([(common(3, m), m)], 3, layout, seed=5), hidden=[common(3, m)])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_not_causal_and_large_queries(layout):
    p = common(8)
    check(make([(p, ONE)], 8, layout, seed=6, causal=False), hidden=[p])
    check(make([(640, [(3, 0), (2, 40), (4, 300)])], 4, layout, seed=7, causal=False))
    check(make([(p, ONE)], 8, layout, seed=8, qamp=40.0), hidden=[p])


@pytest.mark.parametrize("layout", ["raw512", "rope656"])
def test_copies_of_the_prefix(layout):
    """Each request holds the rows in pages of its own."""
    check(make([(common(8), ONE)], 8, layout, seed=9, copies=True))


@pytest.mark.parametrize("layout", ["raw512", "scaled528", "fp4_416"])
def test_requests_shorter_than_the_prefix(layout):
    """What is shared ends with what every first token sees."""
    p = common(8)
    w = make([(p + 900, ONE)], 8, layout, seed=10)
    w["kv"][2] = p + 44
    check(w, hidden=[p])
    w["kv"][2] = 100                                       # below a tile: nobody shares
    check(w)
    w["kv"][3] = 1
    check(w)
    w = make([(p, [(5, 0)] + ONE)], 8, layout, seed=11)
    w["kv"][0] = 3                                         # more new tokens than keys: the first see none
    check(w)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H", [4, 16])
def test_few_requests_behind_a_long_prefix(layout, H):
    """Units over the prefix are spread over most SMs: a row joins dozens of parts."""
    w = make([(40064, [(1, 9), (1, 700), (2, 300)])], H, layout, seed=12)
    check(w, hidden=[39936] if H == 4 else None)


@pytest.mark.parametrize("layout", ["raw512", "rope656", "fp4_288"])
def test_many_requests(layout):
    """More units than every block of the join looks at; a few requests of each group are compared."""
    r = random.Random(13)
    groups = [(512, [(1, r.randint(0, 200)) for _ in range(700)]), (1024, [(1, r.randint(0, 60)) for _ in range(900)])]
    w = make(groups, 8, layout, seed=13)
    check(w, hidden=[512, 1024], only=[0, 1, 350, 698, 699, 700, 701, 1200, 1599])


def test_most_requests():
    r = random.Random(14)
    w = make([(256, [(1, r.randint(0, 9)) for _ in range(4096)])], 4, "raw512", page=16, seed=14)
    check(w, hidden=[256], only=[0, 1, 2000, 4095])
    w = make([(640, [(1, 3), (1, 5)]) for _ in range(300)], 4, "raw512", page=16, seed=15)
    check(w, hidden=[640] * 300, only=[0, 1, 301, 598, 599])
    w = make([], 4, "raw512", page=16, seed=15, alone=([(1, 5)] * 4096, []))           # as many groups as requests
    w["gcu"], w["plens"] = torch.arange(4097, dtype=torch.int32), torch.full((4096,), 128, dtype=torch.int32)
    check(w, only=[0, 1, 4095])


@pytest.mark.parametrize("gcu,plens", [([0, 3, 2, 5], [640, 640, 640]), ([-1, 2, 3, 5], [640] * 3), ([0, 2, 3, 6], [640] * 3),
                                       ([0, 2, 4, 5], [640, -1, 640]), ([5, 3, 1, 0], [640] * 3)])
def test_bad_groups(gcu, plens):
    """Flagged; every request attends alone, so the results are right."""
    w = make([(common(8), ONE[:5])], 8, "raw512", seed=16)
    w["gcu"], w["plens"] = torch.tensor(gcu, dtype=torch.int32), torch.tensor(plens, dtype=torch.int32)
    check(w)                                               # (too small a call to share: the groups are not looked at)
    w["table"] = torch.cat([w["table"], torch.full((5, 200), -1, dtype=torch.int32)], 1)
    check(w, err_want=binding.DSA_DEV_ERR_LENGTH)


def test_prefix_longer_than_anything():
    p = common(8)
    w = make([(p, ONE)], 8, "raw512", seed=17)
    w["plens"][0] = 2 ** 31 - 1
    # every request's keys but its last one are taken for common rows: only those of the first are read
    w["kv"][:] = p + 1
    check(w, hidden=[p])


def test_no_groups():
    w = make([], 8, "rope656", seed=18, alone=([(1, 30), (4, 200)], [(1, 0)]))
    o, lse = check(w)
    o2, lse2, _ = run(w, fn="chunk")
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * o2.float().abs().max()


@pytest.mark.parametrize("layout", ["raw512", "scaled528", "fp4_416"])
def test_bad_lengths_and_pages(layout):
    """A request with offsets out of order or a length beyond the table ends its group's sharing and is flagged, a bad page
    in the first request's row masks its keys for the group."""
    p, n = common(8), len(ONE)
    w = make([(p, ONE)], 8, layout, seed=19, tail=3)
    wide, name = (fp4_ref.expand(w["pool"].numpy()), WIDE[layout]) if layout in WIDE else (w["pool"], layout)
    bound = (lambda table: ref.chunk_attn(w["q"], wide, name, table, 64, w["cu"], w["kv"], SCALE))
    kv1 = int(w["kv"][1])
    w["kv"][1] = 10 ** 6
    o, lse, err = run(w)
    assert err & binding.DSA_DEV_ERR_LENGTH
    ro, rl, otol, ltol, _ = bound(w["table"])
    for t in (0, 2, 3, n - 1):
        assert ((o[t].double() - ro[t]).abs() <= otol[t]).all() and ((lse[t].double() - rl[t]).abs() <= ltol[t]).all()
    w["kv"][1] = kv1
    shown = w["table"].clone()
    w["table"][0, 3] = -7
    o, lse, err = run(w)
    assert err == binding.DSA_DEV_ERR_PAGE_RANGE
    shown[:, 3] = -7
    ro, rl, otol, ltol, _ = bound(shown)
    assert ((o[:n].double() - ro[:n]).abs() <= otol[:n]).all() and ((lse[:n].double() - rl[:n]).abs() <= ltol[:n]).all()
    assert (o[n:] == 7.0).all()


@pytest.mark.parametrize("layout", ["raw512", "scaled528", "fp4_288"])
def test_nan_rows(layout):
    """In the prefix: every result is NaN; behind one request's own rows: its results alone."""
    p = common(8)
    w = make([(p, ONE)], 8, layout, seed=20)
    row = (lambda b, j: int(w["table"][b, j // 64]) * 64 + j % 64)
    clean = w["pool"].clone()
    at = slice(0, 1) if layout == "raw512" else slice(512, 516) if layout == "scaled528" else slice(256, 260)
    nan = torch.tensor([0x7F], dtype=torch.uint8) if layout == "raw512" else torch.full((1,), math.nan).view(torch.uint8)
    w["pool"][row(0, 200), at] = nan
    o, lse, err = run(w)
    assert err == 0 and o.isnan().any(-1).all() and lse.isnan().all()
    w["pool"] = clean.clone()
    w["pool"][row(2, p + 20), at] = nan
    o, lse, err = run(w)
    rest = [t for t in range(len(ONE)) if t != 2]
    assert err == 0 and lse[2].isnan().all() and torch.isfinite(lse[rest]).all() and torch.isfinite(o[rest].float()).all()


@pytest.mark.parametrize("layout", ["raw512", "rope656"])
def test_nan_and_zero_queries(layout):
    """A query row with a NaN or an infinity scores NaN and leaves the rows that it is packed with alone; zero rows average."""
    p = common(8)
    w = make([(p, ONE)], 8, layout, seed=28)
    w["q"][3, 2, 17], w["q"][5, 0, 300], w["q"][6] = math.nan, -math.inf, 0.0
    o, lse, err = run(w, table=hide_shared(w, [p]))
    assert err == 0
    bad = torch.zeros(len(ONE), 8, dtype=torch.bool)
    bad[3, 2] = bad[5, 0] = True
    assert lse[bad].isnan().all() and o[bad].isnan().all()
    w["q"][3, 2, 17] = w["q"][5, 0, 300] = 0.0
    ro, rl, otol, ltol, _ = ref.chunk_attn(w["q"], w["pool"], layout, w["table"], 64, w["cu"], w["kv"], SCALE)
    assert ((o.double() - ro).abs() <= otol)[~bad].all() and ((lse.double() - rl).abs() <= ltol)[~bad].all()


def test_captured_steps():
    """A captured call serves other lengths, groups and prefixes, with a workspace that eager calls use as well."""
    p, B = common(8), len(ONE)
    w = make([(p, ONE)], 8, "rope656", seed=21)
    most = w["kv"].clone()
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    T, H = B, 8
    o, lse = torch.zeros(T, H, 512, dtype=BF, device="cuda"), torch.zeros(T, H, device="cuda")
    ws = binding.prefix_workspace_for(T, H, B, "rope656")

    def step():
        binding.dsa_prefix_attn(d["q"], d["pool"], "rope656", d["table"], 64, d["cu"], d["kv"], d["gcu"], d["plens"], SCALE, o, lse, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for kv0, gcu, plen in ((p, [0, B], p), (300, [0, 5], 200), (p + 1, [2, 3], 640), (130, [0, 0], 0), (p + 9, [1, B], p)):
        w["kv"] = torch.minimum(torch.tensor([kv0 + 1 + 7 * i for i in range(B)], dtype=torch.int32), most)
        w["gcu"], w["plens"] = torch.tensor(gcu, dtype=torch.int32), torch.tensor([plen], dtype=torch.int32)
        for k in ("kv", "gcu", "plens"):
            d[k].copy_(w[k])
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = o.cpu(), lse.cpu()
        want_o, want_lse = check(w, ws=ws)
        assert torch.equal(got[0], want_o) and torch.equal(got[1], want_lse)


def test_streams_and_repeats():
    """Calls on two streams with a workspace each, over and over: the same bits."""
    ws = [make([(5504, [(1, 9 * i) for i in range(20)])], 8, lay, seed=22) for lay in ("raw512", "fp4_416")]
    want = [check(w, only=[0, 7, 19]) for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    dev, outs = [], []
    for w in ws:
        d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
        d["ws"] = binding.prefix_workspace_for(20, 8, 20, w["layout"])
        dev.append(d)
        outs.append([(torch.zeros(20, 8, 512, dtype=BF, device="cuda"), torch.zeros(20, 8, device="cuda")) for _ in range(6)])
    torch.cuda.synchronize()
    for k in range(6):
        for w, d, s, out in zip(ws, dev, streams, outs):
            binding.dsa_prefix_attn(d["q"], d["pool"], w["layout"], d["table"], 64, d["cu"], d["kv"], d["gcu"], d["plens"], SCALE,
                                    *out[k], d["ws"], stream=s)
    torch.cuda.synchronize()
    for (wo, wl), out in zip(want, outs):
        for o, lse in out:
            assert torch.equal(o.cpu(), wo) and torch.equal(lse.cpu(), wl)


@pytest.mark.parametrize("layout", ["raw512", "rope656", "fp4_416"])
def test_wait_that_runs_out(layout):
    """A limit of zero: the call returns, reports the timeout, leaves rows of no request alone, and the next is right."""
    w = make([(5504, [(1, 9 * i) for i in range(20)])], 8, layout, seed=23, lead=2, tail=3)
    old = binding.dsa_set_wait_limit_ns(0)
    try:
        o, lse, err = run(w)
    finally:
        binding.dsa_set_wait_limit_ns(old)
    assert err == binding.DSA_DEV_ERR_TIMEOUT
    out = [0, 1, 22, 23, 24]
    assert (o[out] == 7.0).all() and (lse[out] == 7.0).all()
    check(w)


def test_workspace_of_larger_calls():
    """One workspace for every smaller call."""
    ws = binding.prefix_workspace_for(64, 16, 32, "rope656")
    check(make([(common(8), ONE)], 8, "rope656", seed=24), ws=ws)
    check(make([(640, ONE[:3])], 16, "rope656", seed=25), ws=ws)
    check(make([(640, [(9, 0), (20, 5)])], 16, "rope656", seed=26), ws=ws)


def test_binding_refusals():
    w = make([(200, ONE[:3])], 4, "raw512", seed=27)
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    o, lse = torch.zeros(3, 4, 512, dtype=BF, device="cuda"), torch.zeros(3, 4, device="cuda")
    base = dict(q_bf16=d["q"], pool=d["pool"], layout="raw512", page_table=d["table"], page_size=64, cu_q=d["cu"], kv_lens=d["kv"],
                group_cu=d["gcu"], prefix_lens=d["plens"], sm_scale=SCALE, o=o, lse=lse,
                workspace=binding.prefix_workspace_for(3, 4, 3, "raw512"))
    for kw in (dict(group_cu=d["gcu"][:1]), dict(group_cu=d["gcu"].long()), dict(prefix_lens=d["plens"].cpu()), dict(group_cu=None),
               dict(prefix_lens=d["plens"].float()), dict(workspace=base["workspace"][:-1]), dict(layout="fp4_288"), dict(page_size=0),
               dict(prefix_lens=torch.zeros(4, dtype=torch.int32, device="cuda"), group_cu=torch.zeros(5, dtype=torch.int32, device="cuda")),
               dict(workspace=binding.chunk_workspace_for(3, 4, 3, "raw512")), dict(o=o.float()), dict(lse=lse[:2])):
        with pytest.raises((TypeError, ValueError, binding.DsaError)):
            binding.dsa_prefix_attn(**dict(base, **kw))
    binding.dsa_prefix_attn(**base)
