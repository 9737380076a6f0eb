"""Dense attention over 4-bit rows: against the formula in 64 bits, and bit for bit against the same rows held in 8 bits."""
import math
import random

import pytest
import torch

import dense_ref as ref
import fp4_ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
LAYOUTS = ["fp4_288", "fp4_416"]
WIDE = {"fp4_288": "scaled528", "fp4_416": "rope656"}
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
    q = (torch.randn(T, H, ref.KEY_DIMS[WIDE[layout]], generator=g) * qamp).to(BF)
    return dict(q=q, pool=fp4_ref.make_pool(n_pages * page, layout, g, amp), layout=layout, table=table, page=page,
                cu=torch.tensor(cu, dtype=torch.int32), kv=torch.tensor(kv, dtype=torch.int32), causal=True)


def run(w, pool, layout, stream=None):
    T, H, _ = w["q"].shape
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor) and k != "pool"}
    pool = pool.cuda()
    o = torch.full((T, H, 512), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = binding.chunk_workspace_for(T, H, w["table"].shape[0], layout)
    ws.fill_(0xFF)                                        # what it held before has no effect
    torch.cuda.synchronize()
    binding.dsa_chunk_attn(d["q"], pool, layout, d["table"], w["page"], d["cu"], d["kv"], SCALE, o, lse, ws,
                           causal=w["causal"], err_flag=err, stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), int(err.item())


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == BF else torch.int32), b.view(torch.int16 if b.dtype == BF else torch.int32))


def check(w, err_want=0, exact=True):
    o, lse, err = run(w, w["pool"], w["layout"])
    wide = fp4_ref.expand(w["pool"].numpy())
    o8, lse8, err8 = run(w, wide, WIDE[w["layout"]])
    assert err == err8 == err_want
    assert same(o, o8) and same(lse, lse8)
    if not exact:
        return
    ro, rl, otol, ltol, rerr = ref.chunk_attn(w["q"], wide, WIDE[w["layout"]], w["table"], w["page"], w["cu"], w["kv"],
                                              SCALE, w["causal"])
    assert rerr == err_want
    out = torch.isnan(rl)                                  # rows of no request
    assert (o[out] == 7.0).all() and (lse[out] == 7.0).all()
    o, lse, ro, rl, otol, ltol = (x[~out] for x in (o, lse, ro, rl, otol, ltol))
    none = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), none) and (o[none] == 0).all()
    d = (o.double() - ro).abs() - otol
    assert torch.isfinite(o).all() and (d <= 0).all(), f"O off by {d.max():.3e} beyond the bound"
    d = ((lse.double() - rl).abs() - ltol)[~none]
    assert d.numel() == 0 or (d <= 0).all(), f"LSE off by {d.max():.3e} beyond the bound"


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H", [1, 16, 32, 128])
def test_single_tokens(layout, H):
    check(make([1] * 9, [0, 1, 63, 126, 127, 128, 129, 255, 700], H, layout, seed=H))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256, 1000])
def test_page_sizes(layout, page):
    check(make([1, 5, 40], [300, 77, 130], 8, layout, page=page, seed=page))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("new,ctx", [([2], [0]), ([130], [0]), ([7, 1, 33, 0, 64], [0, 500, 10, 20, 129]), ([200], [301])])
@pytest.mark.parametrize("H", [3, 16])
def test_chunks(layout, new, ctx, H):
    check(make(new, ctx, H, layout, seed=sum(new) + H, lead=2, tail=3))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_long_context_and_many_units(layout):
    """One request over every SM; ranges that begin and end inside requests."""
    check(make([1], [40000], 16, layout, seed=3))
    check(make([3, 1], [20011, 9], 128, layout, seed=4), exact=False)
    r = random.Random(5)
    check(make([r.randint(1, 90) for _ in range(24)], [r.randint(0, 400) for _ in range(24)], 16, layout, seed=5), exact=False)
    check(make([1] * 200, [r.randint(1, 3000) for _ in range(200)], 16, layout, seed=6, page=16), exact=False)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_chunks_over_expanded_rows(layout):
    """Calls of 8192 query rows and 1024 a request, whose rows are expanded once: ragged requests, one without new tokens
    and one without rows, pages of 16 to 256, not causal; what does not fit (smaller pages, bad pages and lengths, too
    many rows) takes the general form, with the same results."""
    new, ctx = [70, 0, 130, 64, 200, 120], [500, 9, 0, 129, 1000, 3]
    for page in (16, 48, 256, 3):
        check(make(new, ctx, 16, layout, page=page, seed=page, lead=2, tail=3), exact=page == 48)
    w = make([600], [1], 16, layout, seed=41)
    w["causal"] = False
    check(w)
    w = make([520, 8], [40, 3], 16, layout, seed=42)
    w["kv"][1] = 0                                         # tokens that see no key
    check(w, exact=False)
    w = make([600, 30], [40, 300], 16, layout, page=16, seed=43)
    w["table"][1, 5], w["table"][0, 7] = -3, 1 << 22
    check(w, err_want=binding.DSA_DEV_ERR_PAGE_RANGE, exact=False)
    w = make([300, 300], [40, 300], 16, layout, page=16, seed=44)
    w["kv"][1] = 10 ** 6
    o, lse, err = run(w, w["pool"], layout)
    assert err & binding.DSA_DEV_ERR_LENGTH
    o8, lse8, err8 = run(w, fp4_ref.expand(w["pool"].numpy()), WIDE[layout])
    assert err == err8 and same(o, o8) and same(lse, lse8)
    w = make([70, 70, 70], [100, 70, 90], 48, layout, page=64, seed=45)       # three pages each
    w["table"] = w["table"][:, :3].repeat(1, 500)[:, :1100]      # 70000 keys a request, over the same pages again and again
    w["kv"][:] = 70000
    check(w, exact=False)


def test_captured_chunk_over_expanded_rows():
    """A captured chunk serves shorter ones, and lengths that do not fit."""
    w = make([600], [700], 16, "fp4_416", seed=46)
    d = {k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)}
    o, lse = torch.zeros(600, 16, 512, dtype=BF, device="cuda"), torch.zeros(600, 16, device="cuda")
    ws = binding.chunk_workspace_for(600, 16, 1, "fp4_416")
    step = (lambda: binding.dsa_chunk_attn(d["q"], d["pool"], "fp4_416", d["table"], 64, d["cu"], d["kv"], SCALE, o, lse, ws))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for kv in (1300, 5, 640, 0, 1300):
        d["kv"].fill_(kv)
        w["kv"][:] = kv
        o.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        o8, lse8, _ = run(w, fp4_ref.expand(w["pool"].numpy()), "rope656")
        assert same(o.cpu(), o8) and same(lse.cpu(), lse8)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_not_causal_and_amplitudes(layout):
    w = make([5, 130, 1], [60, 3, 300], 8, layout, seed=6)
    w["causal"] = False
    check(w)
    check(make([1, 20], [900, 150], 16, layout, seed=7, qamp=40.0))
    check(make([1, 20], [900, 150], 16, layout, seed=8, amp=100.0, qamp=0.05))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_bad_pages(layout):
    """Negative entries and pages behind the pool mask their keys and are flagged."""
    w = make([2, 3], [300, 200], 8, layout, page=16, seed=9)
    w["table"][0, 3], w["table"][1, 7] = -5, 1 << 24
    check(w, err_want=binding.DSA_DEV_ERR_PAGE_RANGE)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_nan_scales(layout):
    """A row with a NaN scale makes the results that see it NaN, and no others; what no query sees has no effect."""
    w = make([4, 1], [100, 200], 8, layout, page=16, seed=10)
    row = lambda b, j: int(w["table"][b, j // 16]) * 16 + j % 16
    nan = torch.full((1,), math.nan).view(torch.uint8)
    w["pool"][row(0, 102), 256:260] = nan
    held = set(w["table"].flatten().tolist())
    for p in range(w["pool"].shape[0] // 16):              # pages of no request, and the rest of the last ones
        if p not in held:
            w["pool"][16 * p:16 * p + 16, 256:272] = nan.repeat(4)
    for b, k in ((0, 104), (1, 201)):
        for j in range(k, ref.pages_of(k, 16) * 16):
            w["pool"][row(b, j), 256:272] = nan.repeat(4)
    o, lse, err = run(w, w["pool"], layout)
    assert err == 0
    assert torch.isfinite(o[[0, 1, 4]].float()).all() and torch.isfinite(lse[[0, 1, 4]]).all()
    assert o[[2, 3]].isnan().all() and lse[[2, 3]].isnan().all()
    check(w, exact=False)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_wait_that_runs_out(layout):
    """A limit of zero: the call returns, reports the timeout, leaves rows of no request alone, and the next is right."""
    w = make([40, 3, 1], [700, 2000, 90], 16, layout, seed=12, lead=1, tail=2)
    old = binding.dsa_set_wait_limit_ns(0)
    try:
        o, lse, err = run(w, w["pool"], layout)
    finally:
        binding.dsa_set_wait_limit_ns(old)
    assert err == binding.DSA_DEV_ERR_TIMEOUT
    out = [0, o.shape[0] - 2, o.shape[0] - 1]
    assert (o[out] == 7.0).all() and (lse[out] == 7.0).all()
    check(w)


def test_captured_over_rows_as_they_are_written():
    """Writer and attention in one graph, replayed with new rows: the bits of the eager calls."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, H, page = 6, 16, 16
    table = torch.arange(6 * 20, dtype=torch.int32, device="cuda").view(6, 20)
    cu, kv = torch.arange(7, dtype=torch.int32, device="cuda"), torch.tensor([300, 1, 17, 128, 129, 256], dtype=torch.int32, device="cuda")
    pool = torch.zeros(6 * 20 * page, 416, dtype=torch.uint8, device="cuda")
    n = pool.shape[0]
    x, pe = torch.zeros(n, 512, dtype=BF, device="cuda"), torch.zeros(n, 64, dtype=BF, device="cuda")
    q = torch.randn(T, H, 576, generator=g, device="cuda").to(BF)
    slots = torch.arange(n, device="cuda")
    ws = binding.chunk_workspace_for(T, H, 6, "fp4_416")
    o, lse = torch.zeros(T, H, 512, dtype=BF, device="cuda"), torch.zeros(T, H, device="cuda")

    def step():
        binding.dsa_kv_write_fp4(x, slots, pool, k_pe=pe)
        binding.dsa_chunk_attn(q, pool, "fp4_416", table, page, cu, kv, SCALE, o, lse, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.copy_(torch.randn(n, 512, generator=g, device="cuda"))
        pe.copy_(torch.randn(n, 64, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        o.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert (o.abs().amax((1, 2)) > 0).all()
