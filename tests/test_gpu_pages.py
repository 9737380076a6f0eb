"""Page tables, slot maps and the return of pages against plain lists."""
import random

import pytest
import torch

import dense_ref as ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def make(B, page, new_hi, ctx_hi, seed, spare=3, pad=5):
    r = random.Random(seed)
    new = [r.randint(0, new_hi) for _ in range(B)]
    seq = [r.choice([0, r.randint(0, ctx_hi), page * r.randint(0, max(0, ctx_hi // page))]) for _ in range(B)]
    width = max(ref.pages_of(s + n, page) for s, n in zip(seq, new)) + 1
    ids = list(range(sum(ref.pages_of(s + n, page) for s, n in zip(seq, new)) + spare))
    r.shuffle(ids)
    table = []
    for s in seq:
        held = ref.pages_of(s, page)
        table.append([ids.pop() for _ in range(held)] + [-1] * (width - held))
    return dict(seq=seq, new=new, table=table, page=page, free=ids + [-7] * 4, count=len(ids), T=sum(new) + pad)


def run_extend(w, in_place=False, stream=None):
    seq, new = torch.tensor(w["seq"], **I32), torch.tensor(w["new"], **I32)
    table, free = torch.tensor(w["table"], **I32), torch.tensor(w["free"], **I32)
    count = torch.tensor([w["count"]], **I32)
    T, B = w["T"], len(w["seq"])
    out = dict(slots=torch.full((T,), 77, dtype=torch.int64, device="cuda"), positions=torch.full((T,), 77, **I32),
               token_seq=torch.full((T,), 77, **I32), cu_q=torch.full((B + 1,), 77, **I32),
               kv_lens=seq if in_place else torch.full((B,), 77, **I32))
    count_out = count if in_place else torch.full((1,), 77, **I32)
    err = torch.zeros(1, **I32)
    torch.cuda.synchronize()
    binding.dsa_pages_extend(seq, new, table, w["page"], free, count, count_out, err_flag=err, stream=stream, **out)
    torch.cuda.synchronize()
    assert free.tolist() == w["free"]
    return {**{k: v.tolist() for k, v in out.items()}, "page_table": table.tolist(),
            "free_count": int(count_out.item()), "err": int(err.item())}


def check_extend(w, **kw):
    want = ref.extend(w["seq"], w["new"], w["table"], w["page"], w["free"], w["count"], w["T"])
    got = run_extend(w, **kw)
    for k in want:
        assert got[k] == want[k], k
    return got


@pytest.mark.parametrize("page", [1, 7, 16, 64, 256])
@pytest.mark.parametrize("B,new_hi,ctx_hi", [(1, 1, 0), (1, 300, 5), (3, 0, 100), (64, 1, 900), (33, 200, 70), (1025, 9, 40)])
def test_extend(B, new_hi, ctx_hi, page):
    check_extend(make(B, page, new_hi, ctx_hi, seed=B * 1000 + page))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T", [16384, 16385, 300000])
def test_extend_many_tokens(T, in_place):
    """The largest call of one CTA, the smallest grid, and more than one pass of a full grid's threads; the padding
    rows count as work."""
    w = make(40, 16, 300, 100, seed=3)
    w["T"] = T
    check_extend(w, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_extend_a_full_grid_of_tokens(in_place):
    check_extend(make(90, 16, 4000, 100, seed=12), in_place=in_place)


def test_extend_most_requests():
    check_extend(make(16384, 64, 2, 3, seed=4))


@pytest.mark.parametrize("B", [5, 300])
def test_extend_in_place(B):
    check_extend(make(B, 16, 40, 100, seed=5), in_place=True)


def test_extend_other_stream():
    s = torch.cuda.Stream()
    check_extend(make(20, 16, 40, 100, seed=6), stream=s)


def test_extend_exact_fit():
    """No spare page, no padding row."""
    w = make(17, 16, 40, 100, seed=7, spare=0, pad=0)
    assert check_extend(w)["free_count"] == 0


@pytest.mark.parametrize("what,bit", [("pages", 32), ("negative_seq", 16), ("negative_new", 16), ("outgrown", 16),
                                      ("tokens", 16), ("count_negative", 16), ("count_high", 16), ("huge", 16)])
def test_extend_refused_changes_nothing(what, bit):
    w = make(9, 16, 40, 100, seed=8)
    w["new"][2] = 33                                       # pages are needed, and the rows have room for them
    w["T"] = sum(w["new"]) + 5
    w["table"] = [row + [-1] * 3 for row in w["table"]]
    if what == "pages":
        w["count"] = 1
    elif what == "negative_seq":
        w["seq"][4] = -1
    elif what == "negative_new":
        w["new"][8] = -3
    elif what == "outgrown":
        w["seq"][1] = len(w["table"][0]) * 16 - 1
        w["new"][1] = 2
    elif what == "tokens":
        w["T"] = sum(w["new"]) - 1
    elif what == "count_negative":
        w["count"] = -1
    elif what == "count_high":
        w["count"] = len(w["free"]) + 1
    else:
        w["seq"][3] = w["new"][3] = 2147483647
    got = check_extend(w)
    assert got["err"] == bit and got["page_table"] == w["table"]


def test_extend_bad_page_ids():
    """A negative id in the stack, and one in a partly filled page's entry."""
    w = make(6, 16, 40, 100, seed=9)
    w["free"][w["count"] - 1] = -4
    w["seq"][2], w["new"][2] = 5, 3
    w["table"][2][0] = -1
    got = check_extend(w)
    assert got["err"] == 2 and -1 in got["slots"][:sum(w["new"])]


def run_release(w, finished, cap=None, in_place=False):
    seq, table = torch.tensor(w["seq"], **I32), torch.tensor(w["table"], **I32)
    free, count = torch.tensor(w["free"], **I32), torch.tensor([w["count"]], **I32)
    out = seq if in_place else torch.full((len(w["seq"]),), 77, **I32)
    count_out = count if in_place else torch.full((1,), 77, **I32)
    err = torch.zeros(1, **I32)
    binding.dsa_pages_release(torch.tensor(finished, device="cuda"), seq, table, w["page"], free, count, count_out, out,
                              err_flag=err)
    torch.cuda.synchronize()
    assert table.tolist() == w["table"]
    return dict(free_pages=free.tolist(), free_count=int(count_out.item()), seq_lens=out.tolist(), err=int(err.item()))


def check_release(w, finished, **kw):
    want = ref.release(finished, w["seq"], w["table"], w["page"], w["free"], w["count"])
    got = run_release(w, finished, **kw)
    assert got == want
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,ctx", [(1, 16, 40), (1, 1, 5000), (7, 64, 0), (64, 64, 900), (600, 16, 300), (16384, 256, 3)])
def test_release(B, page, ctx, in_place):
    r = random.Random(B)
    w = make(B, page, 0, ctx, seed=B + 1)
    w["free"] += [-9] * sum(ref.pages_of(s, page) for s in w["seq"])
    for share in (0.0, 0.3, 1.0):
        check_release(w, [r.random() < share for _ in range(B)], in_place=in_place)


@pytest.mark.parametrize("what,bit", [("room", 32), ("length", 16), ("negative", 16), ("count", 16)])
def test_release_refused_changes_nothing(what, bit):
    w = make(9, 16, 0, 100, seed=10)
    w["seq"][3] = max(w["seq"][3], 17)
    w["table"][3][:2] = [900, 901]
    w["free"] += [-9] * 200
    if what == "room":
        w["free"] = w["free"][:w["count"] + 1]
    elif what == "length":
        w["seq"][5] = len(w["table"][0]) * 16 + 1
    elif what == "negative":
        w["seq"][5] = -2
    else:
        w["count"] = len(w["free"]) + 1
    got = check_release(w, [True] * 9)
    assert got["err"] == bit and got["free_pages"] == w["free"] and got["seq_lens"] == w["seq"]


def test_release_bad_page_is_pushed_and_reported():
    w = make(9, 16, 0, 100, seed=10)
    w["seq"][3] = max(w["seq"][3], 17)
    w["table"][3][:2] = [900, -1]
    w["free"] += [-9] * 200
    assert check_release(w, [True] * 9)["err"] == 2


def test_captured_steps():
    """A captured in-place step, replayed: lengths and the free count move on the GPU alone."""
    w = make(6, 16, 3, 30, seed=11, spare=40)
    B, T = 6, w["T"]
    seq, new = torch.tensor(w["seq"], **I32), torch.tensor(w["new"], **I32)
    table = torch.full((B, 12), -1, **I32)
    table[:, :len(w["table"][0])] = torch.tensor(w["table"], **I32)
    free, count = torch.tensor(w["free"], **I32), torch.tensor([w["count"]], **I32)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    pos, ts, cu = torch.zeros(T, **I32), torch.zeros(T, **I32), torch.zeros(B + 1, **I32)
    g = torch.cuda.CUDAGraph()
    lists = dict(seq=seq.tolist(), table=table.tolist(), count=w["count"])
    with torch.cuda.graph(g):
        binding.dsa_pages_extend(seq, new, table, 16, free, count, count, slots, pos, ts, cu, seq)
    for step in range(4):
        g.replay()
        torch.cuda.synchronize()
        want = ref.extend(lists["seq"], w["new"], lists["table"], 16, w["free"], lists["count"], T)
        assert slots.tolist() == want["slots"] and table.tolist() == want["page_table"], step
        assert seq.tolist() == want["kv_lens"] and int(count.item()) == want["free_count"]
        lists = dict(seq=want["kv_lens"], table=want["page_table"], count=want["free_count"])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T", [4095, 4096, 4097])
def test_extend_around_one_cta(T, in_place):
    """4096 token rows are the largest call of one CTA, one more the smallest with a grid and a finishing launch."""
    w = make(40, 16, 90, 100, seed=13)
    assert sum(w["new"]) <= T
    w["T"] = T
    check_extend(w, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,width", [(63, 65), (64, 64), (17, 241)])
def test_release_around_one_cta(B, width, in_place):
    """Tables of 4095, 4096 and 4097 entries, every page of them held."""
    r = random.Random(B)
    ids = list(range(B * width))
    r.shuffle(ids)
    w = dict(seq=[width * 4 - r.randint(0, 3) for _ in range(B)], new=[0] * B, page=4, count=3, T=1,
             table=[ids[b * width:(b + 1) * width] for b in range(B)], free=[-1, -2, -3] + [-9] * (B * width))
    for share in (0.3, 1.0):
        check_release(w, [r.random() < share for _ in range(B)], in_place=in_place)


def test_captured_steps_of_a_grid():
    """Calls of a grid and its finishing launch, lengths and count in place: pages handed out and returned in one
    captured step, replayed with other lengths each time."""
    r = random.Random(14)
    B, page, width, T = 90, 16, 80, 9000
    n_pages = B * width
    ids = list(range(n_pages))
    r.shuffle(ids)
    w = dict(seq=[0] * B, table=[[-1] * width for _ in range(B)], free=ids, count=n_pages)
    seq, new = torch.tensor(w["seq"], **I32), torch.zeros(B, **I32)
    table, free, count = torch.tensor(w["table"], **I32), torch.tensor(w["free"], **I32), torch.tensor([n_pages], **I32)
    done = torch.zeros(B, dtype=torch.bool, device="cuda")
    slots, pos, ts = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, **I32), torch.zeros(T, **I32)
    cu, err = torch.zeros(B + 1, **I32), torch.zeros(1, **I32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.dsa_pages_extend(seq, new, table, page, free, count, count, slots, pos, ts, cu, seq, err_flag=err)
        binding.dsa_pages_release(done, seq, table, page, free, count, count, seq, err_flag=err)
    for step in range(5):
        grow = [r.randint(0, 190) for _ in range(B)]
        out = [r.random() < 0.3 for _ in range(B)]
        new.copy_(torch.tensor(grow))
        done.copy_(torch.tensor(out))
        g.replay()
        torch.cuda.synchronize()
        a = ref.extend(w["seq"], grow, w["table"], page, w["free"], w["count"], T)
        b = ref.release(out, a["kv_lens"], a["page_table"], page, w["free"], a["free_count"])
        assert slots.tolist() == a["slots"] and pos.tolist() == a["positions"] and ts.tolist() == a["token_seq"], step
        assert cu.tolist() == a["cu_q"] and table.tolist() == a["page_table"]
        assert seq.tolist() == b["seq_lens"] and int(count) == b["free_count"] and free.tolist() == b["free_pages"]
        assert int(err) == a["err"] | b["err"]
        err.zero_()
        w = dict(seq=b["seq_lens"], table=a["page_table"], free=b["free_pages"], count=b["free_count"])
