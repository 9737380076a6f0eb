"""The release of requests that begin with pages of a shared prefix."""
import random

import pytest
import torch

import dense_ref as ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def release_own(finished, shared, seq, table, page, free, count):
    """Lists in, the call's outputs as a dict of lists."""
    room = len(table[0]) * page
    back = [(b, p) for b, f in enumerate(finished) if f for p in range(shared[b], ref.pages_of(seq[b], page))]
    out = dict(free_pages=list(free), free_count=count, seq_lens=list(seq), err=0)
    if any(s < 0 or s > room for s in seq) or any(s < 0 for s in shared) or not 0 <= count <= len(free):
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


def check(finished, shared, seq, table, page, free, count, in_place=False):
    want = release_own(finished, shared, seq, table, page, free, count)
    d = dict(seq=torch.tensor(seq, **I32), free=torch.tensor(free, **I32), count=torch.tensor([count], **I32))
    err = torch.zeros(1, **I32)
    count_out = d["count"] if in_place else torch.full((1,), -7, **I32)
    seq_out = d["seq"] if in_place else torch.full((len(seq),), -7, **I32)
    tab = torch.tensor(table, **I32)
    binding.dsa_pages_release_own(torch.tensor(finished, device="cuda"), torch.tensor(shared, **I32), d["seq"], tab, page,
                                  d["free"], d["count"], count_out, seq_out, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == want["err"]
    assert d["free"].tolist() == want["free_pages"]
    assert int(count_out.item()) == want["free_count"] and seq_out.tolist() == want["seq_lens"]
    assert tab.tolist() == table


def case(B, pages, page, r):
    table = [[r.randrange(10 ** 6) for _ in range(pages)] for _ in range(B)]
    seq = [r.choice([0, 1, page, page + 1, r.randrange(pages * page + 1), pages * page]) for _ in range(B)]
    shared = [r.randrange(ref.pages_of(s, page) + 2) for s in seq]
    return table, seq, shared


@pytest.mark.parametrize("B,pages,page", [(1, 1, 1), (3, 4, 16), (70, 9, 64), (1500, 12, 3)])
@pytest.mark.parametrize("part", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_batches(B, pages, page, part, in_place):
    """One CTA and a grid; none, some and all finished; requests of fewer pages than they share."""
    r = random.Random(B)
    table, seq, shared = case(B, pages, page, r)
    finished = [r.random() < part for _ in range(B)]
    check(finished, shared, seq, table, page, [-1] * (B * pages + 5), 5, in_place)


def test_refusals():
    r = random.Random(3)
    table, seq, shared = case(8, 5, 16, r)
    fin = [True] * 8
    check(fin, shared[:-1] + [-1], seq, table, 16, [0] * 60, 0)
    check(fin, shared, [81] + seq[1:], table, 16, [0] * 60, 0)
    check(fin, [0] * 8, [80] * 8, table, 16, [0] * 39, 0)          # one page too many for the stack
    check(fin, [0] * 7 + [1], [80] * 8, table, 16, [0] * 39, 0)    # as many as it holds
    check(fin, shared, seq, table, 16, [0] * 60, 61)
    table[2][4] = -5
    check(fin, [0] * 8, [80] * 8, table, 16, [0] * 60, 0)          # pushed as it is, flagged
    check(fin, [5] * 8, [80] * 8, table, 16, [0] * 60, 0)          # not a page of its own


def test_nothing_shared_is_the_plain_release():
    r = random.Random(4)
    table, seq, _ = case(40, 6, 16, r)
    fin = torch.tensor([r.random() < 0.5 for _ in range(40)], device="cuda")
    outs = []
    for own in (False, True):
        free, count, so = torch.full((300,), -1, **I32), torch.tensor([3], **I32), torch.zeros(40, **I32)
        args = (torch.tensor(seq, **I32), torch.tensor(table, **I32), 16, free, count, count, so)
        if own:
            binding.dsa_pages_release_own(fin, torch.zeros(40, **I32), *args)
        else:
            binding.dsa_pages_release(fin, *args)
        outs.append((free.tolist(), count.tolist(), so.tolist()))
    assert outs[0] == outs[1]


def test_binding_refusals():
    z = (lambda *s: torch.zeros(*s, **I32))
    base = dict(finished=torch.zeros(2, dtype=torch.bool, device="cuda"), shared_pages=z(2), seq_lens=z(2), page_table=z(2, 3),
                page_size=4, free_pages=z(6), free_count=z(1), free_count_out=z(1), seq_lens_out=z(2))
    for kw in (dict(shared_pages=z(3)), dict(shared_pages=z(2).long()), dict(shared_pages=z(2).cpu()), dict(shared_pages=None),
               dict(finished=z(2)), dict(page_size=0), dict(seq_lens=z(4)[::2])):
        with pytest.raises((TypeError, ValueError, binding.DsaError)):
            binding.dsa_pages_release_own(**dict(base, **kw))
    binding.dsa_pages_release_own(**base)
