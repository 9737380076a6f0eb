"""Attention behind shared prefixes by the number of heads: which calls look at the groups at all, and rows of a token over
several units, packed with others'."""
import pytest
import torch

from sparse_mla_attention_page_gb300 import binding
from test_gpu_prefix_attn import MIXED, ONE, check, common, make, run

pytestmark = pytest.mark.gpu


def widen(w, tiles):
    """The page table with room for that many tiles of 128 keys more."""
    w["table"] = torch.cat([w["table"], torch.full((w["table"].shape[0], tiles * 128 // w["page"]), -1, dtype=torch.int32)], 1)
    return w


def tangle(w):
    """Groups out of order: flagged by a call that looks at them, right results all the same."""
    w["gcu"], w["plens"] = torch.tensor([0, 3, 2, w["table"].shape[0]], dtype=torch.int32), torch.full((3,), 640, dtype=torch.int32)
    return w


@pytest.mark.parametrize("layout", ["raw512", "rope656", "fp4_416"])
@pytest.mark.parametrize("H,B", [(32, 20), (64, 10), (96, 7), (128, 5)])
def test_whole_units_are_not_shared(layout, H, B):
    """Heads that fill the units leave nothing to pack, however wide the page table: the groups are not looked at, and the
    call is dsa_chunk_attn, bit for bit."""
    w = tangle(widen(make([(640, ONE[:B] + ONE[:max(0, B - len(ONE))])], H, layout, seed=H), 2000))
    o, lse = check(w, only=[0, 1, B - 1])
    o2, lse2, err = run(w, fn="chunk")
    assert err == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", ["raw512", "fp4_416"])
@pytest.mark.parametrize("H", [32, 64])
def test_whole_units_of_many_parts(layout, H):
    """Few units, each spread over many SMs: the call goes to the shared kernel for its join, and nothing is shared."""
    few = ONE[:512 // H]
    p = 128 * 300
    check(make([(p, few)], H, layout, seed=H), only=[0, 1, len(few) - 1])
    check(tangle(make([(p, few)], H, layout, seed=H)), err_want=binding.DSA_DEV_ERR_LENGTH, only=[0, 2])


@pytest.mark.parametrize("layout", ["raw512", "rope656", "fp4_416"])
@pytest.mark.parametrize("H", [24, 40, 48, 100])
def test_rows_of_a_token_over_several_units(layout, H):
    """Heads that fill whole units and a part of one: the shared pages are hidden from all requests but the first."""
    p = common(H, MIXED)
    w = make([(p + 77, MIXED)], H, layout, seed=H)
    check(w, hidden=[p], only=[0, 1, 2, 5, len(MIXED) - 1])


@pytest.mark.parametrize("layout", ["scaled528", "fp4_288"])
def test_wide_tokens_in_several_groups(layout):
    """Groups that begin inside a unit of the packed rows, requests of none between them, one without new tokens."""
    p = common(40, MIXED)
    groups = [(p, MIXED), (p // 2, [(0, 9)] + MIXED[:7])]
    w = make(groups, 40, layout, page=16, seed=5, alone=([(1, 60)], [(2, 33)]), lead=2, tail=1)
    check(w, hidden=[p, 0], only=[0, 1, 2, 7, 12, 14, 20, 21])


def test_bound_of_the_saving():
    """The page table has to have room for what packing could save at most: 64 rows of 48 heads are 128 units alone and 96
    packed, 32 x 15 tiles are three for each of 152 SMs, 32 x 14 less."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    enough = -(-3 * sms // 32)
    for tiles, looked in ((enough - 1, False), (enough, True)):
        w = make([], 48, "raw512", seed=1, alone=([(1, 20 + b) for b in range(64)], []))
        w["table"] = torch.cat([w["table"], torch.full((64, tiles * 2), -1, dtype=torch.int32)], 1)[:, :tiles * 2].contiguous()
        check(tangle(w), err_want=binding.DSA_DEV_ERR_LENGTH if looked else 0, only=[0, 31, 63])


@pytest.mark.parametrize("B,H,layout", [(16, 32, "raw512"), (4, 64, "fp4_416"), (16, 16, "rope656"), (2, 128, "scaled528")])
def test_few_long_units(B, H, layout):
    """Units that would be spread over 9 to 24 SMs (of 152) go to the shared kernel from 24 tiles of the page table on."""
    for tiles, looked in ((23, False), (24, True)):
        w = make([], H, layout, seed=2, alone=([(1, tiles * 128 - 1 - 130 * b) for b in range(B)], []))
        w["table"] = w["table"][:, :tiles * 2].contiguous()
        w["gcu"], w["plens"] = torch.tensor([0, B + 1], dtype=torch.int32), torch.tensor([640], dtype=torch.int32)
        check(w, err_want=binding.DSA_DEV_ERR_LENGTH if looked else 0, only=[0, B // 2, B - 1])
