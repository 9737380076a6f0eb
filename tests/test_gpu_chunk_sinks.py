"""Dense attention where a few keys dominate a long tail: the tail's share of the softmax has to reach O.

The bound does not grow with the number of keys.  Per output, beside the BF16 rounding of O (2^-8 |O|), the two E4M3
terms of each weight and the FP32 scores (as in dense_ref.chunk_attn: (2^-8 + 2^-12 + 2 mag) sum_j w_j |v_j|), what
the weights lose to E4M3's smallest step may be 2^-7 sum_j w_j S_j max_j |b_jd|, with b the rows' bytes and S_j the
power of two above row j's largest scale: a 128th of the softmax.  Rounded up or down by position, a weight's operand
is off by 2^-14 2^M at most in the RMS, 2^M <= 2^-lift max_j w_j S_j, so the 128 n keys of a segment leave
sqrt(128 n) 2^-14 2^-lift max_j w_j S_j times the RMS of the bytes.  With lift 1 up to 255 tiles and 2 up to 1023
that is 2^-8.5 at n = 64, 2^-8.2 at 96 and 2^-8 at 547; bytes with a mean, as here, are at most half as large in the
RMS as the largest one, so the bound is three to six times that, and the sum of the weights itself is better still."""
import math

import pytest
import torch

import dense_ref as ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
LAYOUTS = ["raw512", "scaled528", "rope656"]
SCALE = 1 / math.sqrt(576.0)
BF = torch.bfloat16


def rows_of(x, layout):
    """Pool bytes of the latent rows x [n, 512], as the writers leave them (RoPE dims 0)."""
    pool = torch.zeros(x.shape[0], ref.ROW_BYTES[layout], dtype=torch.uint8)
    if layout == "raw512":
        pool[:] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        return pool
    x = x.view(-1, 4, 128)
    s = x.abs().amax(-1, keepdim=True) / 448.0
    pool[:, :512] = torch.where(s > 0, x / s, torch.zeros(())).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 512)
    pool[:, 512:528] = s.reshape(-1, 4).contiguous().view(torch.uint8)
    return pool


def channel(kind, n, g):
    """Dim 0 of the keys, the one that scores look at: 8 is the top."""
    c = torch.zeros(n)
    if kind == "first":
        c[0] = 8
    elif kind == "spread":
        c = (torch.randn(n, generator=g) * 0.7).clamp(-4, 4)
        c[0] = 8
    elif kind == "late":
        c[n // 2 + 5] = 8
    elif kind == "many":
        c[64::1024] = 8
    elif kind == "a_tile":                  # one in every tile, and a larger one in front
        c[7::128] = 4
        c[3] = 8
    elif kind == "falling":
        c = 8 * (1 - torch.arange(n) / n)
    else:
        assert kind == "steps"              # falls and rises again
        c = 8 * (0.5 + 0.5 * torch.cos(torch.arange(n) * (6 * math.pi / n)))
    return c


def check(kind, layout, keys, requests, H, gaps, equal_values=False, seed=0, mean=1.0, dev=0.25):
    """`requests` requests of one token over the same pages; head h scores its top key gaps[h % len] nats above 0."""
    g = torch.Generator().manual_seed(seed)
    x = mean + (0 if equal_values else dev) * torch.randn(keys, 512, generator=g)
    x[:, 0] = channel(kind, keys, g)
    pool = rows_of(x, layout)
    page = 64
    n_pages = ref.pages_of(keys, page)
    ids = torch.randperm(n_pages, generator=g)
    j = torch.arange(keys)
    phys = torch.zeros(n_pages * page, pool.shape[1], dtype=torch.uint8)
    phys[ids[j // page] * page + j % page] = pool
    q = torch.zeros(H, ref.KEY_DIMS[layout])
    q[:, 0] = torch.tensor([gaps[h % len(gaps)] / (8 * SCALE) for h in range(H)])
    q = q.to(BF)
    o = torch.zeros(requests, H, 512, dtype=BF, device="cuda")
    lse = torch.zeros(requests, H, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.dsa_chunk_attn(q.cuda()[None].expand(requests, -1, -1).contiguous(), phys.cuda(), layout,
                           ids.to(torch.int32).cuda()[None].expand(requests, -1).contiguous(), page,
                           torch.arange(requests + 1, dtype=torch.int32, device="cuda"),
                           torch.full((requests,), keys, dtype=torch.int32, device="cuda"), SCALE, o, lse,
                           binding.chunk_workspace_for(requests, H, requests, layout), err_flag=err)
    assert int(err) == 0
    k, v = ref.dequant(pool, layout)
    qd = q.double()
    s = qd[:, :512] @ k[:, :512].T * SCALE
    z = torch.logsumexp(s, -1)
    w = (s - z[:, None]).exp()
    want = w @ v
    mag = (qd[:, :512].abs() @ k[:, :512].abs().T * SCALE).amax(-1) * 2.0 ** -16 + 2.0 ** -18
    S = torch.ones(keys, dtype=torch.float64)
    if layout != "raw512":
        S = 2.0 ** torch.floor(torch.log2(pool[:, 512:528].contiguous().view(torch.float32).double().amax(1)) + 1)
    codes = pool[:, :512].contiguous().view(torch.float8_e4m3fn).double().abs().amax(0)
    tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * mag[:, None]) * (w @ v.abs())
           + 2.0 ** -7 * (w * S).sum(-1)[:, None] * codes)
    d = (o.double().cpu() - want).abs()
    assert (d <= tol).all(), f"O off by up to {(d / want.abs().clamp(min=1e-9)).max():.3f} of it, {(d / tol).max():.1f} times the bound"
    assert ((lse.double().cpu() - z).abs() <= mag + z.abs() * 2.0 ** -22).all()
    return o.double().cpu(), want


GAPS = [6, 7, 8, 9, 9.5, 10, 10.5, 11, 12, 13, 14, 15, 16, 18, 20, 24]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", ["first", "spread", "late", "many", "a_tile"])
@pytest.mark.parametrize("keys,requests,H", [(8192, 160, 16), (12288, 90, 32), (20000, 1, 16), (777, 3, 8)])
def test_tail_of_a_dominant_key(layout, kind, keys, requests, H):
    """Row groups that one SM takes whole, of 16 and 32 query rows, and ones spread over SMs."""
    check(kind, layout, keys, requests, H, GAPS)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", ["first", "spread"])
@pytest.mark.parametrize("keys,requests,H", [(8192, 160, 16), (16384, 90, 32)])
def test_tail_of_large_rows(layout, kind, keys, requests, H):
    """Latents of N(0, 8^2): sums that cancel."""
    check(kind, layout, keys, requests, H, GAPS, mean=0.0, dev=8.0, seed=1)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_weights_sum_to_one(layout):
    """Equal values: O is that value, whatever the scores."""
    o, _ = check("first", layout, 16384, 160, 16, GAPS, equal_values=True)
    # the weights' own errors, 2^-8 each, and their loss, 2^-7 (twice for S above the scale); BF16 adds 2^-8
    assert (o[:, :, 128:] - 1.0).abs().max() <= 2.0 ** -7 * 2 + 2.0 ** -8 * 2


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", ["first", "spread", "many", "falling", "steps"])
def test_long_segments(layout, kind):
    """More than 256 tiles of one SM: the reference of the weights follows the keys down."""
    check(kind, layout, 70001, 160, 8, [10, 12, 14, 16, 20, 40, 90, 300])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("keys,requests,H", [(8192, 160, 16), (12288, 90, 32), (32000, 160, 16)])
def test_library_tolerance(layout, keys, requests, H):
    """|dO| <= 1e-2 + 1e-2 |O|, as for the sparse kernel, for latents of RMS 1 behind a dominant key."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(keys, 512, generator=g)
    x[:, 0] = channel("first", keys, g) / 4
    pool = rows_of(x, layout)
    n = ref.pages_of(keys, 64)
    phys = torch.zeros(n * 64, pool.shape[1], dtype=torch.uint8)
    phys[:keys] = pool
    q = torch.zeros(H, ref.KEY_DIMS[layout])
    q[:, 0] = torch.tensor([GAPS[h % 16] / (2 * SCALE) for h in range(H)])
    q = q.to(BF)
    o, lse = torch.zeros(requests, H, 512, dtype=BF, device="cuda"), torch.zeros(requests, H, device="cuda")
    binding.dsa_chunk_attn(q.cuda()[None].expand(requests, -1, -1).contiguous(), phys.cuda(), layout,
                           torch.arange(n, dtype=torch.int32, device="cuda")[None].expand(requests, -1).contiguous(), 64,
                           torch.arange(requests + 1, dtype=torch.int32, device="cuda"),
                           torch.full((requests,), keys, dtype=torch.int32, device="cuda"), SCALE, o, lse,
                           binding.chunk_workspace_for(requests, H, requests, layout))
    k, v = ref.dequant(pool, layout)
    s = q.double()[:, :512] @ k[:, :512].T * SCALE
    want = s.softmax(-1) @ v
    assert ((o.double().cpu() - want).abs() <= 1e-2 + 1e-2 * want.abs()).all()
    assert ((lse.double().cpu() - torch.logsumexp(s, -1)).abs() <= 1e-3).all()
