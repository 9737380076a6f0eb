"""Multi-axis rotary positions joined with the query concatenation and the 656-byte row writer."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def inputs(T, H, seed, strided=False, axes=3, far=100000):
    g = torch.Generator().manual_seed(seed)
    rnd = (lambda *s: torch.randn(*s, generator=g).to(BF))
    w = dict(q_nope=rnd(T, H, 512), q_pe=rnd(T, H, 64), kv_c=rnd(T, 512) * 3, k_pe=rnd(T, 64))
    w["kv_c"][T // 2] = 0                                 # a zero row: scales 0
    if strided:
        w["q_nope"] = rnd(H, T, 520).transpose(0, 1)[:, :, 8:]       # head-major projection output
        w["q_pe"] = rnd(T, H, 192)[:, :, 128:]
        both = rnd(T, 584)                                 # latent and RoPE dims of one projection
        w["kv_c"], w["k_pe"] = both[:, :512], both[:, 512:576]
    w["positions"] = torch.randint(0, far, (axes, T), generator=g, dtype=torch.int32)
    w["slots"] = torch.randperm(T + 9, generator=g)[:T]
    w["slots"][::7] = -1
    return w


def dev(t):
    """To the GPU with the strides kept."""
    base = torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device="cuda")
    return base.copy_(t)


def run(w, spec, queries=True, rows=True, nope=True, stream=None):
    T, H = w["q_pe"].shape[:2]
    d = {k: dev(v) for k, v in w.items()}
    q_out = torch.full((T, H, 576), 7.0, dtype=BF, device="cuda")
    pool = torch.full((T + 9, 656), 0xA5, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    binding.dsa_rope_qkv656(d["q_nope"] if queries and nope else None, d["q_pe"] if queries else None,
                            q_out if queries else None, *((d[k] if rows else None) for k in ("kv_c", "k_pe", "slots")),
                            pool if rows else None, d["positions"], spec, err_flag=err, stream=stream)
    torch.cuda.synchronize()
    return q_out.cpu(), pool.cpu(), int(err.item())


def check_turned(got, x, w, spec):
    want = ref.turned(x.double().numpy(), w["positions"].numpy(), list(spec.axis), list(spec.inv_freq),
                      bool(spec.interleaved), spec.mscale)
    # cos and sin to 2^-21 of FP32 sums of two products (2^-22), then the BF16 rounding (2^-8 of the value)
    mag = np.abs(x.double().numpy()).max(-1, keepdims=True) * 2
    assert (np.abs(got.double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag * abs(spec.mscale)).all()


def check(w, spec, **kw):
    q, pool, err = run(w, spec, **kw)
    assert err == 0
    T = w["slots"].shape[0]
    assert torch.equal(q[:, :, :512].view(torch.int16), w["q_nope"].contiguous().view(torch.int16))
    check_turned(q[:, :, 512:], w["q_pe"], w, spec)
    put = w["slots"] >= 0
    at = w["slots"][put]
    rest = torch.ones(T + 9, dtype=torch.bool)
    rest[at] = False
    assert (pool[rest] == 0xA5).all()                     # rows of no slot are left alone
    check_turned(pool[at][:, 528:].contiguous().view(BF), w["k_pe"][put], dict(positions=w["positions"][:, put]), spec)
    # the latent part is the existing writer's, byte for byte
    x = torch.cat([w["kv_c"], w["k_pe"]], 1).contiguous().cuda()
    other = torch.zeros(T + 9, 656, dtype=torch.uint8, device="cuda")
    binding.dsa_kv_write_rope656(x, w["slots"].cuda(), other)
    assert torch.equal(pool[at][:, :528], other.cpu()[at][:, :528])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (3, 20), (64, 16), (37, 128), (700, 32)])
def test_shapes(T, H, interleaved):
    check(inputs(T, H, T + H), binding.rope_spec(10000.0, (8, 12, 12), interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_inputs(interleaved):
    check(inputs(50, 12, 5, strided=True), binding.rope_spec(10000.0, (8, 12, 12), interleaved))


@pytest.mark.parametrize("T,H", [(1500, 128)])
def test_several_heads_an_item(T, H):
    """Enough rows that a warp takes several heads of a token."""
    w = inputs(T, H, 6)
    q, _, _ = run(w, binding.rope_spec(10000.0, (8, 12, 12), True))
    assert torch.equal(q[:, :, :512].view(torch.int16), w["q_nope"].view(torch.int16))
    check_turned(q[:, :, 512:], w["q_pe"], w, binding.rope_spec(10000.0, (8, 12, 12), True))


@pytest.mark.parametrize("spec", [
    binding.rope_spec(500000.0, (32,), True),
    binding.rope_spec(10000.0, axis=[i % 3 for i in range(32)], interleaved=False, mscale=1.25),
    binding.rope_spec(inv_freq=[0.0, -0.5, 7.25, 3.0e5] + [1e-6] * 28, sections=(4, 4, 4, 4, 4, 4, 4, 4), interleaved=True),
])
def test_specs(spec):
    """One axis, interleaved axis assignment with a factor, eight axes with unusual frequencies."""
    check(inputs(33, 8, 7, axes=spec.n_axes, far=3000), spec)


def test_far_and_negative_positions():
    w = inputs(40, 8, 8)
    w["positions"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, 40), generator=torch.Generator().manual_seed(1),
                                   dtype=torch.int64).to(torch.int32)
    # frequencies whose products with any position are exact in the reference's doubles
    spec = binding.rope_spec(inv_freq=[2.0 ** -(i // 2) for i in range(32)], sections=(8, 12, 12), interleaved=True)
    q, pool, err = run(w, spec)
    x = w["q_pe"].double().numpy()
    # fraction of a turn with whole numbers: p 2^-k / (2 pi) in 200 bits
    inv_two_pi = 0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E410 # 2^192 / (2 pi), rounded down
    want = np.array(x)
    for i in range(32):
        p = [int(v) for v in w["positions"][spec.axis[i]]]
        frac = np.array([((v * inv_two_pi >> (i // 2)) % (1 << 192)) / float(1 << 192) for v in p])
        c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
        want[..., 2 * i], want[..., 2 * i + 1] = (x[..., 2 * i] * c - x[..., 2 * i + 1] * s,
                                                 x[..., 2 * i + 1] * c + x[..., 2 * i] * s)
    # a double's 1 / (2 pi) and product: 2^-51 of up to 2^31 / 6 turns a position is 2^-22 turns at the farthest
    mag = np.abs(x).max(-1, keepdims=True) * 2
    got = q[:, :, 512:].double().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mag).all()


def test_one_side_only():
    w = inputs(20, 8, 9)
    spec = binding.rope_spec(10000.0, (8, 12, 12), False)
    q, pool, _ = run(w, spec)
    q1, p1, _ = run(w, spec, rows=False)
    assert torch.equal(q1, q) and (p1 == 0xA5).all()
    q2, p2, _ = run(w, spec, queries=False)
    assert (q2 == 7).all() and torch.equal(p2, pool)
    q3, _, _ = run(w, spec, nope=False)
    assert (q3[:, :, :512] == 7).all() and torch.equal(q3[:, :, 512:], q[:, :, 512:])


def test_text_positions_one_row_for_every_axis():
    w = inputs(21, 8, 10, axes=1)
    spec = binding.rope_spec(10000.0, (8, 12, 12), False)
    pos = w["positions"].cuda().expand(3, -1)
    q = torch.zeros(21, 8, 576, dtype=BF, device="cuda")
    binding.dsa_rope_qkv656(w["q_nope"].cuda(), w["q_pe"].cuda(), q, None, None, None, None, pos, spec)
    w["positions"] = w["positions"].expand(3, -1).contiguous()
    check_turned(q[:, :, 512:].cpu(), w["q_pe"], w, spec)


def test_nan_and_inf_stay_in_their_rows():
    w = inputs(16, 8, 11)
    clean, pool_clean, _ = run(w, binding.rope_spec(10000.0, (8, 12, 12), True))
    w["q_pe"][3, 2, 10] = float("nan")
    w["q_nope"][4, 1, 0] = float("inf")
    w["kv_c"][5, 7] = float("nan")
    q, pool, _ = run(w, binding.rope_spec(10000.0, (8, 12, 12), True))
    assert torch.isnan(q[3, 2, 512 + 10]) and torch.isinf(q[4, 1, 0])
    q[3, 2, 512 + 10:512 + 12] = clean[3, 2, 512 + 10:512 + 12]
    q[4, 1, 0] = clean[4, 1, 0]
    assert torch.equal(q.view(torch.int16), clean.view(torch.int16))
    s = int(w["slots"][5])
    keep = [r for r in range(pool.shape[0]) if r != s]
    assert torch.equal(pool[keep], pool_clean[keep])


def test_slot_beyond_the_pool():
    w = inputs(16, 8, 12)
    w["slots"][4] = 25                                     # the pool has 25 rows
    q, pool, err = run(w, binding.rope_spec(10000.0, (8, 12, 12)))
    assert err == binding.DSA_DEV_ERR_SLOT_RANGE


def test_other_stream_and_graph():
    w = inputs(30, 8, 13)
    spec = binding.rope_spec(10000.0, (8, 12, 12), True)
    want, pool, _ = run(w, spec)
    got, pool2, _ = run(w, spec, stream=torch.cuda.Stream())
    assert torch.equal(got, want) and torch.equal(pool, pool2)
    d = {k: dev(v) for k, v in w.items()}
    q = torch.zeros(30, 8, 576, dtype=BF, device="cuda")
    p = torch.full((39, 656), 0xA5, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.dsa_rope_qkv656(d["q_nope"], d["q_pe"], q, d["kv_c"], d["k_pe"], d["slots"], p, d["positions"], spec)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q.cpu(), want) and torch.equal(p.cpu(), pool)


def exact_turned(x, positions, axis, inv_freq, interleaved):
    """x [T, 64] float64 turned by angles that are reduced in 80 decimal digits."""
    import decimal
    with decimal.localcontext() as ctx:
        ctx.prec = 80
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899863")
        out = np.array(x, dtype=np.float64)
        for i in range(32):
            step = decimal.Decimal(float(inv_freq[i]))
            ang = np.array([float((int(p) * step) % two_pi) for p in positions[axis[i]]])
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
            a, b = x[:, ia], x[:, ib]
            out[:, ia], out[:, ib] = a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [1.0, 40.0, 1e4, 1e7])
def test_far_positions_at_any_frequency(top, interleaved):
    """Positions up to 2^31 and frequencies of many turns a step keep full precision."""
    w = inputs(40, 2, seed=21, axes=1, far=2 ** 31 - 1)
    w["positions"][0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1], dtype=torch.int32)
    spec = binding.rope_spec(inv_freq=[top * 0.7 ** i * (-1) ** i for i in range(32)], axis=[0] * 32, interleaved=interleaved)
    q, _, err = run(w, spec)
    assert err == 0
    for h in range(2):
        x = w["q_pe"][:, h].double().numpy()
        want = exact_turned(x, w["positions"].tolist(), [0] * 32, list(spec.inv_freq), interleaved)
        mag = np.abs(x).max(-1, keepdims=True) * 2
        d = np.abs(q[:, h, 512:].double().numpy() - want)
        assert (d <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag).all(), d.max()
