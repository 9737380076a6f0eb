"""Host checks of the dense serving operators: bad arguments are refused before anything is launched."""
import ctypes

import pytest
import torch

from sparse_mla_attention_page_gb300 import binding
from sparse_mla_attention_page_gb300 import build

P = 0x10000          # aligned, never dereferenced
NO_GPU = 8 if not torch.cuda.is_available() else None


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def call(fn, names, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*[a[n] for n in names])


EXT = dict(seq=P, new=P, B=4, table=P, mp=8, ps=64, free=P, cap=32, cnt=P, cnto=P, T=16, slots=P, pos=P, ts=P, cu=P, kv=P,
           err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(B=16385), 2), (dict(mp=0), 2), (dict(ps=0), 2), (dict(mp=1 << 20, ps=1 << 12), 2),
    (dict(cap=0), 2), (dict(T=0), 2), (dict(T=-1), 2), (dict(T=1 << 30), 2), (dict(slots=P + 4), 10), (dict(seq=P + 2), 10), (dict(err=P + 1), 10),
] + [({k: None}, 1) for k in ("seq", "new", "table", "free", "cnt", "cnto", "slots", "pos", "ts", "cu", "kv")])
def test_extend(L, kw, code):
    assert call(L.dsa_pages_extend, EXT, EXT, kw) == code


REL = dict(fin=P + 1, seq=P, B=4, table=P, mp=8, ps=64, free=P, cap=32, cnt=P, cnto=P, out=P, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(B=16385), 2), (dict(mp=0), 2), (dict(ps=-1), 2), (dict(cap=0), 2), (dict(table=P + 2), 10),
] + [({k: None}, 1) for k in ("fin", "seq", "table", "free", "cnt", "cnto", "out")])
def test_release(L, kw, code):
    assert call(L.dsa_pages_release, REL, REL, kw) == code


ROPE = dict(rope=None, pos=P, ps=16, T=16, H=8, qn=P, qnt=4096, qnh=512, qp=P, qpt=512, qph=64, qo=P, kc=P, kcs=512, kp=P,
            kps=64, slots=P, pool=P, rows=64, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 2), (dict(H=0), 2), (dict(rows=-1), 2), (dict(T=0), 0), (dict(pos=None), 1), (dict(qo=None), 1),
    (dict(qp=None), 1), (dict(kp=None), 1), (dict(slots=None), 1), (dict(pool=None), 1), (dict(kc=None), 1),
    (dict(qn=P + 8), 10), (dict(qo=P + 2), 10), (dict(qp=P + 2), 10), (dict(kc=P + 8), 10), (dict(kp=P + 2), 10),
    (dict(slots=P + 4), 10), (dict(pool=P + 8), 10), (dict(qnt=4100), 10), (dict(qnh=-512), 10), (dict(qpt=513), 10),
    (dict(kcs=4), 10), (dict(kps=63), 10), (dict(qnt=1 << 62), 10), (dict(ps=-1), 2),
    (dict(qp=None, qo=None, qn=None, kc=None, kp=None, slots=None, pool=None), 1),
])
def test_rope(L, kw, code):
    spec = binding.rope_spec(10000.0, (8, 12, 12))
    assert call(L.dsa_rope_qkv656, ROPE, dict(ROPE, rope=ctypes.byref(spec)), kw) == code


def test_rope_spec_checked(L):
    for kw in (dict(inv_freq=[float("nan")] * 32), dict(inv_freq=[float("inf")] * 32)):
        assert call(L.dsa_rope_qkv656, ROPE, dict(ROPE, rope=ctypes.byref(binding.rope_spec(**kw))), {}) == 2
    spec = binding.rope_spec()
    for field, bad in (("n_axes", 0), ("n_axes", 9), ("interleaved", 2)):
        s = binding.rope_spec()
        setattr(s, field, bad)
        assert call(L.dsa_rope_qkv656, ROPE, dict(ROPE, rope=ctypes.byref(s)), {}) == 2
    spec.axis[3] = 1
    assert call(L.dsa_rope_qkv656, ROPE, dict(ROPE, rope=ctypes.byref(spec)), {}) == 2
    assert call(L.dsa_rope_qkv656, ROPE, ROPE, {}) == 1
    with pytest.raises(ValueError):
        binding.rope_spec(sections=(8, 12))
    with pytest.raises(ValueError):
        binding.rope_spec(inv_freq=[1.0])


ATT = dict(q=P, T=4, H=16, D=512, pool=P, rows=4096, layout=0, kvd=512, table=P, B=2, mp=8, ps=64, cu=P, kv=P, causal=1,
           sc=0.1, o=P, lse=P, ws=P, wsb=1 << 40, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 2), (dict(T=0), 0), (dict(rows=-1), 2), (dict(rows=0), 2), (dict(rows=1 << 31), 2), (dict(layout=3), 3),
    (dict(layout=-1), 3), (dict(D=576), 4), (dict(layout=2), 4), (dict(kvd=528), 4), (dict(H=0), 6), (dict(H=1025), 6),
    (dict(B=0), 2), (dict(B=16385), 2), (dict(mp=0), 2), (dict(ps=0), 2), (dict(mp=1 << 20, ps=1 << 12), 2),
    (dict(q=P + 8), 10), (dict(pool=P + 8), 10), (dict(o=P + 8), 10), (dict(lse=P + 2), 10), (dict(cu=P + 2), 10),
    (dict(ws=None), 7), (dict(wsb=0), 7), (dict(ws=P + 16), 10),
] + [({k: None}, 1) for k in ("q", "pool", "table", "cu", "kv", "o", "lse")])
def test_chunk_attn(L, kw, code):
    assert call(L.dsa_chunk_attn, ATT, ATT, kw) == code


def test_chunk_workspace(L):
    f = L.dsa_chunk_attn_workspace_bytes
    assert f(1, 16, 1, 0) > 0
    for bad in ((-1, 16, 1, 0), (1, 0, 1, 0), (1, 1025, 1, 0), (1, 16, 0, 0), (1, 16, 16385, 0), (1, 16, 1, 5)):
        assert f(*bad) == 0


def test_chunk_workspace_serves_smaller_calls(L):
    """A call with no more tokens, heads and requests needs no more, also where its query rows group differently."""
    sizes = [(T, H, B) for T in (1, 5, 17, 64, 300, 8192) for H in (1, 16, 128) for B in (1, 7, 64, 500)]
    need = {s: L.dsa_chunk_attn_workspace_bytes(*s, 2) for s in sizes}
    for s in sizes:
        for t in sizes:
            if all(x <= y for x, y in zip(s, t)):
                assert need[s] <= need[t], (s, t)


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_good_arguments_without_a_gpu(L):
    """Valid arguments get as far as the device check."""
    spec = binding.rope_spec(10000.0, (8, 12, 12))
    assert call(L.dsa_pages_extend, EXT, EXT, {}) == NO_GPU
    assert call(L.dsa_pages_release, REL, REL, {}) == NO_GPU
    assert call(L.dsa_rope_qkv656, ROPE, dict(ROPE, rope=ctypes.byref(spec)), {}) == NO_GPU
    assert call(L.dsa_chunk_attn, ATT, ATT, {}) == NO_GPU


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises((TypeError, RuntimeError)):
        binding.dsa_pages_extend(x, x, x.view(1, 4), 16, x, x[:1], x[:1], x.long(), x, x, x, x)
    with pytest.raises((TypeError, RuntimeError)):
        binding.dsa_chunk_attn(torch.zeros(1, 1, 512), x, "raw512", x, 16, x, x, 1.0, x, x, x)


def test_row_width_is_exact():
    """A pool one byte (or a scale, or a RoPE dim) off its layout's row size is not taken for it."""
    for lay, width, dims in ((0, 512, 512), (1, 528, 512), (2, 656, 576)):
        assert binding._kv_row_dim(torch.empty(2, width), lay) == dims
        for off in (-16, -2, -1, 1, 2, 16):
            assert binding._kv_row_dim(torch.empty(2, width + off), lay) != dims
