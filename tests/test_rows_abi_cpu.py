"""Host checks of the 4-bit rows, the reader by request and the release of a request's own pages; the formats' rules."""
import numpy as np
import pytest
import torch

import fp4_ref
from sparse_mla_attention_page_gb300 import binding
from sparse_mla_attention_page_gb300 import build

P = 0x10000          # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


WRITE = dict(kc=P, kcs=512, kp=P, kps=64, n=4, slots=P, pool=P, rows=64, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 2), (dict(rows=-1), 2), (dict(n=0, kc=None, slots=None, pool=None), 0), (dict(kc=None), 1), (dict(slots=None), 1),
    (dict(pool=None), 1), (dict(kc=P + 8), 10), (dict(kp=P + 2), 10), (dict(slots=P + 4), 10), (dict(pool=P + 8), 10),
    (dict(err=P + 2), 10), (dict(kcs=4), 10), (dict(kcs=-512), 10), (dict(kps=63), 10), (dict(kcs=1 << 61), 10),
    (dict(rows=1 << 62), 2), (dict(n=1 << 62), 2),
])
def test_write(L, kw, code):
    assert L.dsa_kv_write_fp4(*dict(WRITE, **kw).values()) == code


READ = dict(pool=P, rows=64, layout=16, table=P, B=2, mp=8, ps=64, cu=P, starts=None, out=P, n=100, stride=512, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 2), (dict(rows=0), 2), (dict(rows=1 << 31), 2), (dict(n=-1), 2), (dict(n=1 << 31), 2), (dict(layout=3), 3),
    (dict(layout=-1), 3), (dict(layout=18), 3), (dict(n=0, pool=None, table=None, cu=None, out=None), 0), (dict(B=0), 2),
    (dict(B=16385), 2), (dict(mp=0), 2), (dict(ps=0), 2), (dict(mp=1 << 20, ps=1 << 12), 2), (dict(stride=511), 2),
    (dict(layout=17), 2), (dict(layout=2), 2), (dict(stride=516), 10), (dict(out=P + 8), 10), (dict(pool=P + 8), 10),
    (dict(cu=P + 2), 10), (dict(starts=P + 1), 10), (dict(table=P + 2), 10), (dict(err=P + 1), 10),
] + [({k: None}, 1) for k in ("pool", "table", "cu", "out")])
def test_read(L, kw, code):
    assert L.dsa_kv_read(*dict(READ, **kw).values()) == code


REL = dict(fin=P + 1, shared=P, seq=P, B=4, table=P, mp=8, ps=64, free=P, cap=32, cnt=P, cnto=P, out=P, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(B=16385), 2), (dict(mp=0), 2), (dict(ps=-1), 2), (dict(cap=0), 2), (dict(table=P + 2), 10),
    (dict(shared=P + 2), 10),
] + [({k: None}, 1) for k in ("fin", "shared", "seq", "table", "free", "cnt", "cnto", "out")])
def test_release_own(L, kw, code):
    assert L.dsa_pages_release_own(*dict(REL, **kw).values()) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_good_arguments_without_a_gpu(L):
    assert L.dsa_kv_write_fp4(*WRITE.values()) == 8
    assert L.dsa_kv_write_fp4(*dict(WRITE, kp=None, kps=-1).values()) == 8
    assert L.dsa_kv_read(*READ.values()) == 8
    assert L.dsa_pages_release_own(*REL.values()) == 8


def test_row_bytes_and_other_entry_points(L):
    """The 4-bit layouts have rows; the entry points over 8-bit rows refuse them."""
    assert L.dsa_kv_row_bytes(16) == 288 and L.dsa_kv_row_bytes(17) == 416 and L.dsa_kv_row_bytes(18) == 0
    for lay in (16, 17):
        assert L.dsa_gather_dequant(P, 64, lay, None, 1, 1, 64, None, P, 4, 8, P, 1 << 30, P, None, None) == 3
        assert L.dsa_gather_dequant_workspace_bytes(4, 8, 64, lay) == 0
        for D in (512, 576):
            assert L.dsa_sparse_attn_decode(P, 4, 16, D, P, 64, lay, D, None, 1, 1, 64, None, P, 128, 0.1, P, P, None, 0,
                                            None, None) == 3
            assert L.dsa_sparse_attn_prefill_q8(P, P, 4, 16, D, P, 64, lay, D, None, 1, 1, 64, None, P, 128, 0.1, P, P, None,
                                                0, None, None) == 3
    assert binding._kv_row_dim(torch.empty(2, 288), 16) == 512 and binding._kv_row_dim(torch.empty(2, 416), 17) == 576


def test_reference_codec():
    """The tests' own codec: nearest codes, and what it encodes is what it decodes to within half a step."""
    z = np.array([0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.0])
    assert fp4_ref.code_of(z).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7]
    x = torch.randn(20, 512, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).float().numpy()
    val, s = fp4_ref.decode(fp4_ref.encode(x))
    y = val * s.repeat(128, 1)
    # half a step: a quarter of the value from 1 on, 0.25 below, 1 at the top (6 to 7); in units of the block's power
    top = np.abs(x.reshape(20, 32, 16)).max(-1).repeat(16, 1)
    assert (np.abs(y - x) <= np.maximum(np.abs(x) / 4, top / 3.5 * 0.25) + 1e-6).all()
    assert (np.abs(y).max(1) <= np.abs(x).max(1) * (1 + 1e-6)).all()
