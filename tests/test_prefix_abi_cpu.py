"""Host checks of the attention behind shared prefixes."""
import pytest
import torch

from sparse_mla_attention_page_gb300 import binding
from sparse_mla_attention_page_gb300 import build

P = 0x10000          # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


ATT = dict(q=P, T=4, H=16, D=512, pool=P, rows=4096, layout=0, kvd=512, table=P, B=2, mp=8, ps=64, cu=P, kv=P, gcu=P, pl=P, G=1,
           causal=1, sc=0.1, o=P, lse=P, ws=P, wsb=1 << 40, err=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 2), (dict(T=0), 0), (dict(T=0, gcu=None, pl=None, q=None), 0), (dict(rows=-1), 2), (dict(rows=0), 2),
    (dict(rows=1 << 31), 2), (dict(layout=3), 3), (dict(layout=-1), 3), (dict(layout=18), 3), (dict(D=576), 4), (dict(layout=2), 4),
    (dict(layout=17), 4), (dict(kvd=528), 4), (dict(H=0), 6), (dict(H=1025), 6), (dict(B=0, G=0), 2), (dict(B=4097), 2),
    (dict(G=-1), 2), (dict(G=3), 2), (dict(mp=0), 2), (dict(ps=0), 2), (dict(mp=1 << 20, ps=1 << 12), 2), (dict(q=P + 8), 10),
    (dict(pool=P + 8), 10), (dict(o=P + 8), 10), (dict(lse=P + 2), 10), (dict(cu=P + 2), 10), (dict(gcu=P + 2), 10),
    (dict(pl=P + 1), 10), (dict(ws=None), 7), (dict(wsb=0), 7), (dict(ws=P + 16), 10),
] + [({k: None}, 1) for k in ("q", "pool", "table", "cu", "kv", "gcu", "pl", "o", "lse")])
def test_arguments(L, kw, code):
    assert L.dsa_prefix_attn(*dict(ATT, **kw).values()) == code


def test_workspace(L):
    """None for sizes out of range; enough for every call of no more tokens, heads and requests; the limit is exact."""
    f = L.dsa_prefix_attn_workspace_bytes
    for bad in ((-1, 16, 1, 0), (1, 0, 1, 0), (1, 1025, 1, 0), (1, 16, 0, 0), (1, 16, 4097, 0), (1, 16, 1, 5)):
        assert f(*bad) == 0
    sizes = [(T, H, B) for T in (1, 5, 17, 64, 300, 8192) for H in (1, 16, 128) for B in (1, 7, 64, 500)]
    need = {s: f(*s, 17) for s in sizes}
    for s in sizes:
        assert need[s] >= L.dsa_chunk_attn_workspace_bytes(*s, 17)
        for t in sizes:
            if all(x <= y for x, y in zip(s, t)):
                assert need[s] <= need[t], (s, t)
    n = f(4, 16, 2, 0)
    assert L.dsa_prefix_attn(*dict(ATT, wsb=n - 1).values()) == 7
    if not torch.cuda.is_available():
        assert L.dsa_prefix_attn(*dict(ATT, wsb=n).values()) == 8
        assert L.dsa_prefix_attn(*dict(ATT, wsb=n, G=0, gcu=None, pl=None).values()) == 8
