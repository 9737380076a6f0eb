"""The Python entry points of the dense serving operators refuse what the kernels could not take, before any launch."""
import ctypes

import pytest
import torch

from sparse_mla_attention_page_gb300 import binding

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
B, T, H, W, PAGE, CAP = 3, 5, 8, 4, 16, 10


def z(*shape, dtype=I32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def extend(**kw):
    a = dict(seq_lens=z(B), new_lens=z(B), page_table=z(B, W), page_size=PAGE, free_pages=z(CAP), free_count=z(1),
             free_count_out=z(1), slots=z(T, dtype=torch.int64), positions=z(T), token_seq=z(T), cu_q=z(B + 1),
             kv_lens=z(B), err_flag=z(1))
    return binding.dsa_pages_extend(**{**a, **kw})


def release(**kw):
    a = dict(finished=z(B, dtype=torch.bool), seq_lens=z(B), page_table=z(B, W), page_size=PAGE, free_pages=z(CAP),
             free_count=z(1), free_count_out=z(1), seq_lens_out=z(B), err_flag=z(1))
    return binding.dsa_pages_release(**{**a, **kw})


def rope(**kw):
    a = dict(q_nope=z(T, H, 512, dtype=BF), q_pe=z(T, H, 64, dtype=BF), q_out=z(T, H, 576, dtype=BF),
             kv_c=z(T, 512, dtype=BF), k_pe=z(T, 64, dtype=BF), slots=z(T, dtype=torch.int64) - 1,
             pool=z(20, 656, dtype=torch.uint8), positions=z(1, T), rope=binding.rope_spec(), err_flag=z(1))
    return binding.dsa_rope_qkv656(**{**a, **kw})


def attn(**kw):
    a = dict(q_bf16=z(T, H, 576, dtype=BF), pool=z(20, 656, dtype=torch.uint8), layout="rope656", page_table=z(B, W),
             page_size=PAGE, cu_q=z(B + 1), kv_lens=z(B), sm_scale=1.0, o=z(T, H, 512, dtype=BF),
             lse=z(T, H, dtype=torch.float32), workspace=binding.chunk_workspace_for(T, H, B, "rope656"), err_flag=z(1))
    return binding.dsa_chunk_attn(**{**a, **kw})


ARGS = {
    extend: ["seq_lens", "new_lens", "page_table", "free_pages", "free_count", "free_count_out", "slots", "positions",
             "token_seq", "cu_q", "kv_lens", "err_flag"],
    release: ["finished", "seq_lens", "page_table", "free_pages", "free_count", "free_count_out", "seq_lens_out", "err_flag"],
    rope: ["q_nope", "q_pe", "q_out", "kv_c", "k_pe", "slots", "pool", "positions", "err_flag"],
    attn: ["q_bf16", "pool", "page_table", "cu_q", "kv_lens", "o", "lse", "workspace", "err_flag"],
}
CASES = [(f, n) for f, names in ARGS.items() for n in names]


def good(f, name):
    """The tensor that f passes for an argument."""
    caught = {}
    real = {"dsa_pages_extend": binding.dsa_pages_extend, "dsa_pages_release": binding.dsa_pages_release,
            "dsa_rope_qkv656": binding.dsa_rope_qkv656, "dsa_chunk_attn": binding.dsa_chunk_attn}
    try:
        for n in real:
            setattr(binding, n, lambda **kw: caught.update(kw))
        f()
    finally:
        for n, fn in real.items():
            setattr(binding, n, fn)
    return caught[name]


@pytest.mark.parametrize("f", list(ARGS), ids=lambda f: f.__name__)
def test_good_arguments(f):
    f()
    torch.cuda.synchronize()


@pytest.mark.parametrize("f,name", CASES, ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_wrong_type(f, name):
    t = good(f, name)
    with pytest.raises((TypeError, ValueError)):
        f(**{name: t.double() if t.dtype != torch.float64 else t.float()})
    with pytest.raises((TypeError, ValueError)):
        f(**{name: t.cpu()})
    with pytest.raises((TypeError, ValueError)):
        f(**{name: t.cpu().view(torch.uint8).numpy() if t.dtype == BF else t.cpu().numpy()})
    with pytest.raises((TypeError, ValueError)):
        f(**{name: [0]})


@pytest.mark.parametrize("f,name", [c for c in CASES if c[1] not in ("err_flag", "workspace")],
                         ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_wrong_shape(f, name):
    t = good(f, name)
    with pytest.raises((TypeError, ValueError, binding.DsaError)):
        f(**{name: t[None]})
    if name not in ("free_pages", "pool"):                       # their length is theirs to choose
        with pytest.raises((TypeError, ValueError, binding.DsaError)):
            f(**{name: torch.cat([t, t])})
    wide = torch.stack([t, t], -1)[..., 0]                       # every second element
    if wide.numel() > 1:
        with pytest.raises((TypeError, ValueError, binding.DsaError)):
            f(**{name: wide})


@pytest.mark.parametrize("f", [extend, release, attn], ids=lambda f: f.__name__)
@pytest.mark.parametrize("page_size", [0, -1, 2 ** 31 - 1])
def test_wrong_page_size(f, page_size):
    with pytest.raises(binding.DsaError):
        f(page_size=page_size)


def test_unknown_layout_and_short_workspace():
    with pytest.raises(ctypes.ArgumentError):                    # as the other entry points do
        attn(layout="rows")
    with pytest.raises((TypeError, ValueError, binding.DsaError)):
        attn(layout="raw512")
    with pytest.raises(binding.DsaError):
        attn(workspace=binding.chunk_workspace_for(T, H, B, "rope656")[:-1].clone())
