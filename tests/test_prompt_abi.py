"""Argument checks of the calls that take a prompt and its answer through the softmax
layers: each bad call returns its status before anything is launched (no GPU
needed)."""
import pytest
import torch

import gated_delta_rule_05_gb300 as kda

A = 0x10000            # a fake, aligned address: never dereferenced
NULL = None
BAD, UNSUPPORTED, WORKSPACE = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
BF16, F32 = kda.KDA_BF16, kda.KDA_FP32


@pytest.fixture(scope="module")
def lib():
    kda.build()
    return kda.lib()


def prompt(lib, **kw):
    args = dict(q=A, k=A * 16, v=A * 32, qs=512, ks=128, vs=128, cu=A * 64, cuk=NULL, N=2, T=10, Tk=10, Hq=8, Hkv=2,
                d=64, dt=BF16, scale=0.1, o=A * 65, ws=A * 256, wsb=256, stream=NULL)
    args.update(kw)
    return lib.kda_prompt_attention(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(N=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=7), BAD),
    (dict(Hq=1), BAD), (dict(Hq=0), BAD), (dict(T=-1), BAD), (dict(Tk=-1), BAD), (dict(T=1 << 31, Tk=1 << 31), BAD),
    (dict(Tk=11), BAD), (dict(cu=NULL), BAD), (dict(cu=NULL, cuk=A, N=1), BAD), (dict(q=NULL), BAD),
    (dict(k=NULL), BAD), (dict(v=NULL), BAD), (dict(o=NULL), BAD), (dict(q=A + 8), BAD), (dict(v=A * 32 + 2), BAD),
    (dict(o=A * 65 + 8), BAD), (dict(cu=A * 64 + 2), BAD), (dict(qs=511), BAD),
    (dict(qs=516), BAD), (dict(ks=120), BAD), (dict(vs=-128), BAD), (dict(qs=1 << 60), BAD), (dict(o=A), BAD), (dict(o=A * 16 + 1024), BAD),
    (dict(o=A * 64 - 16), BAD), (dict(Hkv=1 << 17, Hq=1 << 17, ks=1 << 23, vs=1 << 23, qs=1 << 23), BAD),
    (dict(Hq=1 << 20, Hkv=1, qs=1 << 26), BAD),
    (dict(ws=NULL), WORKSPACE), (dict(wsb=255), WORKSPACE), (dict(ws=A * 256 + 128), WORKSPACE),
    (dict(ws=A * 65), BAD), (dict(ws=A * 32), BAD), (dict(ws=A + 256), BAD),
])
def test_prompt_attention_rejects(lib, kw, code):
    assert prompt(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(cu=A * 256), dict(cu=A * 256 + 252), dict(cu=A * 256 - 8), dict(cuk=A * 256 + 64), dict(cuk=A * 256 - 4)])
def test_prompt_attention_rejects_a_workspace_over_its_offsets(lib, kw):
    assert prompt(lib, **kw) == BAD


def test_prompt_attention_workspace(lib):
    size = kda.kda_prompt_attention_workspace_bytes
    for bad in ((0, 8, 2, 64, BF16), (2, 7, 2, 64, BF16), (2, 8, 2, 48, BF16), (2, 8, 2, 64, 5), (1, 1 << 17, 1 << 17, 16, BF16)):
        assert size(*bad) == 0
    assert size(1, 8, 2, 64, BF16) == 256


def test_prompt_attention_of_no_rows_is_nothing_to_do(lib):
    assert prompt(lib, T=0, Tk=0, q=NULL, k=NULL, v=NULL, o=NULL) == kda.KDA_OK


def append(lib, **kw):
    # a page of 16 rows of 2 heads of 64 channels in 8 bits: 2048 bytes
    args = dict(q=A, k=A * 2, v=A * 3, qs=512, ks=128, vs=128, cu=A * 4, T=10, f=A * 5, rot=64, inter=0, table=A * 6,
                lengths=A * 7, N=2, Hq=8, Hkv=2, d=64, pages=8, page=16, most=4, stride=2048, block=8, dt=BF16,
                qo=A * 8, qos=512, ko=A * 9, kos=128, kc=A * 64, vc=A * 128, kss=A * 10, vss=A * 11, new=A * 12,
                stream=NULL)
    args.update(kw)
    return lib.kda_cache_append_rotary(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(d=48), UNSUPPORTED), (dict(block=129), UNSUPPORTED), (dict(N=0), BAD),
    (dict(Hkv=0), BAD), (dict(Hq=-2), BAD), (dict(Hq=3), BAD), (dict(T=-1), BAD), (dict(T=1 << 31), BAD),
    (dict(rot=0), BAD), (dict(rot=8), BAD), (dict(rot=80), BAD), (dict(rot=24), BAD), (dict(f=NULL), BAD),
    (dict(pages=0), BAD), (dict(page=0), BAD), (dict(most=0), BAD), (dict(most=1 << 28), BAD), (dict(block=-1), BAD),
    (dict(block=5), BAD), (dict(cu=NULL), BAD), (dict(lengths=NULL), BAD), (dict(table=NULL), BAD), (dict(kc=NULL), BAD),
    (dict(vc=NULL), BAD), (dict(kss=NULL), BAD), (dict(vss=NULL), BAD), (dict(k=NULL), BAD), (dict(v=NULL), BAD),
    (dict(q=NULL), BAD), (dict(qo=NULL), BAD), (dict(Hq=0), BAD), (dict(k=A * 2 + 8), BAD), (dict(kc=A * 64 + 8), BAD),
    (dict(qo=A * 8 + 4), BAD), (dict(new=A * 12 + 2), BAD), (dict(kss=A * 10 + 1), BAD), (dict(qs=508), BAD),
    (dict(ks=132), BAD), (dict(qos=511), BAD), (dict(kos=100), BAD), (dict(stride=2047), BAD), (dict(stride=2056), BAD),
    # results over what is read, or over each other
    (dict(qo=A + 16), BAD), (dict(qo=A, qos=1024), BAD), (dict(ko=A * 2 + 256, kos=128), BAD), (dict(qo=A * 3), BAD),
    (dict(ko=A * 8 + 1024), BAD), (dict(kc=A * 3 - 16), BAD), (dict(vc=A * 8), BAD), (dict(kss=A * 9), BAD),
    (dict(vss=A * 10), BAD), (dict(kss=A * 64 + 4096), BAD), (dict(new=A * 7 + 4), BAD), (dict(new=A * 4 + 8), BAD),
    (dict(new=A * 6 + 28), BAD), (dict(new=A * 5 + 124), BAD), (dict(new=A * 2), BAD), (dict(qo=A * 7 - 512), BAD),
    (dict(new=A * 11), BAD),
])
def test_append_rejects(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_rejects_rows_that_meet_within_one_projection(lib):
    # q, k, v beside each other in rows of 768 elements
    fused = dict(qs=768, ks=768, vs=768, qos=768, kos=768, q=A, k=A + 1024, v=A + 1280)
    assert append(lib, **fused, qo=A + 16, ko=A + 1024) == BAD
    assert append(lib, **fused, qo=A, ko=A + 1280) == BAD
    assert append(lib, **fused, qo=A + 512, ko=A + 1024) == BAD


def attention(lib, **kw):
    args = dict(q=A, kc=A * 64, vc=A * 128, ks=A * 2, vs=A * 3, table=A * 4, lengths=A * 5, N=2, Ts=1, Hq=8, Hkv=2,
                d=64, pages=8, page=16, most=4, stride=2048, block=8, dt=BF16, scale=0.1, o=A * 6, ws=A * 256,
                wsb=1 << 30, stream=NULL)
    args.update(kw)
    return lib.kda_cache_attention_e4m3(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(d=48), UNSUPPORTED), (dict(page=1 << 17, block=1 << 10, stride=1 << 24), UNSUPPORTED),
    (dict(N=0), BAD), (dict(Ts=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=3), BAD), (dict(Ts=1 << 18), BAD),
    (dict(pages=0), BAD), (dict(page=0), BAD), (dict(most=0), BAD), (dict(most=1 << 27), BAD), (dict(block=0), BAD),
    (dict(block=3), BAD), (dict(q=NULL), BAD), (dict(kc=NULL), BAD), (dict(vc=NULL), BAD), (dict(ks=NULL), BAD),
    (dict(vs=NULL), BAD), (dict(table=NULL), BAD), (dict(lengths=NULL), BAD), (dict(o=NULL), BAD),
    (dict(q=A + 2), BAD), (dict(vc=A * 128 + 8), BAD), (dict(ks=A * 2 + 2), BAD), (dict(stride=2040), BAD),
    (dict(stride=2056), BAD), (dict(o=A), BAD), (dict(o=A * 64 + 1024), BAD), (dict(o=A * 3), BAD), (dict(o=A * 5), BAD),
    (dict(ws=A * 128), BAD), (dict(ws=A * 6), BAD),
    (dict(ws=NULL), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(ws=A * 256 + 16), WORKSPACE),
])
def test_attention_rejects(lib, kw, code):
    assert attention(lib, **kw) == code


def test_attention_workspace(lib):
    size = kda.kda_cache_attention_e4m3_workspace_bytes
    for bad in ((0, 1, 8, 2, 64, BF16), (2, 0, 8, 2, 64, BF16), (2, 1, 7, 2, 64, BF16), (2, 1, 8, 2, 48, BF16),
                (2, 1, 8, 2, 64, 5), (1, 1 << 20, 1 << 10, 1, 64, BF16), (1, 1, 1 << 30, 1, 64, BF16)):
        assert size(*bad) == 0
    assert size(1, 4, 32, 8, 128, BF16) == size(1000, 4, 32, 8, 128, BF16) > 0


def _calls():
    """Each wrapper with the tensors whose gradients it would drop (on the CPU, where they
    are refused too, for being there)."""
    f, i = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32)
    x, c = f(2, 1, 16), f(3, 4, 1, 16)
    return {
        "kda_prompt_attention": ([x, x, x], []),
        "kda_cache_append_rotary": ([x, x, x], [i(2), f(8), c, c, i(1, 3), i(1)]),
        "kda_cache_attention_e4m3": ([f(1, 1, 1, 16)], [c.to(torch.float8_e4m3fn)] * 2 + [f(3, 1, 1)] * 2 + [i(1, 3), i(1)]),
    }


@pytest.mark.parametrize("name,at", [(n, k) for n, (x, _) in _calls().items() for k in range(len(x))])
def test_gradients_are_refused_not_dropped(name, at):
    call, (floats, rest) = getattr(kda, name), _calls()[name]
    floats = [t.clone().requires_grad_(k == at) for k, t in enumerate(floats)]
    with pytest.raises(RuntimeError, match=name + " has no backward pass"):
        call(*floats, *rest)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
        call(*floats, *rest)
