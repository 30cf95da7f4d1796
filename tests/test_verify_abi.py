"""Argument checks of the calls that verify a tree of drafted tokens: each bad
call returns its status before anything is launched (no GPU needed)."""
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_05_gb300 as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000            # a fake, aligned address: never dereferenced
NULL = None
BAD, UNSUPPORTED, WORKSPACE = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    kda.build()
    return kda.lib()


def attention(lib, **kw):
    args = dict(q=A, k=A * 2, v=A * 3, parent=NULL, kc=A * 256, vc=A * 512, table=A * 4, lengths=A * 5,
                N=2, Ts=4, Hq=8, Hkv=2, d=128, pages=16, page=16, most=8, stride=16 * 2 * 128,
                dt=kda.KDA_BF16, scale=0.1, o=A * 6, ws=A * 1024, wsb=1 << 40, stream=NULL)
    args.update(kw)
    return lib.kda_tree_attention(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(Ts=65), UNSUPPORTED),
    (dict(N=0), BAD), (dict(Ts=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=7), BAD), (dict(Hq=1), BAD),
    (dict(page=0), BAD), (dict(pages=-1), BAD), (dict(most=-1), BAD), (dict(most=1 << 28), BAD),
    (dict(q=NULL), BAD), (dict(k=NULL), BAD), (dict(lengths=NULL), BAD), (dict(o=NULL), BAD),
    (dict(kc=NULL), BAD), (dict(table=NULL), BAD), (dict(q=A + 2), BAD), (dict(vc=A * 512 + 8), BAD),
    (dict(parent=A + 2), BAD), (dict(stride=16 * 2 * 128 - 8), BAD), (dict(stride=16 * 2 * 128 + 4), BAD),
    (dict(o=A), BAD), (dict(o=A * 256 + 1024), BAD),
    (dict(ws=NULL), WORKSPACE), (dict(wsb=64), WORKSPACE), (dict(ws=A * 1024 + 16), WORKSPACE),
])
def test_attention_rejects(lib, kw, code):
    assert attention(lib, **kw) == code


@pytest.mark.parametrize("args", [(0, 4, 8, 2, 128, 0), (2, 0, 8, 2, 128, 0), (2, 65, 8, 2, 128, 0),
                                  (2, 4, 7, 2, 128, 0), (2, 4, 8, 2, 96, 0), (2, 4, 8, 2, 128, 5)])
def test_attention_workspace_of_bad_arguments(lib, args):
    assert lib.kda_tree_attention_workspace_bytes(*args) == 0


def test_attention_workspace_does_not_grow_with_the_batch(lib):
    size = kda.kda_tree_attention_workspace_bytes
    assert size(1, 16, 32, 8, 128, kda.KDA_BF16) == size(1000, 16, 32, 8, 128, kda.KDA_BF16) > 256


def tree(lib, **kw):
    args = dict(q=A, k=A, v=A, g=A, b=A, S=A * 16, parent=A, N=2, Ts=3, H=2, dk=64, dv=64,
                dt=kda.KDA_BF16, o=A * 2, states=A * 64, stream=NULL)
    args.update(kw)
    return lib.kda_decode_tree(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dk=96, dv=96), UNSUPPORTED), (dict(dv=128), UNSUPPORTED), (dict(dt=3), UNSUPPORTED),
    (dict(Ts=65), UNSUPPORTED), (dict(N=0), BAD), (dict(Ts=0), BAD), (dict(H=0), BAD),
    (dict(S=NULL), BAD), (dict(states=NULL), BAD), (dict(v=A + 8), BAD), (dict(parent=A + 1), BAD),
    (dict(states=A * 16), BAD), (dict(o=A * 64), BAD), (dict(o=A * 16), BAD),
    (dict(parent=NULL, N=0), BAD),
])
def test_decode_tree_rejects(lib, kw, code):
    assert tree(lib, **kw) == code


def logprobs(lib, **kw):
    args = dict(x=A, stride=1000, tok=A * 2, T=3, V=1000, J=2, K=4, dt=kda.KDA_FP32, lp=A * 3,
                H=A * 4, ids=A * 5, top=A * 6, stream=NULL)
    args.update(kw)
    return lib.kda_token_logprobs(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dt=kda.KDA_BF16), UNSUPPORTED), (dict(K=33), UNSUPPORTED), (dict(T=0), BAD), (dict(V=0), BAD),
    (dict(J=-1), BAD), (dict(K=-1), BAD), (dict(V=3, stride=3), BAD), (dict(stride=999), BAD),
    (dict(x=NULL), BAD), (dict(tok=NULL), BAD), (dict(lp=NULL), BAD), (dict(ids=NULL), BAD),
    (dict(top=NULL), BAD), (dict(x=A + 4), BAD), (dict(H=A + 2), BAD),
    (dict(J=0, K=0, H=NULL), BAD),
])
def test_logprobs_rejects(lib, kw, code):
    assert logprobs(lib, **kw) == code


def commit(lib, **kw):
    args = dict(k=A, v=A * 2, path=NULL, count=NULL, table=A * 3, lengths=A * 4, layers=2, N=2, Ts=4,
                Hkv=2, d=64, pages=8, page=16, most=4, stride=2048, layer=2048 * 8, dt=kda.KDA_BF16,
                kc=A * 64, vc=A * 128, new=A * 5, stream=NULL)
    args.update(kw)
    return lib.kda_cache_commit(*args.values())


def append(lib, **kw):
    args = dict(k=A, v=A * 2, cu=A * 6, T=10, table=A * 3, lengths=A * 4, layers=2, N=2, Hkv=2, d=64,
                pages=8, page=16, most=4, stride=2048, layer=2048 * 8, dt=kda.KDA_BF16, kc=A * 64,
                vc=A * 128, new=A * 5, stream=NULL)
    args.update(kw)
    return lib.kda_cache_append(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(d=48), UNSUPPORTED), (dict(dt=4), UNSUPPORTED), (dict(layers=0), BAD), (dict(N=0), BAD),
    (dict(Hkv=0), BAD), (dict(pages=0), BAD), (dict(page=0), BAD), (dict(most=0), BAD),
    (dict(k=NULL), BAD), (dict(kc=NULL), BAD), (dict(table=NULL), BAD), (dict(lengths=NULL), BAD),
    (dict(k=A + 8), BAD), (dict(vc=A * 128 + 4), BAD), (dict(stride=2047), BAD), (dict(stride=2052), BAD),
    (dict(layer=2047), BAD), (dict(layer=2048 * 8 + 4), BAD), (dict(k=A * 64), BAD), (dict(v=A * 128), BAD),
    (dict(new=A * 4), BAD), (dict(new=A * 4 + 4), BAD), (dict(new=A * 5 + 2), BAD),
])
def test_cache_calls_reject(lib, kw, code):
    assert commit(lib, **kw) == code
    assert append(lib, **kw) == code


def test_cache_calls_reject_their_own(lib):
    assert commit(lib, Ts=0) == BAD
    assert commit(lib, path=A + 2) == BAD
    assert append(lib, cu=NULL) == BAD
    assert append(lib, T=-1) == BAD
    assert append(lib, T=1 << 31) == BAD


@pytest.mark.parametrize("at", [A * 7, A * 7 + 4, A * 7 - 4])
def test_cache_calls_reject_new_lengths_over_what_they_read(lib, at):
    # N = 2: new_lengths is 8 bytes, and so is count
    assert commit(lib, count=A * 7, new=at) == BAD
    assert commit(lib, path=A * 7, new=at) == BAD
    assert commit(lib, table=A * 7, new=at) == BAD
    assert append(lib, cu=A * 7, new=at) == BAD
    assert append(lib, table=A * 7, new=at) == BAD


@pytest.mark.parametrize("out", ["o", "states"])
@pytest.mark.parametrize("over,size", [("q", 1536), ("k", 1536), ("v", 1536), ("g", 3072), ("b", 48), ("parent", 24)])
def test_decode_tree_rejects_results_over_what_it_reads(lib, out, over, size):
    # N = 2, Ts = 3, H = 2, d = 64, bf16; the last 16-byte piece that lies in the input
    for parent in (A * 9, NULL):
        apart = dict(q=A, k=A * 3, v=A * 4, g=A * 5, b=A * 6, parent=parent)
        if apart[over] is not None:
            for at in (apart[over], apart[over] + (size - 1) // 16 * 16):
                assert tree(lib, **{**apart, out: at}) == BAD


@pytest.mark.parametrize("args", [(1, 64, 1 << 30, 1, 128, 0), (1, 64, 1 << 25, 1, 64, 2), (1, 64, (1 << 14) + 1, 1, 128, 1),
                                  (1, 1, (1 << 20) + 1, 1, 128, 0), (1, 1, 1 << 24, 1 << 24, 128, 0)])
def test_attention_workspace_of_sizes_that_the_call_refuses(args):
    # in a process of its own: an arithmetic exception would end this one
    code = "import gated_delta_rule_05_gb300 as k; print(k.kda_tree_attention_workspace_bytes(*%r))" % (args,)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert out.returncode == 0 and out.stdout.strip() == "0", out
    N, Ts, Hq, Hkv, d, dt = args
    assert attention(kda.lib(), N=N, Ts=Ts, Hq=Hq, Hkv=Hkv, d=d, dt=dt) == BAD


def test_attention_workspace_of_the_widest_call(lib):
    assert kda.kda_tree_attention_workspace_bytes(1, 64, 1 << 14, 1, 128, kda.KDA_BF16) > 256


def _calls():
    """Each wrapper with the tensors whose gradients it would drop (on the CPU, where
    they are refused too, for being there)."""
    f, i = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32)
    x, c = f(1, 2, 1, 16), f(3, 4, 1, 16)
    pool = [f(1, 3, 4, 1, 16), f(1, 3, 4, 1, 16)]
    return {
        "kda_decode_tree": ([x, x, x, x, f(1, 2, 1), f(1, 1, 16, 16)], [i(1, 2)]),
        "kda_tree_attention": ([x, x, x, c, c], [i(1, 3), i(1), i(1, 2)]),
        "kda_token_logprobs": ([f(2, 8)], [i(2, 1)]),
        "kda_cache_commit": ([x[None], x[None]], [i(1, 2), i(1)] + pool + [i(1, 3), i(1)]),
        "kda_cache_append": ([x, x], [i(2)] + pool + [i(1, 3), i(1)]),
    }


@pytest.mark.parametrize("name,at", [(n, k) for n, (x, _) in _calls().items() for k in range(len(x))])
def test_gradients_are_refused_not_dropped(name, at):
    call, (floats, rest) = getattr(kda, name), _calls()[name]
    floats = [t.clone().requires_grad_(k == at) for k, t in enumerate(floats)]
    with pytest.raises(RuntimeError, match=name + " has no backward pass"):
        call(*floats, *rest)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
        call(*floats, *rest)
