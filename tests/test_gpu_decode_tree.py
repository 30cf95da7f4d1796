"""kda_decode_tree: each node one decode step from its parent's state, against
the float64 oracle's decode step applied node by node."""
import numpy as np
import pytest
import torch

import oracle
from tests._parity import TOL, assert_close, compare_out, to64
from tests._tree import lineage, random_trees
from tests.test_gpu_decode_multi import multi_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_05_gb300 as m
    m.build()
    m.lib()
    return m


def reference(q, k, v, g, b, S, parent):
    q, k, v, g, b, S = (to64(x) for x in (q, k, v, g, b, S))
    N, Ts = parent.shape
    o = np.zeros(v.shape)
    states = np.zeros((N, Ts) + S.shape[1:])
    for n in range(N):
        for t in range(Ts):
            if lineage(parent[n], t) is None:
                continue
            p = parent[n, t]
            before = S[n] if p < 0 else states[n, p]
            one = lambda x: x[n, t][None]
            o[n, t], states[n, t] = (x[0] for x in oracle.decode_step(
                one(q), one(k), one(v), one(g), one(b), before[None]))
    return o, states


def run(kda, x, parent, **kw):
    q, k, v, g, b, S = (t.cuda() for t in x)
    states = torch.full(v.shape + (v.shape[-1],), 7.0, device="cuda")
    o, st = kda.kda_decode_tree(q, k, v, g, b, S, torch.from_numpy(parent).cuda(), states=states, **kw)
    torch.cuda.synchronize()
    assert st is states
    return o, st


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,Ts,H", [(5, 7, 3), (2, 24, 1), (1, 1, 2)])
def test_matches_oracle(kda, d, dtype, N, Ts, H):
    _, *x = multi_inputs(N, Ts, H, d, dtype, 900 + d)
    parent = random_trees(N, Ts, np.random.default_rng(d + Ts))
    o, st = run(kda, x, parent)
    o_ref, st_ref = reference(*x, parent)
    compare_out(o, o_ref, TOL[dtype], "o")
    used = np.array([[lineage(p, t) is not None for t in range(Ts)] for p in parent])
    assert_close(to64(st)[used], st_ref[used], TOL[dtype], "states")
    assert torch.all(st[~torch.from_numpy(used).cuda()] == 7.0), "an unused node's state was written"
    assert torch.all(o[~torch.from_numpy(used).cuda()] == 0)


@pytest.mark.parametrize("d", [64, 128])
def test_a_chain_is_decode_multi_bit_for_bit(kda, d):
    N, Ts, H = 3, 6, 2
    _, *x = multi_inputs(N, Ts, H, d, "bf16", 950)
    q, k, v, g, b, S = (t.cuda() for t in x)
    o, st = kda.kda_decode_multi(q, k, v, g, b, S)
    parent = np.tile(np.arange(-1, Ts - 1, dtype=np.int32), (N, 1))
    o2, st2 = run(kda, x, parent)
    assert torch.equal(o, o2) and torch.equal(st, st2)
    o3, st3 = kda.kda_decode_tree(q, k, v, g, b, S)      # no parent: a chain
    assert torch.equal(o, o3) and torch.equal(st, st3)


def test_every_node_on_the_context(kda):
    # a star: each node's state is one decode step from S_in, the same bits
    N, Ts, H, d = 2, 9, 2, 128
    _, *x = multi_inputs(N, Ts, H, d, "bf16", 960)
    o, st = run(kda, x, np.full((N, Ts), -1, np.int32))
    q, k, v, g, b, S = (t.cuda() for t in x)
    for t in range(Ts):
        one = S.clone()
        ot = kda.kda_decode_step(*(y[:, t].contiguous() for y in (q, k, v, g, b)), one)
        assert torch.equal(ot, o[:, t]) and torch.equal(one, st[:, t])


def test_invalid_parents_make_unused_nodes(kda):
    N, Ts, H, d = 1, 6, 1, 64
    _, *x = multi_inputs(N, Ts, H, d, "fp32", 970)
    parent = np.array([[-1, 1, 1, 0, 9, -7]], np.int32)
    x[1][0, 1] = float("nan")
    o, st = run(kda, x, parent)
    o_ref, st_ref = reference(*x, parent)
    assert_close(to64(o), o_ref, TOL["fp32"], "o")
    assert_close(to64(st)[:, [0, 3]], st_ref[:, [0, 3]], TOL["fp32"], "states")
    assert torch.all(st[0, [1, 2, 4, 5]] == 7.0)


def test_sixty_four_nodes_fp32_out(kda):
    N, Ts, H, d = 1, 64, 2, 128
    _, *x = multi_inputs(N, Ts, H, d, "bf16", 980)
    parent = random_trees(N, Ts, np.random.default_rng(3), unused=False)
    o, st = run(kda, x, parent, o_dtype=torch.float32)
    o_ref, st_ref = reference(*x, parent)
    assert_close(to64(o), o_ref, TOL["bf16"], "o")
    assert_close(to64(st), st_ref, TOL["bf16"], "states")


def test_gather_of_an_accepted_node(kda):
    # kda_state_gather takes node + 1 as the accepted count
    N, Ts, H, d = 3, 5, 2, 64
    _, *x = multi_inputs(N, Ts, H, d, "bf16", 990)
    parent = random_trees(N, Ts, np.random.default_rng(4), unused=False)
    _, st = run(kda, x, parent)
    node = torch.tensor([4, -1, 2], dtype=torch.int32, device="cuda")
    S = x[5].cuda()
    out = kda.kda_state_gather(st, S, node + 1)
    assert torch.equal(out[0], st[0, 4]) and torch.equal(out[1], S[1]) and torch.equal(out[2], st[2, 2])


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_sequences(kda, d, dtype):
    # more (sequence, head) pairs than SMs
    N, Ts, H = 170, 9, 2
    _, *x = multi_inputs(N, Ts, H, d, dtype, 1000 + d)
    parent = random_trees(N, Ts, np.random.default_rng(d))
    o, st = run(kda, x, parent)
    few = [0, 1, 76, 151, 152, 169]
    o_ref, st_ref = reference(*(y[few] for y in x), parent[few])
    compare_out(o[few], o_ref, TOL[dtype], "o")
    used = np.array([[lineage(p, t) is not None for t in range(Ts)] for p in parent])
    assert_close(to64(st[few])[used[few]], st_ref[used[few]], TOL[dtype], "states")
    assert torch.all(st[~torch.from_numpy(used).cuda()] == 7.0), "an unused node's state was written"
    assert torch.all(o[~torch.from_numpy(used).cuda()] == 0)


@pytest.mark.parametrize("d", [64, 128])
def test_many_chains_are_decode_multi_bit_for_bit(kda, d):
    N, Ts, H = 90, 6, 2
    _, *x = multi_inputs(N, Ts, H, d, "bf16", 1010)
    q, k, v, g, b, S = (t.cuda() for t in x)
    o, st = kda.kda_decode_multi(q, k, v, g, b, S)
    o2, st2 = kda.kda_decode_tree(q, k, v, g, b, S)
    assert torch.equal(o, o2) and torch.equal(st, st2)


@pytest.mark.parametrize("N,H", [(1, 2), (80, 2)])
@pytest.mark.parametrize("kind", ["comb", "binary", "star of stars"])
def test_many_states_with_children_to_come(kda, kind, N, H):
    # more open states than the kernel holds on chip at once
    Ts, d = 63, 128
    t = np.arange(Ts)
    parent = {"comb": np.where(t < 32, t - 1, t - 32), "binary": (t + 1) // 2 - 1,
              "star of stars": np.where(t < 8, -1, (t - 8) % 8)}[kind].astype(np.int32)
    parent = np.tile(parent, (N, 1))
    _, *x = multi_inputs(N, Ts, H, d, "bf16", 1020)
    o, st = run(kda, x, parent)
    few = [0, N - 1]
    o_ref, st_ref = reference(*(y[few] for y in x), parent[few])
    compare_out(o[few], o_ref, TOL["bf16"], "o")
    assert_close(to64(st[few]), st_ref, TOL["bf16"], "states")
