"""kda_tree_attention against a float64 reference.

Bounds, per element, with A = sum_j p_j |v_j|:
  fp32   |err| <= 1e-4 A: a score is a sum of d <= 128 products, off by at most
         d 2^-24 sum |q k| scale (about 128 * 6e-8 * 12 = 9e-5 at these inputs'
         scores), which is p's relative error; the rest is far below.
  bf16   |err| <= 2^-8 |o| + 2^-8 A + 1e-4 A: the rounding of o, and p rounded
         to bf16 (half an ulp, 2^-9, in the sum and in the normaliser) for the
         second product.  fp32 output from bf16 inputs is held to the fp32 bound
         (its probabilities are not rounded).
"""
import numpy as np
import pytest
import torch

from tests._tree import AttentionInputs, attention_reference, lineage

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_05_gb300 as m
    m.build()
    m.lib()
    return m


def check(o, ref, mag, exact_p):
    o64 = o.double().cpu().numpy()
    bound = 1e-4 * mag + (0 if exact_p else 2.0 ** -8 * mag)
    if o.dtype == BF16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(o64 - ref) <= bound)
    assert not bad.any(), "%d of %d elements off, worst %.3g of the bound" % (
        bad.sum(), bad.size, np.nanmax(np.abs(o64 - ref) / np.maximum(bound, 1e-30)))


def run(kda, inp, **kw):
    o = kda.kda_tree_attention(**inp.on("cuda"), **kw)
    torch.cuda.synchronize()
    return o


CASES = [
    # N, Ts, Hq, Hkv, d, page, lengths
    (1, 1, 1, 1, 16, 1, [1]),
    (1, 1, 8, 8, 128, 16, [0]),
    (3, 1, 8, 2, 64, 16, [63, 64, 65]),
    (4, 5, 6, 2, 128, 48, [0, 1, 127, 129]),
    (2, 64, 2, 1, 64, 7, [128, 300]),
    (2, 33, 8, 1, 128, 128, [511, 1025]),
    (5, 9, 15, 3, 32, 100, [77, 0, 256, 255, 31]),
    (1, 64, 16, 2, 128, 64, [700]),
    (1, 3, 4, 1, 128, 64, [9001]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_matches_reference(kda, case, dtype, out):
    inp = AttentionInputs(*case, dtype, seed=sum(case[:6]))
    o = run(kda, inp, o_dtype=out)
    assert o.dtype == out
    check(o, *attention_reference(inp), exact_p=out == F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chain_is_the_parent_of_each_node_before_it(kda, dtype):
    chain = AttentionInputs(2, 6, 4, 2, 64, 32, [90, 5], dtype, seed=5, parent="chain")
    o = run(kda, chain)
    check(o, *attention_reference(chain), exact_p=dtype == F32)
    chain.parent = np.tile(np.arange(-1, 5, dtype=np.int32), (2, 1))
    assert torch.equal(run(kda, chain), o)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_unused_nodes(kda, dtype, d):
    # invalid parents (itself, a later node, below -1) and a node under one
    parent = np.array([[-1, 1, 1, 0, 9, -7], [-2] * 6], np.int32)
    inp = AttentionInputs(2, 6, 4, 2, d, 16, [40, 40], dtype, seed=6, parent=parent)
    for t in (1, 2, 4, 5):                          # garbage in unused rows reaches nobody
        inp.k[0, t], inp.v[0, t], inp.q[0, t] = float("nan"), float("inf"), float("nan")
    inp.k[1], inp.v[1] = float("nan"), float("nan")
    ref, mag = attention_reference(inp)
    o = run(kda, inp)
    check(o, ref, mag, exact_p=dtype == F32)
    assert torch.all(o[0, [1, 2, 4, 5]] == 0) and torch.all(o[1] == 0)


@pytest.mark.parametrize("dtype,d,Ts,G", [(BF16, 128, 8, 2), (BF16, 64, 40, 4), (F32, 32, 8, 1)])
def test_inf_and_nan_reach_only_the_nodes_that_see_them(kda, dtype, d, Ts, G):
    parent = np.array([[-1] + [0] * (Ts - 1)], np.int32)
    inp = AttentionInputs(1, Ts, 2 * G, 2, d, 16, [30], dtype, seed=7, parent=parent)
    inp.v[0, 2, 0, 1], inp.v[0, 3, 1, 0], inp.k[0, 4, 0] = float("inf"), float("nan"), float("nan")
    o = run(kda, inp).double().cpu().numpy()
    ref, mag = attention_reference(inp)
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(o))
    assert (o[0, 2, :G, 1] == np.inf).all() and np.isnan(o[0, 3, G:, 0]).all()
    assert np.isnan(o[0, 4, :G]).all()
    bound = (2.0 ** -7 + 1e-4) * mag
    assert (np.abs(o - ref)[fine] <= bound[fine]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(kda, dtype):
    # scores of some hundreds: the running maximum has to move the sums with it
    inp = AttentionInputs(2, 4, 4, 2, 128, 16, [600, 333], dtype, seed=8)
    inp.q *= 40
    ref, mag = attention_reference(inp)
    o = run(kda, inp).double().cpu().numpy()
    # p's relative error is the score's absolute one: 128 2^-24 * 12 * 40
    assert (np.abs(o - ref) <= (4e-3 + 2.0 ** -7) * mag).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_page_stride_and_pages_that_do_not_exist(kda, dtype):
    inp = AttentionInputs(2, 3, 4, 2, 64, 16, [70, 50], dtype, seed=9, gap=64)
    check(run(kda, inp), *attention_reference(inp), exact_p=dtype == F32)
    inp.table[0, 1], inp.table[1, 0] = -5, inp.shape[0]
    check(run(kda, inp), *attention_reference(inp), exact_p=dtype == F32)


@pytest.mark.parametrize("dtype,scale", [(BF16, -0.11), (BF16, 0.0), (F32, -0.11)])
def test_other_scales(kda, dtype, scale):
    inp = AttentionInputs(2, 5, 4, 2, 64, 16, [200, 31], dtype, seed=16)
    inp.scale = scale
    check(run(kda, inp), *attention_reference(inp), exact_p=dtype == F32)


@pytest.mark.parametrize("Ts,G", [(1, 128), (43, 3), (64, 3), (64, 4), (50, 7), (64, 9)])
@pytest.mark.parametrize("d", [64, 128])
def test_row_tiles_of_the_tensor_core_kernel(kda, Ts, G, d):
    # 128, 129, 192, 256, 350 and 576 query rows per cache head
    inp = AttentionInputs(2, Ts, 2 * G, 2, d, 32, [391, 12], BF16, seed=Ts + G)
    check(run(kda, inp), *attention_reference(inp), exact_p=False)


def test_lengths_are_clamped(kda):
    inp = AttentionInputs(2, 2, 2, 1, 64, 16, [48, 0], BF16, seed=10)
    args = inp.on("cuda")
    args["lengths"] = torch.tensor([1 << 30, -3], dtype=torch.int32, device="cuda")
    o = kda.kda_tree_attention(**args)
    check(o, *attention_reference(inp), exact_p=False)


def test_no_pages_at_all(kda):
    inp = AttentionInputs(2, 5, 4, 4, 128, 16, [0, 0], BF16, seed=11)
    args = inp.on("cuda")
    args["k_cache"], args["v_cache"] = args["k_cache"][:0], args["v_cache"][:0]
    args["page_table"] = args["page_table"][:, :0].contiguous()
    check(kda.kda_tree_attention(**args), *attention_reference(inp), exact_p=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_sequences(kda, dtype):
    # more sequences than threads of a block, most of them short
    rng = np.random.default_rng(12)
    lengths = rng.integers(0, 40, 700)
    lengths[[5, 300, 699]] = [3000, 2000, 1000]
    inp = AttentionInputs(700, 2, 2, 1, 64, 16, lengths, dtype, seed=12)
    check(run(kda, inp), *attention_reference(inp), exact_p=dtype == F32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Ts,G", [(3, 2), (33, 4), (33, 9)])
def test_many_tiles_in_a_range(kda, Ts, G, d):
    # more tiles than CTAs: ranges of several tiles, items and sequences, also
    # where every item is finished in its own CTA
    rng = np.random.default_rng(17)
    for N, lengths in ((2, [22000, 9000]), (160, rng.integers(0, 300, 160))):
        inp = AttentionInputs(N, Ts, 2 * G, 2, d, 64, lengths, BF16, seed=N + G)
        # the reference of a few nodes is enough
        inp.parent[:, 4:] = np.where(np.arange(4, Ts) % 8 == 0, inp.parent[:, 4:], -2)
        check(run(kda, inp), *attention_reference(inp), exact_p=False)


@pytest.mark.parametrize("dtype,d", [(F32, 16), (F32, 32), (F32, 64), (F32, 128), (BF16, 16), (BF16, 128)])
@pytest.mark.parametrize("Ts,G", [(1, 1), (4, 2), (5, 4), (33, 3)])
def test_many_tiles_in_a_range_of_the_fp32_kernels(kda, Ts, G, dtype, d):
    # 1, 8, 20 and 99 query rows per cache head: the stream and the tiles
    rng = np.random.default_rng(18)
    for N, lengths in ((2, [9000, 5001]), (160, rng.integers(0, 300, 160))):
        inp = AttentionInputs(N, Ts, 2 * G, 2, d, 48, lengths, dtype, seed=N + G)
        inp.parent[:, 5:] = np.where(np.arange(5, Ts) % 8 == 0, inp.parent[:, 5:], -2)
        check(run(kda, inp, o_dtype=F32), *attention_reference(inp), exact_p=True)


@pytest.mark.parametrize("page", [1, 7, 24, 40, 96, 1000])
@pytest.mark.parametrize("Ts,G", [(5, 4), (40, 4)])
def test_page_sizes_over_full_tiles(kda, page, Ts, G):
    # pages that end inside a tile, and inside the boxes of a bulk copy
    inp = AttentionInputs(3, Ts, 2 * G, 2, 128, page, [1500, 129, 1024], BF16, seed=page)
    inp.parent[:, 6:] = -2
    check(run(kda, inp), *attention_reference(inp), exact_p=False)


def test_the_cuda_core_kernels_agree(kda, monkeypatch):
    inp = AttentionInputs(3, 12, 8, 2, 128, 64, [1500, 0, 77], BF16, seed=19)
    ref = attention_reference(inp)
    monkeypatch.setenv("KDA_FORCE_SIMT", "1")
    check(run(kda, inp), *ref, exact_p=False)
    monkeypatch.delenv("KDA_FORCE_SIMT")
    check(run(kda, inp), *ref, exact_p=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_same_bits_every_time_and_on_another_stream(kda, dtype):
    inp = AttentionInputs(3, 16, 8, 2, 128, 64, [4000, 17, 900], dtype, seed=13)
    args = inp.on("cuda")
    first = kda.kda_tree_attention(**args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            again = kda.kda_tree_attention(**args)
        s.synchronize()
        assert torch.equal(first, again)


def test_a_workspace_of_the_given_stream(kda):
    # what the call allocates stays its own while the given stream still runs
    inp = AttentionInputs(1, 4, 8, 2, 128, 64, [4000], BF16, seed=20)
    args = inp.on("cuda")
    want = kda.kda_tree_attention(**args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)               # some 10 ms
    o = kda.kda_tree_attention(**args, stream=s)
    need = kda.kda_tree_attention_workspace_bytes(1, 4, 8, 2, 128, kda.KDA_BF16)
    for _ in range(4):
        torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_offsets_beyond_32_bits(kda):
    # a pool of 2^31 + elements each of K and V; only the last pages are used
    d, Hkv, page = 128, 8, 128
    pages = (1 << 31) // (page * Hkv * d) + 40
    inp = AttentionInputs(2, 3, 16, Hkv, d, page, [700, 130], BF16, seed=14, poison=False)
    args = inp.on("cuda")
    P = inp.shape[0]
    for name in ("k_cache", "v_cache"):
        pool = torch.empty((pages, page, Hkv, d), dtype=BF16, device="cuda")
        pool[-P:] = args[name]
        args[name] = pool
    args["page_table"] = torch.where(args["page_table"] >= 0, args["page_table"] + pages - P,
                                     args["page_table"])
    check(kda.kda_tree_attention(**args), *attention_reference(inp), exact_p=False)


def test_in_a_cuda_graph(kda):
    inp = AttentionInputs(2, 4, 8, 2, 128, 32, [500, 60], BF16, seed=15)
    args = inp.on("cuda")
    need = kda.kda_tree_attention_workspace_bytes(2, 4, 8, 2, 128, kda.KDA_BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(args["q"])
    want = kda.kda_tree_attention(**args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_tree_attention(**args, o=o, workspace=ws)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


@pytest.mark.parametrize("d,Ts,G", [(128, 4, 2), (64, 33, 9)])
def test_waits_that_give_up(kda, monkeypatch, d, Ts, G):
    # Through the library's test hook: the copying warps exit at once, and the other
    # warps' waits run out after their usual limit (about two seconds).  The call
    # returns, the timeout word is set and every row that had anything to see is NaN,
    # of items in one block and of items cut between several; the next call on the
    # same workspace is right.  Nothing here traps or waits without a bound.
    inp = AttentionInputs(3, Ts, 2 * G, 2, d, 64, [4000, 17, 900], BF16, seed=21)
    inp.parent[1, Ts - 1] = -2
    args = inp.on("cuda")
    need = kda.kda_tree_attention_workspace_bytes(3, Ts, 2 * G, 2, d, kda.KDA_BF16)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    o = torch.full_like(args["q"], 5.0)
    monkeypatch.setenv("KDA_TEST_STARVE_CONSUMERS", "1")
    kda.kda_tree_attention(**args, o=o, workspace=ws)
    torch.cuda.synchronize()
    monkeypatch.delenv("KDA_TEST_STARVE_CONSUMERS")
    assert ws[8:12].view(torch.int32).item() & 2, "the timeout bit must be set"
    used = torch.tensor([[lineage(p, t) is not None for t in range(Ts)] for p in inp.parent], device="cuda")
    assert not used.all() and torch.isnan(o[used]).all() and torch.all(o[~used] == 0)
    ws[8:12].zero_()
    kda.kda_tree_attention(**args, o=o, workspace=ws)
    check(o, *attention_reference(inp), exact_p=False)
    assert ws[8:12].view(torch.int32).item() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page,Hkv,pages,odd", [(64, 2, 1, 0), (64, 1, 5, 2), (1, 2, 40, 1), (1, 1, 1, 0)])
def test_strides_of_dimensions_of_one_do_not_matter(kda, dtype, page, Hkv, pages, odd):
    lengths = [min(page * pages - 1, 37), 0]
    inp = AttentionInputs(2, 3, 2 * Hkv, Hkv, 64, page, lengths, dtype, seed=22)
    args = inp.on("cuda")
    for name in ("k_cache", "v_cache"):
        t = args[name][inp.table[0, :pages].tolist()].contiguous()
        stride = list(t.stride())
        stride[odd] = 12345
        args[name] = t.as_strided(t.shape, stride)
    table = torch.arange(args["k_cache"].shape[0], dtype=torch.int32)
    args["page_table"] = torch.stack([table, table]).cuda()
    check(kda.kda_tree_attention(**args), *attention_reference(inp), exact_p=dtype == F32)
