"""kda_prompt_attention against a float64 reference.

Bounds, per element, with A = sum_j p_j |v_j|:
  fp32   |err| <= 1e-4 A: a score is a sum of d <= 128 products, off by at most
         d 2^-24 sum |q k| scale (about 128 * 6e-8 * 12 = 9e-5 at these inputs'
         scores), which is p's relative error; the rest is far below.
         Products of fp16 pairs keep 22 bits of q, k, p and v (2^-22 A and less).
  bf16   |err| <= 2^-8 |o| + 2^-8 A + 1e-4 A: the rounding of o, and p rounded to
         bf16 for the second product (half a step, 2^-8, in the sum; the normaliser
         sums the unrounded).  fp32 output from bf16 inputs is held to the fp32
         bound (its probabilities are not rounded).
"""
import numpy as np
import pytest
import torch

from tests._prompt import prompt_reference

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


def inputs(T, Tk, Hq, Hkv, d, dtype, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dtype)
        return [x[:, a:b] for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))], x
    f = lambda t, h: torch.randn((t, h, d), generator=g).to(dtype)
    return [1.5 * f(T, Hq), f(Tk, Hkv), f(Tk, Hkv)], None


def on_gpu(parts, whole):
    if whole is None:
        return [x.cuda() for x in parts]
    y, out, at = whole.cuda(), [], 0
    for x in parts:
        out.append(y[:, at:at + x.shape[1]])
        at += x.shape[1]
    return out


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def check(o, ref, mag, exact_p):
    o64 = o.double().cpu().numpy()
    bound = 1e-4 * mag + (0 if exact_p else 2.0 ** -8 * mag)
    if o.dtype == BF16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(o64 - ref) <= bound)
    assert not bad.any(), "%d of %d elements off, worst %.3g of the bound, first at %s" % (
        bad.sum(), bad.size, np.nanmax(np.abs(o64 - ref) / np.maximum(bound, 1e-30)), np.argwhere(bad)[0])


def run(kda, parts, whole, cu, cu_k, **kw):
    o = kda.kda_prompt_attention(*on_gpu(parts, whole), i32(cu), i32(cu_k), **kw)
    torch.cuda.synchronize()
    return o


def starts(lens):
    return [0] + np.cumsum(lens).tolist()


CASES = [
    # lengths, key lengths (None: the same), Hq, Hkv, d
    ([1], None, 1, 1, 16),
    ([1], None, 8, 2, 128),
    ([127], None, 4, 4, 128),
    ([128], None, 4, 1, 64),
    ([129, 1, 0, 64], None, 6, 2, 128),
    ([300, 5, 257], None, 8, 8, 64),
    ([511], None, 16, 2, 128),
    ([640, 130], None, 5, 1, 128),
    ([70, 33], None, 14, 2, 32),
    ([1000], None, 7, 7, 64),
    ([33, 0, 200], [200, 17, 200], 4, 2, 128),
    ([1, 1, 1], [1, 300, 128], 8, 1, 128),
    ([65, 140], [400, 139], 3, 1, 64),
    ([50, 20, 9], [3, 0, 9], 4, 2, 128),        # queries before the first key
    ([200], None, 48, 2, 64),
    ([400], None, 12, 3, 16),
    ([2100], None, 2, 1, 128),
    ([40], None, 130, 1, 128),                  # more heads than rows of a tile
]


@pytest.mark.parametrize("lens,keys,Hq,Hkv,d", CASES, ids=lambda c: str(c).replace(" ", ""))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_matches_reference(kda, lens, keys, Hq, Hkv, d, dtype, out):
    cu, cu_k = starts(lens), None if keys is None else starts(keys)
    parts, whole = inputs(cu[-1], (cu_k or cu)[-1], Hq, Hkv, d, dtype, seed=sum(lens) + d)
    o = run(kda, parts, whole, cu, cu_k, o_dtype=out)
    assert o.dtype == out
    check(o, *prompt_reference(*parts, cu, cu_k), exact_p=out == F32)


@pytest.mark.parametrize("lens,keys,Hq,Hkv,d", CASES[3:9] + CASES[11:15], ids=lambda c: str(c).replace(" ", ""))
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, F32)])
def test_cuda_cores_match_reference(kda, monkeypatch, lens, keys, Hq, Hkv, d, dtype, out):
    monkeypatch.setenv("KDA_FORCE_SIMT", "1")
    cu, cu_k = starts(lens), None if keys is None else starts(keys)
    parts, whole = inputs(cu[-1], (cu_k or cu)[-1], Hq, Hkv, d, dtype, seed=sum(lens) + d)
    check(run(kda, parts, whole, cu, cu_k, o_dtype=out), *prompt_reference(*parts, cu, cu_k), exact_p=True)


@pytest.mark.parametrize("spread", [1e-25, 1e25, "rows"])
def test_magnitudes_far_apart(kda, spread):
    # keys and values of very different magnitudes from row to row, queries of the opposite
    (q, k, v), _ = inputs(150, 150, 4, 2, 64, F32, seed=17)
    if spread == "rows":
        f = 10.0 ** torch.randint(-12, 13, (150, 1, 1), generator=torch.Generator().manual_seed(1)).float()
        v = v * f
    else:
        q, k, v = q / spread, k * spread, v * spread
    o = run(kda, (q, k, v), None, None, None)
    ref, mag = prompt_reference(q, k, v)
    check(o, ref, mag, exact_p=True)


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF16, 128, 4, 2), (BF16, 64, 3, 1), (F32, 64, 4, 4), (BF16, 32, 2, 1)])
def test_views_of_one_projection(kda, dtype, d, Hq, Hkv):
    cu = starts([100, 190])
    parts, whole = inputs(290, 290, Hq, Hkv, d, dtype, seed=3, fused=True)
    check(run(kda, parts, whole, cu, None), *prompt_reference(*parts, cu), exact_p=dtype == F32)
    # one sequence without offsets is the same as with them
    a, b = run(kda, parts, whole, None, None), run(kda, parts, whole, [0, 290], None)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d,G", [(BF16, 128, 2), (BF16, 64, 5), (F32, 32, 1)])
def test_inf_and_nan_reach_only_the_queries_that_see_them(kda, dtype, d, G):
    # in the same tile, in the next sequence, in the rows behind the last one
    lens = [150, 60, 40]
    cu = starts(lens)
    parts, _ = inputs(260, 260, 2 * G, 2, d, dtype, seed=7)
    q, k, v = parts
    v[100, 0, 1], v[101, 1, 0], k[120, 0] = float("inf"), float("nan"), float("nan")
    v[150, 1, 2] = float("-inf")
    v[209, 0, 3], v[250:], k[250:] = float("nan"), float("nan"), float("inf")
    q[20, 0] = float("nan")
    keep = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    o = run(kda, parts, None, cu, None, o=keep)
    ref, mag = prompt_reference(*parts, cu, o=torch.full(q.shape, 7.0))
    assert torch.all(o[250:] == 7)
    o64 = o.double().cpu().numpy()
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(o64)), np.argwhere(fine != np.isfinite(o64))[:4]
    # (NaN where p underflows beside an infinity is the reference's 0 * inf)
    assert np.isposinf(o64[100, :G, 1]).all() and np.isnan(o64[120, :G]).all() and np.isneginf(o64[150, G:, 2]).all()
    bound = (2.0 ** -7 + 1e-4) * mag
    assert (np.abs(o64 - ref)[fine] <= bound[fine]).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_rising_scores(kda, dtype, d):
    # maxima that grow along the keys by more than any slack, over many tiles
    T = 700
    q, k, v = inputs(T, T, 2, 1, d, dtype, seed=9)[0]
    k = (torch.linspace(-1, 1, T)[:, None, None] * torch.ones_like(k) * 4).to(dtype)
    q = torch.ones_like(q) * 4
    # scores of 16 d^0.5 * (-1 .. 1): 181 and 128 in the exponent, fp32's rounding of them
    # 2^-24 * 181 * d^0.5 is below the bound of 1e-4
    o = run(kda, [q, k, v], None, None, None)
    ref, mag = prompt_reference(q, k, v)
    check(o, ref, mag * 2, exact_p=dtype == F32)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-3, 2.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales(kda, scale, dtype):
    parts, _ = inputs(200, 200, 4, 2, 64, dtype, seed=11)
    o = run(kda, parts, None, None, None, scale=scale)
    ref, mag = prompt_reference(*parts, scale=scale)
    # the bound's score error grows with the scale: at 2.0 16 times the default's
    check(o, ref, mag * max(1.0, 8 * abs(scale)), exact_p=dtype == F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_sequence_keep_what_they_hold(kda, dtype):
    for cu, cu_k in (([0, 30, 50], None), ([10, 30, 64], None), ([-5, 20, 90], None), ([0, 40, 20], None),
                     ([64, 64, 70], None), ([0, 30, 50], [-3, 40, 200])):
        parts, _ = inputs(64, 64, 4, 2, 64, dtype, seed=12)
        keep = torch.full((64, 4, 64), 3.0, dtype=dtype, device="cuda")
        o = run(kda, parts, None, cu, cu_k, o=keep)
        ref, mag = prompt_reference(*parts, cu, cu_k, o=torch.full((64, 4, 64), 3.0))
        check(o, ref, mag, exact_p=dtype == F32)


def test_many_short_sequences(kda):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 9, 1500).tolist()
    cu = starts(lens)
    parts, _ = inputs(cu[-1], cu[-1], 4, 2, 64, BF16, seed=13)
    check(run(kda, parts, None, cu, None), *prompt_reference(*parts, cu), exact_p=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_other_streams_and_graphs(kda, dtype):
    cu = starts([300, 77])
    (q, k, v), _ = inputs(377, 377, 8, 2, 128, dtype, seed=14)
    a = [x.cuda() for x in (q, k, v)]
    b = [x.flip(0).contiguous() for x in a]
    c = i32(cu)
    want = [kda.kda_prompt_attention(*x, c) for x in (a, b)]
    torch.cuda.synchronize()
    # two at once, each on a stream of its own
    s = [torch.cuda.Stream() for _ in range(2)]
    got = [kda.kda_prompt_attention(*x, c, stream=t) for x, t in zip((a, b), s)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # captured, replayed on other inputs
    hold = [x.clone() for x in a]
    o = torch.empty_like(hold[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_prompt_attention(*hold, c, o=o)
    for x, w in zip((a, b, a), want + want[:1]):
        for y, z in zip(hold, x):
            y.copy_(z)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)


def test_no_rows(kda):
    q, kv = torch.empty((0, 4, 64), dtype=BF16, device="cuda"), torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    assert kda.kda_prompt_attention(q, kv, kv, i32([0, 0])).shape == (0, 4, 64)
    (q, _, _), _ = inputs(5, 5, 4, 2, 64, BF16)
    o = kda.kda_prompt_attention(q.cuda(), kv, kv, i32([0, 5]), i32([0, 0]))
    assert torch.all(o == 0)


def test_kernels_agree(kda, monkeypatch):
    cu = starts([900, 333])
    parts, _ = inputs(1233, 1233, 8, 2, 128, BF16, seed=15)
    tc = run(kda, parts, None, cu, None)
    monkeypatch.setenv("KDA_FORCE_SIMT", "1")
    simt = run(kda, parts, None, cu, None)
    ref, mag = prompt_reference(*parts, cu)
    check(tc, ref, mag, exact_p=False)
    check(simt, ref, mag, exact_p=False)


def test_waits_that_give_up(kda, monkeypatch):
    # the copying warps exit at once: the kernel's waits run out (about 2 s), it returns, sets
    # the workspace's word and marks its rows, and the next call is right
    cu = starts([700, 0, 90, 20])
    parts, _ = inputs(815, 815, 8, 2, 128, BF16, seed=16)
    a, c = on_gpu(parts, None), i32(cu)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    status = ws[8:12].view(torch.int32)
    o = torch.full(a[0].shape, 5.0, dtype=BF16, device="cuda")
    monkeypatch.setenv("KDA_TEST_STARVE_CONSUMERS", "1")
    kda.kda_prompt_attention(*a, c, o=o, workspace=ws)
    torch.cuda.synchronize()
    monkeypatch.delenv("KDA_TEST_STARVE_CONSUMERS")
    assert status.item() & 2
    assert torch.isnan(o[:810]).all() and torch.all(o[810:] == 5)
    status.zero_()
    kda.kda_prompt_attention(*a, c, o=o, workspace=ws)
    ref, mag = prompt_reference(*parts, cu, o=torch.full(a[0].shape, 5.0))
    check(o, ref, mag, exact_p=False)
    assert status.item() == 0


def test_claimed_items_in_graphs_and_on_two_streams(kda):
    # enough items that they are claimed from a counter in the workspace
    cu = starts([2600, 900, 1, 500])
    (q, k, v), _ = inputs(4001, 4001, 16, 8, 64, BF16, seed=18)
    a = [x.cuda() for x in (q, k, v)]
    b = [x.flip(0).contiguous() for x in a]
    c = i32(cu)
    want = [kda.kda_prompt_attention(*x, c) for x in (a, b)]
    ref, mag = prompt_reference(q[:2600], k[:2600], v[:2600])
    check(want[0][:2600], ref, mag, exact_p=False)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [kda.kda_prompt_attention(*x, c, stream=t) for _ in range(4) for x, t in zip((a, b), s)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got))
    hold, o = [x.clone() for x in a], torch.empty_like(a[0])
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[8:12] = 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_prompt_attention(*hold, c, o=o, workspace=ws)
    for x, w in zip((a, b, a), want + want[:1]):
        for y, z in zip(hold, x):
            y.copy_(z)
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 32)])
def test_more_sequences_than_are_held(kda, dtype, d):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 3, 20000).tolist()
    lens[12345] = 400
    cu = starts(lens)
    T = cu[-1]
    parts, _ = inputs(T, T, 2, 1, d, dtype, seed=19)
    o = run(kda, parts, None, cu, None)
    check(o, *prompt_reference(*parts, cu), exact_p=dtype == F32)
    if dtype == BF16:   # a sequence's first token sees itself alone (fp32 values are kept to 22 bits)
        first = [a for a, n in zip(cu, lens) if n > 0]
        assert torch.equal(o[first].cpu(), parts[2][first].expand(-1, 2, -1))


@pytest.mark.parametrize("dtype,simt", [(BF16, False), (F32, False), (F32, True)])
def test_offsets_at_the_ends_of_their_type(kda, monkeypatch, dtype, simt):
    # differences of offsets that do not fit 32 bits
    if simt:
        monkeypatch.setenv("KDA_FORCE_SIMT", "1")
    low, high = -2 ** 31, 2 ** 31 - 1
    for cu, cu_k in (([5, low, 30], None), ([0, 30, low], None), ([low, 20, high], None), ([high, low, high], None),
                     ([0, 30, 50], [high, low, 64]), ([high, low, 40], [7, low, low])):
        parts, _ = inputs(64, 64, 4, 2, 64, dtype, seed=20)
        keep = torch.full((64, 4, 64), 3.0, dtype=dtype, device="cuda")
        o = run(kda, parts, None, cu, cu_k, o=keep)
        ref, mag = prompt_reference(*parts, cu, cu_k, o=torch.full((64, 4, 64), 3.0))
        check(o, ref, mag, exact_p=dtype == F32)


@pytest.mark.parametrize("d", [64, 128])
def test_noted_infinities_outlive_the_next_items(kda, d):
    # long looks at infinities in items of two row tiles, and after those many items of a token, whose own infinities
    # are found meanwhile
    many, few, Lq, Lk = 60, 100, 256, 600
    lens, keys = [Lq] * many + [1] * few, [Lk] * many + [560] * few
    cu, cu_k = starts(lens), starts(keys)
    g = torch.Generator().manual_seed(22)
    f = lambda t: torch.randn((t, 4, d), generator=g).to(BF16)
    q, k, v = f(cu[-1]), f(cu_k[-1]), f(cu_k[-1])
    at = [Lk - 200 + 3 * i for i in range(66)]      # of the long ones' keys
    one = d - 3                                     # and the channel
    wild = v.clone()
    for n in range(many):
        wild[[cu_k[n] + x for x in at], :, one] = float("inf")
        v[[cu_k[n] + x for x in at], :, one] = 0
    for n in range(many, many + few):
        wild[cu_k[n + 1] - 1, :, 0] = float("nan")
        v[cu_k[n + 1] - 1, :, 0] = 0
    o = run(kda, [q, k, wild], None, cu, cu_k)
    ref, mag = prompt_reference(q, k, v, cu, cu_k)
    long = o[:many * Lq].view(many, Lq, 4, d)
    sees = torch.arange(Lq) + Lk - Lq >= at[0]
    assert torch.isposinf(long[:, sees.cuda(), :, one]).all() and torch.isnan(o[many * Lq:, :, 0]).all()
    long[:, sees.cuda(), :, one] = 0
    o[many * Lq:, :, 0] = 0
    ref[:many * Lq].reshape(many, Lq, 4, d)[:, sees.numpy(), :, one] = 0
    ref[many * Lq:, :, 0] = 0
    check(o, ref, mag, exact_p=False)


def test_offsets_of_more_than_one_dimension_are_refused(kda):
    (q, k, v), _ = inputs(30, 30, 4, 2, 64, BF16, seed=23)
    a = on_gpu([q, k, v], None)
    for cu, cu_k in ((i32([[0, 10], [20, 30]]), None), (i32([[0], [30]]), None), (i32([[0, 30]]), i32([[0, 30]]))):
        with pytest.raises(ValueError, match="cu_seqlens"):
            kda.kda_prompt_attention(*a, cu, cu_k)
    with pytest.raises(ValueError, match="cu_seqlens_k"):
        kda.kda_prompt_attention(*a, i32([0, 30]), i32([[0, 30]]))


@pytest.mark.parametrize("dtype,out,d", [(F32, F32, 64), (BF16, F32, 128), (BF16, BF16, 32)])
def test_values_far_above_those_of_the_keys_that_count(kda, dtype, out, d):
    # keys that a row does not see, or sees with a probability of 0, have values of 2^60 and more beside ones of 2^-60
    T = 100
    q, k, v = inputs(T, T, 2, 1, d, dtype, seed=26)[0]
    q, k = torch.full_like(q, d ** 0.5), 0.25 * k
    k[80:] += 128 / d                               # scores some 128 above the others'
    big = torch.zeros(T, 1, 1, dtype=torch.bool)
    big[1:80:2] = True                              # hidden from the rows before, and of probability 0 for the last ones
    v = torch.where(big, v * 2.0 ** 75, v * 2.0 ** -75)
    o = run(kda, (q, k, v), None, None, None, o_dtype=out)
    ref, mag = prompt_reference(q, k, v)
    assert np.abs(ref[80:]).max() < 2.0 ** -70 and np.abs(ref[2:80]).min() > 2.0 ** 50
    check(o[:80], ref[:80], mag[:80], exact_p=out == F32)
    # scores of 128 from d products: 22 bits of each and 8 sums cut off at 2^-23, 128 (2^-22 + 8 2^-23) = 1.5e-4, for
    # two keys that are compared
    check(o[80:], ref[80:], 3 * mag[80:], exact_p=out == F32)


@pytest.mark.parametrize("dtype,out,d", [(F32, F32, 64), (BF16, F32, 64), (F32, F32, 16), (BF16, BF16, 32)])
@pytest.mark.parametrize("gap", [10, 12, 14, 16, 18])
@pytest.mark.parametrize("first", [True, False])
def test_one_key_far_above_many_others(kda, dtype, out, d, gap, first):
    # an attention sink: one key's score lies `gap` above those of 2^15 others, which are all the same, so that
    # errors of their weights add up.  Values of 1 throughout, which the output has to be; then a sink
    # without a value, where the others are all of the output.
    n = 1 << 15
    q = torch.ones((2, 1, d), dtype=dtype)
    k = torch.zeros((n + 2, 1, d), dtype=dtype)
    at = 0 if first else n
    k[at] = gap / d ** 0.5
    v = torch.ones_like(k)
    # The output and, in the thread that has the sink, its divisor are added up in n / 32 steps, each off by half a unit
    # of 2^-23 of a sum between 1 and 2: 2 * 2^10 * 2^-24, always the same way.  The exponentials: 2^-22 each, and
    # 18 log2 e 2^-24 of their argument's rounding.  Scores are exact.
    bound = 2.0 ** -13 + 2.0 ** -20
    # a bf16 output: weights to 11 bits, and the output's rounding
    if out == BF16:
        bound += 2.0 ** -11 + 2.0 ** -8
    for sink in (1.0, 0.0):
        v[at] = sink
        o = run(kda, (q, k, v), None, [0, 2], [0, n + 2], o_dtype=out)
        ref, mag = prompt_reference(q, k, v, [0, 2], [0, n + 2])
        # (with 11 bits and no more, weights below 2^-21 of the largest have fewer: e^-14.6)
        if sink or out == F32 or gap < 14.5:
            assert (np.abs(o.double().cpu().numpy() - ref) <= bound * mag).all()


@pytest.mark.parametrize("dtype,out,d", [(F32, F32, 64), (F32, F32, 128), (BF16, F32, 64), (BF16, F32, 32), (BF16, BF16, 32)])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("power", [118, -118, -124])
def test_magnitudes_near_the_ends_of_fp32(kda, dtype, out, d, which, power):
    # (at 2^-124 a part of the values is subnormal; they are compared as they are)
    q, k, v = inputs(150, 150, 4, 2, d, dtype, seed=24)[0]
    f = 2.0 ** power
    scale = d ** -0.5
    if which != "v":
        scale /= f
    parts = [x * f if y == which else x for x, y in ((q, "q"), (k, "k"), (v, "v"))]
    o = run(kda, parts, None, None, None, scale=scale, o_dtype=out)
    ref, mag = prompt_reference(*parts, scale=scale)
    # what p's rounding to 11 bits adds for a bf16 output is below what that check allows; one around 2^-126 has steps of
    # 2^-133, as it is subnormal: half of that, 2^-134, is 2^-8 of 2^-126
    check(o, ref, mag + (2.0 ** -126 if out == BF16 else 0), exact_p=out == F32)


@pytest.mark.parametrize("which", ["k", "v"])
def test_rows_of_all_magnitudes(kda, which):
    # row by row, over most of fp32's range; the queries match where the keys have it
    q, k, v = inputs(200, 200, 2, 2, 64, F32, seed=25)[0]
    f = 2.0 ** torch.linspace(-120, 120, 200)[torch.randperm(200, generator=torch.Generator().manual_seed(1))][:, None, None]
    scale = 64 ** -0.5
    if which == "v":
        v = v * f
    else:
        k, q, scale = k * f, q * 2.0 ** -118, scale
    o = run(kda, (q, k, v), None, None, None, scale=scale)
    ref, mag = prompt_reference(q, k, v, scale=scale)
    check(o, ref, mag, exact_p=True)


@pytest.mark.parametrize("out", [BF16, F32])
def test_rows_beyond_32_bits(kda, out):
    # more than 2^32 elements of q and o: the last sequences come out as by themselves
    Hq, Hkv, d, n, L = 128, 4, 64, 4200, 128
    T = n * L
    assert T * Hq * d > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(27)
    f = lambda h: torch.empty((T, h, d), dtype=BF16, device="cuda").normal_(generator=g)
    q, k, v = f(Hq), f(Hkv), f(Hkv)
    cu = torch.arange(0, T + 1, L, dtype=torch.int32, device="cuda")
    o = kda.kda_prompt_attention(q, k, v, cu, o_dtype=out)
    for at in (0, T // 2 // L * L, T - 2 * L):
        part = [x[at:at + 2 * L].clone() for x in (q, k, v)]
        assert torch.equal(o[at:at + 2 * L], kda.kda_prompt_attention(*part, i32([0, L, 2 * L]), o_dtype=out))
    # a sequence's first token sees itself alone; an fp32 output has a weight of 22 bits (2^-23), 2^(m - n) and 2^(n - m),
    # 2^-22 each by ex2 (their arguments' rounding is the same and cancels), and three products of 2^-24: below 2^-20
    first = v[::L].repeat_interleave(Hq // Hkv, 1).float()
    assert ((o[::L].float() - first).abs() <= (2.0 ** -20 if out == F32 else 0) * first.abs()).all()
