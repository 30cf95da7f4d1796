"""kda_cache_attention_e4m3 against a float64 reference over the values that the
cache stands for.

Bounds, per element, with A = sum_j p_j |v_j|:
  fp32   |err| <= 1e-4 A: q and p are sums of two fp16 (22 bits), a score is a sum
         of d <= 128 products, off by at most d 2^-24 sum |q k| scale (about 9e-5
         at these inputs' scores), which is p's relative error.
  bf16   |err| <= 2^-8 |o| + 2^-11 A + 1e-4 A: the rounding of o, p rounded to fp16
         (half a step) for the second product.  fp32 output from bf16 is held to the
         fp32 bound.
"""
import numpy as np
import pytest
import torch

from tests._prompt import E4M3, cache_reference, dequantised, eight_bits, prompt_reference, rotate, table_for

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


class Call:
    def __init__(self, N, Ts, Hq, Hkv, d, page, block, lengths, dtype, seed=0, spread=0.0, gap=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        f = lambda *s: torch.randn(s, generator=g)
        self.q = (1.5 * f(N, Ts, Hq, d)).to(dtype)
        self.lengths = np.asarray(lengths, np.int32)
        self.table, P = table_for(np.maximum(lengths, 1), page, rng)
        pools = [f(P, page, Hkv, d) for _ in range(2)]
        if spread:                                  # magnitudes of blocks apart by powers of e^spread
            pools[1] = (pools[1].view(P, page // block, block, Hkv, d)
                        * torch.exp(spread * f(P, page // block, 1, Hkv, 1))).view(P, page, Hkv, d)
        (self.k, self.ks), (self.v, self.vs) = (eight_bits(x, block) for x in pools)
        self.gap, self.page, self.block = gap, page, block
        live = torch.zeros(P, page, dtype=torch.bool)
        for n in range(N):
            for i in range(int(lengths[n])):
                live[self.table[n, i // page], i % page] = True
        # rows and blocks of no sequence hold NaN
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            x.view(torch.uint8)[~live] = 0x7F
            s[~live.view(P, page // block, block).any(2)] = float("nan")

    def on(self, x):
        x = x.view(torch.uint8)
        if not self.gap:
            return x.cuda().view(E4M3)
        P, page, h, d = x.shape
        y = torch.full((P, page * h * d + self.gap), 0x7F, dtype=torch.uint8, device="cuda")
        y[:, :page * h * d] = x.view(P, -1).cuda()
        return y.view(E4M3).as_strided((P, page, h, d), (y.shape[1], h * d, d, 1))

    def args(self):
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
        return dict(q=self.q.cuda(), k_cache=self.on(self.k), v_cache=self.on(self.v), k_scales=self.ks.cuda(),
                    v_scales=self.vs.cuda(), page_table=i32(self.table), lengths=i32(self.lengths))

    def run(self, kda, **kw):
        o = kda.kda_cache_attention_e4m3(**{**self.args(), **kw})
        torch.cuda.synchronize()
        return o

    def reference(self, **kw):
        return cache_reference(self.q, dequantised(self.k, self.ks), dequantised(self.v, self.vs), self.table,
                               self.lengths, **kw)


def check(o, ref, mag, exact_p, more=1.0):
    o64 = o.double().cpu().numpy()
    bound = more * (1e-4 * mag + (0 if exact_p else 2.0 ** -11 * mag))
    if o.dtype == BF16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(o64 - ref) <= bound)
    assert not bad.any(), "%d of %d elements off, worst %.3g of the bound, first at %s" % (
        bad.sum(), bad.size, np.nanmax(np.abs(o64 - ref) / np.maximum(bound, 1e-30)), np.argwhere(bad)[0])


CASES = [
    # N, Ts, Hq, Hkv, d, page, block, lengths
    (1, 1, 1, 1, 16, 1, 1, [1]),
    (1, 1, 8, 2, 128, 16, 16, [0]),
    (3, 1, 8, 2, 64, 16, 8, [63, 64, 65]),
    (4, 5, 6, 2, 128, 48, 24, [0, 1, 127, 129]),
    (2, 8, 16, 2, 128, 64, 64, [500, 3]),       # four row tiles
    (2, 3, 7, 1, 32, 7, 7, [128, 300]),
    (5, 1, 15, 3, 32, 100, 50, [77, 0, 256, 255, 31]),
    (1, 1, 4, 1, 128, 64, 64, [9001]),
    (1, 2, 12, 4, 16, 256, 256, [1500]),
    (40, 1, 4, 2, 64, 32, 16, list(range(0, 400, 10))),
    (1, 64, 2, 1, 128, 16, 4, [1000]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_matches_reference(kda, case, dtype, out):
    c = Call(*case, dtype, seed=sum(case[:7]))
    o = c.run(kda, o_dtype=out)
    assert o.dtype == out
    check(o, *c.reference(), exact_p=out == F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_blocks_of_far_apart_magnitudes(kda, dtype):
    c = Call(3, 2, 8, 2, 128, 32, 16, [700, 40, 333], dtype, seed=3, spread=8.0)
    check(c.run(kda), *c.reference(), exact_p=dtype == F32)
    c = Call(2, 1, 4, 1, 64, 32, 8, [200, 90], dtype, seed=4)
    c.vs[:] = 0.0                                   # nothing but zeros
    o = c.run(kda)
    assert torch.all(o == 0)
    c.vs[:] = 2.0 ** -126
    o = c.run(kda, o_dtype=F32)
    ref, mag = c.reference()
    # the outputs are subnormal or near it: 2^-149 is their step
    assert (np.abs(o.double().cpu().numpy() - ref) <= 2e-3 * mag + 2.0 ** -140).all()


@pytest.mark.parametrize("factor", [1e-30, 1e-6, 1e4])
def test_queries_of_any_magnitude(kda, factor):
    c = Call(2, 1, 8, 2, 64, 32, 32, [100, 333], F32, seed=5)
    c.q *= factor
    scale = 64 ** -0.5 / factor
    check(c.run(kda, scale=scale), *c.reference(scale=scale), exact_p=True)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_scales_of_either_sign(kda, scale):
    c = Call(2, 2, 8, 2, 64, 32, 32, [100, 333], BF16, seed=6)
    # at 1.0 the scores, and with them their rounding, are 8 times the default's
    check(c.run(kda, scale=scale), *c.reference(scale=scale), exact_p=False, more=max(1.0, 8 * scale))


def test_rising_scores(kda):
    c = Call(1, 1, 4, 2, 64, 64, 16, [2000], F32, seed=7)
    ramp = torch.zeros(c.k.shape[:2])
    for i in range(2000):
        ramp[c.table[0, i // 64], i % 64] = i / 1000 - 1
    (c.k, c.ks) = eight_bits((ramp[:, :, None, None] * 4).expand(c.k.shape).contiguous(), 16)
    c.q[:] = 4.0
    ref, mag = c.reference()
    check(c.run(kda), ref, mag, exact_p=True, more=4.0)


def test_page_stride_and_hidden_pages(kda):
    c = Call(2, 1, 4, 2, 128, 16, 8, [100, 60], BF16, seed=8, gap=64)
    c.table[0, 2], c.table[1, 0] = -1, 1 << 20      # hidden
    check(c.run(kda), *c.reference(), exact_p=False)


def test_lengths_are_clamped(kda):
    c = Call(2, 1, 4, 2, 64, 16, 8, [64, 32], BF16, seed=9)
    c.table = np.ascontiguousarray(c.table[:, :2])
    c.lengths = np.array([1000, -5], np.int32)
    check(c.run(kda), *c.reference(), exact_p=False)


def test_nan_scales_reach_only_the_tokens_that_see_their_block(kda):
    c = Call(2, 3, 4, 2, 64, 16, 8, [42, 50], BF16, seed=10)
    # sequence 0: a key block that begins at its last token; sequence 1: a value block in the middle
    c.ks[c.table[0, 2], 1, 0] = float("nan")        # rows 40 .. 47
    c.vs[c.table[1, 1], 0, 1] = float("nan")
    o = c.run(kda).float().cpu()
    ref, mag = c.reference()
    assert torch.isnan(o[0, 1:, :2]).all() and not torch.isnan(o[0, 0]).any() and not torch.isnan(o[0, :, 2:]).any()
    assert torch.isnan(o[1, :, 2:]).all() and not torch.isnan(o[1, :, :2]).any()
    fine = np.isfinite(ref)
    assert (np.abs(o.double().numpy() - ref)[fine] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag)[fine]).all()


def test_streams_graphs_and_workspaces(kda):
    c = Call(3, 1, 8, 2, 128, 32, 16, [5000, 100, 1], BF16, seed=11)
    want = c.run(kda)
    assert torch.equal(c.run(kda, stream=torch.cuda.Stream()), want)
    a = c.args()
    ws = [torch.full((kda.kda_cache_attention_e4m3_workspace_bytes(3, 1, 8, 2, 128, kda.KDA_BF16),), 0xFF,
                     dtype=torch.uint8, device="cuda") for _ in range(2)]
    o = [torch.empty_like(want) for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_cache_attention_e4m3(**a, o=o[i], workspace=ws[i])
        graphs.append(g)
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for x in o:
            x.fill_(0)
        torch.cuda.synchronize()
        for g, t in zip(graphs, s):
            with torch.cuda.stream(t):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0], want) and torch.equal(o[1], want)


def test_offsets_beyond_32_bits(kda):
    page, Hkv, d, block = 64, 8, 128, 64
    P = (1 << 32) // (page * Hkv * d) + 3
    kc, vc = (torch.full((P, page, Hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    small = Call(1, 1, 16, Hkv, d, page, block, [130], BF16, seed=12)
    ks, vs = (torch.full((P, 1, Hkv), float("nan"), device="cuda") for _ in range(2))
    table = np.array([[P - 1, 3, P - 3]], np.int32)
    for i in range(3):
        for big, x in ((kc, small.k.view(torch.uint8)), (vc, small.v.view(torch.uint8)), (ks, small.ks), (vs, small.vs)):
            big[table[0, i]] = x[small.table[0, i]].cuda()
    o = small.run(kda, k_cache=kc.view(E4M3), v_cache=vc.view(E4M3), k_scales=ks, v_scales=vs,
                  page_table=torch.from_numpy(table).cuda())
    check(o, *small.reference(), exact_p=False)


@pytest.mark.parametrize("dtype,d,page,block", [(BF16, 128, 32, 16), (BF16, 64, 48, 24), (F32, 32, 16, 16)])
def test_a_prompt_and_its_answer(kda, dtype, d, page, block):
    """What a softmax layer does with a batch: the prompts' projections are turned and
    appended, the prompts attend to themselves, then tokens come one at a time and
    attend to the cache.  Every step against float64 on what the step was given."""
    Hq, Hkv, steps = 8, 2, 5
    lens = [70, 1, 133]
    rng = np.random.default_rng(2)
    table, P = table_for(np.asarray(lens) + steps, page, rng)
    g = torch.Generator().manual_seed(3)
    f = lambda t: torch.randn((t, Hq + 2 * Hkv, d), generator=g).to(dtype).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    inv_freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float()
    kc, vc = (torch.full((P, page, Hkv, d), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.full((P, page // block, Hkv), float("nan"), device="cuda") for _ in range(2))
    pages = torch.from_numpy(table).cuda()
    cu = [0] + np.cumsum(lens).tolist()
    x = f(cu[-1])
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    plain = q.cpu().clone()
    _, _, lengths = kda.kda_cache_append_rotary(q, k, v, i32(cu), inv_freq.cuda(), kc, vc, pages, i32([0] * 3),
                                                k_scales=ks, v_scales=vs, q_out=q, k_out=k)
    pos = [p for n in lens for p in range(n)]
    want, mag = rotate(plain, pos, inv_freq, False)
    assert (np.abs(q.double().cpu().numpy() - want) <= 2.0 ** -21 * mag + 2.0 ** -8 * np.abs(want)).all()
    o = kda.kda_prompt_attention(q, k, v, i32(cu))
    ref, mag = prompt_reference(q, k, v, cu)
    tight = 0 if dtype == F32 else 2.0 ** -8
    assert (np.abs(o.double().cpu().numpy() - ref) <= (1e-4 + tight) * mag + tight * np.abs(ref)).all()
    for _ in range(steps):
        x = f(3)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        turned, none, lengths = kda.kda_cache_append_rotary(q, k, v, i32([0, 1, 2, 3]), inv_freq.cuda(), kc, vc, pages,
                                                            lengths, k_scales=ks, v_scales=vs)
        assert none is None
        o = kda.kda_cache_attention_e4m3(turned[:, None], kc, vc, ks, vs, pages, lengths)
        check(o, *cache_reference(turned[:, None], dequantised(kc, ks), dequantised(vc, vs), table, lengths.tolist()),
              exact_p=dtype == F32)
    assert lengths.tolist() == [x + steps for x in lens]


@pytest.mark.parametrize("dtype,page,block", [(BF16, 32, 16), (F32, 24, 8)])
def test_waits_that_give_up(kda, monkeypatch, dtype, page, block):
    # no copies are made: the kernel's waits run out (about 2 s), it returns, sets the
    # workspace's word and marks its rows (those of one CTA and joined ones), and the next call is
    # right
    c = Call(3, 2, 8, 2, 64, page, block, [3000, 1, 500], dtype, seed=13)
    args = c.args()
    code = kda.KDA_BF16 if dtype == BF16 else kda.KDA_FP32
    ws = torch.zeros(kda.kda_cache_attention_e4m3_workspace_bytes(3, 2, 8, 2, 64, code), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("KDA_TEST_STARVE_CONSUMERS", "1")
    o = kda.kda_cache_attention_e4m3(**args, workspace=ws)
    torch.cuda.synchronize()
    monkeypatch.delenv("KDA_TEST_STARVE_CONSUMERS")
    assert ws[8:12].view(torch.int32).item() & 2
    assert torch.isnan(o[0]).all() and torch.isnan(o[2]).all()
    ws[8:12].zero_()
    check(kda.kda_cache_attention_e4m3(**args, workspace=ws), *c.reference(), exact_p=dtype == F32)
    assert ws[8:12].view(torch.int32).item() == 0


def test_fp32_over_many_rows(kda):
    # the tensor cores cut off as they add up: sums over a whole context must not be theirs.
    # some 30,000 rows in one block's walk, values with a mean of 2.  A step's own sum over 32
    # keys is cut off by a few units of 2^-23 of it at most (4e-7 or so, not growing); the
    # sums over 625 steps round half a unit of 2^-24 of what they have, at random: 2^-24
    # sqrt(625 / 3) = 9e-7, in the output and in its divisor.  Cutting off instead would add
    # up to 625 2^-24 = 3.7e-5
    n, hi, d, page = 64, 20000, 64, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    pages = -(-hi // page)
    k, v = (torch.randn((pages, page, 4, d), generator=g, device="cuda") + b for b in (0.0, 2.0))
    table = torch.stack([torch.randperm(pages, generator=torch.Generator().manual_seed(i)) for i in range(n)])
    (k, ks), (v, vs) = ([y.cuda() if y.dtype == F32 else y.view(torch.uint8).cuda().view(E4M3) for y in eight_bits(x.cpu(), 64)]
                        for x in (k, v))
    q = torch.randn((n, 1, 4, d), generator=g, device="cuda")
    lengths = torch.full((n,), hi, dtype=torch.int32, device="cuda")
    o = kda.kda_cache_attention_e4m3(q, k, v, ks, vs, table.int().cuda(), lengths).double()
    kd, vd = (x.view(torch.uint8).view(E4M3).double() * s.double().repeat_interleave(page, 1)[..., None] for x, s in ((k, ks), (v, vs)))
    for i in (0, n - 1):
        for h in range(4):
            rows = table[i].cuda()
            w = torch.softmax((kd[rows, :, h].flatten(0, 1)[:hi] @ q[i, 0, h].double()) * d ** -0.5, 0)
            want = w @ vd[rows, :, h].flatten(0, 1)[:hi]
            assert ((o[i, 0, h] - want).norm() / want.norm()).item() < 3e-6


@pytest.mark.parametrize("N,Ts,Hq,Hkv,d,page,block,dtype", [
    (64, 1, 32, 8, 128, 32, 16, BF16), (40, 3, 16, 8, 64, 32, 8, F32), (40, 2, 12, 12, 32, 16, 16, BF16),
    (90, 1, 12, 6, 16, 24, 8, F32), (45, 5, 64, 16, 128, 64, 64, BF16), (48, 1, 8, 4, 128, 8, 8, F32)])
def test_many_sequences(kda, N, Ts, Hq, Hkv, d, page, block, dtype):
    # heads side by side in a thread block, their items cut between thread blocks or not
    rng = np.random.default_rng(N)
    lengths = rng.integers(0, 900, N)
    lengths[:8] = [0, 1, 31, 32, 33, 256, 2000, 5]
    c = Call(N, Ts, Hq, Hkv, d, page, block, lengths, dtype, seed=N, gap=64)
    ref, mag = c.reference()
    args = c.args()
    o = kda.kda_cache_attention_e4m3(**args)
    check(o, ref, mag, exact_p=dtype == F32)
    # a scale of one head, and a page that is not there
    block0 = c.table[6, 0], 0, 1
    args["v_scales"][block0] = float("nan")
    lost = args["page_table"].clone()
    lost[5, :] = -1
    args["page_table"] = lost
    p = kda.kda_cache_attention_e4m3(**args)
    G = Hq // Hkv
    assert torch.isnan(p[6, :, G:2 * G]).all() and (p[5] == 0).all()
    keep = torch.ones(o.shape[:3], dtype=torch.bool)
    keep[6, :, G:2 * G] = keep[5] = False
    assert torch.equal(p[keep.cuda()], o[keep.cuda()])


@pytest.mark.parametrize("N,Ts,Hq,Hkv,lengths", [(2, 200, 16, 2, [700, 150]), (3, 60, 8, 1, [61, 333, 0])])
def test_many_tokens(kda, N, Ts, Hq, Hkv, lengths):
    # so many row tiles that a thread block has all items of one, or that few share them
    c = Call(N, Ts, Hq, Hkv, 64, 32, 16, lengths, BF16, seed=Ts)
    check(c.run(kda), *c.reference(), exact_p=False)


def test_sequences_share_pages(kda):
    # a common prefix: the same pages in every row of the table, and one page twice
    c = Call(1, 1, 8, 2, 128, 32, 16, [500], BF16, seed=21)
    args = c.args()
    one = args["page_table"]
    n = 50
    args["q"] = args["q"].expand(n, 1, 8, 128).contiguous()
    args["page_table"] = one.expand(n, one.shape[1]).contiguous()
    args["lengths"] = args["lengths"].expand(n).contiguous()
    ref, mag = c.reference()
    o = kda.kda_cache_attention_e4m3(**args)
    check(o, ref.repeat(n, 0), mag.repeat(n, 0), exact_p=False)
    args["page_table"][:, 1] = args["page_table"][:, 0]
    c.table[:, 1] = c.table[:, 0]
    ref, mag = c.reference()
    check(kda.kda_cache_attention_e4m3(**args), ref.repeat(n, 0), mag.repeat(n, 0), exact_p=False)


@pytest.mark.parametrize("page,block", [(32, 16), (8, 8), (7, 7)])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_values_far_above_those_of_the_keys_that_count(kda, page, block, dtype, out):
    # rows of probability 0 with values of 2^75 beside ones of 2^-75 that have all of it
    n = 3 * 32 * 7
    c = Call(1, 1, 4, 2, 64, page, block, [n], dtype, seed=31)
    last = c.table[0, -1]
    c.q[:] = 8.0
    c.k.view(torch.uint8)[:] = 0
    c.ks[:] = 1.0
    c.k[last, :] = 2.0                              # scores of 64 * 8 * 2 / 8 = 128
    low = c.vs[last] * 2.0 ** -75
    c.vs *= 2.0 ** 75
    c.vs[last] = low
    ref, mag = c.reference()
    assert 0 < np.abs(ref).max() < 2.0 ** -70
    check(c.run(kda, o_dtype=out), ref, mag, exact_p=out == F32)


@pytest.mark.parametrize("page,block", [(64, 16), (56, 8), (56, 7)])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("gap", [10, 12, 14, 16, 18])
@pytest.mark.parametrize("first", [True, False])
def test_one_row_far_above_many_others(kda, page, block, dtype, out, gap, first):
    # an attention sink: one row's score lies `gap` above those of 2^15 others, which are all the same, so that
    # errors of their weights add up.  Values of 1 throughout, which the output has to be; then a sink
    # without a value, where the others are all of the output.  64 sequences, so that one walk has many rows.
    n, N, d = 1 << 15, 64, 32
    pages = -(-n // page)
    at = (0, 0) if first else ((n - 1) // page, (n - 1) % page)
    one = torch.ones((pages, page, 1, d)).to(E4M3)
    k = torch.zeros((pages, page, 1, d)).to(E4M3)
    k[at] = one[at]
    ks, vs = (torch.ones((pages, page // block, 1)) for _ in range(2))
    ks[at[0], at[1] // block] = gap / d ** 0.5
    table = torch.arange(pages, dtype=torch.int32).expand(N, pages).contiguous()
    lengths = torch.full((N,), n, dtype=torch.int32)
    q = torch.ones((N, 1, 2, d), dtype=dtype)
    # Added up in n / 32 steps at most, each off by half a unit of 2^-23 of a sum between 1 and 2, in the output and in its
    # divisor: 2 * 2^10 * 2^-24, always the same way.  The exponentials: 2^-22 each, and 18 log2 e 2^-24 of their
    # argument's rounding; the scale of that block 2^-24 of a score of 18.
    bound = 2.0 ** -13 + 2.0 ** -19
    if out == BF16:
        bound += 2.0 ** -11 + 2.0 ** -8
    for sink in (1.0, 0.0):
        v = one.clone()
        v[at] = torch.full((1, d), sink).to(E4M3)
        held = [x.view(torch.uint8).cuda().view(E4M3) for x in (k, v)]
        o = kda.kda_cache_attention_e4m3(q.cuda(), *held, ks.cuda(), vs.cuda(), table.cuda(), lengths.cuda(), o_dtype=out)
        ref, mag = cache_reference(q[:1], dequantised(k, ks), dequantised(v, vs), table[:1].numpy(), [n])
        # (with 11 bits and no more, weights below 2^-21 of the largest have fewer: e^-14.6)
        if sink or out == F32 or gap < 14.5:
            assert (np.abs(o.double().cpu().numpy() - ref) <= bound * mag).all()


@pytest.mark.parametrize("page,block", [(32, 16), (24, 8), (7, 7)])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("which,power", [("q", 118), ("q", -118), ("q", -124), ("k", 100), ("k", -100), ("v", 100), ("v", -100)])
def test_magnitudes_near_the_ends_of_fp32(kda, page, block, dtype, out, which, power):
    c = Call(3, 2, 8, 2, 64, page, block, [100, 333, 1], dtype, seed=30)
    f, scale = 2.0 ** power, 64 ** -0.5
    if which == "q":
        c.q = c.q * f
    elif which == "k":
        c.ks = c.ks * f
    else:
        c.vs = c.vs * f
    if which != "v":
        scale /= f
    check(c.run(kda, scale=scale, o_dtype=out), *c.reference(scale=scale), exact_p=out == F32)


@pytest.mark.parametrize("page,block", [(16, 16), (7, 7)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinite_queries(kda, page, block, dtype, value):
    # scores of -inf alone are not the same as no rows; a token that sees no row gives 0 all the same
    c = Call(4, 2, 4, 2, 32, page, block, [1, 2, 300, 0], dtype, seed=32)
    bits = c.k.view(torch.uint8)
    live = (bits & 0x7F) != 0x7F
    bits[live] = (bits[live] & 0x7F) | (0x80 if value > 0 else 0)       # one sign, so that inf * k = -inf in all rows
    for scale in (0.2, -0.2):
        want = c.run(kda, scale=scale).clone()
        q = c.q.clone()
        q[:, 1, 1, 5] = value
        o = c.run(kda, q=q.cuda(), scale=scale)
        hit = torch.zeros(o.shape[:3], dtype=torch.bool, device="cuda")
        hit[:3, 1, 1] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], want[~hit])
        assert torch.all(o[3] == 0) and torch.all(o[0, 0] == 0)
