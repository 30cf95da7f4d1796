"""kda_cache_append_rotary against plain loops.

Turned rows, per element, with M = |x| + |y| of the pair: the angle is off by 2^-32
of a turn (1.5e-9), sine and cosine by at most two units of 2^-24 and the angle's
rounding to fp32 (pi 2^-24), the two products and the sum by 2^-24 M each: within
2^-21 M; in bf16 2^-8 of the value more.  In 8 bits a value is off by half a step of
e4m3, at most max(2^-4 |x|, 2^-10 s), and by the above; rows that were there, and
values, which are not turned, have to be equal bit by bit.
"""
import numpy as np
import pytest
import torch

from tests._prompt import E4M3, eight_bits, power_scale, rotate, spans, table_for

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


def frequencies(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


class Call:
    """Inputs of one call, on the CPU, and what it has to leave behind."""

    def __init__(self, lens, past, Hq, Hkv, d, page, block, dtype, rot=None, interleaved=False, seed=0, cu=None,
                 extra=0, base=10000.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        f = lambda *s: torch.randn(s, generator=g)
        self.cu = [0] + np.cumsum(lens).tolist() if cu is None else cu
        self.T = sum(lens) + extra
        self.past = np.asarray(past, np.int32)
        self.q = f(self.T, Hq, d).to(dtype) if Hq else None
        self.k, self.v = (3 * f(self.T, Hkv, d)).to(dtype), f(self.T, Hkv, d).to(dtype)
        self.inv_freq, self.interleaved = frequencies(rot or d, base), interleaved
        self.table, pages = table_for(np.asarray(lens) + past, page, rng)
        pools = [f(pages, page, Hkv, d) for _ in range(2)]
        self.page, self.block, self.dtype = page, block, dtype
        self.scales = [None, None]
        if block:
            held = [eight_bits(x, block) for x in pools]
            pools, self.scales = [x for x, _ in held], [s for _, s in held]
        else:
            pools = [x.to(dtype) for x in pools]
        self.pools = pools

    def positions(self):
        """(row, sequence, position) of every row that a sequence owns."""
        out = []
        for n, rows in enumerate(spans(self.cu, self.T)):
            if self.past[n] >= 0:
                out += [(r, n, int(self.past[n]) + i) for i, r in enumerate(rows)]
        return out

    def run(self, kda, **kw):
        c = lambda x: None if x is None else x.cuda()
        i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        self.kc, self.vc = (x.view(torch.uint8).cuda().view(E4M3) if self.block else x.cuda() for x in self.pools)
        self.ks, self.vs = c(self.scales[0]), c(self.scales[1])
        kw.setdefault("want_k", True)
        args = dict(q=c(self.q), k=c(self.k), v=c(self.v), cu_seqlens=i32(self.cu), inv_freq=c(self.inv_freq),
                    k_cache=self.kc, v_cache=self.vc, page_table=i32(self.table), lengths=i32(self.past),
                    k_scales=self.ks, v_scales=self.vs, interleaved=self.interleaved)
        args.update(kw)
        out = kda.kda_cache_append_rotary(**args)
        torch.cuda.synchronize()
        return out

    def check_turned(self, got, x):
        rows = [r for r, _, _ in self.positions()]
        want, mag = rotate(x[rows], [p for _, _, p in self.positions()], self.inv_freq, self.interleaved)
        bound = 2.0 ** -21 * mag + (2.0 ** -8 * np.abs(want) if self.dtype == BF16 else 0)
        assert (np.abs(got[rows].double().cpu().numpy() - want) <= bound).all()

    def places(self):
        """{(page, slot): (row, position)} of the rows that have a place."""
        out = {}
        for r, n, p in self.positions():
            at = p // self.page
            if at < self.table.shape[1] and 0 <= self.table[n, at] < self.pools[0].shape[0]:
                out[int(self.table[n, at]), p % self.page] = r, n, p
        return out

    def check_cache(self):
        places = self.places()
        if not self.block:
            for pool, cache, x, turned in ((self.pools[0], self.kc, self.k, True), (self.pools[1], self.vc, self.v, False)):
                want, cache = pool.clone(), cache.cpu()
                for (page, slot), (r, n, p) in places.items():
                    if turned:
                        y, mag = rotate(x[r:r + 1], [p], self.inv_freq, self.interleaved)
                        bound = 2.0 ** -21 * mag[0] + (2.0 ** -8 * np.abs(y[0]) if self.dtype == BF16 else 0)
                        assert (np.abs(cache[page, slot].double().numpy() - y[0]) <= bound).all()
                        want[page, slot] = cache[page, slot]
                    else:
                        want[page, slot] = x[r]
                assert torch.equal(cache, want)
            return
        blocks = {}
        for (page, slot), (r, n, p) in places.items():
            blocks.setdefault((page, slot // self.block), []).append((slot, r, p))
        for pool, scales, cache, got, x, turned in (
                (self.pools[0], self.scales[0], self.kc, self.ks, self.k, True),
                (self.pools[1], self.scales[1], self.vc, self.vs, self.v, False)):
            want, want_s = pool.clone().view(torch.uint8), scales.clone()
            cache, got = cache.view(torch.uint8).cpu(), got.cpu()
            for (page, b), rows in blocks.items():
                rows.sort()
                off = rows[0][0] - b * self.block
                y = x[[r for _, r, _ in rows]].double().numpy()
                mag = np.zeros_like(y)
                if turned:
                    y, mag = rotate(x[[r for _, r, _ in rows]], [p for _, _, p in rows], self.inv_freq, self.interleaved)
                slots = slice(rows[0][0], rows[-1][0] + 1)
                for h in range(x.shape[1]):
                    with np.errstate(invalid="ignore"):
                        top = np.abs(y[:, h]).max()
                    had = float(scales[page, b, h]) if off else 0.0
                    s = power_scale(top)
                    # (turned rows whose largest magnitude lies within the arithmetic's error of a step would not do)
                    assert not (turned and np.isfinite(top)) or power_scale(top * (1 - 1e-6)) == power_scale(top * (1 + 1e-6))
                    s = s if np.isnan(s) or np.isnan(had) else max(s, had)
                    s = float("nan") if np.isnan(had) else s
                    want_s[page, b, h] = s
                    if off and 0 < had < s:
                        old = slice(b * self.block, b * self.block + off)
                        z = want[page, old, h].view(E4M3).float() * (had / s)
                        want[page, old, h] = z.to(E4M3).view(torch.uint8)
                    new = cache[page, slots, h].view(E4M3).double().numpy()
                    if np.isnan(s) or s == 0:
                        assert (new == 0).all()
                    elif turned:
                        bound = np.maximum(2.0 ** -4 * np.abs(y[:, h]), 2.0 ** -10 * s) + 2.0 ** -20 * mag[:, h]
                        assert (np.abs(new * s - y[:, h]) <= bound).all()
                    else:
                        exact = torch.from_numpy(y[:, h] / s).float().to(E4M3)
                        assert np.array_equal(new, exact.double().numpy())
                    want[page, slots, h] = cache[page, slots, h]
            assert torch.equal(cache, want)
            assert np.array_equal(got.numpy(), want_s.numpy(), equal_nan=True)

    def check(self, q, k, new):
        if self.q is not None:
            self.check_turned(q, self.q)
        self.check_turned(k, self.k)
        self.check_cache()
        counts = [len(r) for r in spans(self.cu, self.T)]
        assert new.tolist() == (self.past + counts).tolist()


CASES = [
    # lens, past, Hq, Hkv, d, page, block, rot, interleaved
    ([1], [0], 1, 1, 16, 16, 16, 16, False),
    ([1], [7], 8, 2, 128, 16, 8, 128, False),
    ([5, 0, 33], [3, 9, 64], 6, 2, 64, 24, 24, 32, True),
    ([200, 17], [0, 130], 4, 4, 128, 64, 64, 128, False),
    ([64, 63, 65], [0, 1, 63], 2, 1, 128, 64, 32, 64, False),
    ([40, 1, 90], [100, 31, 6], 0, 3, 32, 30, 10, 16, True),
    ([3] * 40, list(range(40)), 5, 1, 64, 8, 1, 64, False),
    ([300], [500], 3, 1, 128, 128, 128, 128, True),
    ([700], [11], 16, 8, 16, 100, 50, 16, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c[2:]).replace(" ", ""))
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("held", ["own type", "8 bits"])
def test_matches_plain_loops(kda, case, dtype, held):
    lens, past, Hq, Hkv, d, page, block, rot, inter = case
    c = Call(lens, past, Hq, Hkv, d, page, block if held == "8 bits" else 0, dtype, rot, inter, seed=sum(lens) + d)
    c.check(*c.run(kda))


def test_pages_of_odd_sizes(kda):
    for page in (1, 7, 17):
        c = Call([50, 23], [4, 9], 2, 1, 64, page, 0, BF16, seed=page)
        c.check(*c.run(kda))


def test_far_positions(kda):
    # the table names the pages of the far positions alone
    page, far = 64, 33000 * 64 + 17
    c = Call([90], [far], 2, 1, 64, page, 64, F32, seed=5, base=1e6)
    c.table = np.full((1, 33010), -1, np.int32)
    c.table[0, 33000:33003] = [2, 0, 1]
    c.pools = [x[:3] for x in c.pools]
    c.scales = [x[:3] for x in c.scales]
    c.check(*c.run(kda))


def test_in_place_in_one_projection(kda):
    for block in (0, 16):
        c = Call([70, 9], [20, 3], 4, 2, 64, 32, block, BF16, seed=6)
        x = torch.cat([c.q, c.k, c.v], 1).cuda()
        q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
        oq, ok, new = c.run(kda, q=q, k=k, v=v, q_out=q, k_out=k)
        assert oq.data_ptr() == q.data_ptr() and ok.data_ptr() == k.data_ptr()
        assert torch.equal(v.cpu(), c.v)
        c.check(oq, ok, new)


def test_rows_without_a_place_are_turned_all_the_same(kda):
    # past the table, a page that does not exist, rows of no sequence, a negative length
    for block in (0, 8):
        c = Call([20, 20, 6], [12, 0, -1], 2, 1, 32, 8, block, F32, seed=7, extra=5)
        c.table[0, 3:] = -1
        c.table[1, 1] = 999
        keep = torch.full(c.q.shape, 9.0, device="cuda")
        keep_k = torch.full(c.k.shape, 9.0, device="cuda")
        q, k, new = c.run(kda, q_out=keep, k_out=keep_k)
        c.check(q, k, new)
        assert torch.all(q[40:] == 9) and torch.all(k[40:] == 9)


@pytest.mark.parametrize("cu", [[0, 3, 5], [2, 3, 8], [0, 6, 4], [0, 9, 12], [5, 2, 8], [-2, 3, 8], [9, 9, 9]])
@pytest.mark.parametrize("block", [0, 4])
def test_any_cu_seqlens(kda, cu, block):
    c = Call([4, 4], [3, 1], 2, 1, 16, 8, block, F32, seed=8, cu=cu)
    c.table = np.arange(4, dtype=np.int32).reshape(2, 2)
    c.check(*c.run(kda))


def test_infinities_zeros_and_scales_that_grow(kda):
    c = Call([8, 6, 10], [5, 12, 3], 0, 2, 32, 16, 8, F32, seed=9)
    c.v[:4, 0] = 0
    c.k[2, 0, 5], c.v[3, 1, 2] = float("inf"), float("nan")
    c.v[8:14, 0] *= 1e6                             # a begun block's rows are rounded to a larger scale
    c.v[8:14, 1] = 0                                # zeros leave the scale that was there
    c.v[14:24, 1] = 1e-30
    c.k[14:24, 1] *= 1e30
    c.v[14:24, 0] = 1e-42                           # below 448 * 2^-126
    q, k, new = c.run(kda)
    fine = torch.ones(24, dtype=torch.bool)
    fine[2] = False
    rows = [i for i in range(24) if fine[i]]
    want, mag = rotate(c.k[rows], [c.positions()[i][2] for i in rows], c.inv_freq, False)
    assert (np.abs(k.cpu()[rows].double().numpy() - want) <= 2.0 ** -21 * mag).all()
    c.check_cache()


def test_a_block_filled_token_by_token_is_the_block_filled_at_once(kda):
    # but for the roundings of rows that a larger scale met
    d, page, block = 64, 32, 16
    whole = Call([40], [0], 0, 1, d, page, block, F32, seed=10)
    whole.run(kda)
    one = Call([40], [0], 0, 1, d, page, block, F32, seed=10)
    one.pools = [x.clone() for x in whole.pools]
    kc, vc = (x.view(torch.uint8).cuda().view(E4M3) for x in one.pools)
    ks, vs = (s.cuda() for s in one.scales)
    lengths = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(one.table).cuda()
    for t in range(40):
        _, k, lengths = kda.kda_cache_append_rotary(None, one.k[t:t + 1].cuda(), one.v[t:t + 1].cuda(), cu,
                                                    one.inv_freq.cuda(), kc, vc, table, lengths, k_scales=ks,
                                                    v_scales=vs)
        assert k is None
    assert lengths.item() == 40
    assert torch.equal(ks, whole.ks) and torch.equal(vs, whole.vs)
    for a, b, s in ((kc, whole.kc, ks), (vc, whole.vc, vs)):
        a, b = (x.view(torch.uint8).cpu().view(E4M3).double() for x in (a, b))
        # two roundings against one: at most one step more
        assert ((a - b).abs() <= torch.clamp(b.abs() * 2.0 ** -3, min=2.0 ** -9)).all()


def test_streams_and_graphs(kda):
    c = Call([33, 5], [7, 30], 4, 2, 128, 32, 16, BF16, seed=11)
    q, k, new = c.run(kda, stream=torch.cuda.Stream())
    c.check(q, k, new)
    first = [x.clone() for x in (q, k, c.kc.view(torch.uint8), c.vc.view(torch.uint8), c.ks, c.vs)]
    # the same call again changes nothing: what it had to round is rounded
    c2 = Call([33, 5], [7, 30], 4, 2, 128, 32, 16, BF16, seed=11)
    c2.run(kda)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    args = dict(q=c2.q.cuda(), k=c2.k.cuda(), v=c2.v.cuda(), cu_seqlens=torch.tensor(c2.cu, dtype=torch.int32).cuda(),
                inv_freq=c2.inv_freq.cuda(), k_cache=c2.kc, v_cache=c2.vc, page_table=torch.from_numpy(c2.table).cuda(),
                lengths=torch.from_numpy(c2.past).cuda(), k_scales=c2.ks, v_scales=c2.vs, q_out=qo, k_out=ko)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kda.kda_cache_append_rotary(**args)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(first, (qo, ko, c2.kc.view(torch.uint8), c2.vc.view(torch.uint8), c2.ks, c2.vs)):
        assert torch.equal(x, y)
    assert out[2].tolist() == new.tolist()


def test_no_rows(kda):
    c = Call([0, 0], [3, 4], 2, 1, 64, 16, 16, BF16, seed=12)
    q, k, new = c.run(kda)
    assert q.shape[0] == 0 and new.tolist() == [3, 4]
    c.check_cache()


def test_offsets_beyond_32_bits(kda):
    page, Hkv, d, block = 64, 8, 128, 64
    P = (1 << 32) // (page * Hkv * d) + 3
    kc, vc = (torch.empty((P, page, Hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[-2:], vc[-2:] = 1, 2
    ks, vs = (torch.ones((P, 1, Hkv), device="cuda") for _ in range(2))
    k, v = (torch.randn((3, Hkv, d), device="cuda").to(BF16) for _ in range(2))
    table = torch.tensor([[P - 2, P - 1]], dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kda.kda_cache_append_rotary(None, k, v, i32([0, 3]), torch.zeros(64, device="cuda"), kc.view(E4M3), vc.view(E4M3), table,
                                i32([62]), k_scales=ks, v_scales=vs)
    for pool, x, s, fill in ((kc, k, ks, 1), (vc, v, vs, 2)):
        tail = pool[-2:].reshape(-1, Hkv, d)
        # frequencies of 0 turn nothing; the begun block keeps its scale of 1
        by = torch.stack([s[-2, 0], s[-2, 0], s[-1, 0]])[:, :, None]
        assert torch.equal(tail[62:65], (x.float() / by).to(E4M3).view(torch.uint8))
        assert torch.all(tail[:62] == fill) and torch.all(tail[65:] == fill)
        assert torch.all(s[-2] == 1) and torch.all(s[:-2] == 1)


@pytest.mark.parametrize("block", [0, 16])
def test_more_sequences_than_are_held(kda, block):
    rng = np.random.default_rng(4)
    c = Call(rng.integers(0, 4, 1300).tolist(), rng.integers(0, 40, 1300).tolist(), 2, 1, 32, 16, block, BF16, seed=20)
    c.check(*c.run(kda))


@pytest.mark.parametrize("lens,Hkv", [([6000], 4), ([90] * 60, 8)])
def test_heads_in_several_parts(kda, lens, Hkv):
    # more units than SMs and fewer, so that a window's heads go to one thread block or several
    c = Call(lens, [5] * len(lens), Hkv, Hkv, 64, 64, 32, BF16, seed=len(lens))
    c.check(*c.run(kda))


@pytest.mark.parametrize("block", [0, 4])
def test_offsets_at_the_ends_of_their_type(kda, block):
    # differences of offsets that do not fit 32 bits
    low, high = -2 ** 31, 2 ** 31 - 1
    for cu in ([5, low, 8], [low, 3, high], [high, low, 8], [0, 8, low]):
        c = Call([4, 4], [3, 1], 2, 1, 16, 8, block, F32, seed=21, cu=cu)
        c.table = np.arange(6, dtype=np.int32).reshape(2, 3)
        c.pools = [torch.cat([x] * 3)[:6] for x in c.pools]
        c.scales = [x if x is None else torch.cat([x] * 3)[:6] for x in c.scales]
        c.check(*c.run(kda))


def test_more_threads_than_31_bits(kda):
    # a thread block per token of 2^23 sequences and some: 2^31 threads and more
    N, page, d = (1 << 23) + 5, 8, 16
    kc, vc = (torch.zeros((N, page, 1, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((N, 1, 1), device="cuda") for _ in range(2))
    k = torch.randint(-8, 9, (N, 1, d), device="cuda").to(BF16)
    steps = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(N, dtype=torch.int32, device="cuda")
    _, _, new = kda.kda_cache_append_rotary(None, k, -k, steps, torch.zeros(8, device="cuda"), kc.view(E4M3), vc.view(E4M3),
                                            steps[:N, None], zero, k_scales=ks, v_scales=vs)
    assert torch.all(new == 1)
    # whole numbers up to 8 times a power of two are e4m3 values; frequencies of 0 turn nothing
    for cache, s, x in ((kc, ks, k), (vc, vs, -k)):
        assert torch.equal(cache[:, 0].view(E4M3).float() * s, x.float()) and not cache[:, 1:].any()


def test_calls_from_two_threads(kda):
    # blocks whose tables of angles differ in size, through one kernel, without the binding's time between the calls
    import threading

    lib, errors, threads, checks = kda.lib(), [], [], []
    for block in (128, 72) * 2:
        c = Call([block], [0], 0, 1, 128, block, block, BF16, seed=block)
        c.run(kda)
        want = [x.clone() for x in (c.kc.view(torch.uint8), c.vc.view(torch.uint8), c.ks, c.vs)]
        held = [c.k.cuda(), c.v.cuda(), torch.tensor([0, block], dtype=torch.int32).cuda(), c.inv_freq.cuda(),
                torch.from_numpy(c.table).cuda(), torch.from_numpy(c.past).cuda(), torch.cuda.Stream()]
        k, v, cu, freq, table, past, stream = held
        args = (None, k.data_ptr(), v.data_ptr(), 0, 128, 128, cu.data_ptr(), block, freq.data_ptr(), 128, 0, table.data_ptr(),
                past.data_ptr(), 1, 0, 1, 128, c.kc.shape[0], block, table.shape[1], c.kc.stride(0), block, kda.KDA_BF16, None, 0,
                None, 0, c.kc.data_ptr(), c.vc.data_ptr(), c.ks.data_ptr(), c.vs.data_ptr(), None, stream.cuda_stream)

        def work(args=args, stream=stream):
            errors.extend(filter(None, (lib.kda_cache_append_rotary(*args) for _ in range(20000))))
            stream.synchronize()

        checks.append((c, want, held))
        threads.append(threading.Thread(target=work))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c, want, _ in checks:
        assert all(torch.equal(x, y) for x, y in zip((c.kc.view(torch.uint8), c.vc.view(torch.uint8), c.ks, c.vs), want))


@pytest.mark.parametrize("base", [1e4, 5e5])
def test_angles_at_all_positions(kda, base):
    # pairs of (1, 0) become (cos, sin).  Off by 2 pi times 2^-26 + p f 2^-54 + 2^-32 of a turn (the fraction's rounding
    # to fp32, the frequency's 53 bits, the part below 32 bits), and by sincospif: 2 units of 2^-24 of 1
    d = 128
    pos = [0, 1, 1000, 10 ** 6, 2 ** 24 + 1, 2 ** 28 - 1, 2 ** 30 + 12345, 2 ** 31 - 2]
    n = len(pos)
    f = frequencies(d, base)
    q = torch.zeros((n, 1, d))
    q[..., 0::2] = 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kv = torch.zeros((n, 1, d), device="cuda")
    pool = [torch.zeros((1, 8, 1, d), device="cuda") for _ in range(2)]
    got, _, _ = kda.kda_cache_append_rotary(q.cuda(), kv, kv, i32(range(n + 1)), f.cuda(), *pool, i32([[-1]] * n), i32(pos),
                                            interleaved=True)
    want = np.concatenate([rotate(q[i:i + 1], [p], f, True)[0] for i, p in enumerate(pos)])
    bound = 2 * np.pi * (2.0 ** -26 + 2.0 ** -32 + np.outer(pos, f.double().numpy()) * 2.0 ** -54) + 2.0 ** -23
    assert (np.abs(got.double().cpu().numpy() - want) <= np.repeat(bound, 2, 1)[:, None]).all()
