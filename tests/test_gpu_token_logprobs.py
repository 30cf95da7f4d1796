"""kda_token_logprobs against float64.

Bound of a log probability or an entropy: a thread adds up to V / 256 + 32 terms
one after the other and a joining tree follows, each addition off by 2^-24 of
the sum, and each term by a few 2^-24; the logits and lse themselves by 2^-24 of
their size.  So (V / 256 + 64) 2^-23 + 2^-22 max|x|, for the entropy times
(1 + H), whose second sum has terms of that size."""
import numpy as np
import pytest
import torch

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


def reference(x, tokens, K):
    x = x.double().cpu().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        m = x.max(-1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0)
        lse = m + np.log(np.exp(x - m).sum(-1, keepdims=True))
        p = np.exp(x - lse)
        H = (lse[:, 0] - np.where(p > 0, p * x, 0).sum(-1))
    order = np.argsort(-x, axis=-1, kind="stable")[:, :K]
    logp = np.take_along_axis(x, tokens, -1) - lse
    return logp, H, order, np.take_along_axis(x, order, -1) - lse


def check(kda, x, J=3, K=8, seed=0, threads=256):
    T, V = x.shape
    K = min(K, V)
    tokens = np.random.default_rng(seed).integers(0, V, (T, J)).astype(np.int32)
    logp, H, ids, top = kda.kda_token_logprobs(x, torch.from_numpy(tokens).cuda(), K)
    torch.cuda.synchronize()
    rl, rH, rids, rtop = reference(x, tokens, K)
    assert np.array_equal(ids.cpu().numpy(), rids)
    big = np.abs(x.double().cpu().numpy())
    big = float(big[np.isfinite(big)].max())
    tol = (V / threads + 64) * 2.0 ** -23 + 2.0 ** -22 * big
    for got, want in ((logp, rl), (top, rtop)):
        got = got.double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        live = np.isfinite(want)
        assert np.all(np.abs(got - want)[live] <= tol)
    assert np.all(np.abs(H.double().cpu().numpy() - rH) <= tol * (1 + rH))


def logits(T, V, dtype, seed, stride=None, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, stride or V), generator=g, device="cuda") * scale
    return x.to(dtype)[:, :V]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(1, 1), (2, 7), (3, 255), (1, 8192), (2, 8193), (5, 16385),
                                 (1, 50257), (3, 131072), (700, 1000), (65, 33000)])
def test_matches_reference(kda, dtype, T, V):
    check(kda, logits(T, V, dtype, T + V), K=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("stride", [1001, 1003, 1007, 1008, 1024])
def test_row_strides(kda, dtype, stride):
    check(kda, logits(9, 1001, dtype, stride, stride))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [0, 1, 31, 32])
def test_counts_of_alternatives(kda, dtype, K):
    check(kda, logits(4, 20000, dtype, 3), K=K)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 9000, 40000])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values", "steps"])
def test_ties_and_sorted_rows(kda, dtype, V, kind):
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = {"equal": i * 0 + 1.5, "rising": i / V * 8 - 4, "falling": 4 - i / V * 8,
           "two values": (i % 5 == 3).float(), "steps": torch.floor(i / 100) * 0.125}[kind]
    check(kda, row.to(dtype).expand(3, V).contiguous(), K=32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [77, 9001, 66000])
def test_masked_logits(kda, dtype, V):
    x = logits(4, V, dtype, 5)
    x[0, 1:] = float("-inf")                        # one token left
    x[1, ::2] = float("-inf")
    x[2, : V // 2] = float("-inf")
    x[3] = torch.finfo(dtype).min                   # the lowest finite value everywhere
    check(kda, x[:3].contiguous(), K=8)
    _, H, ids, top = kda.kda_token_logprobs(x, None, 2)
    assert abs(H[3].item() - np.log(V)) < 1e-4 and ids[3].tolist() == [0, 1]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [50, 33000])
def test_rows_with_nothing_and_rows_with_nan(kda, dtype, V):
    x = logits(4, V, dtype, 6)
    x[0] = float("-inf")
    x[1, 3] = float("nan")
    x[2, V - 1] = float("inf")
    want = torch.where(torch.isnan(x), float("-inf"), x.float()).double().cpu().numpy()
    tok = torch.tensor([[0, 5]] * 4, dtype=torch.int32, device="cuda")
    logp, H, ids, top = kda.kda_token_logprobs(x, tok, 4)
    assert torch.all(torch.isneginf(logp[0])) and H[0] == 0 and ids[0].tolist() == [0, 1, 2, 3]
    assert torch.all(torch.isneginf(top[0]))
    for r in (1, 2):
        assert torch.isnan(H[r])
        assert ids[r].tolist() == np.argsort(-want[r], kind="stable")[:4].tolist()
    assert torch.all(torch.isnan(logp[1]))
    assert torch.all(torch.isfinite(logp[3])) and torch.isfinite(H[3])


def test_tokens_outside_the_vocabulary_and_no_tokens(kda):
    x = logits(2, 500, F32, 7)
    tok = torch.tensor([[-1, 500, 3], [2, 1 << 30, -9]], dtype=torch.int32, device="cuda")
    logp, *_ = kda.kda_token_logprobs(x, tok)
    want = torch.log_softmax(x.double(), -1)
    assert torch.isneginf(logp[0, :2]).all() and torch.isneginf(logp[1, 1:]).all()
    assert abs(logp[0, 2] - want[0, 3]) < 1e-4 and abs(logp[1, 0] - want[1, 2]) < 1e-4
    empty, H, ids, top = kda.kda_token_logprobs(x)
    assert empty.shape == (2, 0) and ids.shape == top.shape == (2, 0)
    assert torch.allclose(H.double(), -(want.exp() * want).sum(-1), atol=1e-4)


def test_offsets_beyond_32_bits(kda):
    T, V = 2, 1000
    pool = torch.zeros((1 << 31) + 8 * V, dtype=BF16, device="cuda")
    x = pool.as_strided((T, V), (1 << 31, 1))
    x.copy_(logits(T, V, BF16, 8))
    check(kda, x)


def test_another_stream(kda):
    x = logits(3, 40000, BF16, 9)
    a = kda.kda_token_logprobs(x, None, 5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = kda.kda_token_logprobs(x, None, 5)
    s.synchronize()
    for y, z in zip(a, b):
        assert torch.equal(y, z)


# Many rows, whose blocks have 128 threads.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 130, 5003, 20000])
@pytest.mark.parametrize("K", [1, 32])
def test_many_rows(kda, dtype, V, K):
    check(kda, logits(900, V, dtype, V + K), K=K, threads=128)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values"])
def test_many_rows_of_ties_and_sorted_values(kda, dtype, kind):
    V = 7001
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = {"equal": i * 0 + 1.5, "rising": i / V * 8 - 4, "falling": 4 - i / V * 8,
           "two values": (i % 5 == 3).float()}[kind]
    x = row.to(dtype).expand(700, V).contiguous()
    x[1::7, ::2] = float("-inf")
    check(kda, x, K=32, threads=128)


# Finite values as masks.  The bound of an unmasked token's log probability and of
# the entropy goes by the unmasked logits alone: a masked token's probability is 0.
# A masked token's own log probability, and all of a row of nothing but masks, are
# off by what fp32 holds of a number of the mask's size, 2^-23 of it.
FILLS = [-1e4, -1e9, -1e10, -1e12, -1e15, -1e20, -1e30, -1e32, -1e34, -1e36, "lowest"]


def check_finite(kda, x, K, size, threads):
    """Like check, row by row, with ``size`` the magnitude of each row's largest logits.
    Rows repeat from len(size) on and, where they start at the same place in 16 bytes,
    have to give the same bits again."""
    T, V = x.shape
    rows = len(size)
    tokens = np.random.default_rng(V).integers(0, V, (rows, 5)).astype(np.int32)
    tokens[:, 3], tokens[:, 4] = 0, V - 1
    got = kda.kda_token_logprobs(x, torch.from_numpy(tokens).cuda().repeat(T // rows, 1), K)
    for y in got:
        if x.stride(0) % 8 == 0:
            assert torch.equal(y, y[:rows].repeat((T // rows,) + (1,) * (y.dim() - 1)))
    logp, H, ids, top = (y[:rows].double().cpu().numpy() for y in got)
    # relative to the maximum, as float64 would cancel: all four are the same
    top_of = x[:rows].double().amax(-1, keepdim=True)
    rl, rH, rids, rtop = reference(x[:rows].double() - top_of, tokens, K)
    assert np.array_equal(ids, rids)
    size = np.asarray(size, float)[:, None]
    sums = (V / threads + 64) * 2.0 ** -23
    tol = sums + 2.0 ** -22 * size
    for y, want in ((logp, rl), (top, rtop)):
        assert np.all(np.abs(y - want) <= tol + 2.0 ** -23 * np.abs(want)), (y - want, want)
    bound = np.where(size > 1e3, sums, tol)[:, 0]   # differences alone
    assert np.all(np.abs(H - rH) <= bound * (1 + rH)), (H, rH)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("repeat,V", [(1, 50), (1, 1000), (1, 131072), (100, 1000), (100, 5003)])
def test_finite_masks(kda, dtype, fill, repeat, V):
    fill = torch.finfo(dtype).min if fill == "lowest" else fill
    x = logits(7, V, dtype, 11)
    i = torch.arange(V, device="cuda")
    masked = torch.stack([i < 0, i != V // 2, (i // 64) % 2 == 0, i >= V // 2, i < V // 2, i < V - 3, i >= 0])
    x[masked] = fill
    nothing = masked.all(-1, keepdim=True)          # nothing but masks
    size = torch.where(masked & ~nothing, 0, x.float().abs()).amax(-1).tolist()
    rows = torch.zeros((7 * repeat, -(-V // 8) * 8), dtype=dtype, device="cuda")[:, :V]
    rows.copy_(x.repeat(repeat, 1))
    check_finite(kda, rows, 8, size, 128 if repeat > 1 else 256)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset", [1e3, 1e6, 1e8, 1e10, 1e20, 1e30, 1e36, 1e37, 1e38])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("V", [1, 6, 1000, 50001])
def test_large_logits(kda, dtype, offset, sign, V):
    # two values 2^-6 of their size apart
    i = torch.arange(V, device="cuda")
    big = torch.tensor(sign * offset, device="cuda").to(dtype).float()
    x = torch.stack([torch.where((i + r) % 7 == 0, big, big * (1 - 2.0 ** -6)) for r in range(3)])
    x = x.to(dtype)
    check_finite(kda, x, min(V, 8), x.float().abs().amax(-1).tolist(), 256)


@pytest.mark.parametrize("centre", [-(1 << 20), -(1 << 18), 1 << 16, 1 << 20, 1 << 21])
@pytest.mark.parametrize("V", [5, 1000, 50001])
def test_large_logits_close_to_each_other(kda, centre, V):
    # threads' maxima on either side of a power of two, all of them weighty
    g = torch.Generator(device="cuda").manual_seed(V)
    x = centre + 0.5 * torch.randint(-8, 9, (4, V), generator=g, device="cuda").float()
    check_finite(kda, x, 5, [abs(centre) + 4] * 4, 256)


@pytest.mark.parametrize("T", [1, 700])
def test_tokens_outside_the_vocabulary_in_any_column_of_any_row(kda, T):
    # more columns than a block has threads; a NaN row and one of nothing
    V, J = 500, 600
    x = logits(T, V, F32, 12)
    tok = torch.randint(-V // 2, V + V // 2, (T, J), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    outside = ((tok < 0) | (tok >= V)).cuda()
    for fill in (None, float("nan"), float("inf"), float("-inf")):
        if fill is not None:
            x[-1, 7 if fill == fill and fill > 0 else slice(None)] = fill
        logp, *_ = kda.kda_token_logprobs(x, tok.cuda())
        assert torch.isneginf(logp[outside]).all()
        inside = logp[-1][~outside[-1]]
        if fill is None:
            assert torch.isfinite(inside).all()
        elif fill == float("-inf"):
            assert torch.isneginf(inside).all()
        else:
            assert torch.isnan(inside).all()
        x[-1] = logits(1, V, F32, 13)[0]
