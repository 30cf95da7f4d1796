"""kda_cache_commit and kda_cache_append move rows and compute nothing: every
byte of the pool must be what a plain loop leaves there."""
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


def pools(layers, P, page, Hkv, d, dtype, gap=0):
    """K and V pools; with a gap, both live in one buffer of pages."""
    if not gap:
        return [torch.full((layers, P, page, Hkv, d), 9.0 + i, dtype=dtype, device="cuda") for i in range(2)]
    both = torch.full((P, layers, 2, page, Hkv, d), 9.0, dtype=dtype, device="cuda")
    return [both[:, :, i].transpose(0, 1) for i in range(2)]


def table_for(room, page, rng, spare=2):
    need = [max(1, -(-int(x) // page)) for x in room]
    ids = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(room), max(need)), -1, np.int32)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = ids[at:at + c]
        at += c
    return table, len(ids)


def put(pool, x, table, pos, page):
    p = pos // page
    if p < table.shape[0] and 0 <= table[p] < pool.shape[1]:
        pool[:, int(table[p]), pos % page] = x


COMMIT = [(1, 1, 1, 1, 16, 1), (3, 5, 7, 2, 128, 16), (2, 40, 33, 3, 64, 48), (1, 9, 64, 8, 128, 64),
          (2, 3, 200, 1, 32, 7)]


@pytest.mark.parametrize("layers,N,Ts,Hkv,d,page", COMMIT)
@pytest.mark.parametrize("dtype,gap", [(BF16, 0), (F32, 1)])
def test_commit(kda, layers, N, Ts, Hkv, d, page, dtype, gap):
    rng = np.random.default_rng(N + Ts)
    lengths = rng.integers(0, 100, N).astype(np.int32)
    count = rng.integers(0, Ts + 1, N).astype(np.int32)
    count[0] = Ts
    path = np.full((N, Ts), -1, np.int32)
    for n in range(N):
        path[n, :count[n]] = np.sort(rng.permutation(Ts)[:count[n]])
    table, P = table_for(lengths + count, page, rng)
    k, v = (torch.randn((layers, N, Ts, Hkv, d), device="cuda").to(dtype) for _ in range(2))
    kc, vc = pools(layers, P, page, Hkv, d, dtype, gap)
    want = [kc.clone(), vc.clone()]
    for n in range(N):
        for i in range(count[n]):
            for pool, x in zip(want, (k, v)):
                put(pool, x[:, n, path[n, i]], table[n], int(lengths[n]) + i, page)
    c = lambda x: torch.from_numpy(x).cuda()
    new = kda.kda_cache_commit(k, v, c(path), c(count), kc, vc, c(table), c(lengths))
    torch.cuda.synchronize()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert new.tolist() == (lengths + count).tolist()


@pytest.mark.parametrize("layers,lens,Hkv,d,page", [(1, [1], 1, 16, 16), (2, [0, 33, 0, 7, 130, 0], 2, 64, 24),
                                                    (1, [500, 1, 64], 8, 128, 64), (3, [0], 1, 32, 8)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append(kda, layers, lens, Hkv, d, page, dtype):
    rng = np.random.default_rng(sum(lens))
    N, T = len(lens), sum(lens)
    lengths = rng.integers(0, 50, N).astype(np.int32)
    table, P = table_for(lengths + lens, page, rng)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = (torch.randn((layers, T, Hkv, d), device="cuda").to(dtype) for _ in range(2))
    kc, vc = pools(layers, P, page, Hkv, d, dtype)
    want = [kc.clone(), vc.clone()]
    for n in range(N):
        for i in range(lens[n]):
            for pool, x in zip(want, (k, v)):
                put(pool, x[:, cu[n] + i], table[n], int(lengths[n]) + i, page)
    c = lambda x: torch.from_numpy(x).cuda()
    new = kda.kda_cache_append(k, v, c(cu), kc, vc, c(table), c(lengths))
    torch.cuda.synchronize()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert new.tolist() == (lengths + lens).tolist()


def test_rows_without_a_place_are_dropped(kda):
    # past the table, to a page that does not exist, from a node that does not
    # exist; counts beyond Ts are Ts
    page, Ts = 4, 6
    table = np.array([[0, -1], [7, 1]], np.int32)
    lengths = np.array([3, 3], np.int32)
    path = np.array([[0, 1, 2, 3, 4, 5], [0, 9, 2, -1, 4, 5]], np.int32)
    count = np.array([50, 6], np.int32)
    k, v = (torch.randn((1, 2, Ts, 1, 16), device="cuda") for _ in range(2))
    kc, vc = pools(1, 2, page, 1, 16, F32)
    want = [kc.clone(), vc.clone()]
    for pool, x in zip(want, (k, v)):
        put(pool, x[:, 0, 0], table[0], 3, page)
        for i in (2, 4):
            put(pool, x[:, 1, i], table[1], 3 + i, page)
    c = lambda a: torch.from_numpy(a).cuda()
    new = kda.kda_cache_commit(k, v, c(path), c(count), kc, vc, c(table), c(lengths))
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert new.tolist() == [9, 9]
    # negative counts and lengths write nothing
    kc2, vc2 = pools(1, 2, page, 1, 16, F32)
    new = kda.kda_cache_commit(k, v, None, c(np.array([-4, 2], np.int32)), kc2, vc2, c(table),
                               c(np.array([3, -1], np.int32)))
    assert torch.all(kc2 == 9) and torch.all(vc2 == 10) and new[0].item() == 3


def test_append_with_a_broken_cu_seqlens_stays_inside(kda):
    # rows that cu_seqlens gives to no sequence are dropped
    k, v = (torch.randn((1, 8, 1, 16), device="cuda") for _ in range(2))
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    lengths = torch.zeros(2, dtype=torch.int32, device="cuda")
    for cu in ([0, 3, 5], [2, 3, 8], [0, 6, 4]):
        kc, vc = pools(1, 4, 4, 1, 16, F32)
        kda.kda_cache_append(k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), kc, vc, table, lengths)
        torch.cuda.synchronize()
        if cu == [0, 3, 5]:
            assert torch.equal(kc[0, 0, :3], k[0, :3]) and torch.equal(kc[0, 2, :2], k[0, 3:5])
            assert torch.all(kc[0, 1] == 9) and torch.all(kc[0, 2, 2:] == 9)


def test_what_was_appended_is_what_attention_reads(kda):
    from tests._tree import AttentionInputs
    inp = AttentionInputs(2, 1, 4, 2, 64, 16, [37, 20], BF16, seed=3, poison=False)
    args = inp.on("cuda")
    want = kda.kda_tree_attention(**args)
    rows = []
    for name in ("k_cache", "v_cache"):
        flat = [args[name][inp.table[n, i // 16], i % 16] for n in range(2) for i in range(inp.lengths[n])]
        rows.append(torch.stack(flat)[None])
    kc, vc = (torch.full_like(args[x], float("nan")) for x in ("k_cache", "v_cache"))
    cu = torch.tensor([0, 37, 57], dtype=torch.int32, device="cuda")
    new = kda.kda_cache_append(*rows, cu, kc[None], vc[None], args["page_table"], torch.zeros_like(args["lengths"]))
    args.update(k_cache=kc, v_cache=vc, lengths=new)
    assert torch.equal(kda.kda_tree_attention(**args), want)


def test_offsets_beyond_32_bits(kda):
    page, Hkv, d = 64, 8, 128
    P = (1 << 31) // (page * Hkv * d) + 3
    kc, vc = (torch.empty((1, P, page, Hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    kc[:, -2:], vc[:, -2:] = 1.0, 2.0
    k, v = (torch.randn((1, 1, 3, Hkv, d), device="cuda").to(BF16) for _ in range(2))
    table = torch.tensor([[P - 2, P - 1]], dtype=torch.int32, device="cuda")
    kda.kda_cache_commit(k, v, None, None, kc, vc, table, torch.tensor([62], dtype=torch.int32, device="cuda"))
    for pool, x, fill in ((kc, k, 1.0), (vc, v, 2.0)):
        tail = pool[0, -2:].reshape(-1, Hkv, d)
        assert torch.equal(tail[62:65], x[0, 0])
        assert torch.all(tail[:62] == fill) and torch.all(tail[65:] == fill)


@pytest.mark.parametrize("cu", [[0, 3, 5], [2, 3, 8], [0, 6, 4], [0, 9, 12], [5, 2, 8], [-2, 3, 8], [9, 9, 9]])
def test_append_of_any_cu_seqlens_counts_the_rows_that_it_wrote(kda, cu):
    # rows before 0 and from T on do not exist, a sequence that ends before it
    # begins has none
    T, page = 8, 4
    k, v = (torch.randn((2, T, 1, 16), device="cuda") for _ in range(2))
    table = np.arange(6, dtype=np.int32).reshape(2, 3)
    lengths = np.array([3, 1], np.int32)
    kc, vc = pools(2, 6, page, 1, 16, F32)
    want, count = [kc.clone(), vc.clone()], []
    for n in range(2):
        own = range(max(cu[n], 0), min(cu[n + 1], T))
        count.append(len(own))
        for i, r in enumerate(own):
            for pool, x in zip(want, (k, v)):
                put(pool, x[:, r], table[n], int(lengths[n]) + i, page)
    c = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
    new = kda.kda_cache_append(k, v, c(cu), kc, vc, c(table), c(lengths))
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert new.tolist() == (lengths + count).tolist()


@pytest.mark.parametrize("layers,P,page,Hkv,odd", [(2, 1, 8, 2, 1), (1, 3, 8, 2, 0), (2, 3, 1, 2, 2), (2, 3, 8, 1, 3)])
def test_strides_of_dimensions_of_one_do_not_matter(kda, layers, P, page, Hkv, odd):
    kc, vc = pools(layers, P, page, Hkv, 16, F32)
    k, v = (torch.randn((layers, 1, 2, Hkv, 16), device="cuda") for _ in range(2))
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    stride = list(kc.stride())
    stride[odd] = 12345
    kda.kda_cache_commit(k, v, None, None, kc.as_strided(kc.shape, stride), vc.as_strided(vc.shape, stride), table,
                         torch.tensor([1], dtype=torch.int32, device="cuda"))
    for pool, x in ((kc, k), (vc, v)):
        rows = pool.reshape(layers, P * page, Hkv, 16)
        places = [i for i in (1, 2) if i < P * page]
        assert torch.equal(rows[:, places], x[:, 0, :len(places)])
        assert torch.all(rows[:, [i for i in range(P * page) if i not in places]] == (9 if x is k else 10))
