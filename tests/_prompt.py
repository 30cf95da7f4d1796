"""Float64 references of the calls that take a prompt and its answer through the
softmax layers, written as plain loops over sequences and heads, and the inputs their
tests share."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def spans(cu, rows):
    """Rows of each sequence, as far as they exist."""
    return [range(max(int(a), 0), max(min(int(b), rows), max(int(a), 0))) for a, b in zip(cu, cu[1:])]


def softmax_rows(x, v):
    """softmax(x) v and softmax(x) |v| in float64; rows of nothing but -inf give 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        seen = ~(np.isneginf(x))
        top = np.where(seen.any(-1), np.where(seen, x, -np.inf).max(-1, initial=-np.inf), 0.0)
        p = np.where(seen, np.exp(x - top[:, None]), 0.0)
        total = p.sum(-1, keepdims=True)
        p = p / np.where(total == 0, 1.0, total)
        if np.isfinite(v).all():
            return p @ v, p @ np.abs(v)
        o, mag = np.zeros((x.shape[0], v.shape[1])), np.zeros((x.shape[0], v.shape[1]))
        for i in range(x.shape[0]):                # a hidden row's infinities stay hidden
            o[i], mag[i] = p[i, seen[i]] @ v[seen[i]], p[i, seen[i]] @ np.abs(v[seen[i]])
        return o, mag


def prompt_reference(q, k, v, cu=None, cu_k=None, scale=None, o=None):
    """(o, sum of p |v|); rows of no sequence keep o's values."""
    q, k, v = (x.detach().double().cpu().numpy() for x in (q, k, v))
    T, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    cu = [0, T] if cu is None else list(cu)
    cu_k = cu if cu_k is None else list(cu_k)
    scale = d ** -0.5 if scale is None else scale
    o = np.zeros(q.shape) if o is None else o.double().cpu().numpy().copy()
    mag = np.zeros(q.shape)
    for rows, keys in zip(spans(cu, T), spans(cu_k, Tk)):
        i, j = np.arange(len(rows)), np.arange(len(keys))
        hidden = j[None, :] > i[:, None] + len(keys) - len(rows)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            with np.errstate(invalid="ignore", over="ignore"):
                x = scale * (q[rows.start:rows.stop, h] @ k[keys.start:keys.stop, g].T)
            x[hidden] = -np.inf
            a, b = softmax_rows(x, v[keys.start:keys.stop, g])
            o[rows.start:rows.stop, h], mag[rows.start:rows.stop, h] = a, b
    return o, mag


def rotate(x, pos, inv_freq, interleaved):
    """(rows x [n, h, d] turned to positions pos, |x| + |y| of each pair)."""
    y = x.detach().double().cpu().numpy().copy()
    mag = np.abs(y)
    f = inv_freq.double().cpu().numpy()
    r = 2 * len(f)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    # p f mod 2 pi, with p f itself exact in extended precision
    turn = np.fmod(np.asarray(pos, np.longdouble)[:, None] * f.astype(np.longdouble), 2 * np.longdouble(np.pi))
    c, s = (w.astype(np.float64)[:, None, :] for w in (np.cos(turn), np.sin(turn)))
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - w * s, u * s + w * c
    mag[..., a] = mag[..., b] = np.abs(u) + np.abs(w)
    return y, mag


def power_scale(top):
    """The scale of a block whose largest magnitude is `top`."""
    if not np.isfinite(top):
        return float("nan")
    if top == 0:
        return 0.0
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def table_for(room, page, rng, spare=2):
    """A page table over shuffled pages and the number of pages."""
    need = [max(1, -(-int(x) // page)) for x in room]
    ids = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(room), max(need)), -1, np.int32)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = ids[at:at + c]
        at += c
    return table, len(ids)


def eight_bits(x, block):
    """A pool [pages, page, h, d] (fp32) in 8 bits: values and scales."""
    pages, page, h, d = x.shape
    rows = x.view(pages, page // block, block, h, d)
    top = rows.abs().amax((2, 4))
    scales = torch.tensor([power_scale(t) for t in top.flatten().tolist()]).view(top.shape)
    by = torch.where(scales > 0, scales, torch.ones_like(scales))[:, :, None, :, None]
    return (rows / by).to(E4M3).view(x.shape), scales


def dequantised(cache, scales):
    """The values that a pool of 8 bits stands for, in float64."""
    pages, page, h, d = cache.shape
    x = cache.view(torch.uint8).cpu().view(E4M3).double()
    return x * scales.cpu().double().repeat_interleave(page // scales.shape[1], 1)[..., None]


def cache_reference(q, k, v, table, lengths, scale=None):
    """(o, sum of p |v|) of the newest tokens; k, v: pools [pages, page, h, d] in float64."""
    q = q.detach().double().cpu().numpy()
    k, v = k.numpy(), v.numpy()
    N, Ts, Hq, d = q.shape
    pages, page, Hkv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    for n in range(N):
        L = min(max(int(lengths[n]), 0), table.shape[1] * page)
        where = [(table[n, i // page], i % page, i) for i in range(L) if 0 <= table[n, i // page] < pages]
        ps, ss, pos = ([w[c] for w in where] for c in range(3))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            if not where:
                continue
            with np.errstate(invalid="ignore"):
                x = scale * (q[n, :, h] @ k[ps, ss, g].T)
            x[np.array(pos)[None, :] > L - Ts + np.arange(Ts)[:, None]] = -np.inf
            o[n, :, h], mag[n, :, h] = softmax_rows(x, v[ps, ss, g])
    return o, mag
