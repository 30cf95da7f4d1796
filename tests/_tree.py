"""Float64 references of the calls that verify a tree of drafted tokens,
written as plain loops, and the inputs their tests share."""
import numpy as np
import torch


def lineage(parent, t):
    """Nodes from t up to the context; None when t is unused."""
    chain = []
    while t != -1:
        p = int(parent[t])
        if p < -1 or p >= t:
            return None
        chain.append(t)
        t = p
    return chain


def random_trees(N, Ts, rng, unused=True):
    """Random trees, some with unused slots at the end."""
    out = np.full((N, Ts), -2, np.int32)
    for n in range(N):
        used = Ts - int(rng.integers(0, Ts // 2 + 1)) if unused and n % 2 else Ts
        for t in range(used):
            out[n, t] = -1 if t == 0 else max(-1, t - 1 - int(rng.integers(0, 6)))
    return out


class AttentionInputs:
    """Inputs of one kda_tree_attention call.  The cache rows no sequence owns
    (spare pages, rows past a length) hold NaN."""

    def __init__(self, N, Ts, Hq, Hkv, d, page, lengths, dtype, seed=0, parent="tree", gap=0,
                 poison=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        f = lambda *s: torch.randn(s, generator=g)
        self.lengths = np.asarray(lengths, np.int32)
        need = [max(1, -(-int(x) // page)) for x in lengths]
        P = sum(need) + 2
        ids = rng.permutation(P)
        self.table = np.full((N, max(need)), -1, np.int32)
        at = 0
        for n, c in enumerate(need):
            self.table[n, :c] = ids[at:at + c]
            at += c
        self.q = (1.5 * f(N, Ts, Hq, d)).to(dtype)
        self.k, self.v = f(N, Ts, Hkv, d).to(dtype), f(N, Ts, Hkv, d).to(dtype)
        size = page * Hkv * d + gap
        pool = [f(P, size).to(dtype) for _ in range(2)]
        if poison:
            for t in pool:
                rows = t[:, :page * Hkv * d].view(P, page, Hkv, d)
                live = torch.zeros(P, page, dtype=torch.bool)
                for n in range(N):
                    for i in range(int(lengths[n])):
                        live[self.table[n, i // page], i % page] = True
                rows[~live] = float("nan")
                if gap:
                    t[:, page * Hkv * d:] = float("nan")
        self.pool = pool
        self.shape = (P, page, Hkv, d)
        if isinstance(parent, str):
            parent = None if parent == "chain" else random_trees(N, Ts, rng)
        self.parent = parent
        self.scale = d ** -0.5

    def cache(self, device):
        P, page, Hkv, d = self.shape
        out = []
        for t in self.pool:
            t = t.to(device)
            out.append(t.as_strided(self.shape, (t.shape[1], Hkv * d, d, 1)))
        return out

    def on(self, device):
        i32 = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(device)
        kc, vc = self.cache(device)
        return dict(q=self.q.to(device), k=self.k.to(device), v=self.v.to(device), k_cache=kc,
                    v_cache=vc, page_table=i32(self.table), lengths=i32(self.lengths),
                    parent=i32(self.parent), scale=self.scale)


def attention_reference(inp):
    """(o, sum of p |v|) in float64, [N, Ts, Hq, d] each."""
    q, k, v = (x.double().numpy() for x in (inp.q, inp.k, inp.v))
    kc, vc = (x.double().numpy() for x in inp.cache("cpu"))
    N, Ts, Hq, d = q.shape
    P, page, Hkv, _ = kc.shape
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    for n in range(N):
        L = int(inp.lengths[n])
        rows = [(inp.table[n, i // page], i % page) for i in range(L)]
        rows = [(p, s) for p, s in rows if 0 <= p < P]
        ps, ss = [r[0] for r in rows], [r[1] for r in rows]
        parent = np.arange(-1, Ts - 1) if inp.parent is None else inp.parent[n]
        for t in range(Ts):
            chain = lineage(parent, t)
            if chain is None:
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                keys = np.concatenate([kc[ps, ss, g].reshape(-1, d), k[n, chain, g]])
                vals = np.concatenate([vc[ps, ss, g].reshape(-1, d), v[n, chain, g]])
                x = inp.scale * (keys @ q[n, t, h])
                with np.errstate(invalid="ignore"):
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    o[n, t, h], mag[n, t, h] = p @ vals, p @ np.abs(vals)
    return o, mag
