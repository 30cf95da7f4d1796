"""Cases of the operators that verify a tree of drafted tokens in a model that
mixes KDA layers with softmax attention over a paged cache:

  tree_attention   kda_tree_attention: drafted nodes attend to their sequence's
                   cached context and to their ancestors in the tree
  decode_tree      kda_decode_tree: the KDA step of every drafted node from its
                   parent's state
  token_logprobs   kda_token_logprobs: log probabilities of given tokens, the
                   entropy and the largest alternatives of each logits row
  cache_commit     kda_cache_commit: the accepted path's rows into cache pages
  cache_append     kda_cache_append: a prompt's rows into cache pages

Each case runs either in the library (``own`` true) or in a plain form of
elementary torch operations in fp32; ``exact`` evaluates the definitions in
float64.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one request, one new token, a short context: the latency of a call
        dict(name="attn_one_token", op="tree_attention", n=1, ts=1, hq=32, hkv=8, d=128,
             page=16, lo=1023, hi=1023, ragged=False, dtype="bf16"),
        # a serving batch verifying trees of up to 16 nodes, ragged contexts
        # and draft sizes
        dict(name="attn_verify_32x16", op="tree_attention", n=32, ts=16, hq=32, hkv=8, d=128,
             page=64, lo=0, hi=16384, ragged=True, dtype="bf16"),
        # few long contexts, wide trees: 512 query rows per cache head
        dict(name="attn_wide_tree", op="tree_attention", n=4, ts=64, hq=64, hkv=8, d=128,
             page=128, lo=32768, hi=65536, ragged=False, dtype="bf16"),
        # fp32, small heads without sharing, pages that are no power of two
        dict(name="attn_fp32_d64", op="tree_attention", n=8, ts=5, hq=16, hkv=16, d=64,
             page=48, lo=100, hi=4097, ragged=True, dtype="fp32"),
        # one request's KDA layer, a small tree
        dict(name="kda_tree_one", op="decode_tree", n=1, ts=8, h=32, d=128, ragged=False,
             dtype="bf16"),
        # a serving batch's KDA layer, trees of up to 16 nodes
        dict(name="kda_tree_64x16", op="decode_tree", n=64, ts=16, h=32, d=128, ragged=True,
             dtype="bf16"),
        # fp32, smaller heads, odd counts
        dict(name="kda_tree_fp32_d64", op="decode_tree", n=37, ts=5, h=9, d=64, ragged=True,
             dtype="fp32"),
        # one sampled token of one request
        dict(name="logprobs_one_row", op="token_logprobs", t=1, v=32000, pad=0, j=1, k=1,
             dtype="fp32"),
        # the rows of a verified batch: each node's children and alternatives
        dict(name="logprobs_verify", op="token_logprobs", t=512, v=131072, pad=0, j=4, k=8,
             dtype="bf16"),
        # scoring a prompt, fp32 logits, an odd vocabulary in padded rows
        dict(name="logprobs_prompt", op="token_logprobs", t=4096, v=50257, pad=47, j=1, k=20,
             dtype="fp32"),
        # eight layers' accepted rows of a verified batch
        dict(name="commit_32x16", op="cache_commit", layers=8, n=32, ts=16, hkv=8, d=128,
             page=64, lo=0, hi=512, dtype="bf16"),
        # a packed prefill of 16 prompts into empty pages, one layer
        dict(name="append_prefill", op="cache_append", layers=1, n=16, lo=512, hi=16384, hkv=8,
             d=128, page=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree_attention", "tree_attention", "decode_tree", "token_logprobs",
                     "cache_commit", "cache_append"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "tree_attention":
        ts, g = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 7, 8])
        hkv = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 128, 128]) if dtype == "bf16" else rng.choice([16, 32, 64, 128])
        if dtype == "fp32":
            ts = min(ts, 24)
        n = _log_int(rng, 1, 32)
        # the context rows and products stay within the listed cases'
        most = min(65536, (1 << 21) // (n * hkv), (1 << 29) // (n * hkv * ts * g))
        if dtype == "fp32":
            most = min(most, max(64, (1 << 25) // (n * hkv * ts * g)))
        hi = _log_int(rng, 16, max(16, most))
        return dict(op=op, n=n, ts=ts, hq=g * hkv, hkv=hkv, d=d,
                    page=rng.choice([16, 24, 32, 48, 64, 100, 128, 256]),
                    lo=rng.choice([0, hi // 2, hi]), hi=hi, ragged=rng.random() < 0.5,
                    dtype=dtype)
    if op == "decode_tree":
        d, h, ts = rng.choice([16, 32, 64, 128, 128]), rng.choice([1, 3, 8, 16, 32]), _log_int(rng, 1, 24)
        n = _log_int(rng, 1, max(1, min(256, (1 << 29) // (h * (ts + 1) * d * d))))
        return dict(op=op, n=n, ts=ts, h=h, d=d, ragged=rng.random() < 0.5, dtype=dtype)
    if op == "token_logprobs":
        v = rng.choice([1000, 32000, 50257, 65537, 100277, 131072, 163840])
        t = _log_int(rng, 1, max(1, (1 << 28) // v // (2 if dtype == "fp32" else 1)))
        return dict(op=op, t=t, v=v, pad=rng.choice([0, 0, 5, 47]), j=rng.choice([1, 2, 5, 16]),
                    k=rng.choice([0, 1, 5, 8, 20, 32]), dtype=dtype)
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128, 128])
    page = rng.choice([16, 24, 48, 64, 128])
    if op == "cache_commit":
        layers, n, ts = _log_int(rng, 1, 24), _log_int(rng, 1, 48), _log_int(rng, 1, 64)
        most = max(1, (1 << 27) // (layers * n * hkv * d))
        return dict(op=op, layers=layers, n=n, ts=ts, hkv=hkv, d=d, page=page, lo=0,
                    hi=_log_int(rng, 1, min(512, most)), dtype=dtype)
    layers, n = _log_int(rng, 1, 4), _log_int(rng, 1, 24)
    hi = _log_int(rng, 1, max(1, min(16384, (1 << 26) // (layers * n * hkv * d))))
    return dict(op=op, layers=layers, n=n, lo=rng.choice([0, hi // 2, hi]), hi=hi, hkv=hkv, d=d,
                page=page, dtype=dtype)


# --------------------------------------------------------------- the inputs
def _spread(lo, hi, n):
    """n lengths evenly spread over [lo, hi] (the same total for every seed)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _used_counts(case):
    """Drafted nodes per sequence: all, or between half of them and all."""
    n, ts = case["n"], case["ts"]
    return _spread((ts + 1) // 2, ts, n) if case["ragged"] else [ts] * n


def _trees(case, rnd):
    """parent[n][t]: -1 for a child of the context, -2 for an unused slot.
    Drafters extend recent nodes more often than old ones."""
    used = _used_counts(case)
    rnd.shuffle(used)
    return [[-2 if t >= u else (-1 if t == 0 else max(-1, t - int(rnd.expovariate(0.4)) - 1))
             for t in range(case["ts"])] for u in used]


def _pages(lengths, page, rnd):
    """A page table over shuffled pages and the number of pages."""
    need = [max(1, -(-x // page)) for x in lengths]
    ids = list(range(sum(need) + 3))
    rnd.shuffle(ids)
    width, rows, at = max(need), [], 0
    for c in need:
        rows.append(ids[at:at + c] + [-1] * (width - c))
        at += c
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), len(ids)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rnd = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    s = dict(case)
    if op == "tree_attention":
        n, ts, d = case["n"], case["ts"], case["d"]
        lengths = _spread(case["lo"], case["hi"], n)
        rnd.shuffle(lengths)
        s["page_table"], pages = _pages(lengths, case["page"], rnd)
        s["lengths"], s["parent"] = _i32(lengths), _i32(_trees(case, rnd))
        s["q"] = normal(n, ts, case["hq"], d).mul_(1.5).to(dt)
        s["k"], s["v"] = normal(n, ts, case["hkv"], d).to(dt), normal(n, ts, case["hkv"], d).to(dt)
        cache = (pages, case["page"], case["hkv"], d)
        s["k_cache"], s["v_cache"] = normal(*cache).to(dt), normal(*cache).to(dt)
        s["scale"] = d ** -0.5
    elif op == "decode_tree":
        n, ts, h, d = case["n"], case["ts"], case["h"], case["d"]
        k = normal(n, ts, h, d)
        s["q"] = normal(n, ts, h, d).mul_(d ** -0.5).to(dt)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = normal(n, ts, h, d).to(dt)
        s["log_alpha"] = -torch.nn.functional.softplus(normal(n, ts, h, d) - 3.0)
        s["beta"] = torch.sigmoid(normal(n, ts, h))
        s["S"] = normal(n, h, d, d).mul_(0.1)
        s["parent"] = _i32(_trees(case, rnd))
        # the slots of unused nodes keep what they hold
        s["states"] = torch.zeros((n, ts, h, d, d), device="cuda")
    elif op == "token_logprobs":
        t, v = case["t"], case["v"]
        # a model's logits: a few tokens well above the rest
        rows = torch.empty((t, v + case["pad"]), dtype=dt, device="cuda")
        for i in range(0, t, 512):
            x = normal(min(512, t - i), v + case["pad"])
            rows[i:i + 512] = (x * 2.0 + (x > 3.0) * x * 2.0).to(dt)
        s["logits"] = rows[:, :v]
        s["tokens"] = torch.randint(0, v, (t, case["j"]), generator=gen, device="cuda",
                                    dtype=torch.int32)
    else:
        n, hkv, d, layers = case["n"], case["hkv"], case["d"], case["layers"]
        lens = _spread(case["lo"], case["hi"], n)
        rnd.shuffle(lens)
        if op == "cache_commit":
            ts, start = case["ts"], lens
            count = _spread(0, ts, n)
            rnd.shuffle(count)
            path = [sorted(rnd.sample(range(ts), c)) + [-1] * (ts - c) for c in count]
            s["path"], s["count"] = _i32(path), _i32(count)
            rows, room = (layers, n, ts, hkv, d), [x + ts for x in lens]
        else:
            cu = [0]
            for x in lens:
                cu.append(cu[-1] + x)
            s["cu_seqlens"], start = _i32(cu), [0] * n
            s["owner"] = torch.repeat_interleave(torch.arange(n, device="cuda"),
                                                 torch.tensor(lens, device="cuda"))
            rows, room = (layers, cu[-1], hkv, d), lens
        s["k"], s["v"] = normal(*rows).to(dt), normal(*rows).to(dt)
        s["page_table"], pages = _pages(room, case["page"], rnd)
        s["lengths"] = _i32(start)
        cache = (layers, pages, case["page"], hkv, d)
        s["k_cache"], s["v_cache"] = normal(*cache).to(dt), normal(*cache).to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _PLAIN[s["op"]])(s)


def _run_own(s):
    import gated_delta_rule_05_gb300 as kda
    op = s["op"]
    if op == "tree_attention":
        return kda.kda_tree_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                      s["page_table"], s["lengths"], s["parent"],
                                      scale=s["scale"])
    if op == "decode_tree":
        o, states = kda.kda_decode_tree(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S"],
                                        s["parent"], states=s["states"])
        return {"o": o, "states": states}
    if op == "token_logprobs":
        logp, entropy, ids, top = kda.kda_token_logprobs(s["logits"], s["tokens"], s["k"])
        return {"logp": logp, "entropy": entropy, "ids": ids, "top": top}
    if op == "cache_commit":
        new = kda.kda_cache_commit(s["k"], s["v"], s["path"], s["count"], s["k_cache"],
                                   s["v_cache"], s["page_table"], s["lengths"])
    else:
        new = kda.kda_cache_append(s["k"], s["v"], s["cu_seqlens"], s["k_cache"], s["v_cache"],
                                   s["page_table"], s["lengths"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": new}


def _used_and_seen(parent):
    """seen[n, t, j]: node j is t itself or one of its ancestors; used[n, t]:
    t's chain of parents ends at the context."""
    ts = parent.shape[1]
    eye = torch.eye(ts, device=parent.device)
    step = (parent[:, :, None] == torch.arange(ts, device=parent.device)).float()
    seen = torch.linalg.matrix_power(step + eye, max(1, ts)) > 0
    used = (seen & (parent == -1)[:, None, :]).any(-1)
    return used, seen


def _plain_attention(s):
    q, table, lengths = s["q"].float(), s["page_table"], s["lengths"]
    n, ts, hq, d = q.shape
    hkv, page = s["hkv"], s["page"]
    pos = torch.arange(table.shape[1] * page, device=q.device)
    at = table.clamp_min(0)[:, pos // page].long(), (pos % page).expand(n, -1)
    keys = torch.cat([s["k_cache"][at], s["k"]], 1).float().permute(0, 2, 3, 1)
    values = torch.cat([s["v_cache"][at], s["v"]], 1).float().permute(0, 2, 1, 3)
    used, seen = _used_and_seen(s["parent"])
    context = (pos < lengths[:, None])[:, None, :].expand(n, ts, -1)
    mask = torch.cat([context, seen], 2)[:, None, :, None, :]
    rows = q.reshape(n, ts, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)
    x = (rows.reshape(n, hkv, -1, d) @ keys).mul_(s["scale"])
    x = x.view(n, hkv, ts, hq // hkv, -1).masked_fill_(~mask, -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, hkv, -1, p.shape[-1]) @ values).view(n, hkv, ts, hq // hkv, d) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(n, ts, hq, d)
    return (o * used[:, :, None, None]).to(s["q"].dtype)


def _plain_decode_tree(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    alpha, beta, parent = s["log_alpha"].exp(), s["beta"], s["parent"].long()
    n, ts = parent.shape
    used, _ = _used_and_seen(s["parent"])
    rows = torch.arange(n, device=q.device)
    states, outs = s["states"], []
    for t in range(ts):  # a node needs its parent's state
        own_parent = states[rows, parent[:, t].clamp_min(0)]
        prev = torch.where((parent[:, t] < 0)[:, None, None, None], s["S"], own_parent)
        prev = prev * alpha[:, t, :, :, None]
        err = v[:, t] - (prev * k[:, t, :, :, None]).sum(2)
        prev = prev + k[:, t, :, :, None] * (beta[:, t, :, None] * err)[:, :, None, :]
        keep = used[:, t, None, None, None]
        states[:, t] = torch.where(keep, prev, states[:, t])
        outs.append((prev * q[:, t, :, :, None]).sum(2) * keep[..., 0])
    return {"o": torch.stack(outs, 1).to(s["q"].dtype), "states": states}


def _plain_logprobs(s):
    x = s["logits"].float()
    shift = x.amax(-1, keepdim=True)
    e = (x - shift).exp()
    total = e.sum(-1, keepdim=True)
    lse = shift + total.log()
    entropy = total.log()[:, 0] - (e * (x - shift)).sum(-1) / total[:, 0]
    # a key for each logit that orders by value, then by the lower index
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits)
    index = torch.arange(x.shape[1], device=x.device)
    ids = (order * (1 << 20) + ((1 << 20) - 1 - index)).topk(s["k"], -1).indices
    return {"logp": x.gather(1, s["tokens"].long()) - lse, "entropy": entropy,
            "ids": ids.to(torch.int32), "top": x.gather(1, ids) - lse}


def _plain_commit(s):
    n, ts = s["path"].shape
    i = torch.arange(ts, device=s["path"].device)
    pos = s["lengths"][:, None].long() + i
    page = s["page_table"].gather(1, pos // s["page"]).long()
    at = slice(None), page, pos % s["page"]
    path = s["path"].clamp_min(0).long()
    take = slice(None), torch.arange(n, device=path.device)[:, None], path
    keep = (i < s["count"][:, None])[None, :, :, None, None]
    s["k_cache"][at] = torch.where(keep, s["k"][take], s["k_cache"][at])
    s["v_cache"][at] = torch.where(keep, s["v"][take], s["v_cache"][at])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": s["lengths"] + s["count"]}


def _plain_append(s):
    cu, owner = s["cu_seqlens"], s["owner"]
    pos = s["lengths"][owner] + torch.arange(owner.shape[0], device=cu.device) - cu[owner]
    at = slice(None), s["page_table"][owner, pos // s["page"]].long(), pos % s["page"]
    s["k_cache"][at] = s["k"]
    s["v_cache"][at] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "lengths": s["lengths"] + cu[1:] - cu[:-1]}


_PLAIN = {"tree_attention": _plain_attention, "decode_tree": _plain_decode_tree,
          "token_logprobs": _plain_logprobs, "cache_commit": _plain_commit,
          "cache_append": _plain_append}


# ------------------------------------------------- the work, and the answers
def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "tree_attention":
        used = _used_counts(case)
        context = sum(_spread(case["lo"], case["hi"], case["n"]))
        mean = context / case["n"]
        pairs = sum(u * (mean + (1 + u) / 4) for u in used)
        rows = case["hkv"] * (context + sum(used)) * 2 + case["hq"] * sum(used) * 2
        return {"bytes": rows * case["d"] * e, "flops": 4 * case["d"] * case["hq"] * pairs}
    if op == "decode_tree":
        nodes, d, h = sum(_used_counts(case)), case["d"], case["h"]
        return {"bytes": h * ((case["n"] + nodes) * d * d * 4 + nodes * (d * (4 * e + 4) + 4)),
                "flops": 7 * h * nodes * d * d}
    if op == "token_logprobs":
        return {"bytes": case["t"] * (case["v"] * e + 4 + 8 * case["j"] + 8 * case["k"]),
                "flops": 5 * case["t"] * case["v"]}
    if op == "cache_commit":
        rows = sum(_spread(0, case["ts"], case["n"]))
    else:
        rows = sum(_spread(case["lo"], case["hi"], case["n"]))
    return {"bytes": case["layers"] * rows * case["hkv"] * case["d"] * e * 4 + 8 * rows + 8 * case["n"],
            "flops": 0}


def _lineage(parent, t):
    """The nodes from t up to the context, or None for an unused node."""
    chain, t = [], t
    while t != -1:
        if t < 0:
            return None
        chain.append(t)
        t = parent[t]
    return chain


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tree_attention":
        q = s["q"]
        o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        group = case["hq"] // case["hkv"]
        for n, (length, parent) in enumerate(zip(s["lengths"].tolist(), s["parent"].tolist())):
            pages = s["page_table"][n][:-(-length // case["page"])].long()
            nodes = {t: _lineage(parent, t) for t in range(case["ts"])}
            live = [t for t in nodes if nodes[t] is not None]
            bias = torch.full((case["ts"], case["ts"]), -math.inf, dtype=torch.float64)
            for t in live:
                bias[t, nodes[t]] = 0.0
            bias = bias.to(q.device)
            for h in range(case["hkv"]):
                k, v = (torch.cat([c[pages, :, h].reshape(-1, case["d"])[:length], x[n, :, h]]).double()
                        for c, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])))
                for g in range(h * group, (h + 1) * group):
                    x = torch.einsum("td,ld->tl", q[n, live, g].double(), k) * s["scale"]
                    x[:, length:] += bias[live]
                    w = torch.softmax(x, -1)
                    o[n, live, g] = w @ v
        return o
    if op == "decode_tree":
        S = s["S"].double()
        n, ts, h, d = case["n"], case["ts"], case["h"], case["d"]
        states = torch.zeros((n, ts, h, d, d), dtype=torch.float64, device=S.device)
        o = torch.zeros((n, ts, h, d), dtype=torch.float64, device=S.device)
        eye = torch.eye(d, dtype=torch.float64, device=S.device)
        for i, parent in enumerate(s["parent"].tolist()):
            for t in range(ts):
                if _lineage(parent, t) is None:
                    continue
                before = S[i] if parent[t] < 0 else states[i, parent[t]]
                k, v, b = s["k"][i, t].double(), s["v"][i, t].double(), s["beta"][i, t].double()
                turn = eye - b[:, None, None] * k[:, :, None] * k[:, None, :]
                after = turn @ (s["log_alpha"][i, t].double().exp()[:, :, None] * before)
                after = after + b[:, None, None] * k[:, :, None] * v[:, None, :]
                states[i, t] = after
                o[i, t] = torch.einsum("hkv,hk->hv", after, s["q"][i, t].double())
        return {"o": o, "states": states}
    if op == "token_logprobs":
        outs = [[], [], []]
        for row, tokens in zip(s["logits"].split(256), s["tokens"].split(256)):
            logp = torch.log_softmax(row.double(), -1)
            outs[0].append(logp.gather(1, tokens.long()))
            outs[1].append(-(logp.exp() * logp).sum(-1))
            outs[2].append(logp.sort(-1, descending=True).values[:, :case["k"]])
        logp, entropy, top = (torch.cat(x) for x in outs)
        return {"logp": logp, "entropy": entropy, "ids": None, "top": top}
    return None
