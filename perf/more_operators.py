"""Cases of the operators that take a prompt and its answer through the softmax
attention layers of a model that mixes them with KDA layers:

  prompt_attention    kda_prompt_attention: causal attention over packed prompts,
                      whole ones or the rest behind a prefix
  append_rotary       kda_cache_append_rotary: queries and keys rotated to their
                      positions, keys and values into the pages of a cache in the
                      model's type or in 8 bits with a scale per block and head
  cache_attention     kda_cache_attention_e4m3: the newest tokens attend to their
                      sequence's rows in such a cache of 8 bits

Each case runs either in the library (``own`` true) or in a plain form of
elementary torch operations in fp32 (angles in float64); ``exact`` evaluates the
definitions in float64.

The cache of 8 bits holds e4m3 values; a block of rows and head has the scale
2^e, with the smallest e >= -126 for which the block's largest magnitude is at
most 448 * 2^e (0 for a block of zeros).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one short prompt: the latency of a call
        dict(name="prompt_short", op="prompt_attention", n=1, lo=509, hi=509, past=0, hq=32, hkv=8,
             d=128, fused=True, dtype="bf16"),
        # one long prompt
        dict(name="prompt_long", op="prompt_attention", n=1, lo=32768, hi=32768, past=0, hq=32,
             hkv=8, d=128, fused=False, dtype="bf16"),
        # a packed batch of prompts of different lengths
        dict(name="prompt_packed", op="prompt_attention", n=12, lo=512, hi=12288, past=0, hq=32,
             hkv=8, d=128, fused=True, dtype="bf16"),
        # the rest of prompts whose beginnings are cached, smaller heads
        dict(name="prompt_rest", op="prompt_attention", n=5, lo=700, hi=2048, past=6000, hq=16,
             hkv=16, d=64, fused=False, dtype="bf16"),
        # fp32, an odd group of heads
        dict(name="prompt_fp32", op="prompt_attention", n=7, lo=1, hi=1500, past=0, hq=12, hkv=4,
             d=64, fused=False, dtype="fp32"),
        # a packed batch of prompts into empty pages of 8 bits, one layer
        dict(name="append_prompts_8bit", op="append_rotary", n=12, lo=512, hi=12288, past=0, hq=32,
             hkv=8, d=128, rot=128, interleaved=False, page=64, block=64, fused=True, dtype="bf16"),
        # the same into pages of the model's type
        dict(name="append_prompts", op="append_rotary", n=12, lo=512, hi=12288, past=0, hq=32,
             hkv=8, d=128, rot=128, interleaved=False, page=64, block=0, fused=True, dtype="bf16"),
        # one token each of a serving batch, blocks of 16 rows
        dict(name="append_tokens_8bit", op="append_rotary", n=64, lo=1, hi=1, past=8000, hq=32,
             hkv=8, d=128, rot=64, interleaved=True, page=32, block=16, fused=True, dtype="bf16"),
        # one request, one new token: the latency of a call
        dict(name="cache_one_token", op="cache_attention", n=1, ts=1, lo=2047, hi=2047, hq=32, hkv=8,
             d=128, page=64, block=64, dtype="bf16"),
        # one token each of a serving batch, ragged contexts
        dict(name="cache_64x1", op="cache_attention", n=64, ts=1, lo=1000, hi=32000, hq=32, hkv=8,
             d=128, page=64, block=64, dtype="bf16"),
        # drafted chains of four tokens
        dict(name="cache_32x4", op="cache_attention", n=32, ts=4, lo=100, hi=16384, hq=32, hkv=8,
             d=128, page=32, block=16, dtype="bf16"),
        # fp32 queries, small heads without sharing, pages that are no power of two
        dict(name="cache_fp32_d64", op="cache_attention", n=8, ts=1, lo=100, hi=8191, hq=16, hkv=16,
             d=64, page=48, block=24, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt_attention", "append_rotary", "cache_attention"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128, 128]) if dtype == "bf16" else rng.choice([16, 32, 64, 128])
    if op == "prompt_attention":
        n = _log_int(rng, 1, 16)
        # the products stay within the listed cases'
        most = (1 << 34) if dtype == "bf16" else (1 << 27)
        hi = _log_int(rng, 1, max(1, min(16384, int(math.sqrt(most / (n * hkv * g))))))
        past = rng.choice([0, 0, min(hi, 4096)])
        return dict(op=op, n=n, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, past=past, hq=g * hkv,
                    hkv=hkv, d=d, fused=past == 0 and rng.random() < 0.5, dtype=dtype)
    block = rng.choice([8, 16, 24, 32, 64])
    page = block * rng.choice([1, 1, 2, 3, 4])
    if op == "append_rotary":
        n = _log_int(rng, 1, 64)
        rows = (1 << 27) // (n * (g + 2) * hkv * d) // (2 if dtype == "fp32" else 1)
        hi = _log_int(rng, 1, max(1, min(8192, rows)))
        return dict(op=op, n=n, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi,
                    past=rng.choice([0, _log_int(rng, 1, 2048)]), hq=rng.choice([0, g, g]) * hkv,
                    hkv=hkv, d=d, rot=rng.choice([16, d // 2, d]) if d > 16 else 16,
                    interleaved=rng.random() < 0.3, page=page, block=rng.choice([0, block, block]),
                    fused=rng.random() < 0.5, dtype=dtype)
    n, ts = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
    hi = _log_int(rng, 16, max(16, min(65536, (1 << 30) // (n * hkv * d))))
    return dict(op=op, n=n, ts=ts, lo=rng.choice([1, hi // 2, hi]), hi=hi, hq=g * hkv, hkv=hkv, d=d,
                page=page, block=block, dtype=dtype)


# --------------------------------------------------------------- the inputs
def _spread(lo, hi, n):
    """n lengths evenly spread over [lo, hi] (the same total for every seed)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


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


def _starts(lengths):
    cu = [0]
    for x in lengths:
        cu.append(cu[-1] + x)
    return cu


def _heads(x, counts, d, fused):
    """Splits [T, sum(counts) * d] into heads: views of it, or dense copies."""
    parts = [p.unflatten(1, (-1, d)) for p in x.split([c * d for c in counts], 1)]
    return parts if fused else [p.contiguous() for p in parts]


def _power(e):
    """2^e in fp32 for whole numbers e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _eight_bits(x, block):
    """A pool [pages, page, hkv, d] as e4m3 values and the scales of its blocks."""
    p, page, hkv, d = x.shape
    rows = x.view(p, page // block, block, hkv, d)
    mantissa, exponent = torch.frexp(rows.abs().amax((2, 4)))
    scales = _power(exponent - 9 + (mantissa > 0.875).int())
    return (rows / scales[:, :, None, :, None]).to(E4M3).view(x.shape), scales


def prepare(case, seed):
    rnd = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt, n, hq, hkv, d = (case[x] for x in ("op", "dtype", "n", "hq", "hkv", "d"))
    dt = DTYPES[dt]
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    s = dict(case)
    lens = _spread(case["lo"], case["hi"], n)
    rnd.shuffle(lens)
    if op == "cache_attention":
        s["page_table"], pages = _pages(lens, case["page"], rnd)
        s["lengths"] = _i32(lens)
        s["q"] = normal(n, case["ts"], hq, d).mul_(1.5).to(dt)
        pool = (pages, case["page"], hkv, d)
        # keys with channels of different magnitudes
        s["k_cache"], s["k_scales"] = _eight_bits(normal(*pool).mul_(normal(d).mul_(0.3).exp_()), case["block"])
        s["v_cache"], s["v_scales"] = _eight_bits(normal(*pool), case["block"])
        s["scale"] = d ** -0.5
        return s
    cu = _starts(lens)
    s["cu_seqlens"] = _i32(cu)
    past = _spread(0, case["past"], n)
    rnd.shuffle(past)
    if op == "prompt_attention":
        s["starts"] = cu
        if case["past"]:
            s["k_starts"] = _starts([a + b for a, b in zip(lens, past)])
            s["cu_seqlens_k"] = _i32(s["k_starts"])
            s["q"], = _heads(normal(cu[-1], hq * d).to(dt), [hq], d, False)
            s["k"], s["v"] = _heads(normal(s["k_starts"][-1], 2 * hkv * d).to(dt), [hkv, hkv], d, False)
        else:
            s["k_starts"], s["cu_seqlens_k"] = cu, None
            x = normal(cu[-1], (hq + 2 * hkv) * d).to(dt)
            s["q"], s["k"], s["v"] = _heads(x, [hq, hkv, hkv], d, case["fused"])
        s["scale"] = d ** -0.5
        return s
    x = normal(cu[-1], (hq + 2 * hkv) * d).to(dt)
    s["q"], s["k"], s["v"] = _heads(x, [hq, hkv, hkv], d, case["fused"])
    if hq == 0:
        s["q"] = None
    s["owner"] = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lens, device="cuda"))
    s["lengths"] = _i32(past)
    s["page_table"], pages = _pages([a + b for a, b in zip(lens, past)], case["page"], rnd)
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).float().cuda()
    pool = (pages, case["page"], hkv, d)
    s["k_cache"], s["v_cache"] = normal(*pool), normal(*pool)
    s["k_scales"] = s["v_scales"] = None
    if case["block"]:
        s["k_cache"], s["k_scales"] = _eight_bits(s["k_cache"], case["block"])
        s["v_cache"], s["v_scales"] = _eight_bits(s["v_cache"], case["block"])
    else:
        s["k_cache"], s["v_cache"] = s["k_cache"].to(dt), s["v_cache"].to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _PLAIN[s["op"]])(s)


def _run_own(s):
    import gated_delta_rule_05_gb300 as kda
    if s["op"] == "prompt_attention":
        return kda.kda_prompt_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], s["cu_seqlens_k"],
                                        scale=s["scale"])
    if s["op"] == "cache_attention":
        return kda.kda_cache_attention_e4m3(s["q"], s["k_cache"], s["v_cache"], s["k_scales"],
                                            s["v_scales"], s["page_table"], s["lengths"],
                                            scale=s["scale"])
    q, k, lengths = kda.kda_cache_append_rotary(
        s["q"], s["k"], s["v"], s["cu_seqlens"], s["inv_freq"], s["k_cache"], s["v_cache"],
        s["page_table"], s["lengths"], k_scales=s["k_scales"], v_scales=s["v_scales"],
        interleaved=s["interleaved"], want_k=True)
    return _appended(s, q, k, lengths)


def _appended(s, q, k, lengths):
    out = {"k": k, "lengths": lengths, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if q is not None:
        out["q"] = q
    if s["block"]:
        out["k_scales"], out["v_scales"] = s["k_scales"], s["v_scales"]
    return out


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    outs = []
    # a sequence's scores, for as many heads at once as some 16 GB hold
    for r0, r1, c0, c1 in zip(s["starts"], s["starts"][1:], s["k_starts"], s["k_starts"][1:]):
        rows = torch.arange(r1 - r0, device=q.device) + (c1 - c0) - (r1 - r0)
        seen = torch.arange(c1 - c0, device=q.device) <= rows[:, None]
        step = max(1, min(hkv, (1 << 32) // max(1, g * (r1 - r0) * (c1 - c0))))
        parts = []
        for h in range(0, hkv, step):
            m = min(step, hkv - h)
            x = q[r0:r1, h * g:(h + m) * g].float().unflatten(1, (m, g)).permute(1, 2, 0, 3)
            keys = k[c0:c1, h:h + m].float().permute(1, 2, 0)
            x = (x.reshape(m, -1, d) @ keys).view(m, g, r1 - r0, c1 - c0).mul_(s["scale"])
            x.masked_fill_(~seen, -math.inf)
            p = x.sub_(x.amax(-1, keepdim=True)).exp_()
            total = p.sum(-1, keepdim=True)
            o = p.view(m, -1, c1 - c0) @ v[c0:c1, h:h + m].float().transpose(0, 1)
            parts.append((o.view(m, g, r1 - r0, d) / total).permute(2, 0, 1, 3).reshape(r1 - r0, m * g, d))
        outs.append(torch.cat(parts, 1).to(q.dtype))
    return torch.cat(outs)


def _plain_rotate(x, turn, rot, interleaved):
    """x [T, h, d] with its first `rot` channels rotated in pairs by the angles [T, rot / 2]."""
    c, si = turn.cos().float()[:, None], turn.sin().float()[:, None]
    y = x[..., :rot].float()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
    a, b = a * c - b * si, a * si + b * c
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:].float()], -1)


def _plain_scale(top):
    mantissa, exponent = torch.frexp(top)
    return torch.where(top > 0, _power((exponent - 9 + (mantissa > 0.875).int()).clamp_min(-126)), top)


def _plain_blocks(s, x, cache, scales, pos):
    """Rows x [T, hkv, d] (fp32) into the pages of 8 bits."""
    block, page, table = s["block"], s["page"], s["page_table"]
    per = page // block
    pages, _, hkv, d = cache.shape
    flat, rows = scales.view(-1, hkv), cache.view(torch.uint8).view(-1, block, hkv, d)
    at = table[s["owner"], pos // page].long() * per + pos % page // block
    # the largest magnitude of each block's new rows, and what its old rows need
    top = torch.zeros_like(flat).scatter_reduce_(0, at[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    need = _plain_scale(top)
    filled = s["lengths"].long()
    first = table.gather(1, (filled // page)[:, None].clamp_max(table.shape[1] - 1))[:, 0].long() * per + filled % page // block
    old = (torch.arange(block, device=x.device) < (filled % block)[:, None])[:, :, None, None]
    had = torch.where((filled % block > 0)[:, None], flat[first], torch.zeros_like(flat[first]))
    need[first] = torch.maximum(need[first], had)
    touched = torch.zeros(flat.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, at, True)
    flat.copy_(torch.where(touched[:, None], need, flat))
    ratio = torch.where(had > 0, had / flat[first], torch.ones_like(had))[:, None, :, None]
    kept = rows[first].view(E4M3).float()
    rows[first] = torch.where(old, kept * ratio, kept).to(E4M3).view(torch.uint8)
    by = flat[at][:, :, None]
    held = torch.where(by > 0, x / by, torch.zeros_like(x)).to(E4M3).view(torch.uint8)
    rows.view(-1, hkv, d)[at * block + pos % block] = held


def _plain_append(s):
    cu, owner, page = s["cu_seqlens"], s["owner"], s["page"]
    pos = s["lengths"][owner].long() + torch.arange(owner.shape[0], device=cu.device) - cu[owner]
    turn = pos.double()[:, None] * s["inv_freq"].double()
    k = _plain_rotate(s["k"], turn, s["rot"], s["interleaved"])
    q = None
    if s["q"] is not None:
        q = _plain_rotate(s["q"], turn, s["rot"], s["interleaved"]).to(s["q"].dtype)
    if s["block"]:
        _plain_blocks(s, k, s["k_cache"], s["k_scales"], pos)
        _plain_blocks(s, s["v"].float(), s["v_cache"], s["v_scales"], pos)
    else:
        at = s["page_table"][owner, pos // page].long(), pos % page
        s["k_cache"][at] = k.to(s["k"].dtype)
        s["v_cache"][at] = s["v"]
    return _appended(s, q, k.to(s["k"].dtype), s["lengths"] + cu[1:] - cu[:-1])


def _plain_cache_attention(s):
    q, table, lengths = s["q"].float(), s["page_table"], s["lengths"]
    n, ts, hq, d = q.shape
    hkv, page, block = s["hkv"], s["page"], s["block"]
    pos = torch.arange(table.shape[1] * page, device=q.device)
    pages, slot = table.clamp_min(0)[:, pos // page].long(), (pos % page).expand(n, -1)
    keys, values = (s[x + "_cache"].view(torch.uint8)[pages, slot].view(E4M3).float()
                    * s[x + "_scales"][pages, slot // block][..., None] for x in "kv")
    last = lengths[:, None] - ts + torch.arange(ts, device=q.device)
    mask = (pos <= last[:, :, None])[:, None, :, None, :]
    rows = q.reshape(n, ts, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)
    x = (rows.reshape(n, hkv, -1, d) @ keys.permute(0, 2, 3, 1)).mul_(s["scale"])
    x = x.view(n, hkv, ts, hq // hkv, -1).masked_fill_(~mask, -math.inf)
    # a token before the sequence's first row sees nothing
    p = x.sub_(x.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    total = p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = (p.view(n, hkv, -1, p.shape[-1]) @ values.permute(0, 2, 1, 3)).view(n, hkv, ts, hq // hkv, d) / total
    return o.permute(0, 2, 1, 3, 4).reshape(n, ts, hq, d).to(s["q"].dtype)


_PLAIN = {"prompt_attention": _plain_prompt, "append_rotary": _plain_append,
          "cache_attention": _plain_cache_attention}


# ------------------------------------------------- the work, and the answers
def _mean_pairs(lens, past):
    """Query and key pairs of sequences whose pasts are shuffled over them (the mean)."""
    mean = sum(past) / len(past)
    return sum(x * (x + 1) / 2 + x * mean for x in lens)


def work(case):
    op, n, hq, hkv, d, e = (case[x] for x in ("op", "n", "hq", "hkv", "d", "dtype"))
    e = 2 if e == "bf16" else 4
    lens = _spread(case["lo"], case["hi"], n)
    if op == "cache_attention":
        ts = case["ts"]
        rows = sum(lens)
        blocks = sum(-(-x // case["block"]) for x in lens)
        return {"bytes": 2 * rows * hkv * d + 8 * blocks * hkv + 2 * n * ts * hq * d * e,
                "flops": 4 * d * hq * sum(max(0, x - t) for x in lens for t in range(ts))}
    past, t = _spread(0, case["past"], n), sum(lens)
    if op == "prompt_attention":
        keys = t + sum(past)
        return {"bytes": (2 * t * hq + 2 * keys * hkv) * d * e, "flops": 4 * d * hq * _mean_pairs(lens, past)}
    held = 1 if case["block"] else e
    blocks = sum(-(-x // case["block"]) for x in lens) if case["block"] else 0
    return {"bytes": t * d * (2 * hq * e + hkv * (3 * e + 2 * held)) + 8 * blocks * hkv + 8 * t, "flops": 3 * t * (hq + hkv) * case["rot"]}


def _exact_rotation(x, pos, inv_freq, interleaved):
    """x [T, h, d] in float64, its pairs turned as complex numbers."""
    rot = 2 * inv_freq.shape[0]
    y = x.double().clone()
    if interleaved:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    else:
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    z = torch.complex(y[..., first], y[..., second])
    z = z * torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                        pos.double()[:, None, None] * inv_freq.double())
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_power(top):
    """2^e for one magnitude."""
    if top == 0.0:
        return 0.0
    e = math.ceil(math.log2(top)) - 10
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def exact(case, seed):
    op, hq, hkv = case["op"], case["hq"], case["hkv"]
    g = hq // hkv
    if work(case)["flops"] > 1.5e12:
        return None
    s = prepare(case, seed)
    if op == "prompt_attention":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["n"]):
            r0, r1, c0, c1 = s["starts"][i], s["starts"][i + 1], s["k_starts"][i], s["k_starts"][i + 1]
            hidden = torch.ones(r1 - r0, c1 - c0, dtype=torch.bool, device="cuda").triu_(c1 - c0 - (r1 - r0) + 1)
            for h in range(hq):
                x = torch.einsum("td,jd->tj", s["q"][r0:r1, h].double(), s["k"][c0:c1, h // g].double())
                w = torch.softmax((x * s["scale"]).masked_fill(hidden, -math.inf), -1)
                out[r0:r1, h] = w @ s["v"][c0:c1, h // g].double()
        return out
    if op == "cache_attention":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for i, length in enumerate(s["lengths"].tolist()):
            ids = s["page_table"][i][:-(-length // case["page"])].long()
            for h in range(hkv):
                k, v = ((s[x + "_cache"].view(torch.uint8)[ids, :, h].view(E4M3).double()
                         * s[x + "_scales"][ids, :, h].double().repeat_interleave(case["block"], 1)[..., None])
                        .flatten(0, 1)[:length] for x in "kv")
                for t in range(case["ts"]):
                    c = length - case["ts"] + t + 1
                    if c > 0:
                        x = torch.einsum("gd,ld->gl", s["q"][i, t, h * g:(h + 1) * g].double(), k[:c])
                        out[i, t, h * g:(h + 1) * g] = torch.softmax(x * s["scale"], -1) @ v[:c]
        return out
    lens = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).tolist()
    pos = torch.cat([torch.arange(p, p + x, device="cuda") for p, x in zip(s["lengths"].tolist(), lens)])
    k = _exact_rotation(s["k"], pos, s["inv_freq"], case["interleaved"])
    out = {"k": k, "lengths": s["lengths"] + _i32(lens)}
    if s["q"] is not None:
        out["q"] = _exact_rotation(s["q"], pos, s["inv_freq"], case["interleaved"])
    if case["block"] and sum(lens) > 4096:
        # a walk over more blocks than that takes too long: the rotated rows alone
        return out | {x: None for x in ("k_cache", "v_cache", "k_scales", "v_scales")}
    for x, rows in (("k", k), ("v", s["v"].double())):
        cache = s[x + "_cache"].double()
        scales = s[x + "_scales"].double() if case["block"] else None
        step, row = case["block"] or case["page"], 0
        for n, (p, count) in enumerate(zip(s["lengths"].tolist(), lens)):
            end = p + count
            while p < end:
                # the sequence's rows up to the end of their block
                m = min(end, p // step * step + step) - p
                at, slot = int(s["page_table"][n, p // case["page"]]), p % case["page"]
                new = rows[row:row + m]
                if case["block"]:
                    b = slot // step
                    had = scales[at, b] if slot % step else torch.zeros(hkv, dtype=torch.float64, device="cuda")
                    by = torch.tensor([max(_exact_power(u), w) for u, w in zip(new.abs().amax((0, 2)).tolist(), had.tolist())],
                                      dtype=torch.float64, device="cuda")
                    # (values before their rounding)
                    cache[at, b * step:slot] *= torch.where(by > 0, had / by, 1.0)[:, None]
                    new = torch.where(by > 0, 1.0 / by, 0.0)[:, None] * new
                    scales[at, b] = by
                cache[at, slot:slot + m] = new
                p, row = p + m, row + m
        out[x + "_cache"] = cache
        if case["block"]:
            out[x + "_scales"] = scales
    return out
