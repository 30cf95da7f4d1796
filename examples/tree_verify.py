"""Speculative decoding with trees of drafted tokens, in a small hybrid model.

The model (random weights, no training) alternates KDA layers with softmax
attention over a paged cache.  One verification step of a batch is

    kda_decode_tree       in the KDA layers: a state per drafted node
    kda_tree_attention    in the others: the cache and each node's ancestors
    kda_token_logprobs    on the logits: the model's choice after every node

and, once the accepted path of every sequence is known,

    kda_state_gather      the state of its last node
    kda_cache_commit      its keys and values into the cache pages

The prompts go through the same layers in chains of up to 64 tokens.  Their KDA
states come from kda_prefill, their keys and values enter by kda_cache_append.
The drafter is the model without its layers: the head on a token's embedding.

    python examples/tree_verify.py [--dtype bf16] [--d 128]

prints the tokens accepted per step and, for fp32, checks that greedy decoding
one token at a time gives the same tokens.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_05_gb300 as kda  # noqa: E402


class Hybrid:
    """Weights and the layers' calls; ``pairs`` of a KDA and an attention layer."""

    def __init__(self, d, dtype, vocab=512, pairs=2, heads=4, cache_heads=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.d, self.H, self.Hkv, self.V, self.pairs = d, heads, cache_heads, vocab, pairs
        self.dtype, width = dtype, heads * d
        w = lambda i, o: (torch.randn(i, o, generator=g, device="cuda") * i ** -0.5).to(dtype)
        self.embed = torch.randn(vocab, width, generator=g, device="cuda").to(dtype)
        self.head = w(width, vocab)
        self.layers = [dict(q=w(width, width), k=w(width, width), v=w(width, width),
                            gate=w(width, width), beta=w(width, heads), out=w(width, width),
                            aq=w(width, width), ak=w(width, cache_heads * d),
                            av=w(width, cache_heads * d), aout=w(width, width))
                       for _ in range(pairs)]

        # the drafter: what the head makes of the embedding alone
        _, _, ids, _ = kda.kda_token_logprobs(self.embed @ self.head, None, 3)
        self.likely = ids.tolist()

    def forward(self, tokens, kda_layer, attention_layer):
        """tokens [N, Ts] -> logits [N, Ts, V] and the attention layers' k and v
        [pairs, N, Ts, Hkv, d].  The two callbacks are given the layer's number."""
        N, Ts = tokens.shape
        heads = lambda x, n: x.view(N, Ts, n, self.d).contiguous()
        unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(self.dtype)
        norm = lambda x: torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(self.dtype)
        x = self.embed[tokens.long()]
        ks, vs = [], []
        for i, w in enumerate(self.layers):
            y = norm(x)
            log_alpha = -2.0 * torch.sigmoid(heads(y @ w["gate"], self.H).float())
            beta = torch.sigmoid((y @ w["beta"]).float())
            o = kda_layer(i, unit(heads(y @ w["q"], self.H)), unit(heads(y @ w["k"], self.H)),
                          heads(y @ w["v"], self.H), log_alpha, beta)
            x = x + 0.5 * (o.reshape(N, Ts, -1) @ w["out"])
            y = norm(x)
            ks.append(heads(y @ w["ak"], self.Hkv))
            vs.append(heads(y @ w["av"], self.Hkv))
            o = attention_layer(i, heads(y @ w["aq"], self.H), ks[-1], vs[-1])
            x = x + 0.5 * (o.reshape(N, Ts, -1) @ w["aout"])
        return norm(x) @ self.head, torch.stack(ks), torch.stack(vs)


class Sequences:
    """The decoding state of N sequences: KDA states, cache pages, lengths."""

    def __init__(self, model, prompts, room, page=16):
        self.m, N = model, len(prompts)
        longest = max(map(len, prompts)) + room
        per = -(-longest // page)
        pool = (model.pairs, N * per, page, model.Hkv, model.d)
        self.k_cache = torch.empty(pool, dtype=model.dtype, device="cuda")
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.randperm(N * per, device="cuda").int().view(N, per)
        self.lengths = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.S = [torch.zeros(N, model.H, model.d, model.d, device="cuda")
                  for _ in range(model.pairs)]
        # all but the last token of each prompt; that one is the first root
        for n, prompt in enumerate(prompts):
            for at in range(0, len(prompt) - 1, 64):
                self.prefill(n, prompt[at:min(at + 64, len(prompt) - 1)])

    def prefill(self, n, piece):
        m, one = self.m, slice(n, n + 1)
        tokens = torch.tensor([piece], dtype=torch.int32, device="cuda")
        table, lengths = self.table[one].contiguous(), self.lengths[one].clone()

        def kda_layer(i, q, k, v, log_alpha, beta):
            o, S = kda.kda_prefill(q[0], k[0], v[0], log_alpha[0], beta[0],
                                   S0=self.S[i][one].contiguous())
            self.S[i][one] = S
            return o[None]

        def attention_layer(i, q, k, v):
            return kda.kda_tree_attention(q, k, v, self.k_cache[i], self.v_cache[i], table,
                                          lengths)

        _, k, v = m.forward(tokens, kda_layer, attention_layer)
        cu = torch.tensor([0, len(piece)], dtype=torch.int32, device="cuda")
        self.lengths[one] = kda.kda_cache_append(k[:, 0].contiguous(), v[:, 0].contiguous(), cu,
                                                 self.k_cache, self.v_cache, table, lengths)

    def verify(self, tokens, parent):
        """Runs the drafted nodes; returns the model's choice after every node and
        its log probability, [N, Ts]."""
        m = self.m
        N, Ts = tokens.shape
        states = []

        def kda_layer(i, q, k, v, log_alpha, beta):
            o, st = kda.kda_decode_tree(q, k, v, log_alpha, beta, self.S[i], parent)
            states.append(st)
            return o

        def attention_layer(i, q, k, v):
            return kda.kda_tree_attention(q, k, v, self.k_cache[i], self.v_cache[i], self.table,
                                          self.lengths, parent)

        logits, k, v = m.forward(tokens, kda_layer, attention_layer)
        self.pending = states, k, v
        _, _, ids, logp = kda.kda_token_logprobs(logits.view(N * Ts, m.V), None, 1)
        return ids.view(N, Ts), logp.view(N, Ts)

    def accept(self, path, count):
        """Keeps the nodes path[n, :count[n]] of the last verify."""
        states, k, v = self.pending
        last = path.gather(1, (count.long() - 1).clamp(min=0)[:, None])[:, 0]
        node = torch.where(count > 0, last + 1, 0).int()    # 0: the state as it was
        for S, st in zip(self.S, states):
            kda.kda_state_gather(st, S, node, S_out=S)
        self.lengths = kda.kda_cache_commit(k, v, path, count, self.k_cache, self.v_cache,
                                            self.table, self.lengths)


def draft(root, likely, nodes):
    """A tree of at most ``nodes`` tokens under ``root``: the three likeliest
    followers, two of each of those, then one.  Returns (tokens, parent)."""
    tokens, parent, depth = [root], [-1], [0]
    for node in range(nodes):
        if node == len(tokens):
            break
        for token in likely[tokens[node]][:max(3 - depth[node], 1)]:
            if len(tokens) < nodes:
                tokens.append(token)
                parent.append(node)
                depth.append(depth[node] + 1)
    return tokens, parent


def decode(model, prompts, new_tokens, nodes):
    """Greedy decoding, ``nodes`` drafted per step (1: token by token).  Returns
    (tokens per sequence, their log probabilities, steps)."""
    N = len(prompts)
    seqs = Sequences(model, prompts, new_tokens + nodes)
    out, logps = [[] for _ in prompts], [[] for _ in prompts]
    root = [p[-1] for p in prompts]
    steps = 0
    while min(map(len, out)) < new_tokens:
        tokens = np.zeros((N, nodes), np.int32)
        parent = np.full((N, nodes), -2, np.int32)      # -2: an unused node
        for n in range(N):
            if len(out[n]) >= new_tokens:
                continue
            t, p = draft(root[n], model.likely, nodes)
            tokens[n, :len(t)], parent[n, :len(p)] = t, p
        dev = lambda x: torch.from_numpy(x).cuda()
        ids, logp = seqs.verify(dev(tokens), dev(parent))
        ids, logp = ids.cpu().numpy(), logp.cpu().numpy()

        path = np.zeros((N, nodes), np.int32)
        count = np.zeros(N, np.int32)
        for n in range(N):
            node = 0 if parent[n, 0] == -1 else None
            while node is not None:
                path[n, count[n]] = node
                count[n] += 1
                token = int(ids[n, node])
                out[n].append(token)
                logps[n].append(float(logp[n, node]))
                root[n] = token
                if len(out[n]) >= new_tokens:
                    break
                node = next((c for c in range(node + 1, nodes)
                             if parent[n, c] == node and tokens[n, c] == token), None)
        seqs.accept(dev(path), dev(count))
        steps += 1
    return out, logps, steps


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--dtype", choices=["fp32", "bf16"], default="fp32")
    ap.add_argument("--d", type=int, default=64)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--new-tokens", type=int, default=64)
    ap.add_argument("--nodes", type=int, default=13)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    rng = np.random.default_rng(0)
    model = Hybrid(args.d, {"fp32": torch.float32, "bf16": torch.bfloat16}[args.dtype])
    prompts = [rng.integers(0, model.V, 5 + 67 * n).tolist() for n in range(args.sequences)]
    out, logps, steps = decode(model, prompts, args.new_tokens, args.nodes)
    total = sum(map(len, out))
    print("%d tokens in %d steps of %d sequences: %.2f per sequence and step" % (
        total, steps, args.sequences, total / steps / args.sequences))
    plain, plain_logps, _ = decode(model, prompts, args.new_tokens, 1)
    if args.dtype == "fp32":
        assert out == plain, "the tree's tokens differ from one-token decoding"
        worst = max(abs(a - b) for x, y in zip(logps, plain_logps) for a, b in zip(x, y))
        print("the same tokens as one at a time; log probabilities within %.1e" % worst)
    else:
        same = sum(a == b for x, y in zip(out, plain) for a, b in zip(x, y))
        print("%d of %d tokens as one at a time (bf16 roundings differ)" % (same, total))
    return out, plain, steps


if __name__ == "__main__":
    main()
