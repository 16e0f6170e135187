"""A speculative decode loop on the library's calls, as a serving engine makes
them: for every step the pages a drafted tree needs (iq4xs_cache_reserve),
for every layer the quantized q, k, v projection (iq4xs_linear), norm,
rotation and cache append (iq4xs_qk_norm_rope), tree attention over the paged
cache (iq4xs_tree_attention) and the quantized output projection, and after
verification the accepted path committed (iq4xs_cache_commit).  Recurrent layers
(--recurrent) go with them: the projection's convolution, norm and gates
(iq4xs_delta_inputs), the gated delta rule over the same drafted tree from a
state that stays (iq4xs_delta_rule), and the state moved along the accepted path
(iq4xs_delta_commit).  With a vocabulary (--vocab) an output projection's
probabilities (iq4xs_token_probs) choose the path and the token behind it
(iq4xs_verify_drafts).  Sequences are forked and released between steps.

    python -m iq4_xs_quantized_gb300.verify_step [--layers L] [--recurrent R] [--vocab V] [--sequences S] [--tree T] [--steps N]

Weights are seeded random IQ4_XS blocks and a token is a seeded random hidden
state; without a vocabulary a path's acceptance is drawn at random.  What a run
checks is that a sequence that came by drafted trees ends where one that was
decoded token by token ends.
"""
from __future__ import annotations

import argparse
import math
import time

import numpy as np
import torch

from . import binding as B
from . import synth


def tree_mask(parents, words: int | None = None) -> np.ndarray:
    """Mask rows (int64 [T, words]) and depths of a drafted tree: parents[i] <
    i, or -1 for a root; a token sees its ancestors and itself."""
    t = len(parents)
    words = words or max(1, (t + 63) // 64)
    seen, depth = [], []
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError(f"tree_mask: the parent of token {i} is {p}: parents come first")
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    out = np.zeros((t, words), np.uint64)
    for i, bits in enumerate(seen):
        for w in range(words):
            out[i, w] = (bits >> (64 * w)) & (2**64 - 1)
    return out.view(np.int64), np.array(depth, np.int32)


def rope_table(positions: int, rot_dim: int, base: float = 1e6) -> torch.Tensor:
    """fp32 [positions, rot_dim / 2, 2] of (cos, sin), computed in fp64."""
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device="cuda") / rot_dim)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()


class Decoder:
    """The layers of a decoder: `recurrent` ones over a state for each slot, then
    attention layers over a paged cache, one page table for all; an output
    projection to `vocab` tokens."""

    def __init__(self, layers=2, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, page_size=16, pages=256, slots=4,
                 width=32, dtype=torch.float16, seed=0, recurrent=0, vocab=0):
        self.layers, self.hidden, self.hq, self.hkv, self.d = layers, hidden, q_heads, kv_heads, head_dim
        self.page_size, self.slots = page_size, slots
        self.n_qkv = (q_heads + 2 * kv_heads) * head_dim
        self.cache = B.alloc_kv_cache(layers, pages, page_size, kv_heads, head_dim, dtype)
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.refs, self.lens, self.held, self.table = i32(pages), i32(slots), i32(slots), i32(slots, width)
        self.offsets, self.status = i32(slots + 1), i32(slots)
        self.batch = B.KVBatch(self.offsets, self.lens, self.held, self.table)
        self.rope = rope_table(width * page_size, head_dim)
        rng = np.random.default_rng(seed)
        scale = 1.0 / math.sqrt(hidden) / 600  # the blocks' weights spread by about 1300 scale: 2 / sqrt(hidden)
        matrix = lambda n, k: torch.from_numpy(synth.iq4xs_weights(rng, n, k, scale)).cuda()  # noqa: E731
        self.w_qkv = [matrix(self.n_qkv, hidden) for _ in range(layers)]
        self.w_o = [matrix(hidden, q_heads * head_dim) for _ in range(layers)]
        self.norm_q, self.norm_k = (torch.ones(head_dim, device="cuda") for _ in range(2))
        # recurrent layers: 2 query and key heads, 4 value heads of head_dim; a and b from the same projection
        self.vocab, self.recurrent, self.rk, self.rv, self.kept = vocab, recurrent, 2, 4, None
        self.state = None
        if recurrent:
            self.state = B.alloc_delta_state(recurrent, slots, self.rk, self.rv, head_dim, head_dim)
            self.n_in = self.state.channels + 2 * self.rv
            self.w_in = [matrix(self.n_in, hidden) for _ in range(recurrent)]
            self.w_out = [matrix(hidden, self.rv * head_dim) for _ in range(recurrent)]
            normal = lambda *shape: torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).cuda()  # noqa: E731
            self.w_conv = [0.5 * normal(self.state.channels, 4) for _ in range(recurrent)]
            self.a_log, self.dt_bias = normal(recurrent, self.rv), normal(recurrent, self.rv) - 3
        self.w_vocab = matrix(vocab, hidden) if vocab else None  # (last: the other weights are the same without)

    def _buffers(self, m):
        d, ws = self.d, max(B.iq4xs_linear_workspace_bytes(m, self.n_qkv, self.hidden),
                            B.iq4xs_linear_workspace_bytes(m, self.hidden, self.hq * self.d))
        return (torch.empty(m, self.n_qkv, device="cuda"), torch.empty(m, self.hq, d, dtype=self.cache.dtype, device="cuda"),
                torch.empty(m, self.hq * d, device="cuda"), torch.empty(m, self.hidden, device="cuda"),
                torch.empty(ws, dtype=torch.uint8, device="cuda"),
                torch.empty(B.iq4xs_tree_attention_workspace_bytes(m, self.hq, self.cache, self.batch),
                            dtype=torch.uint8, device="cuda"))

    def _recurrent(self, x, max_rows, mask, keep):
        """The recurrent layers.  keep: the states stay, and what a commit needs is kept."""
        st, m, d, c = self.state, x.shape[0], self.d, self.state.channels
        ws = torch.empty(max(B.iq4xs_linear_workspace_bytes(m, self.n_in, self.hidden),
                             B.iq4xs_linear_workspace_bytes(m, self.hidden, self.rv * d)), dtype=torch.uint8, device="cuda")
        f32 = lambda *shape: torch.empty(shape, device="cuda")  # noqa: E731
        proj, out, y = f32(self.recurrent, m, self.n_in), f32(m, self.rv * d), f32(m, self.hidden)
        qkv = torch.empty(self.recurrent, m, c, dtype=self.cache.dtype, device="cuda")
        q, k, v = (t.unflatten(2, (-1, d)) for t in qkv.split((self.rk * d, self.rk * d, self.rv * d), dim=2))
        g, beta, u = f32(self.recurrent, m, self.rv), f32(m, self.rv), f32(self.recurrent, m, self.rv, d) if keep else None
        for i in range(self.recurrent):
            B.iq4xs_linear(self.w_in[i], self.n_in, self.hidden, x, proj[i], ws)
            B.iq4xs_delta_inputs(proj[i, :, :c], self.w_conv[i], proj[i, :, c:c + self.rv], proj[i, :, c + self.rv:], self.a_log[i],
                                 self.dt_bias[i], 1e-6, q[i], k[i], v[i], g[i], beta, st, i, self.batch, tree_mask=mask,
                                 advance=not keep)
            B.iq4xs_delta_rule(q[i], k[i], v[i], g[i], beta, 1.0, out, st, i, self.batch, u=u[i] if keep else None,
                               tree_mask=mask, max_rows=max_rows)
            B.iq4xs_linear(self.w_out[i], self.hidden, self.rv * d, out, y, ws)
            x = x + y
        self.kept = (k, g, u, proj[:, :, :c]) if keep else None
        return x

    def logits(self, x):
        """fp32 [M, vocab] of hidden states [M, hidden]."""
        m = x.shape[0]
        ws = torch.empty(B.iq4xs_linear_workspace_bytes(m, self.vocab, self.hidden), dtype=torch.uint8, device="cuda")
        out = torch.empty(m, self.vocab, device="cuda")
        B.iq4xs_linear(self.w_vocab, self.vocab, self.hidden, x.contiguous(), out, ws)
        return out

    def forward(self, x, rows, positions, mask, keep=False):
        """Hidden states x [M, hidden] of rows[s] new tokens for each sequence
        slot, at `positions`, under `mask` (None: chains) -> hidden states.
        The new tokens' K and V stay in the cache behind lens, not committed;
        recurrent states move on over all of them, or stay with `keep`."""
        self.offsets.copy_(torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32))
        B.iq4xs_cache_reserve(self.batch, self.page_size, self.refs, self.status)
        if bool(self.status.any()):
            raise RuntimeError("the cache has too few pages")
        if self.recurrent:
            x = self._recurrent(x, max(rows), mask, keep)
        m, d = x.shape[0], self.d
        qkv, q, att, y, ws, aws = self._buffers(m)
        at_k, at_v = self.hq * d, (self.hq + self.hkv) * d
        for i in range(self.layers):
            B.iq4xs_linear(self.w_qkv[i], self.n_qkv, self.hidden, x, qkv, ws)
            B.iq4xs_qk_norm_rope(qkv[:, :at_k].unflatten(1, (self.hq, d)), qkv[:, at_k:at_v].unflatten(1, (self.hkv, d)),
                                 qkv[:, at_v:].unflatten(1, (self.hkv, d)), self.norm_q, self.norm_k, 1e-6, self.rope,
                                 positions, q, self.cache, i, self.batch)
            B.iq4xs_tree_attention(q, self.cache, i, self.batch, d ** -0.5, att, aws, tree_mask=mask)
            B.iq4xs_linear(self.w_o[i], self.hidden, self.hq * d, att, y, ws)
            x = x + y
        return x

    def commit(self, paths, accepted):
        if self.kept is not None:
            B.iq4xs_delta_commit(*self.kept, self.state, self.batch, paths, accepted)
            self.kept = None
        B.iq4xs_cache_commit(self.cache, self.batch, self.refs, paths, accepted, self.lens)

    def fork(self, parents, children):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        status = i32([0] * len(parents))
        B.iq4xs_cache_fork(self.cache, self.batch, self.refs, i32(parents), i32(children), status)
        if self.state is not None:
            self.state.s[:, children] = self.state.s[:, parents]
            self.state.conv[:, children] = self.state.conv[:, parents]
        return status

    def release(self, slots):
        B.iq4xs_cache_release(self.batch, self.refs, torch.tensor(slots, dtype=torch.int32, device="cuda"))


def token_states(ids, hidden: int) -> torch.Tensor:
    """A seeded random hidden state for each token id."""
    return torch.stack([torch.randn(hidden, generator=torch.Generator().manual_seed(int(i))) for i in ids]).cuda()


def verified(dec, hidden, tokens, mask, tree, seed):
    """The paths that the output projection's probabilities accept, committed;
    each sequence's accepted tokens (places in its tree) and the token behind them."""
    slots, m = dec.slots, hidden.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    probs = dec.logits(hidden)
    B.iq4xs_token_probs(probs, probs)
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    paths, accepted, ahead = i32(slots, tree), i32(slots), i32(slots)
    rand = torch.rand(m + slots, generator=g, device="cuda")
    B.iq4xs_verify_drafts(probs, tokens, rand[:m], rand[m:], paths, accepted, ahead, dec.batch, tree_mask=mask)
    dec.commit(paths, accepted)
    counts = accepted.tolist()
    return [way[:n] for way, n in zip(paths.tolist(), counts) if n], [t for t, n in zip(ahead.tolist(), counts) if n]


def run(layers=2, sequences=3, tree=8, steps=4, prompt=37, seed=0, dtype=torch.float16, verbose=False, recurrent=0, vocab=0):
    """Decodes `sequences` sequences by drafted trees and again token by token;
    returns the last token's hidden states of both, [sequences, hidden]."""
    rng = np.random.default_rng(seed)
    most = prompt + 5 * (sequences - 1) + steps * tree + tree  # the last prompt is the longest
    width = -(-most // 16) + 1
    dec = Decoder(layers=layers, slots=sequences + 1, width=width, pages=(sequences + 2) * width, dtype=dtype, seed=seed,
                  recurrent=recurrent, vocab=vocab)
    # prompts, and what each sequence comes to hold
    text = [rng.integers(0, 10**6, prompt + 5 * s).tolist() for s in range(sequences)]
    prompts = [list(t) for t in text]
    rows = [len(t) for t in text] + [0]
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    x = token_states([i for t in text for i in t], dec.hidden)
    dec.forward(x, rows, None, None)
    width_p = max(max(rows), tree)
    chain = np.tile(np.arange(width_p, dtype=np.int32), (sequences + 1, 1))
    dec.commit(i32(chain), i32(rows))
    last, ahead = None, rng.integers(0, vocab, sequences).tolist() if vocab else None  # the token that a sequence goes on with
    began = time.perf_counter()
    for step in range(steps):
        parents = [[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, tree)] for _ in range(sequences)]
        ids = [rng.integers(0, vocab or 10**6, tree).tolist() for _ in range(sequences)]
        for s in range(sequences if vocab else 0):
            ids[s][0] = ahead[s]
        built = [tree_mask(p) for p in parents]
        mask = torch.from_numpy(np.concatenate([b[0] for b in built])).cuda()
        lens = [len(t) for t in text]
        positions = i32(np.concatenate([b[1] + n for b, n in zip(built, lens)]))
        out = dec.forward(token_states([i for t in ids for i in t], dec.hidden), [tree] * sequences + [0], positions, mask,
                          keep=True)
        if vocab:
            ways, ahead = verified(dec, out, i32([i for t in ids for i in t]), mask, tree, seed + step)
        else:  # "verification": the way from the root to a drawn token
            paths, ways = np.zeros((sequences + 1, tree), np.int32), []
            for s in range(sequences):
                way, at = [], int(rng.integers(0, tree))
                while at >= 0:
                    way.insert(0, at)
                    at = parents[s][at]
                paths[s, :len(way)] = way
                ways.append(way)
            dec.commit(i32(paths), i32([len(way) for way in ways] + [0]))
        for s, way in enumerate(ways):
            text[s] += [ids[s][i] for i in way]
        last = out[[s * tree + way[-1] for s, way in enumerate(ways)]]
        # a second continuation of the first sequence begins and is given up again
        if bool(dec.fork([0], [sequences]).any()):
            raise RuntimeError("the cache has too few pages")
        dec.release([sequences])
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    # the same texts token by token
    one = Decoder(layers=layers, slots=sequences, width=width, pages=sequences * width + 1, dtype=dtype, seed=seed,
                  recurrent=recurrent)
    one.forward(token_states([i for t in prompts for i in t], one.hidden), [len(t) for t in prompts], None, None)
    one.commit(i32(chain[:sequences]), i32([len(t) for t in prompts]))
    final = torch.empty(sequences, one.hidden, device="cuda")
    step_path = i32(np.zeros((sequences, 1)))
    for i in range(max(len(t) - len(p) for t, p in zip(text, prompts))):
        live = [s for s in range(sequences) if len(prompts[s]) + i < len(text[s])]
        rows = [1 if s in live else 0 for s in range(sequences)]
        out = one.forward(token_states([text[s][len(prompts[s]) + i] for s in live], one.hidden), rows, None, None)
        one.commit(step_path, i32(rows))
        for k, s in enumerate(live):
            if len(prompts[s]) + i + 1 == len(text[s]):
                final[s] = out[k]
    torch.cuda.synchronize()
    if verbose:
        print(f"{steps} steps of {sequences} trees of {tree} tokens, {recurrent} + {layers} layers: {took / steps * 1e3:.2f} ms a step, "
              f"{sum(len(t) for t in text)} tokens cached, {int((dec.refs > 0).sum())} pages held")
    assert B.iq4xs_last_device_error() == 0
    return last, final


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--recurrent", type=int, default=0, help="recurrent layers ahead of the attention layers")
    ap.add_argument("--vocab", type=int, default=0, help="tokens of an output projection that verifies the drafts")
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--tree", type=int, default=16)
    ap.add_argument("--steps", type=int, default=6)
    a = ap.parse_args()
    by_trees, by_tokens = run(a.layers, a.sequences, a.tree, a.steps, verbose=True, recurrent=a.recurrent, vocab=a.vocab)
    off = ((by_trees - by_tokens).norm(dim=1) / by_tokens.norm(dim=1)).max().item()
    print(f"by trees against token by token: {off:.2e} of the hidden state")


if __name__ == "__main__":
    main()
