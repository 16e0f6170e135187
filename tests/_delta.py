"""Plain 64-bit references of the recurrent layers and of verification, and
random batches for them: loops over sequences and rows, written from the
operators' definitions, with bounds on what fp32 arithmetic may be off by."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

from iq4_xs_quantized_gb300 import binding as B

F32 = 2.0**-24  # half a step of fp32, relative
HALF_STEP = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def tree_parents(t, rng, reach=4):
    """A random tree of t tokens: a root, then each with a parent among the `reach` before it."""
    return [-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, t)]


def mask_of(parents_by_seq, words=1):
    rows = []
    for parents in parents_by_seq:
        seen = []
        for i, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        rows += [[(b >> (64 * w)) & (2**64 - 1) for w in range(words)] for b in seen]
    return torch.from_numpy(np.array(rows, np.uint64).reshape(-1, words).view(np.int64)).cuda()


def chains(new):
    return [list(range(-1, n - 1)) for n in new]


class Batch:
    """Sequences of the given lengths and new tokens, their states scattered over
    slots, everything a call reads on the device.  Slots of no sequence and of
    empty ones hold `garbage`; so do the spaces between."""

    def __init__(self, lens, new, hk=2, hv=4, dk=128, dv=128, dtype=torch.float16, layers=1, seed=0, spare=1, mapped=True,
                 garbage=float("nan"), pad=0, first_row=0):
        rng = np.random.default_rng(seed)
        self.lens_n, self.new_n, self.hk, self.hv, self.dk, self.dv, self.dtype = list(lens), list(new), hk, hv, dk, dv, dtype
        b = len(self.lens_n)
        slots = b + spare
        self.slot_n = rng.permutation(slots)[:b] if mapped else np.arange(b)
        self.first_row = first_row
        self.rows = first_row + sum(new)
        self.offsets_n = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + first_row
        self.offsets, self.lens = i32(self.offsets_n), i32(self.lens_n)
        self.batch = B.KVBatch(self.offsets, self.lens, i32(np.zeros(b)), i32(np.zeros((b, 1))))
        self.channels = 2 * hk * dk + hv * dv
        self.g = torch.Generator(device="cuda").manual_seed(seed + 1)
        raw = torch.full((layers, slots, hv * dk * dv + pad), garbage, device="cuda")
        self.s = raw[..., :hv * dk * dv].unflatten(2, (hv, dk, dv))
        rawc = torch.full((layers, slots, 3 * self.channels + pad), garbage, device="cuda")
        self.conv = rawc[..., :3 * self.channels].unflatten(2, (3, self.channels))
        for i, n in enumerate(self.lens_n):
            if n > 0:
                self.s[:, self.slot_n[i]] = 0.3 * self.randn(layers, hv, dk, dv)
                self.conv[:, self.slot_n[i]] = self.randn(layers, 3, self.channels)
        self.raw, self.rawc = raw, rawc
        self.state = B.DeltaState(self.s, self.conv, hk, i32(self.slot_n) if mapped else None)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def rand(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda")

    def operands(self, layers=None, gap=0):
        """Unit keys and queries, values, decays and step sizes; rows `gap` elements apart."""
        lead = () if layers is None else (layers,)

        def rows16(h, d, unit):
            x = self.randn(*lead, self.rows, h, d)
            x = x / x.norm(dim=-1, keepdim=True) if unit else x
            buf = torch.full((*lead, self.rows, h * d + gap), float("nan"), device="cuda", dtype=self.dtype)
            buf[..., :h * d] = x.flatten(-2).to(self.dtype)
            return buf[..., :h * d].unflatten(-1, (h, d))

        q, k, v = rows16(self.hk, self.dk, True), rows16(self.hk, self.dk, True), rows16(self.hv, self.dv, False)
        g = -torch.exp(3 * self.randn(*lead, self.rows, self.hv) - 4)
        return q, k, v, g, torch.sigmoid(self.randn(*lead, self.rows, self.hv))


def rule_ref(bt, q, k, v, g, beta, scale, parents, layer=0, keep=False):
    """out, u, the new states (float64, CPU) and bounds on the error of each.

    Bounds.  A product S^T x is a sum of dk terms, off by at most (dk + 2) 2^-24
    |S_j| |x| in column j (Cauchy and Schwarz); u, the update and the decay add
    a few roundings of what they handle.  A step carries an error of S on
    without growth (e^g <= 1, 0 <= beta |k|^2 <= 2), so a column's error after
    some steps is at most the sum of the steps' own.  Where the rows go in
    blocks, sums of up to 64 further terms stand in for a step's: their lengths
    are added to dk."""
    f = lambda x: x.detach().cpu().double()  # noqa: E731
    q, k, v, g, beta, s_all = f(q), f(k), f(v), f(g), f(beta), f(bt.s[layer])
    group, unit = bt.hv // bt.hk, (bt.dk + 64 + 16) * F32
    out = torch.full((bt.rows, bt.hv, bt.dv), float("nan"), dtype=torch.float64)
    u_out, out_tol, u_tol = out.clone(), out.clone(), out.clone()
    new = s_all.clone()
    s_tol = torch.zeros_like(new)
    for s, n in enumerate(bt.new_n):
        s0 = s_all[bt.slot_n[s]] if bt.lens_n[s] > 0 else torch.zeros(bt.hv, bt.dk, bt.dv, dtype=torch.float64)
        nodes = {-1: (s0, torch.zeros(bt.hv, bt.dv, dtype=torch.float64))}
        for t in range(n):
            r = int(bt.offsets_n[s]) + t
            S, err = nodes[parents[s][t]]
            if not keep:
                nodes.pop(parents[s][t])
            kk, qq = k[r].repeat_interleave(group, 0), q[r].repeat_interleave(group, 0)
            S = S * g[r].exp()[:, None, None]
            size = S.norm(dim=1)
            u = beta[r][:, None] * (v[r] - torch.einsum("hkv,hk->hv", S, kk))
            u_out[r], u_tol[r] = u, err + unit * (size + v[r].abs() + u.abs()) + 1e-30
            S = S + kk[:, :, None] * u[:, None]
            err = err + unit * (size + v[r].abs() + u.abs() + S.norm(dim=1))
            out[r] = scale * torch.einsum("hkv,hk->hv", S, qq)
            out_tol[r] = abs(scale) * qq.norm(dim=1)[:, None] * (err + unit * S.norm(dim=1)) + 1e-30
            nodes[t] = (S, err)
        if n > 0 and not keep:
            new[bt.slot_n[s]], s_tol[bt.slot_n[s]] = nodes[n - 1][0], nodes[n - 1][1][:, None] + 1e-30
    return out, out_tol, u_out, u_tol, new, s_tol


def inputs_ref(bt, x, w, a, b, a_log, dt_bias, eps, parents, layer=0):
    """y (before rounding) of q, k and v with the errors that fp32 allows, g, beta, and the last inputs.

    Bounds.  The convolution: four products and sums, 5 2^-24 of the sum of
    magnitudes m.  SiLU's slope is below 1.1, and its exponential (2 units in
    the last place and 2^-22 |y| from the argument's scaling) and division add
    2^-21 (1 + |y|) of the value.  A norm divides by at least |y| / (1 + eps...),
    so the error relative to the head's norm carries over, twice (the value's
    and the norm's), with a few 2^-24 of the value."""
    f = lambda z: z.detach().cpu().double()  # noqa: E731
    x, w, conv = f(x), f(w), f(bt.conv[layer])
    y, tol = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    last = conv.clone()
    for s, n in enumerate(bt.new_n):
        old = conv[bt.slot_n[s]] if bt.lens_n[s] > 0 else torch.zeros(3, bt.channels, dtype=torch.float64)
        r0 = int(bt.offsets_n[s])
        for t in range(n):
            at, line = t, []
            for _ in range(4):
                line.insert(0, x[r0 + at] if at >= 0 else old[3 + at])
                at = parents[s][at] if at >= 0 else at - 1
            terms = torch.stack(line) * w.T
            z = terms.sum(0)
            y[r0 + t] = z * torch.sigmoid(z)
            tol[r0 + t] = 1.1 * 6 * F32 * terms.abs().sum(0) + 2.0**-21 * (1 + z.abs()) * y[r0 + t].abs() + 1e-30
        if n > 0:
            last[bt.slot_n[s]] = torch.cat((old, x[r0:r0 + n]))[-3:]
    nk = bt.hk * bt.dk
    parts = []
    for i, (lo, hi, h, d) in enumerate(((0, nk, bt.hk, bt.dk), (nk, 2 * nk, bt.hk, bt.dk), (2 * nk, bt.channels, bt.hv, bt.dv))):
        z, e = y[:, lo:hi].unflatten(1, (h, d)), tol[:, lo:hi].unflatten(1, (h, d))
        if i < 2:
            norm = ((z**2).sum(-1, keepdim=True) + eps).sqrt()
            z, e = z / norm, e / norm + z.abs() / norm * (e.norm(dim=-1, keepdim=True) / norm + (d + 8) * F32)
        parts.append((z, e))
    z = f(a) + f(dt_bias)
    g = -f(a_log).exp() * torch.nn.functional.softplus(z, threshold=80)
    g_tol = g.abs() * F32 * (24 + 2 * z.abs() + 2 * f(a_log).abs()) + 1e-37
    beta = torch.sigmoid(f(b))
    beta_tol = beta * F32 * (12 + 2 * f(b).abs()) + 1e-37
    return parts, g, g_tol, beta, beta_tol, last


def commit_ref(bt, k, g, u, x, paths, accepted):
    """The new states and inputs of all layers, and bounds on the states: a few roundings a path row of what it adds."""
    f = lambda z: z.detach().cpu().double()  # noqa: E731
    k, g, u, x, s_all, conv = f(k), f(g), f(u), f(x), f(bt.s).clone(), f(bt.conv).clone()
    group, tol = bt.hv // bt.hk, torch.zeros_like(f(bt.s))
    for s, n in enumerate(accepted):
        if n == 0:
            continue
        slot = bt.slot_n[s]
        rows = [int(bt.offsets_n[s]) + t for t in paths[s][:n]]
        S = s_all[:, slot] if bt.lens_n[s] > 0 else torch.zeros_like(s_all[:, slot])
        size = S.abs()
        for r in rows:
            kk = k[:, r].repeat_interleave(group, 1)
            e = g[:, r].exp()[..., None, None]
            S, size = S * e + kk[..., None] * u[:, r, :, None], size * e + (kk[..., None] * u[:, r, :, None]).abs()
        s_all[:, slot], tol[:, slot] = S, (3 * n + 8) * F32 * (1 + g[:, rows].abs().sum(1)[..., None, None]) * size + 1e-37
        old = conv[:, slot] if bt.lens_n[s] > 0 else torch.zeros_like(conv[:, slot])
        conv[:, slot] = torch.cat((old, x[:, rows]), 1)[:, -3:]
    return s_all, tol, conv


def verify_ref(probs, tokens, accept_u, draw_u, parents, offsets, draft=None, width=None):
    """Paths, accepted and next in exact fractions; q's products as the definition has them."""
    frac = lambda v: Fraction(float(min(v, 1))) if v > 0 else Fraction(0)  # noqa: E731
    P, Q = probs.cpu().double().numpy(), None if draft is None else draft.cpu().double().numpy()
    out = []
    for s in range(len(offsets) - 1):
        first, n = int(offsets[s]), int(offsets[s + 1] - offsets[s])
        if n == 0:
            out.append(([], -1))
            continue
        width_s = n if width is None else width
        way, r, m = [0], [frac(v) for v in P[first]], Fraction(1)
        for t in range(1, n):
            if len(way) == width_s:
                break
            if parents[s][t] != way[-1]:
                continue
            x, u = int(tokens[first + t]), Fraction(float(accept_u[first + t]))
            known = 0 <= x < P.shape[1]
            q = None if Q is None else [frac(v) for v in Q[first + way[-1]]]
            chance = (Fraction(1) if q is None else q[x]) if known else Fraction(0)
            if known and u * m * chance < r[x]:
                way, r, m = way + [t], [frac(v) for v in P[first + t]], Fraction(1)
            elif q is not None:
                r = [max(a - m * b, Fraction(0)) for a, b in zip(r, q)]
                m = sum(r)
            elif known:
                m, r[x] = max(m - r[x], Fraction(0)), Fraction(0)
        total = sum(r)
        if total == 0:
            r = [frac(v) for v in P[first + way[-1]]]
            total = sum(r)
        nxt, upto, border = -1, Fraction(0), Fraction(float(draw_u[s])) * total
        for i, v in enumerate(r):
            upto += v
            if upto > border:
                nxt = i
                break
        out.append((way, nxt))
    return out
