"""64-bit plain forms of key weights, eviction and the gated delta rule for the
tests, with error bounds derived from the arithmetic of the kernels."""
import numpy as np
import torch

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step, relative


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ key weights
def key_weights(q, kc, table, cu, lens, lse, w, ptable=(), plens=(), groups=(0,), causal=True, scale=1.0):
    """(weights, bound): a term's exponent carries the fp32 rounding of its d products, of the scale and of lse; its
    exponential two units in the last place; a key's sum one rounding a term, at most, and one into the weight."""
    T, Hq, d = q.shape
    page, Hkv = kc.shape[1:3]
    G = Hq // Hkv
    out, bound = w.copy(), np.zeros_like(w)
    adds = np.zeros(w.shape)

    def add(t, row, sees):
        i = np.arange(sees)
        p, r = np.asarray(row)[i // page], i % page
        for h in range(Hq):
            if lse[h, t] == -np.inf or not sees:
                continue
            k = kc[p, r, h // G]
            s = k @ q[t, h] * scale
            x = np.exp(s - lse[h, t])
            e = (d + 8) * 2.0 ** -23 * (np.abs(k) @ np.abs(q[t, h])) * abs(scale) + 4 * 2.0 ** -23 * (
                np.abs(s) + abs(lse[h, t])) + 2.0 ** -21
            out[p, r, h // G] += x
            bound[p, r, h // G] += x * e
            adds[p, r, h // G] += 1

    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        for j in range(n):
            t = int(cu[b]) + j
            add(t, table[b], int(lens[b]) - n + j + 1 if causal else int(lens[b]))
            for g in range(len(plens)):
                if groups[g] <= b < groups[g + 1]:
                    add(t, ptable[g], int(plens[g]))
    bound += (adds + 2) * 2.0 ** -24 * np.abs(out) * (adds > 0) + (adds > 0) * 1e-37  # (below it results are flushed)
    return out, bound * 1.01


# ------------------------------------------------------------------ eviction
def evict(weights, table, lens, keep, keep_lens=None, sinks=0, recent=0, per_head=True):
    """(new lengths, kept [B, H, keep]) of weights [pages, page, Hkv] fp32."""
    page, Hkv = weights.shape[1:]
    B, H = len(lens), Hkv if per_head else 1
    left, kept = np.zeros(B, np.int32), np.full((B, H, keep), -1, np.int32)
    for b in range(B):
        n, k = int(lens[b]), keep if keep_lens is None else min(max(int(keep_lens[b]), 0), keep)
        left[b] = min(n, k)
        i = np.arange(n)
        for h in range(H):
            if n <= k:
                kept[b, h, :n] = i
                continue
            w = weights[np.asarray(table[b])[i // page], i % page]
            x = w[:, h].copy()
            if not per_head:
                x = w[:, 0].copy()
                with np.errstate(over="ignore", invalid="ignore"):
                    for j in range(1, Hkv):
                        x = (x + w[:, j]).astype(np.float32)
            first = min(sinks, k)
            last = min(recent, k - first)
            nan = np.isnan(x)
            x[nan] = 0
            mid = i[first:n - last]
            # by weight, NaN behind all, and of equal ones the first
            order = np.lexsort((mid, -x[mid].astype(np.float64), nan[mid]))
            best = np.sort(mid[order[:k - first - last]])
            kept[b, h, :k] = np.concatenate([i[:first], best, i[n - last:]])
    return left, kept


def moved(x, table, to, left, kept):
    """The cache (or weights) [pages, page, Hkv, ...] after the move, by rows."""
    page, Hkv = x.shape[1:3]
    y = x.clone()
    for b in range(len(left)):
        for h in range(Hkv):
            for j in range(int(left[b])):
                i = int(kept[b, h if kept.shape[1] > 1 else 0, j])
                y[to[b][j // page], j % page, h] = x[table[b][i // page], i % page, h]
    return y


# ------------------------------------------------------------------ the gated delta rule
def delta(q, k, v, g, beta, cu, state, scale):
    """(out, final states) in 64 bits, token by token, differentiable by torch."""
    share = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    out, last = [], []
    for b in range(len(cu) - 1):
        S = state[b]
        for t in range(cu[b], cu[b + 1]):
            S = S * torch.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
            S = S + torch.einsum("hk,hv->hkv", k[t], u)
            out.append(torch.einsum("hkv,hk->hv", S, q[t]) * scale)
        last.append(S)
    return (torch.stack(out) if out else v[:0] * 1.0), torch.stack(last)


def delta_check(got, want, what=""):
    """A result of the chunked kernels against 64 bits.

    fp32: a product of tiles adds at most 128 / 16 x 6 times into an accumulator that may cut what it adds to 2^-23, all
    in one direction: 48 x 2^-23 relative; four products follow one another from the inputs to a result, so 2.3e-5 of
    the result's norm, and of its largest element with the factor between a sum of magnitudes and a sum (64 terms of
    random signs: 8) for a single one.  bf16: half a step of each element, and what its 16-bit operands leave
    (3 x 2^-16 a product, four of them, the same factor), a part in 680 of the largest."""
    want = want.detach()
    fp32 = got.dtype == torch.float32
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not want.numel():
        return
    assert torch.isfinite(got).all(), what
    err, top = (got - want).abs(), want.abs().max()
    if fp32:
        assert err.norm() <= 2.3e-5 * want.norm() + 1e-30, (what, float(err.norm() / want.norm()))
        assert err.max() <= 8 * 2.3e-5 * top + 1e-30, (what, float(err.max() / top))
    else:
        assert (err <= 2.0 ** -8 * want.abs() + 8 * 12 * 2.0 ** -16 * top + 1e-30).all(), (what, float(err.max() / top))
