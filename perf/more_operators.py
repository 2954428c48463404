"""What the operators that keep a long context in bounded memory are measured
on: the attention weight that cached keys gather, eviction from the paged cache
by that weight, and the gated delta rule (packed sequences forward and
backward, and one token of each sequence against its state).

`run` computes each operator in a plain form of elementary torch operations
(own = False) or through the library's entry points (own = True); `exact`
gives the same results in 64 bits from the definitions.  Shapes are THD as in
the rest of the library; lengths are drawn from the case's own numbers, values
from the seed.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
_CHUNK = 64  # tokens of a chunk in the plain form of the delta rule


def listed():
    return [
        # one decoding step of 64 requests of ragged length: each key's share of its step's attention
        {"name": "weights decode 64 ragged", "op": "weights", "seqs": 64, "q_max": 1, "own_lo": 128, "own_hi": 8192,
         "prefix": 0, "groups": 0, "hq": 32, "hkv": 8, "d": 128, "page": 16, "hnd": False, "dtype": "bf16", "shape": 1},
        # a chunk of a long prompt against all that came before it: the largest product
        {"name": "weights chunk 2048 at 32768", "op": "weights", "seqs": 1, "q_max": 2048, "q_min": 2048,
         "own_lo": 32768, "own_hi": 32768, "prefix": 0, "groups": 0, "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "hnd": False, "dtype": "bf16", "shape": 2},
        # small chunks of several requests behind a shared document, in the exact type
        {"name": "weights fp32 prefix d64", "op": "weights", "seqs": 9, "q_max": 12, "own_lo": 12, "own_hi": 700,
         "prefix": 1500, "groups": 2, "hq": 8, "hkv": 2, "d": 64, "page": 16, "hnd": True, "dtype": "fp32", "shape": 3},
        # a batch of requests cut down to a fixed budget, each KV head by its own weights
        {"name": "evict 64 to 1024", "op": "evict", "seqs": 64, "n_lo": 700, "n_hi": 8192, "keep": 1024, "sinks": 4,
         "recent": 128, "per_head": True, "hkv": 8, "d": 128, "page": 16, "hnd": False, "dtype": "bf16", "shape": 4},
        # one long prompt behind its prefill
        {"name": "evict one 65536 to 4096", "op": "evict", "seqs": 1, "n_lo": 65536, "n_hi": 65536, "keep": 4096,
         "sinks": 16, "recent": 512, "per_head": True, "hkv": 8, "d": 128, "page": 64, "hnd": False, "dtype": "bf16",
         "shape": 5},
        # the exact type, odd sizes, one choice of tokens for all heads
        {"name": "evict fp32 shared odd", "op": "evict", "seqs": 7, "n_lo": 9, "n_hi": 1301, "keep": 333, "sinks": 1,
         "recent": 32, "per_head": False, "hkv": 2, "d": 64, "page": 16, "hnd": True, "dtype": "fp32", "shape": 6},
        # a training step's packed batch of documents, forward
        {"name": "delta fwd packed 32768", "op": "delta", "bwd": False, "seqs": 24, "len_lo": 128, "len_hi": 8192,
         "tokens": 32768, "hk": 16, "hv": 16, "dk": 128, "dv": 128, "state": False, "dtype": "bf16", "shape": 7},
        # a quarter of that batch, backward (nothing kept from the forward), two value heads for each key head
        {"name": "delta bwd packed 8192", "op": "delta", "bwd": True, "seqs": 7, "len_lo": 100, "len_hi": 4096,
         "tokens": 8192, "hk": 8, "hv": 16, "dk": 128, "dv": 128, "state": False, "dtype": "bf16", "shape": 8},
        # chunks of prompts that go on from the states of the chunks before them, in the exact type
        {"name": "delta fwd fp32 odd states", "op": "delta", "bwd": False, "seqs": 5, "len_lo": 1, "len_hi": 701,
         "tokens": 0, "hk": 2, "hv": 4, "dk": 64, "dv": 64, "state": True, "dtype": "fp32", "shape": 9},
        # the exact type backward, through initial and final states
        {"name": "delta bwd fp32 odd states", "op": "delta", "bwd": True, "seqs": 4, "len_lo": 1, "len_hi": 500,
         "tokens": 0, "hk": 2, "hv": 2, "dk": 64, "dv": 128, "state": True, "dtype": "fp32", "shape": 10},
        # one decoding step of 64 requests
        {"name": "delta step 64", "op": "step", "seqs": 64, "hk": 16, "hv": 32, "dk": 128, "dv": 128, "dtype": "bf16"},
        # one decoding step of three requests: latency
        {"name": "delta step 3", "op": "step", "seqs": 3, "hk": 4, "hv": 8, "dk": 64, "dv": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "evict", "evict", "delta", "delta", "delta", "step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    small = dtype == "fp32"
    shape = rng.randrange(1 << 20)
    if op in ("weights", "evict"):
        hkv = rng.choice([1, 2, 4, 8])
        page, hnd, d = rng.choice([8, 16, 24, 32, 64, 128]), rng.random() < 0.4, rng.choice([64, 128, 128])
        if op == "evict":
            n = _log(rng, 16, 20000)
            keep = _log(rng, 8, n)
            return {"op": op, "seqs": _log(rng, 1, 40), "n_lo": rng.choice([1, n // 2 + 1, n]), "n_hi": n, "keep": keep,
                    "sinks": rng.randint(0, keep // 4), "recent": rng.randint(0, keep // 2),
                    "per_head": rng.random() < 0.6, "hkv": hkv, "d": d, "page": page, "hnd": hnd, "dtype": dtype,
                    "shape": shape}
        groups, q_max = rng.choice([0, 0, 1, 2]), rng.choice([1, 1, 5, _log(rng, 8, 300)])
        most = (2000 if small else 20000) // ((q_max + 15) // 16)
        return {"op": op, "seqs": _log(rng, 1, 12 if q_max > 8 else 64), "q_max": q_max, "own_lo": 1,
                "own_hi": _log(rng, 2, 700 if small else 6000), "prefix": _log(rng, 10, most) if groups else 0,
                "groups": groups, "hq": hkv * rng.choice([1, 2, 4, 7, 8]), "hkv": hkv, "d": d, "page": page, "hnd": hnd,
                "dtype": dtype, "shape": shape}
    hk = rng.choice([1, 2, 4, 8])
    heads = {"hk": hk, "hv": hk * rng.choice([1, 1, 2]), "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]),
             "dtype": dtype}
    if op == "step":
        return {"op": op, "seqs": _log(rng, 1, 128), **heads}
    bwd = rng.random() < 0.5
    hi = _log(rng, 2, 500 if small else 900 if bwd else 2700)
    return {"op": op, "bwd": bwd, "seqs": _log(rng, 1, 6 if small else 12), "len_lo": 1, "len_hi": hi,
            "tokens": 0, "state": rng.random() < 0.5, "shape": shape, **heads}


# ------------------------------------------------------------------ lengths
def _lens(case):
    """The case's lengths: delta: tokens of each sequence; evict: cached tokens; weights: (new tokens, cached tokens
    with the new ones, sequences of each group, each group's prefix length)."""
    rng = random.Random(case["shape"])
    if case["op"] == "delta":
        lens = [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
        if case["tokens"]:  # that many tokens in all, none of a length above len_hi
            while sum(lens) != case["tokens"]:
                at, off = rng.randrange(len(lens)), case["tokens"] - sum(lens)
                lens[at] = min(max(lens[at] + off, case["len_lo"]), case["len_hi"])
        return lens
    if case["op"] == "evict":
        return [_log(rng, case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
    new = [rng.randint(case.get("q_min", 1), case["q_max"]) for _ in range(case["seqs"])]
    kv = [max(_log(rng, case["own_lo"], case["own_hi"]), n) for n in new]
    groups = case["groups"]
    cut = sorted(rng.randint(0, case["seqs"]) for _ in range(groups - 1))
    sizes = [b - a for a, b in zip([0] + cut, cut + [case["seqs"]])] if groups else []
    prefix = [case["prefix"] if g == 0 else rng.randint(0, case["prefix"]) for g in range(groups)]
    return new, kv, sizes, prefix


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = _TYPES[case["dtype"]]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if case["op"] in ("delta", "step"):
        hk, hv, dk, dv, N = case["hk"], case["hv"], case["dk"], case["dv"], case["seqs"]
        lens = _lens(case) if case["op"] == "delta" else [1] * N
        T = sum(lens)
        s["scale"] = 1.0 / math.sqrt(dk)
        # keys and queries of length one, gates as a layer's projections make them: most tokens forget little
        s["q"], s["k"] = (torch.nn.functional.normalize(randn(T, hk, dk).float(), dim=-1).to(dtype) for _ in range(2))
        s["v"] = randn(T, hv, dv)
        s["beta"] = torch.sigmoid(torch.randn(T, hv, generator=gen, device="cuda"))
        s["g"] = -0.15 * torch.nn.functional.softplus(torch.randn(T, hv, generator=gen, device="cuda") * 2 - 1)
        if case["op"] == "step":
            slots = torch.randperm(N + 5, generator=gen, device="cuda")[:N]
            s["slots"], s["state"] = slots.to(torch.int32), torch.randn(N + 5, hv, dk, dv, generator=gen, device="cuda")
            return s
        s["cu"], s["lens"] = ints(_cu(lens)), lens
        if case["state"]:
            s["state"] = torch.randn(N, hv, dk, dv, generator=gen, device="cuda") * 0.3
        if case["bwd"]:
            s["dout"] = randn(T, hv, dv)
            if case["state"]:
                s["dstate"] = torch.randn(N, hv, dk, dv, generator=gen, device="cuda") * 0.3
        s["chunks"] = _chunks(lens)
        return s

    page, hkv, d = case["page"], case["hkv"], case["d"]
    if case["op"] == "evict":
        kv, prefix = _lens(case), []
    else:
        new, kv, sizes, prefix = _lens(case)
    kept = [min(n, case["keep"]) for n in kv] if case["op"] == "evict" else []
    count = [-(-n // page) for n in kv + prefix + kept]
    pages = sum(count) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).tolist()
    tables, at = [], 0
    for lens in (kv, prefix, kept):
        width = max([-(-n // page) for n in lens] + [1])
        table = []
        for n in lens:
            c = -(-n // page)
            table.append(order[at:at + c] + [-1] * (width - c))
            at += c
        tables.append(table)
    s["table"], s["kv_lens"], s["kv_max"] = ints(tables[0]), ints(kv), max(kv)
    shape = (pages, hkv, page, d) if case["hnd"] else (pages, page, hkv, d)
    s["k_cache"], s["v_cache"] = randn(*shape), randn(*shape) if case["op"] == "evict" else None
    # gathered weights: a few keys hold most of it, some have none yet
    w = torch.exp(2.0 * torch.randn(pages, hkv, page, generator=gen, device="cuda"))
    w = w * (0.05 if case["op"] == "evict" else 0.001)
    s["weights"] = torch.where(rand(pages, hkv, page) < 0.05, torch.zeros_like(w), w).transpose(1, 2)
    if case["hnd"]:
        s["k_cache"] = s["k_cache"].transpose(1, 2)
        s["v_cache"] = s["v_cache"].transpose(1, 2) if case["op"] == "evict" else None
    if case["op"] == "evict":
        s["out_table"] = ints(tables[2])
        return s
    T, hq = sum(new), case["hq"]
    s["scale"], s["q"], s["cu"] = 1.0 / math.sqrt(d), randn(T, hq, d), ints(_cu(new))
    s["q_max"], s["prefix_max"] = max(new), max(prefix + [0])
    if sizes:
        s["ptable"], s["prefix_lens"], s["groups"] = ints(tables[1]), ints(prefix), ints(_cu(sizes))
        cu = _cu(new)
        s["group_cu"] = ints([cu[i] for i in _cu(sizes)])
        s["group_max"] = max(cu[b] - cu[a] for a, b in zip(_cu(sizes), _cu(sizes)[1:]))
    # what attention over the cache left: the log-sum-exp of each row
    lse = torch.full((T, hq), -math.inf, device="cuda")
    for scores, seg, j in _scores(s):
        lse = torch.logaddexp(lse, torch.logsumexp(scores, -1).transpose(1, 2)[seg, j].reshape(T, hq))
    s["lse"] = lse.t().contiguous()
    return s


def _chunks(lens):
    """Token indices of each chunk [chunks + 1, _CHUNK] (the number of all tokens where there is none; the last chunk
    is empty), and each sequence's chunks [most chunks, sequences] (the empty one behind the last)."""
    T, index, of, at = sum(lens), [], [], 0
    for n in lens:
        mine = []
        for c in range(0, n, _CHUNK):
            mine.append(len(index))
            index.append([at + i if i < n else T for i in range(c, c + _CHUNK)])
        of.append(mine)
        at += n
    most = max(len(x) for x in of)
    of = [x + [len(index)] * (most - len(x)) for x in of]
    index.append([T] * _CHUNK)
    return torch.tensor(index, device="cuda"), torch.tensor(of, device="cuda").t().contiguous()


# ------------------------------------------------------------------ plain forms
def _members(cu, tokens):
    """The segment of each of the tokens, and its place in it."""
    i = torch.arange(tokens, device="cuda")
    seg = (i[:, None] >= cu[None, 1:]).sum(1)
    return seg, i - cu[seg]


def _places(table, length, page):
    """Page and row of rows 0 .. length - 1 of each table's sequence (pages that are not there: page 0)."""
    i = torch.arange(length, device="cuda")
    return table[:, i // page].long().clamp(min=0), (i % page).expand(table.shape[0], -1)


def _scores(s):
    """For the own keys and for the prefixes: the scaled scores [S, Hkv, most tokens, G, keys], -inf where a token does
    not see a key, and segment and place of each token."""
    q, cu, kv_lens = s["q"], s["cu"], s["kv_lens"]
    T, hq, d = q.shape
    page, hkv = s["k_cache"].shape[1:3]
    new = cu[1:] - cu[:-1]

    def against(cu, count, most, table, length, limit):
        seg, j = _members(cu, T)
        x = torch.zeros(count, most, hkv, hq // hkv, d, device="cuda")
        x[seg, j] = q.float().view(T, hkv, hq // hkv, d)
        sees = torch.zeros(count, most, dtype=torch.int64, device="cuda")
        sees[seg, j] = limit(seg, j)
        k = s["k_cache"][_places(table, length, page)].float().permute(0, 2, 3, 1)
        y = x.transpose(1, 2).reshape(count, hkv, most * (hq // hkv), d) @ k * s["scale"]
        hidden = torch.arange(length, device="cuda") >= sees[:, None, :, None, None]
        return y.view(count, hkv, most, hq // hkv, length).masked_fill(hidden, -math.inf), seg, j

    yield against(cu, len(kv_lens), s["q_max"], s["table"], s["kv_max"],
                  lambda seg, j: (kv_lens[seg] - new[seg] + j + 1).long())
    if "ptable" in s and s["prefix_max"]:
        yield against(s["group_cu"], len(s["prefix_lens"]), s["group_max"], s["ptable"], s["prefix_max"],
                      lambda seg, j: s["prefix_lens"][seg].long())


def _weights(s):
    T, hq, _ = s["q"].shape
    page, hkv = s["k_cache"].shape[1:3]
    for (scores, seg, j), table, lens in zip(_scores(s), (s["table"], s.get("ptable")),
                                             (s["kv_lens"], s.get("prefix_lens"))):
        lse = torch.zeros(scores.shape[:4], device="cuda").transpose(1, 2)
        lse[seg, j] = s["lse"].t().reshape(T, hkv, hq // hkv)
        got = torch.exp(scores - lse.transpose(1, 2)[..., None]).sum((2, 3)).transpose(1, 2)
        pages, rows = _places(table, got.shape[1], page)
        there = torch.arange(got.shape[1], device="cuda") < lens[:, None]
        s["weights"][pages[there], rows[there]] += got[there]
    return s["weights"]


def _evict(s):
    case, lens, page = s["case"], s["kv_lens"].long(), s["k_cache"].shape[1]
    B, hkv, most, keep = len(lens), case["hkv"], s["kv_max"], case["keep"]
    i = torch.arange(most, device="cuda")
    pages, rows = _places(s["table"], most, page)
    w = s["weights"][pages, rows].transpose(1, 2)
    if not case["per_head"]:
        w = sum(w.unbind(1))[:, None]  # in the heads' order
    H = w.shape[1]
    n = lens[:, None]
    safe = (i < case["sinks"]) | (i >= n - case["recent"])
    rank = torch.where(i < n, 1 + safe.long(), 0)[:, None].expand(B, H, most)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.gather(rank, -1, order)
    order = torch.gather(order, -1, torch.sort(rank, dim=-1, descending=True, stable=True).indices)
    left = torch.minimum(lens, torch.tensor(keep, device="cuda"))
    kept = order[..., :keep]
    kept = torch.cat([kept, kept.new_zeros(B, H, keep - kept.shape[-1])], -1)
    there = torch.arange(keep, device="cuda") < left[:, None, None]
    kept = torch.sort(torch.where(there, kept, most), -1).values
    b, h, j = (there.expand(B, hkv, keep)).nonzero(as_tuple=True)
    src = kept.expand(B, hkv, keep)[b, h, j]
    frm = (s["table"][b, src // page].long(), src % page, h)
    to = (s["out_table"][b, j // page].long(), j % page, h)
    for x in (s["k_cache"], s["v_cache"], s["weights"]):
        x[to] = x[frm]
    kept = torch.where(there, kept, -1).to(torch.int32)
    return left.to(torch.int32), kept, s["k_cache"], s["v_cache"], s["weights"]


def _by_chunk(s, *names):
    """The tensors' rows in chunks, [chunks + 1, heads, _CHUNK, d] in 32 bits, 0 where a chunk has no token; q's and
    k's heads repeated for the value heads that share them."""
    index, case = s["chunks"][0], s["case"]
    for name in names:
        x = s[name].float()
        x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[index].transpose(1, 2)
        yield x.repeat_interleave(case["hv"] // case["hk"], 1) if name in ("q", "k") else x


def _tokens(s, x):
    """The rows of chunks [chunks + 1, heads, _CHUNK, ...] as [T, heads, ...]."""
    index = s["chunks"][0].flatten()
    y = x.transpose(1, 2).flatten(0, 1)
    out = y.new_empty(s["q"].shape[0] + 1, *y.shape[1:])
    out[index] = y
    return out[:-1]


def _local(s, k, g, beta):
    """What every chunk has by itself: the sums of its gates, their differences' exponentials on and below the
    diagonal, A = beta_i D_ij k_i k_j below it, and the inverse of I + A by doubling (A is nilpotent)."""
    G = g.cumsum(-1)
    low = torch.ones(_CHUNK, _CHUNK, device="cuda").tril().bool()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf))
    A = (beta[..., None] * D * (k @ k.transpose(-1, -2))).tril(-1)
    inv = torch.eye(_CHUNK, device="cuda") - A
    P = A @ A
    for _ in range(5):
        inv = inv + inv @ P
        P = P @ P
    return G, D, A, inv


def _states(s, k, v, G, beta, inv):
    """The state ahead of each chunk, the values that it writes, and the state behind each sequence."""
    case, of = s["case"], s["chunks"][1]
    W, U = inv @ (k * (beta * G.exp())[..., None]), inv @ (v * beta[..., None])
    last = G[..., -1:]
    K = k * torch.exp(last - G)[..., None]
    S = torch.zeros(case["seqs"], case["hv"], case["dk"], case["dv"], device="cuda")
    S = S + s["state"] if "state" in s else S
    before = S.new_zeros(len(k), *S.shape[1:])
    wrote = torch.zeros_like(v)
    for c in of:
        before[c] = S
        u = U[c] - W[c] @ S
        wrote[c] = u
        S = S * last[c].exp()[..., None] + K[c].transpose(-1, -2) @ u
    return before, wrote, S


def _delta(s):
    q, k, v, g, beta = _by_chunk(s, "q", "k", "v", "g", "beta")
    G, D, A, inv = _local(s, k, g, beta)
    before, wrote, S = _states(s, k, v, G, beta, inv)
    if not s["case"]["bwd"]:
        out = (q * G.exp()[..., None]) @ before + (q @ k.transpose(-1, -2) * D) @ wrote
        out = _tokens(s, out * s["scale"]).to(s["q"].dtype)
        return (out, S) if "state" in s else out
    dout = next(_by_chunk(s, "dout")) * s["scale"]
    eG, eL = G.exp()[..., None], torch.exp(G[..., -1:] - G)[..., None]
    last = G[..., -1:].exp()[..., None]
    P = q @ k.transpose(-1, -2) * D
    near = P.transpose(-1, -2) @ dout  # the gradient of what is written, from the same chunk
    W = inv @ (k * beta[..., None] * eG)
    dS = s["dstate"] if "dstate" in s else torch.zeros_like(S)
    after, dwrote = torch.zeros_like(before), torch.zeros_like(v)
    for c in s["chunks"][1].flip(0):
        after[c] = dS
        du = near[c] + (k * eL)[c] @ dS
        dwrote[c] = du
        dS = dS * last[c] + (q * eG)[c].transpose(-1, -2) @ dout[c] - W[c].transpose(-1, -2) @ du
    dR = inv.transpose(-1, -2) @ dwrote
    kS = k @ before
    dA = -(dR @ wrote.transpose(-1, -2)).tril(-1)
    dP = dout @ wrote.transpose(-1, -2) * D
    M = beta[..., None] * D * dA
    qfar = eG * (dout @ before.transpose(-1, -2))
    kfar = eL * (wrote @ after.transpose(-1, -2))
    kread = -beta[..., None] * eG * (dR @ before.transpose(-1, -2))
    dq = qfar + dP @ k
    dk = dP.transpose(-1, -2) @ q + kfar + kread + (M + M.transpose(-1, -2)) @ k
    dbeta = (dR * (v - eG * kS)).sum(-1) + (dA * D * (k @ k.transpose(-1, -2))).sum(-1)
    E = dP * (q @ k.transpose(-1, -2)) + dA * A
    dG = E.sum(-1) - E.sum(-2) + (qfar * q + kread * k - kfar * k).sum(-1)
    end = (kfar * k).sum((-1, -2)) + (before * after).sum((-1, -2)) * last[..., 0, 0]
    dg = dG.flip(-1).cumsum(-1).flip(-1) + end[..., None]
    share = (len(q), s["case"]["hk"], -1, _CHUNK, s["case"]["dk"])
    dq, dk = (x.view(share).sum(2) for x in (dq, dk))
    grads = [_tokens(s, x).to(s["q"].dtype) for x in (dq, dk, dR * beta[..., None])]
    grads += [_tokens(s, dg), _tokens(s, dbeta)]
    return (*grads, dS) if "state" in s else tuple(grads)


def _step(s):
    case, slots = s["case"], s["slots"].long()
    q, k = (s[n].float().repeat_interleave(case["hv"] // case["hk"], 1) for n in ("q", "k"))
    S = s["state"][slots] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"][slots] = S
    return ((q[..., None] * S).sum(-2) * s["scale"]).to(s["q"].dtype), s["state"]


def run(state):
    s, case = state, state["case"]
    if own:
        import context_varlen_ring_gb300 as ra
        if case["op"] == "weights":
            return ra.paged_attn_key_weights(s["q"], s["k_cache"], s["table"], s["cu"], s["kv_lens"], s["lse"],
                                             s["weights"], prefix_table=s.get("ptable"),
                                             prefix_lens=s.get("prefix_lens"), prefix_groups=s.get("groups"),
                                             scale=s["scale"], max_q_len=s["q_max"])
        if case["op"] == "evict":
            left, kept = ra.kv_cache_evict(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["kv_lens"],
                                           case["keep"], sinks=case["sinks"], recent=case["recent"],
                                           per_head=case["per_head"], out_table=s["out_table"])
            return left, kept, s["k_cache"], s["v_cache"], s["weights"]
        if case["op"] == "step":
            return ra.delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"],
                                      scale=s["scale"]), s["state"]
        if case["bwd"]:
            got = ra.delta_rule_bwd(s["dout"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"],
                                    state=s.get("state"), dstate=s.get("dstate"), scale=s["scale"])
            return got if case["state"] else got[:-1]
        out, last = ra.delta_rule_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], state=s.get("state"),
                                      scale=s["scale"], final_state=case["state"])
        return (out, last) if case["state"] else out
    return {"weights": _weights, "evict": _evict, "delta": _delta, "step": _step}[case["op"]](s)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("delta", "step"):
        return _exact_delta(case, s)
    page, hkv, table = case["page"], case["hkv"], s["table"].tolist()

    def rows(x, row, n):
        return x[torch.tensor(row[:-(-n // page)], device="cuda").long()].double().flatten(0, 1)[:n]

    w = s["weights"].double()
    if case["op"] == "weights":
        new, kv, sizes, prefix = _lens(case)
        cu, G = _cu(new), case["hq"] // hkv
        q, lse = s["q"].double(), s["lse"].double()

        def put(row, n, got):
            for p in range(-(-n // page)):
                part = got[p * page:(p + 1) * page]
                w[row[p], :len(part)] += part

        def of(a, b, keys, sees):
            got = torch.empty(len(keys), hkv, dtype=torch.float64, device="cuda")
            for h in range(hkv):
                x = torch.einsum("tgd,kd->tgk", q[a:b, h * G:(h + 1) * G], keys[:, h]) * s["scale"]
                x = torch.exp(x - lse[h * G:(h + 1) * G, a:b].t()[..., None])
                got[:, h] = (x * sees[:, None]).sum((0, 1))
            return got

        if sum(n * m for n, m in zip(new, kv)) * case["hq"] > 1 << 34:
            return None
        for b, n in enumerate(new):
            at = torch.arange(kv[b], device="cuda")
            sees = (at <= kv[b] - n + torch.arange(n, device="cuda")[:, None]).double()
            put(table[b], kv[b], of(cu[b], cu[b + 1], rows(s["k_cache"], table[b], kv[b]), sees))
        for g, (a, b) in enumerate(zip(_cu(sizes), _cu(sizes)[1:])):
            if cu[b] > cu[a] and prefix[g]:
                row = s["ptable"][g].tolist()
                one = torch.ones(cu[b] - cu[a], prefix[g], dtype=torch.float64, device="cuda")
                put(row, prefix[g], of(cu[a], cu[b], rows(s["k_cache"], row, prefix[g]), one))
        return w

    kv, keep, to = _lens(case), case["keep"], s["out_table"].tolist()
    k, v = s["k_cache"].double(), s["v_cache"].double()
    H = hkv if case["per_head"] else 1
    kept = torch.full((len(kv), H, keep), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(kv):
        mine = rows(s["weights"], table[b], n).float().cpu()
        left, first = min(n, keep), min(case["sinks"], n)
        last = max(n - case["recent"], first)
        for h in range(H):
            x = mine[:, h]
            if not case["per_head"]:
                for j in range(1, hkv):
                    x = x + mine[:, j]
            at = list(range(n))
            if n > keep:
                x = x.tolist()
                best = sorted(range(first, last), key=lambda i: (-x[i], i))[:left - first - (n - last)]
                at = list(range(first)) + sorted(best) + list(range(last, n))
            kept[b, h, :left] = torch.tensor(at, dtype=torch.int32)
        for h in range(hkv):
            at = kept[b, h if case["per_head"] else 0, :left].long()
            p, r = torch.tensor(table[b], device="cuda")[at // page], at % page
            j = torch.arange(left, device="cuda")
            op, orow = torch.tensor(to[b], device="cuda")[j // page], j % page
            for x in (k, v, w):
                x[op, orow, h] = x[p, r, h]
    return torch.tensor([min(n, keep) for n in kv], dtype=torch.int32), kept, k, v, w


def _exact_delta(case, s):
    """Token by token: S <- exp(g) S; u = beta (v - S^T k); S <- S + k u^T; o = scale S^T q, and back."""
    hv, share, scale = case["hv"], case["hv"] // case["hk"], s["scale"]
    q, k = (s[n].double().repeat_interleave(share, 1) for n in ("q", "k"))
    v, beta, a = s["v"].double(), s["beta"].double(), s["g"].double().exp()
    if case["op"] == "step":
        S = s["state"].double()
        for b, slot in enumerate(s["slots"].tolist()):
            x = S[slot] * a[b, :, None, None]
            u = beta[b, :, None] * (v[b] - torch.einsum("hkv,hk->hv", x, k[b]))
            S[slot] = x + torch.einsum("hk,hv->hkv", k[b], u)
        return torch.einsum("bhkv,bhk->bhv", S[s["slots"].long()], q) * scale, S
    lens = s["lens"]
    if case["bwd"] and sum(lens) * hv * case["dk"] * case["dv"] * 8 > 60e9:
        return None
    cu, N = torch.tensor(_cu(lens)[:-1], device="cuda"), len(lens)
    n = torch.tensor(lens, device="cuda")
    S = s["state"].double() if case["state"] else torch.zeros(N, hv, case["dk"], case["dv"], dtype=torch.float64,
                                                              device="cuda")
    out, kept = torch.zeros_like(v), []
    order = sorted(range(N), key=lambda b: -lens[b])  # the sequences that still have a token come first
    S, cu = S[order], cu[order]
    many = [sum(m > t for m in lens) for t in range(max(lens))]
    for t, m in enumerate(many):
        at = cu[:m] + t
        x = S[:m] * a[at][..., None, None]
        e = v[at] - (x.transpose(-1, -2) @ k[at][..., None])[..., 0]
        y = x + k[at][..., None] * (beta[at][..., None] * e)[..., None, :]
        out[at] = (y.transpose(-1, -2) @ q[at][..., None])[..., 0] * scale
        if case["bwd"]:
            kept.append((S[:m].clone(), e))
        S[:m] = y
    back = torch.tensor(order, device="cuda").argsort()
    if not case["bwd"]:
        return (out, S[back]) if case["state"] else out
    dout = s["dout"].double() * scale
    dS = s["dstate"].double()[order] if case["state"] else torch.zeros_like(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(beta), torch.zeros_like(beta)
    for t in range(len(many) - 1, -1, -1):
        m = many[t]
        at = cu[:m] + t
        S0, e = kept.pop()
        x = S0 * a[at][..., None, None]
        u = beta[at][..., None] * e
        y = x + k[at][..., None] * u[..., None, :]
        dq[at] = (y @ dout[at][..., None])[..., 0]
        dy = dS[:m] + q[at][..., None] * dout[at][..., None, :]
        du = (dy.transpose(-1, -2) @ k[at][..., None])[..., 0]
        db[at] = (du * e).sum(-1)
        de = beta[at][..., None] * du
        dv[at] = de
        dk[at] = (dy @ u[..., None])[..., 0] - (x @ de[..., None])[..., 0]
        dx = dy - k[at][..., None] * de[..., None, :]
        dg[at] = (dx * x).sum((-1, -2))
        dS[:m] = dx * a[at][..., None, None]
    dq, dk = (x.view(len(q), case["hk"], share, -1).sum(2) for x in (dq, dk))
    return (dq, dk, dv, dg, db, dS[back]) if case["state"] else (dq, dk, dv, dg, db)


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] in ("delta", "step"):
        hk, hv, dk, dv, N = case["hk"], case["hv"], case["dk"], case["dv"], case["seqs"]
        T = N if case["op"] == "step" else sum(_lens(case))
        rows, state = T * (2 * hk * dk + hv * dv) * e + 8 * T * hv, N * hv * dk * dv * 4
        once = 2 * T * hv * dk * dv  # a product of every token with its state
        if case["op"] == "step":
            return {"bytes": rows + T * hv * dv * e + 2 * state, "flops": 3 * once}
        some = 2 * state if case["state"] else 0
        if not case["bwd"]:
            return {"bytes": rows + T * hv * dv * e + some, "flops": 3 * once}
        return {"bytes": 2 * rows + T * hv * dv * e + 2 * some * 3 // 4, "flops": 8 * once}
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "evict":
        kv = _lens(case)
        left = sum(min(n, case["keep"]) for n in kv)
        H = hkv if case["per_head"] else 1
        return {"bytes": 4 * sum(kv) * hkv + left * hkv * (4 * d * e + 4) + 4 * len(kv) * H * case["keep"],
                "flops": sum(kv) * hkv}
    new, kv, sizes, prefix = _lens(case)
    rows = [sum(new[a:b]) for a, b in zip(_cu(sizes), _cu(sizes)[1:])]
    used = sum(p if n else 0 for p, n in zip(prefix, rows))
    seen = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, kv)) + sum(r * p for r, p in zip(rows, prefix))
    keys = sum(kv) + used
    return {"bytes": keys * hkv * (d * e + 8) + sum(new) * case["hq"] * (d * e + 4),
            "flops": 2 * d * case["hq"] * seen}
