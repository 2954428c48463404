"""What the serving and position operators are measured on: rotary positions
(forward and gradient), appending keys and values to a paged cache with the
rotation applied on the way, and attention over that cache for a batch that
may share a prefix.

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


def listed():
    return [
        # one training step's queries and keys: the packed 32768-token batch, positions restarting in each document
        {"name": "rope fwd packed 32768", "op": "rope", "bwd": False, "tokens": 32768, "hq": 32, "hkv": 8, "d": 128,
         "pairs": 64, "axes": 1, "adjacent": False, "packed": False, "dtype": "bf16"},
        # gradients of a video batch (time, height, width), read from one packed QKV gradient
        {"name": "rope bwd video 8192", "op": "rope", "bwd": True, "tokens": 8192, "hq": 64, "hkv": 8, "d": 128,
         "pairs": 64, "axes": 3, "adjacent": False, "packed": True, "dtype": "bf16"},
        # the exact type, an odd token count, half of each head rotated, neighbouring elements as pairs
        {"name": "rope fwd fp32 odd 2353", "op": "rope", "bwd": False, "tokens": 2353, "hq": 2, "hkv": 2, "d": 64,
         "pairs": 16, "axes": 1, "adjacent": True, "packed": False, "dtype": "fp32"},
        # one decoding step of 64 requests: latency
        {"name": "append decode 64", "op": "append", "seqs": 64, "new_lo": 1, "new_hi": 1, "past_hi": 8192, "hq": 32,
         "hkv": 8, "d": 128, "axes": 1, "page": 16, "hnd": False, "dtype": "bf16", "shape": 1},
        # prefill of packed prompts into fresh pages, straight from the packed QKV projection
        {"name": "append prefill packed", "op": "append", "seqs": 24, "new_lo": 128, "new_hi": 8192, "past_hi": 0,
         "hq": 32, "hkv": 8, "d": 128, "axes": 1, "page": 64, "hnd": False, "dtype": "bf16", "shape": 2},
        # chunks of image prompts in the exact type, three axes, a cache with heads outside the page's tokens
        {"name": "append fp32 chunks", "op": "append", "seqs": 23, "new_lo": 1, "new_hi": 701, "past_hi": 1300, "hq": 8,
         "hkv": 2, "d": 64, "axes": 3, "page": 16, "hnd": True, "dtype": "fp32", "shape": 3},
        # one request, one token: latency over a single long cache
        {"name": "attn one request 8192", "op": "attn", "seqs": 1, "q_max": 1, "own_lo": 8192, "own_hi": 8192,
         "prefix": 0, "groups": 0, "hq": 32, "hkv": 8, "d": 128, "page": 16, "hnd": False, "dtype": "bf16", "shape": 4},
        # a decoding batch without anything shared, ragged lengths
        {"name": "attn batch 64 ragged", "op": "attn", "seqs": 64, "q_max": 1, "own_lo": 128, "own_hi": 8192,
         "prefix": 0, "groups": 0, "hq": 32, "hkv": 8, "d": 128, "page": 16, "hnd": False, "dtype": "bf16", "shape": 5},
        # a decoding batch behind one long document
        {"name": "attn prefix 32768 x 64", "op": "attn", "seqs": 64, "q_max": 1, "own_lo": 128, "own_hi": 2048,
         "prefix": 32768, "groups": 1, "hq": 32, "hkv": 8, "d": 128, "page": 64, "hnd": False, "dtype": "bf16",
         "shape": 6},
        # the largest: many requests and query heads behind one very long document
        {"name": "attn prefix 65536 x 128", "op": "attn", "seqs": 128, "q_max": 1, "own_lo": 128, "own_hi": 1024,
         "prefix": 65536, "groups": 1, "hq": 64, "hkv": 8, "d": 128, "page": 64, "hnd": False, "dtype": "bf16",
         "shape": 7},
        # several tokens a request (drafted tokens being checked), two groups with a prefix each, heads outermost
        {"name": "attn drafts 2 groups", "op": "attn", "seqs": 24, "q_max": 6, "own_lo": 37, "own_hi": 4096,
         "prefix": 6000, "groups": 2, "hq": 32, "hkv": 8, "d": 128, "page": 32, "hnd": True, "dtype": "bf16",
         "shape": 8},
        # the exact type with small heads
        {"name": "attn fp32 d64", "op": "attn", "seqs": 9, "q_max": 2, "own_lo": 5, "own_hi": 700, "prefix": 1500,
         "groups": 1, "hq": 8, "hkv": 2, "d": 64, "page": 16, "hnd": False, "dtype": "fp32", "shape": 9},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128]) if dtype == "bf16" else rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    if op == "rope":
        return {"op": op, "bwd": rng.random() < 0.5, "tokens": _log(rng, 1, 16384), "hq": hq, "hkv": hkv, "d": d,
                "pairs": rng.choice([d // 2, d // 4, d // 2 - 3]), "axes": rng.choice([1, 3]),
                "adjacent": rng.random() < 0.4, "packed": rng.random() < 0.5, "dtype": dtype}
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "append":
        hi = _log(rng, 1, 1500)
        return {"op": op, "seqs": _log(rng, 1, 40), "new_lo": 1, "new_hi": hi, "past_hi": _log(rng, 1, 3000),
                "hq": hq, "hkv": hkv, "d": d, "axes": rng.choice([1, 3]), "page": page, "hnd": rng.random() < 0.4,
                "dtype": dtype, "shape": rng.randrange(1 << 20)}
    groups, q_max = rng.choice([0, 1, 1, 2, 3]), rng.choice([1, 1, 1, 3, 7])
    small = dtype == "fp32"
    most = (3000 if small else 30000) // ((q_max + 1) // 2)
    return {"op": op, "seqs": _log(rng, 1, 16 if small else 100), "q_max": q_max, "own_lo": 1,
            "own_hi": _log(rng, 2, 700 if small else 4096), "prefix": _log(rng, 40, most) if groups else 0,
            "groups": groups, "hq": hq, "hkv": hkv, "d": d, "page": page, "hnd": rng.random() < 0.4, "dtype": dtype, "shape": rng.randrange(1 << 20)}


# ------------------------------------------------------------------ lengths
def _lens(case):
    """The case's lengths: (new tokens, cached tokens with the new ones) of each sequence, sequences of each group,
    and each group's prefix length."""
    rng = random.Random(case["shape"])
    if case["op"] == "append":
        new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
        return new, [n + (rng.randint(0, case["past_hi"]) if case["past_hi"] else 0) for n in new], [], []
    new = [rng.randint(1, case["q_max"]) for _ in range(case["seqs"])]
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


def _inv_freq(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)


def _axes(pairs, axes):
    """The axis of each rotated pair: a quarter of them time, the rest height and width in turn."""
    a = torch.zeros(pairs, dtype=torch.uint8)
    if axes == 3:
        rest = torch.arange(pairs - pairs // 4)
        a[pairs // 4:] = (1 + rest % 2).to(torch.uint8)
    return a


def _positions(tokens, axes, start):
    """[axes, T] int32: a stream of tokens, or patches of a video of 24 x 24 from time `start` on."""
    i = torch.arange(tokens, device="cuda")
    if axes == 1:
        return (i + start)[None].to(torch.int32).contiguous()
    return torch.stack([start + i // 576, i // 24 % 24, i % 24]).to(torch.int32)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = _TYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    rng = random.Random(int(seed))
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "rope":
        T = case["tokens"]
        if case["packed"]:
            qkv = randn(T, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = randn(T, hq, d), randn(T, hkv, d)
        pos = _positions(T, case["axes"], rng.randrange(100000))
        if case["axes"] == 1:  # documents of up to 8192 tokens from one place in a long text on
            pos = pos % 8192 + rng.randrange(1 << 17)
        _rotation(s, case["pairs"], case["axes"], pos.to(torch.int32).contiguous())
        return s

    new, kv, sizes, prefix = _lens(case)
    page, T = case["page"], sum(new)
    s["cu"], s["kv_lens"] = ints(_cu(new)), ints(kv)
    width = max(-(-n // page) for n in kv)
    pwidth = max([-(-n // page) for n in prefix] + [1])
    need = sum(-(-n // page) for n in kv) + sum(-(-n // page) for n in prefix)
    pages = need + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).tolist()
    at = 0
    table, ptable = [], []
    for lens, rows, w in ((kv, table, width), (prefix, ptable, pwidth)):
        for n in lens:
            c = -(-n // page)
            rows.append(order[at:at + c] + [-1] * (w - c))
            at += c
    s["table"] = ints(table)
    shape = (pages, hkv, page, d) if case["hnd"] else (pages, page, hkv, d)
    s["k_cache"], s["v_cache"] = randn(*shape), randn(*shape)
    if case["hnd"]:
        s["k_cache"], s["v_cache"] = s["k_cache"].transpose(1, 2), s["v_cache"].transpose(1, 2)
    if case["op"] == "append":
        qkv = randn(T, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pos = _positions(T, case["axes"], 0)
        if case["axes"] == 1:
            first = [n - a for n, a in zip(kv, new)]
            pos = torch.cat([torch.arange(f, f + n, device="cuda") for f, n in zip(first, new)])[None]
        _rotation(s, d // 2, case["axes"], (pos + rng.randrange(64)).to(torch.int32).contiguous())
        return s
    s["q"] = randn(T, hq, d)
    s["q_max"], s["kv_max"], s["prefix_max"] = max(new), max(kv), max(prefix + [0])
    if sizes:
        s["ptable"], s["prefix_lens"], s["groups"] = ints(ptable), ints(prefix), ints(_cu(sizes))
        cu = _cu(new)
        s["group_cu"] = ints([cu[i] for i in _cu(sizes)])
        s["group_max"] = max(cu[b] - cu[a] for a, b in zip(_cu(sizes), _cu(sizes)[1:]))
    return s


def _rotation(s, pairs, axes, pos):
    s["pos"], s["inv_freq"], s["axes"] = pos, _inv_freq(pairs), _axes(pairs, axes)
    s["inv_freq_dev"], s["axes_dev"] = s["inv_freq"].cuda(), s["axes"].cuda().long()


# ------------------------------------------------------------------ plain forms
def _rotate(x, s, adjacent, inverse):
    """x [T, H, d] with its first 2 * pairs elements of each head rotated; angles in 64 bits, the rest in 32."""
    n = s["inv_freq_dev"].numel()
    angle = s["pos"][s["axes_dev"]].t().double() * s["inv_freq_dev"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    y = x.float()
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if adjacent else (y[..., :n], y[..., n:2 * n])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([ra, rb], -1).flatten(-2) if adjacent else torch.cat([ra, rb], -1)
    return torch.cat([r, y[..., 2 * n:]], -1).to(x.dtype)


def _members(cu, tokens):
    """The segment of each of the tokens, and its place in it."""
    i = torch.arange(tokens, device="cuda")
    seg = (i[:, None] >= cu[None, 1:]).sum(1)
    return seg, i - cu[seg]


def _gather(cache, table, length):
    """Rows 0 .. length - 1 of each table's sequence: [S, Hkv, length, d] in 32 bits (pages that are not there: page 0)."""
    i = torch.arange(length, device="cuda")
    page = cache.shape[1]
    return cache[table[:, i // page].long().clamp(min=0), i % page].float().transpose(1, 2)


def _attend(q, k, v, visible, scale):
    """q [S, H, n, G, d] against k, v [S, H, L, d] where visible [S, n, L]: the running maximum, sum and product."""
    S, H, n, G, d = q.shape
    x = (q.reshape(S, H, n * G, d) @ k.transpose(2, 3)).view(S, H, n, G, -1) * scale
    x = x.masked_fill(~visible[:, None, :, None], -math.inf)
    m = x.amax(-1)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0)[..., None])
    return m, p.sum(-1), (p.view(S, H, n * G, -1) @ v).view(S, H, n, G, d)


def _attention(s):
    q, cu, kv_lens = s["q"], s["cu"], s["kv_lens"]
    T, hq, d = q.shape
    hkv = s["k_cache"].shape[2]
    heads = q.float().view(T, hkv, hq // hkv, d)

    def against(cu, count, most, table, length, limit):
        seg, j = _members(cu, T)
        x = torch.zeros(count, most, hkv, hq // hkv, d, device="cuda")
        x[seg, j] = heads
        visible = torch.zeros(count, most, 1, dtype=torch.int64, device="cuda")
        visible[seg, j, 0] = limit(seg, j)
        visible = torch.arange(length, device="cuda") < visible
        k, v = _gather(s["k_cache"], table, length), _gather(s["v_cache"], table, length)
        return [t.transpose(1, 2)[seg, j] for t in _attend(x.transpose(1, 2), k, v, visible, s["scale"])]

    new = cu[1:] - cu[:-1]
    m, l, acc = against(cu, len(kv_lens), s["q_max"], s["table"], s["kv_max"],
                        lambda seg, j: (kv_lens[seg] - new[seg] + j + 1).long())
    if "ptable" in s and s["prefix_max"]:
        m2, l2, acc2 = against(s["group_cu"], len(s["prefix_lens"]), s["group_max"], s["ptable"], s["prefix_max"],
                               lambda seg, j: s["prefix_lens"][seg].long())
        top = torch.maximum(m, m2)
        safe = top.masked_fill(top == -math.inf, 0.0)
        w, w2 = torch.exp(m - safe), torch.exp(m2 - safe)
        m, l, acc = top, l * w + l2 * w2, acc * w[..., None] + acc2 * w2[..., None]
    out = acc / torch.where(l > 0, l, torch.ones_like(l))[..., None]
    return out.reshape(T, hq, d).to(q.dtype), (m + l.log()).reshape(T, hq).t().contiguous()


def run(state):
    s, case = state, state["case"]
    if own:
        import context_varlen_ring_gb300 as ra
        if case["op"] == "rope":
            call = ra.rope_bwd if case["bwd"] else ra.rope_fwd
            return call(s["q"], s["k"], s["pos"], s["inv_freq"], axes=s["axes"], adjacent=case["adjacent"])
        if case["op"] == "append":
            q = ra.kv_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"],
                                   q=s["q"], pos=s["pos"], inv_freq=s["inv_freq"], axes=s["axes"])
            return q, s["k_cache"], s["v_cache"]
        return ra.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"],
                                 prefix_table=s.get("ptable"), prefix_lens=s.get("prefix_lens"),
                                 prefix_groups=s.get("groups"), scale=s["scale"], max_q_len=s["q_max"])
    if case["op"] == "rope":
        return (_rotate(s["q"], s, case["adjacent"], case["bwd"]), _rotate(s["k"], s, case["adjacent"], case["bwd"]))
    if case["op"] == "append":
        seg, j = _members(s["cu"], s["k"].shape[0])
        new = s["cu"][1:] - s["cu"][:-1]
        i = (s["kv_lens"] - new)[seg] + j
        page = s["table"][seg, i // case["page"]].long()
        s["k_cache"][page, i % case["page"]] = _rotate(s["k"], s, False, False)
        s["v_cache"][page, i % case["page"]] = s["v"]
        return _rotate(s["q"], s, False, False), s["k_cache"], s["v_cache"]
    return _attention(s)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)

    def turned(x, adjacent, sign):
        z = x.double()
        n = s["inv_freq"].numel()
        pos = s["pos"].double().cpu()
        angle = torch.stack([pos[int(a)] * f for a, f in zip(s["axes"], s["inv_freq"])], 1).cuda()
        by = torch.complex(torch.cos(angle), sign * torch.sin(angle))[:, None, :]
        re, im = (z[..., 0:2 * n:2], z[..., 1:2 * n:2]) if adjacent else (z[..., :n], z[..., n:2 * n])
        w = torch.complex(re.contiguous(), im.contiguous()) * by
        y = z.clone()
        if adjacent:
            y[..., 0:2 * n:2], y[..., 1:2 * n:2] = w.real, w.imag
        else:
            y[..., :n], y[..., n:2 * n] = w.real, w.imag
        return y

    if case["op"] == "rope":
        sign = -1.0 if case["bwd"] else 1.0
        return turned(s["q"], case["adjacent"], sign), turned(s["k"], case["adjacent"], sign)
    new, kv, sizes, prefix = _lens(case)
    cu = _cu(new)
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k, table = turned(s["k"], False, 1.0), s["table"].tolist()
        for b, n in enumerate(new):
            at = range(kv[b] - n, kv[b])
            page = torch.tensor([table[b][i // case["page"]] for i in at], device="cuda")
            slot = torch.tensor([i % case["page"] for i in at], device="cuda")
            kc[page, slot], vc[page, slot] = k[cu[b]:cu[b + 1]], s["v"][cu[b]:cu[b + 1]].double()
        return turned(s["q"], False, 1.0), kc, vc

    def keys(cache, row, length):
        c = -(-length // case["page"])
        return cache[row[:c].long()].double().flatten(0, 1)[:length].transpose(0, 1)

    T, hq, d = s["q"].shape
    hkv = case["hkv"]
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device="cuda")
    of = [g for g, n in enumerate(sizes) for _ in range(n)] or [None] * len(new)
    held, pk, pv = -1, None, None
    for b, n in enumerate(new):
        k, v = keys(s["k_cache"], s["table"][b], kv[b]), keys(s["v_cache"], s["table"][b], kv[b])
        shared = 0
        if of[b] is not None:
            shared = prefix[of[b]]
            if of[b] != held:
                held = of[b]
                pk, pv = keys(s["k_cache"], s["ptable"][held], shared), keys(s["v_cache"], s["ptable"][held], shared)
        for j in range(n):
            t, sees = cu[b] + j, kv[b] - n + j + 1
            q = s["q"][t].double().view(hkv, hq // hkv, d)
            x = q @ k[:, :sees].transpose(1, 2)
            if shared:
                x = torch.cat([q @ pk.transpose(1, 2), x], 2)
            x = x * s["scale"]
            z = torch.logsumexp(x, 2)
            p = torch.exp(x - z[..., None])
            y = p[..., shared:] @ v[:, :sees]
            if shared:
                y = y + p[..., :shared] @ pv
            out[t], lse[:, t] = y.reshape(hq, d), z.reshape(hq)
    return out, lse


def work(case):
    e = _BYTES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        T = case["tokens"]
        return {"bytes": 2 * T * (hq + hkv) * d * e + 4 * T * case["axes"], "flops": 6 * T * (hq + hkv) * case["pairs"]}
    new, kv, sizes, prefix = _lens(case)
    T = sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * T * (hq + 2 * hkv) * d * e + 4 * T * case["axes"], "flops": 6 * T * (hq + hkv) * d // 2}
    rows = [sum(new[a:b]) for a, b in zip(_cu(sizes), _cu(sizes)[1:])]
    used = [p if n else 0 for p, n in zip(prefix, rows)]
    seen = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, kv)) + sum(r * p for r, p in zip(rows, prefix))
    return {"bytes": 2 * (sum(kv) + sum(used)) * hkv * d * e + 2 * T * hq * d * e + 4 * T * hq, "flops": 4 * d * hq * seen}
