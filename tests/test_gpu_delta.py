"""The gated delta rule against its plain 64-bit form, token by token
(tests/keep_ref.py), and its gradients against torch's of that form."""
import math
import threading

import numpy as np
import pytest
import torch

import keep_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ra():
    assert torch.cuda.is_available()
    from context_varlen_ring_gb300 import build as b
    b.build()
    import context_varlen_ring_gb300 as m
    m.lib()
    torch.cuda.set_device(0)
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, hk, hv, dk, dv, dtype, gates="usual", seed=0, tail=0, packed=False):
    """Inputs on the GPU of sum(lens) + tail tokens (the tail behind the last sequence)."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)

    def unit(*s):
        return torch.nn.functional.normalize(torch.randn(*s, generator=g), dim=-1).to(TYPES[dtype]).cuda()

    q, k = unit(T, hk, dk), unit(T, hk, dk)
    v = torch.randn(T, hv, dv, generator=g).to(TYPES[dtype]).cuda()
    if packed:  # slices of one projection
        row = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        a, b = hk * dk, 2 * hk * dk
        q, k, v = row[:, :a].view(T, hk, dk), row[:, a:b].view(T, hk, dk), row[:, b:].view(T, hv, dv)
    beta = torch.sigmoid(torch.randn(T, hv, generator=g))
    gate = -0.2 * torch.nn.functional.softplus(torch.randn(T, hv, generator=g) * 2)
    if gates == "none":       # nothing is forgotten
        gate = torch.zeros(T, hv)
    elif gates == "strong":   # almost all is forgotten, each token
        gate = gate * 60
    elif gates == "reset":    # now and then everything, by -inf and by values that no exponential can tell from it
        hit = torch.rand(T, hv, generator=g)
        gate = torch.where(hit < 0.05, torch.tensor(-math.inf), torch.where(hit < 0.1, torch.tensor(-3e5), gate))
        gate = torch.where((hit > 0.1) & (hit < 0.15), torch.tensor(-900.0), gate)
    elif gates == "edges":    # tokens that write nothing, or all of it
        beta = torch.where(torch.rand(T, hv, generator=g) < 0.3, torch.zeros(()), beta)
        beta = torch.where(torch.rand(T, hv, generator=g) < 0.3, torch.ones(()), beta)
    return q, k, v, gate.cuda(), beta.cuda(), cu, ints(cu)


def states(n, hv, dk, dv, seed):
    return (torch.randn(n, hv, dk, dv, generator=torch.Generator().manual_seed(seed)) * 0.3).cuda()


def ref(q, k, v, g, beta, cu, state, scale, dout=None, dstate=None):
    """64 bits on the CPU; with dout the gradients too."""
    leaves = [x.detach().double().cpu() for x in (q, k, v, g, beta)]
    leaves[3] = leaves[3].clamp(min=-1e4)  # (the gradient of -inf by autograd would be nan)
    zero = torch.zeros(len(cu) - 1, v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64)
    leaves.append(zero if state is None else state.double().cpu())
    if dout is None:
        return R.delta(*leaves[:5], cu, leaves[5], scale)
    for x in leaves:
        x.requires_grad_()
    out, last = R.delta(*leaves[:5], cu, leaves[5], scale)
    total = (out * dout.double().cpu()[:cu[-1]]).sum()
    if dstate is not None:
        total = total + (last * dstate.double().cpu()).sum()
    return torch.autograd.grad(total, leaves, allow_unused=True)


CASES = [  # lens, hk, hv, dk, dv, dtype, gates, state, packed
    ([1], 1, 1, 64, 64, "bf16", "usual", False, False),
    ([64], 1, 2, 128, 128, "bf16", "usual", True, False),
    ([65], 2, 2, 128, 64, "bf16", "strong", False, True),
    ([63, 1, 0, 130, 17], 2, 4, 64, 128, "bf16", "usual", True, True),
    ([200, 64, 128], 1, 3, 128, 128, "bf16", "none", False, False),
    ([0, 0, 5], 2, 2, 64, 64, "bf16", "edges", True, False),
    ([90, 70], 1, 2, 128, 128, "bf16", "reset", True, False),
    ([1, 1, 1, 1], 1, 1, 64, 128, "fp32", "usual", True, False),
    ([129, 33], 2, 2, 64, 64, "fp32", "usual", False, True),
    ([63, 64, 65, 0], 1, 2, 128, 128, "fp32", "edges", True, False),
    ([150], 1, 1, 128, 64, "fp32", "reset", True, False),
    ([100, 100], 2, 4, 64, 128, "fp32", "strong", True, False),
    ([300], 1, 1, 64, 64, "fp32", "none", False, False),
]


@pytest.mark.parametrize("lens,hk,hv,dk,dv,dtype,gates,state,packed", CASES)
def test_forward(ra, lens, hk, hv, dk, dv, dtype, gates, state, packed):
    q, k, v, g, beta, cu, cud = make(lens, hk, hv, dk, dv, dtype, gates, seed=dk + sum(lens), tail=3, packed=packed)
    s0 = states(len(lens), hv, dk, dv, 1) if state else None
    scale = 0.3
    want, last = ref(q, k, v, g, beta, cu, s0, scale)
    out = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    got, s1 = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, final_state=True, scale=scale, out=out)
    assert got is out and ra.device_status() == 0
    R.delta_check(got[:cu[-1]], want, "out")
    R.delta_check(s1, last, "state")
    assert (got[cu[-1]:] == 7.0).all()  # (rows behind the last sequence)
    # without the last state: fewer bits inside, the same result to the type's rounding
    got, none = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, scale=scale)
    assert none is None
    R.delta_check(got[:cu[-1]], want, "out alone")
    if state:  # in place in a pool, the sequences' places in any order, one of them none
        pool = states(len(lens) + 3, hv, dk, dv, 2)
        slots = [len(lens) + 1 - i for i in range(len(lens))]
        for b, s in enumerate(slots):
            pool[s] = s0[b]
        before = pool.clone()
        got2, same = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=pool, slots=ints(slots), state_out=pool, scale=scale)
        assert same is pool and torch.equal(pool[slots], s1)
        rest = [i for i in range(len(pool)) if i not in slots]
        assert torch.equal(pool[rest], before[rest])
        pool = before.clone()
        got3, _ = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=pool, slots=ints([-1] + slots[1:]), state_out=pool,
                                    scale=scale)
        assert torch.equal(pool[slots[0]], before[slots[0]]) and torch.equal(got3[cu[1]:cu[-1]], got2[cu[1]:cu[-1]])
        s0z = s0.clone()
        s0z[0] = 0
        R.delta_check(got3[:cu[-1]], ref(q, k, v, g, beta, cu, s0z, scale)[0], "no slot")
        assert ra.device_status() == 0


@pytest.mark.parametrize("lens,hk,hv,dk,dv,dtype,gates,state,packed", CASES)
def test_gradients(ra, lens, hk, hv, dk, dv, dtype, gates, state, packed):
    q, k, v, g, beta, cu, cud = make(lens, hk, hv, dk, dv, dtype, gates, seed=dv + sum(lens), tail=2, packed=packed)
    s0 = states(len(lens), hv, dk, dv, 1) if state else None
    ds = states(len(lens), hv, dk, dv, 3) if state else None
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(9)).to(v.dtype).cuda()
    scale = 0.4
    want = ref(q, k, v, g, beta, cu, s0, scale, dout, ds)
    got = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=ds, scale=scale)
    assert ra.device_status() == 0 and (got[5] is not None) == state
    n = cu[-1]
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        R.delta_check(x[:n], y[:n], name)
    if state:
        R.delta_check(got[5], want[5], "dstate0")
        again = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=torch.cat([s0 * 0, s0]),
                                  slots=ints([len(lens) + i for i in range(len(lens))]), dstate=ds, scale=scale)
        assert all(torch.equal(a[:n] if i < 5 else a, b[:n] if i < 5 else b) for i, (a, b) in enumerate(zip(again, got)))


def test_gradients_match_differences(ra):
    """fp32, a central difference along a random direction of all inputs.  The loss is a sum of 64-bit products of fp32
    outputs that are 2.3e-5 off at most (tests/keep_ref.py): |dL| <= 2 x 2.3e-5 |out| |dout| / (2 h), and the difference's
    own error is O(h^2)."""
    q, k, v, g, beta, cu, cud = make([70, 9], 1, 2, 64, 64, "fp32", "usual", 5)
    s0 = states(2, 2, 64, 64, 6)
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).cuda()
    dlast = states(2, 2, 64, 64, 7)
    grads = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=dlast)
    x = [q, k, v, g, beta, s0]
    gen = torch.Generator().manual_seed(2)
    dirs = [torch.randn(t.shape, generator=gen).cuda() * (0.01 if i == 3 else 0.1) for i, t in enumerate(x)]
    h = 1 / 32

    def loss(sign):
        y = [t + sign * h * d for t, d in zip(x, dirs)]
        out, last = ra.delta_rule_fwd(*y[:5], cud, state=y[5], final_state=True)
        return float((out.double() * dout).sum() + (last.double() * dlast).sum()), float(out.norm() * dout.norm())

    (hi, size), (lo, _) = loss(1), loss(-1)
    along = sum(float((a.double() * d).sum()) for a, d in zip(grads, dirs))
    # third differences: the exact derivative along h is known to the same formula at h / 2
    h2, h = h, h / 2
    (hi2, _), (lo2, _) = loss(1), loss(-1)
    d1, d2 = (hi - lo) / (2 * h2), (hi2 - lo2) / (2 * h)
    best = (4 * d2 - d1) / 3
    assert abs(along - best) <= abs(d1 - d2) + 3 * 2.3e-5 * size / h, (along, best, d1, d2)


@pytest.mark.parametrize("hk,hv,dk,dv,dtype", [(1, 1, 64, 64, "bf16"), (2, 4, 128, 128, "bf16"), (1, 3, 64, 128, "fp32"),
                                               (2, 2, 128, 64, "fp32")])
@pytest.mark.parametrize("B", [1, 5, 33])
def test_step(ra, hk, hv, dk, dv, dtype, B):
    q, k, v, g, beta, cu, cud = make([1] * B, hk, hv, dk, dv, dtype, "edges", B, packed=True)
    g[0] = -math.inf
    s0 = states(B, hv, dk, dv, 4)
    want, last = ref(q, k, v, g, beta, cu, s0, 0.2)
    pool = states(B + 2, hv, dk, dv, 5)
    slots = [(i + 2) % (B + 2) for i in range(B)]
    pool[slots] = s0
    before = pool.clone()
    got = ra.delta_rule_step(q, k, v, g, beta, pool, slots=ints(slots), scale=0.2)
    R.delta_check(got, want, "out")
    R.delta_check(pool[slots], last, "state")
    rest = [i for i in range(B + 2) if i not in slots]
    assert torch.equal(pool[rest], before[rest])
    # the pool as it is, and a padded row
    alone = s0.clone()
    assert torch.equal(ra.delta_rule_step(q, k, v, g, beta, alone, scale=0.2), got) and torch.equal(alone, pool[slots])
    pool = before.clone()
    out = torch.full(v.shape, 3.0, dtype=v.dtype, device="cuda")
    ra.delta_rule_step(q, k, v, g, beta, pool, slots=ints(slots[:-1] + [-1]), scale=0.2, out=out)
    assert torch.equal(out[:-1], got[:-1]) and (out[-1] == 0).all() and torch.equal(pool[slots[-1]], before[slots[-1]])
    assert ra.device_status() == 0


def test_steps_continue_a_packed_call(ra):
    """A prompt by the packed call and its next tokens by steps: the outputs and the state of the whole in one call, to
    the states' fp32 bound."""
    q, k, v, g, beta, cu, cud = make([100, 37], 2, 2, 64, 128, "bf16", "usual", 3)
    whole, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, final_state=True)
    cut = [80, 17]
    rows = list(range(80)) + list(range(100, 117))
    out, s = ra.delta_rule_fwd(*(x[rows] for x in (q, k, v, g, beta)), ints([0, 80, 97]), final_state=True)
    assert (out[:80].float() - whole[:80].float()).abs().max() <= 2.0 ** -7 * whole.float().abs().max()
    for i in range(20):
        at = [cut[0] + i, 100 + cut[1] + i]
        got = ra.delta_rule_step(*(x[at] for x in (q, k, v, g, beta)), s)
        err = (got.float() - whole[at].float()).abs()
        assert (err <= 2.0 ** -7 * whole[at].float().abs() + 1e-3 * whole.float().abs().max()).all()
    assert (s - last).norm() <= 4.6e-5 * last.norm()


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_long_chains_stay_exact(ra, dk, dv):
    """2200 tokens that forget nothing: the state keeps its 24 bits through 35 chunks."""
    q, k, v, g, beta, cu, cud = make([2200], 1, 1, dk, dv, "bf16", "none", 8)
    out, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, final_state=True)
    want, wl = ref(q, k, v, g, beta, cu, None, dk ** -0.5)
    R.delta_check(out, want, "out")
    R.delta_check(last, wl, "state")


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, "fp32"), (128, 64, "fp32"), (64, 128, "fp32"), (128, 128, "fp32"),
                                         (64, 64, "bf16"), (128, 64, "bf16"), (64, 128, "bf16")])
@pytest.mark.parametrize("hk,hv", [(1, 2), (4, 16)])
def test_few_and_many_heads(ra, hk, hv, dk, dv, dtype):
    """Few heads: narrow slices of the state, two CTAs a chunk's gradients.  Many: wide slices, one."""
    lens = [70, 3, 64, 130, 0, 1]
    q, k, v, g, beta, cu, cud = make(lens, hk, hv, dk, dv, dtype, "usual", 11, tail=1)
    s0, ds = states(6, hv, dk, dv, 1), states(6, hv, dk, dv, 2)
    want, last = ref(q, k, v, g, beta, cu, s0, 0.3)
    got, s1 = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, final_state=True, scale=0.3)
    R.delta_check(got[:cu[-1]], want, "out")
    R.delta_check(s1, last, "state")
    R.delta_check(ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, scale=0.3)[0][:cu[-1]], want, "out")
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(9)).to(v.dtype).cuda()
    want = ref(q, k, v, g, beta, cu, s0, 0.3, dout, ds)
    got = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=ds, scale=0.3)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        R.delta_check(x[:cu[-1]], y[:cu[-1]], name)
    R.delta_check(got[5], want[5], "dstate0")
    again = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=ds, scale=0.3)
    assert all(torch.equal(x[:cu[-1]] if i < 5 else x, y[:cu[-1]] if i < 5 else y) for i, (x, y) in enumerate(zip(got, again)))
    assert ra.device_status() == 0


@pytest.mark.parametrize("state", [False, True])
def test_every_end_of_a_chunk(ra, state):
    """Last chunks that end inside, at and behind each 16 tokens: nothing of the next sequence's rows is written."""
    lens = [1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 79, 80, 81, 128, 129, 200]
    q, k, v, g, beta, cu, cud = make(lens, 1, 2, 128, 128, "bf16", "usual", 12, tail=1)
    s0 = states(len(lens), 2, 128, 128, 1) if state else None
    want, last = ref(q, k, v, g, beta, cu, s0, 0.3)
    out = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    got, s1 = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, final_state=state, scale=0.3, out=out)
    R.delta_check(got[:cu[-1]], want, "out")
    assert (got[cu[-1]:] == 7.0).all() and ra.device_status() == 0
    if state:
        R.delta_check(s1, last, "state")


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_many_sequences(ra, dk, dv):
    """More sequences than the plan lines up at a time, and than it sorts."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 4, 4500).tolist()
    q, k, v, g, beta, cu, cud = make(lens, 1, 1, dk, dv, "bf16", "usual", 9)
    out, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, final_state=True)
    want, wl = ref(q, k, v, g, beta, cu, None, dk ** -0.5)
    R.delta_check(out, want, "out")
    R.delta_check(last, wl, "state")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_empty_calls(ra, dtype):
    q, k, v, g, beta, cu, cud = make([0, 0], 1, 2, 64, 128, dtype, "usual", 1)
    s0, ds = states(2, 2, 64, 128, 1), states(2, 2, 64, 128, 2)
    out, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, final_state=True)
    assert out.shape == (0, 2, 128) and torch.equal(last, s0)
    got = ra.delta_rule_bwd(out, q, k, v, g, beta, cud, state=s0, dstate=ds)
    assert [x.shape[0] for x in got[:5]] == [0] * 5 and torch.equal(got[5], ds)
    out, last = ra.delta_rule_fwd(q, k, v, g, beta, ints([0]))
    assert out.numel() == 0 and last is None
    none = torch.empty(0, 2, 64, 128, device="cuda")
    assert ra.delta_rule_step(q, k, v, g, beta, none).numel() == 0
    # tokens, and all of them behind the last sequence
    q, k, v, g, beta, cu, _ = make([], 1, 2, 64, 128, dtype, "usual", 1, tail=70)
    keep = torch.full(v.shape, 5.0, dtype=v.dtype, device="cuda")
    ra.delta_rule_fwd(q, k, v, g, beta, ints([0, 0, 0]), out=keep)
    assert (keep == 5.0).all() and ra.device_status() == 0


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_nan_stays_in_its_sequence(ra, dk, dv):
    """A NaN or an infinity reaches its own sequence's tokens of its chunk and behind, and nothing else: not the sequence
    ahead either, whose last chunk ends where it begins."""
    lens = [130, 70, 64]
    for bad, dtype, seq in ((math.nan, "bf16", 0), (math.inf, "fp32", 0), (math.nan, "bf16", 1), (math.inf, "bf16", 1)):
        q, k, v, g, beta, cu, cud = make(lens, 1, 2, dk, dv, dtype, "usual", 2)
        clean, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, final_state=True)
        alone = ra.delta_rule_fwd(q, k, v, g, beta, cud)[0]
        dout = torch.randn_like(v)
        at = cu[seq] + (70 if seq == 0 else 2)
        others = [t for t in range(cu[-1]) if not cu[seq] <= t < cu[seq + 1] or (seq == 0 and t < 64)]
        rest = [t for t in range(cu[-1]) if not cu[seq] <= t < cu[seq + 1]]
        seqs = [b for b in range(3) if b != seq]
        for x in (q, k, v, dout):
            y = x.clone()
            y[at, 0, 3] = bad
            args = [y if z is x else z for z in (q, k, v)]
            if x is not dout:
                out, s = ra.delta_rule_fwd(*args, g, beta, cud, final_state=True)
                assert torch.equal(out[others], clean[others]) and torch.equal(s[seqs], last[seqs])
                assert not torch.isfinite(out[at]).all()
                assert torch.equal(ra.delta_rule_fwd(*args, g, beta, cud)[0][others], alone[others])
            got = ra.delta_rule_bwd(y if x is dout else dout, *args, g, beta, cud)
            want = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud)
            assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got[:5], want[:5]))
    assert ra.device_status() == 0


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_bad_arrays_are_recorded(ra, dk, dv):
    """Boundaries that decrease or leave the tokens: recorded, nothing written.  A slot outside the pool: recorded, the
    sequence begins at zero and its state is dropped."""
    q, k, v, g, beta, cu, cud = make([40, 50], 1, 1, dk, dv, "bf16", "usual", 1)
    for bad in ([0, 60, 50], [0, 40, 91], [-1, 40, 90]):
        out = torch.full_like(v, 2.0)
        s = torch.full((2, 1, dk, dv), 2.0, device="cuda")
        ra.delta_rule_fwd(q, k, v, g, beta, ints(bad), state_out=s, out=out)
        assert ra.device_status() == 6 and (out == 2.0).all() and (s == 2.0).all()
        grads = ra.delta_rule_bwd(v, q, k, v, g, beta, ints(bad))
        assert ra.device_status() == 6 and len(grads) == 6
    pool = states(2, 1, dk, dv, 1)
    keep = pool.clone()
    out, _ = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=pool, slots=ints([1, 2]), state_out=pool)
    assert ra.device_status() == 6 and torch.equal(pool[0], keep[0]) and not torch.equal(pool[1], keep[1])
    zero = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=keep, slots=ints([1, -1]))[0]
    R.delta_check(out, zero.double().cpu(), "dropped")
    out = ra.delta_rule_step(q[:2], k[:2], v[:2], g[:2], beta[:2], pool, slots=ints([5, 0]))
    assert ra.device_status() == 6 and (out[0] == 0).all() and (out[1] != 0).any()


def test_python_refusals(ra):
    q, k, v, g, beta, cu, cud = make([40], 1, 2, 64, 64, "bf16", "usual", 1)
    s = states(1, 2, 64, 64, 1)
    fwd = ra.delta_rule_fwd
    for args, kw in [((q, k[:39], v, g, beta, cud), {}), ((q, k, v[:39], g, beta, cud), {}),
                     ((q, k, v, g[:39], beta, cud), {}), ((q, k, v, g, beta.t().contiguous().t(), cud), {}),
                     ((q, k, v, g, beta, cud), {"state": s[:, :1]}), ((q, k, v, g, beta, cud), {"slots": ints([0])}),
                     ((q, k, v, g, beta, cud), {"state": torch.cat([s, s])}),
                     ((q, k, v, g, beta, cud), {"state": torch.cat([s, s]), "final_state": True}),
                     ((q, k, v, g, beta, cud), {"state": s, "slots": ints([0]), "final_state": True}),
                     ((q, k, v, g, beta, cud), {"state": s, "slots": ints([0, 1])}),
                     ((q, k, v, g, beta, cud.cpu()), {}), ((q.float(), k, v, g, beta, cud), {}),
                     ((q, k, v, g, beta, cud), {"out": v.float()}), ((q.transpose(1, 2), k, v, g, beta, cud), {})]:
        with pytest.raises(ValueError):
            fwd(*args, **kw)
    with pytest.raises(TypeError):
        fwd(q, k, v, g.double(), beta, cud)
    with pytest.raises(TypeError):
        fwd(q, k, v, g, beta, cud.long())
    with pytest.raises(TypeError):
        fwd(q.half(), k.half(), v.half(), g, beta, cud)
    with pytest.raises(ra.RaError):  # heads of other sizes
        fwd(q[..., :32].contiguous(), k[..., :32].contiguous(), v, g, beta, cud)
    with pytest.raises(ra.RaError):  # value heads that no key head divides
        fwd(torch.cat([q] * 3, 1), torch.cat([k] * 3, 1), v, g, beta, cud)
    with pytest.raises(ra.RaError):
        fwd(q, k, v, g, beta, cud, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ra.RaError):
        fwd(q, k, v, g, beta, cud, scale=math.inf)
    with pytest.raises(ValueError):
        ra.delta_rule_bwd(v[:39], q, k, v, g, beta, cud)
    with pytest.raises(ValueError):
        ra.delta_rule_bwd(v, q, k, v, g, beta, cud, dstate=torch.cat([s, s]))
    with pytest.raises(ValueError):
        ra.delta_rule_step(q, k, v, g, beta, s)
    assert ra.device_status() == 0


def test_same_bits_from_any_workspace(ra):
    q, k, v, g, beta, cu, cud = make([150, 20, 300], 2, 4, 128, 128, "bf16", "usual", 4)
    dout = torch.randn_like(v)
    got = []
    for fill in (0, 255):
        ws = [torch.full((ra.delta_rule_workspace_bytes(len(q), 3, 2, 4, 128, 128, 0, b),), fill, dtype=torch.uint8,
                         device="cuda") for b in (False, True)]
        out, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, final_state=True, workspace=ws[0])
        got.append([out, last, *ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, workspace=ws[1])[:5]])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_in_a_graph_and_on_another_stream(ra, dk, dv):
    """Captured calls follow their arrays' contents; a call on a side stream runs there."""
    lens = [70, 64, 10]
    q, k, v, g, beta, cu, cud = make(lens, 1, 2, dk, dv, "bf16", "usual", 6, tail=20)
    dout = torch.randn_like(v)
    pool = states(4, 2, dk, dv, 1)
    slots = ints([2, 0, 3])
    start = pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up, and a call away from the default stream
        ra.delta_rule_fwd(q, k, v, g, beta, cud, state=pool, slots=slots, state_out=pool)
        ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=pool, slots=slots)
        ra.delta_rule_step(q[:3], k[:3], v[:3], g[:3], beta[:3], pool, slots=slots)
    torch.cuda.current_stream().wait_stream(side)
    pool.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=pool, slots=slots, state_out=pool)
        grads = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=pool, slots=slots)
        one = ra.delta_rule_step(q[:3], k[:3], v[:3], g[:3], beta[:3], pool, slots=slots)
    for new, places in ((lens, [2, 0, 3]), ([1, 0, 150], [0, 1, 2]), ([144, 10, 0], [3, 2, 1])):
        c = [0]
        for n in new:
            c.append(c[-1] + n)
        cud.copy_(ints(c))
        slots.copy_(ints(places))
        pool.copy_(start)
        out.zero_()
        graph.replay()
        p = start.clone()
        want, _ = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=p, slots=slots, state_out=p)
        wg = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=p, slots=slots)
        w1 = ra.delta_rule_step(q[:3], k[:3], v[:3], g[:3], beta[:3], p, slots=slots)
        n = c[-1]
        assert torch.equal(out[:n], want[:n]) and torch.equal(pool, p) and torch.equal(one, w1)
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(grads[:5], wg[:5])) and torch.equal(grads[5], wg[5])
    assert ra.device_status() == 0


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_calls_from_several_threads(ra, dk, dv):
    ins = [make([30 + 50 * i, 5], 1, 1 + i % 2, dk, dv, "bf16", "usual", i) for i in range(4)]
    want = [ra.delta_rule_fwd(*x[:5], x[6], final_state=True) for x in ins]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = ra.delta_rule_fwd(*ins[i][:5], ins[i][6], final_state=True)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    assert all(torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) for a, b in zip(got, want))


def test_rows_behind_32_bits_of_elements(ra):
    """Rows 2^31 / 60 elements apart: the last of 70 lies behind 2^31 elements."""
    stride = 2 ** 31 // 60 // 8 * 8
    T = 70
    flat = torch.zeros(T * stride + 64, dtype=torch.bfloat16, device="cuda")
    q, k, v, g, beta, cu, cud = make([T], 1, 1, 64, 64, "bf16", "usual", 1)
    far = []
    for i, x in enumerate((q, k, v)):
        y = torch.as_strided(flat, (T, 1, 64), (stride, 64, 1), i * 128)
        y.copy_(x)
        far.append(y)
    a, b = ra.delta_rule_fwd(*far, g, beta, cud)[0], ra.delta_rule_fwd(q, k, v, g, beta, cud)[0]
    assert torch.equal(a, b)
    d = torch.as_strided(flat, (T, 1, 64), (stride, 64, 1), 512)
    d.copy_(v)
    got, want = ra.delta_rule_bwd(d, *far, g, beta, cud), ra.delta_rule_bwd(v, q, k, v, g, beta, cud)
    assert all(torch.equal(x, y) for x, y in zip(got[:5], want[:5]))


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, "bf16"), (64, 128, "bf16"), (128, 128, "bf16"), (128, 128, "fp32")])
@pytest.mark.parametrize("gates", ["none", "usual"])
def test_outputs_do_not_depend_on_the_last_state(ra, dk, dv, dtype, gates):
    """The same call without the states behind the sequences gives the same bits, also at the end of long chains."""
    q, k, v, g, beta, cu, cud = make([1500, 70, 1], 1, 2, dk, dv, dtype, gates, 8)
    s0 = states(3, 2, dk, dv, 1)
    want = ref(q, k, v, g, beta, cu, s0, dk ** -0.5)[0]
    out, _ = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, final_state=True)
    R.delta_check(out, want, "out")
    assert torch.equal(ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0)[0], out)
    assert ra.device_status() == 0


def ref_by_sequence(q, k, v, g, beta, cu, state, scale, dout, dstate):
    """The gradients in 64 bits, a sequence at a time on the GPU: (dq, dk, dv, dg, dbeta, dstate0) on the CPU."""
    parts = []
    for b in range(len(cu) - 1):
        at = slice(cu[b], cu[b + 1])
        x = [t[at].detach().double() for t in (q, k, v, g, beta)] + [state[b:b + 1].double()]
        for t in x:
            t.requires_grad_()
        out, last = R.delta(*x[:5], [0, cu[b + 1] - cu[b]], x[5], scale)
        total = (out * dout[at].double()).sum() + (last * dstate[b:b + 1].double()).sum()
        parts.append([t.cpu() for t in torch.autograd.grad(total, x)])
    return [torch.cat(p) for p in zip(*parts)]


@pytest.mark.parametrize("hv", [8, 16])
def test_gradients_of_more_chunks_than_sms(ra, hv):
    """bf16 heads of 128: several (chunk, key head) units to each CTA of the gradients, more walks than SMs, sequences of
    up to 11 chunks, value heads that share a key head, ragged ends."""
    rng = np.random.default_rng(hv)
    lens = rng.integers(1, 300, 29).tolist() + [700]
    q, k, v, g, beta, cu, cud = make(lens, 8, hv, 128, 128, "bf16", "usual", 13, tail=5)
    s0, ds = states(30, hv, 128, 128, 1), states(30, hv, 128, 128, 2)
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(9)).to(v.dtype).cuda()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(-(-n // 64) for n in lens) * 8 > 2.5 * sms and 30 * hv > sms
    got = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=ds, scale=0.3)
    want = ref_by_sequence(q, k, v, g, beta, cu, s0, 0.3, dout, ds)
    n = cu[-1]
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        R.delta_check(x[:n], y, name)
    R.delta_check(got[5], want[5], "dstate0")
    for _ in range(3):
        again = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=ds, scale=0.3)
        assert all(torch.equal(a[:n] if i < 5 else a, b[:n] if i < 5 else b) for i, (a, b) in enumerate(zip(again, got)))
    assert ra.device_status() == 0


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, "bf16"), (128, 128, "bf16"), (128, 128, "fp32")])
@pytest.mark.parametrize("gates", ["none", "usual"])
def test_gradients_of_long_chains(ra, dk, dv, dtype, gates):
    """1000 tokens, 16 chunks of a walk; the states' gradients keep their 24 bits as the states do.

    A product of the tensor cores adds up to 24 instructions in one accumulator (three parts of depth 128), and each cuts at
    most 2^-23 of it, 2^-24 on average, always towards 0: 1.5e-6 of a product.  What follows multiplies that by operands of
    random signs, and a gated or contracting state does not let it grow: the errors of a chunk's four products add up as
    squares, 2.9e-6 of the norm."""
    q, k, v, g, beta, cu, cud = make([1000, 65], 1, 2, dk, dv, dtype, gates, 21)
    s0, ds = states(2, 2, dk, dv, 1), states(2, 2, dk, dv, 2)
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(9)).to(v.dtype).cuda()
    scale = dk ** -0.5
    got = ra.delta_rule_bwd(dout, q, k, v, g, beta, cud, state=s0, dstate=ds)
    want = ref_by_sequence(q, k, v, g, beta, cu, s0, scale, dout, ds)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate0"), got, want):
        R.delta_check(x, y, name)
    _, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, state=s0, final_state=True)
    _, wl = R.delta(*(t.double() for t in (q, k, v, g, beta)), cu, s0.double(), scale)
    for name, x, y in (("state", last, wl.cpu()), ("dstate0", got[5], want[5])):
        err = (x.double().cpu() - y).norm() / y.norm()
        assert err <= 2.9e-6, (name, float(err))
    assert ra.device_status() == 0


def test_wide_rows_behind_32_bits_of_elements(ra):
    """The same for heads of 128, whose rows come by tensor maps: the last of 150 tokens lies behind 2^31 elements."""
    stride = 2 ** 31 // 140 // 8 * 8
    T = 150
    flat = torch.zeros(T * stride + 1024, dtype=torch.bfloat16, device="cuda")
    q, k, v, g, beta, cu, cud = make([70, 80], 1, 2, 128, 128, "bf16", "usual", 1)
    at, far = 0, []
    for x in (q, k, v, v.flip(0)):
        y = torch.as_strided(flat, tuple(x.shape), (stride, 128, 1), at)
        y.copy_(x)
        far.append(y)
        at += x.shape[1] * 128
    a, b = ra.delta_rule_fwd(*far[:3], g, beta, cud)[0], ra.delta_rule_fwd(q, k, v, g, beta, cud)[0]
    assert torch.equal(a, b)
    got, want = ra.delta_rule_bwd(far[3], *far[:3], g, beta, cud), ra.delta_rule_bwd(v.flip(0), q, k, v, g, beta, cud)
    assert all(torch.equal(x, y) for x, y in zip(got[:5], want[:5])) and ra.device_status() == 0


@pytest.mark.parametrize("n", [2047, 2048, 2049])
def test_sequences_in_order_of_length_or_not(ra, n):
    """Up to 2048 sequences are walked by their length, more in their own order: the results are the same."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 3, n - 1).tolist() + [200]
    q, k, v, g, beta, cu, cud = make(lens, 1, 1, 64, 64, "bf16", "usual", 9)
    out, last = ra.delta_rule_fwd(q, k, v, g, beta, cud, final_state=True)
    want, wl = ref(q, k, v, g, beta, cu, None, 0.125)
    R.delta_check(out, want, "out")
    R.delta_check(last, wl, "state")
