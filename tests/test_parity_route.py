"""w4_route and w4_combine against 64-bit numpy implementations.

ids, offsets, order and pos are whole numbers and have to be equal.  A weight
is one fp32 rounding (2^-24) of an fp64 value whose own error is below
1100 * 2^-53; 2^-23 covers both.  w4_combine sums k + 1 terms in fp32 and rounds
once: |out - ref| <= 2^-8 (|ref| + e) + e with e = (k + 2) 2^-24 * sum of the
terms' magnitudes.
"""
import numpy as np
import pytest

from bit_gemm_quant_b200 import synth
from parity import dev_bf16, dev_f32, host_bf16_as_f64


@pytest.fixture(scope="module")
def w4():
    from bit_gemm_quant_b200 import build
    build.build()
    import bit_gemm_quant_b200 as w4
    w4.lib()
    return w4


def choose(x, k, sigmoid=False, bias=None, groups=1, keep=1, group_top=1, renorm=True, scale=1.0):
    """The definition, one token after the other; x fp64 [T, E]."""
    T, E = x.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        live = ~np.isneginf(x[t])
        score = np.zeros(E)
        if sigmoid:
            with np.errstate(over="ignore"):
                score[live] = 1 / (1 + np.exp(-x[t][live]))
        elif live.any():
            score[live] = np.exp(x[t][live] - x[t][live].max())
            score /= score.sum()
        choice = score + (0.0 if bias is None else bias.astype(np.float64))
        ok = live.copy()
        if groups > 1:
            per = E // groups
            value = []
            for g in range(groups):
                m = sorted((choice[e] for e in range(g * per, (g + 1) * per) if live[e]), reverse=True)[:group_top]
                value.append(sum(m) if m else -np.inf)
            best = sorted(range(groups), key=lambda g: (-value[g], g))[:keep]
            for g in range(groups):
                if g not in best:
                    ok[g * per:(g + 1) * per] = False
        top = sorted(np.flatnonzero(ok), key=lambda e: (-choice[e], e))[:k]
        ids[t, :len(top)] = top
        weights[t, :len(top)] = score[top]
        total = weights[t].sum()
        if renorm:
            weights[t] = weights[t] / total if total > 0 else 0.0
        weights[t] *= scale
    return ids, weights


def plan(ids, E):
    flat = ids.reshape(-1)
    offsets, order, pos = np.zeros(E + 1, np.int32), [], np.full(flat.size, -1, np.int32)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        pos[mine] = len(order) + np.arange(mine.size)
        order += list(mine)
        offsets[e + 1] = len(order)
    return offsets, np.array(order + [-1] * (flat.size - len(order)), np.int32), pos.reshape(ids.shape)


def check(w4, x, k, f32=True, sigmoid=False, bias=None, groups=1, keep=1, group_top=1, renorm=True, scale=1.0):
    x = np.asarray(x, np.float32)
    if f32:
        d = dev_f32(x)
    else:
        bits = synth.to_bf16_bits(x)
        d, x = dev_bf16(bits), synth.bf16_bits_to_f32(bits)
    r = w4.route(d, k, scoring=w4.SIGMOID if sigmoid else w4.SOFTMAX, bias=None if bias is None else dev_f32(bias),
                 n_groups=groups, topk_groups=keep, group_top=group_top, renormalize=renorm, scale=scale)
    ids, weights = choose(x.astype(np.float64), k, sigmoid, bias, groups, keep, group_top, renorm, scale)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = r.weights.cpu().numpy().astype(np.float64)
    assert (np.abs(got - weights) <= 2.0 ** -23 * np.abs(weights) + 1e-44).all()
    for a, b, what in zip((r.offsets, r.order, r.pos), plan(ids, x.shape[1]), ("offsets", "order", "pos")):
        assert np.array_equal(a.cpu().numpy(), b), what
    return r


def logits(T, E, seed=0):
    return 2.0 * np.random.default_rng([T, E, seed]).standard_normal((T, E))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 5, 5), (3, 8, 2), (1, 31, 4), (7, 32, 32), (9, 33, 3), (64, 60, 6),
                                   (1, 256, 8), (33, 257, 8), (5, 512, 10), (3, 513, 4), (2, 1024, 32), (700, 16, 4),
                                   (129, 128, 1), (40, 96, 8), (31, 128, 8), (32, 128, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_choice_and_plan(w4, T, E, k, sigmoid):
    check(w4, logits(T, E), k, sigmoid=sigmoid)
    check(w4, logits(T, E, 1), k, f32=False, sigmoid=sigmoid, renorm=False, scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,groups,keep,group_top", [(1, 256, 8, 8, 4, 2), (50, 64, 4, 8, 3, 1), (9, 64, 4, 64, 5, 2),
                                                         (20, 12, 3, 4, 1, 2), (17, 384, 6, 4, 4, 1), (5, 1024, 8, 32, 9, 2),
                                                         (6, 120, 5, 40, 33, 1), (3, 960, 3, 64, 2, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_and_bias(w4, T, E, k, groups, keep, group_top, sigmoid):
    bias = 0.3 * np.random.default_rng(E).standard_normal(E).astype(np.float32)
    for b in (None, bias, bias - 2.0):                 # the last makes every choice negative
        check(w4, logits(T, E, 2), k, sigmoid=sigmoid, bias=b, groups=groups, keep=keep, group_top=group_top)


@pytest.mark.gpu
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_ties_go_to_the_lowest_index(w4, sigmoid, groups, keep):
    """Few different logits, so that most choices and many groups are equal."""
    x = np.random.default_rng(5).integers(0, 3, (60, 64)).astype(np.float32)
    x[0] = 0.0
    x[1, ::2] = -0.0
    x[1, 1::2] = 0.0
    check(w4, x, 7, sigmoid=sigmoid, groups=groups, keep=keep, group_top=2)
    check(w4, x, 7, f32=False, sigmoid=sigmoid, groups=groups, keep=keep, bias=np.full(64, -1.0, np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_masked_experts_and_tokens(w4, sigmoid, groups, keep):
    """-inf logits: single ones, all but a few, whole rows; a row of the type's
    lowest value is not masked."""
    x = logits(40, 64, 3).astype(np.float32)
    rng = np.random.default_rng(8)
    x[rng.random(x.shape) < 0.4] = -np.inf
    x[3] = x[17] = x[39] = -np.inf
    x[5, :] = -np.inf
    x[5, 63] = 1.0
    x[6, 1:] = -np.inf
    x[7] = np.finfo(np.float32).min
    bias = 0.5 * rng.standard_normal(64).astype(np.float32) - 1.0
    for b in (None, bias):
        r = check(w4, x, 6, sigmoid=sigmoid, bias=b, groups=groups, keep=keep, group_top=2)
        assert (r.ids[3] == -1).all() and (r.weights[3] == 0).all() and (r.pos[3] == -1).all()
    check(w4, np.full((3, 16), -np.inf), 4, sigmoid=sigmoid)


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_not_a_number_keeps_the_plan_valid(w4, sigmoid, groups):
    """NaN and +inf spoil their own token's weights; ids stay distinct and in
    range, and the other tokens are untouched."""
    x = logits(12, 32, 4).astype(np.float32)
    clean = dev_f32(x.copy())
    x[2, 5] = np.nan
    x[4] = np.nan
    x[6, 7] = np.inf
    kw = dict(scoring=w4.SIGMOID if sigmoid else w4.SOFTMAX, n_groups=groups, topk_groups=max(1, groups // 2))
    a, b = w4.route(dev_f32(x), 5, **kw), w4.route(clean, 5, **kw)
    ids = a.ids.cpu().numpy()
    assert ((ids >= -1) & (ids < 32)).all()
    for row in ids:
        row = row[row >= 0]
        assert len(set(row)) == len(row)
    keep = [t for t in range(12) if t not in (2, 4, 6)]
    assert np.array_equal(ids[keep], b.ids.cpu().numpy()[keep])
    assert np.array_equal(a.weights.cpu().numpy()[keep], b.weights.cpu().numpy()[keep])
    for got, want in zip((a.offsets, a.order, a.pos), plan(ids, 32)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.gpu
def test_near_scores_are_told_apart(w4):
    """Logits one fp32 step apart: their fp32 softmax scores are equal."""
    x = np.full((1, 64), 1.0, np.float32)
    x[0, 40] = np.nextafter(np.float32(1), np.float32(2))
    x[0, 50] = np.nextafter(x[0, 40], np.float32(2))
    r = check(w4, x, 3)
    assert r.ids[0].tolist() == [50, 40, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(5000, 24, 3), (2049, 128, 8), (8192, 256, 8), (1025, 4, 1), (2731, 40, 12),
                                   (4096, 64, 8), (4097, 64, 8), (6000, 1024, 16), (40000, 1, 1), (16500, 3, 2)])
def test_long_plans(w4, T, E, k):
    check_ids = np.argsort(-logits(T, E, 6).astype(np.float32), axis=1, kind="stable")[:, :k].astype(np.int32)
    r = w4.route(dev_f32(logits(T, E, 6)), k)
    assert np.array_equal(r.ids.cpu().numpy(), check_ids)
    for a, b in zip((r.offsets, r.order, r.pos), plan(check_ids, E)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(300, 16, 2), (9000, 40, 4)])
def test_long_plans_with_masked_tokens(w4, T, E, k):
    """Pairs without an expert, in front, in the middle and at the end."""
    x = logits(T, E, 9).astype(np.float32)
    dead = np.random.default_rng(1).random(T) < 0.3
    dead[:5] = dead[-7:] = True
    x[dead] = -np.inf
    r = w4.route(dev_f32(x), k)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    ids[dead] = -1
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    for a, b in zip((r.offsets, r.order, r.pos), plan(ids, E)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.gpu
def test_choice_without_a_plan(w4):
    import torch
    x = dev_f32(logits(9, 32))
    r = w4.route(x, 4)
    ids = torch.empty_like(r.ids)
    weights = torch.empty_like(r.weights)
    st = w4.w4_route(x.data_ptr(), 1, None, 9, 32, 4, w4.SOFTMAX, 1, 1, 1, 1, 1.0, ids.data_ptr(), weights.data_ptr(),
                     None, None, None, torch.cuda.current_stream().cuda_stream)
    assert st == w4.W4_OK and torch.equal(ids, r.ids) and torch.equal(weights, r.weights)


# Dynamic sizes just under 48 KB, where the kernels' static shared memory takes them over the limit without an
# opt-in: route_fused_kernel has 1024 static bytes and T (E + 64) 8 dynamic ones with groups, plan_many_kernel 128
# and 34 E 4.  In a process of its own: an earlier call with more memory would have opted the kernel in.
BETWEEN = [dict(T=16, E=313 + 7, k=8, groups=8, keep=4), dict(T=15, E=344, k=8, groups=8, keep=4),
           dict(T=14, E=368, k=8, groups=8, keep=4), dict(T=8, E=704, k=8, groups=8, keep=4),
           dict(T=16, E=320, k=8, groups=8, keep=4, group_top=2, sigmoid=True),
           dict(T=8, E=704, k=8, groups=8, keep=4, group_top=2, sigmoid=True),
           dict(T=1030, E=361, k=32)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", BETWEEN, ids=lambda c: "T%d_E%d%s" % (c["T"], c["E"], "_fp64" if "sigmoid" in c else ""))
def test_shared_memory_around_48_kb(case):
    import json
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import json, sys; sys.path[:0] = [%r, %r]\n"
            "import bit_gemm_quant_b200 as w4, test_parity_route as t\n"
            "c = json.loads(sys.argv[1]); T, E, k = (c.pop(n) for n in ('T', 'E', 'k'))\n"
            "t.check(w4, t.logits(T, E, 12), k, **c)\n" % (here, os.path.dirname(here)))
    r = subprocess.run([sys.executable, "-c", code, json.dumps(case)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def pairs_of_choices(sigmoid, count, seed):
    """(logits, scores' leading parts, what is left) of `count` fp32 logits whose exact score lies within 2^-30
    of an fp32 value, so that the rest of it, score - fp32(score), is an fp32 value to 2^-54 of the score."""
    # (a sigmoid above 16 is 1 to fp32)
    x = np.random.default_rng(seed).uniform(-40, 16 if sigmoid else 0, 1 << 20).astype(np.float32)
    e = np.exp(-np.abs(x.astype(np.longdouble)))         # 64 bits of mantissa
    s = np.where(x < 0, e / (1 + e), 1 / (1 + e))         # softmax of (x, 0) is the sigmoid of x
    lead = s.astype(np.float32)
    rest = s - lead
    near = np.flatnonzero(np.abs(rest) <= 2.0 ** -30 * s)[:count]
    assert near.size == count and np.finfo(np.longdouble).nmant >= 63
    return x[near], s[near], lead[near], rest[near]


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_the_last_bits_of_the_scores(w4, sigmoid):
    """Scores to their last bits, as the choice with a bias sees them.

    Of each token two experts compete: one with the logit x and the bias -fp32(score), whose choice is what is
    left of its score (the subtraction of near values is exact), and one with a score of 0 (logit -2000) and a
    bias just below or above the exact rest.  Which is chosen tells the score to the distance between the two.

    Distance, in u = 2^-53 of the score.  exp of v <= 0: its reduced argument is off by at most 0.7 u, the two
    last steps of the polynomial by u (1 + 0.6), those before and the truncation by 0.3: 2.6.  Sigmoid: 1 + e
    1 + 2.6 / 2, its reciprocal 1.1, and for x < 0 the exponential (whose own error then counts once in all) and
    the product 1: below 6.  Softmax of x and 0: 2.6, the sum 1 + 1.3, its reciprocal 1, the product 1: below 7."""
    u = 2.0 ** -53
    tol = (6 if sigmoid else 7) * u
    T = 511
    x, s, lead, rest = pairs_of_choices(sigmoid, T, 3)
    E = 2 * T + 1
    logits = np.full((T, E), -np.inf, np.float32)
    t = np.arange(T)
    logits[t, 2 * t], logits[t, 2 * t + 1] = x, -2000.0
    logits[:, E - 1] = 0.0                               # the softmax's other term, never chosen
    for side in (-1, 1):
        edge = rest + side * tol * s
        other = edge.astype(np.float32)
        wrong = (other - edge) * side < 0                # rounded towards the rest: one step outwards
        other[wrong] = np.nextafter(other[wrong], np.float32(side * np.inf))
        # the fp32 steps leave the edge close: no more than another 2^-53 away
        assert (np.abs(other - edge) <= u * s).all()
        bias = np.empty(E, np.float32)
        bias[0:-1:2], bias[1:-1:2], bias[-1] = -lead, other, -4.0
        got = w4.route(dev_f32(logits), 1, scoring=w4.SIGMOID if sigmoid else w4.SOFTMAX, bias=dev_f32(bias))
        assert np.array_equal(got.ids.cpu().numpy()[:, 0], 2 * t + (side > 0)), "side %d" % side


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_near_scores_are_told_apart_with_a_bias(w4, sigmoid):
    """Logits one fp32 step apart on the path that orders by fp64 scores."""
    x = np.full((2, 64), 1.0, np.float32)
    x[:, 40] = np.nextafter(np.float32(1), np.float32(2))
    x[:, 50] = np.nextafter(x[:, 40], np.float32(2))
    r = check(w4, x, 3, sigmoid=sigmoid, bias=np.full(64, 0.25, np.float32))
    assert r.ids[0].tolist() == [50, 40, 0]
    r = check(w4, x, 3, sigmoid=sigmoid, groups=8, keep=3, group_top=2)
    assert r.ids[1].tolist() == [50, 40, 0]


# -------------------------------------------------------------- combine --

@pytest.mark.gpu
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (5, 32, 264), (40, 3, 1001), (300, 6, 512),
                                   (2000, 4, 136)])
@pytest.mark.parametrize("add", [False, True])
def test_combine(w4, T, k, N, add):
    rng = np.random.default_rng([T, k, N])
    P = T * k
    Y = synth.activations(T + k, P, N, 0.02, 30.0)
    pos = rng.permutation(P).astype(np.int32).reshape(T, k)
    pos[rng.random(pos.shape) < 0.2] = -1
    pos[T // 2] = -1                                   # a token without any expert
    if P > 3:
        pos[0, 0] = P                                   # out of range: adds nothing either
    w = rng.random((T, k)).astype(np.float32)
    A = synth.activations(9, T, N, 0.0, 1.0) if add else None
    got = combine_dev(w4, Y, pos, w, A)
    y = synth.bf16_bits_to_f32(Y).astype(np.float64)
    terms = np.where(((pos >= 0) & (pos < P))[..., None], y[np.clip(pos, 0, P - 1)], 0.0) * w[..., None]
    ref, mag = terms.sum(1), np.abs(terms).sum(1)
    if add:
        a = synth.bf16_bits_to_f32(A).astype(np.float64)
        ref, mag = ref + a, mag + np.abs(a)
    e = (k + 2) * 2.0 ** -24 * mag
    assert (np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + e) + e).all()


def combine_dev(w4, Y, pos, w, A):
    import torch
    out = w4.combine(dev_bf16(Y), torch.from_numpy(pos).cuda(), dev_f32(w), add=None if A is None else dev_bf16(A))
    return host_bf16_as_f64(out)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [136, 77])
def test_combine_in_place_and_unwritten_rows(w4, N):
    """out over add; NaN in rows of Y that no pair names stays out of the sums."""
    import torch
    Y = torch.randn(8, N, device="cuda").bfloat16()
    Y[6:] = float("nan")
    pos = torch.tensor([[0, 5], [-1, 2], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.rand(3, 2, device="cuda")
    A = torch.randn(3, N, device="cuda").bfloat16()
    want = w4.combine(Y, pos, w, add=A)
    assert torch.isfinite(want).all() and torch.equal(want[2], A[2])
    got = w4.combine(Y, pos, w, add=A, out=A)
    assert got.data_ptr() == A.data_ptr() and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8192, 8191])
def test_combine_past_32_bits(w4, N):
    import torch
    P, k = 2 ** 31 // N + 40, 2
    Y = torch.zeros(P, N, dtype=torch.bfloat16, device="cuda")
    Y[-1] = 1.0
    Y[0] = 2.0
    pos = torch.full((P, k), -1, dtype=torch.int32, device="cuda")
    pos[-1, 0], pos[-1, 1], pos[0, 1] = P - 1, 0, P - 1
    w = torch.full((P, k), 0.5, device="cuda")
    out = w4.combine(Y, pos, w)
    assert (out[-1] == 1.5).all() and (out[0] == 0.5).all() and (out[1:-1] == 0).all()


# ------------------------------------------------------------- refusals --

FAKE = 1 << 20


def call_route(w4, logits=FAKE, kind=1, bias=None, T=4, E=64, k=4, scoring=0, groups=1, keep=1, group_top=1, scale=1.0,
               ids=FAKE, weights=FAKE, offsets=FAKE, order=FAKE, pos=FAKE):
    return w4.w4_route(logits, kind, bias, T, E, k, scoring, groups, keep, group_top, 1, scale, ids, weights, offsets,
                       order, pos, None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(ids=None), dict(weights=None), dict(offsets=None), dict(order=None), dict(pos=None),
    dict(kind=2), dict(scoring=2), dict(T=0), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(E=3, k=4),
    dict(groups=0), dict(groups=5), dict(groups=128, E=256), dict(keep=0), dict(groups=4, keep=5), dict(group_top=0),
    dict(group_top=3), dict(groups=32, keep=1, k=3), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(logits=FAKE + 2), dict(kind=0, logits=FAKE + 1), dict(bias=FAKE + 2), dict(ids=FAKE + 2)])
def test_route_refusals(w4, bad):
    assert call_route(w4, **bad) == w4.W4_ERR_INVALID_ARG


@pytest.mark.parametrize("big", [dict(T=1 << 25), dict(T=(1 << 26) + 1, E=16, k=16),
                                 dict(T=1 << 40, E=1, k=1, offsets=None, order=None, pos=None)])
def test_route_unsupported(w4, big):
    assert call_route(w4, **big) == w4.W4_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(Y=None), dict(pos=None), dict(w=None), dict(out=None), dict(P=0), dict(T=0),
                                 dict(N=0), dict(k=0), dict(k=33), dict(Y=FAKE + 1), dict(pos=FAKE + 2), dict(w=FAKE + 1),
                                 dict(add=FAKE + 1), dict(out=FAKE + 1), dict(T=1 << 61)])
def test_combine_refusals(w4, bad):
    a = dict(Y=FAKE, P=8, pos=FAKE, w=FAKE, T=4, k=2, N=64, add=None, out=FAKE)
    a.update(bad)
    assert w4.w4_combine(a["Y"], a["P"], a["pos"], a["w"], a["T"], a["k"], a["N"], a["add"], a["out"],
                         None) == w4.W4_ERR_INVALID_ARG


def test_helper_refusals(w4):
    import torch
    x = torch.zeros(4, 8)
    for bad in (x, x.half(), x[0], x.t()):
        with pytest.raises(ValueError):
            w4.route(bad, 2)
    y, pos, w = torch.zeros(8, 4, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args in ((y, pos, w), (y.float(), pos, w), (y, pos.long(), w), (y, pos, w[:2])):
        with pytest.raises(ValueError):
            w4.combine(*args)
