"""The router's choice (ep_route) and its gradient (ep_route_grad) against
plain 64-bit arithmetic, token by token.

Ids are compared exactly: keys are the logits themselves, or taken in 64 bits
on both sides, where two keys of these inputs are either the same by
construction (same logit, same bias) or further apart than 1e-12. Tolerances of
weights and gradients count roundings of 32 bits (2^-24 of a value each): an
exponential of an argument v is off by (|v| + 16) * 2^-23 (the argument's
scaling to base 2 loses |v| * 2^-24, the rest is a few units in the last
place).
"""
import math

import pytest
import torch

from combine_get_layout_amd import ep
from test_experts_gpu import F32, F64, HALF_BF16, U23, check_there

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
TINY = 1e-20


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.lib()


def scores(row, score):
    """Scores of one token's logits (a list of floats, -inf masked)."""
    if score == ep.EP_SCORE_SIGMOID:
        return [1 / (1 + math.exp(-l)) if l > -700 else 0.0 for l in row]
    top = max(row)
    if top == -INF:
        return [0.0] * len(row)
    p = [1.0 if l == top else 0.0 if l == -INF else math.exp(l - top) for l in row]
    s = math.fsum(p)
    return [v / s for v in p]


def choose(row, K, G, score, top_groups=None, group_top=1, bias=None):
    """Ids and scores of one token, from the definition."""
    E = len(row)
    row = [-INF if math.isnan(l) else l for l in row]
    s = scores(row, score)
    top_groups = G if top_groups is None else top_groups
    if bias is None and (top_groups == G or group_top == 1):
        key = list(row)
    else:
        key = [-INF if l == -INF else v + (0.0 if bias is None else b) for l, v, b in
               zip(row, s, [0.0] * E if bias is None else bias)]
        key = [-INF if math.isnan(k) else k for k in key]
    if top_groups < G:
        size = E // G
        ranks = []
        for g in range(G):
            best = sorted((k for k in key[g * size:(g + 1) * size] if k > -INF), reverse=True)[:group_top]
            ranks.append((-sum(best) if best else INF, g))
        allowed = {g for _, g in sorted(ranks)[:top_groups]}
        key = [k if e // size in allowed else -INF for e, k in enumerate(key)]
    order = sorted(range(E), key=lambda e: (-key[e], e))
    ids = [e for e in order[:K] if key[e] > -INF]
    return ids + [-1] * (K - len(ids)), s


def reference(logits, K, G, router):
    score, norm, scale = router["score"], router.get("normalize", True), router.get("scale", 1.0)
    bias = router.get("bias")
    bias = None if bias is None else bias.tolist()
    ids, ws, ss = [], [], []
    for row in logits.tolist():
        i, s = choose(row, K, G, score, router.get("top_groups"), router.get("group_top", 1), bias)
        lane = [s[e] if e >= 0 else 0.0 for e in i]
        total = math.fsum(lane) + TINY if norm else 1.0
        ids.append(i)
        ws.append([scale * v / total for v in lane])
        ss.append(s)
    return torch.tensor(ids), torch.tensor(ws, dtype=F64), torch.tensor(ss, dtype=F64)


def spread(logits, score):
    """The largest argument of an exponential that does not vanish."""
    l = logits.double()
    l = torch.where(torch.isfinite(l), l, torch.zeros(()))
    if score == ep.EP_SCORE_SIGMOID:
        return l.abs().clamp(max=90).max().item()
    top = torch.where(torch.isfinite(logits), logits.double(), torch.tensor(-1e30, dtype=F64)).amax(1, keepdim=True)
    d = (top - logits.double())
    return d[torch.isfinite(d) & (d < 90)].max().item() if bool((torch.isfinite(d) & (d < 90)).any()) else 0.0


def weight_rel(logits, score, E):
    """An exponential, the sum of them (E / 64 in a lane, 8 more), the quotient, the sum of the chosen
    and its quotient, the scale: relative, each of two sums of positive terms."""
    one = (spread(logits, score) + 16) * U23
    return 2 * one + (E / 64 + 8 + 64 + 12) * U23


def route(logits, K, G, router, want_err=0):
    T, E = logits.shape
    shape = ep.make_shape(T, 8, K, E, G, G)
    ws = ep.alloc_workspace(shape)
    idx = torch.full((T + 2, K), 77, dtype=torch.int64, device="cuda")
    w = torch.full((T + 2, K), 7.0, device="cuda")
    router = dict(router, bias=None if router.get("bias") is None else router["bias"].cuda())
    ep.ep_route(shape, logits.cuda(), router, idx, w, ws)
    assert ep.ep_check_sticky_errors(ws) == want_err
    assert (idx[T:] == 77).all() and (w[T:] == 7).all()
    only = torch.empty((T, K), dtype=torch.int64, device="cuda")
    ep.ep_route(shape, logits.cuda(), router, only, None, ws)
    assert torch.equal(only, idx[:T])
    return idx[:T].cpu(), w[:T].cpu()


def check_route(logits, K, G, router, want_err=0):
    idx, w = route(logits, K, G, router, want_err)
    ids, ws, _ = reference(logits, K, G, router)
    assert torch.equal(idx, ids), (idx != ids).nonzero()[:4]
    check_there(w, ws, weight_rel(logits, router["score"], logits.shape[1]) * ws.abs() + 1e-30, "weights")
    return ids


def logit_case(T, E, seed, masked=0.0, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    l = scale * torch.randn((T, E), generator=g)
    l[torch.rand((T, E), generator=g) < masked] = -INF
    return l


# (T, E, K): one expert, all of them, sizes around 64 lanes and each number of experts a lane.
PLAIN = [(1, 1, 1), (5, 8, 8), (3, 5, 9), (7, 64, 8), (13, 72, 6), (9, 130, 4), (6, 257, 8), (50, 256, 8), (3, 1000, 64),
         (2, 2047, 3), (2, 4096, 64)]
SOFTMAX, SIGMOID = 0, 1


@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("case", PLAIN, ids=str)
def test_route(case, score, bias):
    T, E, K = case
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(5)) if bias else None
    for masked, normalize in ((0.0, True), (0.3, False)):
        check_route(logit_case(T, E, 3, masked), K, 1,
                    dict(score=score, normalize=normalize, scale=2.5, bias=b))


# (T, E, K, G, top_groups): groups in powers of two and others, one to 64, and the largest
# number of experts to a lane (4,092 experts in 33 groups: 124).
GROUPED = [(9, 256, 8, 8, 4), (5, 160, 6, 8, 3), (4, 36, 4, 3, 1), (4, 64, 5, 64, 7), (3, 4096, 8, 64, 3),
           (2, 4092, 64, 33, 5), (3, 90, 4, 9, 8), (5, 40, 8, 5, 2), (6, 16, 2, 16, 16), (8, 8, 8, 2, 1)]


@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("case", GROUPED, ids=str)
def test_route_in_groups(case, score, group_top, bias):
    T, E, K, G, top_groups = case
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(5)) if bias else None
    for masked in (0.0, 0.4):
        check_route(logit_case(T, E, 4, masked), K, G,
                    dict(score=score, top_groups=top_groups, group_top=group_top, scale=1.0, bias=b))


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
def test_route_ties_go_to_the_lowest_id(score, bias):
    """Logits of few distinct values, the same bias everywhere; groups of the same sums."""
    g = torch.Generator().manual_seed(7)
    l = torch.randint(-1, 2, (40, 96), generator=g).float()
    b = torch.full((96,), 0.25) if bias else None
    check_route(l, 8, 1, dict(score=score, bias=b))
    check_route(l, 8, 6, dict(score=score, bias=b, top_groups=2, group_top=1))
    check_route(torch.zeros((3, 96)), 8, 6, dict(score=score, bias=b, top_groups=2, group_top=2))


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
def test_route_masked_and_extreme_rows(score):
    """Rows with nothing left, with fewer experts than lanes, of the type's lowest value, with infinities, of
    large differences, of denormals."""
    E, K, low = 16, 4, torch.finfo(F32).min
    l = logit_case(9, E, 8)
    l[0] = -INF
    l[1] = -INF
    l[1, 5] = 0.5
    l[2] = low
    l[3] = low
    l[3, 9] = 1.0
    l[4, [3, 11]] = INF
    l[5] = torch.linspace(-80, 80, E)
    l[6] = INF
    l[7] = -INF
    l[7, [2, 15]] = torch.tensor([low, INF])
    l[8] = 1e-40
    for norm in (True, False):
        for G, top in ((1, 1), (4, 1), (4, 2)):
            ids = check_route(l, K, G, dict(score=score, normalize=norm, scale=1.5, top_groups=top))
            assert (ids[0] == -1).all() and ids[1].tolist() == [5, -1, -1, -1]


def test_route_biases_that_mask_and_force():
    E, K = 70, 5
    l = logit_case(6, E, 9)
    b = torch.zeros(E)
    b[::3] = -INF
    b[1] = INF
    ids = check_route(l, K, 1, dict(score=SIGMOID, bias=b))
    assert (ids[:, 0] == 1).all() and (ids % 3 != 0).all()


def test_route_reports_nan():
    """A NaN is no choice and is reported; the rest of the row is chosen from as if it were masked."""
    E, K = 24, 3
    l = logit_case(4, E, 10)
    l[2, 7] = NAN
    l[3] = NAN
    for router in (dict(score=SOFTMAX), dict(score=SIGMOID), dict(score=SOFTMAX, bias=torch.zeros(E))):
        ids = check_route(l, K, 1, router, want_err=ep.EP_DEVERR_LOGIT)
        assert (ids[3] == -1).all() and (ids[2] != 7).all()
    b = torch.zeros(E)
    b[4] = NAN
    ids = check_route(logit_case(4, E, 10), K, 1, dict(score=SIGMOID, bias=b), want_err=ep.EP_DEVERR_LOGIT)
    assert (ids != 4).all()


def test_route_many_tokens():
    """Two tokens apart by more than a launch of one workgroup a CU; a sample against the definition."""
    T, E, K, G = 30_001, 64, 4, 4
    l = logit_case(T, E, 11)
    router = dict(score=SIGMOID, top_groups=2, group_top=2, bias=0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)))
    idx, w = route(l, K, G, router)
    at = torch.arange(0, T, 997)
    ids, ws, _ = reference(l[at], K, G, router)
    assert torch.equal(idx[at], ids)
    check_there(w[at], ws, weight_rel(l, SIGMOID, E) * ws.abs(), "weights")
    assert torch.equal(idx[-1], reference(l[-1:], K, G, router)[0][0])


def test_route_of_more_tokens_than_one_launch():
    """2^21 workgroups of four tokens and a few tokens more, and their gradient."""
    T, E, cut = (1 << 23) + 5, 2, 1 << 22
    l = torch.randn((T, E), generator=torch.Generator().manual_seed(3))
    router = dict(score=SOFTMAX, normalize=False)
    idx, w = route(l, 1, 1, router)
    assert torch.equal(idx[:, 0], l.argmax(1))
    d_w = torch.ones((T, 1))
    d = grad(l, idx, d_w, router)
    for part in (slice(0, cut), slice(cut, T)):
        assert torch.equal(route(l[part], 1, 1, router)[1], w[part])
        assert torch.equal(grad(l[part], idx[part], d_w[part], router), d[part])
    check_there(w[-9:], reference(l[-9:], 1, 1, router)[1], weight_rel(l, SOFTMAX, E) * w[-9:], "weights")


# --------------------------------------------------------------------------
# Gradient
# --------------------------------------------------------------------------

def grad_reference(logits, idx, d_w, router):
    """The gradient and a bound on its error, in 64 bits, by the formula."""
    T, E = logits.shape
    score, norm, scale = router["score"], router.get("normalize", True), router.get("scale", 1.0)
    clean = torch.where(torch.isnan(logits), -INF, logits)
    s = torch.tensor([scores(r, score) for r in clean.tolist()], dtype=F64)
    ok = (idx >= 0) & (idx < E)
    at = torch.where(ok, idx, 0)
    lane = torch.where(ok, s.gather(1, at), 0.0)
    g = torch.where(ok, scale * d_w.double(), 0.0)
    mag = g.abs()
    if norm:
        S = lane.sum(1, keepdim=True) + TINY
        dot, dot_mag = (g * lane).sum(1, keepdim=True) / S, (g.abs() * lane).sum(1, keepdim=True) / S
        g, mag = torch.where(ok, (g - dot) / S, 0.0), torch.where(ok, (g.abs() + dot_mag) / S, 0.0)
    ds = torch.zeros((T, E), dtype=F64).scatter_add_(1, at, torch.where(lane > 0, g, 0.0))
    ds_mag = torch.zeros((T, E), dtype=F64).scatter_add_(1, at, torch.where(lane > 0, mag, 0.0))
    noise = 2.0 ** -50 * s * (ds_mag * s).sum(1, keepdim=True)  # of this reference's own mean
    if score == SIGMOID:
        not_s = torch.tensor([scores(r, score) for r in (-clean).tolist()], dtype=F64)
        d, m = ds * s * not_s, ds_mag * s * not_s
    else:
        d = s * (ds - (ds * s).sum(1, keepdim=True))
        # The mean of normalised weights vanishes but for TINY; without it it has these magnitudes.
        m = s * (ds_mag + (0 if norm else (ds_mag * s).sum(1, keepdim=True)))
        if norm:
            m = m + d.abs()
    rel = 3 * (spread(clean, score) + 16) * U23 + (E / 64 + 8 + 2 * 64 + 24) * U23
    return d, rel * m + noise + 1e-30


def grad(logits, idx, d_w, router, G=1, dtype=F32, want_err=0):
    T, E = logits.shape
    K = idx.shape[1]
    shape = ep.make_shape(T, 8, K, E, G, G)
    ws = ep.alloc_workspace(shape)
    d = torch.full((T + 1, E), 7.0, dtype=dtype, device="cuda")
    ep.ep_route_grad(shape, logits.cuda(), router, idx.cuda(), d_w.cuda(), d,
                     ep.EP_GRAD_F32 if dtype == F32 else ep.EP_GRAD_BF16, ws)
    assert ep.ep_check_sticky_errors(ws) == want_err
    assert (d[T:] == 7).all()
    return d[:T].cpu()


def grad_case(T, E, K, seed, masked=0.2):
    g = torch.Generator().manual_seed(seed)
    l = logit_case(T, E, seed, masked)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] if K <= E else torch.arange(K) % E for _ in range(T)])
    ids[torch.rand(ids.shape, generator=g) < 0.1] = -1
    return l, ids, torch.randn((T, K), generator=g)


@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "scores"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("case", [(1, 1, 1), (5, 8, 8), (4, 5, 9), (13, 72, 6), (33, 256, 8), (3, 1003, 64), (2, 4096, 8),
                                  (11, 63, 2), (6, 68, 3)], ids=str)
def test_route_grad(case, score, normalize):
    T, E, K = case
    l, ids, d_w = grad_case(T, E, K, 6)
    router = dict(score=score, normalize=normalize, scale=2.5)
    ref, bound = grad_reference(l, ids, d_w, router)
    check_there(grad(l, ids, d_w, router), ref, bound, "d_logits")
    check_there(grad(l, ids, d_w, router, dtype=torch.bfloat16), ref, bound + HALF_BF16 * (ref.abs() + bound), "bf16")


@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "scores"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
def test_route_grad_against_differences(score, normalize):
    """Central differences, in 64 bits, of sum d_w * weights with the choice held. Steps of 1e-5 leave
    1e-10 of third derivatives (at most about 20 |d_w|) and 1e-16 / 1e-5 of rounding: under 1e-8."""
    T, E, K = 3, 12, 4
    l, ids, d_w = grad_case(T, E, K, 21, masked=0.0)
    router = dict(score=score, normalize=normalize, scale=2.5)

    def loss(x):
        s = torch.sigmoid(x) if score == SIGMOID else torch.softmax(x, 1)
        lane = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), 0.0)
        w = lane / (lane.sum(1, keepdim=True) + TINY) if normalize else lane
        return (2.5 * w * d_w.double()).sum(1)

    num, step = torch.zeros((T, E), dtype=F64), 1e-5
    for e in range(E):
        a, b = l.double(), l.double()
        a[:, e] += step
        b[:, e] -= step
        num[:, e] = (loss(a) - loss(b)) / (2 * step)
    _, bound = grad_reference(l, ids, d_w, router)
    check_there(grad(l, ids, d_w, router), num, bound + 1e-7 * 2.5 * (1 + d_w.abs().max().item()), "against differences")


def test_route_grad_of_repeated_bad_and_masked_ids():
    """An id twice adds up; bad ids are reported and skipped, also those that 32 bits would take for
    valid ones; a masked expert in a lane has no part."""
    l, _, _ = grad_case(4, 20, 4, 30, masked=0.0)
    l[3, 6] = -INF
    ids = torch.tensor([[3, 3, 5, 3], [1, 99, -5, 2], [(1 << 32) + 1, -1, 4, 7], [6, 6, 2, 8]])
    d_w = torch.tensor([[0.5, -1.0, 2.0, 0.25]] * 4)
    for score in (SOFTMAX, SIGMOID):
        for norm in (True, False):
            router = dict(score=score, normalize=norm)
            ref, bound = grad_reference(l, ids, d_w, router)
            got = grad(l, ids, d_w, router, want_err=ep.EP_DEVERR_EXPERT_ID)
            check_there(got, ref, bound, "d_logits")
            assert got[3, 6] == 0


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
def test_route_grad_of_extreme_rows(score):
    """Rows without an expert, with infinities and the type's lowest value: zeros or the limit, no NaN."""
    E, low = 10, torch.finfo(F32).min
    l = logit_case(6, E, 31)
    l[0] = -INF
    l[1, 4] = INF
    l[2] = low
    l[3] = torch.linspace(-80, 80, E)
    l[4] = NAN
    l[5, 2:] = -INF
    ids = torch.tensor([[-1, -1], [4, 0], [0, 1], [9, 8], [-1, -1], [0, 1]])
    d_w = torch.ones((6, 2)) * torch.tensor([1.0, -0.5])
    for norm in (True, False):
        router = dict(score=score, normalize=norm)
        ref, bound = grad_reference(l, ids, d_w, router)
        check_there(grad(l, ids, d_w, router), ref, bound, "d_logits")


def test_route_without_tokens():
    shape = ep.make_shape(0, 8, 2, 16, 1)
    ws = ep.alloc_workspace(shape)
    ep.ep_route(shape, None, dict(score=SOFTMAX), None, None, ws)
    ep.ep_route_grad(shape, None, dict(score=SOFTMAX), None, None, None, ep.EP_GRAD_F32, ws)
    assert ep.ep_check_sticky_errors(ws) == 0


def test_route_in_a_graph_and_on_two_streams():
    """Captured once, replayed with new logits; two streams share one workspace (for its error words)."""
    T, E, K, G = 500, 160, 6, 8
    shape = ep.make_shape(T, 8, K, E, G, G)
    ws = ep.alloc_workspace(shape)
    ep.ep_clear_errors(ws)
    ls = [logit_case(T, E, s, 0.2).cuda() for s in (40, 41, 42)]
    d_w = torch.randn((T, K), device="cuda")
    router = dict(score=SIGMOID, top_groups=3, group_top=2, bias=0.1 * torch.randn(E, device="cuda"))

    def step(l, b):
        if not b:
            b += [torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda"),
                  torch.empty((T, E), device="cuda")]
        ep.ep_route(shape, l, router, b[0], b[1], ws)
        ep.ep_route_grad(shape, l, router, b[0], d_w, b[2], ep.EP_GRAD_F32, ws)
        return b

    ref = [[t.clone() for t in step(l, [])] for l in ls]
    static, b = ls[0].clone(), []
    step(static, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, b)
    for i in (0, 1, 2, 0, 2):
        static.copy_(ls[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(b, ref[i])), i
        step(ls[1], [])
        torch.randn(1000, device="cuda").sum().item()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for n in range(8):
        with torch.cuda.stream(streams[n % 2]):
            got.append((n % 3, step(ls[n % 3], [])))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, ref[i]))
    assert ep.ep_check_sticky_errors(ws) == 0
