"""The expert products (ep_expert_matmul, ep_expert_swiglu, ep_swiglu_grad,
ep_expert_wgrad) and the few-token layer (ep_moe_few) against plain 64-bit
arithmetic on the CPU.

Tolerances are bounds by arithmetic, computed per element beside each
reference:
  - a sum of n products held in 32 bits is off by at most n * 2^-23 * sum|a b|
    (one unit in the last place a step, which covers either rounding of the
    matrix instruction's adder);
  - one rounding to bf16 is off by at most 2^-8 of the value, to e4m3 by 2^-4
    of it, or by half its smallest step, 2^-10, near zero;
  - 1 / (1 + exp(-g)) in 32 bits is off by (|g| + 16) * 2^-23 of its value
    (the argument's scaling to base 2 loses |g| * 2^-24, the rest is a few
    units in the last place).
"""
import numpy as np
import pytest
import torch

from combine_get_layout_amd import ep

pytestmark = pytest.mark.gpu

BF16, F32, F64, U8, F8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.float8_e4m3fn
U23, HALF_BF16, HALF_E4M3 = 2.0 ** -23, 2.0 ** -8, 2.0 ** -4


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.lib()


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, dtype=F32) * scale).to(BF16)


def routing(T, K, E, seed, skip=0.0, skew=0.0, repeat=False):
    """Expert ids [T, K] (distinct unless `repeat`), and weights."""
    r = np.random.default_rng(seed)
    if repeat:
        idx = r.integers(0, E, size=(T, K))
    else:
        keys = r.gumbel(size=(T, E)) - skew * np.log(np.arange(1, E + 1))
        idx = np.argsort(-keys, axis=1)[:, :K]
    idx = np.where(r.random((T, K)) < skip, -1, idx).astype(np.int64)
    w = r.random((T, K)).astype(np.float32) - 0.3  # weights of either sign
    return torch.from_numpy(idx), torch.from_numpy(w)


def grouped(idx, E):
    """Expand rows of idx in plain Python: offsets, slot, expert of each row."""
    T, K = idx.shape
    rows = sorted((int(idx[t, k]), t, k) for t in range(T) for k in range(K) if idx[t, k] >= 0)
    slot = torch.full((T, K), -1, dtype=torch.int32)
    for i, (_, t, k) in enumerate(rows):
        slot[t, k] = i
    experts = torch.tensor([e for e, _, _ in rows], dtype=torch.int64)
    counts = torch.bincount(experts, minlength=E) if rows else torch.zeros(E, dtype=torch.int64)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = counts.cumsum(0)
    return off, slot, experts


def per_expert(off, f, like):
    """Rows [off[e], off[e+1]) of f(e, slice), one after the other."""
    parts = [f(e, slice(int(off[e]), int(off[e + 1]))) for e in range(len(off) - 1)]
    return torch.cat(parts) if parts else like


def check(got, ref, bound, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    over = (got - ref).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert worst <= 0, f"{what}: {worst:.3g} over its bound at {np.unravel_index(int(over.argmax()), over.shape)}"


def gpu(*ts):
    return [t.cuda() for t in ts]


# (tokens, K, E, k_dim, n_dim, options): one row, no row, sizes that fill no
# tile, tails of every kind of a 256-row tile, skewed and empty experts.
PRODUCTS = [
    (1, 1, 1, 8, 8, {}),
    (1, 2, 4, 64, 256, {}),
    (5, 3, 7, 72, 264, dict(skip=0.3)),
    (64, 2, 1 + 1, 136, 520, {}),
    (129, 2, 3, 200, 96, {}),
    (300, 2, 2, 320, 512, {}),
    (700, 4, 5, 128, 248, dict(skew=1.5)),
    (40, 4, 600, 64, 128, {}),      # more experts than threads in a workgroup
    (257, 1, 1, 1032, 24, {}),
    (33, 64, 64, 48, 40, dict(repeat=True)),
]


def product_case(case, seed):
    T, K, E, k, n, opt = case
    g = torch.Generator().manual_seed(seed)
    idx, w = routing(T, K, E, seed, **opt)
    off, slot, experts = grouped(idx, E)
    N = len(experts)
    shape = ep.make_shape(T, 128, K, E, 1)
    return g, idx, w, off, slot, N, shape, ep.alloc_workspace(shape)


@pytest.mark.parametrize("back", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("case", PRODUCTS, ids=str)
def test_matmul(case, back):
    g, idx, w, off, slot, N, shape, ws = product_case(case, 11)
    E, k, n = case[2], case[3], case[4]
    spare = 3  # rows behind the last expert's stay as they were
    x = randn(g, N + spare, k)
    wt = randn(g, *((E, k, n) if back else (E, n, k)), scale=k ** -0.5)
    y = torch.full((N + spare, n), 7.0, dtype=BF16, device="cuda")
    xd, wd, od = gpu(x, wt, off)
    ep.ep_expert_matmul(shape, dict(expert_offsets=od), xd, N + spare, k, wd, n,
                        ep.EP_WEIGHT_KN if back else ep.EP_WEIGHT_NK, y, ws)
    assert ep.ep_check_errors(ws) == 0
    m = wt.double() if back else wt.double().transpose(1, 2)
    ref = per_expert(off, lambda e, s: x[s].double() @ m[e], None)
    mag = per_expert(off, lambda e, s: x[s].double().abs() @ m[e].abs(), None)
    acc = k * U23 * mag
    check(y[:N], ref, acc + HALF_BF16 * (ref.abs() + acc), "y")
    assert (y[N:] == 7.0).all()


def silu_parts(gu, F):
    gate, up = gu[:, :F], gu[:, F:]
    s = torch.sigmoid(gate)
    return gate, up, s, gate * s * up


def act_bound(gate, up, s, act, dg, du):
    """How far silu(g) u in 32 bits is off for g, u off by dg, du (|silu'| <= 1.1)."""
    return 1.1 * dg * (up.abs() + du) + (gate * s).abs() * du + (gate.abs() + 20) * U23 * act.abs()


# Rows of an expert on both sides of every tile height (64, 128, 160, 192, 224,
# 256 rows), of two and three tiles, and none.
HEIGHTS = [0, 1, 33, 64, 65, 128, 0, 129, 160, 161, 192, 193, 224, 225, 256, 257, 300, 515, 0]


def by_counts(counts, H=128):
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    N, E = int(off[-1]), len(counts)
    shape = ep.make_shape(max(N, 1), H, 1, E, 1)
    return off, N, shape, ep.alloc_workspace(shape)


@pytest.mark.parametrize("k", [8, 96, 136, 200])  # one to four steps of the contracted axis, odd and even
@pytest.mark.parametrize("back", [False, True], ids=["nk", "kn"])
def test_matmul_tile_heights(back, k):
    off, N, shape, ws = by_counts(HEIGHTS)
    E, n = len(HEIGHTS), 264
    g = torch.Generator().manual_seed(k)
    x, wt = randn(g, N, k), randn(g, *((E, k, n) if back else (E, n, k)), scale=k ** -0.5)
    y = torch.full((N, n), 7.0, dtype=BF16, device="cuda")
    xd, wd, od = gpu(x, wt, off)
    ep.ep_expert_matmul(shape, dict(expert_offsets=od), xd, N, k, wd, n,
                        ep.EP_WEIGHT_KN if back else ep.EP_WEIGHT_NK, y, ws)
    m = wt.double() if back else wt.double().transpose(1, 2)
    ref = per_expert(off, lambda e, s: x[s].double() @ m[e], None)
    acc = k * U23 * per_expert(off, lambda e, s: x[s].double().abs() @ m[e].abs(), None)
    check(y, ref, acc + HALF_BF16 * (ref.abs() + acc), "y")


def test_swiglu_tile_heights():
    H, F = 72, 384
    off, N, shape, ws = by_counts(HEIGHTS, H)
    g = torch.Generator().manual_seed(3)
    x, w13 = randn(g, N, H), randn(g, len(HEIGHTS), 2 * F, H, scale=H ** -0.5)
    act = torch.empty((N, F), dtype=BF16, device="cuda")
    q, sc = torch.empty((N, 2 * F), dtype=U8, device="cuda"), torch.empty((N, 2 * F // 128), device="cuda")
    xd, wd, od = gpu(x, w13, off)
    ep.ep_expert_swiglu(shape, dict(expert_offsets=od), xd, N, wd, F, act, q, sc, ws)
    gu = per_expert(off, lambda e, s: x[s].double() @ w13[e].double().T, None)
    acc = H * U23 * per_expert(off, lambda e, s: x[s].double().abs() @ w13[e].double().abs().T, None)
    gate, up, s, ref = silu_parts(gu, F)
    b = act_bound(gate, up, s, ref, acc[:, :F], acc[:, F:])
    check(act, ref, b + HALF_BF16 * (ref.abs() + b), "act")
    rep = sc.double().cpu().repeat_interleave(128, 1)
    off_by = acc + 4 * U23 * gu.abs()
    check(q.cpu().view(F8).double() * rep, gu, off_by + HALF_E4M3 * (gu.abs() + off_by) + 2.0 ** -10 * rep, "checkpoint")


@pytest.mark.parametrize("back", [False, True], ids=["nk", "kn"])
def test_matmul_more_tiles_than_workgroups(back):
    """Several tiles to a workgroup, of different heights one after the other."""
    counts = [(37 * e) % 290 for e in range(40)]
    off, N, shape, ws = by_counts(counts)
    E, k, n = len(counts), 200, 2056
    g = torch.Generator().manual_seed(5)
    x, wt = randn(g, N, k), randn(g, *((E, k, n) if back else (E, n, k)), scale=k ** -0.5)
    y = torch.full((N, n), 7.0, dtype=BF16, device="cuda")
    xd, wd, od = gpu(x, wt, off)
    ep.ep_expert_matmul(shape, dict(expert_offsets=od), xd, N, k, wd, n,
                        ep.EP_WEIGHT_KN if back else ep.EP_WEIGHT_NK, y, ws)
    m = wt.double() if back else wt.double().transpose(1, 2)
    ref = per_expert(off, lambda e, s: x[s].double() @ m[e], None)
    acc = k * U23 * per_expert(off, lambda e, s: x[s].double().abs() @ m[e].abs(), None)
    check(y, ref, acc + HALF_BF16 * (ref.abs() + acc), "y")


SWIGLU = [
    (1, 1, 1, 8, 128, {}),
    (3, 2, 5, 72, 128, {}),
    (65, 2, 3, 200, 256, dict(skip=0.2)),
    (300, 3, 4, 264, 384, dict(skew=1.0)),
    (140, 8, 9, 512, 640, {}),
    (512, 1, 1, 64, 128, {}),
]


@pytest.mark.parametrize("case", SWIGLU, ids=str)
def test_swiglu_with_checkpoint(case):
    T, K, E, H, F, opt = case
    g, idx, w, off, slot, N, _, _ = product_case(case, 23)
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_workspace(shape)
    spare = 2
    x, w13 = randn(g, N + spare, H), randn(g, E, 2 * F, H, scale=H ** -0.5)
    act = torch.full((N + spare, F), 7.0, dtype=BF16, device="cuda")
    q = torch.full((N + spare, 2 * F), 0x55, dtype=U8, device="cuda")
    sc = torch.full((N + spare, 2 * F // 128), 7.0, device="cuda")
    xd, wd, od = gpu(x, w13, off)
    ep.ep_expert_swiglu(shape, dict(expert_offsets=od), xd, N + spare, wd, F, act, q, sc, ws)
    alone = torch.full_like(act, 7.0)
    ep.ep_expert_swiglu(shape, dict(expert_offsets=od), xd, N + spare, wd, F, alone, None, None, ws)
    assert ep.ep_check_errors(ws) == 0
    assert torch.equal(alone, act)
    assert (act[N:] == 7.0).all() and (q[N:] == 0x55).all() and (sc[N:] == 7.0).all()

    gu = per_expert(off, lambda e, s: x[s].double() @ w13[e].double().T, None)
    acc = H * U23 * per_expert(off, lambda e, s: x[s].double().abs() @ w13[e].double().abs().T, None)
    gate, up, s, ref = silu_parts(gu, F)
    b = act_bound(gate, up, s, ref, acc[:, :F], acc[:, F:])
    check(act[:N], ref, b + HALF_BF16 * (ref.abs() + b), "act")
    # Scales: amax / 448; the largest magnitude is off by the sums' error.
    blocks = gu.reshape(N, -1, 128).abs().amax(2)
    dacc = acc.reshape(N, -1, 128).amax(2)
    check(sc[:N], blocks / 448, dacc / 448 + 4 * U23 * blocks / 448, "scales")
    # Values: v * (1 / scale) rounded to e4m3, for the scale as written.
    rep = sc[:N].double().cpu().repeat_interleave(128, 1)
    val = q[:N].cpu().view(F8).double() * rep
    off_by = acc + 4 * U23 * gu.abs()
    check(val, gu, off_by + HALF_E4M3 * (gu.abs() + off_by) + 2.0 ** -10 * rep, "checkpoint")
    assert (q[:N].cpu().view(F8).float().abs().reshape(N, -1, 128).amax(2) == 448).all()


@pytest.mark.parametrize("F", [8, 72, 136, 1000])
def test_swiglu_without_checkpoint_takes_odd_sizes(F):
    T, K, E, H = 90, 2, 4, 104
    g, idx, w, off, slot, N, _, _ = product_case((T, K, E, H, F, {}), 5)
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_workspace(shape)
    x, w13 = randn(g, N, H), randn(g, E, 2 * F, H, scale=H ** -0.5)
    act = torch.empty((N, F), dtype=BF16, device="cuda")
    xd, wd, od = gpu(x, w13, off)
    ep.ep_expert_swiglu(shape, dict(expert_offsets=od), xd, N, wd, F, act, None, None, ws)
    gu = per_expert(off, lambda e, s: x[s].double() @ w13[e].double().T, None)
    acc = H * U23 * per_expert(off, lambda e, s: x[s].double().abs() @ w13[e].double().abs().T, None)
    gate, up, s, ref = silu_parts(gu, F)
    b = act_bound(gate, up, s, ref, acc[:, :F], acc[:, F:])
    check(act, ref, b + HALF_BF16 * (ref.abs() + b), "act")


def test_swiglu_zero_and_nonfinite_rows():
    """An all-zero row stores scales of 1 and zeros; a row with an infinity
    reads back as NaN where it matters and leaves its neighbours alone."""
    H, F, N = 64, 128, 5
    g = torch.Generator().manual_seed(1)
    x, w13 = randn(g, N, H), randn(g, 1, 2 * F, H)
    x[1] = 0
    x[3, 7] = float("inf")
    shape = ep.make_shape(N, H, 1, 1, 1)
    ws = ep.alloc_workspace(shape)
    off = torch.tensor([0, N], dtype=torch.int32)
    act = torch.empty((N, F), dtype=BF16, device="cuda")
    q = torch.empty((N, 2 * F), dtype=U8, device="cuda")
    sc = torch.empty((N, 2), device="cuda")
    xd, wd, od = gpu(x, w13, off)
    ep.ep_expert_swiglu(shape, dict(expert_offsets=od), xd, N, wd, F, act, q, sc, ws)
    assert (sc[1] == 1).all() and (q[1].view(F8).float() == 0).all() and (act[1] == 0).all()
    val = q.view(F8).float() * sc.repeat_interleave(128, 1)
    assert torch.isnan(val[3]).all()
    for i in (0, 2, 4):
        assert torch.isfinite(val[i]).all() and torch.isfinite(act[i]).all() and (sc[i] != 1).all()


def checkpoint(g, N, F, scale=1.0):
    v = torch.randn((N, 2 * F), generator=g) * scale
    s = v.reshape(N, -1, 128).abs().amax(2) / 448
    return (v / s.repeat_interleave(128, 1)).to(F8), s


GRAD = [(1, 1, 1, 128, {}), (7, 3, 5, 256, dict(skip=0.3)), (50, 8, 16, 640, {}), (33, 2, 4, 1152, {}),
        (20, 4, 4, 2176, dict(repeat=True))]


def grad_reference(idx, w, slot, q, sc, d, F):
    N = len(q)
    gu = q.double() * sc.double().repeat_interleave(128, 1)
    row_w = torch.zeros((N, 1), dtype=F64)
    has = slot >= 0
    row_w[slot[has].long(), 0] = w[has].double()
    return gu, row_w, has


@pytest.mark.parametrize("scale", [1.0, 12.0], ids=["", "wide"])
@pytest.mark.parametrize("case", GRAD, ids=str)
def test_swiglu_grad(case, scale):
    T, K, E, F, opt = case
    g = torch.Generator().manual_seed(31)
    idx, w = routing(T, K, E, 3, **opt)
    off, slot, experts = grouped(idx, E)
    N = len(experts)
    q, sc = checkpoint(g, N, F, scale)
    d = randn(g, N, F)
    shape = ep.make_shape(T, 128, K, E, 1)
    ws = ep.alloc_workspace(shape)
    spare = 2
    d_gu = torch.full((N + spare, 2 * F), 7.0, dtype=BF16, device="cuda")
    act_w = torch.full((N + spare, F), 7.0, dtype=BF16, device="cuda")
    d_w = torch.full((T, K), 7.0, device="cuda")
    pad = lambda t: torch.cat([t.cuda(), torch.zeros((spare, t.shape[1]), device="cuda").to(t.dtype)])
    L = dict(expert_slot=slot.cuda())
    ep.ep_swiglu_grad(shape, L, F, pad(q), pad(sc), pad(d), N + spare, w.cuda(), d_gu, act_w, d_w, ws)
    assert ep.ep_check_errors(ws) == 0
    assert (d_gu[N:] == 7.0).all() and (act_w[N:] == 7.0).all()

    gu, row_w, has = grad_reference(idx, w, slot, q, sc, d, F)
    gate, up, s, act = silu_parts(gu, F)
    dd = d.double()
    rel = (gate.abs() + 24) * U23
    ref_g = row_w * dd * up * s * (1 + gate * (1 - s))
    ref_u = row_w * dd * gate * s
    # 1 + g (1 - s) may cancel: its error goes by the size of its terms.
    bg = (row_w * dd * up * s).abs() * (1 + gate.abs()) * rel
    bu = ref_u.abs() * rel
    check(d_gu[:N, :F], ref_g, bg + HALF_BF16 * (ref_g.abs() + bg), "d_gate")
    check(d_gu[:N, F:], ref_u, bu + HALF_BF16 * (ref_u.abs() + bu), "d_up")
    ref_a = row_w * act
    ba = ref_a.abs() * rel
    check(act_w[:N], ref_a, ba + HALF_BF16 * (ref_a.abs() + ba), "act_w")
    ref_w = torch.zeros((T, K), dtype=F64)
    bw = torch.zeros((T, K), dtype=F64)
    ref_w[has] = (dd * act).sum(1)[slot[has].long()]
    bw[has] = ((dd * act).abs() * (rel + F * U23)).sum(1)[slot[has].long()]
    check(d_w, ref_w, bw, "d_topk_weights")
    # Optional outputs left out: the others stay the same.
    again = torch.empty_like(d_gu)
    ep.ep_swiglu_grad(shape, L, F, pad(q), pad(sc), pad(d), N + spare, w.cuda(), again, None, None, ws)
    assert torch.equal(again[:N], d_gu[:N])


def test_swiglu_grad_against_differences():
    """The gradient against central differences, in 64 bits, of
    sum w d silu(g) u at the checkpoint's values: steps of 1e-4 leave errors of
    about 1e-8 |w d| (1 + |u|), far under the result's bf16 rounding."""
    T, K, E, F = 6, 2, 3, 128
    g = torch.Generator().manual_seed(77)
    idx, w = routing(T, K, E, 8)
    off, slot, experts = grouped(idx, E)
    N = len(experts)
    q, sc = checkpoint(g, N, F)
    d = randn(g, N, F)
    shape = ep.make_shape(T, 128, K, E, 1)
    ws = ep.alloc_workspace(shape)
    d_gu = torch.empty((N, 2 * F), dtype=BF16, device="cuda")
    ep.ep_swiglu_grad(shape, dict(expert_slot=slot.cuda()), F, q.cuda(), sc.cuda(), d.cuda(), N, w.cuda(), d_gu,
                      None, None, ws)
    gu, row_w, _ = grad_reference(idx, w, slot, q, sc, d, F)
    f = lambda a, b: row_w * d.double() * a * torch.sigmoid(a) * b
    gate, up, h = gu[:, :F], gu[:, F:], 1e-4
    num = torch.cat([(f(gate + h, up) - f(gate - h, up)), (f(gate, up + h) - f(gate, up - h))], 1) / (2 * h)
    small = 1e-7 * (row_w * d.double()).abs().repeat(1, 2) * (1 + up.abs().repeat(1, 2)) * (8 + gate.abs().repeat(1, 2))
    check(d_gu, num, small + HALF_BF16 * (num.abs() + small), "d_gu against differences")


WGRAD = [
    (1, 1, 1, 8, 128, {}),
    (5, 3, 9, 72, 128, dict(skip=0.3)),
    (100, 2, 3, 264, 384, {}),
    (300, 2, 2, 520, 256, dict(skew=1.0)),
    (64, 1, 1, 256, 256, {}),
    (65, 1, 1, 24, 640, {}),
]


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("fp8", [False, True], ids=["rows", "fp8rows"])
@pytest.mark.parametrize("case", WGRAD, ids=str)
def test_wgrad(case, fp8, wide):
    T, K, E, n, k, opt = case
    g, idx, w, off, slot, N, shape, ws = product_case((T, K, E, k, n, opt), 41)
    dy = randn(g, N + 1, n)
    if fp8:
        q, sc = checkpoint(g, N + 1, k // 2)
        x = q.double() * sc.double().repeat_interleave(128, 1)
        rows = dict(x_fp8=q.cuda(), x_scales=sc.cuda())
    else:
        xb = randn(g, N + 1, k)
        x, rows = xb.double(), dict(x=xb.cuda())
    dw = torch.full((E, n, k), 7.0, dtype=F32 if wide else BF16, device="cuda")
    dyd, od = gpu(dy, off)
    ep.ep_expert_wgrad(shape, dict(expert_offsets=od), dyd, N + 1, n, rows, k, dw,
                       ep.EP_GRAD_F32 if wide else ep.EP_GRAD_BF16, ws)
    assert ep.ep_check_errors(ws) == 0
    parts = [slice(int(off[e]), int(off[e + 1])) for e in range(E)]
    ref = torch.stack([dy[p].double().T @ x[p] for p in parts])
    mag = torch.stack([dy[p].double().abs().T @ x[p].abs() for p in parts])
    most = max(p.stop - p.start for p in parts)
    acc = most * U23 * mag + (HALF_BF16 * mag * (1 + most * U23) + U23 * mag if fp8 else 0)
    check(dw, ref, acc if wide else acc + HALF_BF16 * (ref.abs() + acc), "dw")
    # The sum over one row more is the old one plus that row's product: the
    # gradient is linear in the rows (a difference, exact up to roundings).
    if wide and not fp8 and E == 1:
        od2 = torch.tensor([0, N + 1], dtype=torch.int32, device="cuda")
        more = torch.empty_like(dw)
        ep.ep_expert_wgrad(shape, dict(expert_offsets=od2), dyd, N + 1, n, rows, k, more, ep.EP_GRAD_F32, ws)
        outer = dy[N].double().unsqueeze(1) * x[N].unsqueeze(0)
        both = mag[0] + outer.abs()
        check((more.double() - dw.double())[0], outer, 2 * (N + 1) * U23 * both, "difference by one row")


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("fp8", [False, True], ids=["rows", "fp8rows"])
def test_wgrad_many_tiles_of_all_lengths(fp8, wide):
    """Several tiles to a workgroup: experts without rows, of one row, of 1, 2, 3
    and more steps of 64 rows, one after the other in one stream."""
    counts = [0, 1, 0, 63, 64, 65, 128, 0, 0, 129, 192, 200, 5, 300, 0, 1, 256, 70, 10, 0]
    off, N, shape, ws = by_counts(counts)
    E, n, k = len(counts), 1032, 768
    g = torch.Generator().manual_seed(7)
    dy = randn(g, N, n)
    if fp8:
        q, sc = checkpoint(g, N, k // 2)
        x, rows = q.double() * sc.double().repeat_interleave(128, 1), dict(x_fp8=q.cuda(), x_scales=sc.cuda())
    else:
        xb = randn(g, N, k)
        x, rows = xb.double(), dict(x=xb.cuda())
    dw = torch.full((E, n, k), 7.0, dtype=F32 if wide else BF16, device="cuda")
    dyd, od = gpu(dy, off)
    ep.ep_expert_wgrad(shape, dict(expert_offsets=od), dyd, N, n, rows, k, dw,
                       ep.EP_GRAD_F32 if wide else ep.EP_GRAD_BF16, ws)
    parts = [slice(int(off[e]), int(off[e + 1])) for e in range(E)]
    for e, p in enumerate(parts):
        ref = dy[p].double().T @ x[p]
        mag = dy[p].double().abs().T @ x[p].abs()
        acc = counts[e] * U23 * mag + (HALF_BF16 * mag * (1 + counts[e] * U23) + U23 * mag if fp8 else 0)
        check(dw[e], ref, acc if wide else acc + HALF_BF16 * (ref.abs() + acc), f"dw of expert {e}")


def test_wgrad_of_one_expert_repeats_bit_for_bit():
    """No order of summation depends on timing."""
    off, N, shape, ws = by_counts([400, 0, 333])
    g = torch.Generator().manual_seed(8)
    dy, x = randn(g, N, 520).cuda(), randn(g, N, 264).cuda()
    od = off.cuda()
    outs = []
    for _ in range(3):
        dw = torch.empty((3, 520, 264), device="cuda")
        ep.ep_expert_wgrad(shape, dict(expert_offsets=od), dy, N, 520, dict(x=x), 264, dw, ep.EP_GRAD_F32, ws)
        outs.append(dw)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def near(got, ref, mag, n, what):
    """One rounding to bf16 and n products summed in 32 bits."""
    check(got, ref.cpu(), (n * U23 * mag + HALF_BF16 * (ref.abs() + n * U23 * mag)).cpu(), what)


def test_offsets_past_32_bits():
    """Rows, weights and results behind the first 4 GiB of their arrays."""
    g = torch.Generator(device="cuda").manual_seed(1)
    k, n = 8192, 64
    counts = [290_000, 40]
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    N = sum(counts)
    x = torch.randn((N, k), generator=g, device="cuda", dtype=BF16)  # 4.75 GB
    w = torch.randn((2, n, k), generator=g, device="cuda", dtype=BF16)
    shape = ep.make_shape(8, k, 1, 2, 1)
    ws = ep.alloc_workspace(shape)
    y = torch.empty((N, n), dtype=BF16, device="cuda")
    L = dict(expert_offsets=off)
    ep.ep_expert_matmul(shape, L, x, N, k, w, n, ep.EP_WEIGHT_NK, y, ws)
    for e, rows in ((0, slice(289_900, 290_000)), (1, slice(290_000, N))):
        a, b = x[rows].double(), w[e].double()
        near(y[rows], a @ b.T, a.abs() @ b.abs().T, k, "rows")
    # Results past 4 GiB: the other way round.
    back = torch.empty((N, k), dtype=BF16, device="cuda")
    ep.ep_expert_matmul(shape, L, y, N, n, w, k, ep.EP_WEIGHT_KN, back, ws)
    a, b = y[290_000:].double(), w[1].double()
    near(back[290_000:], a @ b, a.abs() @ b.abs(), n, "results")
    # The gradient of the last expert reads only its rows.
    dw = torch.empty((2, n, k), device="cuda")
    ep.ep_expert_wgrad(shape, L, y, N, n, dict(x=x), k, dw, ep.EP_GRAD_F32, ws)
    a, b = y[290_000:].double(), x[290_000:].double()
    check(dw[1], (a.T @ b).cpu(), (40 * U23 * (a.abs().T @ b.abs())).cpu(), "dw")
    del x, y, back, dw
    # Weights past 4 GiB, of the products and of the few-token layer.
    E, H, F = 90, 4096, 4096
    w13 = torch.randn((E, 2 * F, H), generator=g, device="cuda", dtype=BF16).mul_(H ** -0.5)  # 6 GB
    w2 = torch.randn((E, H, F), generator=g, device="cuda", dtype=BF16).mul_(F ** -0.5)
    T = 3
    xt = torch.randn((T, H), generator=g, device="cuda", dtype=BF16)
    idx = torch.tensor([[E - 1], [E - 2], [0]], device="cuda")
    wt = torch.ones((T, 1), device="cuda")
    s2 = ep.make_shape(T, H, 1, E, 1)
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    ep.ep_moe_few(s2, dict(x=xt, topk_idx=idx, topk_weights=wt), dict(F=F, w13=w13, w2=w2), out,
                  ep.alloc_few_workspace(s2, F))
    act = torch.empty((1, F), dtype=BF16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 1
    ep.ep_expert_swiglu(s2, dict(expert_offsets=off), xt[:1].contiguous(), 1, w13, F, act, None, None,
                        ep.alloc_workspace(s2))
    for t in range(T):
        e = int(idx[t, 0])
        ref, bound = few_reference(xt[t:t + 1].cpu(), w13[e:e + 1].cpu(), w2[e:e + 1].cpu(),
                                   torch.zeros((1, 1), dtype=torch.int64), wt[:1].cpu(), F)
        check(out[t:t + 1], ref, bound, f"token {t}")
    gu = xt[:1].double() @ w13[E - 1].double().T
    acc = H * U23 * (xt[:1].double().abs() @ w13[E - 1].double().abs().T)
    gate, up, sg, ref = silu_parts(gu, F)
    b = act_bound(gate, up, sg, ref, acc[:, :F], acc[:, F:])
    check(act, ref.cpu(), (b + HALF_BF16 * (ref.abs() + b)).cpu(), "act")


FEW = [
    # (T, H, F, E, K, options)
    (1, 256, 512, 16, 2, {}),
    (1, 8, 8, 1, 1, {}),
    (2, 72, 40, 3, 2, {}),
    (13, 264, 136, 40, 3, dict(skip=0.2)),
    (16, 640, 384, 8, 8, {}),
    (17, 128, 256, 5, 4, dict(repeat=True)),
    (40, 200, 264, 4, 2, {}),
    (128, 136, 72, 2, 1, {}),            # 64 tokens and more to one expert
    (36, 128, 128, 1, 1, {}),            # three token tiles of one expert
    (128, 128, 128, 4096, 4, {}),        # the largest number of experts
    (100, 64, 48, 3, 64, dict(repeat=True)),
    (5, 1032, 712, 6, 6, {}),
    (103, 512, 1024, 10, 8, {}),         # workgroups that share outputs, many tokens to each expert
]


def few_reference(x, w13, w2, idx, w, F):
    """out and its bound in 64 bits."""
    T, H = x.shape
    out, bound = torch.zeros((T, H), dtype=F64), torch.zeros((T, H), dtype=F64)
    xd = x.double()
    lanes = 0
    for e in range(len(w13)):
        hit = (idx == e)
        ts = hit.any(1).nonzero()[:, 0]
        if not len(ts):
            continue
        lanes += 1
        a, b2 = w13[e].double(), w2[e].double()
        gu = xd[ts] @ a.T
        acc = H * U23 * (xd[ts].abs() @ a.abs().T)
        gate, up, s, act = silu_parts(gu, F)
        da = act_bound(gate, up, s, act, acc[:, :F], acc[:, F:])
        da = da + 2.0 ** -16 * (act.abs() + da)  # two bf16 values: the rest is rounded, 2^-8 of 2^-8
        we = (w.double() * hit).sum(1)[ts].unsqueeze(1)
        wabs = (w.double().abs() * hit).sum(1)[ts].unsqueeze(1)
        out[ts] += we * (act @ b2.T)
        mag = (act.abs() + da) @ b2.abs().T
        bound[ts] += wabs * (da @ b2.abs().T + F * U23 * mag) + 80 * U23 * wabs * mag
    bound = bound + 8 * U23 * out.abs()
    return out, bound + HALF_BF16 * (out.abs() + bound)


def eight(w):
    """e4m3 weights, scales and the values they stand for."""
    E, n, k = w.shape
    s = w.float().reshape(E, n, -1, 128).abs().amax(3).clamp(min=1e-20) / 448
    q = (w.float() / s.repeat_interleave(128, 2)).to(F8)
    return q, s, q.double() * s.double().repeat_interleave(128, 2)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", FEW, ids=str)
def test_few(case, fp8):
    T, H, F, E, K, opt = case
    if fp8:  # the same cases at the next sizes that FP8 takes
        H, F = -(-H // 128) * 128, -(-F // 128) * 128
        if E == 4096:
            E = 1024
    g = torch.Generator().manual_seed(9)
    idx, w = routing(T, K, E, 17, **opt)
    x, w13, w2 = randn(g, T, H), randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5)
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_few_workspace(shape, F).fill_(0xAB)
    ep.ep_clear_errors(ws)
    if fp8:
        (q13, s13, w13), (q2, s2, w2) = eight(w13), eight(w2)
        experts = dict(F=F, w13_fp8=q13.cuda(), w13_scales=s13.cuda(), w2_fp8=q2.cuda(), w2_scales=s2.cuda())
    else:
        experts = dict(F=F, w13=w13.cuda(), w2=w2.cuda())
    out = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    tokens = dict(x=x.cuda(), topk_idx=idx.cuda(), topk_weights=w.cuda())
    ep.ep_moe_few(shape, tokens, experts, out, ws)
    assert ep.ep_check_errors(ws) == 0
    ref, bound = few_reference(x, w13, w2, idx, w, F)
    check(out, ref, bound, "out")
    again = torch.empty_like(out)
    ep.ep_moe_few(shape, tokens, experts, again, ws)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_few_keeps_nonfinite_values_with_their_tokens():
    """NaN and infinite weights of one expert reach only its tokens; a token of
    NaN only itself; a token without a lane gets zeros; bad ids are reported
    and skipped."""
    T, H, F, E, K = 6, 128, 256, 4, 2
    g = torch.Generator().manual_seed(2)
    x, w13, w2 = randn(g, T, H), randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5)
    idx = torch.tensor([[0, 1], [1, 2], [-1, -1], [3, 0], [0, 99], [-7, 1]])
    w = torch.full((T, K), 0.5)
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_few_workspace(shape, F)
    clean = torch.where((idx < 0) | (idx >= E), -1, idx)
    ref, bound = few_reference(x, w13, w2, clean, w, F)
    bad13, bad2, badx = w13.clone(), w2.clone(), x.clone()
    bad13[2, 3, :] = float("inf")     # expert 2: token 1 only
    bad2[2, 5, 9] = float("nan")
    bad2[3] = float("nan")            # expert 3: token 3 only
    badx[4] = float("nan")            # token 4 only
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    ep.ep_moe_few(shape, dict(x=badx.cuda(), topk_idx=idx.cuda(), topk_weights=w.cuda()),
                  dict(F=F, w13=bad13.cuda(), w2=bad2.cuda()), out, ws)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_EXPERT_ID
    for t in (0, 2, 5):
        check(out[t], ref[t], bound[t], f"token {t}")
    assert (out[2] == 0).all()
    assert torch.isnan(out[3]).all() and torch.isnan(out[4]).all() and not torch.isfinite(out[1]).all()


def test_rows_past_the_capacity_are_left_out():
    E, k, n, N = 3, 64, 72, 50
    g = torch.Generator().manual_seed(4)
    off = torch.tensor([0, 20, 40, N], dtype=torch.int32)
    have = 33
    x, wt = randn(g, have, k), randn(g, E, n, k, scale=k ** -0.5)
    shape = ep.make_shape(N, 128, 1, E, 1)
    ws = ep.alloc_workspace(shape)
    ep.ep_clear_errors(ws)
    y = torch.empty((have, n), dtype=BF16, device="cuda")
    xd, wd, od = gpu(x, wt, off)
    ep.ep_expert_matmul(shape, dict(expert_offsets=od), xd, have, k, wd, n, ep.EP_WEIGHT_NK, y, ws)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_CAPACITY
    cut = off.clamp(max=have)
    ref = per_expert(cut, lambda e, s: x[s].double() @ wt[e].double().T, None)
    mag = per_expert(cut, lambda e, s: x[s].double().abs() @ wt[e].double().abs().T, None)
    check(y, ref, k * U23 * mag + HALF_BF16 * (ref.abs() + k * U23 * mag), "y")
    # A lane whose row lies past the capacity: reported, gradient 0.
    F = 128
    slot = torch.tensor([[0], [33]], dtype=torch.int32, device="cuda")
    s2 = ep.make_shape(2, 128, 1, E, 1)
    ep.ep_clear_errors(ws)
    q, sc = checkpoint(g, have, F)
    d_w = torch.full((2, 1), 7.0, device="cuda")
    d_gu = torch.full((have, 2 * F), 7.0, dtype=BF16, device="cuda")
    ep.ep_swiglu_grad(s2, dict(expert_slot=slot), F, q.cuda(), sc.cuda(), randn(g, have, F).cuda(), have,
                      torch.ones((2, 1), device="cuda"), d_gu, None, d_w, ws)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_CAPACITY
    assert d_w[1, 0] == 0 and d_w[0, 0] != 7.0 and (d_gu[1:] == 7.0).all()


def test_no_rows_and_no_tokens():
    E, k, n = 5, 64, 128
    shape = ep.make_shape(4, 128, 2, E, 1)
    ws = ep.alloc_workspace(shape)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    wt = torch.zeros((E, n, k), dtype=BF16, device="cuda")
    y = torch.full((8, n), 7.0, dtype=BF16, device="cuda")
    x = torch.zeros((8, n), dtype=BF16, device="cuda")
    L = dict(expert_offsets=off)
    ep.ep_expert_matmul(shape, L, x, 8, k, wt, n, ep.EP_WEIGHT_NK, y, ws)
    ep.ep_expert_matmul(shape, L, None, 0, k, wt, n, ep.EP_WEIGHT_NK, None, ws)
    assert (y == 7.0).all()
    for rows, dy, xs in ((8, y, dict(x=x)), (0, None, {})):
        dw = torch.full((E, n, k), 7.0, device="cuda")
        ep.ep_expert_wgrad(shape, L, dy, rows, n, xs, k, dw, ep.EP_GRAD_F32, ws)
        assert (dw == 0).all()
    s0 = ep.make_shape(0, 128, 2, E, 1)
    w0 = ep.alloc_few_workspace(s0, 8).fill_(0xAB)
    ep.ep_moe_few(s0, {}, dict(F=8, w13=wt, w2=wt), None, w0)
    assert ep.ep_check_errors(w0) == 0


def layer_case(T=150, H=256, F=256, E=8, K=3, skip=0.1):
    g = torch.Generator().manual_seed(6)
    idx, w = routing(T, K, E, 21, skip=skip)
    x, dout = randn(g, T, H), randn(g, T, H)
    w13, w2 = randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5)
    return idx, w, x, dout, w13, w2


def layer_step(shape, F, idx, w, x, dout, w13, w2, bufs=None):
    """Forward and backward of a whole layer by the entry points; every
    intermediate in a dict."""
    T, H, K, E = shape.T, shape.H, shape.K, shape.E
    b = bufs if bufs is not None else {}
    N = T * K

    def buf(name, *size, dtype=BF16):
        if name not in b:
            b[name] = torch.zeros(size, dtype=dtype, device="cuda")
        return b[name]

    if "L" not in b:
        b["L"], b["ws"] = ep.alloc_layout(shape, expand=True), ep.alloc_workspace(shape)
        b["recv"] = ep.alloc_recv(shape, N)
        b["d_recv"] = ep.alloc_recv(shape, N, meta=False)
        b["ones"] = torch.ones((T, K), device="cuda")
    L, ws = b["L"], b["ws"]
    ep.ep_get_layout(shape, idx, L, ws)
    ep.ep_dispatch_expand(shape, L, dict(x=x, topk_idx=idx, topk_weights=w), b["recv"], N, ws)
    xr = b["recv"]["x"]
    act, q = buf("act", N, F), buf("q", N, 2 * F, dtype=U8)
    sc = buf("sc", N, 2 * F // 128, dtype=F32)
    ep.ep_expert_swiglu(shape, L, xr, N, w13, F, act, q, sc, ws)
    y, out = buf("y", N, H), buf("out", T, H)
    ep.ep_expert_matmul(shape, L, act, N, F, w2, H, ep.EP_WEIGHT_NK, y, ws)
    ep.ep_combine_expand(shape, L, y, N, 2 * H, ep.EP_FMT_PLAIN, 0, w, out, ws)

    ep.ep_dispatch_expand(shape, L, dict(x=dout, topk_idx=idx), b["d_recv"], N, ws)
    dy = b["d_recv"]["x"]
    d_act, d_gu, act_w = buf("d_act", N, F), buf("d_gu", N, 2 * F), buf("act_w", N, F)
    d_w = buf("d_w", T, K, dtype=F32)
    ep.ep_expert_matmul(shape, L, dy, N, H, w2, F, ep.EP_WEIGHT_KN, d_act, ws)
    ep.ep_swiglu_grad(shape, L, F, q, sc, d_act, N, w, d_gu, act_w, d_w, ws)
    dw2, dw13 = buf("dw2", E, H, F, dtype=F32), buf("dw13", E, 2 * F, H, dtype=F32)
    ep.ep_expert_wgrad(shape, L, dy, N, H, dict(x=act_w), F, dw2, ep.EP_GRAD_F32, ws)
    ep.ep_expert_wgrad(shape, L, d_gu, N, 2 * F, dict(x=xr), H, dw13, ep.EP_GRAD_F32, ws)
    dxr, dx = buf("dxr", N, H), buf("dx", T, H)
    ep.ep_expert_matmul(shape, L, d_gu, N, 2 * F, w13, H, ep.EP_WEIGHT_KN, dxr, ws)
    ep.ep_combine_expand(shape, L, dxr, N, 2 * H, ep.EP_FMT_PLAIN, 0, b["ones"], dx, ws)
    return b


def test_whole_layer_forward_and_backward():
    """A layer's training step against automatic differentiation in 64 bits.

    The forward output passes three roundings to bf16 (act, y, out): each
    2^-8 at most, so the 2-norm is off by at most 3 * 2^-8 of itself for values
    of random sign. The backward also uses g and u from 8 bits (2^-4 at most
    of each value, uniformly spread: 2^-4 / sqrt(3) in 2-norm for the largest
    mantissa step, less on average), which enters the gradients through
    products of g and u: twice that, and the bf16 roundings, bound them by
    2 * 2^-4 + 4 * 2^-8 of their norm."""
    T, H, F, E, K = 150, 256, 256, 8, 3
    idx, w, x, dout, w13, w2 = layer_case(T, H, F, E, K)
    shape = ep.make_shape(T, H, K, E, 1)
    b = layer_step(shape, F, *gpu(idx, w, x, dout, w13, w2))
    assert ep.ep_check_errors(b["ws"]) == 0
    X, W13, W2, W = (t.double().requires_grad_() for t in (x, w13, w2, w))
    out = torch.zeros((T, H), dtype=F64)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        gu = X[t] @ W13[e].T
        a = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        out = out.index_add(0, t, W[t, k].unsqueeze(1) * (a @ W2[e].T))
    out.backward(dout.double())
    rel = lambda a, r: ((a.double().cpu() - r).norm() / r.norm()).item()
    assert rel(b["out"], out.detach()) <= 3 * HALF_BF16
    for name, ref in (("dx", X.grad), ("dw13", W13.grad), ("dw2", W2.grad), ("d_w", W.grad)):
        assert rel(b[name], ref) <= 2 * HALF_E4M3 + 4 * HALF_BF16, name
    # The few-token layer computes the same output.
    s2 = ep.make_shape(128, H, K, E, 1)
    ws = ep.alloc_few_workspace(s2, F)
    few = torch.empty((128, H), dtype=BF16, device="cuda")
    ep.ep_moe_few(s2, dict(x=x[:128].cuda(), topk_idx=idx[:128].cuda().contiguous(),
                           topk_weights=w[:128].cuda().contiguous()), dict(F=F, w13=w13.cuda(), w2=w2.cuda()), few, ws)
    assert rel(few, out.detach()[:128]) <= 3 * HALF_BF16


def test_whole_layer_in_a_graph():
    """The training step and the few-token layer captured once and replayed
    with new inputs, other work and waits between the replays; every replay
    equals the eager result bit for bit."""
    T, H, F, E, K = 100, 128, 128, 6, 2
    shape = ep.make_shape(T, H, K, E, 1)
    inputs = [gpu(*layer_case(T, H, F, E, K)), None, None]
    for i in (1, 2):
        idx, w = routing(T, K, E, 50 + i, skip=0.2)
        g = torch.Generator().manual_seed(60 + i)
        inputs[i] = [idx.cuda(), w.cuda(), randn(g, T, H).cuda(), randn(g, T, H).cuda(), inputs[0][4], inputs[0][5]]
    names = ("out", "dx", "dw13", "dw2", "d_w", "few")

    def step(args, b):
        layer_step(shape, F, *args, bufs=b)
        if "few" not in b:
            b["few"], b["few_ws"] = torch.zeros((T, H), dtype=BF16, device="cuda"), ep.alloc_few_workspace(shape, F)
        ep.ep_moe_few(shape, dict(x=args[2], topk_idx=args[0], topk_weights=args[1]),
                      dict(F=F, w13=args[4], w2=args[5]), b["few"], b["few_ws"])

    eager = []
    for args in inputs:
        b = {}
        step(args, b)
        torch.cuda.synchronize()
        eager.append({n: b[n].clone() for n in names})
    static, b = [t.clone() for t in inputs[0]], {}
    step(static, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, b)
    for i in (0, 1, 2, 1, 0):
        for s, t in zip(static, inputs[i]):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(b[n].view(U8), eager[i][n].view(U8)), (i, n)
        torch.randn(1000, device="cuda").sum().item()
        step(inputs[i], {})  # eager work on buffers of its own between replays


def test_calls_run_on_the_given_stream():
    """Each call on a stream of its own, ordered behind work queued there."""
    T, H, F, E, K = 16, 128, 128, 4, 2
    idx, w, x, dout, w13, w2 = gpu(*layer_case(T, H, F, E, K))
    shape = ep.make_shape(T, H, K, E, 1)
    ref = layer_step(shape, F, idx, w, x, dout, w13, w2)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    x2, b = torch.zeros_like(x), {}
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        big = torch.randn(2048, 2048, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-3
        x2.copy_(x)
        layer_step(shape, F, idx, w, x2, dout, w13, w2, bufs=b)
    st.synchronize()
    for n in ("out", "dx", "dw13", "dw2", "d_w"):
        assert torch.equal(b[n], ref[n]), n


def test_calls_at_once():
    """Two streams at once: the few-token layer on a workspace each, the
    products on one workspace between them (they use its error words alone)."""
    T, H, F, E, K = 32, 512, 384, 12, 4
    idx, w, x, dout, w13, w2 = gpu(*layer_case(T, H, F, E, K))
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_workspace(shape)
    counts = [50, 0, 300, 7, 90, 1, 256, 33, 64, 12, 100, 5]
    off, N, _, _ = by_counts(counts)
    off = off.cuda()
    rows = randn(torch.Generator().manual_seed(3), N, H).cuda()
    d = randn(torch.Generator().manual_seed(4), N, F).cuda()
    L = dict(expert_offsets=off)

    def work(few_ws):
        out = torch.empty((T, H), dtype=BF16, device="cuda")
        ep.ep_moe_few(shape, dict(x=x, topk_idx=idx, topk_weights=w), dict(F=F, w13=w13, w2=w2), out, few_ws)
        act = torch.empty((N, F), dtype=BF16, device="cuda")
        q, sc = torch.empty((N, 2 * F), dtype=U8, device="cuda"), torch.empty((N, 2 * F // 128), device="cuda")
        ep.ep_expert_swiglu(shape, L, rows, N, w13, F, act, q, sc, ws)
        y = torch.empty((N, H), dtype=BF16, device="cuda")
        ep.ep_expert_matmul(shape, L, act, N, F, w2, H, ep.EP_WEIGHT_NK, y, ws)
        dw = torch.empty((E, F, H), device="cuda")
        ep.ep_expert_wgrad(shape, L, d, N, F, dict(x=rows), H, dw, ep.EP_GRAD_F32, ws)
        return out, act, q, sc, y, dw

    ref = work(ep.alloc_few_workspace(shape, F))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [ep.alloc_few_workspace(shape, F) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st, few_ws in zip(streams, spaces):
            with torch.cuda.stream(st):
                got.append(work(few_ws))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, ref):
            assert torch.equal(a.view(U8), b.view(U8))


def test_offsets_that_decrease():
    """The products compute nothing and say so; weight gradients stay inside the arrays."""
    N, k, n, F = 48, 64, 72, 128
    shape = ep.make_shape(N, k, 1, 3, 1)
    g = torch.Generator().manual_seed(4)
    x, w, w13 = gpu(randn(g, N, k), randn(g, 3, n, k), randn(g, 3, 2 * F, k))
    off = torch.tensor([0, 40, 16, 48], dtype=torch.int32, device="cuda")
    ws = ep.alloc_workspace(shape)
    y = torch.full((N, n), 7.0, dtype=BF16, device="cuda")
    act = torch.full((N, F), 7.0, dtype=BF16, device="cuda")
    for call in (lambda: ep.ep_expert_matmul(shape, dict(expert_offsets=off), x, N, k, w, n, ep.EP_WEIGHT_NK, y, ws),
                 lambda: ep.ep_expert_swiglu(shape, dict(expert_offsets=off), x, N, w13, F, act, None, None, ws)):
        ep.ep_clear_errors(ws)
        call()
        assert ep.ep_check_errors(ws) == ep.EP_DEVERR_CAPACITY
    assert (y == 7.0).all() and (act == 7.0).all()
    dy = randn(g, N, n)
    dw = torch.empty((3, n, k), dtype=F32, device="cuda")
    ep.ep_expert_wgrad(shape, dict(expert_offsets=off), dy.cuda(), N, n, dict(x=x), k, dw, ep.EP_GRAD_F32, ws)
    assert (dw[1] == 0).all()
    for e, s in ((0, slice(0, 40)), (2, slice(16, 48))):
        a, b = dy[s].double(), x[s].cpu().double()
        check(dw[e], a.T @ b, 48 * U23 * (a.abs().T @ b.abs()), "dw")


def test_few_repeats_bit_for_bit():
    """Workgroups that share outputs finish in any order; eager calls and replays agree."""
    T, H, F, E, K = 40, 264, 1032, 12, 4
    g = torch.Generator().manual_seed(8)
    idx, w = routing(T, K, E, 3)
    x, w13, w2 = gpu(randn(g, T, H), randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5))
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_few_workspace(shape, F).fill_(0xAB)
    ep.ep_clear_errors(ws)
    tokens = dict(x=x, topk_idx=idx.cuda(), topk_weights=w.cuda())
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    ep.ep_moe_few(shape, tokens, dict(F=F, w13=w13, w2=w2), out, ws)
    first = out.clone()
    ref, bound = few_reference(x.cpu(), w13.cpu(), w2.cpu(), idx, w, F)
    check(first, ref, bound, "out")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_moe_few(shape, tokens, dict(F=F, w13=w13, w2=w2), out, ws)
    for n in range(20):
        out.fill_(7.0)
        if n % 2:
            graph.replay()
        else:
            ep.ep_moe_few(shape, tokens, dict(F=F, w13=w13, w2=w2), out, ws)
        assert torch.equal(out, first), n
    assert ep.ep_check_errors(ws) == 0


def cleared(shape):
    ws = ep.alloc_workspace(shape)
    ep.ep_clear_errors(ws)
    return ws


# Offsets that no layout gives, over 48 rows: a decrease, one behind which the last is
# in range, a last one past the rows (alone, and with an inner one).
BAD_OFFSETS = [(0, 40, 16, 48), (0, 60, 50, 48), (0, 60, 40, 40), (0, 20, 40, 49), (0, 48, 52, 60)]


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("fp8", [False, True], ids=["rows", "fp8rows"])
@pytest.mark.parametrize("offs", BAD_OFFSETS, ids=str)
def test_wgrad_reports_bad_offsets(offs, fp8, wide):
    """The error is set; each expert's gradient is that of its range, cut to the arrays."""
    N, n, k = 48, 72, 128
    shape = ep.make_shape(N, 128, 1, 3, 1)
    g = torch.Generator().manual_seed(4)
    dy = randn(g, N, n)
    if fp8:
        q, sc = checkpoint(g, N, k // 2)
        x, rows = q.double() * sc.double().repeat_interleave(128, 1), dict(x_fp8=q.cuda(), x_scales=sc.cuda())
    else:
        xb = randn(g, N, k)
        x, rows = xb.double(), dict(x=xb.cuda())
    dyd = dy.cuda()
    ws = cleared(shape)
    dw = torch.full((3, n, k), 7.0, dtype=F32 if wide else BF16, device="cuda")
    call = lambda o: ep.ep_expert_wgrad(shape, dict(expert_offsets=torch.tensor(o, dtype=torch.int32, device="cuda")),
                                        dyd, N, n, rows, k, dw, ep.EP_GRAD_F32 if wide else ep.EP_GRAD_BF16, ws)
    call(offs)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_CAPACITY
    for e in range(3):
        lo = min(offs[e], N)
        s = slice(lo, min(max(offs[e + 1], lo), N))
        a, b = dy[s].double(), x[s]
        mag = a.abs().T @ b.abs()
        acc = 48 * U23 * mag + (HALF_BF16 * mag * (1 + 48 * U23) + U23 * mag if fp8 else 0)
        check(dw[e], a.T @ b, acc if wide else acc + HALF_BF16 * ((a.T @ b).abs() + acc), f"dw of expert {e}")
    ep.ep_clear_errors(ws)
    call((0, 20, 20, 48))
    assert ep.ep_check_errors(ws) == 0


def test_wgrad_reports_bad_offsets_of_many_experts():
    """A decrease anywhere among more experts than a workgroup has threads."""
    E, N, n, k = 1500, 64, 8, 8
    shape = ep.make_shape(N, 128, 1, E, 1)
    g = torch.Generator().manual_seed(4)
    dy, x = gpu(randn(g, N, n), randn(g, N, k))
    dw = torch.empty((E, n, k), dtype=BF16, device="cuda")
    ws = cleared(shape)
    for at in (None, 1, 511, 512, 513, 1024, E - 1):
        off = torch.full((E + 1,), 32, dtype=torch.int32)
        off[0] = 0
        if at is not None:
            off[at] = 33
        ep.ep_clear_errors(ws)
        ep.ep_expert_wgrad(shape, dict(expert_offsets=off.cuda()), dy, N, n, dict(x=x), k, dw, ep.EP_GRAD_BF16, ws)
        assert ep.ep_check_errors(ws) == (0 if at is None else ep.EP_DEVERR_CAPACITY), at


def test_products_without_rows_report_offsets_past_them():
    E, k, n, F = 3, 64, 72, 128
    shape = ep.make_shape(8, k, 1, E, 1)
    g = torch.Generator().manual_seed(4)
    w, w13 = gpu(randn(g, E, n, k), randn(g, E, 2 * F, k))
    ws = cleared(shape)
    calls = [lambda L: ep.ep_expert_matmul(shape, L, None, 0, k, w, n, ep.EP_WEIGHT_NK, None, ws),
             lambda L: ep.ep_expert_matmul(shape, L, None, 0, n, w, k, ep.EP_WEIGHT_KN, None, ws),
             lambda L: ep.ep_expert_swiglu(shape, L, None, 0, w13, F, None, None, None, ws)]
    for offs, want in (((0, 0, 0, 0), 0), ((0, 0, 3, 3), ep.EP_DEVERR_CAPACITY), ((0, 1, 0, 0), ep.EP_DEVERR_CAPACITY)):
        L = dict(expert_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda"))
        for i, call in enumerate(calls):
            ep.ep_clear_errors(ws)
            call(L)
            assert ep.ep_check_errors(ws) == want, (offs, i)


def test_negative_offsets_are_bad_ones():
    """An expert cannot begin before the first row: products compute nothing, all report."""
    N, k, n, F, E = 48, 64, 72, 128, 3
    shape = ep.make_shape(N, k, 1, E, 1)
    g = torch.Generator().manual_seed(4)
    x, w, w13, dy = gpu(randn(g, N, k), randn(g, E, n, k), randn(g, E, 2 * F, k), randn(g, N, n))
    ws = cleared(shape)
    y = torch.full((N, n), 7.0, dtype=BF16, device="cuda")
    act = torch.full((N, F), 7.0, dtype=BF16, device="cuda")
    dw = torch.empty((E, n, k), device="cuda")
    for offs in ((-5, 10, 20, 48), (-3, -2, -1, 48), (-4, -3, -2, -1)):
        L = dict(expert_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda"))
        for call in (lambda: ep.ep_expert_matmul(shape, L, x, N, k, w, n, ep.EP_WEIGHT_NK, y, ws),
                     lambda: ep.ep_expert_swiglu(shape, L, x, N, w13, F, act, None, None, ws),
                     lambda: ep.ep_expert_wgrad(shape, L, dy, N, n, dict(x=x), k, dw, ep.EP_GRAD_F32, ws)):
            ep.ep_clear_errors(ws)
            call()
            assert ep.ep_check_errors(ws) == ep.EP_DEVERR_CAPACITY, offs
    assert (y == 7.0).all() and (act == 7.0).all()


def few_by_hand(x, w13, w2, F, T, weight=1.0):
    """ep_moe_few of one expert with the given (mostly zero) matrices."""
    H = x.shape[1]
    shape = ep.make_shape(T, H, 1, 1, 1)
    ws = ep.alloc_few_workspace(shape, F)
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    tokens = dict(x=x.cuda(), topk_idx=torch.zeros((T, 1), dtype=torch.int64, device="cuda"),
                  topk_weights=torch.full((T, 1), weight, device="cuda"))
    ep.ep_moe_few(shape, tokens, dict(F=F, w13=w13.cuda(), w2=w2.cuda()), out, ws)
    assert ep.ep_check_errors(ws) == 0
    return out.double().cpu()


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_few_inner_values_past_the_largest_bf16(sign, T):
    """gate = 2^64, up = +-(2^64 - 2^54): silu(gate) * up = +-2^128 (1 - 2^-10) is finite in
    32 bits and rounds to infinity in bf16; times 2^-100 it is 2^28 (1 - 2^-10), all powers
    and sums exact but the last rounding."""
    H, F = 16, 8
    x = torch.zeros((T, H), dtype=BF16)
    x[:, 0] = x[:, 1] = 2.0 ** 32
    w13, w2 = torch.zeros((1, 2 * F, H), dtype=BF16), torch.zeros((1, H, F), dtype=BF16)
    w13[0, 0, 0] = 2.0 ** 32
    w13[0, F, 0], w13[0, F, 1] = sign * 2.0 ** 32, -sign * 2.0 ** 22
    w2[0, :, 0] = 2.0 ** -100
    ref = torch.full((T, H), sign * 2.0 ** 28 * (1 - 2.0 ** -10), dtype=F64)
    # exp(-2^64) is 0: silu(gate) is exact; what the two bf16 values leave is 2^-16 of it.
    b = 2.0 ** -16 * ref.abs()
    check(few_by_hand(x, w13, w2, F, T), ref, b + HALF_BF16 * (ref.abs() + b), "out")


@pytest.mark.parametrize("F", [8, 264, 512])
def test_few_keeps_the_sign_of_infinite_second_weights(F):
    """One infinite W2 entry meets inner values that bf16 holds exactly (their rest is 0),
    and ones that it rounds up and down (their rest has either sign): the output is the
    infinity of the value's sign, as the sum's definition says; other outputs stay."""
    T, H = 11, 16
    g = torch.Generator().manual_seed(12)
    x = randn(g, T, H)
    x[:, 0] = 1.0
    w13, w2 = randn(g, 1, 2 * F, H, scale=H ** -0.5), randn(g, 1, H, F, scale=F ** -0.5)
    w13[0, 0], w13[0, F] = 0, 0
    w13[0, 0, 0], w13[0, F, 0] = 96.0, 0.5  # silu(96) * 0.5 = 48: no rest
    clean, bound = few_reference(x, w13, w2, torch.zeros((T, 1), dtype=torch.int64), torch.full((T, 1), 0.5), F)
    w2[0, 3, 0], w2[0, 4, F - 1], w2[0, 5, 2] = float("inf"), float("-inf"), float("inf")
    out = few_by_hand(x, w13, w2, F, T, weight=0.5)
    gu = x.double() @ w13[0].double().T
    act = silu_parts(gu, F)[3]
    assert (act[:, [0, 2, F - 1]].abs() > 1e-6).all()  # far from zero against the 32-bit sums' error
    for h, f, v in ((3, 0, 1.0), (4, F - 1, -1.0), (5, 2, 1.0)):
        assert torch.equal(out[:, h], v * torch.sign(act[:, f]) * float("inf")), h
    rest = [h for h in range(H) if h not in (3, 4, 5)]
    check(out[:, rest], clean[:, rest], bound[:, rest], "other outputs")


def test_swiglu_leaves_out_rows_past_the_capacity():
    E, H, F, N, have = 3, 64, 128, 50, 33
    g = torch.Generator().manual_seed(4)
    x, w13 = randn(g, have, H), randn(g, E, 2 * F, H, scale=H ** -0.5)
    off = torch.tensor([0, 20, 40, N], dtype=torch.int32)
    shape = ep.make_shape(N, H, 1, E, 1)
    ws = cleared(shape)
    act = torch.empty((have, F), dtype=BF16, device="cuda")
    xd, wd, od = gpu(x, w13, off)
    ep.ep_expert_swiglu(shape, dict(expert_offsets=od), xd, have, wd, F, act, None, None, ws)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_CAPACITY
    cut = off.clamp(max=have)
    gu = per_expert(cut, lambda e, s: x[s].double() @ w13[e].double().T, None)
    acc = H * U23 * per_expert(cut, lambda e, s: x[s].double().abs() @ w13[e].double().abs().T, None)
    gate, up, s, ref = silu_parts(gu, F)
    b = act_bound(gate, up, s, ref, acc[:, :F], acc[:, F:])
    check(act, ref, b + HALF_BF16 * (ref.abs() + b), "act")


def check_there(got, ref, bound, what):
    """check, on the device that holds the values (large results)."""
    over = (got.double() - ref).abs() - bound
    assert not torch.isnan(over).any(), f"{what}: NaN"
    assert (over <= 0).all(), f"{what}: {over.max().item():.3g} over its bound"


@pytest.mark.parametrize("save", [False, True], ids=["act", "checkpoint"])
def test_swiglu_more_tiles_than_workgroups(save):
    """Three tiles to a workgroup, of different heights and experts one after the other:
    the next tile's first steps arrive while block maxima and results are written."""
    counts = [(37 * e) % 290 for e in range(40)]
    H, F = 200, 2176 if save else 2184
    off, N, shape, ws = by_counts(counts, H)
    assert sum(-(-c // 256) for c in counts) * -(-F // 128) > 2 * 256
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((N, H), generator=g, device="cuda").to(BF16)
    w13 = (torch.randn((len(counts), 2 * F, H), generator=g, device="cuda") * H ** -0.5).to(BF16)
    act = torch.full((N, F), 7.0, dtype=BF16, device="cuda")
    q = torch.full((N, 2 * F), 0x55, dtype=U8, device="cuda") if save else None
    sc = torch.full((N, 2 * F // 128), 7.0, device="cuda") if save else None
    ep.ep_expert_swiglu(shape, dict(expert_offsets=off.cuda()), x, N, w13, F, act, q, sc, ws)
    assert ep.ep_check_errors(ws) == 0
    for e in range(len(counts)):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.stop == r.start:
            continue
        a, b = x[r].double(), w13[e].double()
        gu, acc = a @ b.T, H * U23 * (a.abs() @ b.abs().T)
        gate, up, s, ref = silu_parts(gu, F)
        d = act_bound(gate, up, s, ref, acc[:, :F], acc[:, F:])
        check_there(act[r], ref, d + HALF_BF16 * (ref.abs() + d), f"act of expert {e}")
        if save:
            m = gu.reshape(len(gu), -1, 128).abs().amax(2)
            check_there(sc[r], m / 448, acc.reshape(len(gu), -1, 128).amax(2) / 448 + 4 * U23 * m / 448, f"scales {e}")
            rep = sc[r].double().repeat_interleave(128, 1)
            by = acc + 4 * U23 * gu.abs()
            check_there(q[r].view(F8).double() * rep, gu, by + HALF_E4M3 * (gu.abs() + by) + 2.0 ** -10 * rep,
                        f"checkpoint of expert {e}")


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("fp8", [False, True], ids=["rows", "fp8rows"])
def test_wgrad_streams_over_many_tiles(fp8, wide):
    """Four tiles and more to a workgroup, each of another expert than the last: tiles of
    no rows, of one, two, three and more steps between two others, with and without edges."""
    counts = [0, 1, 0, 63, 64, 65, 128, 0, 0, 129, 192, 200, 5, 300, 0, 1, 256, 70, 10, 0] * 2
    off, N, shape, ws = by_counts(counts)
    E, n, k = len(counts), 1032, 1408
    assert E * -(-n // 256) * -(-k // 256) >= 4 * 256
    g = torch.Generator(device="cuda").manual_seed(7)
    dy = torch.randn((N, n), generator=g, device="cuda").to(BF16)
    if fp8:
        v = torch.randn((N, k), generator=g, device="cuda")
        sc = v.reshape(N, -1, 128).abs().amax(2) / 448
        q = (v / sc.repeat_interleave(128, 1)).to(F8)
        x, rows = q.double() * sc.double().repeat_interleave(128, 1), dict(x_fp8=q, x_scales=sc)
    else:
        xb = torch.randn((N, k), generator=g, device="cuda").to(BF16)
        x, rows = xb.double(), dict(x=xb)
    dw = torch.full((E, n, k), 7.0, dtype=F32 if wide else BF16, device="cuda")
    ep.ep_expert_wgrad(shape, dict(expert_offsets=off.cuda()), dy, N, n, rows, k, dw,
                       ep.EP_GRAD_F32 if wide else ep.EP_GRAD_BF16, ws)
    assert ep.ep_check_errors(ws) == 0
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        a, b = dy[r].double(), x[r]
        ref, mag = a.T @ b, a.abs().T @ b.abs()
        acc = counts[e] * U23 * mag + (HALF_BF16 * mag * (1 + counts[e] * U23) + U23 * mag if fp8 else 0)
        check_there(dw[e], ref, acc if wide else acc + HALF_BF16 * (ref.abs() + acc), f"dw of expert {e}")


@pytest.mark.parametrize("how", ["none", "default", "null", "object", "handle"])
def test_calls_take_a_stream(how):
    """No stream, the default one, and another as torch's object or its handle."""
    T, H, F, E, K = 16, 128, 128, 4, 2
    idx, w, x, _, w13, w2 = gpu(*layer_case(T, H, F, E, K))
    shape = ep.make_shape(T, H, K, E, 1)
    tokens, experts = dict(x=x, topk_idx=idx, topk_weights=w), dict(F=F, w13=w13, w2=w2)
    ref = torch.empty((T, H), dtype=BF16, device="cuda")
    ep.ep_moe_few(shape, tokens, experts, ref, ep.alloc_few_workspace(shape, F))
    out, ws = torch.zeros_like(ref), ep.alloc_few_workspace(shape, F)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    stream = dict(none=None, default=torch.cuda.default_stream(), null=0, object=st, handle=st.cuda_stream)[how]
    ep.ep_moe_few(shape, tokens, experts, out, ws, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


MOST = 1 << 20  # EP_MAX_DIM


def device_randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(BF16)


@pytest.mark.parametrize("k,n", [(MOST, 8), (8, MOST), (MOST - 8, 264), (264, MOST - 8)])
def test_products_at_the_largest_dimensions(k, n):
    """Both weight orders and the weight gradient; rows of two experts around an empty one."""
    off = torch.tensor([0, 3, 3, 5], dtype=torch.int32, device="cuda")
    N, E = 5, 3
    shape = ep.make_shape(N, 128, 1, E, 1)
    ws = cleared(shape)
    L = dict(expert_offsets=off)
    x, w = device_randn(1, N, k), device_randn(2, E, n, k, scale=k ** -0.5)
    y = torch.full((N, n), 7.0, dtype=BF16, device="cuda")
    for order in (ep.EP_WEIGHT_NK, ep.EP_WEIGHT_KN):
        wt = w if order == ep.EP_WEIGHT_NK else w.transpose(1, 2).contiguous()
        ep.ep_expert_matmul(shape, L, x, N, k, wt, n, order, y, ws)
        for e, r in ((0, slice(0, 3)), (2, slice(3, 5))):
            a, b = x[r].double(), w[e].double()
            ref, acc = a @ b.T, k * U23 * (a.abs() @ b.abs().T)
            check_there(y[r], ref, acc + HALF_BF16 * (ref.abs() + acc), f"y of expert {e}, order {order}")
    dw = torch.full((E, n, k), 7.0, device="cuda")
    ep.ep_expert_wgrad(shape, L, y, N, n, dict(x=x), k, dw, ep.EP_GRAD_F32, ws)
    for e, r in ((0, slice(0, 3)), (1, slice(0, 0)), (2, slice(3, 5))):
        a, b = y[r].double(), x[r].double()
        check_there(dw[e], a.T @ b, 3 * U23 * (a.abs().T @ b.abs()), f"dw of expert {e}")
    assert ep.ep_check_errors(ws) == 0


@pytest.mark.parametrize("H,F", [(MOST, 8), (8, MOST), (8192, 65528)])
def test_swiglu_at_the_largest_dimensions(H, F):
    """The last is the largest matrix of one expert: 4 F H just below 2^31 - 16."""
    N, E = 3, 1
    shape = ep.make_shape(N, H, 1, E, 1)
    ws = cleared(shape)
    x, w13 = device_randn(1, N, H), device_randn(2, E, 2 * F, H, scale=H ** -0.5)
    act = torch.full((N, F), 7.0, dtype=BF16, device="cuda")
    off = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    ep.ep_expert_swiglu(shape, dict(expert_offsets=off), x, N, w13, F, act, None, None, ws)
    assert ep.ep_check_errors(ws) == 0
    xd = x.double()
    for lo in range(0, F, 1 << 14):
        hi = min(F, lo + (1 << 14))
        w = torch.cat([w13[0, lo:hi], w13[0, F + lo:F + hi]]).double()
        gu, acc = xd @ w.T, H * U23 * (xd.abs() @ w.abs().T)
        m = hi - lo
        gate, up, s, ref = silu_parts(gu, m)
        b = act_bound(gate, up, s, ref, acc[:, :m], acc[:, m:])
        check_there(act[:, lo:hi], ref, b + HALF_BF16 * (ref.abs() + b), f"act from {lo}")


def test_swiglu_grad_at_the_largest_dimension():
    F, T = MOST, 2
    shape = ep.make_shape(T, 128, 1, 1, 1)
    ws = cleared(shape)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((T, 2 * F), generator=g, device="cuda").to(F8)
    sc = torch.rand((T, 2 * F // 128), generator=g, device="cuda") + 0.5
    d, w = device_randn(4, T, F), torch.tensor([[0.5], [-0.25]], device="cuda")
    slot = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    d_gu, act_w = torch.empty((T, 2 * F), dtype=BF16, device="cuda"), torch.empty((T, F), dtype=BF16, device="cuda")
    d_w = torch.empty((T, 1), device="cuda")
    ep.ep_swiglu_grad(shape, dict(expert_slot=slot), F, q, sc, d, T, w, d_gu, act_w, d_w, ws)
    assert ep.ep_check_errors(ws) == 0
    gate, up, s, act = silu_parts(q.double() * sc.double().repeat_interleave(128, 1), F)
    row_w, dd, rel = w.flip(0).double(), d.double(), (gate.abs() + 24) * U23
    ref = torch.cat([row_w * dd * up * s * (1 + gate * (1 - s)), row_w * dd * gate * s], 1)
    b = torch.cat([(row_w * dd * up * s).abs() * (1 + gate.abs()) * rel, ref[:, F:].abs() * rel], 1)
    check_there(d_gu, ref, b + HALF_BF16 * (ref.abs() + b), "d_gu")
    ref = row_w * act
    check_there(act_w, ref, ref.abs() * rel + HALF_BF16 * ref.abs() * (1 + rel), "act_w")
    # A lane's partial sums hold F / 64 terms each, six more join them.
    each = (dd * act).abs()
    check_there(d_w.flip(0)[:, 0], (dd * act).sum(1), (each * (rel + (F // 64 + 8) * U23)).sum(1), "d_topk_weights")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,F", [(MOST, 8), (8, MOST)])
def test_few_at_the_largest_dimensions(H, F, fp8):
    T, K, E = 3, 2, 2
    if fp8:
        H, F = max(H, 128), max(F, 128)
    x = device_randn(1, T, H)
    w13, w2 = device_randn(2, E, 2 * F, H, scale=H ** -0.5), device_randn(3, E, H, F, scale=F ** -0.5)
    idx = torch.tensor([[0, 1], [1, -1], [0, 0]])
    w = torch.tensor([[0.5, -0.5], [1.0, 3.0], [0.25, 0.5]])
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_few_workspace(shape, F).fill_(0xAB)
    ep.ep_clear_errors(ws)
    if fp8:
        (q13, s13, w13), (q2, s2, w2) = eight(w13), eight(w2)
        experts = dict(F=F, w13_fp8=q13, w13_scales=s13, w2_fp8=q2, w2_scales=s2)
    else:
        experts = dict(F=F, w13=w13, w2=w2)
    out = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    ep.ep_moe_few(shape, dict(x=x, topk_idx=idx.cuda(), topk_weights=w.cuda()), experts, out, ws)
    assert ep.ep_check_errors(ws) == 0
    ref, bound = few_reference(x.cpu(), w13.cpu(), w2.cpu(), idx, w, F)
    check(out, ref, bound, "out")


def test_few_with_most_lanes_and_experts():
    """128 tokens of 64 lanes over 4,096 experts: 8,192 lanes, most experts used."""
    T, K, E, H, F = 128, 64, 4096, 24, 16
    g = torch.Generator().manual_seed(9)
    idx, w = routing(T, K, E, 17)
    x, w13, w2 = randn(g, T, H), randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5)
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_few_workspace(shape, F).fill_(0xAB)
    ep.ep_clear_errors(ws)
    out = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    ep.ep_moe_few(shape, dict(x=x.cuda(), topk_idx=idx.cuda(), topk_weights=w.cuda()),
                  dict(F=F, w13=w13.cuda(), w2=w2.cuda()), out, ws)
    assert ep.ep_check_errors(ws) == 0
    ref, bound = few_reference(x, w13, w2, idx, w, F)
    # few_reference allows 80 sums of experts' parts; these tokens have 64 each: enough.
    check(out, ref, bound, "out")


@pytest.mark.parametrize("F", [128, 2056])
def test_few_without_any_lane(F):
    """All lanes skipped, or of ids that 32 bits would take for valid ones: zeros, and for the
    latter the error (F: with and without shared outputs)."""
    T, H, E, K = 9, 264, 4, 3
    x, w13, w2 = device_randn(1, T, H), device_randn(2, E, 2 * F, H), device_randn(3, E, H, F)
    w = torch.full((T, K), float("nan"), device="cuda")
    shape = ep.make_shape(T, H, K, E, 1)
    ws = ep.alloc_few_workspace(shape, F).fill_(0xAB)
    for ident, want in ((-1, 0), ((1 << 32) + 1, ep.EP_DEVERR_EXPERT_ID), (-(1 << 32), ep.EP_DEVERR_EXPERT_ID)):
        ep.ep_clear_errors(ws)
        out = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
        ep.ep_moe_few(shape, dict(x=x, topk_idx=torch.full((T, K), ident, device="cuda"), topk_weights=w),
                      dict(F=F, w13=w13, w2=w2), out, ws)
        assert ep.ep_check_errors(ws) == want
        assert (out == 0).all()
