"""The few-token layer with 4-bit weights (ep_moe_few_w4) against plain 64-bit
arithmetic on the values that codes and scales stand for, and the layers that
the norm, the router and the expert operators make together.

Tolerances as in test_experts_gpu.py: a sum of n products in 32 bits is off by
at most n * 2^-23 of the sum of their magnitudes. EP_W4_INT's magnitudes are taken
as x * (code + 8) * scale, which is more than the x * |code - 8| * scale that it sums.
"""
import pytest
import torch

from combine_get_layout_amd import ep
from test_experts_gpu import (BF16, F32, F64, HALF_BF16, HALF_E4M3, U8, U23, act_bound, check, cleared, gpu, randn, routing,
                              silu_parts)

pytestmark = pytest.mark.gpu

INT, E2M1 = 0, 1
TABLE = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=F64)
FORMS = pytest.mark.parametrize("form", [INT, E2M1], ids=["int", "e2m1"])


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.lib()


def values(code, scales, form):
    """The values, and the magnitudes that enter the sums, of [..., n, k / 2] packed codes."""
    c = torch.stack([code & 15, code >> 4], -1).flatten(-2).long()
    if form == INT:
        s = scales.double().repeat_interleave(128, -1)
        return (c - 8).double() * s, (c + 8).double() * s.abs()
    v = TABLE.to(c.device)[c] * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)
    return v, v.abs()


def four(g, E, n, k, form, spread=3):
    """Random codes and scales of matrices that keep a vector's size."""
    code = torch.randint(0, 256, (E, n, k // 2), generator=g).to(U8)
    if form == INT:
        s = (torch.rand((E, n, k // 128), generator=g) + 0.5) * (k ** -0.5 / 4.6)
        s *= torch.where(torch.rand(s.shape, generator=g) < 0.3, -1.0, 1.0)
        return code, s.to(BF16)
    mid = 127 - round(torch.tensor(k ** 0.5 * 3).log2().item())
    return code, torch.randint(mid - spread, mid + spread, (E, n, k // 32), generator=g).to(U8)


def few_reference(x, w13, w2, idx, w, F, form):
    """out and its bound in 64 bits; w13, w2: (codes, scales)."""
    T, H = x.shape
    out, bound = torch.zeros((T, H), dtype=F64), torch.zeros((T, H), dtype=F64)
    xd = x.double()
    for e in range(len(w13[0])):
        hit = (idx == e)
        ts = hit.any(1).nonzero()[:, 0]
        if not len(ts):
            continue
        (a, am), (b2, bm) = values(w13[0][e], w13[1][e], form), values(w2[0][e], w2[1][e], form)
        gu = xd[ts] @ a.T
        acc = H * U23 * (xd[ts].abs() @ am.T)
        gate, up, s, act = silu_parts(gu, F)
        da = act_bound(gate, up, s, act, acc[:, :F], acc[:, F:])
        da = da + 2.0 ** -16 * (act.abs() + da)  # two bf16 values: the rest is rounded, 2^-8 of 2^-8
        we = (w.double() * hit).sum(1)[ts].unsqueeze(1)
        wabs = (w.double().abs() * hit).sum(1)[ts].unsqueeze(1)
        out[ts] += we * (act @ b2.T)
        mag = (act.abs() + da) @ bm.T
        bound[ts] += wabs * (da @ b2.abs().T + F * U23 * mag) + 80 * U23 * wabs * mag
    bound = bound + 8 * U23 * out.abs()
    return out, bound + HALF_BF16 * (out.abs() + bound)


def experts(w13, w2, F, form):
    return dict(F=F, form=form, w13=w13[0].cuda(), w13_scales=w13[1].cuda(), w2=w2[0].cuda(), w2_scales=w2[1].cuda())


def few_call(x, idx, w, X, E, ws=None, out=None):
    T, H = x.shape
    shape = ep.make_shape(T, H, idx.shape[1], E, 1)
    if ws is None:
        ws = ep.alloc_few_w4_workspace(shape, X["F"]).fill_(0xAB)
        ep.ep_clear_errors(ws)
    if out is None:
        out = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    ep.ep_moe_few_w4(shape, dict(x=x.cuda(), topk_idx=idx.cuda(), topk_weights=w.cuda()), X, out, ws)
    return out, ws


FEW = [
    # (T, H, F, E, K, options): sizes in steps of 32 (of 128 for integers)
    (1, 256, 512, 16, 2, {}),
    (1, 32, 32, 1, 1, {}),
    (2, 96, 64, 3, 2, {}),
    (13, 288, 160, 40, 3, dict(skip=0.2)),
    (16, 640, 384, 8, 8, {}),
    (17, 128, 256, 5, 4, dict(repeat=True)),
    (33, 224, 288, 4, 2, {}),
    (128, 160, 96, 2, 1, {}),            # 64 tokens and more to one expert
    (36, 128, 128, 1, 1, {}),            # three token tiles of one expert
    (128, 128, 128, 1024, 4, {}),        # many experts
    (100, 64, 96, 3, 64, dict(repeat=True)),
    (5, 1056, 736, 6, 6, {}),
    (103, 512, 1024, 10, 8, {}),         # workgroups that share outputs, many tokens to each expert
    (32, 1024, 512, 12, 5, {}),
    (9, 2080, 544, 7, 2, {}),
    (65, 1312, 672, 30, 6, dict(skip=0.1)),
]


def few_case(case, form):
    T, H, F, E, K, opt = case
    if form == INT:
        H, F = -(-H // 128) * 128, -(-F // 128) * 128
    g = torch.Generator().manual_seed(9)
    idx, w = routing(T, K, E, 17, **opt)
    return H, F, randn(g, T, H), idx, w, four(g, E, 2 * F, H, form), four(g, E, H, F, form)


@FORMS
@pytest.mark.parametrize("case", FEW, ids=str)
def test_few_w4(case, form):
    H, F, x, idx, w, w13, w2 = few_case(case, form)
    X = experts(w13, w2, F, form)
    out, ws = few_call(x, idx, w, X, case[3])
    assert ep.ep_check_errors(ws) == 0
    ref, bound = few_reference(x, w13, w2, idx, w, F, form)
    check(out, ref, bound, "out")
    again, _ = few_call(x, idx, w, X, case[3], ws=ws)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@FORMS
def test_few_w4_every_code(form):
    """Identity inputs read each weight back: every code at every place of a row, exactly."""
    H, F = 256, 128
    T = 64
    code13 = torch.zeros((1, 2 * F, H // 2), dtype=U8)
    r, c = torch.arange(2 * F).unsqueeze(1), torch.arange(H)
    full = (r + c + c // 16).remainder(16).to(U8)
    code13[0] = full[:, 0::2] | full[:, 1::2] << 4
    s13 = torch.ones((1, 2 * F, H // 128)).to(BF16) if form == INT else torch.full((1, 2 * F, H // 32), 127).to(U8)
    v13 = values(code13, s13, form)[0][0]
    # Gate rows of +8 and more saturate; compare the first product through up rows only: gate = 64.
    code13[0, :F] = 0x88 if form == INT else 0
    code2 = torch.zeros((1, H, F // 2), dtype=U8)
    one = 9 if form == INT else 2  # the code of 1
    eight = torch.full((F // 2,), 0x88 if form == INT else 0, dtype=torch.long)
    for h in range(F):
        row = eight.clone()
        row[h // 2] = (row[h // 2] & (0xF0 if h % 2 == 0 else 0x0F)) | one << (4 * (h % 2))
        code2[0, h] = row.to(U8)
    code2[0, F:] = 0x88 if form == INT else 0
    s2 = torch.ones((1, H, F // 128)).to(BF16) if form == INT else torch.full((1, H, F // 32), 127).to(U8)
    # The last column carries the gate: x = e_t + 64 e_last, gate rows have 1 there; t < 255.
    code13[0, :F, -1] = (code13[0, :F, -1] & 0x0F) | one << 4
    v13 = values(code13, s13, form)[0][0]
    for t0 in range(0, H - 1, T):
        n = min(T, H - 1 - t0)
        x = torch.zeros((n, H))
        x[torch.arange(n), t0 + torch.arange(n)] = 1.0
        x[:, -1] = 64.0
        x = x.to(BF16)
        out, ws = few_call(x, torch.zeros((n, 1), dtype=torch.int64), torch.ones((n, 1)),
                           experts((code13, s13), (code2, s2), F, form), 1)
        gu = x.double() @ v13.T
        assert (gu[:, :F] == 64).all()  # silu(64) = 64 in 32 bits
        ref = 64 * gu[:, F:]            # exact in 32 bits; one rounding to bf16
        check(out[:, :F], ref, HALF_BF16 * ref.abs() + 4 * U23 * ref.abs(), "weights read back")
        assert (out[:, F:] == 0).all()


def test_few_w4_scales_of_all_sizes():
    """Powers of two from 2^-127 to 2^60 and NaN (255), in the second matrix, one row each."""
    T, H, F = 3, 256, 32
    g = torch.Generator().manual_seed(3)
    x, w13 = randn(g, T, H), four(g, 1, 2 * F, H, E2M1)
    code2 = torch.randint(0, 256, (1, H, F // 2), generator=g).to(U8)
    s2 = torch.arange(H).clamp(max=187).to(U8).reshape(1, H, 1).clone()
    s2[0, 200] = 255
    idx, w = torch.zeros((T, 1), dtype=torch.int64), torch.ones((T, 1))
    out, _ = few_call(x, idx, w, experts(w13, (code2, s2), F, E2M1), 1)
    assert torch.isnan(out[:, 200]).all()
    keep = [h for h in range(H) if h != 200]
    ref, bound = few_reference(x, w13, (code2, torch.where(s2 == 255, 127, s2.long()).to(U8)), idx, w, F, E2M1)
    # Below 2^-126 products and sums lose bits: a step of 2^-149 each.
    check(out[:, keep].double(), ref[:, keep], bound[:, keep] + F * 2.0 ** -133 * 64, "out")


@FORMS
def test_few_w4_keeps_nonfinite_values_with_their_tokens(form):
    """A NaN scale of one expert, NaN and infinite inputs reach only their own tokens; bad ids are
    reported and skipped; a token without a lane gets zeros."""
    T, H, F, E, K = 6, 128, 256, 4, 2
    g = torch.Generator().manual_seed(2)
    x, w13, w2 = randn(g, T, H), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    idx = torch.tensor([[0, 1], [1, 2], [-1, -1], [3, 0], [0, 99], [-7, 1]])
    w = torch.full((T, K), 0.5)
    clean = torch.where((idx < 0) | (idx >= E), -1, idx)
    ref, bound = few_reference(x, w13, w2, clean, w, F, form)
    bad13, bad2, badx = (w13[0], w13[1].clone()), (w2[0], w2[1].clone()), x.clone()
    bad13[1][2, 3, 0] = float("nan") if form == INT else 255  # expert 2: token 1 only
    bad2[1][3] = float("nan") if form == INT else 255         # expert 3: token 3 only
    badx[4] = float("nan")                                    # token 4 only
    out, ws = few_call(badx, idx, w, experts(bad13, bad2, F, form), E)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_EXPERT_ID
    for t in (0, 2, 5):
        check(out[t], ref[t], bound[t], f"token {t}")
    assert (out[2] == 0).all()
    assert torch.isnan(out[3]).all() and torch.isnan(out[4]).all() and torch.isnan(out[1]).all()


@FORMS
@pytest.mark.parametrize("F", [256, 2560])
def test_few_w4_keeps_nonfinite_values_among_many_tokens(form, F):
    """The same where an expert's tokens are multiplied in tiles of 16 and more."""
    copies, H, E, K = 16, 128, 4, 2
    g = torch.Generator().manual_seed(22)
    T = 6 * copies
    x, w13, w2 = randn(g, T, H), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    idx = torch.tensor([[0, 1], [1, 2], [-1, -1], [3, 0], [0, 99], [-7, 1]]).repeat(copies, 1)
    w = torch.full((T, K), 0.5)
    clean = torch.where((idx < 0) | (idx >= E), -1, idx)
    ref, bound = few_reference(x, w13, w2, clean, w, F, form)
    bad13, bad2, badx = (w13[0], w13[1].clone()), (w2[0], w2[1].clone()), x.clone()
    bad13[1][2, 3, 0] = float("nan") if form == INT else 255
    bad2[1][3] = float("nan") if form == INT else 255
    badx[4::6] = float("nan")
    out, ws = few_call(badx, idx, w, experts(bad13, bad2, F, form), E)
    assert ep.ep_check_errors(ws) == ep.EP_DEVERR_EXPERT_ID
    for t in (0, 2, 5):
        check(out[t::6], ref[t::6], bound[t::6], f"tokens {t}, {t + 6}, ...")
    assert (out[2::6] == 0).all()
    for t in (1, 3, 4):
        assert torch.isnan(out[t::6]).all()


@pytest.mark.parametrize("H,F", [(128, 128), (640, 384), (256, 1152)])
def test_few_w4_keeps_the_sign_of_infinite_scales(H, F):
    """An infinite scale of the second matrix makes an infinity of its block's sum's sign (sums far
    from zero), and none of a NaN where a row's columns or the steps behind its end have no value."""
    T = 5
    g = torch.Generator().manual_seed(14)
    x, w13, w2 = randn(g, T, H), four(g, 1, 2 * F, H, INT), four(g, 1, H, F, INT)
    w2[1][0, 3, 0] = float("inf")
    w2[1][0, 7, F // 128 - 1] = float("-inf")
    idx, w = torch.zeros((T, 1), dtype=torch.int64), torch.full((T, 1), 0.5)
    out, _ = few_call(x, idx, w, experts(w13, w2, F, INT), 1)
    finite = (w2[0], torch.where(torch.isfinite(w2[1]), w2[1], torch.ones((), dtype=BF16)))
    act = silu_parts(x.double() @ values(w13[0][0], w13[1][0], INT)[0].T, F)[3]
    codes, mags = values(finite[0][0], torch.ones_like(finite[1][0]), INT)
    for h, block, sign in ((3, 0, 1.0), (7, F // 128 - 1, -1.0)):
        cut = slice(block * 128, block * 128 + 128)
        part = act[:, cut] @ codes[h, cut]
        sure = part.abs() > 1e-3 * (act[:, cut].abs() @ mags[h, cut])
        assert sure.any()
        assert torch.equal(out[sure.cuda(), h].cpu().double(), sign * torch.sign(part[sure]) * float("inf")), h
    keep = [h for h in range(H) if h not in (3, 7)]
    ref, bound = few_reference(x, w13, finite, idx, w, F, INT)
    check(out[:, keep], ref[:, keep], bound[:, keep], "other outputs")


def by_power(m, form, rows=slice(None), power=0):
    """(codes, scales) with the scales of some rows times 2^power, exactly."""
    sc = m[1].clone()
    sc[:, rows] = (sc[:, rows].double() * 2.0 ** power).to(BF16) if form == INT else (sc[:, rows].int() + power).to(U8)
    return m[0], sc


def set_codes(code, e, rows, cols, values):
    """The codes of some rows and columns of expert e."""
    full = torch.stack([code[e] & 15, code[e] >> 4], -1).flatten(-2)
    full[rows, cols] = torch.as_tensor(values, dtype=U8)
    code[e] = full[:, 0::2] | full[:, 1::2] << 4


# (T, F, E, K): each launch's forms for one token, for few and for many tokens an expert.
EXTREME = [(1, 256, 1, 1), (5, 384, 2, 1), (64, 1024, 16, 2), (96, 256, 1, 1), (128, 256, 24, 5)]


def extreme_values(case, form):
    T, F, E, K = case
    H = 256
    g = torch.Generator().manual_seed(31)
    x, w13, w2 = randn(g, T, H), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    idx, w = routing(T, K, E, 17)
    up, most = slice(F, None), 122 if form == INT else 119
    return idx, w, dict(inputs=(x * 2.0 ** 124, by_power(w13, form, power=-116), w2),
                        inner=(x, by_power(w13, form, up, most), by_power(w2, form, power=-114)),
                        small=(x * 2.0 ** -104, by_power(w13, form, power=100), w2))


@FORMS
@pytest.mark.parametrize("case", EXTREME, ids=str)
def test_few_w4_of_large_and_small_finite_values(case, form):
    """Inputs, then inner values, close to bf16's largest (sums of eight of them pass 32 bits), and inputs of
    2^-104, whose scales bring the results back to common sizes: the same bounds as for common inputs."""
    F, E = case[1:3]
    idx, w, cases = extreme_values(case, form)
    for name, (x, w13, w2) in cases.items():
        assert torch.isfinite(x).all()
        ref, bound = few_reference(x, w13, w2, idx, w, F, form)
        out, ws = few_call(x, idx, w, experts(w13, w2, F, form), E)
        assert ep.ep_check_errors(ws) == 0
        check(out, ref, bound, name)


@FORMS
@pytest.mark.parametrize("case", EXTREME, ids=str)
def test_few_w4_keeps_the_sign_of_infinite_inputs(case, form):
    """An infinite input makes infinite inner values, and outputs of the sign that the values give; tokens
    of finite inputs keep theirs."""
    T, F, E, K = case
    H = 256
    g = torch.Generator().manual_seed(32)
    x, w13, w2 = randn(g, T, H), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    idx, w = routing(T, K, E, 17)
    w = w.abs() + 0.1
    plus, minus = (11, 2) if form == INT else (3, 12)
    w13, w2 = (w13[0], w13[1].abs()), (w2[0], w2[1].abs())
    x[0::2, 77] = float("inf")
    sign = torch.where(torch.arange(H) % 2 == 0, 1.0, -1.0)
    for e in range(E):  # each gate and up is +infinity, each output's weights have one sign
        set_codes(w13[0], e, slice(None), 77, plus)
        set_codes(w2[0], e, slice(None), slice(None), torch.where(sign > 0, plus, minus).unsqueeze(1).expand(H, F))
    out, _ = few_call(x, idx, w, experts(w13, w2, F, form), E)
    assert torch.equal(out[0::2].float().cpu(), (sign * float("inf")).expand(len(out[0::2]), H))
    ref, bound = few_reference(x[1::2], w13, w2, idx[1::2], w[1::2], F, form)
    check(out[1::2], ref, bound, "tokens of finite inputs")


@FORMS
@pytest.mark.parametrize("case", EXTREME, ids=str)
def test_few_w4_keeps_the_sign_of_infinite_inner_values(case, form):
    """Finite inputs and weights whose inner value 77 passes 32 bits, to +infinity in even experts and
    -infinity in odd ones: outputs of its sign times the weight's, NaN where the weight is 0 or the token
    has experts of both kinds."""
    T, F, E, K = case
    H, at = 256, 77
    g = torch.Generator().manual_seed(33)
    x, w13, w2 = randn(g, T, H).abs(), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    idx, w = routing(T, K, E, 17)
    w = w.abs() + 0.1
    zero, plus, minus = (8, 11, 2) if form == INT else (0, 3, 12)
    w13, w2 = (w13[0], w13[1].abs()), (w2[0], w2[1].abs())
    w13 = by_power(w13, form, slice(F + at, F + at + 1), 130 if form == INT else 127)
    pick = torch.arange(H) % 3
    for e in range(E):
        set_codes(w13[0], e, at, slice(None), plus)
        set_codes(w13[0], e, F + at, slice(None), plus if e % 2 == 0 else minus)
        set_codes(w2[0], e, slice(None), at, torch.tensor([plus, minus, zero])[pick])
        for m in (w13, w2):
            assert torch.isfinite(values(m[0][e], m[1][e], form)[0].to(BF16)).all()
    out = few_call(x, idx, w, experts(w13, w2, F, form), E)[0].float().cpu()
    for t in range(T):
        kinds = {e % 2 for e in idx[t].tolist()}
        if len(kinds) == 2:
            assert torch.isnan(out[t]).all(), t
            continue
        inf = -float("inf") if kinds == {1} else float("inf")
        assert (out[t, pick == 0] == inf).all() and (out[t, pick == 1] == -inf).all(), t
        assert torch.isnan(out[t, pick == 2]).all(), t


@FORMS
@pytest.mark.parametrize("case", [(1, 32, 32, 1, 1, {}), (1, 288, 160, 2, 2, {}), (3, 96, 416, 4, 1, {})], ids=str)
def test_few_w4_scales_at_the_end_of_their_memory(case, form):
    """The shortest rows of scales, which end where their memory does: a workgroup asks for whole vectors of
    more rows than there are, and takes none of what lies behind the array. The same results as with each
    array in the middle of other values."""
    H, F, x, idx, w, w13, w2 = few_case(case, form)
    X = experts(w13, w2, F, form)
    out, _ = few_call(x, idx, w, X, case[3])
    for name in ("w13_scales", "w2_scales"):
        around = torch.full((1 << 16,), 0x7F, dtype=U8, device="cuda")
        raw = X[name].view(U8).flatten()
        last, middle = around.clone(), around.clone()
        last[len(last) - len(raw):], middle[4096:4096 + len(raw)] = raw, raw
        for t, at in ((last, len(last) - len(raw)), (middle, 4096)):
            again, _ = few_call(x, idx, w, dict(X, **{name: t[at:at + len(raw)]}), case[3])
            assert torch.equal(again.view(torch.int16), out.view(torch.int16)), name


@FORMS
@pytest.mark.parametrize("F", [128, 2048])
def test_few_w4_without_any_lane(form, F):
    """All lanes skipped, or of ids that 32 bits would take for valid ones: zeros, and for the latter
    the error (F: with and without shared outputs)."""
    T, H, E, K = 9, 256, 4, 3
    g = torch.Generator().manual_seed(1)
    X = experts(four(g, E, 2 * F, H, form), four(g, E, H, F, form), F, form)
    w = torch.full((T, K), float("nan"))
    for ident, want in ((-1, 0), ((1 << 32) + 1, ep.EP_DEVERR_EXPERT_ID), (-(1 << 32), ep.EP_DEVERR_EXPERT_ID)):
        out, ws = few_call(randn(g, T, H), torch.full((T, K), ident), w, X, E)
        assert ep.ep_check_errors(ws) == want
        assert (out == 0).all()


@FORMS
def test_few_w4_with_most_lanes_and_experts(form):
    """128 tokens of 64 lanes over 4,096 experts: 8,192 lanes, most experts used."""
    T, K, E = 128, 64, 4096
    H, F = (128, 128) if form == INT else (32, 64)
    g = torch.Generator().manual_seed(9)
    idx, w = routing(T, K, E, 17)
    x, w13, w2 = randn(g, T, H), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    out, ws = few_call(x, idx, w, experts(w13, w2, F, form), E)
    assert ep.ep_check_errors(ws) == 0
    ref, bound = few_reference(x, w13, w2, idx, w, F, form)
    check(out, ref, bound, "out")


@FORMS
@pytest.mark.parametrize("case", [(64, 256, 896, 12, 8, {}), (36, 384, 480, 20, 16, dict(skip=0.1)),
                                  (40, 128, 672, 48, 10, {}), (128, 1024, 2080, 5, 5, {})], ids=str)
def test_few_w4_many_tokens_an_expert(case, form):
    """16, 32, 64 and 128 tokens of an expert at a time, and what is left of them."""
    test_few_w4(case, form)


@FORMS
@pytest.mark.parametrize("case", [(1, 512, 16384, 1, 5, dict(repeat=True)), (2, 1056, 8224, 2, 5, dict(repeat=True)),
                                  (3, 1312, 5472, 3, 6, dict(repeat=True)), (4, 1024, 4096, 4, 8, dict(repeat=True)),
                                  (4, 512, 8192, 4, 8, dict(repeat=True)), (1, 256, 6144, 1, 64, dict(repeat=True))], ids=str)
def test_few_w4_of_few_tokens_whose_lanes_repeat_experts(case, form):
    """One to four tokens with more than four lanes an expert, which take the first launch's forms of 32 and
    64 values of f to a workgroup; rows of one to three steps a wave, F that fills no tile of 32."""
    test_few_w4(case, form)


@FORMS
@pytest.mark.parametrize("case", [(8, 256, 2080, 8, 5, {}), (7, 2336, 3296, 5, 4, {}), (64, 256, 1024, 16, 2, {}),
                                  (20, 256, 1056, 16, 4, {}), (24, 1312, 864, 20, 6, dict(skip=0.1)),
                                  (24, 1312, 864, 20, 7, {}), (40, 544, 672, 25, 5, dict(repeat=True))], ids=str)
def test_few_w4_32_columns_a_workgroup(case, form):
    """Four to eight lanes an expert, for 8 and for 16 tokens at a time: the first launch's form of 32 values
    of f to a workgroup, tiles that F fills in part, rows of one to three steps a wave; and, with the last but
    one, the form for many tokens beside it."""
    test_few_w4(case, form)


@FORMS
@pytest.mark.parametrize("case", [(1, 1024, 8192, 4, 4, {}), (3, 256, 2080, 16, 6, {}), (4, 1056, 1024, 32, 8, {}),
                                  (5, 2048, 1056, 32, 8, {}), (12, 2080, 1056, 32, 3, dict(skip=0.1)),
                                  (17, 96, 1056, 40, 2, {})], ids=str)
def test_few_w4_short_rows(case, form):
    """One to a few tokens an expert in the first launch's form for many, on both sides of the row lengths
    that take it."""
    test_few_w4(case, form)


@FORMS
@pytest.mark.parametrize("case", [(32, 160, 2048, 33, 4, {}), (32, 160, 4192, 16, 4, {}), (9, 224, 2336, 30, 4, dict(skip=0.1)),
                                  (2, 96, 2048, 128, 64, {}), (1, 544, 4192, 40, 16, {})], ids=str)
def test_few_w4_64_columns_of_the_second_launch(case, form):
    """256 units of 256 values of f and more: the second launch's form of 64 outputs to a workgroup, which H
    fills in part, with scales in LDS and from memory."""
    test_few_w4(case, form)


@FORMS
def test_few_w4_many_tokens_of_the_longest_rows_in_lds(form):
    """Scales of 512 bytes a row in LDS, beside 128 tokens' rows."""
    T, H, F, E, K = 128, 16384 if form == E2M1 else 32768, 128, 80, 40
    g = torch.Generator().manual_seed(19)
    some = [four(g, 4, n, k, form) for n, k in ((2 * F, H), (H, F))]
    w13, w2 = [tuple(t.repeat(E // 4, 1, 1) for t in m) for m in some]
    x = randn(g, T, H)
    idx, w = routing(T, K, E, 18)
    out, ws = few_call(x, idx, w, experts(w13, w2, F, form), E)
    assert ep.ep_check_errors(ws) == 0
    # A sample of the tokens: each is a sum of its own.
    at = torch.arange(0, T, 17)
    ref, bound = few_reference(x[at], w13, w2, idx[at], w[at], F, form)
    check(out.cpu()[at], ref, bound, "out")


@FORMS
@pytest.mark.parametrize("wide", ["H", "F"])
def test_few_w4_at_the_largest_dimensions(form, wide):
    small = 128 if form == INT else 32
    H, F = (1 << 20, small) if wide == "H" else (small, 1 << 20)
    T, K, E = 3, 2, 2
    g = torch.Generator().manual_seed(5)
    idx = torch.tensor([[0, 1], [1, -1], [0, 0]])
    w = torch.tensor([[0.5, -0.5], [1.0, 3.0], [0.25, 0.5]])
    x, w13, w2 = randn(g, T, H), four(g, E, 2 * F, H, form), four(g, E, H, F, form)
    out, ws = few_call(x, idx, w, experts(w13, w2, F, form), E)
    assert ep.ep_check_errors(ws) == 0
    ref, bound = few_reference(x, w13, w2, idx, w, F, form)
    check(out, ref, bound, "out")


@FORMS
def test_few_w4_in_graphs_and_on_two_streams(form):
    """Two captured calls on a workspace each, replayed in turn with new inputs beside eager calls;
    then two streams at once. Every result equals the first eager one, bit for bit."""
    T, H, F, E, K = 40, 256, 1024, 12, 4
    g = torch.Generator().manual_seed(8)
    X = experts(four(g, E, 2 * F, H, form), four(g, E, H, F, form), F, form)
    inputs = [gpu(randn(g, T, H), *routing(T, K, E, s, skip=0.1)) for s in (1, 2)]
    ref = [few_call(*i, X, E)[0].clone() for i in inputs]
    static = [[t.clone() for t in i] for i in inputs]
    spaces = [few_call(*i, X, E)[1] for i in inputs]
    outs = [torch.empty_like(r) for r in ref]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in inputs]
    for n, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            few_call(*static[n], X, E, ws=spaces[n], out=outs[n])
    for turn in range(6):
        for n in (0, 1):
            for s, t in zip(static[n], inputs[(n + turn) % 2]):
                s.copy_(t)
            graphs[n].replay()
        few_call(*inputs[0], X, E)
        torch.cuda.synchronize()
        for n in (0, 1):
            assert torch.equal(outs[n], ref[(n + turn) % 2]), (turn, n)
        torch.randn(1000, device="cuda").sum().item()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for turn in range(6):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got.append((n, few_call(*inputs[n], X, E, ws=spaces[n])[0]))
    torch.cuda.synchronize()
    for n, out in got:
        assert torch.equal(out, ref[n])


# --------------------------------------------------------------------------
# Together: norm, router, experts
# --------------------------------------------------------------------------

def rel(a, r):
    return ((a.double().cpu() - r).norm() / r.norm()).item()


@FORMS
@pytest.mark.parametrize("T", [1, 24])
def test_decoding_layers(T, form):
    """Three layers of a decoding step, the stream updated in place: norm, router product, router, expert
    layer. Each against 64 bits on its own inputs, and the ids those of the definition.

    y is rounded once (2^-8), the layer's output once; a layer's output is off by the former in 2-norm
    times what the experts do to a relative change of their input: silu(g) u is at most quadratic, so 2 *
    2^-8 and 2^-8 of its own rounding bound the norm."""
    H, F, E, K, G = 256, 384, 16, 4, 4
    g = torch.Generator().manual_seed(12)
    stream = torch.randn((T, H), generator=g).to(BF16).cuda()
    x = randn(g, T, H).cuda()
    shape = ep.make_shape(T, H, K, E, G, G)
    ws, few_ws = cleared(shape), ep.alloc_few_w4_workspace(shape, F)
    ep.ep_clear_errors(few_ws)
    for layer in range(3):
        gain = (1 + 0.2 * torch.randn(H, generator=g)).to(BF16).cuda()
        wr = torch.randn((E, H), generator=g).cuda() * H ** -0.5
        bias = 0.05 * torch.randn(E, generator=g).cuda()
        w13, w2 = four(g, E, 2 * F, H, form), four(g, E, H, F, form)
        before = stream.double() + x.double()
        y = torch.empty((T, H), dtype=BF16, device="cuda")
        ep.ep_rms_norm(shape, x, stream, ep.EP_STREAM_BF16, gain, 1e-6, dict(h=stream, y=y))
        logits = y.float() @ wr.T
        router = dict(score=ep.EP_SCORE_SIGMOID, top_groups=2, group_top=2, scale=2.5, bias=bias)
        idx, w = torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda")
        ep.ep_route(shape, logits, router, idx, w, ws)
        x = torch.empty((T, H), dtype=BF16, device="cuda")
        ep.ep_moe_few_w4(shape, dict(x=y, topk_idx=idx, topk_weights=w), experts(w13, w2, F, form), x, few_ws)
        assert ep.ep_check_sticky_errors(ws) == 0 and ep.ep_check_sticky_errors(few_ws) == 0

        assert rel(stream, before.cpu()) <= HALF_BF16
        h = stream.double()
        y64 = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + 1e-6) * gain.double()
        s = torch.sigmoid(logits.double())
        key = s + bias.double()
        best = key.view(T, G, E // G).topk(2, dim=2).values.sum(2).topk(2, dim=1).indices
        allowed = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, best, True)
        key = torch.where(allowed.repeat_interleave(E // G, 1), key, -1e9)
        assert torch.equal(key.topk(K, dim=1).indices, idx)
        lane = s.gather(1, idx)
        ref, _ = few_reference(y64.cpu(), w13, w2, idx.cpu(), (2.5 * lane / lane.sum(1, keepdim=True)).cpu(), F, form)
        assert rel(x, ref) <= 3 * HALF_BF16, layer


def training_step(shape, F, router, args, b):
    """Norm, router, dispatch of bf16 and 8-bit rows, experts, combine, and all of it backward."""
    x, res, gain, wr, w13, w2, dout, d_h_later = args
    T, H, K, E = shape.T, shape.H, shape.K, shape.E
    N = T * K

    def buf(name, *size, dtype=BF16):
        if name not in b:
            b[name] = torch.zeros(size, dtype=dtype, device="cuda")
        return b[name]

    if "L" not in b:
        b["L"], b["ws"] = ep.alloc_layout(shape, expand=True), ep.alloc_workspace(shape)
        ep.ep_clear_errors(b["ws"])
        b["nws"] = ep.alloc_norm_workspace(shape)
        b["recv"] = ep.alloc_recv(shape, N, fp8=True, scales=True)
        b["d_recv"] = ep.alloc_recv(shape, N, meta=False)
        b["ones"] = torch.ones((T, K), device="cuda")
        b["one_expert"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    L, ws = b["L"], b["ws"]
    h, y, rstd = buf("h", T, H, dtype=F32), buf("y", T, H), buf("rstd", T, dtype=F32)
    y8, ys = buf("y8", T, H, dtype=U8), buf("ys", T, H // 128, dtype=F32)
    ep.ep_rms_norm(shape, x, res, ep.EP_STREAM_F32, gain, 1e-6, dict(h=h, y=y, y_fp8=y8, y_scales=ys, rstd=rstd))
    logits = buf("logits", T, E, dtype=F32)
    torch.matmul(y.float(), wr.float().T, out=logits)
    idx, w = buf("idx", T, K, dtype=torch.int64), buf("w", T, K, dtype=F32)
    ep.ep_route(shape, logits, router, idx, w, ws)
    ep.ep_get_layout(shape, idx, L, ws)
    ep.ep_dispatch_expand(shape, L, dict(x=y, x_fp8=y8, x_scales=ys, topk_idx=idx, topk_weights=w), b["recv"], N, ws)
    act, q, sc = buf("act", N, F), buf("q", N, 2 * F, dtype=U8), buf("sc", N, 2 * F // 128, dtype=F32)
    ep.ep_expert_swiglu(shape, L, b["recv"]["x"], N, w13, F, act, q, sc, ws)
    ye, out = buf("ye", N, H), buf("out", T, H)
    ep.ep_expert_matmul(shape, L, act, N, F, w2, H, ep.EP_WEIGHT_NK, ye, ws)
    ep.ep_combine_expand(shape, L, ye, N, 2 * H, ep.EP_FMT_PLAIN, 0, w, out, ws)

    ep.ep_dispatch_expand(shape, L, dict(x=dout, topk_idx=idx), b["d_recv"], N, ws)
    dye = b["d_recv"]["x"]
    d_act, d_gu, act_w = buf("d_act", N, F), buf("d_gu", N, 2 * F), buf("act_w", N, F)
    d_w, d_logits = buf("d_w", T, K, dtype=F32), buf("d_logits", T, E)
    ep.ep_expert_matmul(shape, L, dye, N, H, w2, F, ep.EP_WEIGHT_KN, d_act, ws)
    ep.ep_swiglu_grad(shape, L, F, q, sc, d_act, N, w, d_gu, act_w, d_w, ws)
    dw2, dw13 = buf("dw2", E, H, F, dtype=F32), buf("dw13", E, 2 * F, H, dtype=F32)
    ep.ep_expert_wgrad(shape, L, dye, N, H, dict(x=act_w), F, dw2, ep.EP_GRAD_F32, ws)
    rows8 = dict(x_fp8=b["recv"]["x_fp8"], x_scales=b["recv"]["x_scales"])
    ep.ep_expert_wgrad(shape, L, d_gu, N, 2 * F, rows8, H, dw13, ep.EP_GRAD_F32, ws)
    dxr, dy = buf("dxr", N, H), buf("dy", T, H)
    ep.ep_expert_matmul(shape, L, d_gu, N, 2 * F, w13, H, ep.EP_WEIGHT_KN, dxr, ws)
    ep.ep_combine_expand(shape, L, dxr, N, 2 * H, ep.EP_FMT_PLAIN, 0, b["ones"], dy, ws)
    ep.ep_route_grad(shape, logits, router, idx, d_w, d_logits, ep.EP_GRAD_BF16, ws)
    dense, L1 = ep.make_shape(T, H, 1, 1, 1), dict(expert_offsets=b["one_expert"])
    dwr, dyr = buf("dwr", 1, E, H, dtype=F32), buf("dyr", T, H)
    ep.ep_expert_wgrad(dense, L1, d_logits, T, E, dict(x=y), H, dwr, ep.EP_GRAD_F32, ws)
    ep.ep_expert_matmul(dense, L1, d_logits, T, E, wr, H, ep.EP_WEIGHT_KN, dyr, ws)
    dy.add_(dyr)
    d_h, d_x, d_gain = buf("d_h", T, H, dtype=F32), buf("d_x", T, H), buf("d_gain", H, dtype=F32)
    ep.ep_rms_norm_grad(shape, h, ep.EP_STREAM_F32, gain, rstd, dy, d_h_later, d_h, d_x, d_gain, b["nws"])
    return b


def training_case(T, H, F, E, seed=6):
    g = torch.Generator().manual_seed(seed)
    return [randn(g, T, H), torch.randn((T, H), generator=g), (1 + 0.2 * torch.randn(H, generator=g)).to(BF16),
            randn(g, E, H, scale=H ** -0.5), randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5),
            randn(g, T, H), torch.randn((T, H), generator=g)]


@pytest.mark.parametrize("score", [ep.EP_SCORE_SOFTMAX, ep.EP_SCORE_SIGMOID], ids=["softmax", "sigmoid"])
def test_training_layer_forward_and_backward(score):
    """A layer's training step from the stream on, against automatic differentiation in 64 bits with the
    same choice of experts.

    The output passes four roundings to bf16 (y twice as strong, silu(g) u being at most quadratic; act,
    ye, out): 5 * 2^-8. The backward uses g and u from 8 bits and the rows from 8 bits (2^-4 at most each,
    which enters through products of two: 2 * 2^-4) beside bf16 roundings on the way, at most eight."""
    T, H, F, E, K = 150, 256, 256, 8, 3
    args = training_case(T, H, F, E)
    shape = ep.make_shape(T, H, K, E, 1)
    router = dict(score=score, normalize=True, scale=1.5)
    b = training_step(shape, F, router, gpu(*args), {})
    assert ep.ep_check_sticky_errors(b["ws"]) == 0
    x, res, gain, wr, w13, w2 = (t.double().requires_grad_() for t in args[:6])
    h = x + res
    y = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + 1e-6) * gain
    logits = y @ wr.T
    s = torch.softmax(logits, 1) if score == ep.EP_SCORE_SOFTMAX else torch.sigmoid(logits)
    idx = b["idx"].cpu()
    w = s.gather(1, idx)
    w = 1.5 * w / w.sum(1, keepdim=True)
    out = torch.zeros((T, H), dtype=F64)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        gu = y[t] @ w13[e].T
        a = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        out = out.index_add(0, t, w[t, k].unsqueeze(1) * (a @ w2[e].T))
    ((out * args[6].double()).sum() + (h * args[7].double()).sum()).backward()
    assert rel(b["out"], out.detach()) <= 5 * HALF_BF16
    grads = dict(d_h=res.grad, d_x=x.grad, d_gain=gain.grad, dw13=w13.grad, dw2=w2.grad)
    for name, ref in grads.items():
        assert rel(b[name], ref) <= 2 * HALF_E4M3 + 8 * HALF_BF16, name
    assert rel(b["dwr"][0], wr.grad) <= 2 * HALF_E4M3 + 8 * HALF_BF16


def test_training_layer_in_a_graph():
    """Captured while the buffers of an eager step live, replayed with new inputs and eager work between;
    every replay equals the eager result bit for bit."""
    T, H, F, E, K = 100, 128, 128, 8, 2  # the router's products take E in multiples of 8
    shape = ep.make_shape(T, H, K, E, 1)
    router = dict(score=ep.EP_SCORE_SOFTMAX, normalize=False)
    inputs = [gpu(*training_case(T, H, F, E, seed)) for seed in (1, 2, 3)]
    names = ("h", "out", "idx", "d_h", "d_x", "d_gain", "dw13", "dw2", "dwr", "d_logits")
    eager = []
    for args in inputs:
        b = training_step(shape, F, router, args, {})
        torch.cuda.synchronize()
        eager.append({n: b[n].clone() for n in names})
    static, b = [t.clone() for t in inputs[0]], {}
    training_step(shape, F, router, static, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        training_step(shape, F, router, static, b)
    for i in (0, 1, 2, 1, 0):
        for s, t in zip(static, inputs[i]):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(b[n].view(U8), eager[i][n].view(U8)), (i, n)
        torch.randn(1000, device="cuda").sum().item()
        training_step(shape, F, router, inputs[i], {})
