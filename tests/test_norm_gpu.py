"""The norm of the residual stream (ep_rms_norm) and its gradient
(ep_rms_norm_grad) against plain 64-bit arithmetic.

Tolerances are bounds by arithmetic. Half a step is 2^-24 of a value in 32
bits, 2^-8 in bf16, 2^-4 in e4m3 (2^-10 near zero).
  - A sum over a row: each of at least 64 threads adds every 64th vector of 8
    (H / 64 values, at least 8), then at most 6 + 16 of their sums join, so
    it is off by (max(H / 64, 8) + 22) * 2^-24 of the sum of magnitudes.
  - 1 / sqrt(sum / H + eps): half the sum's error, and half a step each for the
    quotient, the addition, the root and the reciprocal: 2 steps in all.
"""
import pytest
import torch

from combine_get_layout_amd import ep
from test_experts_gpu import BF16, F8, F32, F64, HALF_BF16, HALF_E4M3, U8, U23, check_there, randn

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
EPS = 1e-5
MOST = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ep.lib()


def row_steps(H):
    return (max(H // 64, 8) + 22) * U24


def stream(g, T, H, wide):
    v = torch.randn((T, H), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    return v.to(F32 if wide else BF16)


def kind(wide):
    return ep.EP_STREAM_F32 if wide else ep.EP_STREAM_BF16


def norm_case(T, H, wide, residual, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = randn(g, T, H).cuda()
    res = stream(g, T, H, wide).cuda() if residual else None
    return x, res, (1 + 0.3 * torch.randn(H, generator=g)).to(BF16).cuda()


def check_norm(x, res, gain, out, wide, eps=EPS):
    """Every output against 64 bits; the norm against that of the stored stream."""
    H = x.shape[1]
    h = x.double() if res is None else x.double() + res.double()
    if "h" in out:
        half = U24 if wide else HALF_BF16
        # The sum in 32 bits, then rounded to the stream's type.
        check_there(out["h"], h, U24 * h.abs() + half * h.abs() * (1 + U24), "h")
        h = out["h"].double()
    elif res is not None:
        h = (x.float() + res.float()).to(res.dtype).double()
    r = 1 / torch.sqrt(h.pow(2).mean(1, keepdim=True) + eps)
    rel = row_steps(H) / 2 + 2 * U23
    if "rstd" in out:
        check_there(out["rstd"], r[:, 0], rel * r[:, 0], "rstd")
    v = h * r * gain.double()
    off = v.abs() * (rel + 2 * U24) * (1 + 2.0 ** -10)  # two products more
    if "y" in out:
        check_there(out["y"], v, off + HALF_BF16 * (v.abs() + off), "y")
    if "y_fp8" in out:
        m = v.reshape(len(v), -1, 128).abs().amax(2)
        # The largest magnitude times 1 / 448, that and the product rounded.
        check_there(out["y_scales"], m / 448, (rel + 4 * U24 + 2 * U24) * m / 448, "y_scales")
        rep = out["y_scales"].double().repeat_interleave(128, 1)
        val = out["y_fp8"].view(F8).double() * rep
        off = off + 4 * U23 * v.abs()  # the reciprocal and its product
        check_there(val, v, off + HALF_E4M3 * (v.abs() + off) + 2.0 ** -10 * rep, "y_fp8")


def outputs(T, H, wide, names, spare=0):
    make = dict(h=lambda: torch.full((T + spare, H), 7.0, dtype=F32 if wide else BF16, device="cuda"),
                y=lambda: torch.full((T + spare, H), 7.0, dtype=BF16, device="cuda"),
                y_fp8=lambda: torch.full((T + spare, H), 0x55, dtype=U8, device="cuda"),
                y_scales=lambda: torch.full((T + spare, H // 128), 7.0, device="cuda"),
                rstd=lambda: torch.full((T + spare,), 7.0, device="cuda"))
    return {n: make[n]() for n in names}


# Row lengths on both sides of every change of kernel: 64 to 1,024 threads to a row, one to
# four vectors of eight to a thread, and rows in two passes.
LENGTHS = [8, 72, 512, 520, 1024, 1032, 2048, 2056, 3080, 4096, 4104, 5120, 5128, 6144, 6152, 7168, 7176, 8192, 8200, 16384, 16392, 32768, 32776, 40960]


@pytest.mark.parametrize("residual", [True, False], ids=["residual", "alone"])
@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", LENGTHS)
def test_norm(H, wide, residual):
    T, spare = 5, 2
    x, res, gain = norm_case(T, H, wide, residual)
    names = ["h", "y", "rstd"] + (["y_fp8", "y_scales"] if H % 128 == 0 else [])
    out = outputs(T, H, wide, names, spare)
    ep.ep_rms_norm(ep.make_shape(T, H, 1, 1, 1), x, res, kind(wide), gain, EPS, out)
    for n, t in out.items():  # rows behind the last stay as they were
        assert (t[T:] == (0x55 if n == "y_fp8" else 7)).all(), n
    check_norm(x, res, gain, {n: t[:T] for n, t in out.items()}, wide)
    # One output at a time gives the same.
    for n in ("h", "y", "rstd"):
        alone = outputs(T, H, wide, [n])
        ep.ep_rms_norm(ep.make_shape(T, H, 1, 1, 1), x, res, kind(wide), gain, EPS, alone)
        assert torch.equal(alone[n], out[n][:T]), n


@pytest.mark.parametrize("T,H", [(1, 7168), (1, 128), (300, 384), (1, 1024), (64, 2048), (1000, 1152), (3, MOST)])
def test_norm_rows(T, H):
    x, res, gain = norm_case(T, H, False, True, seed=T)
    out = outputs(T, H, False, ["h", "y", "y_fp8", "y_scales", "rstd"])
    ep.ep_rms_norm(ep.make_shape(T, H, 1, 1, 1), x, res, ep.EP_STREAM_BF16, gain, EPS, out)
    check_norm(x, res, gain, out, False)
    # 8-bit rows alone, as dispatch takes them.
    eight = outputs(T, H, False, ["y_fp8", "y_scales"])
    ep.ep_rms_norm(ep.make_shape(T, H, 1, 1, 1), x, res, ep.EP_STREAM_BF16, gain, EPS, eight)
    assert torch.equal(eight["y_fp8"], out["y_fp8"]) and torch.equal(eight["y_scales"], out["y_scales"])


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [264, 4096, 32776])
def test_norm_takes_the_stream_in_place(H, wide):
    """The stream updated where it lies, as a decoding loop keeps it."""
    T = 9
    x, res, gain = norm_case(T, H, wide, True)
    shape = ep.make_shape(T, H, 1, 1, 1)
    ref = outputs(T, H, wide, ["h", "y"])
    ep.ep_rms_norm(shape, x, res, kind(wide), gain, EPS, ref)
    y, same = torch.empty_like(x), res.clone()
    ep.ep_rms_norm(shape, x, same, kind(wide), gain, EPS, dict(h=same, y=y))
    assert torch.equal(same, ref["h"]) and torch.equal(y, ref["y"])


@pytest.mark.parametrize("H", [128, 4096, 40960])
def test_norm_of_zero_and_nonfinite_rows(H):
    """A row of zeros: rstd 1 / sqrt(eps), zeros, scales of 1. A row with a NaN is all NaN, one with an
    infinity has rstd 0: NaN where the infinity is, zeros elsewhere. Neighbours keep theirs."""
    T = 5
    x, _, gain = norm_case(T, H, False, False)
    gain[:] = 1.0
    clean = x.clone()
    x[1] = 0
    x[2, H - 3] = float("nan")
    x[4, 1] = float("-inf")
    shape = ep.make_shape(T, H, 1, 1, 1)
    out = outputs(T, H, False, ["y", "y_fp8", "y_scales", "rstd"])
    ep.ep_rms_norm(shape, x, None, ep.EP_STREAM_BF16, gain, EPS, out)
    val = out["y_fp8"].view(F8).double() * out["y_scales"].double().repeat_interleave(128, 1)
    assert (out["y"][1] == 0).all() and (val[1] == 0).all() and (out["y_scales"][1] == 1).all()
    assert abs(out["rstd"][1].item() * EPS ** 0.5 - 1) < 1e-6
    assert torch.isnan(out["y"][2]).all() and torch.isnan(val[2]).all()
    assert out["rstd"][4] == 0 and torch.isnan(out["y"][4, 1]) and torch.isnan(val[4, 1])
    rest = [c for c in range(H) if c != 1]
    assert (out["y"][4, rest] == 0).all() and (val[4, rest] == 0).all()
    for t in (0, 3):
        check_norm(clean[t:t + 1], None, gain, {n: v[t:t + 1] for n, v in out.items()}, False)


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [8, 512, 1032, 2048, 2056, 4096, 5120, 6144, 7168, 8192, 16384, 32768, 40960, MOST])
def test_norm_of_rows_whose_squares_add_up_past_32_bits(H, wide):
    """Values of about 1e19: the mean of their squares is a number of 32 bits, the sum is not. One value of
    2^63.5 sqrt(H) alone; a row of 3e19, whose mean passes too, has rstd 0. Neighbours keep theirs."""
    x, res, gain = norm_case(6, H, wide, True)
    x[1], res[1] = 0.5e19 * (1 + torch.rand(H, device="cuda")), 0.5e19
    x[2], res[2] = 0, 0
    x[2, H // 2] = 2.0 ** 63.5 * H ** 0.5
    x[4], res[4] = 3e19, 0
    h = x.double() + res.double()
    assert h[1].pow(2).mean() < 3e38 and (h[1].pow(2).sum() > 4e38 or H < 8) and h[2].pow(2).mean() < 3e38
    assert h[4].pow(2).mean() > 4e38
    names = ["h", "y", "rstd"] + (["y_fp8", "y_scales"] if H % 128 == 0 else [])
    out = outputs(6, H, wide, names)
    shape = ep.make_shape(6, H, 1, 1, 1)
    ep.ep_rms_norm(shape, x, res, kind(wide), gain, EPS, out)
    assert out["rstd"][4] == 0 and (out["y"][4] == 0).all()
    keep = [0, 1, 3, 5]
    check_norm(x[keep], res[keep], gain, {n: t[keep] for n, t in out.items()}, wide)
    check_norm(x[2:3], res[2:3], gain, {n: out[n][2:3] for n in ("h", "y", "rstd")}, wide)
    if H % 128 == 0:  # its other blocks are zeros
        v = h[2] * out["rstd"][2].double() * gain.double()
        block = H // 2 // 128
        scale = torch.ones(H // 128, dtype=F64, device="cuda")
        scale[block] = v.abs().max() / 448
        check_there(out["y_scales"][2], scale, 4 * U24 * scale, "y_scales of one value")
        got = out["y_fp8"][2].view(F8).float()
        assert (got != 0).sum() == 1 and got[H // 2] == 448 * torch.sign(v[H // 2])
    # Without the stored stream, and in place of the residual.
    y = outputs(6, H, wide, ["y"])
    ep.ep_rms_norm(shape, x, res, kind(wide), gain, EPS, y)
    assert torch.equal(y["y"], out["y"])
    y, same = outputs(6, H, wide, ["y"]), res.clone()
    ep.ep_rms_norm(shape, x, same, kind(wide), gain, EPS, dict(y, h=same))
    assert torch.equal(y["y"], out["y"]) and torch.equal(same, out["h"])


def test_norm_of_small_blocks():
    """A block whose largest magnitude is below 1e-33 has a scale of 1 and zeros."""
    H = 256
    x, _, gain = norm_case(3, H, False, False)
    gain[:128] = 1e-36
    out = outputs(3, H, False, ["y_fp8", "y_scales"])
    ep.ep_rms_norm(ep.make_shape(3, H, 1, 1, 1), x, None, ep.EP_STREAM_BF16, gain, EPS, out)
    assert (out["y_scales"][:, 0] == 1).all() and (out["y_fp8"][:, :128].view(F8).float() == 0).all()
    assert (out["y_fp8"][:, 128:].view(F8).float().abs().amax(1) == 448).all()


def test_norm_of_more_rows_than_one_launch():
    """2^21 workgroups of four rows and a few rows more: the same as in two calls."""
    T, H, cut = (1 << 23) + 7, 8, 1 << 22
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF16)
    gain = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    out = outputs(T, H, False, ["y", "rstd"], spare=2)
    ep.ep_rms_norm(ep.make_shape(T, H, 1, 1, 1), x, None, ep.EP_STREAM_BF16, gain, EPS, out)
    assert (out["y"][T:] == 7).all() and (out["rstd"][T:] == 7).all()
    for part in (slice(0, cut), slice(cut, T)):
        alone = outputs(part.stop - part.start, H, False, ["y", "rstd"])
        ep.ep_rms_norm(ep.make_shape(part.stop - part.start, H, 1, 1, 1), x[part], None, ep.EP_STREAM_BF16, gain, EPS, alone)
        for n in alone:
            assert torch.equal(alone[n], out[n][part]), n
    check_norm(x[-9:], None, gain, {n: t[T - 9:T] for n, t in out.items()}, False)


def test_norm_offsets_past_32_bits():
    """More than 2^32 bytes of each array; the last rows are right."""
    T, H = 300_000, 8192
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    last, res, gain = norm_case(4, H, False, True)
    x[-4:] = last
    out = dict(y=torch.empty_like(x), rstd=torch.empty(T, device="cuda"))
    shape = ep.make_shape(T, H, 1, 1, 1)
    ep.ep_rms_norm(shape, x, None, ep.EP_STREAM_BF16, gain, EPS, out)
    check_norm(last, None, gain, {n: t[-4:] for n, t in out.items()}, False)
    dy = out["y"]
    ws = ep.alloc_norm_workspace(shape)
    d_h, d_gain = torch.empty_like(x), torch.empty(H, device="cuda")
    ep.ep_rms_norm_grad(shape, x, ep.EP_STREAM_BF16, gain, out["rstd"], dy, None, d_h, None, d_gain, ws)
    check_grad(last, gain, out["rstd"][-4:], dy[-4:], None, dict(d_h=d_h[-4:]), False)
    _, _, dg, dg_off = grad_bounds(last, gain, out["rstd"][-4:], dy[-4:], None, 4)  # the other rows add zeros
    check_there(d_gain, dg, dg_off, "d_gain")


# --------------------------------------------------------------------------
# Gradient
# --------------------------------------------------------------------------

def grad_bounds(h, gain, r, dy, ds, T):
    """d, d_gain and how far 32 bits are off, in 64 bits."""
    H = h.shape[1]
    h, dy, g, r = h.double(), dy.double(), gain.double(), r.double().unsqueeze(1)
    a = dy * g
    k = r * r * (a * h).mean(1, keepdim=True)
    d = r * (a - k * h)
    # The dot product: its sum, the products' rounding, then / H and r^2: 4 steps.
    dk = r * r * (a * h).abs().mean(1, keepdim=True) * (row_steps(H) + 4 * U23)
    off = r * (h.abs() * dk + 4 * U24 * (a.abs() + (k * h).abs()))
    if ds is not None:
        d = d + ds.double()
        off = off + U24 * (d.abs() + ds.double().abs())
    each = dy * h * r
    # Each term rounded twice; at most T additions follow each other.
    return d, off, each.sum(0), (T + 4) * U24 * each.abs().sum(0)


def check_grad(h, gain, r, dy, ds, out, wide):
    d, off, dg, dg_off = grad_bounds(h, gain, r, dy, ds, len(h))
    if out.get("d_h") is not None:
        half = U24 if wide else HALF_BF16
        check_there(out["d_h"], d, off + half * (d.abs() + off), "d_h")
    if out.get("d_x") is not None:
        check_there(out["d_x"], d, off + HALF_BF16 * (d.abs() + off), "d_x")
    if out.get("d_gain") is not None:
        check_there(out["d_gain"], dg, dg_off, "d_gain")


def grad_case(T, H, wide, add, seed=2):
    g = torch.Generator().manual_seed(seed)
    h = stream(g, T, H, wide).cuda()
    gain = (1 + 0.3 * torch.randn(H, generator=g)).to(BF16).cuda()
    r = (1 / torch.sqrt(h.double().pow(2).mean(1) + EPS)).float()
    dy = randn(g, T, H).cuda()
    ds = stream(g, T, H, wide).cuda() if add else None
    return h, gain, r, dy, ds


def grad_call(shape, case, wide, ws, d_h=True, d_x=True, d_gain=True, spare=0):
    h, gain, r, dy, ds = case
    T, H = shape.T, shape.H
    out = dict(d_h=torch.full((T + spare, H), 7.0, dtype=h.dtype, device="cuda") if d_h else None,
               d_x=torch.full((T + spare, H), 7.0, dtype=BF16, device="cuda") if d_x else None,
               d_gain=torch.full((H,), 7.0, device="cuda") if d_gain else None)
    ep.ep_rms_norm_grad(shape, h, kind(wide), gain, r, dy, ds, out["d_h"], out["d_x"], out["d_gain"], ws)
    return out


@pytest.mark.parametrize("add", [True, False], ids=["stream", "alone"])
@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", LENGTHS)
def test_norm_grad(H, wide, add):
    T = 7
    case = grad_case(T, H, wide, add)
    shape = ep.make_shape(T, H, 1, 1, 1)
    ws = ep.alloc_norm_workspace(shape).fill_(0xAB)
    out = grad_call(shape, case, wide, ws, spare=2)
    assert (out["d_h"][T:] == 7).all() and (out["d_x"][T:] == 7).all()
    out = dict(out, d_h=out["d_h"][:T], d_x=out["d_x"][:T])
    check_grad(*case, out, wide)
    for only in ("d_h", "d_x", "d_gain"):
        alone = grad_call(shape, case, wide, ws, **{n: n == only for n in ("d_h", "d_x", "d_gain")})
        assert torch.equal(alone[only], out[only]), only


@pytest.mark.parametrize("T,H", [(1, 7168), (1, 8), (4099, 72), (2500, 2056), (1111, 9000), (130, 33000), (2, MOST)])
def test_norm_grad_rows(T, H):
    """One row, and more rows than the workgroups take at once."""
    case = grad_case(T, H, False, True, seed=T)
    shape = ep.make_shape(T, H, 1, 1, 1)
    ws = ep.alloc_norm_workspace(shape).fill_(0xAB)
    out = grad_call(shape, case, False, ws, d_x=False)
    check_grad(*case, out, False)
    again = grad_call(shape, case, False, ws, d_x=False)
    assert torch.equal(again["d_gain"], out["d_gain"]) and torch.equal(again["d_h"], out["d_h"])


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1500, 512), (2049, 512), (512, 8192), (513, 8192), (1024, 8192), (300, 16384), (70, 20480),
                                 (1, 32768), (300, 32768)])
def test_norm_grad_in_one_launch_and_in_two(T, H, wide):
    """The gain's gradient beside the rows and behind them, and rows held and read twice, in both streams."""
    case = grad_case(T, H, wide, True, seed=T)
    shape = ep.make_shape(T, H, 1, 1, 1)
    ws = ep.alloc_norm_workspace(shape).fill_(0xAB)
    out = grad_call(shape, case, wide, ws)
    check_grad(*case, out, wide)
    for only in ("d_h", "d_gain"):
        alone = grad_call(shape, case, wide, ws, **{n: n == only for n in ("d_h", "d_x", "d_gain")})
        assert torch.equal(alone[only], out[only]), only


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [264, 4096, 32776])
def test_norm_grad_in_place(H, wide):
    T = 9
    h, gain, r, dy, ds = case = grad_case(T, H, wide, True)
    shape = ep.make_shape(T, H, 1, 1, 1)
    ws = ep.alloc_norm_workspace(shape)
    ref = grad_call(shape, case, wide, ws, d_gain=False)
    same = ds.clone()
    ep.ep_rms_norm_grad(shape, h, kind(wide), gain, r, dy, same, same, None, None, ws)
    assert torch.equal(same, ref["d_h"])


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [8, 512, 1024, 1032, 2056, 4104, 7168, 8192, 16384, 32768, 40960])
def test_norm_grad_of_small_and_large_rows(H, wide):
    """With eps of 1e-40: a row of zeros, whose 1 / sqrt(eps) squared passes 32 bits, one of about 1e-21, an
    ordinary one, and rows of about 1e19, with gradients of 1e19 too, whose products pass 32 bits."""
    eps = 1e-40
    h, gain, _, dy, ds = grad_case(5, H, wide, True, seed=9)
    h = h / h.double().pow(2).mean(1, keepdim=True).sqrt().to(h.dtype)
    h[0], h[1] = 0, h[1] * 1e-21
    h[3:] *= 1e19
    dy[4] *= 1e19
    shape = ep.make_shape(5, H, 1, 1, 1)
    rstd = torch.empty(5, device="cuda")
    # The forward's rstd, of the 32-bit stream's rows by the definition (x has 16 bits).
    r = (1 / torch.sqrt(h.double().pow(2).mean(1) + torch.tensor(eps, dtype=F32).double().item())).float()
    if not wide:
        ep.ep_rms_norm(shape, h, None, ep.EP_STREAM_BF16, gain, eps, dict(rstd=rstd))
        check_there(rstd, r.double(), (row_steps(H) / 2 + 2 * U23) * r.double() + 2.0 ** -149 * r.double() / (2 * eps), "rstd")
    ws = ep.alloc_norm_workspace(shape).fill_(0xAB)
    for rows in ([0, 1, 2, 3, 4], [0], [3, 4]):
        case = [t[rows].contiguous() for t in (h, r, dy, ds)]
        case.insert(1, gain)
        out = grad_call(ep.make_shape(len(rows), H, 1, 1, 1), case, wide, ws)
        check_grad(*case, out, wide)


def test_norm_grad_against_differences():
    """The gradient against central differences, in 64 bits, of sum dy * y + sum ds * h as ep_rms_norm
    defines y. With steps of 1e-4 and third derivatives of at most about 6 r^3 |a| sqrt(H) the
    differences are off by under 1e-7 of r |a| sqrt(H)."""
    T, H = 3, 24
    h, gain, r, dy, ds = (t.cpu() for t in grad_case(T, H, True, True))
    shape = ep.make_shape(T, H, 1, 1, 1)
    ws = ep.alloc_norm_workspace(shape)
    out = grad_call(shape, [t.cuda() for t in (h, gain, r, dy, ds)], True, ws, d_x=False)

    def loss(h, g):
        return (dy.double() * (h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + EPS) * g)).sum() + (ds.double() * h).sum()

    H64, G64, step = h.double(), gain.double(), 1e-4
    num, num_g = torch.zeros_like(H64), torch.zeros_like(G64)
    for t in range(T):
        for c in range(H):
            a, b = H64.clone(), H64.clone()
            a[t, c] += step
            b[t, c] -= step
            num[t, c] = (loss(a, G64) - loss(b, G64)) / (2 * step)
    for c in range(H):
        a, b = G64.clone(), G64.clone()
        a[c] += step
        b[c] -= step
        num_g[c] = (loss(H64, a) - loss(H64, b)) / (2 * step)
    d, off, dg, dg_off = grad_bounds(h, gain, r, dy, ds, T)
    small = 1e-6 * (r.double().unsqueeze(1) * (dy.double() * G64).norm(dim=1, keepdim=True) + 1)
    # r comes from 32 bits: each term it enters is off by 3 * 2^-24 more.
    r_off = 3 * U23 * ((d - ds.double()).abs() + r.double().unsqueeze(1) * (dy.double() * G64).abs())
    check_there(out["d_h"].cpu(), num, off + small + r_off + U24 * num.abs(), "d_h against differences")
    check_there(out["d_gain"].cpu(), num_g, dg_off + 1e-6 * (1 + num_g.abs()), "d_gain against differences")


def test_norm_without_tokens():
    H = 256
    shape = ep.make_shape(0, H, 1, 1, 1)
    ws = ep.alloc_norm_workspace(shape)
    ep.ep_rms_norm(shape, None, None, ep.EP_STREAM_BF16, None, EPS, {})
    d_gain = torch.full((H,), 7.0, device="cuda")
    ep.ep_rms_norm_grad(shape, None, ep.EP_STREAM_BF16, None, None, None, None, None, None, d_gain, ws)
    assert (d_gain == 0).all()


def test_norm_in_a_graph_and_on_two_streams():
    """Captured once and replayed with new inputs, with eager work between; two streams at once on a
    workspace each. Every result equals the eager one."""
    T, H = 700, 2056
    shape = ep.make_shape(T, H, 1, 1, 1)
    cases = [grad_case(T, H, False, True, seed=s) for s in (3, 4)]
    xs = [norm_case(T, H, False, True, seed=s)[0] for s in (5, 6)]

    def step(x, case, ws, b):
        h, gain, r, dy, ds = case
        out = b.setdefault("out", outputs(T, H, False, ["h", "y", "rstd"]))
        ep.ep_rms_norm(shape, x, h, ep.EP_STREAM_BF16, gain, EPS, out)
        g = b.setdefault("g", dict(d_h=torch.empty_like(h), d_gain=torch.empty(H, device="cuda")))
        ep.ep_rms_norm_grad(shape, out["h"], ep.EP_STREAM_BF16, gain, out["rstd"], dy, ds, g["d_h"], None, g["d_gain"], ws)
        return [out["h"], out["y"], out["rstd"], g["d_h"], g["d_gain"]]

    ref = []
    for x, case in zip(xs, cases):
        ref.append([t.clone() for t in step(x, case, ep.alloc_norm_workspace(shape), {})])
    torch.cuda.synchronize()
    static_x, static, b, ws = xs[0].clone(), [t.clone() for t in cases[0]], {}, ep.alloc_norm_workspace(shape)
    step(static_x, static, ws, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static_x, static, ws, b)
    for i in (0, 1, 1, 0, 1):
        static_x.copy_(xs[i])
        for s, t in zip(static, cases[i]):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for a, r in zip(got, ref[i]):
            assert torch.equal(a, r)
        step(xs[1 - i], cases[1 - i], ep.alloc_norm_workspace(shape), {})
        torch.randn(1000, device="cuda").sum().item()
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [ep.alloc_norm_workspace(shape) for _ in range(2)]
    bufs = [{}, {}]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                last = step(xs[i], cases[i], spaces[i], bufs[i])
                bufs[i]["last"] = last
    torch.cuda.synchronize()
    for i in range(2):
        for a, r in zip(bufs[i]["last"], ref[i]):
            assert torch.equal(a, r)
