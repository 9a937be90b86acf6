"""Measured cases of the operators around the experts: the root-mean-square
norm with the residual's addition and 8-bit rows, its gradient, the router's
selection, its gradient, and the few-token layer with 4-bit weights.

A case is a dict of plain values. `prepare` makes what a program holds before
the call, `run` makes one pass: with `own` false in elementary torch
operations, with `own` true by the library's entry points. `exact` states the
same results in 64 bits.
"""
import math

import torch

own = False

BF16, F8, F32, F64 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64
E4M3_MAX = 448.0
BLOCK = 128       # channels that share a scale (8-bit rows, 4-bit integers)
SMALL_BLOCK = 32  # channels that share a scale (4-bit floating point)
EPS = 1e-6        # of the norm
TINY = 1e-20      # of the weights' sum
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    def norm(name, T, H, residual=True, wide=False, fp8=False, save=False):
        return dict(name=name, op="norm", T=T, H=H, residual=residual, wide=wide, fp8=fp8, save=save)

    def norm_grad(name, T, H, wide=False, stream=True):
        return dict(name=name, op="norm_grad", T=T, H=H, wide=wide, stream=stream)

    def route(name, op, T, E, K, sigmoid, G=1, top_groups=1, group_top=1, bias=False, normalize=True, masked=0.0):
        return dict(name=name, op=op, T=T, E=E, K=K, sigmoid=sigmoid, G=G, top_groups=top_groups,
                    group_top=group_top, bias=bias, normalize=normalize, masked=masked)

    def few(name, T, H, F, E, K, form, drop=0.0):
        return dict(name=name, op="few", T=T, H=H, F=F, E=E, K=K, form=form, drop=drop)

    return [
        # One decoded token before its expert layer: latency.
        norm("norm_token", 1, 7168),
        # A training step's tokens: residual added, bf16 and 8-bit rows for dispatch, what the gradient needs.
        norm("norm_train", 4096, 7168, fp8=True, save=True),
        # A small batch of an odd width on a residual stream kept in 32 bits.
        norm_grad("norm_grad_odd", 201, 2056, wide=True),
        # The gradient of the training step's norm, the later layers' gradient of the stream added.
        norm_grad("norm_grad_train", 4096, 7168),
        # A decode batch with a padded part (experts masked by -infinity), softmax, no groups: latency.
        route("route_decode", "route", 13, 72, 6, sigmoid=False, masked=0.1),
        # A training step's tokens: sigmoid scores with a balancing bias, 4 of 8 groups, 8 of 256 experts.
        route("route_train", "route", 4096, 256, 8, sigmoid=True, G=8, top_groups=4, group_top=2, bias=True),
        # Gradient of a small batch's router, softmax weights as they are.
        route("route_grad_small", "route_grad", 333, 48, 3, sigmoid=False, normalize=False),
        # Gradient of the training step's router.
        route("route_grad_train", "route_grad", 4096, 256, 8, sigmoid=True, G=8, top_groups=4, group_top=2,
              bias=True),
        # One token through a small model with 4-bit experts: latency.
        few("few4_tiny", 1, 256, 512, 16, 2, "int"),
        # One decoded token through a large layer: eight experts' weights are streamed once.
        few("few4_token", 1, 7168, 2048, 64, 8, "int"),
        # A decode batch with skipped lanes and sizes that fill no tile.
        few("few4_odd", 13, 2080, 736, 40, 3, "e2m1", drop=0.1),
        # A decode batch that touches nearly every expert.
        few("few4_batch", 32, 7168, 2048, 64, 8, "e2m1"),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["norm", "norm", "norm_grad", "route", "route_grad", "few", "few"])
    if op in ("norm", "norm_grad"):
        fp8 = op == "norm" and rng.random() < 0.5
        H = log(128, 7168, BLOCK if fp8 else 8)
        T = min(log(1, 16384), 4096 * 7168 // H // 2)
        wide = rng.random() < 0.4
        if op == "norm":
            return dict(op=op, T=T, H=H, residual=rng.random() < 0.8, wide=wide, fp8=fp8, save=rng.random() < 0.5)
        return dict(op=op, T=T, H=H, wide=wide, stream=rng.random() < 0.7)
    if op in ("route", "route_grad"):
        G = rng.choice([1, 1, 4, 8])
        E = log(8, 512, G)
        T = min(log(1, 16384), 4096 * 256 // E)
        sigmoid, bias = rng.random() < 0.5, rng.random() < 0.5
        top_groups = rng.randint(max(1, G // 2), G)
        group_top = rng.choice([1, 2]) if G > 1 else 1
        K = rng.randint(1, min(8, E // G * top_groups))
        return dict(op=op, T=T, E=E, K=K, sigmoid=sigmoid, G=G, top_groups=top_groups, group_top=group_top,
                    bias=bias, normalize=K > 1 and rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.1]))
    form = rng.choice(["int", "e2m1"])
    step = BLOCK if form == "int" else SMALL_BLOCK
    K = rng.randint(1, 8)
    T = log(1, 128)
    return dict(op=op, T=T, H=log(256, 7168, step), F=log(128, 2048, step), E=rng.randint(8, 64), K=K, form=form,
                drop=rng.choice([0.0, 0.0, 0.1]) if T * K >= 16 else 0.0)


def work(c):
    T = c["T"]
    if c["op"] == "norm":
        H, w = c["H"], 4 if c["wide"] else 2
        stored = 2 * w if c["residual"] else 0  # the stream, read and written
        out = 2 + (1 + 4 / BLOCK if c["fp8"] else 0)
        return dict(bytes=T * H * (2 + stored + out) + 2 * H + (4 * T if c["save"] else 0), flops=T * H * 8)
    if c["op"] == "norm_grad":
        H, w = c["H"], 4 if c["wide"] else 2
        rows = 2 + w + (w if c["stream"] else 0) + w + (2 if c["wide"] else 0)
        return dict(bytes=T * H * rows + 6 * H + 4 * T, flops=T * H * 10)
    if c["op"] == "route":
        return dict(bytes=T * c["E"] * 4 + T * c["K"] * 12 + (4 * c["E"] if c["bias"] else 0), flops=T * c["E"] * 8)
    if c["op"] == "route_grad":
        # Sigmoid scores need the chosen logits alone.
        read = c["K"] if c["sigmoid"] else c["E"]
        return dict(bytes=T * read * 4 + T * c["K"] * 12 + T * c["E"] * 4, flops=T * c["E"] * 8)
    H, F, E, K = c["H"], c["F"], c["E"], c["K"]
    lanes = T * K - _dropped(c)
    # Expected experts that T tokens with K distinct lanes each reach.
    used = E * (1.0 - (1.0 - K * (1.0 - c["drop"]) / E) ** T)
    per = 3 * F * H * (0.5 + (2.0 / BLOCK if c["form"] == "int" else 1.0 / SMALL_BLOCK))
    return dict(bytes=used * per + T * H * 4 + T * K * 12, flops=lanes * 6 * F * H)


def _dropped(c):
    """Skipped lanes."""
    return int(c["T"] * c["K"] * c["drop"])


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _stream_rows(c, g):
    """Rows of a residual stream: a few channels are much larger than the others, rows differ in size."""
    T, H = c["T"], c["H"]
    v = torch.randn((T, H), generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))
    v *= torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return v.to(F32 if c["wide"] else BF16)


def _logits(c, g):
    """Router logits, some experts masked by -infinity, and padded tokens with nothing but those."""
    T, E = c["T"], c["E"]
    l = 1.5 * torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    if c["masked"]:
        l[torch.rand((T, E), generator=g, device="cuda") < c["masked"]] = -math.inf
        l[torch.rand(T, generator=g, device="cuda") < c["masked"]] = -math.inf
    return l


def _four_bit(c, g, rows, cols):
    """Codes (two a byte, the even column's in the low half) and scales of a matrix per expert, as rounding
    normal values gives them."""
    E = c["E"]
    w = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device="cuda")
    table = torch.tensor(E2M1, device="cuda", dtype=BF16)
    middles = ((table[1:] + table[:-1]) / 2).contiguous()
    for e in range(E):
        v = torch.randn((rows, cols), generator=g, device="cuda", dtype=BF16)
        if c["form"] == "int":
            code = ((v * 2.5).round_().clamp_(-8, 7) + 8).to(torch.uint8)
        else:
            v *= 2
            code = torch.bucketize(v.abs(), middles).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        w[e] = code[:, 0::2] | (code[:, 1::2] << 4)
    if c["form"] == "int":
        s = (torch.rand((E, rows, cols // BLOCK), generator=g, device="cuda") + 0.5) * (cols ** -0.5 / 2.5)
        return w, s.to(BF16)
    # Biased exponents: 2^(s - 127), each a factor of 4 around the matrix's.
    mid = 127 + round(math.log2(cols ** -0.5 / 2))
    s = torch.randint(mid - 1, mid + 2, (E, rows, cols // SMALL_BLOCK), generator=g, device="cuda")
    return w, s.to(torch.uint8)


def prepare(case, seed):
    c = case
    T = c["T"]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(c)
    if c["op"] == "norm":
        H = c["H"]
        s["x"] = torch.randn((T, H), generator=g, device="cuda").to(BF16)
        s["res"] = _stream_rows(c, g) if c["residual"] else None
        s["gain"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    elif c["op"] == "norm_grad":
        H = c["H"]
        s["h"] = _stream_rows(c, g)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["gain"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
        s["dy"] = torch.randn((T, H), generator=g, device="cuda").to(BF16)
        s["d_stream"] = torch.randn((T, H), generator=g, device="cuda").to(s["h"].dtype) if c["stream"] else None
    elif c["op"] in ("route", "route_grad"):
        s["logits"] = _logits(c, g)
        s["bias"] = 0.05 * torch.randn(c["E"], generator=g, device="cuda") if c["bias"] else None
        if c["op"] == "route_grad":
            s["idx"] = _select(s)
            s["d_w"] = torch.randn((T, c["K"]), generator=g, device="cuda")
    else:
        H, F, E, K = c["H"], c["F"], c["E"], c["K"]
        idx = torch.rand((T, E), generator=g, device="cuda").topk(K, dim=1).indices.contiguous()
        if c["drop"]:
            idx.view(-1)[torch.randperm(T * K, generator=g, device="cuda")[:_dropped(c)]] = -1
        s["idx"], s["w"] = idx, torch.softmax(torch.randn((T, K), generator=g, device="cuda"), dim=1)
        s["x"] = torch.randn((T, H), generator=g, device="cuda").to(BF16)
        s["w13"], s["w13_scales"] = _four_bit(c, g, 2 * F, H)
        s["w2"], s["w2_scales"] = _four_bit(c, g, H, F)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


def _quantise(v):
    """e4m3 values and scales = amax / 448 for each row and 128 channels."""
    b = v.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return (b / scale).flatten(-2).to(F8), scale.squeeze(-1)


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["residual"]:
        out["h"] = (h + s["res"].float()).to(s["res"].dtype)
        h = out["h"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    v = h * rstd.unsqueeze(1) * s["gain"].float()
    out["y"] = v.to(BF16)
    if s["fp8"]:
        out["y_fp8"], out["y_scales"] = _quantise(v)
    if s["save"]:
        out["rstd"] = rstd
    return out


def _plain_norm_grad(s):
    h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    a = dy * s["gain"].float()
    n = h * r
    d = r * (a - n * (a * n).mean(1, keepdim=True))
    if s["stream"]:
        d = d + s["d_stream"].float()
    out = dict(d_h=d.to(s["h"].dtype), d_gain=(dy * n).sum(0))
    if s["wide"]:
        out["d_x"] = d.to(BF16)
    return out


def _scores(s, dtype):
    """Scores of the experts in dtype; 0 for masked ones."""
    l = s["logits"].to(dtype)
    if s["sigmoid"]:
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    p = torch.exp(l - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _select(s):
    """Expert ids [T, K]: the largest of the allowed groups, ties to the lowest id; -1 where none is left.
    Without bias and sums of two the logits order as the scores do; with them the scores are taken in 64
    bits, as two may lie next to each other."""
    l, T, E, G, K = s["logits"], s["T"], s["E"], s["G"], s["K"]
    masked = torch.isinf(l)
    key = l
    if s["bias"] is not None or s["group_top"] > 1:
        key = _scores(s, F64)
        if s["bias"] is not None:
            key = key + s["bias"].double()
    key = torch.where(masked, -math.inf, key)
    if s["top_groups"] < G:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :s["group_top"]]
        group = torch.where(torch.isinf(best), 0.0, best).sum(2)
        group = torch.where(torch.isinf(best[:, :, 0]), -math.inf, group)
        chosen = group.sort(stable=True, dim=1, descending=True).indices[:, :s["top_groups"]]
        allowed = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, chosen, True)
        key = torch.where(allowed.repeat_interleave(E // G, 1), key, -math.inf)
    top = key.sort(stable=True, dim=1, descending=True)
    return torch.where(torch.isinf(top.values[:, :K]), -1, top.indices[:, :K]).contiguous()


def _plain_route(s):
    idx = _select(s)
    w = torch.gather(_scores(s, F32), 1, idx.clamp(min=0)) * (idx >= 0)
    if s["normalize"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    return dict(topk_idx=idx, topk_weights=2.5 * w)


def _plain_route_grad(s):
    idx = s["idx"]
    p = _scores(s, F32)
    lane = torch.gather(p, 1, idx.clamp(min=0)) * (idx >= 0)
    d = 2.5 * s["d_w"] * (idx >= 0)
    if s["normalize"]:
        total = lane.sum(1, keepdim=True) + TINY
        d = (d - (d * lane).sum(1, keepdim=True) / total) / total * (idx >= 0)
    ds = torch.zeros((s["T"], s["E"] + 1), device="cuda").scatter_(1, torch.where(idx < 0, s["E"], idx), d)[:, :s["E"]]
    if s["sigmoid"]:
        return ds * p * (1.0 - p)
    return p * (ds - (ds * p).sum(1, keepdim=True))


def _codes(w):
    """The 4-bit codes of packed bytes, column by column."""
    return torch.stack([w & 15, w >> 4], -1).flatten(-2)


def _wide(s, name, used):
    """The 32-bit values of the used experts' matrix `name`."""
    code, scales = _codes(s[name][used]), s[name + "_scales"][used]
    if s["form"] == "int":
        v, size, f = code.float() - 8.0, BLOCK, scales.float()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
        v, size, f = table[code.int()], SMALL_BLOCK, torch.exp2(scales.float() - 127.0)
    return (v.unflatten(-1, (-1, size)) * f.unsqueeze(-1)).flatten(-2)


def _plain_few(s):
    T, K, E = s["T"], s["K"], s["E"]
    # Routing weights [T, E] (repeated lanes add up), and the experts in use: at most T * K.
    lanes = torch.where(s["idx"] < 0, E, s["idx"])
    route = torch.zeros((T, E + 1), device="cuda").scatter_add_(1, lanes, s["w"])
    hits = torch.zeros(E + 1, device="cuda").index_add_(0, lanes.reshape(-1), torch.ones(T * K, device="cuda"))
    used = hits[:E].topk(min(E, T * K)).indices
    gu = torch.matmul(s["x"].float(), _wide(s, "w13", used).transpose(1, 2))  # [U, T, 2F]
    gate, up = gu[..., :s["F"]], gu[..., s["F"]:]
    act = gate / (1.0 + torch.exp(-gate)) * up * route[:, used].t().unsqueeze(-1)
    return torch.matmul(act, _wide(s, "w2", used).transpose(1, 2)).sum(0).to(BF16)


_PLAIN = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, route=_plain_route, route_grad=_plain_route_grad,
              few=_plain_few)


def _run_own(s):
    from combine_get_layout_amd import ep

    T, op = s["T"], s["op"]

    def new(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "norm":
        H = s["H"]
        shape = ep.make_shape(T, H, 1, 1, 1)
        out = dict(y=new(T, H))
        if s["residual"]:
            out["h"] = torch.empty_like(s["res"])
        if s["fp8"]:
            out["y_fp8"], out["y_scales"] = new(T, H, dtype=F8), new(T, H // BLOCK, dtype=F32)
        if s["save"]:
            out["rstd"] = new(T, dtype=F32)
        ep.ep_rms_norm(shape, s["x"], s["res"], ep.EP_STREAM_F32 if s["wide"] else ep.EP_STREAM_BF16, s["gain"], EPS,
                       out)
        return out
    if op == "norm_grad":
        H = s["H"]
        shape = ep.make_shape(T, H, 1, 1, 1)
        if "ws" not in s:  # a training program keeps its workspace
            s["ws"] = ep.alloc_norm_workspace(shape)
        out = dict(d_h=torch.empty_like(s["h"]), d_gain=new(H, dtype=F32))
        if s["wide"]:
            out["d_x"] = new(T, H)
        ep.ep_rms_norm_grad(shape, s["h"], ep.EP_STREAM_F32 if s["wide"] else ep.EP_STREAM_BF16, s["gain"], s["rstd"],
                            s["dy"], s["d_stream"], out["d_h"], out.get("d_x"), out["d_gain"], s["ws"])
        return out
    if op in ("route", "route_grad"):
        E, K = s["E"], s["K"]
        shape = ep.make_shape(T, 8, K, E, s["G"], s["G"])
        if "ws" not in s:
            s["ws"] = ep.alloc_workspace(shape)
        router = dict(score=ep.EP_SCORE_SIGMOID if s["sigmoid"] else ep.EP_SCORE_SOFTMAX, top_groups=s["top_groups"],
                      group_top=s["group_top"], normalize=s["normalize"], scale=2.5, bias=s["bias"])
        if op == "route":
            out = dict(topk_idx=new(T, K, dtype=torch.int64), topk_weights=new(T, K, dtype=F32))
            ep.ep_route(shape, s["logits"], router, out["topk_idx"], out["topk_weights"], s["ws"])
            return out
        d_logits = new(T, E, dtype=F32)
        ep.ep_route_grad(shape, s["logits"], router, s["idx"], s["d_w"], d_logits, ep.EP_GRAD_F32, s["ws"])
        return d_logits
    H, F, E, K = s["H"], s["F"], s["E"], s["K"]
    shape = ep.make_shape(T, H, K, E, 1)
    if "ws" not in s:
        s["ws"] = ep.alloc_few_w4_workspace(shape, F)
    out = new(T, H)
    experts = dict(F=F, form=ep.EP_W4_INT if s["form"] == "int" else ep.EP_W4_E2M1, w13=s["w13"],
                   w13_scales=s["w13_scales"], w2=s["w2"], w2_scales=s["w2_scales"])
    ep.ep_moe_few_w4(shape, dict(x=s["x"], topk_idx=s["idx"], topk_weights=s["w"]), experts, out, s["ws"])
    return out


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------

def _matrix64(s, name, e):
    w = s[name][e].long()
    code = torch.empty((w.shape[0], 2 * w.shape[1]), dtype=torch.long, device="cuda")
    code[:, 0::2], code[:, 1::2] = w % 16, w // 16
    if s["form"] == "int":
        return (code - 8).to(F64) * s[name + "_scales"][e].to(F64).repeat_interleave(BLOCK, 1)
    # Sign, two bits of exponent, one of fraction.
    ex, fr = code // 2 % 4, (code % 2).to(F64)
    v = torch.where(ex == 0, fr / 2, (1 + fr / 2) * 2.0 ** (ex - 1).to(F64)) * (1 - 2 * (code // 8)).to(F64)
    return v * torch.pow(2.0, s[name + "_scales"][e].to(F64) - 127).repeat_interleave(SMALL_BLOCK, 1)


def _scores64(s):
    l = s["logits"].to(F64)
    return torch.sigmoid(l) if s["sigmoid"] else torch.nan_to_num(torch.softmax(l, 1), nan=0.0)


def _first_largest(v):
    """Largest value of each row and the first column that has it."""
    top = v.max(1, keepdim=True).values
    return top.squeeze(1), torch.where(v == top, torch.arange(v.shape[1], device="cuda"), v.shape[1]).min(1).values


def _select64(s, p):
    """The K experts one after the other, the groups before them."""
    T, E, G = s["T"], s["E"], s["G"]
    t = torch.arange(T, device="cuda")
    key = s["logits"].to(F64) if s["bias"] is None and s["group_top"] == 1 else p.clone()
    if s["bias"] is not None:
        key += s["bias"].to(F64)
    key[s["logits"] == -math.inf] = -math.inf
    if s["top_groups"] < G:
        rest, total = key.reshape(T * G, E // G).clone(), torch.zeros(T * G, dtype=F64, device="cuda")
        empty = (rest == -math.inf).all(1)
        for _ in range(s["group_top"]):
            top, at = _first_largest(rest)
            total += torch.where(top == -math.inf, 0.0, top)
            rest[torch.arange(T * G, device="cuda"), at.clamp(max=E // G - 1)] = -math.inf
        total = torch.where(empty, -math.inf, total).reshape(T, G)
        left = torch.ones((T, G), dtype=torch.bool, device="cuda")
        for _ in range(s["top_groups"]):
            top, at = _first_largest(total)
            left[t, at] = False
            total[t, at] = -math.inf
        key.reshape(T, G, E // G)[left] = -math.inf
    idx = torch.empty((T, s["K"]), dtype=torch.long, device="cuda")
    for k in range(s["K"]):
        top, at = _first_largest(key)
        idx[:, k] = torch.where(top == -math.inf, -1, at)
        key[t, at] = -math.inf
    return idx


def exact(case, seed):
    s = prepare(case, seed)
    op, T = s["op"], s["T"]
    if op == "norm":
        h = s["x"].to(F64)
        out = {}
        if s["residual"]:
            h = h + s["res"].to(F64)
            out["h"] = h
            # The norm is of the stored values.
            h = h.float().to(s["res"].dtype).to(F64)
        rstd = (h.pow(2).sum(1) / s["H"] + EPS) ** -0.5
        y = torch.einsum("th,t,h->th", h, rstd, s["gain"].to(F64))
        out["y"] = y
        if s["fp8"]:
            amax = y.reshape(T, -1, BLOCK).abs().amax(2)
            scale = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
            out["y_fp8"], out["y_scales"] = y / scale.repeat_interleave(BLOCK, 1), scale
        if s["save"]:
            out["rstd"] = rstd
        return out
    if op == "norm_grad":
        h, dy, r, g = s["h"].to(F64), s["dy"].to(F64), s["rstd"].to(F64).view(-1, 1), s["gain"].to(F64)
        dot = torch.einsum("th,th,h->t", h, dy, g).view(-1, 1)
        d = r * g * dy - r ** 3 / s["H"] * dot * h
        if s["stream"]:
            d = d + s["d_stream"].to(F64)
        out = dict(d_h=d, d_gain=torch.einsum("th,th,t->h", dy, h, s["rstd"].to(F64)))
        if s["wide"]:
            out["d_x"] = d
        return out
    if op in ("route", "route_grad"):
        p = _scores64(s)
        idx = _select64(s, p) if op == "route" else s["idx"]
        t, k = (idx >= 0).nonzero(as_tuple=True)
        e = idx[t, k]
        lane = torch.zeros(idx.shape, dtype=F64, device="cuda")
        lane[t, k] = p[t, e]
        if op == "route":
            w = lane / (lane.sum(1, keepdim=True) + TINY) if s["normalize"] else lane
            return dict(topk_idx=None, topk_weights=2.5 * w)
        g = 2.5 * s["d_w"].to(F64)
        if s["normalize"]:
            D = lane.sum(1, keepdim=True) + TINY
            g = g / D - (g * lane).sum(1, keepdim=True) / D ** 2
        ds = torch.zeros((T, s["E"]), dtype=F64, device="cuda")
        ds[t, e] = g[t, k]
        if s["sigmoid"]:
            return ds * torch.sigmoid(s["logits"].to(F64)) * torch.sigmoid(-s["logits"].to(F64))
        return p * ds - p * torch.einsum("te,te->t", ds, p).view(-1, 1)
    F = s["F"]
    out = torch.zeros((T, s["H"]), dtype=F64, device="cuda")
    x = s["x"].to(F64)
    for e in range(s["E"]):
        t, k = (s["idx"] == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        w13 = _matrix64(s, "w13", e)
        gate, up = x[t] @ w13[:F].T, x[t] @ w13[F:].T
        y = (gate * torch.sigmoid(gate) * up) @ _matrix64(s, "w2", e).T
        out.index_add_(0, t, y * s["w"][t, k].to(F64).unsqueeze(1))
    return out
