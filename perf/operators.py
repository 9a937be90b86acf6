"""Measured cases of the expert operators: the whole layer for a few tokens,
the grouped expert products, the fused SwiGLU product with its 8-bit
checkpoint, its gradient, and the weight gradient.

A case is a dict of plain values. `prepare` makes what a program holds before
the call (rows grouped by expert, offsets, weights), `run` makes one pass:
with `own` false in elementary torch operations in 32 bits, with `own` true by
the library's entry points. `exact` states the same results in 64 bits.
"""
import math

import torch

own = False

BF16, F8, F32, F64 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64
E4M3_MAX = 448.0
BLOCK = 128  # channels that share a scale


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    def few(name, T, H, F, E, K, fp8=False, drop=0.0):
        return dict(name=name, op="few", T=T, H=H, F=F, E=E, K=K, fp8=fp8, drop=drop, skew=0.0)

    def rows(name, op, T, H, F, E, K, drop=0.0, skew=0.0, **more):
        return dict(name=name, op=op, T=T, H=H, F=F, E=E, K=K, drop=drop, skew=skew, **more)

    return [
        # One token through a small model: launch latency decides.
        few("few_tiny", 1, 256, 512, 16, 2),
        # One decoded token through a large layer: eight experts' weights are streamed once.
        few("few_one", 1, 7168, 2048, 64, 8),
        # A small decode batch with skipped lanes and sizes that fill no tile.
        few("few_odd", 13, 2056, 712, 40, 3, drop=0.1),
        # A decode batch that touches nearly every expert, weights held in 8 bits.
        few("few_batch_fp8", 32, 7168, 2048, 64, 8, fp8=True),
        # Gate/up product of a small training batch with its 8-bit checkpoint.
        rows("swiglu_small", "swiglu", 128, 256, 512, 16, 2, save=True),
        # Gate/up product of a training step (4,096 tokens, top-8), checkpoint kept.
        rows("swiglu_large", "swiglu", 4096, 7168, 2048, 32, 8, save=True),
        # Down product of the same step: rows of 2,048 to rows of 7,168.
        rows("matmul_down", "matmul", 4096, 7168, 2048, 32, 8, back=False, gate_up=False),
        # Gradient of the gate/up product's rows, skewed routing, odd sizes, empty experts.
        rows("matmul_back_odd", "matmul", 1000, 2056, 712, 48, 6, drop=0.05, skew=1.2, back=True, gate_up=True),
        # SwiGLU gradient from the 8-bit checkpoint of a training step.
        rows("grad_large", "grad", 4096, 7168, 2048, 32, 8),
        # The same for a small batch with skipped lanes: latency counts.
        rows("grad_small", "grad", 333, 1024, 640, 16, 3, drop=0.1),
        # Weight gradient of the gate/up product from the dispatched 8-bit rows.
        rows("wgrad_fp8", "wgrad", 4096, 7168, 2048, 32, 8, fp8=True, wide=False, gate_up=True),
        # Weight gradient kept in 32 bits, skewed routing, empty experts, odd sizes.
        rows("wgrad_wide_odd", "wgrad", 1500, 1032, 520, 48, 4, skew=1.2, fp8=False, wide=True, gate_up=False),
    ]


def draw(rng):
    def log(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["few", "few", "swiglu", "matmul", "grad", "wgrad"])
    K = rng.randint(1, 8)
    E = rng.randint(max(8, K), 64)
    drop = rng.choice([0.0, 0.0, 0.1])
    if op == "few":
        fp8 = rng.random() < 0.4
        step = BLOCK if fp8 else 8
        T = log(1, 128, 1)
        drop = drop if T * K >= 16 else 0.0
        return dict(op=op, T=T, H=log(256, 7168, step), F=log(128, 2048, step), E=E, K=K,
                    fp8=fp8, drop=drop, skew=0.0)
    H, F = log(256, 4096, 8), log(128, 2048, 8)
    T = log(16, 4096, 1)
    skew = rng.choice([0.0, 0.0, 1.2])
    if skew:
        T = min(T, 2048)
    c = dict(op=op, T=T, H=H, F=F, E=E, K=K, drop=drop, skew=skew)
    if op == "swiglu":
        c["save"] = rng.random() < 0.7
        if c["save"]:
            c["F"] = log(128, 2048, BLOCK)
    elif op == "matmul":
        c["back"], c["gate_up"] = rng.random() < 0.5, rng.random() < 0.5
    elif op == "grad":
        c["F"] = log(128, 2048, BLOCK)
    else:
        c["fp8"] = rng.random() < 0.5
        c["wide"], c["gate_up"] = not c["fp8"] and rng.random() < 0.5, rng.random() < 0.5
        if c["fp8"]:
            c["H"] = log(256, 4096, BLOCK)
            c["gate_up"] = True
    return c


def work(c):
    T, H, F, E, K = c["T"], c["H"], c["F"], c["E"], c["K"]
    lanes = T * K - _dropped(c)
    if c["op"] == "few":
        # Expected experts that T tokens with K distinct lanes each reach.
        used = E * (1.0 - (1.0 - K * (1.0 - c["drop"]) / E) ** T)
        per = 3 * F * H * (1.0 + 4.0 / BLOCK if c["fp8"] else 2.0)
        return dict(bytes=used * per + T * H * 4 + T * K * 12, flops=lanes * 6 * F * H)
    if c["op"] == "swiglu":
        kept = 2 * F + 8 * F / BLOCK if c["save"] else 0
        return dict(bytes=lanes * (2 * H + 2 * F + kept) + E * 4 * F * H, flops=lanes * 4 * F * H)
    if c["op"] == "matmul":
        k, n = _product_dims(c)
        return dict(bytes=lanes * 2 * (k + n) + E * 2 * k * n, flops=lanes * 2 * k * n)
    if c["op"] == "grad":
        return dict(bytes=lanes * (2 * F + 8 * F / BLOCK + 2 * F + 4 * F + 2 * F) + T * K * 12,
                    flops=lanes * 20 * F)
    k, n = _wgrad_dims(c)
    x = k * (1 + 4.0 / BLOCK) if c["fp8"] else 2 * k
    return dict(bytes=lanes * (2 * n + x) + E * n * k * (4 if c["wide"] else 2), flops=lanes * 2 * k * n)


def _dropped(c):
    """Skipped lanes."""
    return int(c["T"] * c["K"] * c["drop"])


def _product_dims(c):
    """(contracted, produced) sizes of a matmul case."""
    k, n = (c["H"], 2 * c["F"]) if c["gate_up"] else (c["F"], c["H"])
    return (n, k) if c["back"] else (k, n)


def _wgrad_dims(c):
    """(columns, rows) of each expert's weight."""
    return (c["H"], 2 * c["F"]) if c["gate_up"] else (c["F"], c["H"])


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _routing(c, g):
    """Distinct experts per token (by the largest keys; skew > 0: a Zipf law by
    Gumbel keys), some lanes skipped (-1), and softmax weights."""
    T, E, K = c["T"], c["E"], c["K"]
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7)
    keys = -torch.log(-torch.log(u))
    if c["skew"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        keys = keys - c["skew"] * torch.log(rank)
    idx = keys.topk(K, dim=1).indices.contiguous()
    if c["drop"]:
        idx.view(-1)[torch.randperm(T * K, generator=g, device="cuda")[:_dropped(c)]] = -1
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), dim=1)
    return idx, w


def _expand(idx, E):
    """expert_offsets [E+1], expert_slot [T, K] and each expand row's expert."""
    flat = idx.reshape(-1)
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    slot = torch.empty_like(flat)
    slot[order] = torch.arange(flat.numel(), device="cuda")
    slot = torch.where(flat < 0, -1, slot).to(torch.int32).reshape(idx.shape)
    return offsets, slot, int(counts.sum()), int(counts.max())


def prepare(case, seed):
    c = case
    T, H, F, E, K = c["T"], c["H"], c["F"], c["E"], c["K"]
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        t = torch.randn(shape, generator=g, device="cuda", dtype=BF16)
        return t.mul_(scale) if scale != 1.0 else t

    def eight(rows, cols, scale):
        """e4m3 values and one scale for each row and 128 channels."""
        q = (torch.randn((rows, cols), generator=g, device="cuda", dtype=BF16) * 64).clamp_(-E4M3_MAX, E4M3_MAX).to(F8)
        s = (torch.rand((rows, cols // BLOCK), generator=g, device="cuda") + 0.5) * (scale / 64)
        return q, s

    idx, w = _routing(c, g)
    s = dict(c, idx=idx, w=w)
    if c["op"] == "few":
        s["x"] = normal(T, H)
        if c["fp8"]:
            q, sc = eight(E * 2 * F, H, H ** -0.5)
            s["w13"], s["w13_scales"] = q.view(E, 2 * F, H), sc.view(E, 2 * F, H // BLOCK)
            q, sc = eight(E * H, F, F ** -0.5)
            s["w2"], s["w2_scales"] = q.view(E, H, F), sc.view(E, H, F // BLOCK)
        else:
            s["w13"], s["w2"] = normal(E, 2 * F, H, scale=H ** -0.5), normal(E, H, F, scale=F ** -0.5)
        return s
    s["offsets"], s["slot"], s["rows"], s["most"] = _expand(idx, E)
    N = s["rows"]
    if c["op"] == "swiglu":
        s["x"], s["w13"] = normal(N, H), normal(E, 2 * F, H, scale=H ** -0.5)
    elif c["op"] == "matmul":
        k, n = _product_dims(c)
        s["x"] = normal(N, k)
        s["wt"] = normal(*((E, k, n) if c["back"] else (E, n, k)), scale=k ** -0.5)
    elif c["op"] == "grad":
        s["q"], s["scales"] = eight(N, 2 * F, 1.0)
        s["d_act"] = normal(N, F)
    else:
        k, n = _wgrad_dims(c)
        s["dy"] = normal(N, n)
        if c["fp8"]:
            s["x8"], s["x_scales"] = eight(N, k, 1.0)
        else:
            s["x"] = normal(N, k)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


def _wide(q, scales):
    """The 32-bit values of e4m3 rows with a scale for each 128 channels."""
    v = q.float().unflatten(-1, (-1, BLOCK)) * scales.unsqueeze(-1)
    return v.flatten(-2)


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _plain_few(s):
    T, K, E = s["T"], s["K"], s["E"]
    # Routing weights [T, E] (repeated lanes add up), and the experts in use: at most U.
    route = torch.zeros((T, E + 1), device="cuda").scatter_add_(1, torch.where(s["idx"] < 0, E, s["idx"]), s["w"])
    hits = torch.zeros(E + 1, device="cuda").index_add_(
        0, torch.where(s["idx"] < 0, E, s["idx"]).reshape(-1), torch.ones(T * K, device="cuda"))
    used = hits[:E].topk(min(E, T * K)).indices
    w13, w2 = s["w13"][used], s["w2"][used]
    if s["fp8"]:
        w13, w2 = _wide(w13, s["w13_scales"][used]), _wide(w2, s["w2_scales"][used])
    else:
        w13, w2 = w13.float(), w2.float()
    gu = torch.matmul(s["x"].float(), w13.transpose(1, 2))              # [U, T, 2F]
    act = _silu(gu[..., :s["F"]]) * gu[..., s["F"]:]
    act = act * route[:, used].t().unsqueeze(-1)
    return torch.matmul(act, w2.transpose(1, 2)).sum(0).to(BF16)


def _padded(s, x):
    """Rows of each expert side by side: [E, most, columns], zeros behind the last."""
    at = s["offsets"][:-1].long().unsqueeze(1) + torch.arange(s["most"], device="cuda")
    inside = at < s["offsets"][1:].unsqueeze(1)
    return x[at.clamp(max=max(s["rows"] - 1, 0))] * inside.unsqueeze(-1)


def _dense(s, y):
    """The rows of _padded, one after the other again."""
    i = torch.arange(s["rows"], device="cuda")
    e = torch.searchsorted(s["offsets"].long(), i, right=True) - 1
    return y[e, i - s["offsets"].long()[e]]


def _quantise(v):
    """e4m3 values and scales = amax / 448 for each row and 128 channels."""
    b = v.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return (b / scale).flatten(-2).to(F8), scale.squeeze(-1)


def _plain_swiglu(s):
    gu = _dense(s, torch.bmm(_padded(s, s["x"].float()), s["w13"].float().transpose(1, 2)))
    act = (_silu(gu[:, :s["F"]]) * gu[:, s["F"]:]).to(BF16)
    return (act, *_quantise(gu)) if s["save"] else (act,)


def _plain_matmul(s):
    w = s["wt"].float()
    return _dense(s, torch.bmm(_padded(s, s["x"].float()), w if s["back"] else w.transpose(1, 2))).to(BF16)


def _plain_grad(s):
    F, N = s["F"], s["rows"]
    lane = s["slot"].reshape(-1).long()
    row_w = torch.zeros(N + 1, device="cuda")
    row_w[torch.where(lane < 0, N, lane)] = s["w"].reshape(-1)
    row_w = row_w[:N].unsqueeze(1)
    gu = _wide(s["q"], s["scales"])
    g, u, d = gu[:, :F], gu[:, F:], s["d_act"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig * u
    d_gate = row_w * d * u * sig * (1.0 + g * (1.0 - sig))
    d_up = row_w * d * g * sig
    d_w = torch.cat([(d * act).sum(1), torch.zeros(1, device="cuda")])[lane].reshape(s["w"].shape)
    return torch.cat([d_gate, d_up], 1).to(BF16), (row_w * act).to(BF16), d_w


def _plain_wgrad(s):
    x = _wide(s["x8"], s["x_scales"]) if s["fp8"] else s["x"].float()
    dw = torch.bmm(_padded(s, s["dy"].float()).transpose(1, 2), _padded(s, x))
    return dw if s["wide"] else dw.to(BF16)


_PLAIN = dict(few=_plain_few, swiglu=_plain_swiglu, matmul=_plain_matmul, grad=_plain_grad, wgrad=_plain_wgrad)


def _run_own(s):
    from combine_get_layout_amd import ep

    T, H, F, E, K = s["T"], s["H"], s["F"], s["E"], s["K"]
    shape = ep.make_shape(T, H, K, E, 1)
    if s["op"] == "few":
        if "ws" not in s:  # a decoding program keeps its workspace
            s["ws"] = ep.alloc_few_workspace(shape, F)
        out = torch.empty((T, H), dtype=BF16, device="cuda")
        experts = dict(F=F)
        if s["fp8"]:
            experts.update(w13_fp8=s["w13"], w13_scales=s["w13_scales"], w2_fp8=s["w2"], w2_scales=s["w2_scales"])
        else:
            experts.update(w13=s["w13"], w2=s["w2"])
        ep.ep_moe_few(shape, dict(x=s["x"], topk_idx=s["idx"], topk_weights=s["w"]), experts, out, s["ws"])
        return out
    if "ws" not in s:
        s["ws"] = ep.alloc_workspace(shape)
    layout, N = dict(expert_offsets=s["offsets"], expert_slot=s["slot"]), s["rows"]
    if s["op"] == "swiglu":
        act = torch.empty((N, F), dtype=BF16, device="cuda")
        if not s["save"]:
            ep.ep_expert_swiglu(shape, layout, s["x"], N, s["w13"], F, act, None, None, s["ws"])
            return (act,)
        q = torch.empty((N, 2 * F), dtype=F8, device="cuda")
        scales = torch.empty((N, 2 * F // BLOCK), dtype=F32, device="cuda")
        ep.ep_expert_swiglu(shape, layout, s["x"], N, s["w13"], F, act, q, scales, s["ws"])
        return act, q, scales
    if s["op"] == "matmul":
        k, n = _product_dims(s)
        y = torch.empty((N, n), dtype=BF16, device="cuda")
        order = ep.EP_WEIGHT_KN if s["back"] else ep.EP_WEIGHT_NK
        ep.ep_expert_matmul(shape, layout, s["x"], N, k, s["wt"], n, order, y, s["ws"])
        return y
    if s["op"] == "grad":
        d_gu = torch.empty((N, 2 * F), dtype=BF16, device="cuda")
        act = torch.empty((N, F), dtype=BF16, device="cuda")
        d_w = torch.empty((T, K), dtype=F32, device="cuda")
        ep.ep_swiglu_grad(shape, layout, F, s["q"], s["scales"], s["d_act"], N, s["w"], d_gu, act, d_w, s["ws"])
        return d_gu, act, d_w
    k, n = _wgrad_dims(s)
    dw = torch.empty((E, n, k), dtype=F32 if s["wide"] else BF16, device="cuda")
    rows = dict(x_fp8=s["x8"], x_scales=s["x_scales"]) if s["fp8"] else dict(x=s["x"])
    ep.ep_expert_wgrad(shape, layout, s["dy"], N, n, rows, k, dw, ep.EP_GRAD_F32 if s["wide"] else ep.EP_GRAD_BF16,
                       s["ws"])
    return dw


# --------------------------------------------------------------------------
# The definition in 64 bits, expert by expert
# --------------------------------------------------------------------------

def _wide64(q, scales):
    return q.to(F64) * scales.to(F64).repeat_interleave(BLOCK, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op, F, E = s["op"], s["F"], s["E"]
    if op == "few":
        out = torch.zeros((s["T"], s["H"]), dtype=F64, device="cuda")
        x = s["x"].to(F64)
        for e in range(E):
            t, k = (s["idx"] == e).nonzero(as_tuple=True)
            if not len(t):
                continue
            w13 = _wide64(s["w13"][e], s["w13_scales"][e]) if s["fp8"] else s["w13"][e].to(F64)
            w2 = _wide64(s["w2"][e], s["w2_scales"][e]) if s["fp8"] else s["w2"][e].to(F64)
            gate, up = x[t] @ w13[:F].T, x[t] @ w13[F:].T
            y = (gate * torch.sigmoid(gate) * up) @ w2.T
            out.index_add_(0, t, y * s["w"][t, k].to(F64).unsqueeze(1))
        return out
    off = s["offsets"].tolist()
    parts = [slice(off[e], off[e + 1]) for e in range(E)]
    if op == "swiglu":
        gu = torch.cat([s["x"][p].to(F64) @ s["w13"][e].to(F64).T for e, p in enumerate(parts)])
        act = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        if not s["save"]:
            return (act,)
        amax = gu.reshape(len(gu), -1, BLOCK).abs().amax(2)
        scale = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
        return act, (gu / scale.repeat_interleave(BLOCK, 1)).float().to(F8), scale
    if op == "matmul":
        return torch.cat([s["x"][p].to(F64) @ (s["wt"][e].to(F64) if s["back"] else s["wt"][e].to(F64).T)
                          for e, p in enumerate(parts)])
    if op == "grad":
        gu, d = _wide64(s["q"], s["scales"]), s["d_act"].to(F64)
        t, k = (s["slot"] >= 0).nonzero(as_tuple=True)
        row = s["slot"][t, k].long()
        w = torch.zeros((s["rows"], 1), dtype=F64, device="cuda")
        w[row, 0] = s["w"][t, k].to(F64)
        g, u = gu[:, :F], gu[:, F:]
        sg = torch.sigmoid(g)
        a = g * sg * u
        d_w = torch.zeros(s["w"].shape, dtype=F64, device="cuda")
        d_w[t, k] = (d * a).sum(1)[row]
        return torch.cat([w * d * u * (sg + g * sg * (1 - sg)), w * d * g * sg], 1), w * a, d_w
    x = _wide64(s["x8"], s["x_scales"]) if s["fp8"] else s["x"].to(F64)
    return torch.stack([s["dy"][p].to(F64).T @ x[p] for p in parts])
