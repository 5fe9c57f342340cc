"""Measured cases of the routing, router-gradient and dense-projection operators.

Five calls of the MoE layer's library, as a user of the layer makes them:

  route          moe_route_grouped           scores, bias for balance, groups, top-k, gate weights
  route_bwd      moe_route_grouped_backward  gradient of the gate weights to the router's logits
  combine_bwd    moe_combine_backward        gradient of the top-k reduce to the expert rows and the gate weights
  linear         moe_linear                  dense product with bias, activation and residual (shared expert, projections)
  linear_bwd     moe_linear_backward         its gradients to the input, the weights and the bias

With `own` false, `run` computes the same in elementary torch operations (fp32;
fp64 where a border between two scores decides an index).
"""
import math

import torch

own = False

DEV = "cuda:0"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One token of a serving step through a 256-expert router (the decode layer's): balance bias, 8 groups of 32, 4 kept.
        dict(name="route_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, masked=False),
        # A whole prompt batch through the same router.
        dict(name="route_prompt", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, masked=False),
        # A ragged, padded batch: softmax scores, 8 groups of 20, padding rows without any expert, experts masked out.
        dict(name="route_padded", op="route", T=4099, E=160, k=6, score="softmax", bias=False, n_group=8, topk_group=3,
             group_top=1, renorm=False, scale=16.0, masked=True),
        # Training step of the 256-expert router: only the chosen experts' logits get a gradient.
        dict(name="route_bwd_sigmoid", op="route_bwd", T=16384, E=256, k=8, score="sigmoid", renorm=True, scale=2.5,
             masked=False),
        # Training step of the fine-grained layer's router: full softmax, every logit gets a gradient.
        dict(name="route_bwd_softmax", op="route_bwd", T=8192, E=64, k=6, score="softmax", renorm=False, scale=1.0,
             masked=True),
        # Gradient of the combine at the Mixtral-shaped layer: every slot local.
        dict(name="combine_bwd_all", op="combine_bwd", T=4096, H=4096, k=2, E=8, E_loc=8, tile_m=256),
        # The same on an expert-parallel share: most slots belong to other ranks, a ragged number of tokens.
        dict(name="combine_bwd_share", op="combine_bwd", T=5003, H=4096, k=8, E=64, E_loc=8, tile_m=256),
        # Serving, one token: the shared expert's gate and up products at the decode layer's width.
        dict(name="linear_token", op="linear", M=1, N=2048, K=7168, act="swiglu", bias=False, residual=False,
             out="bf16", save=False),
        # Shared expert's down product on a ragged batch, added to the routed experts' fp32 output.
        dict(name="linear_residual", op="linear", M=4099, N=2048, K=2816, act="none", bias=False, residual=True,
             out="fp32", save=False),
        # A dense SwiGLU layer of the Mixtral shape, pre-activations kept for the backward pass: the largest.
        dict(name="linear_swiglu", op="linear", M=4096, N=14336, K=4096, act="swiglu", bias=False, residual=False,
             out="bf16", save=True),
        # Training: the fine-grained layer's shared expert (two units wide), gate and up.
        dict(name="linear_bwd_swiglu", op="linear_bwd", M=8192, N=2816, K=2048, act="swiglu", bias=False, out="bf16"),
        # Training on odd sizes: a GELU projection with bias.
        dict(name="linear_bwd_ragged", op="linear_bwd", M=1003, N=1001, K=1416, act="gelu", bias=True, out="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "combine_bwd", "linear", "linear", "linear", "linear_bwd", "linear_bwd"])
    if op in ("route", "route_bwd"):
        if rng.random() < 0.5:  # the usual routers
            E, n_group = rng.choice([(8, 1), (16, 1), (64, 1), (64, 8), (128, 8), (128, 1), (256, 8), (256, 1), (512, 16)])
        else:  # any number of groups of any size
            n_group = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
            E = n_group * rng.randint(2, max(2, min(64, 640 // n_group)))
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(12, topk_group * (E // n_group)))
        c = dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.3)
        if op == "route":
            c.update(bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group, group_top=rng.choice([1, 2]))
        return c
    if op == "combine_bwd":
        E, k = rng.choice([(8, 2), (64, 6), (64, 8), (32, 4), (16, 1), (48, 5)])
        return dict(op=op, T=_log(rng, 1, 8192), H=4 * _log(rng, 16, 1100), k=k, E=E, E_loc=rng.choice([E, E // 2, E // 8]),
                    tile_m=rng.choice([16, 64, 256]))
    while True:
        M, N, K = _log(rng, 1, 8192), _log(rng, 1, 8192), 8 * _log(rng, 1, 1024)
        if 2.0 * M * N * K <= 2.0e11:
            break
    if rng.random() < 0.5 and N > 64:
        N = N // 64 * 64
    act = rng.choice(["none", "gelu", "silu", "swiglu", "swiglu"])
    c = dict(op=op, M=M, N=N, K=K, act=act, bias=rng.random() < 0.4, out=rng.choice(["bf16", "fp32"]))
    if op == "linear":
        c.update(residual=rng.random() < 0.4, save=rng.random() < 0.3)
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _logits(c, g):
    """Router logits, a little wider than N(0, 1); masked: one token in ten is padding (no expert), one expert in twenty is barred."""
    x = torch.randn(c["T"], c["E"], device=DEV, generator=g) * 1.5
    if c["masked"]:
        barred = torch.rand(c["T"], c["E"], device=DEV, generator=g) < 0.05
        barred |= torch.rand(c["T"], 1, device=DEV, generator=g) < 0.1
        x.masked_fill_(barred, float("-inf"))
    return x


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "route":
        return dict(logits=_logits(c, g), bias=torch.randn(c["E"], device=DEV, generator=g) * 0.1 if c["bias"] else None)
    if c["op"] == "route_bwd":
        x = _logits(c, g)
        v, i = torch.topk(x, c["k"], dim=1)
        return dict(logits=x, idx=torch.where(v > float("-inf"), i, -1).to(torch.int32).contiguous(),
                    d_w=torch.randn(c["T"], c["k"], device=DEV, generator=g))
    if c["op"] == "combine_bwd":
        T, H, k, E, El, tm = (c[n] for n in ("T", "H", "k", "E", "E_loc", "tile_m"))
        e = torch.rand(T, E, device=DEV, generator=g).topk(k, dim=1).indices.reshape(-1)  # distinct experts of a token
        order = torch.argsort(e * (T * k) + torch.arange(T * k, device=DEV))              # by expert, then token
        counts = torch.bincount(e, minlength=E)
        pad = (counts + tm - 1) // tm * tm
        first, off = torch.cumsum(counts, 0) - counts, torch.cumsum(pad, 0) - pad
        es = e[order]
        row = off[es] + torch.arange(T * k, device=DEV) - first[es]
        inv = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
        inv[order] = torch.where(es < El, row, -1).to(torch.int32)                        # this share owns experts 0 .. E_loc - 1
        R = T * min(k, El) + El * (tm - 1)
        w = torch.softmax(torch.randn(T, k, device=DEV, generator=g), dim=1)
        return dict(d_out=torch.randn(T, H, device=DEV, generator=g), y=torch.randn(R, H, device=DEV, generator=g),
                    inv=inv.view(T, k), w=w)
    M, N, K, act = c["M"], c["N"], c["K"], c["act"]
    odt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    rb = lambda *s, std=1.0: (torch.randn(*s, device=DEV, generator=g) * std).to(torch.bfloat16)  # noqa: E731
    d = dict(x=rb(M, K), w=rb(N, K, std=0.02), w_up=rb(N, K, std=0.02) if act == "swiglu" else None)
    bias = torch.randn(N, device=DEV, generator=g) * 0.1 if c["bias"] else None
    bias_up = torch.randn(N, device=DEV, generator=g) * 0.1 if c["bias"] and act == "swiglu" else None
    if c["op"] == "linear":
        d.update(bias=bias, bias_up=bias_up, residual=torch.randn(M, N, device=DEV, generator=g).to(odt) if c["residual"] else None)
        return d
    d["d_out"] = torch.randn(M, N, device=DEV, generator=g).to(odt)
    z = lambda w, b: (d["x"].float() @ w.float().T + (0.0 if b is None else b)).to(torch.bfloat16)  # noqa: E731
    d["z"] = z(d["w"], bias) if act != "none" else None
    d["z_up"] = z(d["w_up"], bias_up) if act == "swiglu" else None
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    c = case
    # What a serving or training program keeps from call to call: output buffers, and the operator's workspace.
    if c["op"] == "route":
        d["topk_idx"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV)
        d["topk_w"] = torch.empty(c["T"], c["k"], device=DEV)
    elif c["op"] == "route_bwd":
        d["d_logits"] = torch.empty(c["T"], c["E"], device=DEV)
    elif c["op"] == "combine_bwd":
        d["d_y"] = torch.zeros_like(d["y"])  # rows behind an expert's last token are never written
        d["d_topk_w"] = torch.empty(c["T"], c["k"], device=DEV)
    elif c["op"] == "linear":
        odt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        d["out"] = torch.empty(c["M"], c["N"], dtype=odt, device=DEV)
        z = c["save"] and c["act"] != "none"
        d["z"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device=DEV) if z else None
        d["z_up"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device=DEV) if z and c["act"] == "swiglu" else None
    else:
        dual = c["act"] == "swiglu"
        d["d_x"], d["d_w"] = torch.empty_like(d["x"]), torch.empty_like(d["w"])
        d["d_w_up"] = torch.empty_like(d["w"]) if dual else None
        d["d_bias"] = torch.empty(c["N"], device=DEV) if c["bias"] else None
        d["d_bias_up"] = torch.empty(c["N"], device=DEV) if c["bias"] and dual else None
    if own:
        from mixture_experts_layer_moe_amd import ffi
        if c["op"] == "linear":
            d["ws"] = ffi.alloc_linear_workspace(c["M"], c["N"], c["K"], c["act"], DEV)
        elif c["op"] == "linear_bwd":
            d["ws"] = ffi.alloc_linear_backward_workspace(c["M"], c["N"], c["K"], c["act"], DEV)
    return d


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        from mixture_experts_layer_moe_amd import ffi
        if c["op"] == "route":
            return ffi.moe_route_grouped(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_group=c["n_group"],
                                         topk_group=c["topk_group"], group_top=c["group_top"], renormalize=c["renorm"],
                                         scale=c["scale"], topk_idx=s["topk_idx"], topk_w=s["topk_w"])
        if c["op"] == "route_bwd":
            return ffi.moe_route_grouped_backward(s["logits"], s["idx"], s["d_w"], score=c["score"],
                                                  renormalize=c["renorm"], scale=c["scale"], d_logits=s["d_logits"])
        if c["op"] == "combine_bwd":
            return ffi.moe_combine_backward(s["d_out"], s["y"], s["inv"], s["w"], d_y_perm=s["d_y"], d_topk_w=s["d_topk_w"])
        if c["op"] == "linear":
            out = ffi.moe_linear(s["x"], s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"], act=c["act"],
                                 residual=s["residual"], out=s["out"], z=s["z"], z_up=s["z_up"], ws=s["ws"])
            return [t for t in (out, s["z"], s["z_up"]) if t is not None]
        ffi.moe_linear_backward(s["d_out"], s["x"], s["w"], w_up=s["w_up"], act=c["act"], z=s["z"], z_up=s["z_up"],
                                d_x=s["d_x"], d_w=s["d_w"], d_w_up=s["d_w_up"], d_bias=s["d_bias"],
                                d_bias_up=s["d_bias_up"], ws=s["ws"])
        return [t for t in (s["d_x"], s["d_w"], s["d_w_up"], s["d_bias"], s["d_bias_up"]) if t is not None]
    return {"route": _route, "route_bwd": _route_bwd, "combine_bwd": _combine_bwd, "linear": _linear,
            "linear_bwd": _linear_bwd}[c["op"]](s, c)


_BIG = torch.finfo(torch.float32).max


def _scores(logits, score):
    """Scores in 64 bits (their order decides indices) and which experts can be chosen at all."""
    x = logits.double()
    ok = x > float("-inf")  # false for NaN too
    x = torch.where(ok, x, 0.0).clamp(max=_BIG)
    if score == "sigmoid":
        return torch.where(ok, 1.0 / (1.0 + torch.exp(-x)), 0.0), ok
    top = torch.where(ok, x, -_BIG).amax(dim=1, keepdim=True)
    e = torch.where(ok, torch.exp(x - top), 0.0)
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300), ok


def _route(s, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    p, ok = _scores(s["logits"], c["score"])
    key = p if s["bias"] is None else p + s["bias"].double()
    none = float("-inf")
    key = torch.where(ok, key, none)
    best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[:, :, :c["group_top"]]
    gkey = torch.where(best > none, best, 0.0).sum(dim=2)
    gkey = torch.where(best[:, :, 0] > none, gkey, none)
    kept = torch.sort(gkey, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
    keep = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, kept, True)
    key = torch.where(keep.repeat_interleave(E // G, dim=1), key, none)
    v, i = torch.sort(key, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    has = v > none
    w = torch.where(has, p.gather(1, i), 0.0)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return torch.where(has, i, -1).to(torch.int32), (w * c["scale"]).float()


def _route_bwd(s, c):
    p, _ = _scores(s["logits"], c["score"])
    p = p.float()
    has = s["idx"] >= 0
    i = s["idx"].clamp(min=0).long()
    ps = torch.where(has, p.gather(1, i), 0.0)
    g = torch.where(has, s["d_w"] * c["scale"], 0.0)
    if c["renorm"]:
        total = ps.sum(dim=1, keepdim=True).clamp(min=1e-30)
        q = ps / total
        d = (g - (q * g).sum(dim=1, keepdim=True))
        d = q * d * (1.0 - ps) if c["score"] == "sigmoid" else q * d
        out = torch.zeros_like(s["logits"])
    elif c["score"] == "sigmoid":
        d = g * ps * (1.0 - ps)
        out = torch.zeros_like(s["logits"])
    else:
        d = g * ps
        out = -p * d.sum(dim=1, keepdim=True)
    return out.scatter_add_(1, i, torch.where(has, d, 0.0))


def _combine_bwd(s, c):
    inv = s["inv"].long()
    has = inv >= 0
    rows = inv.clamp(min=0)
    y = s["y"][rows.view(-1)].view(c["T"], c["k"], c["H"])
    d_w = torch.where(has, (y * s["d_out"][:, None, :]).sum(dim=2), 0.0)
    d_y = torch.zeros_like(s["y"])
    t = torch.arange(c["T"], device=inv.device)[:, None].expand(-1, c["k"])[has]
    d_y[inv[has]] = s["d_out"][t] * s["w"][has][:, None]
    return d_y, d_w


def _linear(s, c):
    x = s["x"].float()
    z = x @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    u = None
    if c["act"] == "swiglu":
        u = x @ s["w_up"].float().T
        if s["bias_up"] is not None:
            u = u + s["bias_up"]
        y = z * torch.sigmoid(z) * u
    elif c["act"] == "silu":
        y = z * torch.sigmoid(z)
    elif c["act"] == "gelu":
        y = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    else:
        y = z
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = [y.to(s["out"].dtype)]
    if s["z"] is not None:
        out.append(z.to(torch.bfloat16))
    if s["z_up"] is not None:
        out.append(u.to(torch.bfloat16))
    return out


def _linear_bwd(s, c):
    g, x, w = s["d_out"].float(), s["x"].float(), s["w"].float()
    z = s["z"].float() if s["z"] is not None else None
    if c["act"] == "swiglu":
        u, sg = s["z_up"].float(), torch.sigmoid(z)
        dz, du = g * u * (sg * (1.0 + z * (1.0 - sg))), g * (z * sg)
        wu = s["w_up"].float()
        out = [(dz @ w + du @ wu), dz.T @ x, du.T @ x]
        sums = [dz.sum(dim=0), du.sum(dim=0)]
    else:
        if c["act"] == "silu":
            sg = torch.sigmoid(z)
            dz = g * (sg * (1.0 + z * (1.0 - sg)))
        elif c["act"] == "gelu":
            dz = g * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
        else:
            dz = g
        out = [dz @ w, dz.T @ x]
        sums = [dz.sum(dim=0)]
    return [t.to(torch.bfloat16) for t in out] + (sums if c["bias"] else [])


# ---------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": 4 * c["T"] * c["E"] + 8 * c["T"] * c["k"] + (4 * c["E"] if c["bias"] else 0), "flops": 8 * c["T"] * c["E"]}
    if c["op"] == "route_bwd":
        dense = c["score"] == "softmax" and not c["renorm"]  # else only the chosen logits have to be read
        return {"bytes": 4 * c["T"] * (c["E"] + (c["E"] if dense else c["k"]) + 2 * c["k"]), "flops": 6 * c["T"] * (c["E"] if dense else c["k"])}
    if c["op"] == "combine_bwd":
        rows = c["T"] * c["k"] * c["E_loc"] / c["E"]
        return {"bytes": 4 * c["H"] * (c["T"] + 2 * rows) + 12 * c["T"] * c["k"], "flops": 3 * rows * c["H"]}
    M, N, K = c["M"], c["N"], c["K"]
    mats, ob = (2 if c["act"] == "swiglu" else 1), (2 if c["out"] == "bf16" else 4)
    kept = mats if c["act"] != "none" else 0
    if c["op"] == "linear":
        b = 2 * M * K + 2 * mats * N * K + M * N * ob * (2 if c["residual"] else 1)
        b += (2 * M * N * kept if c["save"] else 0) + (4 * N * mats if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K * mats}
    b = M * N * ob + 2 * M * N * kept + 4 * M * K + 4 * mats * N * K + (4 * N * mats if c["bias"] else 0)
    return {"bytes": b, "flops": 4 * M * N * K * mats}


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    f = torch.float64
    if c["op"] == "route":
        # Only the weights are computed numbers; the definition over the chosen set, found by ranking with counts.
        x = d["logits"].to(f)
        free = ~(torch.isnan(x) | torch.isneginf(x))
        lse = torch.logsumexp(torch.where(free, x, torch.tensor(-1e300, dtype=f, device=x.device)), dim=1, keepdim=True)
        p = torch.where(free, torch.sigmoid(x) if c["score"] == "sigmoid" else torch.exp(x - lse), torch.zeros((), dtype=f, device=x.device))
        key = p.clone()
        if d["bias"] is not None:
            key += d["bias"].to(f)
        key[~free] = -1e18
        Eg = c["E"] // c["n_group"]
        top = key.view(c["T"], c["n_group"], Eg).topk(c["group_top"], dim=2).values
        gk = torch.where(top > -1e17, top, torch.zeros((), dtype=f, device=x.device)).sum(2)
        gk[top[:, :, 0] < -1e17] = -1e18
        number = torch.arange(c["n_group"], device=x.device)
        ahead = (gk[:, None, :] > gk[:, :, None]) | ((gk[:, None, :] == gk[:, :, None]) & (number[None, None, :] < number[None, :, None]))
        drop = ahead.sum(2) >= c["topk_group"]
        key[drop.repeat_interleave(Eg, dim=1)] = -1e18
        v, i = key.topk(c["k"], dim=1)
        w = torch.where(v > -1e17, p.gather(1, i), torch.zeros((), dtype=f, device=x.device))
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(w))
        return None, w * c["scale"]
    if c["op"] == "route_bwd":
        x = torch.where(torch.isneginf(d["logits"]), torch.tensor(-1e6, device=DEV), d["logits"]).to(f).requires_grad_()
        has = d["idx"] >= 0
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1)
        w = torch.where(has, p.gather(1, d["idx"].clamp(min=0).long()), torch.zeros((), dtype=f, device=x.device))
        if c["renorm"]:
            w = w / torch.where(has.any(1, keepdim=True), w.sum(1, keepdim=True), torch.ones((), dtype=f, device=x.device))
        return torch.autograd.grad((w * c["scale"] * torch.where(has, d["d_w"].to(f), torch.zeros((), dtype=f, device=x.device))).sum(), x)[0]
    if c["op"] == "combine_bwd":
        if c["T"] * c["k"] * c["H"] > 3e8:
            return None
        flat = d["inv"].view(-1).long()
        pair = torch.nonzero(flat >= 0).view(-1)
        g = d["d_out"].to(f)[pair // c["k"]]
        d_y = torch.zeros(d["y"].shape, dtype=f, device=DEV)
        d_y.index_copy_(0, flat[pair], g * d["w"].to(f).view(-1)[pair][:, None])
        d_w = torch.zeros(c["T"] * c["k"], dtype=f, device=DEV)
        d_w[pair] = torch.linalg.vecdot(g, d["y"].to(f)[flat[pair]])
        return d_y, d_w.view(c["T"], c["k"])
    x, w = d["x"].to(f), d["w"].to(f)
    wu = d["w_up"].to(f) if d["w_up"] is not None else None
    norm_cdf = lambda t: 0.5 * torch.erfc(-t / math.sqrt(2.0))  # noqa: E731
    if c["op"] == "linear":
        z = torch.nn.functional.linear(x, w, None if d["bias"] is None else d["bias"].to(f))
        u = torch.nn.functional.linear(x, wu, None if d["bias_up"] is None else d["bias_up"].to(f)) if wu is not None else None
        y = {"none": lambda: z.clone(), "gelu": lambda: z * norm_cdf(z), "silu": lambda: z / (1 + torch.exp(-z)),
             "swiglu": lambda: z / (1 + torch.exp(-z)) * u}[c["act"]]()
        if d["residual"] is not None:
            y += d["residual"].to(f)
        kept = [z, u] if c["act"] == "swiglu" else [z] if c["act"] != "none" else []
        return [y] + (kept if c["save"] else [])
    g = d["d_out"].to(f)
    z = d["z"].to(f).requires_grad_() if d["z"] is not None else None
    if c["act"] == "swiglu":
        u = d["z_up"].to(f).requires_grad_()
        dz, du = torch.autograd.grad((torch.nn.functional.silu(z) * u * g).sum(), (z, u))
        return [torch.mm(dz, w) + torch.mm(du, wu), torch.mm(dz.T, x), torch.mm(du.T, x)] + ([dz.sum(0), du.sum(0)] if c["bias"] else [])
    dz = g
    if c["act"] != "none":
        y = torch.nn.functional.silu(z) if c["act"] == "silu" else torch.nn.functional.gelu(z)
        dz = torch.autograd.grad((y * g).sum(), z)[0]
    return [torch.mm(dz, w), torch.mm(dz.T, x)] + ([dz.sum(0)] if c["bias"] else [])
