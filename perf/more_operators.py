"""Cases that measure a block's operators between its matrix products, each in a plain form and through the library.

drop   dropout from a counter-based generator, with or without a residual added: forward, backward, or both
route  routing of tokens to experts: weights, experts, places in the experts' order, and the gradient of the logits
rows   rows to the experts and back: dispatch, weighted combine, and their backward passes
gn     group norm with an activation, channels last: forward, backward (with the weight's and bias's gradients), or both
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def f32(x):
    """x rounded to float32, as the library takes its scalars."""
    return float(torch.tensor(x, dtype=torch.float32))


GN_EPS = f32(1e-5)
LOW = 0xFFFFFFFF


# ---------------------------------------------------------------- cases

def listed():
    return [
        # an adapter's hidden rows of a few tokens: launch latency counts
        {"name": "drop_small", "op": "drop", "rows": 48, "width": 768, "type": "f32", "p": 0.1, "residual": True, "dir": "fwd"},
        # an odd width in half precision, forward and backward
        {"name": "drop_odd", "op": "drop", "rows": 4099, "width": 1601, "type": "f16", "p": 0.25, "residual": False, "dir": "both"},
        # a training micro-batch of 32 K tokens: the residual stream's dropout and add
        {"name": "drop_large", "op": "drop", "rows": 32768, "width": 4096, "type": "bf16", "p": 0.1, "residual": True, "dir": "fwd"},
        # a few tokens being generated: weights and experts of each
        {"name": "route_decode", "op": "route", "tokens": 7, "experts": 64, "k": 6, "score": "softmax", "groups": 1, "top_groups": 1,
         "bias": False, "renorm": False, "type": "bf16", "padded": 0.0, "dir": "fwd"},
        # a training micro-batch over many experts in groups, balanced by a bias, padded tokens at its end
        {"name": "route_groups", "op": "route", "tokens": 8192, "experts": 256, "k": 8, "score": "sigmoid", "groups": 8, "top_groups": 4,
         "bias": True, "renorm": True, "type": "f32", "padded": 0.125, "dir": "both"},
        # 64 K tokens over 128 experts by softmax, as a large data-parallel batch routes them
        {"name": "route_large", "op": "route", "tokens": 65536, "experts": 128, "k": 8, "score": "softmax", "groups": 1, "top_groups": 1,
         "bias": False, "renorm": True, "type": "bf16", "padded": 0.0, "dir": "both"},
        # a few generated tokens' rows joined again after the experts
        {"name": "rows_decode", "op": "rows", "tokens": 5, "width": 4096, "k": 4, "experts": 64, "type": "bf16", "padded": 0.0, "dir": "combine"},
        # an odd width in full precision, there and back
        {"name": "rows_odd", "op": "rows", "tokens": 2051, "width": 1601, "k": 3, "experts": 24, "type": "f32", "padded": 0.125, "dir": "both"},
        # a training micro-batch of 8 K tokens, eight experts each, there and back
        {"name": "rows_large", "op": "rows", "tokens": 8192, "width": 4096, "k": 8, "experts": 128, "type": "bf16", "padded": 0.0, "dir": "both"},
        # every head of a few thousand tokens normalised by itself
        {"name": "gn_heads", "op": "gn", "samples": 4096, "positions": 1, "channels": 4096, "groups": 64, "type": "bf16", "weight": "f32",
         "act": "none", "dir": "fwd"},
        # odd lengths and a group width off the 16-byte grid, forward and backward
        {"name": "gn_odd", "op": "gn", "samples": 3, "positions": 1021, "channels": 330, "groups": 30, "type": "f32", "weight": "f32",
         "act": "silu", "dir": "both"},
        # a training micro-batch of sixteen sequences, backward
        {"name": "gn_bwd_large", "op": "gn", "samples": 16, "positions": 4096, "channels": 1024, "groups": 32, "type": "bf16", "weight": "f32",
         "act": "silu", "dir": "bwd"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["drop", "route", "rows", "gn"])
    kind = rng.choice(["f32", "f16", "bf16"])
    size = SIZE[kind]
    if op == "drop":
        width = _log(rng, 48, 8192)
        width = width if rng.random() < 0.4 else (width + 7) // 8 * 8
        way = rng.choice(["fwd", "bwd", "both"])
        # a pass in full precision, or in both directions, gets as many fewer rows
        most = 32768 * 4096 * 2 // (size * width) // (2 if way == "both" else 1)
        return {"op": op, "rows": _log(rng, 1, min(32768, most)), "width": width, "type": kind, "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                "residual": rng.random() < 0.5, "dir": way}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4 if groups == 1 else 2, 512 // groups)
        top = 1 if groups == 1 else rng.randint(1, groups)
        k = rng.randint(1, min(16, experts // groups * top))
        most = min(65536, 65536 * 128 * 8 // (experts * k) * 2 // size, 65536 * 128 * 2 // (experts * size))
        return {"op": op, "tokens": _log(rng, 1, max(2, most)), "experts": experts, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "groups": groups, "top_groups": top, "bias": rng.random() < 0.5, "renorm": rng.random() < 0.5, "type": kind,
                "padded": rng.choice([0.0, 0.125]), "dir": rng.choice(["fwd", "both"])}
    if op == "rows":
        width = _log(rng, 48, 8192)
        width = width if rng.random() < 0.4 else (width + 7) // 8 * 8
        k = rng.randint(1, 8)
        most = min(32768, 8192 * 4096 * 8 * 2 // (size * width * (k + 1)))
        return {"op": op, "tokens": _log(rng, 1, most), "width": width, "k": k, "experts": k * _log(rng, 1, 16), "type": kind,
                "padded": rng.choice([0.0, 0.125]), "dir": rng.choice(["dispatch", "combine", "both"])}
    groups = _log(rng, 1, 64)
    channels = groups * _log(rng, 2, 4096 // groups)
    if rng.random() < 0.6:
        channels = (channels + 8 * groups - 1) // (8 * groups) * 8 * groups
    way = rng.choice(["fwd", "bwd", "both"])
    # a pass in full precision, or in both directions, gets as much less
    most = max(1, 16 * 4096 * 1024 * 2 * 3 // (channels * size * (5 if way == "both" else 3)))
    positions = _log(rng, 1, min(8192, most))
    return {"op": op, "samples": _log(rng, 1, max(1, min(4096, most // positions))), "positions": positions, "channels": channels, "groups": groups,
            "type": kind, "weight": rng.choice(["f32", kind]), "act": rng.choice(["none", "silu"]), "dir": way}


def pad(case):
    """How many of the last tokens are padding."""
    return int(case["tokens"] * case["padded"])


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind = TYPES[case["type"]]
    normal = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    state = {"case": case}
    if case["op"] == "drop":
        rows, width = case["rows"], case["width"]
        state.update(x=normal(rows, width).to(kind), residual=(2 * normal(rows, width)).to(kind) if case["residual"] else None,
                     dy=normal(rows, width).to(kind), p=f32(case["p"]), seed=1000003 * seed + (seed << 33), site=3,
                     steps=torch.tensor([100 + seed % 1000], dtype=torch.int32, device=DEV))
        if own:
            from adamw_optimizer_step_tensor_gb300 import FusedDropout
            state["drop"] = FusedDropout(state["p"], seed=state["seed"], site=state["site"])
        return state
    if case["op"] == "route":
        tokens, experts, k = case["tokens"], case["experts"], case["k"]
        logits = (1.5 * normal(tokens, experts)).to(kind)
        live = tokens - pad(case)
        logits[live:] = -math.inf              # padding: no expert may take it
        # the bias has moved by steps of 0.001 for a while
        steps = torch.randint(-40, 41, (experts,), device=DEV, generator=g)
        state.update(logits=logits, bias=steps.float() * 0.001 if case["bias"] else None, dweights=normal(tokens, k))
        if own:
            from adamw_optimizer_step_tensor_gb300 import FusedRouter
            state["router"] = FusedRouter(tokens, experts, k, score=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                                          group_score="top2", renormalise=case["renorm"])
        return state
    if case["op"] == "rows":
        tokens, width, k, experts = case["tokens"], case["width"], case["k"], case["experts"]
        ids = torch.rand(tokens, experts, device=DEV, generator=g).argsort(1)[:, :k]
        ids[tokens - pad(case):] = experts     # padding sorts behind every expert
        order = ids.flatten().argsort(stable=True)
        slots = torch.empty(tokens * k, dtype=torch.int64, device=DEV)
        slots[order] = torch.arange(tokens * k, device=DEV)
        slots = slots.view(tokens, k)
        live = tokens - pad(case)
        slots[live:] = -1
        weights = torch.softmax(normal(tokens, k), 1)
        weights[live:] = 0
        state.update(slots=slots.to(torch.int32), weights=weights, x=normal(tokens, width).to(kind))
        if case["dir"] != "dispatch":
            state["ys"] = normal(tokens * k, width).to(kind)
        if case["dir"] == "both":
            state["dy"], state["dxs"] = normal(tokens, width).to(kind), normal(tokens * k, width).to(kind)
            state["dys"] = torch.zeros(tokens * k, width, dtype=kind, device=DEV)
        if case["dir"] != "combine":
            state["xs"] = torch.zeros(tokens * k, width, dtype=kind, device=DEV)
        if own:
            from adamw_optimizer_step_tensor_gb300 import FusedRouter
            state["router"] = FusedRouter(tokens, experts, k)
        return state
    n, length, channels, groups, wkind = case["samples"], case["positions"], case["channels"], case["groups"], TYPES[case["weight"]]
    # channels have means and scales of their own
    x = (normal(n, length, channels) * (0.5 + torch.rand(channels, device=DEV, generator=g)) + 0.5 * normal(channels)).to(kind)
    state.update(x=x, weight=(1 + 0.1 * normal(channels)).to(wkind), bias=(0.1 * normal(channels)).to(wkind))
    if case["dir"] != "fwd":
        state["dy"] = normal(n, length, channels).to(kind)
    if case["dir"] == "bwd":                     # the forward pass left these
        xg = x.float().view(n, length, groups, channels // groups)
        state["mean"] = xg.mean((1, 3))
        state["rstd"] = 1 / torch.sqrt((xg - state["mean"][:, None, :, None]).square().mean((1, 3)) + GN_EPS)
    if own:
        from adamw_optimizer_step_tensor_gb300 import FusedGroupNorm
        state["norm"] = FusedGroupNorm(channels, groups, max_samples=n, eps=GN_EPS, activation=case["act"])
    return state


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return {"drop": _drop, "route": _route, "rows": _rows, "gn": _gn}[case["op"]](s, case)


def _philox(blocks, step, site, seed):
    """Four 32-bit words (in int64) for each counter in ``blocks``: Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw 2011)."""
    c = [blocks & LOW, blocks >> 32, (step.long() & LOW).expand(blocks.shape), torch.full_like(blocks, site)]
    k0, k1 = seed & LOW, seed >> 32 & LOW
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & LOW) ^ c[1] ^ k0, b & LOW, (a >> 32 & LOW) ^ c[3] ^ k1, a & LOW]
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return c


def _keep(s, n):
    words = _philox(torch.arange((n + 3) // 4, device=DEV), s["steps"], s["site"], s["seed"])
    return torch.stack(words, 1).flatten()[:n] >= round(s["p"] * 2 ** 32)


def _drop(s, case):
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    out = []
    if own:
        if fwd:
            out.append(s["drop"].forward(s["x"], s["steps"], s["residual"]))
        if bwd:
            out.append(s["drop"].backward(s["dy"], s["steps"]))
        return out
    x, scale = s["x"], f32(1 / (1 - s["p"]))
    keep = _keep(s, x.numel()).view(x.shape)
    zero = torch.zeros((), device=DEV)
    if fwd:
        y = torch.where(keep, x.float() * scale, zero)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out.append(y.to(x.dtype))
    if bwd:
        out.append(torch.where(keep, s["dy"].float() * scale, zero).to(x.dtype))
    return out


def _route(s, case):
    both = case["dir"] == "both"
    if own:
        out = s["router"].route(s["logits"], s["bias"])
        return (*out, s["router"].backward(s["dweights"], s["logits"], out[1])) if both else out
    tokens, experts, k, groups = case["tokens"], case["experts"], case["k"], case["groups"]
    z = s["logits"].double()                    # in 64 bits: experts' scores may lie close to one another
    there = z > -math.inf
    if case["score"] == "softmax":
        e = torch.where(there, torch.exp(z - z.max(1, keepdim=True).values), torch.zeros_like(z))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1 / (1 + torch.exp(-z))
    low = torch.full_like(z, -math.inf)
    key = torch.where(there, score if s["bias"] is None else score + s["bias"].double(), low)
    if s["bias"] is None and groups == 1:
        key = z                                  # the scores' order
    if groups > 1:
        two = key.view(tokens, groups, -1).sort(dim=2, descending=True).values[:, :, :2]
        of_group = two.sum(2)
        best = of_group.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        chosen = torch.zeros(tokens, groups, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        key = torch.where(chosen.repeat_interleave(experts // groups, 1), key, low)
    top = key.sort(dim=1, descending=True, stable=True)
    ids = top.indices[:, :k]
    live = top.values[:, :k] > -math.inf
    zero = torch.zeros((), dtype=z.dtype, device=DEV)
    w = torch.where(live, score.gather(1, ids), zero)
    total = w.sum(1, keepdim=True).clamp(min=1e-300)
    if case["renorm"]:
        w = w / total
    of = torch.where(live, ids, torch.full_like(ids, experts)).flatten()
    order = of.sort(dim=0, stable=True).indices
    slots = torch.empty_like(of)
    slots[order] = torch.arange(of.numel(), device=DEV)
    slots = torch.where(live, slots.view(tokens, k), torch.full_like(ids, -1))
    starts = (of[:, None] < torch.arange(experts + 1, device=DEV)).sum(0) if of.numel() < 1 << 16 else torch.cat(
        [torch.zeros(1, dtype=torch.int64, device=DEV), torch.bincount(of, minlength=experts + 1)[:experts].cumsum(0)])
    out = (w.float(), torch.where(live, ids, torch.full_like(ids, -1)).int(), slots.int(), starts.int())
    if not both:
        return out
    dw = s["dweights"].double()
    dz = torch.zeros_like(z)
    chosen_score = torch.where(live, score.gather(1, ids), zero)
    if case["renorm"]:
        part = w * (dw - (dw * w).sum(1, keepdim=True))
        dz.scatter_(1, ids, part * (1 - chosen_score) if case["score"] == "sigmoid" else part)
    elif case["score"] == "sigmoid":
        dz.scatter_(1, ids, dw * w * (1 - w))
    else:
        dz.scatter_(1, ids, torch.where(live, dw, zero))
        dz = score * (dz - (dw * w).sum(1, keepdim=True))
    return (*out, dz.to(s["logits"].dtype))


def _rows(s, case):
    way = case["dir"]
    out = []
    if own:
        r = s["router"]
        if way != "combine":
            out.append(r.dispatch(s["x"], s["slots"], xs=s["xs"]))
        if way != "dispatch":
            out.append(r.combine(s["ys"], s["slots"], s["weights"]))
        if way == "both":
            out += r.combine_backward(s["dy"], s["ys"], s["slots"], s["weights"], dys=s["dys"])
            out.append(r.combine(s["dxs"], s["slots"]))
        return out
    slots, k = s["slots"].long(), case["k"]
    live = slots >= 0
    at = slots.clamp(min=0)
    if way != "combine":
        for j in range(k):
            s["xs"][slots[live[:, j], j]] = s["x"][live[:, j]]
        out.append(s["xs"])

    def join(rows, weights):
        y = torch.zeros(case["tokens"], case["width"], device=DEV)
        for j in range(k):
            w = live[:, j].float() if weights is None else weights[:, j]
            y += torch.where(live[:, j, None], rows[at[:, j]].float(), torch.zeros((), device=DEV)) * w[:, None]
        return y.to(rows.dtype)

    if way != "dispatch":
        out.append(join(s["ys"], s["weights"]))
    if way == "both":
        dy = s["dy"].float()
        dw = torch.zeros(case["tokens"], k, device=DEV)
        for j in range(k):
            m = live[:, j]
            s["dys"][slots[m, j]] = (dy[m] * s["weights"][m, j, None]).to(s["dys"].dtype)
            dw[:, j] = torch.where(m, (dy * s["ys"][at[:, j]].float()).sum(1), torch.zeros((), device=DEV))
        out += [s["dys"], dw, join(s["dxs"], None)]
    return out


def _gn(s, case):
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    out = []
    if own:
        norm = s["norm"]
        mean, rstd = (None, None) if fwd else (s["mean"], s["rstd"])
        if fwd:
            y, mean, rstd = norm.forward(s["x"], s["weight"], s["bias"])
            out += [y, mean, rstd]
        if bwd:
            out += norm.backward(s["dy"], s["x"], s["weight"], s["bias"], mean, rstd)
        return out
    n, length, channels, groups = case["samples"], case["positions"], case["channels"], case["groups"]
    kind, wkind = s["x"].dtype, s["weight"].dtype
    split = (n, length, groups, channels // groups)
    wide = lambda t: t[:, None, :, None]  # noqa: E731
    x = s["x"].float().view(split)
    if fwd:
        mean = x.mean((1, 3))
        rstd = 1 / torch.sqrt((x - wide(mean)).square().mean((1, 3)) + GN_EPS)
    else:
        mean, rstd = s["mean"], s["rstd"]
    xhat = ((x - wide(mean)) * wide(rstd)).view(n, length, channels)
    w = s["weight"].float()
    z = xhat * w + s["bias"].float()
    sig = 1 / (1 + torch.exp(-z)) if case["act"] == "silu" else None
    if fwd:
        out += [(z if sig is None else z * sig).to(kind), mean, rstd]
    if bwd:
        dz = s["dy"].float()
        if sig is not None:
            dz = dz * (sig * (1 + z * (1 - sig)))
        a, xg = (dz * w).view(split), xhat.view(split)
        dx = wide(rstd) * (a - wide(a.mean((1, 3))) - xg * wide((a * xg).mean((1, 3))))
        out += [dx.reshape(n, length, channels).to(kind), (dz * xhat).sum((0, 1)).to(wkind), dz.sum((0, 1)).to(wkind)]
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = SIZE[case["type"]]
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    if case["op"] == "drop":
        n = case["rows"] * case["width"]
        passes = (2 + case["residual"] if fwd else 0) + (2 if bwd else 0)
        return {"bytes": passes * n * size, "flops": (2 * n if fwd else 0) + (n if bwd else 0)}
    if case["op"] == "route":
        tokens, experts, k = case["tokens"], case["experts"], case["k"]
        moved = tokens * experts * size + 12 * tokens * k + 4 * (experts + 1) + (4 * experts if case["bias"] else 0)
        if bwd:
            moved += 8 * tokens * k + tokens * experts * size
            dense = case["score"] == "softmax" and not case["renorm"]
            moved += tokens * (experts if dense else k) * size
        return {"bytes": moved, "flops": tokens * experts * (8 if bwd else 4)}
    if case["op"] == "rows":
        row, k = case["width"] * size, case["k"]
        live = case["tokens"] - pad(case)
        one = live * row * (1 + k) + 4 * case["tokens"] * k
        zeros = pad(case) * row                  # a padded token's row comes out as zeros
        weights = 4 * case["tokens"] * k
        moved = {"dispatch": one, "combine": one + zeros + weights,
                 "both": 3 * one + 2 * zeros + 2 * weights + live * row * (1 + 2 * k) + 8 * case["tokens"] * k}[case["dir"]]
        return {"bytes": moved, "flops": live * k * case["width"] * {"dispatch": 0, "combine": 2, "both": 6}[case["dir"]]}
    n, wsize = case["samples"] * case["positions"] * case["channels"], SIZE[case["weight"]]
    stats = 8 * case["samples"] * case["groups"]
    moved = 2 * n * size + 2 * case["channels"] * wsize + stats if fwd else 0
    moved += 3 * n * size + 4 * case["channels"] * wsize + stats if bwd else 0
    act = 4 if case["act"] == "silu" else 0
    return {"bytes": moved, "flops": ((8 + act) * n if fwd else 0) + ((14 + 2 * act) * n if bwd else 0)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _mulhilo(a, b):
    """High and low halves of 32-bit products, by 16-bit pieces."""
    a0, a1, b0, b1 = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    mid = a1 * b0 + (a0 * b0 >> 16)
    low = (mid & 0xFFFF) + a0 * b1
    return a1 * b1 + (mid >> 16) + (low >> 16), (low << 16 | (a0 * b0 & 0xFFFF)) & LOW


def _mask(s, first, n):
    """Which of the elements first .. first + n - 1 are kept (first a multiple of four)."""
    x = torch.arange(first // 4, (first + n + 3) // 4, device=DEV)
    k = (s["seed"] % 2 ** 32, s["seed"] // 2 ** 32 % 2 ** 32)
    w0, w1 = x % 2 ** 32, x // 2 ** 32
    w2, w3 = torch.zeros_like(x) + int(s["steps"]), torch.zeros_like(x) + s["site"]
    for r in range(10):
        hi0, lo0 = _mulhilo(w0, 0xD2511F53)
        hi2, lo2 = _mulhilo(w2, 0xCD9E8D57)
        w0, w1, w2, w3 = (hi2 ^ w1 ^ ((k[0] + r * 0x9E3779B9) % 2 ** 32), lo2, hi0 ^ w3 ^ ((k[1] + r * 0xBB67AE85) % 2 ** 32), lo0)
    return (torch.stack((w0, w1, w2, w3), -1).view(-1)[:n].double() / 2 ** 32) >= s["p"]


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "drop":
        n, out = s["x"].numel(), []
        wide = d if n < 1 << 26 else torch.float32
        for name, on in (("x", case["dir"] != "bwd"), ("dy", case["dir"] != "fwd")):
            if not on:
                continue
            y = torch.empty(n, dtype=wide, device=DEV)
            src = s[name].view(-1)
            for at in range(0, n, 1 << 24):
                m = min(1 << 24, n - at)
                t = src[at:at + m].to(d) / (1 - s["p"]) * _mask(s, at, m)
                y[at:at + m] = t + s["residual"].view(-1)[at:at + m] if name == "x" and s["residual"] is not None else t
            out.append(y.view(s["x"].shape))
        return out
    if case["op"] == "route":
        tokens, experts, k, groups = case["tokens"], case["experts"], case["k"], case["groups"]
        z = s["logits"].to(d)
        live_rows = tokens - pad(case)
        score = torch.softmax(z[:live_rows], 1) if case["score"] == "softmax" else torch.sigmoid(z[:live_rows])
        key = score.cpu().numpy()
        if s["bias"] is not None:
            key = key + s["bias"].cpu().numpy().astype(np.float64)
        if groups > 1:
            by = key.reshape(live_rows, groups, experts // groups)
            of = np.sort(by, 2)[:, :, -2:].sum(2) if experts // groups > 1 else by[:, :, 0]
            allowed = np.argsort(np.argsort(-of, 1, kind="stable"), 1, kind="stable") < case["top_groups"]
            key = np.where(allowed[:, :, None], by, -np.inf).reshape(live_rows, experts)
        ids = np.full((tokens, k), -1, np.int64)
        ids[:live_rows] = np.argsort(-key, 1, kind="stable")[:, :k]
        flat = ids[:live_rows].reshape(-1)
        slots = np.full((tokens, k), -1, np.int64)
        place = np.empty(flat.size, np.int64)
        place[np.argsort(flat, kind="stable")] = np.arange(flat.size)
        slots[:live_rows] = place.reshape(live_rows, k)
        starts = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=experts))])
        at = torch.from_numpy(ids[:live_rows]).to(DEV)
        leaf = z[:live_rows].clone().requires_grad_()
        w = (torch.softmax(leaf, 1) if case["score"] == "softmax" else torch.sigmoid(leaf)).gather(1, at)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        weights = torch.zeros(tokens, k, dtype=d, device=DEV)
        weights[:live_rows] = w.detach()
        whole = [torch.from_numpy(a).to(DEV).to(torch.int32) for a in (ids, slots, starts)]
        if case["dir"] == "fwd":
            return (weights, *whole)
        dz = torch.zeros_like(z)
        if live_rows:
            dz[:live_rows] = torch.autograd.grad(w, leaf, s["dweights"][:live_rows].to(d))[0]
        return (weights, *whole, dz)
    if case["op"] == "rows":
        tokens, k, width, live = case["tokens"], case["k"], case["width"], case["tokens"] - pad(case)
        slots = s["slots"][:live].long()
        wide = d if tokens * k * width < 1 << 26 else torch.float32
        owner = torch.arange(live, device=DEV).repeat_interleave(k)[slots.flatten().argsort()]      # token of each row
        col = slots.flatten().argsort() % k

        def behind(rows):
            full = torch.zeros(tokens * k, width, dtype=rows.dtype, device=DEV)
            full[:live * k] = rows
            return full

        def total(rows, weights):
            y = torch.zeros(tokens, width, dtype=d, device=DEV)
            for at in range(0, live, 512):
                part = rows[slots[at:at + 512]].to(d)
                y[at:at + 512][:part.shape[0]] = part.sum(1) if weights is None else torch.einsum("tkd,tk->td", part, weights[at:at + 512][:part.shape[0]].to(d))
            return y

        out = []
        if case["dir"] != "combine":
            out.append(behind(s["x"][owner]))
        if case["dir"] != "dispatch":
            out.append(total(s["ys"], s["weights"]))
        if case["dir"] == "both":
            dys = torch.zeros(tokens * k, width, dtype=wide, device=DEV)
            dw = torch.zeros(tokens, k, dtype=d, device=DEV)
            for at in range(0, live * k, 4096):
                o, c = owner[at:at + 4096], col[at:at + 4096]
                dy = s["dy"][o].to(d)
                dys[at:at + 4096][:o.numel()] = (dy * s["weights"][o, c, None].to(d)).to(wide)
                dw[o, c] = torch.einsum("rd,rd->r", dy, s["ys"][at:at + 4096][:o.numel()].to(d))
            out += [dys, dw, total(s["dxs"], None)]
        return out
    n, length, channels, groups = case["samples"], case["positions"], case["channels"], case["groups"]
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    w, b, per = s["weight"].to(d), s["bias"].to(d), channels // groups
    wide = d if s["x"].numel() < 1 << 25 else torch.float32
    y, dx = (torch.empty(s["x"].shape, dtype=wide, device=DEV) if on else None for on in (fwd, bwd))
    mean, rstd = (torch.empty(n, groups, dtype=d, device=DEV) for _ in range(2))
    dw, db = (torch.zeros(channels, dtype=d, device=DEV) for _ in range(2))
    step = max(1, (1 << 24) // (length * channels))
    for at in range(0, n, step):
        x = s["x"][at:at + step].to(d)
        m = x.shape[0]
        if fwd:
            sums = torch.einsum("nlgc->ng", x.view(m, length, groups, per)) / (length * per)
            squares = torch.einsum("nlgc,nlgc->ng", x.view(m, length, groups, per), x.view(m, length, groups, per)) / (length * per)
            mean[at:at + m], rstd[at:at + m] = sums, (squares - sums * sums + GN_EPS).rsqrt()
        else:
            mean[at:at + m], rstd[at:at + m] = s["mean"][at:at + m].to(d), s["rstd"][at:at + m].to(d)
        of_channel = lambda t: t[at:at + m].repeat_interleave(per, 1)[:, None, :]  # noqa: B023, E731
        xhat = (x - of_channel(mean)) * of_channel(rstd)
        z = torch.addcmul(b, xhat, w)
        if fwd:
            y[at:at + m] = (torch.nn.functional.silu(z) if case["act"] == "silu" else z).to(wide)
        if bwd:
            dz = s["dy"][at:at + m].to(d)
            if case["act"] == "silu":
                dz = dz * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
            dw += torch.einsum("nlc,nlc->c", dz, xhat)
            db += torch.einsum("nlc->c", dz)
            a = torch.einsum("nlc,c->nc", dz, w).view(m, groups, per).sum(2) / (length * per)
            q = torch.einsum("nlc,nlc,c->nc", dz, xhat, w).view(m, groups, per).sum(2) / (length * per)
            dx[at:at + m] = ((dz * w - a.repeat_interleave(per, 1)[:, None] - xhat * q.repeat_interleave(per, 1)[:, None]) * of_channel(rstd)).to(wide)
    return ([y, mean, rstd] if fwd else []) + ([dx, dw, db] if bwd else [])
