"""Cases that measure the operators around the optimizer step, each in a plain form and through the library.

norm    global gradient norm over a plan's tensors with the scale that clips it; with ``step`` the clipped AdamW step too
logps   log-probability of the given token per row of logits (scoring by the old and the reference policy)
policy  clipped policy loss with a KL term: loss, log-probabilities and the gradient of the logits
pref    preference loss over chosen / rejected sequences: loss, rewards and the gradient of the logits
ln      layer norm: forward, backward (with the weight's and bias's gradients), or both
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def f32(x):
    """x rounded to float32, as the library takes its scalars."""
    return float(torch.tensor(x, dtype=torch.float32))


B1, B2, EPS, LR, WD, MAX_NORM = f32(0.9), f32(0.999), f32(1e-8), f32(1e-3), f32(0.1), f32(0.1)
LN_EPS = f32(1e-5)
CLIP_LO, CLIP_HI, KL = f32(0.2), f32(0.28), f32(0.05)
BETA, SMOOTH = f32(0.1), f32(0.05)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # GPT-2 small's parameter list (148 tensors, 124 M) as data-parallel training clips it each step
        {"name": "norm_gpt2_small", "op": "norm", "layers": 12, "width": 768, "vocab": 50257, "type": "bf16", "step": False},
        # a small model or adapter: launch latency counts; norm, clip and step
        {"name": "norm_step_small", "op": "norm", "layers": 2, "width": 96, "vocab": 1009, "type": "f32", "step": True},
        # mixed precision at 0.35 G parameters: loss-scaled fp16 grads, norm, clip and step
        {"name": "norm_step_medium_amp", "op": "norm", "layers": 24, "width": 1024, "vocab": 50257, "type": "f16", "step": True},
        # a sampler scoring the token it just drew, a few sequences at once
        {"name": "logps_decode", "op": "logps", "rows": 7, "vocab": 128256, "type": "bf16", "masked": 0.0},
        # a short completion of a small policy: latency
        {"name": "policy_short", "op": "policy", "rows": 24, "vocab": 32000, "type": "f16", "masked": 0.25},
        # GPT-2's odd vocabulary, where rows start off the 16-byte grid
        {"name": "policy_odd_vocab", "op": "policy", "rows": 4001, "vocab": 50257, "type": "bf16", "masked": 0.25},
        # a micro-batch of Llama-3's vocabulary: 8192 tokens, prompts masked
        {"name": "policy_llama3_vocab", "op": "policy", "rows": 8192, "vocab": 128256, "type": "bf16", "masked": 0.25},
        # two short pairs in full precision, odd vocabulary
        {"name": "pref_short", "op": "pref", "pairs": 2, "rows": 203, "vocab": 50257, "type": "f32", "masked": 0.25},
        # a preference micro-batch: 4 pairs of about 512 tokens a side
        {"name": "pref_llama3_vocab", "op": "pref", "pairs": 4, "rows": 4096, "vocab": 128256, "type": "bf16", "masked": 0.25},
        # the final norm while decoding a few tokens
        {"name": "ln_decode", "op": "ln", "rows": 5, "width": 4096, "type": "bf16", "weight": "bf16", "dir": "fwd"},
        # an odd width in full precision, forward and backward
        {"name": "ln_train_odd", "op": "ln", "rows": 4099, "width": 1601, "type": "f32", "weight": "f32", "dir": "both"},
        # a training micro-batch of 32 K tokens, fp32 weights under bf16 activations
        {"name": "ln_bwd_large", "op": "ln", "rows": 32768, "width": 4096, "type": "bf16", "weight": "f32", "dir": "bwd"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "logps", "policy", "pref", "ln"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        return {"op": op, "layers": rng.randint(1, 20), "width": 8 * _log(rng, 8, 128), "vocab": _log(rng, 500, 50257), "type": kind,
                "step": rng.random() < 0.5}
    if op == "ln":
        width = _log(rng, 48, 8192)
        width = width if rng.random() < 0.4 else (width + 7) // 8 * 8
        rows = _log(rng, 1, min(32768, 32768 * 4096 * 2 // (SIZE[kind] * width)))
        return {"op": op, "rows": rows, "width": width, "type": kind, "weight": rng.choice(["f32", kind]),
                "dir": rng.choice(["fwd", "bwd", "both"])}
    vocab = _log(rng, 500, 131072)
    vocab = vocab if rng.random() < 0.4 else (vocab + 63) // 64 * 64
    most = min(8192, (8192 if op != "pref" else 4096) * 128256 * 2 // (SIZE[kind] * vocab))
    case = {"op": op, "vocab": vocab, "type": kind, "masked": rng.choice([0.0, 0.25, 0.5])}
    if op == "pref":
        pairs = rng.randint(1, 8)
        case.update(pairs=pairs, rows=_log(rng, 4 * pairs, min(most, 1024 * pairs)))
    else:
        case["rows"] = _log(rng, 1, most)
    return case


def shapes(case):
    """Element counts of a decoder's parameter list, matrices (decayed) and vectors (not)."""
    d = case["width"]
    layer = [(d, False), (d, False), (3 * d * d, True), (3 * d, False), (d * d, True), (d, False),
             (d, False), (d, False), (4 * d * d, True), (4 * d, False), (4 * d * d, True), (d, False)]
    return [(case["vocab"] * d, True)] + layer * case["layers"] + [(d, False), (d, False)]


def hidden(case):
    """Which rows count for nothing: the last part of every stretch, as padding (as many of them whatever the seed)."""
    stretch = max(4, case["rows"] // 16)
    return [t % stretch >= stretch - int(case["masked"] * stretch) for t in range(case["rows"])]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    state = {"case": case}
    kind = TYPES[case["type"]]
    if case["op"] == "norm":
        sizes = shapes(case)
        starts, total = [], 0
        for n, _ in sizes:
            starts.append(total)
            total += (n + 127) // 128 * 128       # tensors start where an allocator would put them
        scale = 1024.0 if case["type"] == "f16" else 1.0
        grads, wd = torch.zeros(total, dtype=kind, device=DEV), torch.zeros(total, device=DEV)
        params = torch.zeros(total, device=DEV)
        for (n, decayed), at in zip(sizes, starts):
            # matrices' gradients are smaller than vectors'
            x = torch.randn(n, device=DEV, generator=g) * (scale * (1e-3 if decayed else 1e-2))
            grads[at:at + n] = x.to(kind)
            params[at:at + n] = torch.randn(n, device=DEV, generator=g) * 0.02
            if decayed:
                wd[at:at + n] = WD
        m = torch.zeros(total, device=DEV)
        v = torch.zeros(total, device=DEV)
        state.update(grads=grads, params=params, wd=wd, m=m, v=v, lr=torch.tensor([LR], device=DEV),
                     steps=torch.zeros(1, dtype=torch.int32, device=DEV), scale=torch.tensor([scale], device=DEV),
                     norm=torch.zeros(1, device=DEV), clip_scale=torch.zeros(1, device=DEV), found_inf=torch.zeros(1, device=DEV))
        if own:
            from adamw_optimizer_step_tensor_gb300 import FusedAdamW
            cut = [[x[at:at + n] for (n, _), at in zip(sizes, starts)] for x in (params, grads, m, v)]
            state["opt"] = FusedAdamW(*cut, [WD if decayed else 0.0 for _, decayed in sizes])
        return state
    if case["op"] == "ln":
        rows, width, wkind = case["rows"], case["width"], TYPES[case["weight"]]
        x = (torch.randn(rows, width, device=DEV, generator=g) * 1.5 + 0.25).to(kind)
        state.update(x=x, dy=torch.randn(rows, width, device=DEV, generator=g).to(kind),
                     weight=(1 + 0.1 * torch.randn(width, device=DEV, generator=g)).to(wkind),
                     bias=(0.1 * torch.randn(width, device=DEV, generator=g)).to(wkind))
        if case["dir"] == "bwd":                 # the forward pass left these
            xf = x.float()
            state["mean"] = xf.mean(1)
            state["rstd"] = 1 / torch.sqrt((xf - state["mean"][:, None]).square().mean(1) + LN_EPS)
        if own:
            from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm
            state["norm"] = FusedLayerNorm(width, eps=LN_EPS)
        return state
    rows, vocab = case["rows"], case["vocab"]
    logits = torch.empty(rows, vocab, dtype=kind, device=DEV)
    for at in range(0, rows, 1024):
        logits[at:at + 1024] = (2 * torch.randn(min(1024, rows - at), vocab, device=DEV, generator=g)).to(kind)
    labels = torch.randint(0, vocab - 8, (rows,), device=DEV, generator=g)
    # the taken token is mostly a likely one; the vocabulary's last columns are padding that is never produced
    at = torch.arange(rows, device=DEV)
    logits[at, labels] += (4 + 12 * torch.rand(rows, device=DEV, generator=g)).to(kind)
    logits[:, vocab - 8:] = -math.inf
    live = ~torch.tensor(hidden(case), device=DEV)
    labels[~live] = -100
    weights = live.float()
    normal = lambda: torch.randn(rows, device=DEV, generator=g)  # noqa: E731
    # fp16 gradients carry a loss scale
    state.update(logits=logits, labels=labels, dlogits=torch.empty_like(logits),
                 scale=torch.tensor([4096.0 if case["type"] == "f16" else 1.0], device=DEV))
    if case["op"] != "logps":
        logp = torch.cat([_logps(logits[k:k + 1024], labels[k:k + 1024])[0] for k in range(0, rows, 1024)])
    if case["op"] == "policy":
        # the policy moved a little since it sampled; no ratio sits right at a clip bound, where one rounding would decide
        delta = 0.15 * normal()
        for edge in (math.log(1 - CLIP_LO), math.log(1 + CLIP_HI)):
            off = delta - edge
            delta = torch.where(off.abs() < 1e-3, edge + torch.where(off < 0, -1e-3, 1e-3), delta)
        state.update(weights=weights / max(1.0, float(weights.sum())), advantages=normal() + 0.5, old=logp - delta, ref=logp + 0.2 * normal())
    if case["op"] == "pref":
        inner = torch.randperm(rows - 1, device=DEV, generator=g)[:2 * case["pairs"] - 1].sort().values + 1
        ends = torch.tensor([rows], device=DEV)
        state.update(weights=weights, ref=logp - 0.05 + 0.2 * normal(), starts=torch.cat([torch.zeros_like(ends), inner, ends]).to(torch.int32))
    if own:
        from adamw_optimizer_step_tensor_gb300 import FusedTokenLoss
        state["loss"] = FusedTokenLoss(rows, max_pairs=case.get("pairs", 0))
    return state


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    return {"norm": _norm, "ln": _ln, "logps": _score, "policy": _policy, "pref": _pref}[case["op"]](s, case)


def _norm(s, case):
    if own:
        s["opt"].grad_norm(s["norm"], max_norm=MAX_NORM, grad_scale=s["scale"], clip_scale=s["clip_scale"], found_inf=s["found_inf"])
        if case["step"]:
            s["opt"].step(s["lr"], s["steps"], betas=(B1, B2), eps=EPS, grad_scale=s["clip_scale"], found_inf=s["found_inf"])
        out = {k: s[k] for k in ("norm", "clip_scale", "found_inf")}
    else:
        g = s["grads"].float() / s["scale"]
        norm = g.square().sum().sqrt().reshape(1)
        coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        out = {"norm": norm, "clip_scale": s["scale"] / coef, "found_inf": 1 - torch.isfinite(norm).float()}
        if case["step"]:
            g = g * coef
            s["steps"] += 1
            t = s["steps"].float()
            s["m"].mul_(B1).add_(g * (1 - B1))
            s["v"].mul_(B2).add_(g.square() * (1 - B2))
            root = s["v"].sqrt() / (1 - B2 ** t.double()).sqrt().float() + EPS
            s["params"].copy_(s["params"] * (1 - LR * s["wd"]) - s["m"] / root * (LR / (1 - B1 ** t.double())).float())
    if case["step"]:
        out.update(params=s["params"], m=s["m"], v=s["v"])
    return out


def _logps(logits, labels):
    """(log-probability of the label and log of the sum of exponentials, 0 where there is no label; probabilities)"""
    z = logits.float()
    top = z.max(1).values
    e = torch.exp(z - top[:, None])
    total = e.sum(1)
    live = (labels >= 0) & (labels < z.shape[1])
    zy = z.gather(1, torch.where(live, labels, torch.zeros_like(labels))[:, None])[:, 0]
    logp = (zy - top) - torch.log(total)
    zero = torch.zeros_like(logp)
    return torch.where(live, logp, zero), torch.where(live, top + torch.log(total), zero), e / total[:, None]


def _dlogits(probs, labels, per_row, kind):
    live = (labels >= 0) & (per_row != 0)
    c = torch.where(live, per_row, torch.zeros_like(per_row))
    d = probs * -c[:, None]
    d.scatter_add_(1, torch.where(live, labels, torch.zeros_like(labels))[:, None], c[:, None])
    return d.to(kind)


def _score(s, case):
    if own:
        return s["loss"].logps(s["logits"], s["labels"])
    return _logps(s["logits"], s["labels"])[:2]


def _policy(s, case):
    if own:
        return s["loss"].policy(s["logits"], s["labels"], s["weights"], s["advantages"], s["old"], s["ref"], clip=(CLIP_LO, CLIP_HI),
                                kl_coef=KL, grad_scale=s["scale"], dlogits=s["dlogits"])
    logp, _, probs = _logps(s["logits"], s["labels"])
    a, w = s["advantages"], s["weights"]
    live = w != 0
    logp = torch.where(live, logp, torch.zeros_like(logp))
    ratio = torch.exp(logp - s["old"])
    bound = ratio.clamp(1 - CLIP_LO, 1 + CLIP_HI)
    clipped = bound * a < ratio * a
    back = s["ref"] - logp
    over = torch.exp(back)
    policy = -torch.where(clipped, bound, ratio) * a
    kl = over - back - 1
    zero = torch.zeros_like(w)
    policy_term, kl_term = torch.where(live, w * policy, zero).sum(), torch.where(live, w * kl, zero).sum()
    stats = torch.stack([policy_term + KL * kl_term, policy_term, kl_term, torch.where(live & clipped, w, zero).sum()])
    per_row = w * (torch.where(clipped, zero, -a * ratio) + KL * (1 - over))
    return stats, logp, _dlogits(probs, s["labels"], per_row * s["scale"], s["logits"].dtype)


def _pref(s, case):
    if own:
        return s["loss"].preference(s["logits"], s["labels"], s["weights"], s["ref"], s["starts"], beta=BETA, label_smoothing=SMOOTH,
                                    grad_scale=s["scale"], dlogits=s["dlogits"])
    logp, _, probs = _logps(s["logits"], s["labels"])
    pairs, rows, w = case["pairs"], case["rows"], s["weights"]
    live = w != 0
    logp = torch.where(live, logp, torch.zeros_like(logp))
    gap = torch.where(live, w * (logp - s["ref"]), torch.zeros_like(w))
    at = torch.arange(rows, device=w.device)
    inside = (at >= s["starts"][:-1, None]) & (at < s["starts"][1:, None])       # [2 pairs, rows]
    rewards = BETA * torch.where(inside, gap, torch.zeros_like(gap)).sum(1)
    margin = rewards[:pairs] - rewards[pairs:]
    minus_log_sig = lambda d: torch.log(1 + torch.exp(-d.abs())) + (-d).clamp(min=0)  # noqa: E731
    losses = (1 - SMOOTH) * minus_log_sig(margin) + SMOOTH * minus_log_sig(-margin)
    stats = torch.stack([losses.mean(), (margin > 0).float().mean(), rewards[:pairs].mean(), rewards[pairs:].mean()])
    slope = (SMOOTH - 1 / (1 + torch.exp(margin))) * (BETA / pairs)              # d loss / d (a chosen sequence's sum)
    per_row = w * (inside.float() * torch.cat([slope, -slope])[:, None]).sum(0)
    return stats, rewards, logp, _dlogits(probs, s["labels"], per_row * s["scale"], s["logits"].dtype)


def _ln(s, case):
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    out = []
    if own:
        norm = s["norm"]
        mean, rstd = (None, None) if fwd else (s["mean"], s["rstd"])
        if fwd:
            y, mean, rstd = norm.forward(s["x"], s["weight"], s["bias"])
            out += [y, mean, rstd]
        if bwd:
            out += norm.backward(s["dy"], s["x"], s["weight"], mean, rstd)
        return out
    x, w = s["x"].float(), s["weight"].float()
    if fwd:
        mean = x.mean(1)
        rstd = 1 / torch.sqrt((x - mean[:, None]).square().mean(1) + LN_EPS)
        xhat = (x - mean[:, None]) * rstd[:, None]
        out += [(xhat * w + s["bias"].float()).to(s["x"].dtype), mean, rstd]
    else:
        mean, rstd = s["mean"], s["rstd"]
        xhat = (x - mean[:, None]) * rstd[:, None]
    if bwd:
        dy = s["dy"].float()
        a = dy * w
        dx = rstd[:, None] * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
        out += [dx.to(s["x"].dtype), (dy * xhat).sum(0).to(w_type(s)), dy.sum(0).to(w_type(s))]
    return out


def w_type(s):
    return s["weight"].dtype


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "norm":
        n = sum(k for k, _ in shapes(case))
        return {"bytes": n * size + (n * (size + 24) if case["step"] else 0), "flops": 2 * n + (14 * n if case["step"] else 0)}
    if case["op"] == "ln":
        n, wsize = case["rows"] * case["width"], SIZE[case["weight"]]
        fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
        moved = 2 * n * size + case["width"] * 2 * wsize + 8 * case["rows"] if fwd else 0
        moved += 3 * n * size + case["width"] * 3 * wsize + 8 * case["rows"] if bwd else 0
        return {"bytes": moved, "flops": (8 * n if fwd else 0) + (14 * n if bwd else 0)}
    rows, vocab = case["rows"], case["vocab"]
    live = rows - sum(hidden(case))
    read = live * vocab * size
    if case["op"] == "logps":
        return {"bytes": read + 16 * rows, "flops": 4 * live * vocab}
    return {"bytes": read + rows * vocab * size + 28 * rows, "flops": 8 * live * vocab}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "norm":
        g = s["grads"].to(d) / s["scale"].to(d)
        norm = torch.linalg.vector_norm(g).reshape(1)
        coef = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6))
        out = {"norm": norm, "clip_scale": s["scale"].to(d) / coef, "found_inf": torch.zeros_like(norm)}
        if case["step"]:
            g *= coef
            m, v = (1 - B1) * g, (1 - B2) * g * g
            p = s["params"].to(d)
            p = p - LR * s["wd"].to(d) * p - LR * (m / (1 - B1)) / (torch.sqrt(v / (1 - B2)) + EPS)
            out.update(params=p, m=m, v=v)
        return out
    if case["op"] == "ln":
        x, w, n = s["x"].to(d), s["weight"].to(d), case["width"]
        out = []
        if case["dir"] == "bwd":
            mean, rstd = s["mean"].to(d), s["rstd"].to(d)
        else:
            mean = x.sum(1) / n
            rstd = ((x * x).sum(1) / n - mean * mean + LN_EPS).rsqrt()
        xhat = torch.addcmul(-(mean * rstd)[:, None], x, rstd[:, None])
        if case["dir"] != "bwd":
            out += [torch.addcmul(s["bias"].to(d), xhat, w), mean, rstd]
        if case["dir"] != "fwd":
            dy = s["dy"].to(d)
            k1, k2 = dy @ w / n, torch.einsum("rc,rc,c->r", dy, xhat, w) / n
            out += [(dy * w - k1[:, None] - xhat * k2[:, None]) * rstd[:, None], torch.einsum("rc,rc->c", dy, xhat), torch.einsum("rc->c", dy)]
        return out
    rows, kind = case["rows"], s["logits"].dtype
    labels = s["labels"]
    live = labels >= 0
    y = labels.clamp(min=0)
    logp, lse = torch.empty(rows, dtype=d, device=DEV), torch.empty(rows, dtype=d, device=DEV)
    for k in range(0, rows, 512):
        z = s["logits"][k:k + 512].to(d)
        lse[k:k + 512] = torch.logsumexp(z, 1)
        logp[k:k + 512] = z.gather(1, y[k:k + 512, None])[:, 0] - lse[k:k + 512]
    logp[~live] = 0
    lse[~live] = 0
    if case["op"] == "logps":
        return logp, lse
    w = s["weights"].to(d)
    if case["op"] == "policy":
        a, ratio, x = s["advantages"].to(d), (logp - s["old"].to(d)).exp(), s["ref"].to(d) - logp
        lo, hi = 1 - CLIP_LO, 1 + CLIP_HI
        cut = ((a > 0) & (ratio > hi)) | ((a < 0) & (ratio < lo))
        pg = -a * torch.where(cut, torch.where(a > 0, torch.full_like(a, hi), torch.full_like(a, lo)), ratio)
        kl = torch.expm1(x) - x
        keep = w > 0
        terms = [(w * t)[keep].sum() for t in (pg, kl, cut.to(d))]
        head = [torch.stack([terms[0] + KL * terms[1], *terms]), logp]
        coef = w * (-a * ratio * (~cut) - KL * torch.expm1(x))
    else:
        pairs, at = case["pairs"], s["starts"].tolist()
        gap = w * (logp - s["ref"].to(d))
        sums = torch.stack([gap[i:j].sum() for i, j in zip(at, at[1:])]) * BETA
        margin = sums[:pairs] - sums[pairs:]
        sp = torch.nn.functional.softplus
        each = (1 - SMOOTH) * sp(-margin) + SMOOTH * sp(margin)
        head = [torch.stack([each.mean(), (margin > 0).to(d).mean(), sums[:pairs].mean(), sums[pairs:].mean()]), sums, logp]
        slope = BETA / pairs * (SMOOTH * torch.sigmoid(margin) - (1 - SMOOTH) * torch.sigmoid(-margin))
        coef = torch.zeros_like(w)
        for i, j, c in zip(at, at[1:], torch.cat([slope, -slope])):
            coef[i:j] = w[i:j] * c
    coef = coef * s["scale"].to(d)
    grad = torch.empty(s["logits"].shape, dtype=d if s["logits"].numel() < 1 << 28 else torch.float32, device=DEV)
    for k in range(0, rows, 512):
        p = torch.exp(s["logits"][k:k + 512].to(d) - lse[k:k + 512, None]) * -coef[k:k + 512, None]
        p[torch.arange(p.shape[0], device=DEV), y[k:k + 512]] += coef[k:k + 512]
        grad[k:k + 512] = torch.where(live[k:k + 512, None], p, torch.zeros_like(p)).to(grad.dtype)
    return (*head, grad)
