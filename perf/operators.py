"""Work for the operators that stand around the block-scaled linear layers in a training or
serving step: the norms before and after a block with its gate and residual scale
(block_norm), tokens sorted by expert and back (expert_sort, expert_gather, expert_combine)
and the global gradient norm with clipping (clip_grad_norm), forward and backward.

`run` computes each of them either in a plain form of elementary torch operations (own = False)
or through this package's entry points (own = True), on the same inputs.
"""
import math

import torch

own = False

EPS_NORM = 1e-6
EPS_CLIP = 1e-6


def listed():
    return [
        # one token of a decoder of width 4096: RMS norms on both sides of the block (latency)
        dict(name="norm_fwd_one_token", op="norm_fwd", kind="rms", rows=1, cols=4096, dtype="bf16", params="bf16",
             groups=1, post=True, bias=False, gate=False, scale=1.0, offset=1.0),
        # ViT-L/16, 32 frames of 1600 tokens: layer norm of the next sublayer, LayerScale, no norm after
        dict(name="norm_fwd_vitl_large", op="norm_fwd", kind="layer", rows=51200, cols=1024, dtype="bf16",
             params="bf16", groups=1, post=False, bias=True, gate=True, scale=1.0, offset=0.0),
        # an odd width and row count in fp32, a gate for each of 7 samples
        dict(name="norm_fwd_odd_fp32", op="norm_fwd", kind="layer", rows=4097 * 7, cols=1001, dtype="fp32",
             params="fp32", groups=7, post=True, bias=True, gate=True, scale=0.5, offset=0.0),
        # ViT-B/16 at its training shape, 14 frames of 1024 tokens: gradients of both norms and of LayerScale
        dict(name="norm_bwd_vitb", op="norm_bwd", kind="layer", rows=14336, cols=768, dtype="bf16", params="bf16",
             groups=1, post=True, bias=True, gate=True, scale=1.0, offset=0.0),
        # a wide decoder's training step: RMS norms on both sides, 8 sequences with a gate each
        dict(name="norm_bwd_wide", op="norm_bwd", kind="rms", rows=16384, cols=8192, dtype="bf16", params="fp32",
             groups=8, post=True, bias=False, gate=True, scale=0.7, offset=1.0),
        # one token to 8 of 64 experts while serving (latency)
        dict(name="experts_dispatch_one_token", op="dispatch", tokens=1, topk=8, experts=64, cols=4096, align=1,
             dtype="bf16", drop=0.0),
        # ViT-L width, 7 frames of 1024 tokens, expert segments padded to the 128-row scale tiles, some tokens dropped
        dict(name="experts_dispatch_vitl", op="dispatch", tokens=7168, topk=2, experts=16, cols=1024, align=128,
             dtype="bf16", drop=0.02),
        # many small experts: the weighted sum of 8 expert rows a token, odd token count
        dict(name="experts_combine_fine", op="combine", tokens=16381, topk=8, experts=128, cols=2048, align=1,
             dtype="bf16", drop=0.0),
        # gradient of the weighted sum, to the expert rows and to the router's weights
        dict(name="experts_combine_bwd", op="combine_bwd", tokens=14336, topk=4, experts=64, cols=2048, align=128,
             dtype="bf16", drop=0.01),
        # an adapter's or a head's few tensors (latency), fp32
        dict(name="clip_head", op="clip", layers=1, width=64, align=1, dtype="fp32", level=1e-2, max_norm=1.0),
        # one ViT-L/16 in bf16 with fp32 vectors: some hundred tensors
        dict(name="clip_vitl_bf16", op="clip", layers=24, width=1024, align=128, dtype="bf16", level=1e-3,
             max_norm=1.0),
        # an odd width, tensors packed without gaps, fp32
        dict(name="clip_odd_fp32", op="clip", layers=12, width=1537, align=1, dtype="fp32", level=1e-4, max_norm=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_bwd", "dispatch", "combine", "combine_bwd", "gather_bwd", "clip"])
    if op in ("norm_fwd", "norm_bwd"):
        cols = _log_int(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = max(64, cols // 64 * 64)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        groups = rng.choice([1, 1, 2, 5])
        most = (1 << 26) // cols
        rows = max(1, _log_int(rng, 1, most) // groups) * groups
        return dict(op=op, kind=rng.choice(["rms", "layer"]), rows=rows, cols=cols, dtype=dtype,
                    params=rng.choice(["bf16", "fp32"]), groups=groups, post=rng.random() < 0.7,
                    bias=rng.random() < 0.5, gate=groups > 1 or rng.random() < 0.6, scale=rng.choice([1.0, 0.5]),
                    offset=rng.choice([0.0, 1.0]))
    if op == "clip":
        return dict(op="clip", layers=rng.randint(1, 20), width=_log_int(rng, 16, 1100), align=rng.choice([1, 8, 128]),
                    dtype=rng.choice(["bf16", "fp32"]), level=10.0 ** rng.uniform(-5, -1),
                    max_norm=rng.choice([0.1, 1.0, 5.0]))
    experts = rng.choice([4, 8, 32, 60, 128, 256])
    cols = _log_int(rng, 64, 4096)
    if rng.random() < 0.7:
        cols = cols // 64 * 64
    topk = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= experts])
    tokens = _log_int(rng, 1, max(2, (1 << 26) // (cols * topk)))
    return dict(op=op, tokens=tokens, topk=topk, experts=experts, cols=cols, align=rng.choice([1, 1, 16, 128]),
                dtype=rng.choice(["bf16", "bf16", "fp32"]), drop=rng.choice([0.0, 0.0, 0.05, 0.3]))


# ---------------------------------------------------------------- inputs
_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _rms(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS_NORM)


def _stats_of(v, kind):
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return mean, _rms(v - mean)


def _prepare_norm(case, gen):
    dt, pt = _DTYPE[case["dtype"]], _DTYPE[case["params"]]
    rows, cols, groups = case["rows"], case["cols"], case["groups"]

    def rnd(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, device="cuda", generator=gen) * std + mean

    center = 1.0 - case["offset"]  # weights are stored without the offset that is added to them
    # residual stream: a row scale that varies from token to token, and a few large channels
    x = rnd(rows, cols) * torch.exp(0.5 * rnd(rows, 1)) + 0.2
    x[:, :: max(1, cols // 5)] *= 20
    s = dict(case=case, h=rnd(rows, cols, std=0.7, mean=0.05).to(dt), x=x.to(dt), post_weight=None, post_bias=None,
             gate=None, pre_weight=rnd(cols, std=0.1, mean=center).to(pt),
             pre_bias=rnd(cols, std=0.1).to(pt) if case["bias"] else None)
    if case["post"]:
        s["post_weight"] = rnd(cols, std=0.1, mean=center).to(pt)
        s["post_bias"] = rnd(cols, std=0.1).to(pt) if case["bias"] else None
    if case["gate"]:
        gate = rnd(groups, cols, std=0.3, mean=0.3).to(pt)
        s["gate"] = gate if groups > 1 else gate.reshape(cols)
    if case["op"] == "norm_bwd":  # what the forward pass kept, and the gradients that arrive
        x_out, _, stats = _norm_fwd_plain(s, rounded=False)
        s["x_out"], s["stats"] = x_out.to(dt), stats
        s["dx_out"] = rnd(rows, cols, std=1e-3).to(dt)
        s["dy"] = rnd(rows, cols, std=1e-3).to(dt)
        del s["x"]
    return s


def _prepare_experts(case, gen):
    dt = _DTYPE[case["dtype"]]
    tokens, topk, experts, cols = case["tokens"], case["topk"], case["experts"], case["cols"]

    def rnd(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * std

    # a router's logits with a taste of its own for each expert: loads are uneven, experts may stay empty
    logits = rnd(tokens, experts) + rnd(1, experts)
    best, ids = logits.topk(topk, dim=-1)
    if case["drop"] > 0:
        lost = torch.rand(tokens, topk, device="cuda", generator=gen) < case["drop"]
        ids = torch.where(lost, torch.full_like(ids, -1), ids)
    s = dict(case=case, ids=ids, weights=torch.exp(best - best.amax(-1, keepdim=True)))
    s["weights"] = s["weights"] / s["weights"].sum(-1, keepdim=True)
    if case["op"] == "dispatch":
        s["x"] = rnd(tokens, cols).to(dt)
        return s
    counts, offsets, position, slot = _sort_plain(ids, experts, case["align"])
    s.update(counts=counts, offsets=offsets, position=position, slot=slot)
    s["y"] = rnd(slot.numel(), cols).to(dt)
    s["dout"] = rnd(tokens, cols, std=1e-3).to(dt)
    return s


def _clip_sizes(case):
    """(elements, is a matrix) of each tensor: the linear layers, biases and norms of `layers` blocks."""
    w = case["width"]
    block = [(w * w, True), (w, False)] * 4 + [(4 * w * w, True), (4 * w, False), (4 * w * w, True), (w, False)] + \
        [(w, False)] * 4
    return block * case["layers"] + [(w, False), (w, False)]


def _prepare_clip(case, gen):
    # matrices in the case's type, vectors in fp32, each type in a bucket of its own
    mt, sizes, align = _DTYPE[case["dtype"]], _clip_sizes(case), case["align"]
    s = dict(case=case, grads=[], outs=[])
    for name, dt, matrix in (("matrices", mt, True), ("vectors", torch.float32, False)):
        places, total = [], 0
        for n, is_matrix in sizes:
            if is_matrix == matrix:
                places.append((total, n))
                total += -(-n // align) * align
        bucket = torch.randn(total, device="cuda", generator=gen).mul_(case["level"]).to(dt)
        s[name] = torch.zeros(total, device="cuda", dtype=dt)  # where the clipped gradients go
        s["grads"] += [bucket[a:a + n] for a, n in places]
        s["outs"] += [s[name][a:a + n] for a, n in places]
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _prepare_norm(case, gen)
    return _prepare_clip(case, gen) if op == "clip" else _prepare_experts(case, gen)


# ---------------------------------------------------------------- plain forms
def _rows_of_gate(s, rows):
    """The gate as a broadcastable fp32 matrix."""
    gate = s["gate"].float()
    return gate if gate.dim() == 1 else gate.repeat_interleave(rows // gate.shape[0], 0)


def _weight(w, offset):
    return w.float() + offset


def _norm_fwd_plain(s, rounded=True):
    case = s["case"]
    kind, offset = case["kind"], case["offset"]
    n = s["h"].float()
    post = torch.zeros(case["rows"], 2, device="cuda")
    if case["post"]:
        mean, rstd = _stats_of(n, kind)
        post = torch.cat([mean, rstd], 1)
        n = (n - mean) * rstd * _weight(s["post_weight"], offset)
        if s["post_bias"] is not None:
            n = n + s["post_bias"].float()
    if s["gate"] is not None:
        n = n * _rows_of_gate(s, case["rows"])
    x_out = s["x"].float() * case["scale"] + n
    mean, rstd = _stats_of(x_out, kind)
    y = (x_out - mean) * rstd * _weight(s["pre_weight"], offset)
    if s["pre_bias"] is not None:
        y = y + s["pre_bias"].float()
    stats = torch.cat([post, mean, rstd], 1)
    if not rounded:
        return x_out, y, stats
    dt = s["h"].dtype
    return x_out.to(dt), y.to(dt), stats


def _norm_grad(g, xhat, rstd, kind):
    """Gradient through (v - mean) * rstd, from the gradient g of that."""
    out = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        out = out - g.mean(-1, keepdim=True)
    return out * rstd


def _norm_bwd_plain(s):
    case = s["case"]
    kind, offset, rows, groups = case["kind"], case["offset"], case["rows"], case["groups"]
    dt = s["h"].dtype
    stats, h, dy = s["stats"], s["h"].float(), s["dy"].float()
    out = {}
    xhat = (s["x_out"].float() - stats[:, 2:3]) * stats[:, 3:4]
    out["dpre_weight"] = (dy * xhat).sum(0)
    if s["pre_bias"] is not None:
        out["dpre_bias"] = dy.sum(0)
    d = s["dx_out"].float() + _norm_grad(dy * _weight(s["pre_weight"], offset), xhat, stats[:, 3:4], kind)
    out["dx"] = (d * case["scale"]).to(dt)
    n = h
    if case["post"]:
        xhat = (h - stats[:, 0:1]) * stats[:, 1:2]
        n = xhat * _weight(s["post_weight"], offset)
        if s["post_bias"] is not None:
            n = n + s["post_bias"].float()
    if s["gate"] is not None:
        dgate = d * n
        out["dgate"] = dgate.sum(0) if groups == 1 else dgate.reshape(groups, rows // groups, -1).sum(1)
        d = d * _rows_of_gate(s, rows)
    if case["post"]:
        out["dpost_weight"] = (d * xhat).sum(0)
        if s["post_bias"] is not None:
            out["dpost_bias"] = d.sum(0)
        d = _norm_grad(d * _weight(s["post_weight"], offset), xhat, stats[:, 1:2], kind)
    out["dh"] = d.to(dt)
    return out


def _capacity(slots, experts, align):
    """Rows that hold every expert's segment, padded to `align`, whatever the router says."""
    return -(-(slots + min(experts, slots) * (align - 1)) // align) * align


def _sort_plain(ids, experts, align):
    flat = ids.reshape(-1)
    slots = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    sorted_key, order = torch.sort(key, stable=True)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    padded = (counts + align - 1) // align * align
    zero = torch.zeros(1, device=flat.device, dtype=torch.int64)
    offsets = torch.cat([zero, padded.cumsum(0)])
    begins = torch.cat([zero, counts.cumsum(0)])  # where each expert begins among the sorted slots; the dropped last
    rank = torch.arange(slots, device=flat.device) - begins[sorted_key]
    row = torch.where(sorted_key < experts, offsets[sorted_key] + rank, torch.full_like(rank, -1))
    position = torch.empty_like(row)
    position[order] = row
    slot = torch.full((_capacity(slots, experts, align) + 1,), -1, device=flat.device, dtype=torch.int64)
    slot[row] = order  # the dropped ones write the last place, which is cut off
    return counts.int(), offsets.int(), position.int().reshape(ids.shape), slot[:-1].int()


def _gather_plain(x, slot, topk):
    rows = x[slot.clamp(min=0) // topk]
    return torch.where(slot[:, None] >= 0, rows, torch.zeros_like(rows))


def _combine_plain(y, position, weights):
    rows = y[position.clamp(min=0)].float()
    if weights is not None:
        rows = rows * weights[..., None]
    return torch.where(position[..., None] >= 0, rows, torch.zeros_like(rows)).sum(1).to(y.dtype)


def _combine_bwd_plain(dout, y, position, slot, weights):
    topk = position.shape[1]
    grad = dout[slot.clamp(min=0) // topk].float() * weights.reshape(-1)[slot.clamp(min=0)][:, None]
    dy = torch.where(slot[:, None] >= 0, grad, torch.zeros_like(grad)).to(y.dtype)
    dots = (y[position.clamp(min=0)].float() * dout.float()[:, None, :]).sum(-1)
    return dy, torch.where(position >= 0, dots, torch.zeros_like(dots))


def _clip_plain(s):
    case = s["case"]
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    coef = (case["max_norm"] / (total + EPS_CLIP)).clamp(max=1.0)
    _ = [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
    return dict(norm=total, matrices=s["matrices"], vectors=s["vectors"])


def _named(counts, offsets, position, slot, rows):
    return dict(counts=counts, offsets=offsets, position=position, slot=slot, rows=rows)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        x_out, y, stats = _norm_fwd_plain(s)
        return dict(x_out=x_out, y=y, stats=stats)
    if op == "norm_bwd":
        return _norm_bwd_plain(s)
    if op == "dispatch":
        counts, offsets, position, slot = _sort_plain(s["ids"], case["experts"], case["align"])
        return _named(counts, offsets, position, slot, _gather_plain(s["x"], slot, case["topk"]))
    if op == "combine":
        return _combine_plain(s["y"], s["position"], s["weights"])
    if op == "gather_bwd":
        return _combine_plain(s["y"], s["position"], None)
    if op == "combine_bwd":
        dy, dweights = _combine_bwd_plain(s["dout"], s["y"], s["position"], s["slot"], s["weights"])
        return dict(dy=dy, dweights=dweights)
    return _clip_plain(s)


# ---------------------------------------------------------------- this package's operators
def _run_own(s):
    import block_scaled_precision_bsq_gb300 as bsq

    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        r = bsq.block_norm(s["h"], s["x"], kind=case["kind"], post_norm=case["post"], post_weight=s["post_weight"],
                           post_bias=s["post_bias"], gate=s["gate"], residual_scale=case["scale"],
                           pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], weight_offset=case["offset"],
                           eps=EPS_NORM)
        return dict(x_out=r.x_out, y=r.y, stats=r.stats)
    if op == "norm_bwd":
        r = bsq.block_norm_backward(s["dx_out"], s["dy"], s["x_out"], s["h"], s["stats"], kind=case["kind"],
                                    post_norm=case["post"], post_weight=s["post_weight"], post_bias=s["post_bias"],
                                    gate=s["gate"], residual_scale=case["scale"], pre_weight=s["pre_weight"],
                                    pre_bias=s["pre_bias"], weight_offset=case["offset"])
        return {k: v for k, v in r._asdict().items() if v is not None}
    if op == "dispatch":
        r = bsq.expert_sort(s["ids"], case["experts"], align=case["align"])
        return _named(r.counts, r.offsets, r.position, r.slot, bsq.expert_gather(s["x"], r.position, r.slot))
    if op == "combine":
        return bsq.expert_combine(s["y"], s["position"], s["weights"])
    if op == "gather_bwd":
        return bsq.expert_gather_backward(s["y"], s["position"])
    if op == "combine_bwd":
        dy, dweights = bsq.expert_combine_backward(s["dout"], s["y"], s["position"], s["slot"], s["weights"])
        return dict(dy=dy, dweights=dweights)
    norm = bsq.clip_grad_norm(s["grads"], case["max_norm"], eps=EPS_CLIP, outs=s["outs"])
    return dict(norm=norm, matrices=s["matrices"], vectors=s["vectors"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        es = 2 if case["dtype"] == "bf16" else 4
        ps = 2 if case["params"] == "bf16" else 4
        rows, cols = case["rows"], case["cols"]
        vectors = cols * (1 + case["bias"] + case["post"] * (1 + case["bias"]) + case["gate"] * case["groups"])
        if op == "norm_fwd":  # h, x in; x_out, y, four statistics a row out
            return dict(bytes=4 * rows * cols * es + 16 * rows + vectors * ps, flops=rows * cols * 16)
        # dx_out, dy, x_out, h, statistics in; dx, dh and fp32 parameter gradients out. h is needed for the norm after
        # the block and for the gate's gradient alone.
        need_h = case["post"] or case["gate"]
        return dict(bytes=(5 + need_h) * rows * cols * es + 16 * rows + vectors * (ps + 4), flops=rows * cols * 36)
    if op == "clip":
        es = 2 if case["dtype"] == "bf16" else 4
        sizes = _clip_sizes(case)
        matrices = sum(n for n, m in sizes if m)
        vectors = sum(n for n, m in sizes if not m)
        return dict(bytes=2 * (matrices * es + vectors * 4) + 4, flops=3 * (matrices + vectors))
    es = 2 if case["dtype"] == "bf16" else 4
    tokens, topk, cols = case["tokens"], case["topk"], case["cols"]
    slots = tokens * topk
    live = slots * (1 - case["drop"])
    capacity = _capacity(slots, case["experts"], case["align"])
    if op == "dispatch":  # ids and x in; positions, slots and every row of the capacity out
        return dict(bytes=slots * 8 + tokens * cols * es + slots * 4 + capacity * (4 + cols * es) + case["experts"] * 8,
                    flops=slots)
    if op in ("combine", "gather_bwd"):
        return dict(bytes=slots * 8 + (live + tokens) * cols * es, flops=2 * live * cols)
    # combine_bwd: dout, y, weights and the map in; dy over the capacity and the weights' gradient out
    return dict(bytes=slots * 12 + capacity * 4 + (tokens + live + capacity) * cols * es, flops=3 * live * cols)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_norm(s):
    case = s["case"]
    f64 = torch.float64
    h = s["h"].to(f64)
    rows, cols, offset, layer = case["rows"], case["cols"], case["offset"], case["kind"] == "layer"
    w2 = s["pre_weight"].to(f64) + offset
    gate = torch.ones(1, 1, dtype=f64, device="cuda")
    if s["gate"] is not None:
        gate = s["gate"].to(f64).reshape(case["groups"], 1, cols).expand(-1, rows // case["groups"], -1).reshape(rows, cols)

    def moments(v):
        mu = v.sum(1, keepdim=True) / cols if layer else torch.zeros(rows, 1, dtype=f64, device="cuda")
        return mu, 1 / torch.sqrt(torch.sum((v - mu) ** 2, 1, keepdim=True) / cols + EPS_NORM)

    def affine(v, w, b):
        return v * w if b is None else v * w + b.to(f64)

    if case["op"] == "norm_fwd":
        mu1 = torch.zeros(rows, 1, dtype=f64, device="cuda")
        r1, n = mu1, h
        if case["post"]:
            mu1, r1 = moments(h)
            n = affine((h - mu1) * r1, s["post_weight"].to(f64) + offset, s["post_bias"])
        x_out = case["scale"] * s["x"].to(f64) + gate * n
        mu2, r2 = moments(x_out)
        return dict(x_out=x_out, y=affine((x_out - mu2) * r2, w2, s["pre_bias"]), stats=torch.cat([mu1, r1, mu2, r2], 1))
    mu1, r1, mu2, r2 = s["stats"].to(f64).split(1, dim=1)

    def back(g, v, mu, r):
        z = (v - mu) * r
        along = torch.sum(g * z, 1, keepdim=True) / cols
        flat = torch.sum(g, 1, keepdim=True) / cols if layer else 0.0
        return r * (g - flat - z * along)

    dy, x_out = s["dy"].to(f64), s["x_out"].to(f64)
    total = s["dx_out"].to(f64) + back(dy * w2, x_out, mu2, r2)
    out = dict(dx=case["scale"] * total, dpre_weight=torch.sum(dy * (x_out - mu2) * r2, 0))
    if s["pre_bias"] is not None:
        out["dpre_bias"] = torch.sum(dy, 0)
    dn = total * gate
    n = h
    if case["post"]:
        w1 = s["post_weight"].to(f64) + offset
        n = affine((h - mu1) * r1, w1, s["post_bias"])
        out["dpost_weight"] = torch.sum(dn * (h - mu1) * r1, 0)
        if s["post_bias"] is not None:
            out["dpost_bias"] = torch.sum(dn, 0)
        out["dh"] = back(dn * w1, h, mu1, r1)
    else:
        out["dh"] = dn.expand(rows, cols)
    if s["gate"] is not None:
        out["dgate"] = torch.sum((total * n).reshape(case["groups"], -1, cols), 1).reshape(s["gate"].shape)
    return out


def _exact_experts(s):
    case = s["case"]
    f64 = torch.float64
    topk, experts, align = case["topk"], case["experts"], case["align"]
    if case["op"] == "dispatch":
        ids = s["ids"].reshape(-1).cpu().tolist()
        lists = [[] for _ in range(experts)]
        for i, e in enumerate(ids):
            if 0 <= e < experts:
                lists[e].append(i)
        slot, offsets, position = [], [0], [-1] * len(ids)
        for members in lists:
            for i in members:
                position[i] = len(slot)
                slot.append(i)
            slot += [-1] * (-len(slot) % align if len(slot) % align else 0)
            offsets.append(len(slot))
        slot += [-1] * (_capacity(len(ids), experts, align) - len(slot))
        at = torch.tensor(slot, device="cuda")
        rows = torch.zeros(len(slot), case["cols"], dtype=f64, device="cuda")
        live = at >= 0
        rows[live] = s["x"].to(f64)[at[live] // topk]
        whole = dict(dtype=torch.int32, device="cuda")
        return _named(torch.tensor([len(m) for m in lists], **whole), torch.tensor(offsets, **whole),
                      torch.tensor(position, **whole).reshape(s["ids"].shape), at.int(), rows)
    y = s["y"].to(f64)
    position = s["position"]
    live = position >= 0
    if case["op"] in ("combine", "gather_bwd"):
        w = s["weights"].to(f64) if case["op"] == "combine" else torch.ones_like(s["weights"], dtype=f64)
        out = torch.zeros(case["tokens"], case["cols"], dtype=f64, device="cuda")
        for j in range(topk):
            t = torch.nonzero(live[:, j]).reshape(-1)
            out[t] += w[t, j, None] * y[position[t, j].long()]
        return out
    dout = s["dout"].to(f64)
    dy, dweights = torch.zeros_like(y), torch.zeros_like(s["weights"], dtype=f64)
    for j in range(topk):
        t = torch.nonzero(live[:, j]).reshape(-1)
        p = position[t, j].long()
        dy[p] = s["weights"].to(f64)[t, j, None] * dout[t]
        dweights[t, j] = torch.einsum("tc,tc->t", dout[t], y[p])
    return dict(dy=dy, dweights=dweights)


def _exact_clip(s):
    total = 0.0
    for g in s["grads"]:
        total += float(torch.linalg.vector_norm(g.double()) ** 2)
    norm = math.sqrt(total)
    coef = min(1.0, s["case"]["max_norm"] / (norm + EPS_CLIP))
    out = dict(norm=torch.tensor(norm, dtype=torch.float64, device="cuda"))
    for name in ("matrices", "vectors"):
        out[name] = torch.zeros(s[name].numel(), dtype=torch.float64, device="cuda")
    for g, o in zip(s["grads"], s["outs"]):
        name = "matrices" if o.untyped_storage().data_ptr() == s["matrices"].untyped_storage().data_ptr() else "vectors"
        out[name][o.storage_offset():o.storage_offset() + o.numel()] = g.double() * coef
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s)
    return _exact_clip(s) if case["op"] == "clip" else _exact_experts(s)
