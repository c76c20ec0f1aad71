"""Work for the linear layers of dense and expert blocks beyond the plain product: products grouped
by expert over ragged segments of rows (expert_gemm, its gradient towards the rows and its weight
gradient) and products with bias, activation and residual in their epilogue (gemm_act, and the
gradient through the activation), on block-scaled operands.

`run` computes each of them either in a plain form of elementary torch operations (own = False)
or through this package's entry points (own = True), on the same inputs.
"""
import math

import torch

own = False

_FMT = {"mxfp8": 1, "nvfp4": 2, "mxfp4": 3}
_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token to 8 of 64 experts while serving: rows packed without gaps (latency, the weights' bytes)
        dict(name="expert_one_token", op="expert_fwd", fmt="mxfp4", tokens=1, topk=8, experts=64, n=2048, k=4096, align=1,
             bias=False, act="", pre=False),
        # ViT-L widths, 7 frames of 1024 tokens to 2 of 16 experts: fc1 with GELU in training, which keeps its argument
        dict(name="expert_fwd_vitl", op="expert_fwd", fmt="mxfp8", tokens=7168, topk=2, experts=16, n=4096, k=1024,
             align=128, bias=True, act="gelu", pre=True),
        # many small experts over an odd number of tokens: prefill while serving
        dict(name="expert_fwd_fine", op="expert_fwd", fmt="nvfp4", tokens=16381, topk=8, experts=128, n=1024, k=2048,
             align=1, bias=False, act="", pre=False),
        # the gradient through fc2 and the GELU before it, with fc1's bias gradient
        dict(name="expert_bwd_vitl", op="expert_bwd", fmt="mxfp8", tokens=7168, topk=2, experts=16, n=1024, k=4096,
             align=128, act="gelu", dbias=True),
        # the gradient through fc1 towards the rows, many experts
        dict(name="expert_bwd_fine", op="expert_bwd", fmt="nvfp4", tokens=8191, topk=4, experts=64, n=2048, k=2048,
             align=128, act="", dbias=False),
        # the experts' weight gradients
        dict(name="expert_wgrad_vitl", op="expert_wgrad", fmt="mxfp8", tokens=7168, topk=2, experts=16, n=4096, k=1024,
             align=128, dtype="bf16"),
        # weight gradients of many experts for fp32 accumulation, FP4
        dict(name="expert_wgrad_fine", op="expert_wgrad", fmt="mxfp4", tokens=8191, topk=4, experts=64, n=1024, k=2048,
             align=128, dtype="fp32"),
        # one token through a square layer onto the residual stream (latency)
        dict(name="act_one_token", op="act", fmt="nvfp4", rows=1, n=4096, k=4096, bias=True, act="", residual="bf16",
             pre=False),
        # ViT-L fc2 of 32 frames of 1600 tokens, added to the residual stream
        dict(name="act_fc2_residual", op="act", fmt="mxfp4", rows=51200, n=1024, k=4096, bias=True, act="",
             residual="bf16", pre=False),
        # fc1 of an odd number of tokens in training, keeps its argument
        dict(name="act_fc1_odd", op="act", fmt="nvfp4", rows=7203, n=4096, k=1024, bias=True, act="gelu", residual="",
             pre=True),
        # ViT-L fc2's gradient through the GELU before it, with fc1's bias gradient
        dict(name="act_bwd_vitl", op="act_bwd", fmt="mxfp8", rows=14336, n=1024, k=4096, act="gelu", dbias=True),
        # the same of a decoder's layer with SiLU, an odd number of tokens
        dict(name="act_bwd_odd", op="act_bwd", fmt="nvfp4", rows=2049, n=4096, k=8192, act="silu", dbias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["expert_fwd", "expert_fwd", "expert_bwd", "expert_wgrad", "act", "act", "act_bwd"])
    n, k = (max(1, _log_int(rng, 128, 4096) // 128) * 128 for _ in range(2))
    act = rng.choice(["", "gelu", "gelu_tanh", "silu", "relu"])
    case = dict(op=op, fmt=rng.choice(["mxfp8", "nvfp4", "mxfp4"]), n=n, k=k)
    most = (1 << 38) // (2 * n * k)  # rows that cost no more than the largest listed case
    if op.startswith("act"):
        case["rows"] = _log_int(rng, 1, min(60000, most))
        if op == "act_bwd":
            return dict(case, act=act, dbias=rng.random() < 0.7)
        return dict(case, bias=rng.random() < 0.7, act=act, residual=rng.choice(["", "bf16", "fp32"]),
                    pre=rng.random() < 0.4)
    case["experts"] = rng.choice([4, 8, 16, 60, 128])
    case["topk"] = rng.choice([t for t in (1, 2, 4, 8) if t <= case["experts"]])
    case["tokens"] = _log_int(rng, 1, max(2, min(60000, most // case["topk"])))
    if op == "expert_wgrad":
        return dict(case, align=128, dtype=rng.choice(["bf16", "fp32"]))
    case["align"] = rng.choice([1, 1, 128])
    if op == "expert_bwd":
        return dict(case, act=act, dbias=rng.random() < 0.5)
    return dict(case, bias=rng.random() < 0.5, act=act, pre=rng.random() < 0.4)


# ---------------------------------------------------------------- inputs
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_codes(v):
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    code = torch.bucketize(v.abs(), borders, out_int32=True).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tile(scales):
    """Scale bytes (rows x scale columns) in tiles of 128 rows x 4 columns."""
    rows, cols = scales.shape
    whole = torch.zeros(-(-rows // 128) * 128, -(-cols // 4) * 4, dtype=torch.uint8, device=scales.device)
    whole[:rows, :cols] = scales
    return whole.reshape(-1, 4, 32, whole.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _quantized(fmt, x):
    """A matrix as a block-scaled operand: what the quantizer leaves in the program's hands."""
    rows, cols = x.shape
    x = x.float()
    block = 16 if fmt == "nvfp4" else 32
    xb = x.reshape(rows, cols // block, block)
    amax = xb.abs().amax(-1)
    g = None
    if fmt == "nvfp4":
        g = (x.abs().amax() / 2688).reshape(1)
        s = (amax / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn)
        step = s.float() * g
        v = torch.where(step[..., None] > 0, xb / step[..., None], torch.zeros_like(xb))
        s = s.view(torch.uint8)
    else:
        e = (torch.frexp(amax).exponent - 1 - (8 if fmt == "mxfp8" else 2)).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        v = torch.ldexp(xb, -e[..., None])
        s = (e + 127).to(torch.uint8)
    v = v.reshape(rows, cols)
    codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "mxfp8" else _e2m1_codes(v)
    scales = _tile(s)
    if fmt == "nvfp4":  # the tail: g, the largest magnitude, two zeros
        tail = torch.cat([g, g * 2688, torch.zeros(2, device=x.device)])
        scales = torch.cat([scales, tail.view(torch.uint8)])
    return dict(fmt=fmt, rows=rows, cols=cols, codes=codes.reshape(-1), scales=scales, g=g)


def _segments(case, gen):
    """Rows of each expert, their first rows, and which of all rows are live: a router's choices with mild tastes."""
    tokens, topk, experts, align = case["tokens"], case["topk"], case["experts"], case["align"]
    logits = torch.randn(tokens, experts, device="cuda", generator=gen) + \
        0.3 * torch.randn(1, experts, device="cuda", generator=gen)
    ids = logits.topk(topk, dim=-1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=experts)
    padded = (counts + align - 1) // align * align
    offsets = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), padded.cumsum(0)])
    slots = tokens * topk
    capacity = -(-(slots + min(experts, slots) * (align - 1)) // align) * align
    row = torch.arange(capacity, device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), row, right=True).clamp(max=experts - 1)
    live = (row >= offsets[expert]) & (row < offsets[expert] + counts[expert])
    return counts.int(), offsets.int(), live


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def rnd(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * std

    def tokens_like(rows, cols, std):  # a row scale that varies from token to token, and a few large channels
        x = rnd(rows, cols) * torch.exp(0.5 * rnd(rows, 1)) * std
        x[:, :: max(1, cols // 5)] *= 8
        return x

    op, fmt, n, k = case["op"], case["fmt"], case["n"], case["k"]
    s = dict(case=case, bias=None, residual=None, before=None)
    experts = 1
    if op.startswith("expert"):
        experts = case["experts"]
        s["counts"], s["offsets"], live = _segments(case, gen)
        rows = live.numel()
    else:
        rows, live = case["rows"], torch.ones(case["rows"], device="cuda", dtype=torch.bool)
    if op == "expert_wgrad":
        s["dy"] = _quantized(fmt, torch.where(live[:, None], tokens_like(rows, n, 1e-3), 0).t().contiguous())
        s["x"] = _quantized(fmt, torch.where(live[:, None], tokens_like(rows, k, 1.0), 0).t().contiguous())
        return s
    w = rnd(experts * n, k, std=k ** -0.5)
    if op in ("act", "expert_fwd"):
        s["x"] = _quantized(fmt, torch.where(live[:, None], tokens_like(rows, k, 1.0), 0))
        s["w"] = _quantized(fmt, w)
        if case["bias"]:
            s["bias"] = rnd(experts, n, std=0.1).to(torch.bfloat16).reshape((experts, n) if op == "expert_fwd" else (n,))
        if case.get("residual"):
            s["residual"] = tokens_like(rows, n, 1.0).to(_DTYPE[case["residual"]])
        return s
    s["dy"] = _quantized(fmt, torch.where(live[:, None], tokens_like(rows, n, 1e-3), 0))
    s["w"] = _quantized(fmt, w.t().contiguous())  # the column-wise operand: k x (experts n), blocks along n
    if case["act"]:
        s["before"] = torch.where(live[:, None], rnd(rows, k, std=1.5), 0).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms
def _decode(q):
    """The values of an operand in fp32, without the per-tensor scale."""
    rows, cols, fmt = q["rows"], q["cols"], q["fmt"]
    block = 16 if fmt == "nvfp4" else 32
    if fmt == "mxfp8":
        v = q["codes"].view(torch.float8_e4m3fn).float().reshape(rows, cols)
    else:
        table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=q["codes"].device)
        v = torch.stack([table[(q["codes"] & 15).int()], table[(q["codes"] >> 4).int()]], -1).reshape(rows, cols)
    wide = -(-(cols // block) // 4)
    tiles = q["scales"][:-(-rows // 128) * wide * 512].reshape(-1, wide, 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = tiles.reshape(-1, wide * 4)[:rows, :cols // block].contiguous()
    s = s.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(s.float() - 127)
    return (v.reshape(rows, cols // block, block) * s[..., None]).reshape(rows, cols)


def _alpha(a, b):
    return 1.0 if a["g"] is None else a["g"] * b["g"]


def _act(name, v):
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v.clamp(min=0) if name == "relu" else v


def _slope(name, v):
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-v))
        return sg * (1 + v * (1 - sg))
    return (v > 0).to(v.dtype)


def _experts_of(q, experts, active):
    """The operand of some experts' weights alone, out of that of all (stacked along the rows)."""
    rows, tail = q["rows"] // experts, 16 if q["fmt"] == "nvfp4" else 0
    body = q["scales"][:q["scales"].numel() - tail]
    return dict(q, rows=rows * active.numel(), codes=q["codes"].reshape(experts, -1)[active].reshape(-1),
                scales=body.reshape(experts, -1)[active].reshape(-1))


def _places(s, rows):
    """The experts that have rows; for each, the places of its rows (as many as the largest has) and which are its own."""
    counts, offsets = s["counts"].long(), s["offsets"].long()
    active = counts.nonzero().reshape(-1)
    at = offsets[active][:, None] + torch.arange(int(counts.max()), device=counts.device)
    return active, at.clamp(max=rows - 1), at < (offsets[active] + counts[active])[:, None]


def _whole(values, at, mine, rows):
    """Rows of the experts' batches back in their places, zeros in rows of none."""
    out = torch.zeros(rows, values.shape[-1], device=values.device, dtype=values.dtype)
    out[at[mine]] = values[mine]
    return out


def _run_plain(s):
    case = s["case"]
    op, n, k = case["op"], case["n"], case["k"]
    if op == "act":
        v = _decode(s["x"]) @ _decode(s["w"]).t() * _alpha(s["x"], s["w"])
        if s["bias"] is not None:
            v = v + s["bias"].float()
        out = _act(case["act"], v)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        out = dict(out=out.to(s["residual"].dtype if s["residual"] is not None else torch.bfloat16))
        if case["pre"]:
            out["pre"] = v.to(torch.bfloat16)
        return out
    if op == "act_bwd":
        d = _decode(s["dy"]) @ _decode(s["w"]).t() * _alpha(s["dy"], s["w"])
        if s["before"] is not None:
            d = d * _slope(case["act"], s["before"].float())
        return dict(dpre=d.to(torch.bfloat16), dbias=d.sum(0)) if case["dbias"] else dict(dpre=d.to(torch.bfloat16))
    experts = case["experts"]
    if op == "expert_wgrad":
        rows = s["x"]["cols"]
        active, at, mine = _places(s, rows)
        x = torch.where(mine[..., None], _decode(s["x"]).t()[at], 0)
        dy = torch.where(mine[..., None], _decode(s["dy"]).t()[at], 0)
        dw = torch.zeros(experts, n, k, device=x.device)
        dw[active] = torch.bmm(dy.transpose(1, 2), x) * _alpha(s["dy"], s["x"])
        return dw.to(_DTYPE[case["dtype"]])
    if op == "expert_fwd":
        rows = s["x"]["rows"]
        active, at, mine = _places(s, rows)
        w = _decode(_experts_of(s["w"], experts, active)).reshape(-1, n, k)
        v = torch.bmm(_decode(s["x"])[at], w.transpose(1, 2)) * _alpha(s["x"], s["w"])
        if s["bias"] is not None:
            v = v + s["bias"].float()[active][:, None, :]
        out = dict(out=_whole(_act(case["act"], v).to(torch.bfloat16), at, mine, rows))
        if case["pre"]:
            out["pre"] = _whole(v.to(torch.bfloat16), at, mine, rows)
        return out
    rows = s["dy"]["rows"]
    active, at, mine = _places(s, rows)
    w = _decode(s["w"]).reshape(k, experts, n)[:, active]
    d = torch.bmm(_decode(s["dy"])[at], w.permute(1, 2, 0)) * _alpha(s["dy"], s["w"])
    if s["before"] is not None:
        d = d * _slope(case["act"], s["before"].float()[at])
    out = dict(dpre=_whole(d.to(torch.bfloat16), at, mine, rows))
    if case["dbias"]:
        out["dbias"] = torch.zeros(experts, k, device=d.device)
        out["dbias"][active] = torch.where(mine[..., None], d, 0).sum(1)
    return out


# ---------------------------------------------------------------- this package's operators
def _run_own(s):
    import block_scaled_precision_bsq_gb300 as bsq

    def operand(q):
        return bsq.QTensor(_FMT[q["fmt"]], q["rows"], q["cols"], q["codes"], q["scales"], q["g"])

    case = s["case"]
    op = case["op"]
    if op == "act":
        r = bsq.gemm_act(operand(s["x"]), operand(s["w"]), s["bias"], activation=case["act"] or None,
                         residual=s["residual"], save_pre=case["pre"])
        return dict(out=r.out, pre=r.pre) if case["pre"] else dict(out=r.out)
    if op == "act_bwd":
        r = bsq.gemm_act_backward(operand(s["dy"]), operand(s["w"]), s["before"], activation=case["act"] or None,
                                  bias_grad=case["dbias"])
        return dict(dpre=r.dpre, dbias=r.dbias) if case["dbias"] else dict(dpre=r.dpre)
    if op == "expert_wgrad":
        return bsq.expert_gemm_wgrad(operand(s["dy"]), operand(s["x"]), s["counts"], s["offsets"],
                                     dtype=_DTYPE[case["dtype"]])
    if op == "expert_fwd":
        r = bsq.expert_gemm(operand(s["x"]), operand(s["w"]), s["counts"], s["offsets"], s["bias"],
                            activation=case["act"] or None, save_pre=case["pre"])
        return dict(out=r.out, pre=r.pre) if case["pre"] else dict(out=r.out)
    r = bsq.expert_gemm_backward(operand(s["dy"]), operand(s["w"]), s["counts"], s["offsets"], s["before"],
                                 activation=case["act"] or None, bias_grad=case["dbias"])
    return dict(dpre=r.dpre, dbias=r.dbias) if case["dbias"] else dict(dpre=r.dpre)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, fmt, n, k = case["op"], case["fmt"], case["n"], case["k"]
    value = {"mxfp8": 1 + 1 / 32, "nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32}[fmt]
    experts, live, rows = 1, case.get("rows"), case.get("rows")
    if op.startswith("expert"):
        slots, align = case["tokens"] * case["topk"], case["align"]
        live, rows = slots, -(-(slots + min(case["experts"], slots) * (align - 1)) // align) * align
        experts = case["experts"]
    # the experts that some token chooses, as for even odds
    active = experts * (1 - (1 - case["topk"] / experts) ** case["tokens"]) if op.startswith("expert") else 1
    flops = 2 * live * n * k
    if op == "expert_wgrad":
        return dict(bytes=live * (n + k) * value + experts * n * k * (2 if case["dtype"] == "bf16" else 4), flops=flops)
    if op in ("act", "expert_fwd"):
        out = 4 if case.get("residual") == "fp32" else 2
        each = out + (2 if case["pre"] else 0)
        read = live * n * out if case.get("residual") else 0
        return dict(bytes=live * k * value + active * n * k * value + rows * n * each + read +
                    (active * n * 2 if case["bias"] else 0), flops=flops)
    return dict(bytes=live * n * value + active * n * k * value + rows * k * 2 + (live * k * 2 if case["act"] else 0) +
                (experts * k * 4 if case["dbias"] else 0), flops=flops)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_values(q):
    """An operand's values with its per-tensor scale in fp64, element by element from the bytes."""
    rows, cols, fmt = q["rows"], q["cols"], q["fmt"]
    f64, codes, block = torch.float64, q["codes"], 16 if q["fmt"] == "nvfp4" else 32

    def e4m3(b):
        b = b.to(torch.int32)
        e, m = (b >> 3) & 15, (b & 7).to(f64)
        size = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).to(f64)))
        return torch.where(b >= 128, -size, size)

    if fmt == "mxfp8":
        v = e4m3(codes)
    else:
        c = torch.empty(rows * cols, device=codes.device, dtype=torch.int32)
        c[0::2], c[1::2] = codes % 16, codes // 16
        e, m = (c % 8) // 2, (c % 2).to(f64)
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).to(f64)))
        v = torch.where(c >= 8, -v, v)
    r = torch.arange(rows, device=codes.device)[:, None]
    c = torch.arange(cols // block, device=codes.device)[None, :]
    across = (cols // block + 3) // 4
    byte = q["scales"][((r // 128) * across + c // 4) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + c % 4]
    scale = e4m3(byte) * q["g"].to(f64) if fmt == "nvfp4" else torch.exp2(byte.to(f64) - 127)
    return v.reshape(rows, cols) * scale.repeat_interleave(block, 1)


def _exact_act(name, v):
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "silu":
        return v * torch.sigmoid(v)
    return torch.where(v > 0, v, torch.zeros_like(v)) if name == "relu" else v


def _exact_slope(name, v):
    v = v.detach().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(_exact_act(name, v).sum(), v)[0]


def exact(case, seed):
    s = prepare(case, seed)
    op, n, k, act = case["op"], case["n"], case["k"], case.get("act")
    f64 = torch.float64
    if op.startswith("act"):
        experts, spans = 1, [(0, case["rows"])]
    else:
        experts = case["experts"]
        spans = [(a, a + c) for a, c in zip(s["offsets"].tolist(), s["counts"].tolist())]
    if op == "expert_wgrad":
        x, dy = _exact_values(s["x"]), _exact_values(s["dy"])
        return torch.stack([dy[:, a:b] @ x[:, a:b].t() for a, b in spans])
    w = _exact_values(s["w"])
    if op in ("act", "expert_fwd"):
        x = _exact_values(s["x"])
        v, out = (torch.zeros(x.shape[0], n, dtype=f64, device="cuda") for _ in range(2))
        for e, (a, b) in enumerate(spans):
            v[a:b] = x[a:b] @ w[e * n:(e + 1) * n].t()
            if s["bias"] is not None:
                v[a:b] += s["bias"].reshape(experts, n)[e].to(f64)
            out[a:b] = _exact_act(act, v[a:b])
        if s["residual"] is not None:
            out += s["residual"].to(f64)
        return dict(out=out, pre=v) if case["pre"] else dict(out=out)
    dy = _exact_values(s["dy"])
    d, dbias = torch.zeros(dy.shape[0], k, dtype=f64, device="cuda"), torch.zeros(experts, k, dtype=f64, device="cuda")
    for e, (a, b) in enumerate(spans):
        d[a:b] = dy[a:b] @ w[:, e * n:(e + 1) * n].t()
        if s["before"] is not None:
            d[a:b] *= _exact_slope(act, s["before"][a:b].to(f64))
        dbias[e] = d[a:b].sum(0)
    if op == "act_bwd":
        dbias = dbias[0]
    return dict(dpre=d, dbias=dbias) if case["dbias"] else dict(dpre=d)
