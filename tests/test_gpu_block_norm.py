"""block_norm and block_norm_backward against the formulas in 64 bits.

Tolerances count roundings (u = 2^-24 for fp32, half a step of the output type at the end), carried
through the formulas term by term: a sum of n terms in any order is off by at most n u times the sum
of magnitudes; the row sums here add at most 16 values in a lane, 5 shuffles and one value a warp,
so k = 32 + warps covers them with the few operations around them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F64 = torch.float64


def _bsq():
    import block_scaled_precision_bsq_gb300 as bsq

    return bsq


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def depth(cols):
    return 32 + cols // 256


def rand(gen, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(dtype)


class Case:
    """Inputs of one shape, and what the formulas make of them in 64 bits with error bounds."""

    def __init__(self, rows, cols, kind="layer", dtype=torch.bfloat16, params=torch.bfloat16, post=True, bias=True,
                 gate=True, groups=1, scale=0.75, offset=0.0, eps=1e-6, seed=0, mean=0.3):
        self.rows, self.cols, self.kind, self.dtype = rows, cols, kind, dtype
        self.post, self.groups, self.scale, self.offset, self.eps = post, groups, scale, offset, eps
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.h = rand(g, rows, cols, std=0.7, mean=mean, dtype=dtype)
        self.x = rand(g, rows, cols, std=2.0, mean=mean, dtype=dtype)
        self.w1 = rand(g, cols, std=0.2, mean=1 - offset, dtype=params) if post else None
        self.b1 = rand(g, cols, std=0.2, dtype=params) if post and bias else None
        self.gate = rand(g, *((groups, cols) if groups > 1 else (cols,)), std=0.5, mean=0.2, dtype=params) \
            if gate else None
        self.w2 = rand(g, cols, std=0.2, mean=1 - offset, dtype=params)
        self.b2 = rand(g, cols, std=0.2, dtype=params) if bias else None
        self.dxo = rand(g, rows, cols, std=0.1, dtype=dtype)
        self.dy = rand(g, rows, cols, std=0.1, dtype=dtype)

    def kw(self):
        return dict(kind=self.kind, post_norm=self.post, post_weight=self.w1, post_bias=self.b1, gate=self.gate,
                    residual_scale=self.scale, pre_weight=self.w2, pre_bias=self.b2, weight_offset=self.offset)

    def d(self, t, default):
        return torch.full((1,), default, device="cuda", dtype=F64) if t is None else t.to(F64)

    def weight(self, t):
        return torch.ones(1, device="cuda", dtype=F64) if t is None else t.to(F64) + self.offset

    def gate_rows(self):
        if self.gate is None:
            return torch.ones(1, device="cuda", dtype=F64)
        gt = self.gate.to(F64)
        return gt if gt.dim() == 1 else gt.repeat_interleave(self.rows // self.groups, 0)

    def moments(self, v):
        mu = v.mean(1, keepdim=True) if self.kind == "layer" else torch.zeros_like(v[:, :1])
        return mu, ((v - mu).square().mean(1, keepdim=True) + self.eps).rsqrt()

    def norm(self, v, ev, w, b):
        """(norm(v) * w + b, its bound, mean, rstd) for v off by at most ev."""
        k = depth(self.cols)
        mu, r = self.moments(v)
        layer = self.kind == "layer"
        emu = ev.mean(1, keepdim=True) + k * U * v.abs().mean(1, keepdim=True) if layer else torch.zeros_like(mu)
        dv = (v - mu).abs()
        # relative error of rstd: half that of the mean square, which moves by 2 |v - mu| (ev + emu)
        er = r * r * (dv * (ev + emu)).mean(1, keepdim=True) + 0.5 * r * r * (ev + emu).square().mean(1, keepdim=True) + k * U
        z = (v - mu) * r
        y = z * w + b
        ey = (w * r).abs() * (ev + emu) + (z * w).abs() * (er + 6 * U) + 2 * U * b.abs()
        return y, ey, mu, r

    def forward(self):
        h, x = self.h.to(F64), self.x.to(F64)
        zero = torch.zeros(self.rows, 1, device="cuda", dtype=F64)
        mu1 = r1 = zero
        n, en = h, torch.zeros_like(h)
        if self.post:
            n, en, mu1, r1 = self.norm(h, en, self.weight(self.w1), self.d(self.b1, 0.0))
        gt = self.gate_rows()
        xo = self.scale * x + gt * n
        exo = gt.abs() * en + 3 * U * ((gt * n).abs() + (self.scale * x).abs())
        y, ey, mu2, r2 = self.norm(xo, exo, self.weight(self.w2), self.d(self.b2, 0.0))
        hs = half_step(self.dtype)
        return dict(x_out=(xo, exo + hs * (xo.abs() + exo)), y=(y, ey + hs * (y.abs() + ey)),
                    stats=torch.cat([mu1, r1, mu2, r2], 1))

    def backward(self, x_out, stats):
        """Gradients from the stored x_out and statistics (inputs of the backward pass)."""
        k = depth(self.cols)
        layer = self.kind == "layer"
        mu1, r1, mu2, r2 = stats.to(F64).split(1, 1)

        def back(g, eg, v, mu, r):
            z = (v - mu) * r
            ez = 3 * U * z.abs()
            m1 = (g * z).mean(1, keepdim=True)
            em1 = (eg * z.abs() + g.abs() * ez).mean(1, keepdim=True) + k * U * (g * z).abs().mean(1, keepdim=True)
            m0 = g.mean(1, keepdim=True) if layer else torch.zeros_like(m1)
            em0 = eg.mean(1, keepdim=True) + k * U * g.abs().mean(1, keepdim=True) if layer else torch.zeros_like(m1)
            t = g - m0 - z * m1
            et = eg + em0 + z.abs() * em1 + m1.abs() * ez + 4 * U * (g.abs() + m0.abs() + (z * m1).abs())
            return r * t, r * et + 2 * U * (r * t).abs(), z, ez

        def column(v, ev, groups=1):
            n = self.rows // groups
            v, ev = v.reshape(groups, n, -1), ev.reshape(groups, n, -1)
            return v.sum(1), ev.sum(1) + (n + 8) * U * v.abs().sum(1)

        out = {}
        dy, h = self.dy.to(F64), self.h.to(F64)
        w2 = self.weight(self.w2)
        g2 = dy * w2
        t, et, z2, ez2 = back(g2, 3 * U * g2.abs(), x_out.to(F64), mu2, r2)
        out["dpre_weight"] = column(dy * z2, dy.abs() * ez2 + U * (dy * z2).abs())
        out["dpre_bias"] = column(dy, torch.zeros_like(dy))
        d = self.dxo.to(F64) + t
        ed = et + 2 * U * (d.abs() + t.abs())
        hs = half_step(self.dtype)

        def rounded(v, ev):
            return v, ev + hs * (v.abs() + ev)

        out["dx"] = rounded(self.scale * d, abs(self.scale) * ed + U * (self.scale * d).abs())
        gt, w1, b1 = self.gate_rows(), self.weight(self.w1), self.d(self.b1, 0.0)
        if self.post:
            z1 = (h - mu1) * r1
            ez1 = 3 * U * z1.abs()
        else:
            z1, ez1 = h, torch.zeros_like(h)
        a1, ea1 = column(d * z1, ed * z1.abs() + d.abs() * ez1 + 2 * U * (d * z1).abs(), self.groups)
        a0, ea0 = column(d, ed, self.groups)
        out["dgate"] = (w1 * a1 + b1 * a0, w1.abs() * ea1 + b1.abs() * ea0 + 4 * U * ((w1 * a1).abs() + (b1 * a0).abs()))
        gg = self.d(self.gate, 1.0).reshape(self.groups if self.gate is not None else 1, -1)
        terms = self.groups + 4
        out["dpost_weight"] = ((gg * a1).sum(0), (gg.abs() * ea1 + terms * U * (gg * a1).abs()).sum(0))
        out["dpost_bias"] = ((gg * a0).sum(0), (gg.abs() * ea0 + terms * U * (gg * a0).abs()).sum(0))
        g1, eg1 = d * gt, ed * gt.abs() + 2 * U * (d * gt).abs()
        if self.post:
            g1, eg1 = g1 * w1, eg1 * w1.abs() + 3 * U * (g1 * w1).abs()
            g1, eg1, _, _ = back(g1, eg1, h, mu1, r1)
        out["dh"] = rounded(g1, eg1)
        return out


def check(got, want, what):
    ref, tol = want
    assert got.shape == ref.squeeze(0).shape or got.numel() == ref.numel(), (what, got.shape, ref.shape)
    err = (got.to(F64).reshape(ref.shape) - ref).abs()
    tol = tol + 1e-37
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its tolerance" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).max()))


def run(c, rows=None):
    bsq = _bsq()
    f = bsq.block_norm(c.h, c.x, eps=c.eps, **c.kw())
    want = c.forward()
    check(f.x_out, want["x_out"], "x_out")
    check(f.y, want["y"], "y")
    rel = (f.stats.to(F64) - want["stats"]).abs()
    scale = want["stats"].abs()
    scale[:, 0] += c.h.to(F64).abs().mean(1)
    scale[:, 2] += want["x_out"][0].abs().mean(1)
    # a mean is off by k u mean|v|, rstd by k u of itself and what the mean and x_out move it by
    assert (rel <= 8 * depth(c.cols) * U * scale + 1e-37).all(), float((rel / (scale + 1e-37)).max())
    r = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    want = c.backward(f.x_out, f.stats)
    for name, given in (("dx", True), ("dh", True), ("dpost_weight", c.w1), ("dpost_bias", c.b1), ("dgate", c.gate),
                        ("dpre_weight", c.w2), ("dpre_bias", c.b2)):
        v = getattr(r, name)
        assert (v is None) == (given is None), name
        if v is not None:
            check(v, want[name], name)
    return f, r


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 31, 64, 100, 512, 520, 768, 1001, 1024, 1032, 2056, 4096, 4100, 5000, 8192])
def test_widths(cols, dtype, kind):
    run(Case(19, cols, kind, dtype, seed=cols))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 8200), (torch.bfloat16, 8201), (torch.bfloat16, 20000),
                                        (torch.bfloat16, 65536), (torch.float32, 4104), (torch.float32, 12289),
                                        (torch.float32, 32768)])
def test_rows_over_a_cluster(cols, dtype, kind):
    run(Case(5, cols, kind, dtype, seed=cols))
    run(Case(330, cols, kind, dtype, groups=2, seed=cols))


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 151, 1217, 5000])
@pytest.mark.parametrize("cols", [64, 264, 1024, 4096])
def test_row_counts(rows, cols):
    run(Case(rows, cols, "layer", torch.bfloat16, seed=rows))
    run(Case(rows, cols, "rms", torch.bfloat16, bias=False, post=False, seed=rows))


@pytest.mark.parametrize("params", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,bias,gate,offset", [(True, True, True, 0.0), (True, False, False, 1.0),
                                                   (False, True, True, 0.0), (False, False, False, 0.0),
                                                   (True, True, False, 0.0), (True, False, True, 1.0)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_parts(kind, post, bias, gate, offset, dtype, params):
    run(Case(37, 392, kind, dtype, params, post, bias, gate, offset=offset, seed=5))


@pytest.mark.parametrize("rows,groups", [(12, 12), (700, 7), (330, 2), (64, 16), (96, 32), (1000, 1000), (5000, 5)])
@pytest.mark.parametrize("cols", [96, 1001, 4096])
def test_gate_groups(rows, groups, cols):
    run(Case(rows, cols, "layer", torch.bfloat16, groups=groups, seed=groups))


def test_large_mean_small_spread():
    # mean 100 spreads: the second moment about a rough mean would lose most of its bits
    run(Case(40, 2000, "layer", torch.float32, torch.float32, mean=300.0, seed=3))


def test_outlier_channels_and_tiny_rows():
    c = Case(40, 1024, "layer", torch.bfloat16, seed=4)
    c.x[:, ::200] *= 64
    c.h[7] = 0
    c.x[7] = 0
    c.h[9] *= 2.0 ** -60
    run(c)


def test_first_norm_without_a_block():
    bsq = _bsq()
    for kind in ("rms", "layer"):
        c = Case(33, 520, kind, scale=1.0)
        f = bsq.block_norm(None, c.x, kind=kind, pre_weight=c.w2, pre_bias=c.b2)
        assert f.x_out is None
        x = c.x.to(F64)
        y, ey, _, _ = c.norm(x, torch.zeros_like(x), c.weight(c.w2), c.d(c.b2, 0.0))
        check(f.y, (y, ey + half_step(c.dtype) * (y.abs() + ey)), "y")
        r = bsq.block_norm_backward(None, c.dy, c.x, None, f.stats, kind=kind, pre_weight=c.w2, pre_bias=c.b2)
        c.dxo = torch.zeros_like(c.dxo)
        want = c.backward(c.x, f.stats)
        assert r.dh is None and r.dgate is None and r.dpost_weight is None
        for name in ("dx", "dpre_weight", "dpre_bias"):
            check(getattr(r, name), want[name], name)


def test_last_block_without_a_norm_after():
    bsq = _bsq()
    c = Case(33, 520, "rms", bias=False)
    kw = dict(kind="rms", post_norm=True, post_weight=c.w1, gate=c.gate, residual_scale=c.scale)
    f = bsq.block_norm(c.h, c.x, pre_norm=False, **kw)
    assert f.y is None
    check(f.x_out, c.forward()["x_out"], "x_out")
    r = bsq.block_norm_backward(c.dxo, None, None, c.h, f.stats, **kw)
    c.dy = torch.zeros_like(c.dy)
    stats = f.stats.clone()
    stats[:, 3] = 1.0
    want = c.backward(f.x_out, stats)
    assert r.dpre_weight is None
    for name in ("dx", "dh", "dpost_weight", "dgate"):
        check(getattr(r, name), want[name], name)


def test_row_strides_and_odd_addresses():
    """Rows inside wider matrices, and buffers that start one element off 16 bytes."""
    bsq = _bsq()
    for shift in (0, 1):
        for dtype in (torch.bfloat16, torch.float32):
            c = Case(21, 768, "layer", dtype)
            for name in ("h", "x", "dxo", "dy"):
                wide = torch.full((21, 800), float("nan"), dtype=dtype, device="cuda")
                view = wide[:, 8 + shift:776 + shift]
                view.copy_(getattr(c, name))
                setattr(c, name, view)
            run(c)
    # one row repeated (stride 0), as the gradient of a broadcast has it
    c = Case(21, 768, "layer")
    c.dy = c.dy[:1].expand(21, 768)
    run(c)
    del bsq


def test_in_place_outputs_give_the_same_bits():
    bsq = _bsq()
    c = Case(300, 1024, "layer")
    f = bsq.block_norm(c.h, c.x, **c.kw())
    h, x = c.h.clone(), c.x.clone()
    stats = torch.empty(300, 4, device="cuda")
    g = bsq.block_norm(h, x, out=bsq.BlockNorm(x, h, stats), **c.kw())
    assert torch.equal(g.x_out, f.x_out) and torch.equal(g.y, f.y) and torch.equal(stats, f.stats)


def test_nan_and_infinity_stay_in_their_rows():
    bsq = _bsq()
    c = Case(40, 1000, "layer")
    clean = bsq.block_norm(c.h, c.x, **c.kw())
    c.h[3, 17] = float("nan")
    c.x[11, 999] = float("inf")
    f = bsq.block_norm(c.h, c.x, **c.kw())
    rows = [r for r in range(40) if r not in (3, 11)]
    assert torch.equal(f.y[rows], clean.y[rows]) and torch.equal(f.x_out[rows], clean.x_out[rows])
    assert f.y[3].isnan().all() and f.x_out[3].isnan().all()
    assert f.y[11].isnan().all() and torch.isinf(f.x_out[11, 999]) and torch.equal(f.x_out[11, :999], clean.x_out[11, :999])


def test_no_rows():
    bsq = _bsq()
    c = Case(2, 64)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    f = bsq.block_norm(empty, empty, **c.kw())
    assert f.y.shape == (0, 64) and f.stats.shape == (0, 4)
    r = bsq.block_norm_backward(empty, empty, f.x_out, empty, f.stats, **c.kw())
    for name in ("dpost_weight", "dpost_bias", "dgate", "dpre_weight", "dpre_bias"):
        assert torch.equal(getattr(r, name), torch.zeros(64, device="cuda"))


@pytest.mark.parametrize("cols", [768, 4096, 9000])
def test_same_bits_every_time_and_on_another_stream_and_in_a_graph(cols):
    bsq = _bsq()
    c = Case(901, cols, "layer")
    f = bsq.block_norm(c.h, c.x, **c.kw())
    r = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f2 = bsq.block_norm(c.h, c.x, stream=s, **c.kw())
    r2 = bsq.block_norm_backward(c.dxo, c.dy, f2.x_out, c.h, f2.stats, stream=s.cuda_stream, **c.kw())
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f3 = bsq.block_norm(c.h, c.x, **c.kw())
        r3 = bsq.block_norm_backward(c.dxo, c.dy, f3.x_out, c.h, f3.stats, **c.kw())
    for t in (*f3, *r3):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, d in zip((*f, *r), (*f2, *r2), (*f3, *r3)):
        assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_against_differences(kind):
    """Central differences of the 64-bit forward formula along random directions, for every input."""
    bsq = _bsq()
    c = Case(6, 88, kind, torch.float32, torch.float32, groups=2, seed=9)
    gen = torch.Generator(device="cuda").manual_seed(10)

    def loss():
        w = c.forward()
        return float((w["x_out"][0] * c.dxo.to(F64)).sum() + (w["y"][0] * c.dy.to(F64)).sum())

    f = bsq.block_norm(c.h, c.x, **c.kw())
    r = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    for name, grad in (("h", r.dh), ("x", r.dx), ("w1", r.dpost_weight), ("b1", r.dpost_bias), ("gate", r.dgate),
                       ("w2", r.dpre_weight), ("b2", r.dpre_bias)):
        keep = getattr(c, name)
        v = rand(gen, *keep.shape).to(F64)
        step = 1e-5
        setattr(c, name, keep.to(F64) + step * v)
        up = loss()
        setattr(c, name, keep.to(F64) - step * v)
        down = loss()
        setattr(c, name, keep)
        want = (up - down) / (2 * step)
        got = float((grad.to(F64) * v).sum())
        # fp32 gradients of about 500 values each: 1e-4 of the sum of magnitudes is far above both errors
        assert abs(got - want) <= 1e-5 * float((grad.to(F64) * v).abs().sum()) + 1e-7, (name, got, want)


def test_more_than_2_31_elements():
    """Rows on both sides of element 2^31 against the formulas."""
    bsq = _bsq()
    cols = 8192
    rows = (1 << 31) // cols + 5
    small = Case(8, cols, "rms", bias=False)
    reps = -(-rows // 8)
    big = {n: getattr(small, n).repeat(reps, 1)[:rows] for n in ("h", "x", "dxo", "dy")}
    f = bsq.block_norm(big["h"], big["x"], **small.kw())
    fs = bsq.block_norm(small.h, small.x, **small.kw())
    r = bsq.block_norm_backward(big["dxo"], big["dy"], f.x_out, big["h"], f.stats, param_grads=False, **small.kw())
    rs = bsq.block_norm_backward(small.dxo, small.dy, fs.x_out, small.h, fs.stats, **small.kw())
    for a, b in ((f.x_out, fs.x_out), (f.y, fs.y), (r.dx, rs.dx), (r.dh, rs.dh)):
        for at in (0, (1 << 30) // cols // 8 * 8, (1 << 31) // cols // 8 * 8 - 8, rows // 8 * 8):
            n = min(8, rows - at)
            assert torch.equal(a[at:at + n], b[:n])
    assert r.dgate is None


def test_small_workspace_is_refused():
    bsq = _bsq()
    c = Case(64, 256)
    f = bsq.block_norm(c.h, c.x, **c.kw())
    need = bsq.bsq_block_norm_backward_workspace(bsq.FLAG_POST_NORM, 64, 256, 1)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dw = torch.empty(256, device="cuda")

    def call(nbytes):
        p = lambda t: t.data_ptr()  # noqa: E731
        return bsq.bsq_block_norm_backward(bsq.BlockNormGradArgs(
            kind=2, flags=bsq.FLAG_POST_NORM, rows=64, cols=256, gate_groups=1, residual_scale=1.0, dx_out=p(c.dxo),
            dy=p(c.dy), x_out=p(f.x_out), h=p(c.h), dx_out_stride=256, dy_stride=256, x_out_stride=256, h_stride=256,
            stats=p(f.stats), pre_weight=p(c.w2), dpre_weight=p(dw), workspace=p(ws), workspace_bytes=nbytes))

    assert call(need - 1) == bsq.ERR_ARG and call(need) == bsq.OK
    assert bsq.device_status() == 0


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1, 7, 64, 100, 250, 256, 264, 505, 512, 520, 768, 1001, 1024, 2056, 4089, 4096, 4100,
                                  5000, 8192, 8200, 12352, 15200, 16384, 16385])
def test_widths_with_rows_enough_for_every_sm(cols, dtype, kind):
    """More rows than SMs: several rows a CTA at once, more elements a thread."""
    run(Case(460, cols, kind, dtype, torch.float32, seed=cols))
    run(Case(460, cols, kind, dtype, post=False, bias=False, seed=cols))


@pytest.mark.parametrize("rows", [153, 304, 2433])
@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("cols", [126, 743, 2816])
def test_rows_that_do_not_fill_the_last_round(rows, groups, cols):
    rows = rows // groups * groups
    run(Case(rows, cols, "layer", torch.bfloat16, groups=groups, seed=rows))
    run(Case(rows, cols, "rms", torch.float32, torch.float32, bias=False, groups=groups, seed=rows))


@pytest.mark.parametrize("cols", [1000, 1001, 9001])
@pytest.mark.parametrize("rows", [40, 700])
def test_nan_rows_do_not_reach_their_neighbours_gradients(rows, cols):
    """Rows that share 16-byte vectors with a row of NaN: forward and both input gradients."""
    bsq = _bsq()
    c = Case(rows, cols, "layer")
    f = bsq.block_norm(c.h, c.x, **c.kw())
    r = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    for t in (c.h, c.x, c.dxo, c.dy):
        t[3] = float("nan")
        t[rows - 1, cols - 1] = float("inf")
    f2 = bsq.block_norm(c.h, c.x, **c.kw())
    r2 = bsq.block_norm_backward(c.dxo, c.dy, f2.x_out, c.h, f2.stats, **c.kw())
    rest = [i for i in range(rows - 1) if i != 3]
    for a, b in ((f.x_out, f2.x_out), (f.y, f2.y), (f.stats, f2.stats), (r.dx, r2.dx), (r.dh, r2.dh)):
        assert torch.equal(a[rest], b[rest])
    assert f2.y[3].isnan().all() and r2.dx[3].isnan().all() and r2.dh[3].isnan().all()


def test_in_place_gradients_and_odd_widths_in_place():
    bsq = _bsq()
    for cols in (1024, 1001):
        c = Case(700, cols, "layer")
        f = bsq.block_norm(c.h, c.x, **c.kw())
        h, x = c.h.clone(), c.x.clone()
        stats = torch.empty(700, 4, device="cuda")
        g = bsq.block_norm(h, x, out=bsq.BlockNorm(x, h, stats), **c.kw())
        assert torch.equal(g.x_out, f.x_out) and torch.equal(g.y, f.y) and torch.equal(stats, f.stats)
        r = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, param_grads=False, **c.kw())
        dy, dh = c.dy.clone(), torch.empty_like(c.h)
        p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        a = bsq.BlockNormGradArgs(kind=2, flags=bsq.FLAG_POST_NORM, rows=700, cols=cols, gate_groups=1,
                                  residual_scale=c.scale, weight_offset=0.0, dx_out=p(c.dxo), dy=p(dy), x_out=p(f.x_out),
                                  h=p(c.h), dx_out_stride=cols, dy_stride=cols, x_out_stride=cols, h_stride=cols,
                                  stats=p(f.stats), post_weight=p(c.w1), post_bias=p(c.b1), gate=p(c.gate),
                                  pre_weight=p(c.w2), pre_bias=p(c.b2), dx=p(dy), dh=p(dh))
        assert bsq.bsq_block_norm_backward(a) == bsq.OK
        assert torch.equal(dy, r.dx) and torch.equal(dh, r.dh)


@pytest.mark.parametrize("after", [0, 1, 3])
@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 8192), (torch.bfloat16, 9001), (torch.float32, 32768)])
def test_a_wait_that_runs_out_reports_a_timeout(dtype, cols, after):
    """One CTA of each cluster falls silent: the others give up after the limit, nothing hangs, and the
    next call is whole again. Armed past launches on short rows."""
    import time

    bsq = _bsq()
    c = Case(700, cols, "layer", dtype)
    f = bsq.block_norm(c.h, c.x, **c.kw())
    want = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    assert bsq.device_status() == 0
    assert bsq.bsq_test_inject_stall(bsq.KERNEL_NORM, after, 2_000_000) == bsq.OK
    s = Case(40, 256, "layer")
    fs = bsq.block_norm(s.h, s.x, **s.kw())
    bsq.block_norm_backward(s.dxo, s.dy, fs.x_out, s.h, fs.stats, **s.kw())
    assert bsq.device_status() == 0
    begin = time.monotonic()
    bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    assert bsq.device_status() == bsq.ERR_TIMEOUT
    assert time.monotonic() - begin < 1.0
    got = bsq.block_norm_backward(c.dxo, c.dy, f.x_out, c.h, f.stats, **c.kw())
    assert bsq.device_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [1, 5, 17, 40, 121, 128, 300, 385])
@pytest.mark.parametrize("cols", [64, 137, 768, 1100, 2368, 4096])
@pytest.mark.parametrize("groups", [1, 5])
def test_few_rows_join_their_sums_in_one_launch(rows, cols, groups):
    rows = -(-rows // groups) * groups
    run(Case(rows, cols, "layer", torch.bfloat16, groups=groups, seed=rows))
    run(Case(rows, cols, "rms", torch.float32, torch.float32, bias=False, groups=groups, seed=rows))
