"""Training steps of one residual block of experts with block-scaled linear layers.

    x -> norm -> router -> tokens sorted by expert -> fc1, GELU, fc2 of each expert (MXFP8) ->
    weighted sum back in token order -> norm after the block, LayerScale, residual -> next norm

and back through all of it, ending with the global gradient norm, clipping and an SGD update.
Everything around the linear layers runs in this package's operators (block_norm, expert_*,
clip_grad_norm); the router's small softmax and the GELU's derivative are torch's.

Run it on a GB300: python examples/expert_block_step.py [--tokens 4096] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_bsq_gb300 as bsq  # noqa: E402

FMT = "mxfp8"
ALIGN = 128  # an expert's rows fill whole scale tiles: its segment is a GEMM operand by itself


class ExpertBlock:
    def __init__(self, width=1024, hidden=2048, experts=8, topk=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape, std):
            return torch.randn(*shape, device="cuda", generator=gen) * std

        self.width, self.hidden, self.experts, self.topk = width, hidden, experts, topk
        # fp32 master parameters; the linear layers quantize bf16 copies
        self.params = dict(router=rnd(experts, width, std=0.02), fc1=rnd(experts, hidden, width, std=0.02),
                           fc2=rnd(experts, width, hidden, std=0.02), gate=torch.full((width,), 0.1, device="cuda"),
                           in_weight=torch.ones(width, device="cuda"), in_bias=torch.zeros(width, device="cuda"),
                           post_weight=torch.ones(width, device="cuda"), post_bias=torch.zeros(width, device="cuda"),
                           out_weight=torch.ones(width, device="cuda"), out_bias=torch.zeros(width, device="cuda"))

    def step(self, x, target, lr=0.1, max_norm=1.0):
        """One step on x (tokens x width, bf16); returns (loss, gradient norm before clipping)."""
        p, f32, bf16 = self.params, torch.float32, torch.bfloat16
        # --- forward
        first = bsq.block_norm(None, x, pre_weight=p["in_weight"], pre_bias=p["in_bias"])
        probs = torch.softmax(first.y.to(f32) @ p["router"].t(), dim=-1)
        chosen, ids = probs.topk(self.topk, dim=-1)
        weights = (chosen / chosen.sum(-1, keepdim=True)).contiguous()
        order = bsq.expert_sort(ids, self.experts, align=ALIGN)
        rows = bsq.expert_gather(first.y, order.position, order.slot)
        offsets = order.offsets.tolist()  # the experts' segments, for the GEMMs' launches
        out_rows = torch.zeros_like(rows)
        kept = []
        for e in range(self.experts):
            a, b = offsets[e], offsets[e + 1]
            if a == b:
                kept.append(None)
                continue
            w1_row, w1_col = bsq.quantize_dual(FMT, p["fc1"][e].to(bf16))
            w2_row, w2_col = bsq.quantize_dual(FMT, p["fc2"][e].to(bf16))
            x_row, x_col = bsq.quantize_dual(FMT, rows[a:b])
            pre = bsq.gemm(x_row, w1_row)
            h_row, h_col = bsq.quantize_dual(FMT, torch.nn.functional.gelu(pre))
            bsq.gemm(h_row, w2_row, out=out_rows[a:b])
            kept.append((pre, x_col, w1_col, h_col, w2_col))
        h = bsq.expert_combine(out_rows, order.position, weights)
        norm = dict(post_norm=True, post_weight=p["post_weight"], post_bias=p["post_bias"], gate=p["gate"],
                    pre_weight=p["out_weight"], pre_bias=p["out_bias"])
        last = bsq.block_norm(h, x, **norm)
        error = last.y.to(f32) - target.to(f32)
        loss = error.square().mean()

        # --- backward
        g = {}
        dy = (error * (2.0 / error.numel())).to(bf16)
        back = bsq.block_norm_backward(None, dy, last.x_out, h, last.stats, **norm)
        g.update(post_weight=back.dpost_weight, post_bias=back.dpost_bias, gate=back.dgate,
                 out_weight=back.dpre_weight, out_bias=back.dpre_bias)
        dout_rows, dweights = bsq.expert_combine_backward(back.dh, out_rows, order.position, order.slot, weights)
        drows = torch.zeros_like(rows)
        g["fc1"], g["fc2"] = torch.zeros_like(p["fc1"]), torch.zeros_like(p["fc2"])
        for e in range(self.experts):
            if kept[e] is None:
                continue
            a, b = offsets[e], offsets[e + 1]
            pre, x_col, w1_col, h_col, w2_col = kept[e]
            dh_rows, dw2 = bsq.linear_backward(dout_rows[a:b], h_col, w2_col)
            v = pre.to(f32)
            slope = 0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) * 0.3989422804014327
            dx_rows, dw1 = bsq.linear_backward((dh_rows.to(f32) * slope).to(bf16), x_col, w1_col)
            drows[a:b] = dx_rows
            g["fc1"][e], g["fc2"][e] = dw1.to(f32), dw2.to(f32)
        dy_in = bsq.expert_gather_backward(drows, order.position).to(f32)
        # router: through the renormalised weights of the chosen experts and the softmax
        total = chosen.sum(-1, keepdim=True)
        dchosen = (dweights - (dweights * weights).sum(-1, keepdim=True)) / total
        dprobs = torch.zeros_like(probs).scatter_(1, ids, dchosen)
        dlogits = probs * (dprobs - (dprobs * probs).sum(-1, keepdim=True))
        g["router"] = dlogits.t() @ first.y.to(f32)
        dy_in = (dy_in + dlogits @ p["router"]).to(bf16)
        back_in = bsq.block_norm_backward(None, dy_in, x, None, first.stats, pre_weight=p["in_weight"],
                                          pre_bias=p["in_bias"])
        g.update(in_weight=back_in.dpre_weight, in_bias=back_in.dpre_bias)

        # --- update
        names = sorted(g)
        total_norm = bsq.clip_grad_norm([g[n] for n in names], max_norm)
        for n in names:
            p[n].sub_(g[n], alpha=lr)
        self.grads, self.dx = g, back.dx + back_in.dx
        return loss, total_norm


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    args = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(args.tokens, args.width, device="cuda", generator=gen).to(torch.bfloat16)
    target = torch.randn(args.tokens, args.width, device="cuda", generator=gen).to(torch.bfloat16)
    block = ExpertBlock(args.width, args.hidden)
    for i in range(args.steps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        loss, norm = block.step(x, target, lr=2.0, max_norm=0.5)
        end.record()
        torch.cuda.synchronize()
        print("step %d  loss %.5f  gradient norm %.4f  %.2f ms" % (i, float(loss), float(norm), begin.elapsed_time(end)))
    status = bsq.device_status()
    assert status == bsq.OK, bsq.bsq_strerror(status)


if __name__ == "__main__":
    main()
