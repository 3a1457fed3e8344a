"""A mixture-of-experts block in MXFP8: training steps, and single tokens through it.

    out = x + sum over the chosen experts e of w_e * down_e(silu(gate_e(h)) * up_e(h)),   h = layer_norm(x)

Everything between the products runs on the library's own calls: layer_norm, route, moe_plan,
moe_dispatch, the quantizers and grouped GEMMs, moe_combine, their gradients, and
clip_grad_norm over all of the block's gradients.  The router's own product (FP32) and, unless the
block keeps it in 8 bits, the activation between the projections are plain torch.

With checkpoint8 the activation's input is kept for the backward pass in 8 bits (activation,
activation_backward) instead of 16, and its output not at all.  quantize_for_serving keeps the experts'
weights in MXFP4 too, and decode() runs rows through them: half the bytes that a token's experts cost.

    python examples/moe_block.py                      # a few training steps, then one token at a time
    python examples/moe_block.py --tokens 16384 --hidden 4096 --inter 2048 --experts 128 --topk 8 --steps 3
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mxfp8_microscaled_precision_gb300 import mxq, workloads  # noqa: E402


class MoEBlock:
    """hidden a multiple of 128, inter a multiple of 128 (the grouped GEMMs' shapes)."""

    def __init__(self, hidden, inter, experts, topk, seed=0, device="cuda", checkpoint8=False):
        self.H, self.I, self.E, self.k = hidden, inter, experts, topk
        self.checkpoint8 = checkpoint8
        self.norm_w = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.norm_b = torch.zeros(hidden, dtype=torch.bfloat16, device=device)
        self.router = workloads.normal((experts, hidden), 0.02, seed + 1, device=device).float()
        self.bias = torch.zeros(experts, device=device)   # balances the load, moved by balance()
        self.w_gate_up = workloads.normal((experts, 2 * inter, hidden), 0.02, seed + 2, device=device)
        self.w_down = workloads.normal((experts, hidden, inter), 0.02, seed + 3, device=device)
        self.quantize_weights()

    def parameters(self):
        return [self.norm_w, self.norm_b, self.router, self.w_gate_up, self.w_down]

    def quantize_weights(self):
        """Row copies (forward) and column copies (dgrad) of the experts' weights."""
        E, H, I = self.E, self.H, self.I
        q, s, qc, sc = mxq.quant_1x32_dual_batched(self.w_gate_up)
        self.gu = (q.view(E * 2 * I, H), s.view(-1)), (qc.view(E * H, 2 * I), sc.view(-1))
        q, s, qc, sc = mxq.quant_1x32_dual_batched(self.w_down)
        self.dn = (q.view(E * H, I), s.view(-1)), (qc.view(E * I, H), sc.view(-1))

    def _experts(self, a, weight, offsets, N, K):
        q, s, _, _ = mxq.quant_1x32_dual(a, col=False)
        return mxq.grouped_gemm(q, s, *weight, offsets, N, K, workspace="alloc")

    def forward(self, x, token_mask=None):
        """x bf16 [T, H]; token_mask: 0 for padding tokens, which pass through.  Returns
        (out [T, H], what backward needs)."""
        h, mean, rstd = mxq.layer_norm(x, self.norm_w, self.norm_b)
        logits = h.float() @ self.router.t()
        ids, weights = mxq.route(logits, self.k, score="sigmoid", bias=self.bias, token_mask=token_mask)
        offsets, rows = mxq.moe_plan(ids, self.E)
        a = mxq.moe_dispatch(h, rows)
        z = self._experts(a, self.gu[0], offsets, 2 * self.I, self.H)
        if self.checkpoint8:
            act, *z = mxq.activation(z)   # what is kept of z: payload and scales
        else:
            act = torch.nn.functional.silu(z[:, :self.I]) * z[:, self.I:]
        y = self._experts(act, self.dn[0], offsets, self.H, self.I)
        if self.checkpoint8:
            act = None   # computed again in the backward pass
        out = x + mxq.moe_combine(y, rows, weights)
        return out, (x, h, mean, rstd, logits, ids, weights, offsets, rows, a, z, act, y)

    def backward(self, dout, saved):
        """(dx, gradients in the order of parameters())."""
        x, h, mean, rstd, logits, ids, weights, offsets, rows, a, z, act, y = saved
        I, N = self.I, a.shape[0]
        dy, dweights = mxq.moe_combine_backward(dout, y, rows, weights)
        dact = self._experts(dy, self.dn[1], offsets, I, self.H)
        if self.checkpoint8:
            dz, act = mxq.activation_backward(dact, *z)
        else:
            g, u = z[:, :I].float(), z[:, I:].float()
            sig = torch.sigmoid(g)
            dz = torch.cat([dact * u * sig * (1 + g * (1 - sig)), dact * g * sig], 1).to(torch.bfloat16)
        da = self._experts(dz, self.gu[1], offsets, self.H, 2 * I)
        cols = lambda t: mxq.quant_cols_grouped(t, offsets)  # noqa: E731
        d_down = mxq.grouped_gemm_wgrad(*cols(dy), *cols(act), offsets, N)
        d_gate_up = mxq.grouped_gemm_wgrad(*cols(dz), *cols(a), offsets, N)
        dlogits = mxq.route_backward(dweights, logits, ids, score="sigmoid")
        dh = (mxq.moe_combine(da, rows).float() + dlogits @ self.router).to(torch.bfloat16)
        d_router = dlogits.t() @ h.float()
        dx, d_norm_w, d_norm_b = mxq.layer_norm_backward(dh, x, self.norm_w, mean, rstd)
        return dx + dout, [d_norm_w, d_norm_b, d_router, d_gate_up, d_down]

    def quantize_for_serving(self):
        """The experts' weights in MXFP4, for decode()."""
        E, H, I = self.E, self.H, self.I
        self.gu4 = mxq.quant_mxfp4(self.w_gate_up, col=False)[:2]
        self.dn4 = mxq.quant_mxfp4(self.w_down, col=False)[:2]

    def decode(self, x, token_mask=None):
        """The block's output for x bf16 [T, H] through the MXFP4 weights; nothing is kept."""
        h, _, _ = mxq.layer_norm(x, self.norm_w, self.norm_b)
        ids, weights = mxq.route(h.float() @ self.router.t(), self.k, score="sigmoid", bias=self.bias, token_mask=token_mask)
        offsets, rows = mxq.moe_plan(ids, self.E)
        z = mxq.grouped_gemm_mxfp4(*mxq.quant_mxfp4_grouped(mxq.moe_dispatch(h, rows), offsets), *self.gu4, offsets,
                                   2 * self.I, self.H)
        act, _, _ = mxq.activation(z, checkpoint=False)
        y = mxq.grouped_gemm_mxfp4(*mxq.quant_mxfp4_grouped(act, offsets), *self.dn4, offsets, self.H, self.I)
        return x + mxq.moe_combine(y, rows, weights)

    def balance(self, offsets, rate=1e-3):
        """Moves the bias of experts with more rows than the mean down, of the others up."""
        load = (offsets[1:] - offsets[:-1]).float()
        self.bias += rate * torch.sign(load.mean() - load)

    def step(self, x, target, lr=0.3, max_norm=1.0):
        """One step of gradient descent on the squared error of a token, the mean over the
        tokens; (loss, gradient norm) on the device."""
        out, saved = self.forward(x)
        diff = out.float() - target.float()
        dout = (diff * (2.0 / diff.shape[0])).to(torch.bfloat16)
        _, grads = self.backward(dout, saved)
        norm, grads = mxq.clip_grad_norm(grads, max_norm, out=grads)
        for p, g in zip(self.parameters(), grads):
            p.sub_((lr * g.float()).to(p.dtype))
        self.balance(saved[7])
        self.quantize_weights()
        return diff.square().sum(1).mean(), norm


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 2048), ("hidden", 512), ("inter", 256), ("experts", 16), ("topk", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--lr", type=float, default=1.0)
    ap.add_argument("--checkpoint8", action="store_true", help="keep the activation's input in 8 bits")
    a = ap.parse_args()
    block = MoEBlock(a.hidden, a.inter, a.experts, a.topk, checkpoint8=a.checkpoint8)
    x = workloads.normal((a.tokens, a.hidden), 1.0, 7, device="cuda")
    target = workloads.normal((a.tokens, a.hidden), 1.0, 7, device="cuda") * 0.5
    for i in range(a.steps):
        torch.cuda.synchronize()
        began = time.perf_counter()
        loss, norm = block.step(x, target, lr=a.lr)
        torch.cuda.synchronize()
        took = (time.perf_counter() - began) * 1e3
        print(f"step {i}: loss {float(loss):.5f}  gradient norm {float(norm):.4g}  {took:.2f} ms")
    for t in range(3):   # one token at a time
        torch.cuda.synchronize()
        began = time.perf_counter()
        out, _ = block.forward(x[t:t + 1])
        torch.cuda.synchronize()
        print(f"token {t}: {(time.perf_counter() - began) * 1e6:.0f} us, |out| {float(out.float().norm()):.4f}")
    block.quantize_for_serving()
    for t in range(3):   # the same through the weights in 4 bits
        torch.cuda.synchronize()
        began = time.perf_counter()
        out = block.decode(x[t:t + 1])
        torch.cuda.synchronize()
        print(f"token {t} in 4 bits: {(time.perf_counter() - began) * 1e6:.0f} us, |out| {float(out.float().norm()):.4f}")
    status = mxq.get_device_status()
    if status:
        raise RuntimeError(mxq.status_string(status))


if __name__ == "__main__":
    main()
