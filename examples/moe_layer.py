"""One MoE layer, forward and backward, on the library's operators alone.

    python examples/moe_layer.py [--tokens 4096] [--width 3584] [--hidden 3072] [--experts 32] [--top-k 8]

Forward: router scores (a dense linear), top-k routing, the row plan, tokens to their experts' rows, gate/up
projection fused with SiTU-GLU, down projection, weighted rows back into the residual stream. Backward: the
fused down-projection gradient + SiTU-GLU backward + router gradient, weight gradients in fp32 (what the streamed
Adam step takes), the gate/up input gradient, rows back to tokens, and the router. The expert outputs o are not
kept: the router's gradient comes from the fused backward ("Kimi K3 模型结构（9）：显存", section "MoE 反向").

The script runs a training step and a decoding step and prints their times.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_situ_glu_gb300 as sg  # noqa: E402


class MoELayer:
    """y = x + Σ_k p_k · W_down,e · SiTU(W_gate,e x, W_up,e x) over the top-k experts e of each token.

    width D (a multiple of 64), hidden H (of 16), experts E (of 8); all weights bf16 in the nn.Linear layout."""

    def __init__(self, width, hidden, experts, top_k, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s: (torch.randn(*s, generator=g, device=device) / s[-1] ** 0.5).to(torch.bfloat16)  # noqa: E731
        self.experts, self.top_k = experts, top_k
        self.w_router = new(experts, width)
        self.w_gate_up = new(experts, 2 * hidden, width)
        self.w_down = new(experts, width, hidden)
        self.saved = None

    def forward(self, x, train=True):
        """x bf16 [T, D] -> y bf16 [T, D]; with ``train`` what backward() needs is kept."""
        logits = sg.situ_linear(x, self.w_router, out_dtype=torch.float32)
        p, ids = sg.situ_route_topk(logits, self.top_k)
        offsets, row_of, _, p_rows = sg.situ_dispatch_plan(ids, self.experts, p=p)
        h = sg.situ_dispatch(x, row_of, offsets)
        pre, act = sg.situ_glu_fwd_gateup(h, self.w_gate_up, offsets)
        o = sg.situ_linear(act, self.w_down, expert_offsets=offsets)
        if train:
            self.saved = (x, p, ids, offsets, row_of, p_rows, h, pre, act)
        return sg.situ_combine(o, row_of, weights=p, residual=x)

    def backward(self, dy):
        """dy bf16 [T, D] -> dict of dx (bf16) and the weights' gradients (fp32)."""
        x, p, ids, offsets, row_of, p_rows, h, pre, act = self.saved
        self.saved = None
        dy_rows = sg.situ_dispatch(dy, row_of, offsets)
        dpre, dp_rows = sg.situ_glu_bwd_router_dgrad_wd(pre, dy_rows, self.w_down, offsets, p_rows)
        do = sg.situ_dispatch(dy, row_of, offsets, weights=p)                # the experts' output gradient
        _, dw_down, _ = sg.situ_linear_bwd(do, act, self.w_down, offsets, bias=False, need_da=False)
        dh, dw_gate_up, _ = sg.situ_linear_bwd(dpre, h, self.w_gate_up, offsets, bias=False)
        dlogits = sg.situ_route_topk_bwd(ids, p, dp_rows, self.experts, dtype=torch.bfloat16, row_of=row_of)
        dx_router, dw_router, _ = sg.situ_linear_bwd(dlogits, x, self.w_router, bias=False)
        dx = sg.situ_combine(dh, row_of, residual=dy)                        # rows back to tokens, and the residual path
        return dict(dx=dx.add_(dx_router), dw_router=dw_router, dw_gate_up=dw_gate_up, dw_down=dw_down)


def timed(f, n=10):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=3584)
    ap.add_argument("--hidden", type=int, default=3072)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=8)
    a = ap.parse_args()
    layer = MoELayer(a.width, a.hidden, a.experts, a.top_k)
    x = torch.randn(a.tokens, a.width, device="cuda").to(torch.bfloat16)
    dy = torch.randn_like(x)

    def step():
        layer.forward(x)
        return layer.backward(dy)

    grads = step()
    assert all(torch.isfinite(g.sum()) for g in grads.values())
    print(f"training step, {a.tokens} tokens, {a.experts} experts, top {a.top_k}: {timed(step):.3f} ms")
    one = x[:8].contiguous()
    print(f"decoding step, 8 tokens: {timed(lambda: layer.forward(one, train=False)):.3f} ms")


if __name__ == "__main__":
    main()
