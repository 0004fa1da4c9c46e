"""One MoE layer trained by its own kernels: route, dispatch, expert FFN,
combine, and back, with SGD on the router and the experts.

    python examples/train_step.py [--layer tiny|granite|dsv2lite|...] [--tokens T] [--steps S] [--block] [--packed]

--block puts the layer into its block: a norm before it, and behind it a norm, a
gate for each channel and the residual.  --packed keeps what the backward pass
needs in 8 bits.
The forward routes with moe_route (the inference layer's router); the rest are
the training calls of include/moe_train.h.  The router's own linear map is a
plain matrix product, so its gradient is two more of those.  The target is a
fixed random linear map of the tokens (synthetic data, random weights).
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import expert_routing_ffn_gb300 as moe  # noqa: E402
from workloads import CONFIGS  # noqa: E402


class TrainLayer:
    """The weights of one MoE layer, the buffers of a step of T tokens, and the
    step's calls.  The library's calls work in buffers allocated once; the plain
    products around them (the router's linear map, the update) take their own."""

    def __init__(self, cfg, T, capacity=0, balance=0.01, renorm=True, seed=0, device="cuda", packed=False):
        self.cfg, self.T, self.capacity, self.balance, self.packed = cfg, T, capacity, balance, packed
        self.D = moe.make_dims(T, cfg.d, cfg.N, cfg.k, cfg.I, wtype=cfg.wtype, renorm_topk=int(renorm))
        self.renorm = renorm
        d, N, k, I = cfg.d, cfg.N, cfg.k, cfg.I
        kind = torch.bfloat16 if cfg.wtype == "bf16" else torch.float32
        gen = torch.Generator(device).manual_seed(seed)

        def weight(*shape):
            return torch.empty(shape, dtype=kind, device=device).normal_(0.0, 0.02, generator=gen)

        def buf(*shape, dtype=kind):
            return torch.empty(shape, dtype=dtype, device=device)

        i32, f32 = torch.int32, torch.float32
        self.w_router, self.w_gate, self.w_up, self.w_down = weight(N, d), weight(N, I, d), weight(N, I, d), weight(N, I, d)
        self.ws_route = torch.zeros(moe.moe_workspace_size(self.D), dtype=torch.uint8, device=device)
        self.ws = torch.zeros(moe.moe_train_workspace_size(self.D), dtype=torch.uint8, device=device)
        # routing
        self.topk_idx, self.topk_gate, self.prob = buf(T, k, dtype=i32), buf(T, k, dtype=f32), buf(T, N, dtype=f32)
        self.delta_hat, self.prefetch_mask = buf(T, dtype=i32), buf(T, dtype=torch.int64)
        # rows grouped by expert
        M = T * k
        self.x_perm, self.y_perm, self.h = buf(M, d), buf(M, d), buf(M, I)
        self.offsets, self.perm, self.inv = buf(N + 1, dtype=i32), buf(M, dtype=i32), buf(M, dtype=i32)
        self.out = buf(T, d)
        if packed:
            # kept until the backward pass: x once a token, g, u and y once a slot.  Nothing above is, so
            # the 16-bit rows could serve every layer of a model in turn, and here y's serve dx's
            self.x8, self.y8 = moe.packed_rows(T, d, device), moe.packed_rows(M, d, device)
            self.g8, self.u8 = moe.packed_rows(M, I, device), moe.packed_rows(M, I, device)
            self.dx_perm = self.y_perm
        else:  # kept: x_perm, y_perm, h and
            self.g, self.u = buf(M, I), buf(M, I)
            self.dx_perm = buf(M, d)
        # gradients; the weights' in float32, so that micro-batches may add up
        self.dy_perm, self.dx = buf(M, d), buf(T, d)
        self.dg, self.du = buf(M, I), buf(M, I)
        self.dgate, self.dlogits, self.loss = buf(T, k, dtype=f32), buf(T, N, dtype=f32), buf(1, dtype=f32)
        self.dw_gate, self.dw_up, self.dw_down = (torch.zeros((N, I, d), dtype=f32, device=device) for _ in range(3))
        self.dw_router = torch.zeros((N, d), dtype=f32, device=device)

    def forward(self, x):
        D = self.D
        moe.moe_route(D, x, self.w_router, None, None, None, None, None, 0.5, 0, self.topk_idx, self.topk_gate, self.prob,
                      self.delta_hat, self.prefetch_mask, None, None, self.ws_route)
        self.gate = self.topk_gate / self.topk_gate.sum(1, keepdim=True) if self.renorm else self.topk_gate
        moe.moe_dispatch_rows(D, x, self.topk_idx, self.capacity, self.x_perm, self.offsets, self.perm, self.inv, self.ws)
        if self.packed:
            moe.moe_pack_rows(x, *self.x8)
            moe.moe_experts_up_packed(D, self.x_perm, self.offsets, self.w_gate, self.w_up, *self.g8, *self.u8, self.h, self.ws)
        else:
            moe.moe_experts_up(D, self.x_perm, self.offsets, self.w_gate, self.w_up, self.g, self.u, self.h, self.ws)
        moe.moe_experts_down(D, self.h, self.offsets, self.w_down, self.y_perm, self.ws)
        if self.packed:
            moe.moe_pack_rows(self.y_perm, *self.y8)
        moe.moe_combine_rows(D, self.y_perm, self.gate, self.inv, None, self.out)
        return self.out

    def backward(self, x, dout, accumulate=False):
        """Gradients of <dout, out> + the balance loss for x and all weights."""
        D = self.D
        if self.packed:
            moe.moe_combine_rows_grad_packed(D, dout, *self.y8, self.gate, self.inv, self.dy_perm, self.dgate)
            moe.moe_experts_down_grad_packed(D, self.dy_perm, *self.g8, *self.u8, self.offsets, self.w_down, self.h, self.dg,
                                             self.du, self.dw_down, accumulate, self.ws)
            moe.moe_unpack_rows(*self.x8, self.perm, self.cfg.k, self.x_perm)
        else:
            moe.moe_combine_rows_grad(D, dout, self.y_perm, self.gate, self.inv, self.dy_perm, self.dgate)
            moe.moe_experts_down_grad(D, self.dy_perm, self.h, self.g, self.u, self.offsets, self.w_down, self.dg, self.du,
                                      self.dw_down, accumulate, self.ws)
        moe.moe_experts_up_grad(D, self.dg, self.du, self.x_perm, self.offsets, self.w_gate, self.w_up, self.dx_perm,
                                self.dw_gate, self.dw_up, accumulate, self.ws)
        moe.moe_gate_grad(D, self.prob, self.topk_idx, self.dgate, self.balance, self.dlogits, self.loss, self.ws)
        # the router's linear map: dlogits back to the tokens and to its weights
        through_router = (self.dlogits @ self.w_router.float()).to(self.dx.dtype)
        if accumulate:
            self.dw_router += self.dlogits.T @ x.float()
        else:
            torch.matmul(self.dlogits.T, x.float(), out=self.dw_router)
        moe.moe_dispatch_rows_grad(D, self.dx_perm, self.inv, through_router, self.dx)
        return self.dx

    def weights(self):
        """(weight, its gradient)"""
        return [(self.w_router, self.dw_router), (self.w_gate, self.dw_gate), (self.w_up, self.dw_up), (self.w_down, self.dw_down)]

    def step(self, lr):
        for w, dw in self.weights():
            w.sub_(lr * dw)

    def check(self):
        st, det = moe.moe_check(self.ws)
        if st != moe.MOE_OK:
            raise RuntimeError(f"{moe.status_string(st)} ({det})")


class TrainBlock(TrainLayer):
    """The layer in its block: n = norm(x), y = layer(n), out = x + scale gate norm(y),
    and out's norm, which is the next block's input."""

    def __init__(self, cfg, T, scale=0.5, **kw):
        super().__init__(cfg, T, **kw)
        kind, f32, d, device = self.out.dtype, torch.float32, cfg.d, self.out.device
        self.block = moe.make_block(residual_scale=scale, gate=moe.MOE_GATE_CHANNEL)
        self.w_pre, self.w_post, self.w_next = (torch.ones(d, dtype=kind, device=device) for _ in range(3))
        self.w_chan = torch.ones(d, dtype=kind, device=device)
        self.n, self.stream, self.next, self.dlayer, self.dres, self.din = (torch.empty((T, d), dtype=kind, device=device) for _ in range(6))
        self.rstd_pre, self.rstd_post, self.rstd_next = (torch.empty(T, dtype=f32, device=device) for _ in range(3))
        self.dw_pre, self.dw_post, self.dw_next, self.dw_chan = (torch.zeros(d, dtype=f32, device=device) for _ in range(4))

    def forward(self, x):
        moe.moe_norm_rows(self.D, x, self.w_pre, self.block.eps, self.block.weight_offset, self.n, self.rstd_pre)
        y = super().forward(self.n)
        moe.moe_block_out(self.D, self.block, y, x, self.w_chan, self.w_post, self.w_next, self.stream, self.next, self.rstd_post,
                          self.rstd_next)
        return self.next

    def backward(self, x, dnext, accumulate=False, dstream=None):
        """Gradients of <dnext, next> + <dstream, stream> + the balance loss."""
        D = self.D
        moe.moe_block_out_grad(D, self.block, dstream, dnext, self.out, self.stream, self.w_chan, self.w_post, self.w_next,
                               self.rstd_post, self.rstd_next, self.dres, self.dlayer, self.dw_chan, self.dw_post, self.dw_next,
                               accumulate, self.ws)
        dn = super().backward(self.n, self.dlayer, accumulate)
        moe.moe_norm_rows_grad(D, dn, x, self.rstd_pre, self.w_pre, self.block.weight_offset, self.dres, self.din, self.dw_pre,
                               accumulate, self.ws)
        return self.din

    def weights(self):
        return super().weights() + [(self.w_pre, self.dw_pre), (self.w_post, self.dw_post), (self.w_next, self.dw_next),
                                    (self.w_chan, self.dw_chan)]


def train(layer="tiny", tokens=64, steps=20, lr=None, seed=0, block=False, packed=False):
    """SGD on a fixed random linear target; the losses, step by step.  The
    gradients grow with the width, and the curvature with the width over the
    tokens where these are few, so the default rate falls with both."""
    cfg = CONFIGS[layer]
    lr = 300.0 / cfg.d * min(1.0, 8.0 * tokens / cfg.d) if lr is None else lr
    L = (TrainBlock if block else TrainLayer)(cfg, tokens, seed=seed, packed=packed)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    kind = L.out.dtype
    target_map = torch.randn(cfg.d, cfg.d, device="cuda", generator=gen) / cfg.d ** 0.5
    x = torch.randn(tokens, cfg.d, device="cuda", generator=gen).to(kind)
    target = 0.1 * (x.float() @ target_map)
    losses = []
    for _ in range(steps):
        diff = L.forward(x).float() - target
        losses.append(0.5 * diff.square().sum(1).mean())
        L.backward(x, (diff / tokens).to(kind))
        L.step(lr)
    L.check()
    return [float(v) for v in losses]


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--layer", default="tiny", choices=sorted(CONFIGS))
    a.add_argument("--tokens", type=int, default=64)
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--lr", type=float, default=None)
    a.add_argument("--block", action="store_true")
    a.add_argument("--packed", action="store_true")
    a = a.parse_args()
    for i, loss in enumerate(train(a.layer, a.tokens, a.steps, a.lr, block=a.block, packed=a.packed)):
        print(f"step {i:3d}  loss {loss:.5f}")


if __name__ == "__main__":
    main()
