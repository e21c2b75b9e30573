"""One MoE layer with the library's calls, serving and training.

    python examples/moe_layer.py            # a decode step, then a training step, each checked

`ServedLayer` routes and dispatches a batch, multiplies every expert's rows by its 4-bit weights
(gate and up with silu, then down) and combines: four calls, all of which a CUDA graph can hold.
`TrainedLayer` computes the layer with per-expert scales in the experts' place, the router's
balance and z loss, and the gradients of rows, experts and router logits.  `TrainedBlock` is a whole
block of a model that trains: residual addition and RMS norm, router, experts with bf16 weights,
combine, and the gradients of its inputs and of all its weights.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_moe_route_06_gb300 as moe  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantize(w):
    """Weights [E, rows, K] to E2M1 codes, an E4M3 scale per 16 columns and a factor per expert."""
    E, rows, K = w.shape
    factor = w.abs().amax((1, 2)).float() / (448 * 6)
    whole = torch.where(factor > 0, factor, 1.0)             # (an expert of zeros stays one)
    groups = w.float().view(E, rows, K // 16, 16) / whole[:, None, None, None]
    scales = (groups.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    q = groups / scales.float().clamp(min=2.0 ** -9).unsqueeze(-1)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = (torch.bucketize(q.abs(), mids) + 8 * (q < 0)).to(torch.uint8).view(E, rows, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scales.view(torch.uint8), factor


def dequantize(codes, scales, factor):
    E, rows, half = codes.shape
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    w = values[torch.stack((codes & 15, codes >> 4), -1).int()].view(E, rows, half // 8, 16)
    scales = scales.view(torch.float8_e4m3fn).float() * factor[:, None, None]
    return (w * scales.unsqueeze(-1)).view(E, rows, 2 * half)


def packed(codes, scales, gated):
    E, rows, half = codes.shape
    w4 = torch.empty(moe.moe_w4_bytes(E, rows // 2 if gated else rows, 2 * half, gated),
                     dtype=torch.uint8, device=codes.device)
    moe.moe_w4_pack(codes, scales, w4, gated=gated)
    return w4


class ServedLayer:
    """E experts of width F with 4-bit weights: gate_up [E, 2F, H], down [E, H, F]."""

    def __init__(self, T, H, F, E, k, P, gate_up, down, block_rows):
        self.path = moe.MoePath(1, T, H, E, k, P, layout="masked", block_rows=block_rows)
        self.block_rows = block_rows
        codes, scales, self.f_gate_up = quantize(gate_up)
        self.gate_up = packed(codes, scales, True)
        codes, scales, self.f_down = quantize(down)
        self.down = packed(codes, scales, False)
        rows = E * block_rows
        self.h = torch.empty((rows, F), dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(max(moe.moe_expert_product_w4_workspace_bytes(rows, E, F, H),
                                  moe.moe_expert_product_w4_workspace_bytes(rows, E, H, F)),
                              dtype=torch.uint8, device="cuda")

    def step(self, logits, x):
        p = self.path
        p.dispatch_fused(logits, x)
        by = dict(masked_counts=p.masked_counts, block_rows=self.block_rows, dev_status=p.dev_status)
        moe.moe_expert_product_w4(p.recv, self.gate_up, self.f_gate_up, self.h, self.ws, gated=True, **by)
        moe.moe_expert_product_w4(self.h, self.down, self.f_down, self.y, self.ws, **by)
        p.combine(self.y)
        return p.out


class TrainedLayer:
    """y_e = scale_e x in the experts' place; balance and z loss with their coefficients."""

    def __init__(self, S, T, H, E, k, P, balance=0.01, z=0.001):
        f32, i32, bf16 = (dict(dtype=d, device="cuda")
                          for d in (torch.float32, torch.int32, torch.bfloat16))
        self.path = moe.MoePath(S, T, H, E, k, P)
        self.d_losses = torch.tensor([balance, z], **f32)
        self.counts, self.prob = torch.empty((S, E), **i32), torch.empty((S, E), **f32)
        self.lse, self.n_valid = torch.empty((S, T), **f32), torch.empty((S,), **i32)
        self.losses = torch.empty((2,), **f32)
        self.ws = torch.empty(moe.moe_balance_loss_workspace_bytes(S, T, E), dtype=torch.uint8,
                              device="cuda")
        self.ones = torch.ones((S, T, k), **f32)
        rows = self.path.cap_recv
        self.d_y, self.d_recv = (torch.empty((rows, H), **bf16) for _ in range(2))
        self.d_w = torch.empty((S, T, k), **f32)
        self.d_x = torch.empty((S, T, H), **bf16)
        self.d_logits = torch.empty((S, T, E), **f32)

    def forward(self, logits, x, scale, mask=None):
        """The layer's output, and the losses [2] before their coefficients."""
        p = self.path
        out = p.step(logits, x, scale)
        moe.moe_balance_loss(logits, p.topk_ids, self.counts, self.prob, self.lse, self.n_valid,
                             self.losses, self.ws, token_mask=mask, dev_status=p.dev_status)
        return out, self.losses

    def backward(self, d_out, logits, scale, mask=None):
        """Gradients of the rows and of the router logits, from the output's and the losses'."""
        p = self.path
        moe.moe_combine_backward(d_out, p.y, p.pair_row, p.topk_w, self.d_y, self.d_w,
                                 recv_pair=p.recv_pair, dev_status=p.dev_status)
        # the experts' own backward: here y = scale x, so the rows' gradients are scaled
        moe.moe_expert_scale(self.d_y, p.expert_offsets, scale, self.d_recv)
        # a row was copied to its pairs: its gradient is their sum
        moe.moe_combine(self.d_recv, p.pair_row, self.ones, self.d_x, p.dev_status)
        moe.moe_route_backward(logits, p.topk_ids, p.topk_w, self.d_w, self.lse, self.counts,
                               self.n_valid, self.d_losses, self.d_logits, token_mask=mask,
                               dev_status=p.dev_status)
        return self.d_x, self.d_logits


class TrainedBlock:
    """h = x + residual, out = experts(norm(h)) by the router's picks; the block's outputs are out and h.

    norm [H], router [E, H], gate_up [E, 2F, H] and down [E, H, F] are its weights, the last three bf16.
    """

    def __init__(self, T, H, F, E, k, P, norm, router, gate_up, down):
        f32, bf16, u8 = (dict(dtype=d, device="cuda") for d in (torch.float32, torch.bfloat16, torch.uint8))
        self.norm, self.router, self.gate_up, self.down = norm, router, gate_up, down
        self.path = moe.MoePath(1, T, H, E, k, P)
        rows = self.path.cap_recv
        self.h, self.normed, self.d_x, self.d_normed = (torch.empty((1, T, H), **bf16) for _ in range(4))
        self.pre, self.d_pre = (torch.empty((rows, 2 * F), **bf16) for _ in range(2))
        self.act = torch.empty((rows, F), **bf16)
        self.y, self.d_y, self.d_recv = (torch.empty((rows, H), **bf16) for _ in range(3))
        self.d_w, self.ones = torch.empty((1, T, k), **f32), torch.ones((1, T, k), **f32)
        self.d_logits = torch.empty((1, T, E), **f32)
        self.d_gate_up, self.d_down = torch.empty(gate_up.shape, **f32), torch.empty(down.shape, **f32)
        self.d_norm = torch.empty(norm.shape, **f32)
        self.ws = torch.empty(max(moe.moe_expert_product_workspace_bytes(rows, E, F, H, True),
                                  moe.moe_expert_product_workspace_bytes(rows, E, H, F),
                                  moe.moe_expert_product_backward_workspace_bytes(rows, E, 2 * F, H),
                                  moe.moe_expert_product_backward_workspace_bytes(rows, E, H, F),
                                  moe.moe_rms_norm_backward_workspace_bytes(T, H)), **u8)

    def forward(self, x, residual):
        p = self.path
        moe.moe_rms_norm(x, self.norm, y=self.normed, residual=residual, residual_out=self.h)
        p.dispatch_fused((self.normed @ self.router.t()).float(), self.normed)
        by = dict(expert_offsets=p.expert_offsets, dev_status=p.dev_status)
        moe.moe_expert_product(p.recv, self.gate_up, self.act, self.ws, gated=True, pre=self.pre, **by)
        moe.moe_expert_product(self.act, self.down, self.y, self.ws, **by)
        p.combine(self.y)
        return p.out, self.h

    def backward(self, d_out, d_h):
        """Gradients of x and residual (the same) and of norm, router, gate_up and down."""
        p = self.path
        by = dict(expert_offsets=p.expert_offsets, dev_status=p.dev_status)
        moe.moe_combine_backward(d_out, self.y, p.pair_row, p.topk_w, self.d_y, self.d_w,
                                 recv_pair=p.recv_pair, dev_status=p.dev_status)
        moe.moe_expert_product_backward(self.d_y, self.act, self.down, self.ws, d_a=self.d_pre,
                                        d_w=self.d_down, pre=self.pre, **by)
        moe.moe_expert_product_backward(self.d_pre, p.recv, self.gate_up, self.ws, d_a=self.d_recv,
                                        d_w=self.d_gate_up, **by)
        moe.moe_combine(self.d_recv, p.pair_row, self.ones, self.d_normed, p.dev_status)
        moe.moe_route_backward(None, p.topk_ids, p.topk_w, self.d_w, None, None, None, None,
                               self.d_logits, dev_status=p.dev_status)
        d_logits = self.d_logits[0].bfloat16()
        d_router = d_logits.t() @ self.normed[0]
        d_normed = self.d_normed + (d_logits @ self.router).unsqueeze(0)
        moe.moe_rms_norm_backward(d_normed, self.h, self.norm, self.d_x, self.ws, d_weight=self.d_norm,
                                  d_residual=d_h)
        return self.d_x, self.d_norm, d_router, self.d_gate_up, self.d_down


def relative(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def check_served(T=64, H=512, F=256, E=32, k=4, P=8, block_rows=64):
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate_up, down = randn(E, 2 * F, H) / math.sqrt(H), randn(E, H, F) / math.sqrt(F)
    logits, x = randn(1, T, E), randn(1, T, H).bfloat16()
    layer = ServedLayer(T, H, F, E, k, P, gate_up, down, block_rows)
    out = layer.step(logits, x)
    w1, w2 = dequantize(*quantize(gate_up)), dequantize(*quantize(down))
    top, ids = torch.topk(logits[0], k)
    both = torch.einsum("tkfh,th->tkf", w1[ids], x[0].float())
    h = torch.nn.functional.silu(both[..., :F]) * both[..., F:]
    y = torch.einsum("tkhf,tkf->tkh", w2[ids], h)
    want = (torch.softmax(top, -1).unsqueeze(-1) * y).sum(1)
    assert int(layer.path.dev_status.item()) == 0
    return relative(out[0], want)


def check_trained(S=2, T=96, H=256, E=16, k=3, P=4):
    g = torch.Generator(device="cuda").manual_seed(2)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    logits, x, d_out = randn(S, T, E), randn(S, T, H).bfloat16(), randn(S, T, H).bfloat16()
    scale = 0.5 + torch.rand(E, generator=g, device="cuda")
    mask = (torch.arange(T, device="cuda") < torch.tensor([[T], [T - 20]], device="cuda")[:S]).to(torch.uint8)
    d_out = d_out * mask.unsqueeze(-1).bfloat16()
    layer = TrainedLayer(S, T, H, E, k, P)
    out, losses = layer.forward(logits, x, scale, mask)
    d_x, d_logits = layer.backward(d_out, logits, scale, mask)
    # the same by automatic differentiation in 64 bits
    l64, x64 = logits.double().requires_grad_(), x.double().requires_grad_()
    top, ids = torch.topk(l64, k)
    want = ((torch.softmax(top, -1) * scale.double()[ids]).sum(-1, keepdim=True)) * x64
    m, n = mask.double(), mask.double().sum(1)
    prob = (torch.softmax(l64, -1) * m.unsqueeze(-1)).sum(1) / n[:, None]
    hot = (torch.nn.functional.one_hot(ids, E).sum(2) * m.unsqueeze(-1)).sum(1)
    balance = (E / (k * n) * (hot * prob).sum(-1)).mean()
    z = ((torch.logsumexp(l64, -1) ** 2 * m).sum(1) / n).mean()
    ((want * d_out.double()).sum() + 0.01 * balance + 0.001 * z).backward()
    assert int(layer.path.dev_status.item()) == 0
    return {"out": relative(out, want.detach()),
            "losses": relative(losses, torch.stack((balance, z)).detach()),
            "d_x": relative(d_x, x64.grad), "d_logits": relative(d_logits, l64.grad)}


def check_block(T=200, H=512, F=264, E=16, k=3, P=4):
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, residual, d_out, d_h = (randn(1, T, H).bfloat16() for _ in range(4))
    weights = [1 + 0.2 * randn(H)] + [(randn(*s) / math.sqrt(s[-1])).bfloat16()
                                      for s in ((E, H), (E, 2 * F, H), (E, H, F))]
    block = TrainedBlock(T, H, F, E, k, P, *weights)
    out, h = block.forward(x, residual)
    grads = block.backward(d_out, d_h)
    # the same by automatic differentiation in 64 bits, for the picks that were made
    ids = block.path.topk_ids[0].long()
    x64, r64, *w64 = (t.double().requires_grad_() for t in (x[0], residual[0], *weights))
    norm, router, gate_up, down = w64
    h64 = x64 + r64
    y64 = h64 / (h64.square().mean(-1, keepdim=True) + 1e-6).sqrt() * norm
    w = torch.softmax((y64 @ router.t()).gather(1, ids), -1)
    want = torch.zeros_like(y64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = (y64[t] @ gate_up[e].t()).chunk(2, -1)
        want = want.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ down[e].t()))
    ((want * d_out[0].double()).sum() + (h64 * d_h[0].double()).sum()).backward()
    assert int(block.path.dev_status.item()) == 0
    errors = {"out": relative(out[0], want.detach()), "h": relative(h[0], h64.detach()),
              "d_x": relative(grads[0][0], x64.grad)}
    errors.update({f"d_{name}": relative(got, leaf.grad) for name, got, leaf in
                   zip(("norm", "router", "gate_up", "down"), grads[1:], w64)})
    return errors


if __name__ == "__main__":
    moe.build()
    print(f"served: relative error of the output {check_served():.1e}")
    print("trained: relative errors " + ", ".join(f"{k} {v:.1e}" for k, v in check_trained().items()))
    print("block: relative errors " + ", ".join(f"{k} {v:.1e}" for k, v in check_block().items()))
