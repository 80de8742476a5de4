"""A mixture-of-experts block between two norms, its tokens exchanged compressed: the operators together as they are used.

    pre_norm -> router -> route -> dispatch -> zipped all-to-all -> experts -> zipped all-to-all back -> combine -> post_norm

``MoEBlock`` holds experts_per_rank experts on each rank of a torch.distributed group and trains: the exchange's
gradient is the exchange the other way round, as compressed as the forward one.  The experts' products are library
matrix products.  Run it on one GPU (a group of one rank) with

    python examples/moe_block.py
"""
import os
import sys

import torch
import torch.distributed as dist

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lossless_bf16_exponent_zc_gb300 import torch_ops, zc  # noqa: E402,F401  (registers torch.ops.zc)
from lossless_bf16_exponent_zc_gb300.exchange import zipped_all_to_all  # noqa: E402

ops = torch.ops.zc


class ZippedExchange(torch.autograd.Function):
    """Rows sorted by destination rank to their ranks, compressed with the exact histogram's codebook of what is sent.
    Rows behind those (of slots that are not routed) stay here and get no gradient."""

    @staticmethod
    def forward(ctx, rows, send, recv, status, group=None):
        ctx.send, ctx.recv, ctx.status, ctx.group, ctx.rows = send, recv, status, group, rows.shape[0]
        return ZippedExchange.move(rows, send, recv, status, group)

    @staticmethod
    def backward(ctx, drows):
        back = ZippedExchange.move(drows.contiguous(), ctx.recv, ctx.send, ctx.status, ctx.group)
        kept = back.new_zeros((ctx.rows - back.shape[0], back.shape[1]))
        return torch.cat([back, kept]) if len(kept) else back, None, None, None, None

    @staticmethod
    def move(rows, send, recv, status, group=None):
        hidden = rows.shape[1]
        bits = rows[:sum(send)].reshape(-1).view(torch.int16)
        cb, _ = zc.histogram_topk(bits, zc.workspace(bits.numel(), rows.device), status)
        pieces = zipped_all_to_all(list(bits.split([n * hidden for n in send])), [n * hidden for n in recv], cb, status,
                                   group=group)
        return torch.cat(pieces).view(torch.bfloat16).view(-1, hidden)


class MoEBlock(torch.nn.Module):
    """x, h -> x_new, h_next: h is x normed for this block, h_next x_new normed for the next one."""

    def __init__(self, hidden, inner, experts_per_rank, k, residual_scale=1.0, group=None, device="cuda"):
        super().__init__()
        self.group, self.world, self.k = group, dist.get_world_size(group), k
        self.experts = experts_per_rank * self.world
        self.residual_scale, self.eps = residual_scale, 1e-6
        kw = dict(device=device, dtype=torch.bfloat16)

        def weight(*shape):
            return torch.nn.Parameter(torch.randn(shape, **kw) * shape[-2] ** -0.5)

        self.router = torch.nn.Parameter(torch.randn((hidden, self.experts), **kw) * hidden ** -0.5)
        self.up, self.down = weight(experts_per_rank, hidden, inner), weight(experts_per_rank, inner, hidden)
        self.norm_weight = torch.nn.Parameter(torch.ones(hidden, **kw))
        self.next_weight = torch.nn.Parameter(torch.ones(hidden, **kw))
        self.gate = torch.nn.Parameter(torch.full((1, hidden), 0.5, **kw))
        self.register_buffer("bias", torch.zeros(self.experts, device=device))  # balances the load, fp32
        self.status = zc.new_status(device)

    def counts(self, offsets):
        """Rows for every expert from every rank: [world][experts] on the host (the one wait for the device)."""
        mine = offsets.diff()
        every = [torch.empty_like(mine) for _ in range(self.world)]
        if self.world > 1:
            dist.all_gather(every, mine, group=self.group)
        else:
            every = [mine]
        return torch.stack(every).tolist()

    def run_experts(self, rows, counts):
        """The rows of each rank lie one after another, each rank's sorted by expert."""
        outs, at = [], 0
        for of_rank in counts:
            for e, n in enumerate(of_rank):
                outs.append(torch.nn.functional.silu(rows[at:at + n] @ self.up[e]) @ self.down[e])
                at += n
        return torch.cat(outs)

    def forward(self, x, h):
        weights, experts = ops.moe_route(h @ self.router, self.bias, self.k, "sigmoid", True, 1.0)
        rows, positions, _, offsets = ops.moe_dispatch(h, experts, self.experts)
        counts = self.counts(offsets)
        per, rank = self.experts // self.world, dist.get_rank(self.group)
        send = [sum(counts[rank][r * per:(r + 1) * per]) for r in range(self.world)]
        here = [c[rank * per:(rank + 1) * per] for c in counts]
        recv = [sum(c) for c in here]
        got = ZippedExchange.apply(rows, send, recv, self.status, self.group)
        back = ZippedExchange.apply(self.run_experts(got, here), recv, send, self.status, self.group)
        y, combined = ops.moe_combine(back, weights, positions)
        torch.maximum(self.status, combined, out=self.status)
        return ops.post_pre_norm(y, x, self.norm_weight, self.gate, self.next_weight, self.residual_scale, self.eps)


def main():
    if not dist.is_initialized():
        dist.init_process_group("gloo", init_method="tcp://127.0.0.1:29571", rank=0, world_size=1)
    torch.manual_seed(0)
    block = MoEBlock(hidden=512, inner=1024, experts_per_rank=8, k=2, residual_scale=0.9)
    first = torch.nn.Parameter(torch.ones(512, device="cuda", dtype=torch.bfloat16))
    opt = torch.optim.SGD([first, *block.parameters()], lr=0.5)
    x = torch.randn(1024, 512, device="cuda").to(torch.bfloat16)
    target = torch.randn(1024, 512, device="cuda")
    losses = []
    for _ in range(5):  # training
        opt.zero_grad()
        x_new, _ = block(x, ops.pre_norm(x, first, 1e-6))
        loss = (x_new.float() - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    with torch.no_grad():  # a decoding step of four tokens
        x_new, h = block(x[:4], ops.pre_norm(x[:4], first, 1e-6))
    assert zc.status_value(block.status) == 0, zc.status_string(zc.status_value(block.status))
    print("loss", " ".join(f"{v:.4f}" for v in losses), "| decoded", tuple(h.shape))
    return losses


if __name__ == "__main__":
    main()
