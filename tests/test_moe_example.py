"""The example block's exchange: its gradient has a row for every row that went in, sent or not, and it runs over the
block's group.  On CPU the exchange itself is a stand-in; on the GPU the whole block runs with closed experts."""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def example(monkeypatch):
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    import moe_block
    return moe_block


@pytest.mark.parametrize("sent", [0, 3, 5])
def test_gradient_of_rows_that_are_not_sent(example, monkeypatch, sent):
    """Unrouted rows stand behind the others and stay here: zeros for them, the exchanged gradient for the rest."""
    monkeypatch.setattr(example.ZippedExchange, "move",
                        staticmethod(lambda rows, send, recv, status, *group: 2 * rows[:sum(send)]))
    rows = torch.randn((5, 4), requires_grad=True)
    out = example.ZippedExchange.apply(rows, [sent], [sent], None)
    assert torch.equal(out, 2 * rows[:sent])
    g = torch.randn((sent, 4))
    out.backward(g)
    assert torch.equal(rows.grad[:sent], 2 * g) and not rows.grad[sent:].any()


def test_the_group_is_that_of_the_block(example, monkeypatch):
    """Both directions exchange over the group whose ranks the counts are of, not over all ranks."""
    groups = []

    def exchange(chunks, recv_counts, cb, status, ws=None, group=None):
        groups.append(group)
        return list(chunks)

    monkeypatch.setattr(example, "zipped_all_to_all", exchange)
    monkeypatch.setattr(example.zc, "workspace", lambda *a: None)
    monkeypatch.setattr(example.zc, "histogram_topk", lambda *a: (None, None))
    rows, group = torch.randn((5, 4)).bfloat16().requires_grad_(True), object()
    example.ZippedExchange.apply(rows, [2, 3], [2, 3], None, group).sum().backward()
    assert groups == [group, group] and torch.equal(rows.grad, torch.ones_like(rows))


@pytest.mark.gpu
def test_block_of_a_group_of_its_own(zc, example):
    """The whole block over a group that is not the default one (one rank here)."""
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method="tcp://127.0.0.1:29574", rank=0, world_size=1)
    try:
        outs = []
        for group in (None, dist.new_group([0])):
            torch.manual_seed(4)
            block = example.MoEBlock(hidden=64, inner=64, experts_per_rank=4, k=2, group=group)
            outs.append(block(*torch.randn((2, 30, 64), device="cuda").bfloat16()))
        for a, b in zip(*outs):
            assert torch.equal(a, b)
    finally:
        dist.destroy_process_group()


@pytest.mark.gpu
@pytest.mark.parametrize("open_experts", [0, 1, 3])
def test_block_with_closed_experts(zc, example, open_experts):
    """Fewer open experts than slots: what is not routed adds nothing, and training still gets every gradient."""
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method="tcp://127.0.0.1:29573", rank=0, world_size=1)
    try:
        torch.manual_seed(3)
        block = example.MoEBlock(hidden=64, inner=64, experts_per_rank=6, k=2)
        block.bias[open_experts:] = -math.inf
        x = torch.randn((50, 64), device="cuda").bfloat16().requires_grad_(True)
        h = torch.randn((50, 64), device="cuda").bfloat16().requires_grad_(True)
        x_new, h_next = block(x, h)
        (x_new.float().square().sum() + h_next.float().sum()).backward()
        assert zc.status_value(block.status) == 0
        for name, p in [("x", x), ("h", h), *block.named_parameters()]:
            assert p.grad is not None and torch.isfinite(p.grad).all(), name
        assert not block.up.grad[open_experts:].any()
        if open_experts == 0:  # no expert's output: the block passes x on
            assert torch.equal(x_new, x) and not h.grad.any()
        else:
            assert block.up.grad[:open_experts].any() and h.grad.any()
    finally:
        dist.destroy_process_group()
