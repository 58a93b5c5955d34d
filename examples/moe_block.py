"""A mixture-of-experts block on the package's kernels: layer norm, router,
FP8 experts, residual.  Trains it on a fixed random map for a few steps, then
runs it one token at a time.

    python examples/moe_block.py [--tokens 2048 --width 2048 --hidden 1408 --experts 64 --k 6 --steps 5]

Every step of the block but the router's matrix product (tokens x experts, in
torch) is a call of the library, forward and backward.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_matmul_amd as fp8mm  # noqa: E402


class MoEBlock(torch.nn.Module):
    """y = x + experts(norm(x)), tokens routed by sigmoid scores with a balance
    bias over groups of experts, weights renormalised."""

    def __init__(self, width, hidden, experts, k, groups=1, group_topk=None, device="cuda"):
        super().__init__()
        self.k, self.groups, self.group_topk = k, groups, group_topk
        kw = dict(device=device, dtype=torch.bfloat16)
        self.gamma = torch.nn.Parameter(torch.ones(width, **kw))
        self.beta = torch.nn.Parameter(torch.zeros(width, **kw))
        self.router = torch.nn.Parameter(torch.randn((width, experts), **kw) * width ** -0.5)
        self.w_in = torch.nn.Parameter(torch.randn((experts, 2 * hidden, width), **kw) * width ** -0.5)
        self.w_out = torch.nn.Parameter(torch.randn((experts, width, hidden), **kw) * hidden ** -0.5)
        self.register_buffer("balance", torch.zeros(experts, device=device))

    def forward(self, x):
        n = fp8mm.layer_norm(x, self.gamma, self.beta)
        ids, weights = fp8mm.moe_route(n @ self.router, self.k, "sigmoid", self.balance, self.groups, self.group_topk,
                                       "top2" if self.groups > 1 else "max")
        if self.training:
            self._rebalance(ids)
        return x + fp8mm.fp8_moe(n, self.w_in, self.w_out, ids, weights)

    @torch.no_grad()
    def _rebalance(self, ids, rate=1e-3):
        """Raise the bias of experts with fewer tokens than their share, lower the others'."""
        offsets, _ = fp8mm.moe_plan(ids, self.balance.numel())
        load = torch.diff(offsets, prepend=offsets.new_zeros(1)).float()
        self.balance += rate * torch.sign(load.mean() - load)


def main(tokens=2048, width=2048, hidden=1408, experts=64, k=6, steps=5, lr=0.05, decode=8, seed=0, say=print):
    """Returns the losses of the steps."""
    torch.manual_seed(seed)
    groups = 4 if experts % 4 == 0 and experts // 2 >= k else 1
    block = MoEBlock(width, hidden, experts, k, groups, 2 if groups > 1 else None)
    x = torch.randn((tokens, width), device="cuda").bfloat16()
    target = (x.float() + torch.randn((tokens, width), device="cuda")).bfloat16()
    optimizer = torch.optim.SGD(block.parameters(), lr=lr * tokens, momentum=0.0)
    losses = []
    for step in range(steps):
        torch.cuda.synchronize()
        began = time.perf_counter()
        optimizer.zero_grad(set_to_none=True)
        loss = torch.nn.functional.mse_loss(block(x).float(), target.float())
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
        torch.cuda.synchronize()
        say(f"step {step}: loss {losses[-1]:.4f}, {(time.perf_counter() - began) * 1e3:.2f} ms", flush=True)
    block.eval()
    with torch.no_grad():
        whole = block(x[:decode])
        single = torch.cat([block(x[t:t + 1]) for t in range(decode)])
    # tokens do not see each other: one at a time gives what all at once give
    say(f"one token at a time: largest difference {float((whole - single).abs().max()):.3g}", flush=True)
    return losses, whole, single


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 2048), ("hidden", 1408), ("experts", 64), ("k", 6), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
