#!/usr/bin/env python3
"""A training step of a small layer with experts, its device-wide steps by counted_notify_sync_gb300:

    python examples/expert_training_step.py [--steps N] [--block]

routing with a load-balancing bias (run_route), the tokens' rows sorted by expert (run_dispatch), each expert's product
on its rows, these back to their tokens with the routing's weights (run_combine), all their gradients inside torch's
autograd, and clipping all gradients by their global norm before the optimiser reads them (run_grad_clip).  With --block
the layer stands between a root-mean-square norm (run_rms_norm) and the residual that it is added to.  Needs a GB300.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import counted_notify_sync_gb300 as cns  # noqa: E402


class RoutedGradient(torch.autograd.Function):
    """The logits' gradient from the weights'.  It has no derivative of its own, and says so."""

    @staticmethod
    def forward(ctx, logits, dweights, ids, route):
        return cns.run_route_backward(route, logits, dweights.contiguous(), ids=ids, stream=torch.cuda.current_stream())

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the routing is differentiable once")


class Routed(torch.autograd.Function):
    """Weights of the chosen experts; `route` holds the ids and the plan afterwards."""

    @staticmethod
    def forward(ctx, logits, bias, route):
        stream = torch.cuda.current_stream()
        cns.run_route(route, logits, bias=bias, stream=stream)
        ctx.route = route
        ids = route.ids[:logits.shape[0]].clone()
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return route.weights[:logits.shape[0]].clone(), ids

    @staticmethod
    def backward(ctx, dweights, _):
        logits, ids = ctx.saved_tensors
        return RoutedGradient.apply(logits, dweights, ids, ctx.route), None, None


def once(name, gradient):
    """An autograd function that takes a gradient from all that it depends on.  It has no derivative of its own, and
    says so."""

    def forward(ctx, *args):
        return gradient(*args)

    def backward(ctx, *_):
        raise RuntimeError(f"{name} is differentiable once")

    return type(name + "Gradient", (torch.autograd.Function,), {"forward": staticmethod(forward),
                                                                "backward": staticmethod(backward)})


DispatchedGradient = once("Dispatched", lambda drows, places, route: cns.run_dispatch_backward(
    route, drows.contiguous(), places=places, stream=torch.cuda.current_stream()))
CombinedGradient = once("Combined", lambda dy, rows, weights, places, route: cns.run_combine_backward(
    route, rows, dy.contiguous(), weights=weights, places=places, stream=torch.cuda.current_stream()))
NormedGradient = once("Normed", lambda dh, dy, h, gain, norm: cns.run_rms_norm_backward(
    norm, h, gain, dy.contiguous(), dh=dh.contiguous(), stream=torch.cuda.current_stream()))


class Dispatched(torch.autograd.Function):
    """The tokens' rows in their experts' order."""

    @staticmethod
    def forward(ctx, x, places, route):
        ctx.route = route
        ctx.save_for_backward(places)
        return cns.run_dispatch(route, x, places=places, stream=torch.cuda.current_stream())

    @staticmethod
    def backward(ctx, drows):
        return DispatchedGradient.apply(drows, *ctx.saved_tensors, ctx.route), None, None


class Combined(torch.autograd.Function):
    """The rows back to their tokens, weighted, and added to a base (or None)."""

    @staticmethod
    def forward(ctx, rows, weights, base, places, route):
        ctx.route, ctx.base = route, base is not None
        ctx.save_for_backward(rows, weights, places)
        return cns.run_combine(route, rows, weights=weights, places=places, base=base, stream=torch.cuda.current_stream())

    @staticmethod
    def backward(ctx, dy):
        drows, dweights = CombinedGradient.apply(dy, *ctx.saved_tensors, ctx.route)
        return drows, dweights, dy if ctx.base else None, None, None


class Normed(torch.autograd.Function):
    """(h, y): h = x + residual, and h normalised."""

    @staticmethod
    def forward(ctx, x, residual, gain, norm):
        h, y, _, _ = cns.run_rms_norm(norm, x, gain, residual=residual, stream=torch.cuda.current_stream())
        ctx.norm = norm
        ctx.save_for_backward(h, gain)
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        dx, dgain = NormedGradient.apply(dh, dy, *ctx.saved_tensors, ctx.norm)
        return dx, dx, dgain.to(ctx.saved_tensors[1].dtype), None


class Experts(torch.nn.Module):
    def __init__(self, tokens, width, hidden, experts, top_k, groups=4, top_groups=2):
        super().__init__()
        self.router = torch.nn.Parameter(torch.randn(width, experts, device="cuda") * width ** -0.5)
        self.up = torch.nn.Parameter(torch.randn(experts, width, hidden, device="cuda") * width ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(experts, hidden, width, device="cuda") * hidden ** -0.5)
        self.register_buffer("bias", torch.zeros(experts, device="cuda"))
        self.route = cns.new_route(tokens, experts, top_k, score=cns.CNS_SCORE_SIGMOID, groups=groups,
                                   top_groups=top_groups, group_top=2)

    def forward(self, x, base=None):
        weights, _ = Routed.apply(x @ self.router, self.bias, self.route)
        places = self.route.places[:x.shape[0]].clone()
        # each expert's product on its own rows, which lie in a row
        starts = self.route.offsets.tolist()
        rows = Dispatched.apply(x, places, self.route)[:starts[-1]].split([b - a for a, b in zip(starts, starts[1:])])
        out = torch.cat([torch.relu(r @ self.up[e]) @ self.down[e] for e, r in enumerate(rows)])
        return Combined.apply(out, weights, base, places, self.route)

    def balance(self, rate=1e-3):
        """Move the bias against the load: experts with more than their share become less likely to be chosen."""
        load = self.route.offsets.diff().float()
        self.bias += rate * torch.sign(load.mean() - load)


class Block(torch.nn.Module):
    """x + residual, and the experts of its norm added to that."""

    def __init__(self, tokens, width, hidden, experts, top_k, **kw):
        super().__init__()
        self.gain = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.norm = cns.new_rms_norm(width)
        self.experts = Experts(tokens, width, hidden, experts, top_k, **kw)
        self.balance = self.experts.balance

    def forward(self, x, residual=None):
        h, y = Normed.apply(x, torch.zeros_like(x) if residual is None else residual, self.gain, self.norm)
        return self.experts(y, base=h)


def train(steps=30, tokens=512, width=64, hidden=128, experts=16, top_k=2, seed=0, max_norm=0.05, rate=1.0, kind=Experts):
    """Fit a fixed random map; returns the losses, and the gradient norm before and after clipping of each step."""
    torch.manual_seed(seed)
    layer = kind(tokens, width, hidden, experts, top_k)
    target = torch.randn(width, width, device="cuda") * width ** -0.5
    params = list(layer.parameters())
    for p in params:
        p.grad = torch.zeros_like(p)
    clip = cns.new_grad_clip([p.grad for p in params], max_norm)   # in place; the gradients stay where they are
    losses, norms = [], []
    for _ in range(steps):
        x = torch.randn(tokens, width, device="cuda")
        torch._foreach_zero_([p.grad for p in params])
        loss = (layer(x) - torch.tanh(x @ target)).square().mean()
        loss.backward()
        before = cns.run_grad_clip(clip, stream=torch.cuda.current_stream()).clone()
        after = cns.run_grad_norm(clip, stream=torch.cuda.current_stream()).clone()
        with torch.no_grad():
            for p in params:
                p -= rate * p.grad
            layer.balance()
        losses.append(loss.detach())
        norms.append((before, after))
    return [float(v) for v in losses], [(float(a), float(b)) for a, b in norms]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--block", action="store_true")
    a = ap.parse_args()
    losses, norms = train(a.steps, kind=Block if a.block else Experts)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}  gradient norm {norms[i][0]:.3f} -> {norms[i][1]:.3f}")
    print(f"last       loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
