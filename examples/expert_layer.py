"""An expert layer on encoded weights, from the weights to its answers and gradients.

The experts' weights are encoded (IQ1_S, IQ2_XS or IQ1_M), decoded, and laid out
once as 8-bit integers with a scale per output channel.  A batch of tokens is
then routed to its experts and served in 8-bit integers:

    router -> expert_sort -> quantize_rows -> int8_expert_matmul -> expert_combine

and the same routing is run as a training step runs it, with the gradients of
the tokens, of the experts' answers and of the router's weights.  The served
answers are compared with those of the decoded weights in 64 bits.

    python examples/expert_layer.py --experts 16 --channels 1536 --depth 4096 --tokens 512
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ggml_iq_codebook_amd as iq  # noqa: E402
import workloads  # noqa: E402


def encoded_experts(experts, channels, depth, fmt):
    """Payload of the experts' weights and the grid it was encoded with."""
    grid = workloads.iq2xs_grid() if fmt == "iq2_xs" else workloads.iq1s_grid()
    grid = torch.from_numpy(grid).cuda()
    weight = torch.from_numpy(workloads.normal_weight((experts, channels, depth), 5)).cuda()
    importance = torch.from_numpy(workloads.lognormal_importance((experts, depth), 6)).cuda()
    return iq.encode(weight, grid, importance, fmt=fmt), grid


def int8_experts(payload, grid, fmt):
    """The decoded weights as 8-bit integers, expert by expert: (codes, scales)."""
    experts, channels, blocks, _ = payload.shape
    codes = torch.empty((experts, channels, blocks * 256), dtype=torch.int8, device="cuda")
    scales = torch.empty((experts, channels), dtype=torch.float32, device="cuda")
    for e in range(experts):
        codes[e], scales[e] = iq.quantize_rows(iq.dequant(payload[e], grid, fmt=fmt))
    return codes, scales


def serve(x, choice, weights, codes, scales, status):
    """The layer's answers; nothing here waits for the GPU."""
    order, position, offsets = iq.expert_sort(choice, codes.shape[0], status=status, check=False)
    q, q_scale = iq.quantize_rows(x, status=status, check=False)
    y = iq.int8_expert_matmul(q, q_scale, codes, scales, offsets, order, top_k=choice.shape[1],
                              dtype=x.dtype)
    return iq.expert_combine(y, position, offsets, weights)


def train_step(x, choice, weights, experts_forward, experts_backward, out_grad, experts):
    """Forward and backward of a layer whose experts are the caller's: (answers,
    gradient of x, gradient of the router's weights)."""
    order, position, offsets = iq.expert_sort(choice, experts)
    sorted_x = iq.expert_dispatch(x, position, offsets)
    y = experts_forward(sorted_x, offsets)
    out = iq.expert_combine(y, position, offsets, weights)
    y_grad, weights_grad = iq.expert_combine_backward(out_grad, y, position, offsets, weights)
    sorted_grad = experts_backward(y_grad, offsets)
    return out, iq.expert_dispatch_backward(sorted_grad, position, offsets), weights_grad


def reference(x, choice, weights, payload, grid, fmt):
    """The answers with the decoded weights in 64 bits."""
    out = torch.zeros((x.shape[0], payload.shape[1]), dtype=torch.float64, device="cuda")
    for e in range(payload.shape[0]):
        token, slot = torch.nonzero(choice == e, as_tuple=True)
        w = iq.dequant(payload[e], grid, fmt=fmt).double()
        out.index_add_(0, token, (x[token].double() @ w.T) * weights[token, slot, None].double())
    return out


def run(experts=16, channels=1536, depth=4096, tokens=512, top_k=2, fmt="iq1_s", repeats=20):
    """Returns the served answers' relative error, the largest of the training step's
    (answers, gradients of the tokens and of the router's weights) and the microseconds
    of a served call."""
    payload, grid = encoded_experts(experts, channels, depth, fmt)
    codes, scales = int8_experts(payload, grid, fmt)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, depth), generator=g, device="cuda").bfloat16()
    router = torch.randn((depth, experts), generator=g, device="cuda") / depth ** 0.5
    top, choice = torch.topk(x.float() @ router, top_k, dim=1)
    weights = torch.softmax(top, dim=1)

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = serve(x, choice, weights, codes, scales, status)
    want = reference(x, choice, weights, payload, grid, fmt)
    error = float((out.double() - want).norm() / want.norm())

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(repeats):
        serve(x, choice, weights, codes, scales, status)
    end.record()
    torch.cuda.synchronize()
    if int(status.item()):
        raise iq.IQError(int(status.item()), "serve")

    # A training step around experts that only scale their rows.
    def scaled(rows, offsets):
        return rows * 2.0

    out_grad = torch.randn((tokens, depth), generator=g, device="cuda").bfloat16()
    out, x_grad, weights_grad = train_step(x, choice, weights, scaled, scaled, out_grad, experts)
    total = weights.sum(dim=1, keepdim=True)
    dots = (out_grad.double() * x.double()).sum(dim=1, keepdim=True)
    train_error = max(float((got.double() - want).norm() / want.norm()) for got, want in (
        (out, 2.0 * total * x.double()), (x_grad, 2.0 * total * out_grad.double()),
        (weights_grad, 2.0 * dots.expand_as(weights))))
    return error, train_error, start.elapsed_time(end) / repeats * 1e3


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--channels", type=int, default=1536)
    p.add_argument("--depth", type=int, default=4096)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--top-k", type=int, default=2)
    p.add_argument("--fmt", choices=sorted(iq.FORMATS), default="iq1_s")
    a = p.parse_args()
    error, train_error, us = run(a.experts, a.channels, a.depth, a.tokens, a.top_k, a.fmt)
    print("%d tokens, %d of %d experts of %d x %d (%s): %.1f us a call, %.2f %% from 64 bits; "
          "training step %.2f %%" % (a.tokens, a.top_k, a.experts, a.channels, a.depth, a.fmt, us,
                                100 * error, 100 * train_error))


if __name__ == "__main__":
    main()
