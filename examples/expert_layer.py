"""Trains one sparse expert layer on synthetic data, then serves single tokens.

    python examples/expert_layer.py [--steps N] [--tokens T] [--experts E] [--width D] [--hidden F]

Every step: logits, routing, the experts' products, a squared error against a
random target map, all gradients, clipping by their global norm, and plain
gradient descent on fp32 copies of the parameters.  The bias of the router is
moved after every step towards experts with fewer tokens.  At the end the
routing matrix R is taken as CSR and R^T R, the number of tokens that two
experts share, is made by the library's sparse product.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spgemm_symbolic_row_amd as sg


def train(steps=30, tokens=4096, experts=16, width=256, hidden=128, k=2, lr=0.5, seed=0):
    """Losses of all steps, the last routing, the tokens of every expert, and the parameters."""
    dev, bf = "cuda", torch.bfloat16
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev) * scale

    target = randn(width, width, scale=width ** -0.5)
    main = {"router": randn(experts, width, scale=width ** -0.5),
            "w_in": randn(experts, 2 * hidden, width, scale=width ** -0.5),
            "w_out": randn(experts, width, hidden, scale=hidden ** -0.5)}
    bias = torch.zeros(experts, device=dev)
    losses = []
    for _ in range(steps):
        x = randn(tokens, width).to(bf)
        want = torch.tanh(x.float() @ target.t())
        w_in, w_out = main["w_in"].to(bf), main["w_out"].to(bf)

        logits = x.float() @ main["router"].t()
        r = sg.route(logits, k, scores="sigmoid", bias=bias)
        y, kept = sg.experts(x, w_in, w_out, r.col, r.val, keep=True)

        err = y.float() - want
        losses.append(err.square().mean())
        dy = (err * (2.0 / tokens)).to(bf)

        _, dw_in, dw_out, dval = sg.experts_backward(dy, kept)
        dlogits = sg.route_backward(logits, r, dval)
        grads = {"router": dlogits.t() @ x.float(), "w_in": dw_in, "w_out": dw_out}
        clipped = {n: torch.empty_like(main[n]) for n in main}
        sg.clip_grad_norm(grads.values(), 1.0, out=clipped.values())
        for n in main:
            main[n] -= lr * clipped[n]

        row_ptr, _ = sg.dispatch(r.col, experts)
        load = row_ptr.diff().float()
        bias += 0.01 * torch.sign(load.mean() - load)
    return [float(v) for v in losses], r, load, main


def shared_tokens(r):
    """R^T R of a routing: entry (a, b) counts the tokens that went to a and to b."""
    R = r.csr()
    R.val = torch.ones_like(R.val)
    return sg.matmul(sg.transpose(R), R)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 30), ("tokens", 4096), ("experts", 16), ("width", 256), ("hidden", 128)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    losses, r, load, params = train(a.steps, a.tokens, a.experts, a.width, a.hidden)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i}: loss {losses[i]:.4f}")
    print(f"last loss {losses[-1]:.4f}; tokens per expert {[int(v) for v in load]}")
    row_ptr, col, val = shared_tokens(r)
    print(f"pairs of experts that share tokens: {int(row_ptr[-1])} of {a.experts ** 2}")

    # Single tokens: the same layer, without what training keeps.
    w_in, w_out = params["w_in"].bfloat16(), params["w_out"].bfloat16()
    x = torch.randn(1, a.width, device="cuda").bfloat16()
    for _ in range(3):
        t = sg.route(x.float() @ params["router"].t(), 2, scores="sigmoid")
        x = sg.experts(x, w_in, w_out, t.col, t.val)
        print("token to experts", t.col[0].tolist())


if __name__ == "__main__":
    main()
