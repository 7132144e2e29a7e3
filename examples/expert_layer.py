"""A layer of a language model with per-request adapters and experts, served and trained on the
library's grouped products.

    python examples/expert_layer.py [tokens]

Serving: every row goes through a shared projection with the low-rank adapter of its request, a
router sends it to its experts, and a gated expert layer answers.  Training: one expert product with
its weighted sum, a squared error, the gradients of the product, of the weighted sum and of the
router's logits, and a step of plain gradient descent that lowers the error.  At the end the routing
is used as the sparse matrix that it is: the library's SpGEMM counts how often two experts
serve the same token.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_gemm_irregular_gb300 as sg  # noqa: E402


def make(tokens, dim=1024, hidden=512, experts=16, adapters=5, rank=16, seed=0, device="cuda"):
    """Weights and a batch; the last row is padding (its logits are -inf), some rows have no adapter."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, fan_in):
        return (torch.randn(*shape, device=device, generator=g) * fan_in ** -0.5).bfloat16()

    m = dict(w_in=normal(dim, dim, fan_in=dim), a=normal(adapters, rank, dim, fan_in=dim),
             b=normal(adapters, dim, rank, fan_in=rank), scale=torch.ones(adapters, device=device),
             w_router=normal(experts, dim, fan_in=dim), bias=torch.zeros(experts, device=device),
             w_up=normal(experts, 2 * hidden, dim, fan_in=dim), w_down=normal(experts, dim, hidden, fan_in=hidden),
             w_train=normal(experts, dim, dim, fan_in=dim))
    x = normal(tokens, dim, fan_in=1)
    ids = torch.randint(-1, adapters, (tokens,), device=device, generator=g).int()
    return m, x, ids


def logits_of(m, h):
    l = torch.matmul(h, m["w_router"].t()).float()
    l[-1] = float("-inf")
    return l


def serve(m, x, ids, top_k=4):
    """(output, routing) of the layer."""
    h = sg.adapted_product(x, m["w_in"], m["a"], m["b"], ids, m["scale"])
    r = sg.route(logits_of(m, h), top_k, bias=m["bias"], score="sigmoid", groups=4, groups_kept=2, group_score="top2")
    return h + sg.experts(h, m["w_up"], m["w_down"], r), r


def train_step(m, h, target, top_k=2, rate=0.05):
    """One step on w_train and the router; returns the mean squared error before it."""
    l = logits_of(m, h)
    r = sg.route(l, top_k)
    y = sg.expert_product(h, m["w_train"], r)
    out = sg.combine(y, r)
    error = out.float() - target.float()
    dout = (2.0 / h.shape[0] * error).bfloat16()
    dy, dweights = sg.combine_backward(dout, y, r)
    _, dw = sg.expert_product_backward(dy, h, m["w_train"], r, need_dx=False)
    dlogits = sg.route_backward(l, r, dweights)
    m["w_train"] = (m["w_train"].float() - rate * dw.float()).bfloat16()
    m["w_router"] = (m["w_router"].float() - rate * torch.matmul(dlogits.t(), h.float())).bfloat16()
    return float(error.square().mean())


def together(r):
    """experts x experts: the number of tokens that two experts serve together."""
    ones = sg.group_rows(r.ids, r.groups)  # the same choice with weights of one
    row_ptr, col, val = sg.multiply(ones.transposed_csr(), ones.to_csr()).to_host()
    out = torch.zeros(r.groups, r.groups)
    for e in range(r.groups):
        out[e, torch.from_numpy(col[row_ptr[e]:row_ptr[e + 1]]).long()] = torch.from_numpy(
            val[row_ptr[e]:row_ptr[e + 1]]).float()
    return out


def main(tokens=2048):
    m, x, ids = make(tokens)
    out, r = serve(m, x, ids)
    count = (r.offsets[1:] - r.offsets[:-1]).cpu()
    print("served %d rows of %d; rows per expert %d to %d" % (out.shape[0], out.shape[1], count.min(), count.max()))
    target = torch.matmul(x, m["w_in"].t())
    errors = [train_step(m, x, target) for _ in range(8)]
    print("training error %.4f -> %.4f" % (errors[0], errors[-1]))
    pairs = together(r)
    pairs.fill_diagonal_(0)
    print("experts serving together most often: %s (%d tokens)" % (divmod(int(pairs.argmax()), r.groups), pairs.max()))
    sg.grouped_status()
    return out, errors, pairs


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 2048)
