"""A gated feed-forward block, from training to serving:

  1. quantization-aware steps on fp32 latent weights: FakeQuantize, GLU, the
     down projection in torch, plain SGD;
  2. the trained weights packed;
  3. a prompt and then single tokens through glu and, with one adapter a
     request, lora_matmul.

    python examples/ffn_block.py [--rows 512 --model 1024 --hidden 3584 --steps 4]

Prints the loss of each step and how far the served block is from the trained
one (they share the codes; the trained one rounds code * scale to bf16).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ternary_weight_only_amd as tq  # noqa: E402


def train(x, target, latent, G, steps, rate):
    """SGD on the latent weights; the loss of each step."""
    losses = []
    for _ in range(steps):
        gate, up, down = (tq.FakeQuantize.apply(w, G).to(torch.bfloat16) for w in latent)
        y = tq.GLU.apply(x, gate, up).float() @ down.float().t()
        loss = ((y - target) ** 2).mean()
        loss.backward()
        with torch.no_grad():
            for w in latent:
                w -= rate * w.grad / w.grad.norm()
                w.grad = None
        losses.append(loss.item())
    return losses


def serve(x, packed, adapters, ids, G, status):
    """The block on packed weights, each row with its request's adapter."""
    gate, up, (down, scales) = packed
    M, K = x.shape
    a, b, scaling = adapters
    N, R = b.shape[1], a.shape[1]
    hidden = a.shape[2]
    h = tq.glu(x, gate, up, hidden, K, G, status=status)
    return tq.lora_matmul(h, down, scales, ids, a, b, scaling, N, hidden, G, status=status)


def run(rows=512, model=1024, hidden=3584, G=64, steps=4, requests=6, rank=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    x = normal(rows, model).to(torch.bfloat16)
    target = normal(rows, model)
    latent = [normal(hidden, model, std=model ** -0.5).requires_grad_(),
              normal(hidden, model, std=model ** -0.5).requires_grad_(),
              normal(model, hidden, std=hidden ** -0.5).requires_grad_()]
    losses = train(x, target, latent, G, steps, rate=2.0)

    status = tq.new_status(x.device)
    with torch.no_grad():
        packed = [tq.quantize_pack(w.to(torch.bfloat16), G, status=status) for w in latent]
        hats = [tq.dequantize(p, s, *w.shape, G, status=status) for (p, s), w in zip(packed, latent)]
        adapters = (normal(requests, rank, hidden, std=hidden ** -0.5).to(torch.bfloat16),
                    normal(requests, model, rank, std=0.1).to(torch.bfloat16),
                    torch.full((requests,), 0.5, device="cuda"))
        # runs of rows, one a request; the last rows have no adapter
        ids = torch.arange(rows, device="cuda", dtype=torch.int32) * (requests + 1) // rows
        ids = torch.where(ids == requests, -1, ids).to(torch.int32)
        prompt = serve(x, packed, adapters, ids, G, status)
        # a step of decoding: the last row of each request
        last = torch.stack([torch.nonzero(ids == r).max() for r in range(requests)])
        token = serve(x[last].contiguous(), packed, adapters, ids[last].contiguous(), G, status)

        # the same block on the weights as bf16, adapters in fp32
        h = tq.glu_forward(x, hats[0], hats[1])[0].float()
        y = h @ hats[2].float().t()
        a, b, scaling = adapters
        for r in range(requests):
            rows_r = ids == r
            y[rows_r] += scaling[r] * (h[rows_r] @ a[r].float().t()) @ b[r].float().t()
        error = ((prompt - y).norm() / y.norm()).item()
        apart = ((token - prompt[last]).norm() / prompt[last].norm()).item()
    if int(status.item()):
        raise RuntimeError("device status %d" % int(status.item()))
    return losses, error, apart


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--rows", type=int, default=512)
    p.add_argument("--model", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=3584)
    p.add_argument("--group", type=int, default=64, choices=(64, 128))
    p.add_argument("--steps", type=int, default=4)
    args = p.parse_args()
    losses, error, apart = run(args.rows, args.model, args.hidden, args.group, args.steps)
    print("loss:", " ".join("%.4f" % v for v in losses))
    print("packed block against bf16 weights: relative difference %.2e" % error)
    print("single tokens against the prompt's rows: relative difference %.2e" % apart)


if __name__ == "__main__":
    main()
