"""A training step of one parameter group on one GPU, from token ids to updated parameters.

    python examples/training_step.py [--steps 30]

The group is an embedding table and a layer norm.  C contributors (their buffers on this GPU stand for
data-parallel ranks) each look their tokens up, normalise them and make bf16 gradients, straight into
the per-parameter tensors that the reduce-scatter reads in place.  The reduce-scatter leaves R fp32
shards; they are clipped by their global norm, the fp32 master shards take a step of gradient descent,
and the all-gather placement puts the new bf16 parameters back.  The loss is the squared distance of the
normalised vectors from a fixed vector for each token, so that it can be seen to fall.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from all_gather_placement_amd import (Layout, clip_grad_norm, embedding, embedding_bwd, layer_norm, layer_norm_bwd)


def train(steps=30, vocab=1000, dim=264, tokens=2000, contributors=4, ranks=4, lr=0.5, max_norm=1.0, report=print):
    """Runs the steps; returns the loss and the gradient norm before clipping of each."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(0)

    def normal(*shape):
        return torch.empty(shape, device=dev).normal_(generator=gen)

    scale = dim ** 0.5
    params = [(normal(vocab, dim) / scale).bfloat16(), torch.ones(dim, device=dev, dtype=torch.bfloat16),
              torch.zeros(dim, device=dev, dtype=torch.bfloat16)]
    table, weight, bias = params
    goal = normal(vocab, dim)
    grads = [[torch.empty_like(p) for p in params] for _ in range(contributors)]
    losses, norms = [], []
    with Layout([tuple(p.shape) for p in params], ranks) as layout:
        stage = torch.empty(ranks * layout.S, device=dev, dtype=torch.bfloat16)
        layout.slot_pack(params, stage)
        master = stage.float()  # rank-major, as the shards
        flat = torch.empty(ranks * layout.S, device=dev)
        shards = list(flat.split(layout.S))
        reduce = layout.bind_rs(grads, shards)
        place = layout.bind_ag(stage, params)
        try:
            for step in range(steps):
                loss = torch.zeros((), device=dev)
                for c in range(contributors):
                    ids = torch.randint(0, vocab, (tokens,), device=dev, generator=gen)
                    ids[::50] = -1  # padded positions
                    h = embedding(ids, table, scale)
                    y, mean, rstd = layer_norm(h, weight, bias)
                    off = torch.where((ids >= 0)[:, None], y.float() - goal[ids], 0.0)
                    loss += off.square().sum() / (2 * contributors * tokens)
                    dy = (off / (contributors * tokens)).bfloat16()
                    dtable, dweight, dbias = grads[c]
                    layer_norm_bwd(dy, h, weight, mean, rstd, dx=dy, dweight=dweight, dbias=dbias)
                    embedding_bwd(ids, dy, vocab, scale, out=dtable)
                reduce.launch()
                norm = clip_grad_norm(shards, max_norm)
                master.add_(flat, alpha=-lr)
                stage.copy_(master)
                place.launch()
                losses.append(loss)
                norms.append(norm)
        finally:
            torch.cuda.synchronize()
            reduce.close()
            place.close()
    losses, norms = [float(x) for x in losses], [float(x) for x in norms]
    for step in range(0, steps, max(1, steps // 10)):
        report(f"step {step:4d}  loss {losses[step]:9.4f}  gradient norm {norms[step]:.4f}")
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    args = ap.parse_args()
    losses, _ = train(args.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
