"""Trains a vocabulary-parallel head with the library's losses, on one GPU.

    python examples/train_head.py [--ranks 4] [--steps 40]

A head W [V, D], split by rows over the ranks, learns from hidden states X that
hide their word: first from labels (fcc_linear_xent and its gradient), then a
second head from the first one's top logits (fcc_linear_distill and its
gradient).  No step ever holds the T x V logits.  The gradients of X, which a
model would send on to its last layer, are computed too.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--words", type=int, default=8000)
    ap.add_argument("--hidden", type=int, default=256)
    a = ap.parse_args()
    import gemm_collective_gb300 as fcc

    R, T, V, D, K = a.ranks, a.tokens, a.words // a.ranks * a.ranks, a.hidden, 32
    gen = torch.Generator(device="cuda").manual_seed(0)
    words = torch.randn(V, D, device="cuda", generator=gen)
    word = torch.randint(0, V, (T,), device="cuda", generator=gen)
    X = (words[word] + 0.5 * torch.randn(T, D, device="cuda", generator=gen)).bfloat16()
    labels = word.to(torch.int32)
    labels[: T // 8] = -100  # a prompt's tokens: no loss
    live = (labels >= 0).sum()
    dloss = torch.full((T,), 1.0, device="cuda") / live  # the mean over the live tokens

    def head():
        return [torch.zeros(V // R, D, device="cuda") for _ in range(R)]

    def copies(dtype, *shape):
        return [torch.empty(*shape, device="cuda", dtype=dtype) for _ in range(R)]

    Xs = [X] * R  # (every rank's copy)
    loss, lse = copies(torch.float32, T), copies(torch.float32, T)
    dX, dW = copies(torch.bfloat16, T, D), copies(torch.bfloat16, V // R, D)

    def train(name, master, forward, backward, rate):
        """Plain gradient descent on f32 master weights; the first and last mean loss."""
        seen = []
        for _ in range(a.steps):
            W = [w.bfloat16() for w in master]
            forward(W)
            seen.append(loss[0].sum() / live)
            backward(W)
            for w, g in zip(master, dW):
                w -= rate * g.float()
        if (status := fcc.fcc_stream_status()) != fcc.FCC_OK:
            raise RuntimeError(fcc.fcc_status_string(status))
        first, last = float(seen[0]), float(seen[-1])
        print(f"{name}: mean loss {first:.4f} -> {last:.4f} in {a.steps} steps, "
              f"|dX| {float(dX[0].float().norm()):.3e}")
        if not last < 0.8 * first:
            raise SystemExit(f"{name}: the loss did not fall")

    teacher = head()
    train("cross entropy", teacher,
          lambda W: fcc.fcc_linear_xent(R, Xs, W, labels, T, V, D, loss, lse, smoothing=0.01),
          lambda W: fcc.fcc_linear_xent_grad(R, Xs, W, labels, lse, dloss, T, V, D, dX, dW,
                                             smoothing=0.01), rate=20.0)
    top = torch.topk(X.float() @ torch.cat(teacher).T, K, dim=1)
    idx = torch.where(labels[:, None] < 0, -1, top.indices).to(torch.int32)
    logits = top.values.contiguous()
    train("distillation", head(),
          lambda W: fcc.fcc_linear_distill(R, Xs, W, idx, logits, T, V, D, K, loss, lse,
                                           temperature=2.0),
          lambda W: fcc.fcc_linear_distill_grad(R, Xs, W, idx, logits, lse, dloss, T, V, D, K, dX,
                                                dW, temperature=2.0), rate=20.0)


if __name__ == "__main__":
    main()
