"""A pre-norm residual MLP block of sparse layers trained with its activations kept in 8 bits.

    h' = h + down(gelu(up(rmsnorm(h) * gain)))

Between the forward and the backward pass the block keeps h in bf16 (the residual stream), one float a row, and the
checkpoints of three activations: the inputs of both layers and of the GELU, 33/32 of a byte a value.

    python examples/checkpointed_block.py [--rows 1024] [--width 768] [--hidden 3072] [--sparsity 90] [--format int8]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import coo_spmm_amd as L  # noqa: E402


def sparse_layer(out_features, in_features, sparsity, rows, gen):
    """Positions drawn uniformly, values of a variance that keeps the activations' size."""
    cells = out_features * in_features
    nnz = max(1, cells * (100 - sparsity) // 100)
    pos = torch.randperm(cells, device="cuda", generator=gen)[:nnz].sort().values
    vals = torch.randn(nnz, device="cuda", generator=gen) * (out_features / nnz) ** 0.5
    return L.SnackLayer(out_features, in_features, (pos // in_features).int(), (pos % in_features).int(), vals,
                        seed=1, max_batch=rows)


class CheckpointedBlock:
    def __init__(self, width, hidden, sparsity, rows, fmt=L.INT8, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.up = sparse_layer(hidden, width, sparsity, rows, gen)
        self.down = sparse_layer(width, hidden, sparsity, rows, gen)
        self.gain = torch.ones(width, device="cuda")
        self.fmt, self.kept = fmt, None

    def forward(self, x, residual):
        """The block's output for the hidden state residual (bf16) + x (fp32), as (branch, hidden state)."""
        h, y, rstd, ck_y = L.rmsnorm_fwd(x, self.gain, 1e-6, residual=residual, q_format=self.fmt)
        g, ck_a, ck_g = L.gelu_ckpt_fwd(self.up.forward(y), self.fmt)
        self.kept = (h, rstd, ck_y, ck_a, ck_g)
        return self.down.forward(g), h

    def kept_bytes(self):
        h, rstd, *cks = self.kept
        return h.numel() * h.element_size() + rstd.numel() * 4 + sum(c.nbytes for c in cks)

    def backward(self, d_out):
        """Gradients from that of branch + hidden state: (d_x, d_gain, d_up, d_down)."""
        h, rstd, ck_y, ck_a, ck_g = self.kept
        d_g, d_down = self.down.backward_ckpt(ck_g, d_out)
        d_y, d_up = self.up.backward_ckpt(ck_y, L.gelu_ckpt_bwd(ck_a, d_g))
        d_x, d_gain = L.rmsnorm_bwd(h, self.gain, rstd, d_y, dR=d_out)
        return d_x, d_gain, d_up, d_down

    def step(self, x, residual, target, lr):
        """One step on the mean squared error of branch + hidden state; the loss, as a device tensor."""
        branch, h = self.forward(x, residual)
        err = branch + h.float() - target
        _, d_gain, d_up, d_down = self.backward(err * (2.0 / err.numel()))
        self.gain -= lr * d_gain
        self.up.sgd_step(d_up, lr)
        self.down.sgd_step(d_down, lr)
        return (err * err).mean()

    def close(self):
        self.up.close()
        self.down.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--width", type=int, default=768)
    ap.add_argument("--hidden", type=int, default=3072)
    ap.add_argument("--sparsity", type=int, default=90)
    ap.add_argument("--format", choices=("int8", "e4m3"), default="int8")
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--lr", type=float, default=20.0)
    a = ap.parse_args()
    if a.steps < 1:
        ap.error("--steps must be at least 1")
    block = CheckpointedBlock(a.width, a.hidden, a.sparsity, a.rows, L.INT8 if a.format == "int8" else L.E4M3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    residual = torch.randn(a.rows, a.width, device="cuda", generator=gen).bfloat16()
    x = torch.randn(a.rows, a.width, device="cuda", generator=gen) * 0.1
    target = torch.randn(a.rows, a.width, device="cuda", generator=gen)
    first = float(block.step(x, residual, target, a.lr))
    full = 4 * a.rows * (2 * a.width + 2 * a.hidden)
    print(f"kept for the backward pass: {block.kept_bytes() / 1e6:.2f} MB ({full / 1e6:.2f} MB in fp32)")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(a.steps):
        loss = block.step(x, residual, target, a.lr)
        if (i + 1) % max(1, a.steps // 10) == 0:
            for layer in (block.up, block.down):      # a dynamic-sparsity step
                layer.prune_regrow(layer.nnz // 50)
            print(f"step {i + 1}: loss {float(loss):.4f}", flush=True)
    torch.cuda.synchronize()
    print(f"loss {first:.4f} -> {float(loss):.4f}, {(time.perf_counter() - t0) / a.steps * 1e3:.3f} ms a step")
    block.close()


if __name__ == "__main__":
    main()
