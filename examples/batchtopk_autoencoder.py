"""Trains a BatchTopK sparse autoencoder on synthetic activations, every step in the library's kernels.

    python examples/batchtopk_autoencoder.py --steps 200

A step is: encode (linear with ReLU), keep the K = rows x k largest activations of the batch (select_global),
reconstruct from them (decode), the squared error, its gradients through the decoder (decode_backward) and through
the selected activations to the encoder (linear_backward_selected), clipping of all gradients by their common norm
(clip_grad_norm_), and a step of Adam.  The data are sparse mixtures of hidden directions, so the loss has a way down.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import top_selection_prof_gb300 as tk  # noqa: E402


class Autoencoder:
    def __init__(self, width, features, k, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn(features, width, device="cuda", generator=g)
        w /= w.norm(dim=1, keepdim=True)
        self.k = k
        self.params = {"w_enc": w.clone(), "b_enc": torch.zeros(features, device="cuda"), "w_dec": w,
                       "b_dec": torch.zeros(width, device="cuda")}
        self.moments = {n: (torch.zeros_like(p), torch.zeros_like(p)) for n, p in self.params.items()}
        self.dtype, self.steps = dtype, 0

    def gradients(self, x):
        """(loss, reconstruction, gradients by name) for a batch x (rows, width): the squared error of a row, averaged."""
        p = {n: t.to(self.dtype) for n, t in self.params.items()}
        rows = x.shape[0]
        acts = tk.linear(x, p["w_enc"], p["b_enc"], act="relu")
        vals, idx = tk.select_global(acts, rows * self.k)
        y = tk.decode(vals, idx, p["w_dec"], rows, bias=p["b_dec"])
        err = y.float() - x.float()
        loss = err.square().sum() / rows
        dy = (err * (2.0 / rows)).to(self.dtype)
        dvals, dw_dec, db_dec = tk.decode_backward(dy, vals, idx, p["w_dec"])
        _, dw_enc, db_enc = tk.linear_backward_selected(dvals, vals, idx, x, p["w_enc"], act="relu",
                                                        need=(False, True, True))
        return loss, y, {"w_enc": dw_enc, "b_enc": db_enc, "w_dec": dw_dec, "b_dec": db_dec}

    def step(self, x, lr=2e-3, max_norm=1.0, betas=(0.9, 0.999), eps=1e-8):
        """One training step; returns (loss, gradient norm)."""
        loss, _, grads = self.gradients(x)
        norm = tk.clip_grad_norm_(list(grads.values()), max_norm)
        self.steps += 1
        c1, c2 = 1 - betas[0] ** self.steps, 1 - betas[1] ** self.steps
        for n, p in self.params.items():
            g, (m, v) = grads[n].float(), self.moments[n]
            m.lerp_(g, 1 - betas[0])
            v.lerp_(g * g, 1 - betas[1])
            p.sub_(lr * (m / c1) / ((v / c2).sqrt() + eps))
        return loss, norm


def batches(width, directions, active, rows, dtype=torch.bfloat16, seed=1):
    """Batches of sums of a few of `directions` fixed directions."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = torch.randn(directions, width, device="cuda", generator=g) / width ** 0.5
    while True:
        code = torch.rand(rows, directions, device="cuda", generator=g)
        code = torch.where(torch.rand(rows, directions, device="cuda", generator=g) < active / directions, code + 0.5, 0.0)
        yield (code @ d).to(dtype)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--features", type=int, default=4096)
    ap.add_argument("--k", type=int, default=32)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    model, data = Autoencoder(a.width, a.features, a.k), batches(a.width, a.features // 4, 24, a.rows)
    for i in range(a.steps):
        loss, norm = model.step(next(data))
        if i % 20 == 0 or i == a.steps - 1:
            print("step %4d  loss %.5f  gradient norm %.4f" % (i, float(loss), float(norm)))


if __name__ == "__main__":
    main()
