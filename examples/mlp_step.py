"""A gated MLP in 2 bits, distilled from its own frozen 4-bit copy.

The student's gate, up and down projections are LC-VQ layers (2-bit codes, straight-through
backward). What its backward needs of the activations is kept in 8-bit checkpoints: the
input X once for gate and up, G and U for the gate, H for down, about half the bytes of
bfloat16. The teacher is the same MLP with MXFP4 weights; training runs it on the 4-bit
matrix cores, and at the end it decodes a single token from the same weights.

    python examples/mlp_step.py [--tokens 4096] [--hidden 4096] [--inner 11008] [--steps 20]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_lc_amd as P  # noqa: E402

D = 8


class Student:
    """One LC-VQ projection [N, K], started on the uniform grid {-1.5, -.5, .5, 1.5} sigma."""

    def __init__(self, W):
        s = float(W.std())
        self.A = s * torch.eye(D, device=W.device)
        self.B = torch.full((D,), -1.5 * s, device=W.device)
        self.Wp = (W / s + 1.5).contiguous()
        self.scale = s

    def forward(self, X):
        out = P.linear_fwd(X, self.Wp, self.A, self.B, D)
        self.packed, self.mask = out["packed"], out["mask"]
        return out["Y"]

    def backward(self, dY, X8):
        self.grad = P.linear_bwd_ckpt8(dY, *X8, self.packed, self.mask, self.A, self.B, D)
        return self.grad["dX"]

    def update(self, lr):
        # dWp carries a factor A (about sigma), as the weight A Wp + B does
        self.Wp -= lr / self.scale ** 2 * self.grad["dWp"]


class MLP:
    def __init__(self, hidden, inner, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        shapes = {"gate": (inner, hidden), "up": (inner, hidden), "down": (hidden, inner)}
        self.student, self.teacher = {}, {}
        for name, (n, k) in shapes.items():
            W = torch.randn(n, k, generator=g, device=device) * k ** -0.5
            self.student[name] = Student(W)
            self.teacher[name] = P.mx_quantize(W, P.LCVQ_MXFP4)

    def teach(self, X, quantize_x=None):
        """The 4-bit MLP; the activations are MXFP4 too only with quantize_x (training)."""
        t = self.teacher
        G = P.mxfp4_linear(X, *t["gate"], quantize_x)
        U = P.mxfp4_linear(X, *t["up"], quantize_x)
        H = torch.empty_like(G)
        P.lcvq_silu_gate_fwd(G, U, H)
        return P.mxfp4_linear(H, *t["down"], quantize_x)

    def forward(self, X):
        s = self.student
        self.X8 = P.mx_quantize(X, P.LCVQ_MXINT8)
        self.gate = P.silu_gate_fwd(s["gate"].forward(X), s["up"].forward(X))
        return s["down"].forward(self.gate.pop("H"))

    def backward(self, dY):
        s = self.student
        dH = s["down"].backward(dY, self.gate["H8"])
        dG, dU = P.silu_gate_bwd(dH, self.gate["G8"], self.gate["U8"])
        return s["gate"].backward(dG, self.X8) + s["up"].backward(dU, self.X8)

    def saved_bytes(self):
        pairs = [self.X8, self.gate["G8"], self.gate["U8"], self.gate["H8"]]
        return sum(t.numel() for p in pairs for t in p)


def train_step(mlp, X, lr):
    """Mean squared distance to the teacher, its gradients, one descent step."""
    T = mlp.teach(X, quantize_x=True)
    Y = mlp.forward(X)
    err = Y.float() - T.float()
    loss = err.square().mean()
    mlp.dX = mlp.backward((err * (2 / X.shape[0])).bfloat16())
    for layer in mlp.student.values():
        layer.update(lr)
    return loss


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=11008)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    mlp = MLP(a.hidden, a.inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    for i in range(a.steps):
        loss = train_step(mlp, X, a.lr)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i}: loss {float(loss):.5f}", flush=True)
    wide = 2 * a.tokens * (a.hidden + 3 * a.inner)
    print(f"kept for the backward: {mlp.saved_bytes() / 2**20:.1f} MiB "
          f"({wide / 2**20:.1f} MiB in bfloat16)")
    y1, y4 = mlp.teach(X[:1].contiguous()), mlp.teach(X[:1].contiguous(), quantize_x=True)
    print(f"one token decoded with 4-bit weights: |Y| {float(y1.float().norm()):.3f}, with 4-bit "
          f"activations too: {float((y1 - y4).float().norm() / y1.float().norm()):.3f} apart")


if __name__ == "__main__":
    main()
