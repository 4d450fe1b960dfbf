"""Quantisation-aware distillation of a small two-layer student, every product in 4 bits.

A teacher (bf16) maps token features to logits: tanh(x W1^T) W2^T.  The student has the same weights, held as FP32
masters and quantised to MXFP4 for every product, and is trained on the teacher's top log-probabilities:

    forward    h = tanh(Q(x) Q(W1)^T),  z = Q(h) Q(W2)^T              (W4A4 products)
    loss       KL(teacher || student) on the teacher's top entries and one class for the rest, with dz in one pass
    backward   dh = Q(dz) Q_c(W2),  dW = Q_c(dY)^T Q_c(X)             (straight-through quantisers)

Run it on a GB300:  python examples/qad_step.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_weight_only_02_gb300 import binding as nv  # noqa: E402


class Student:
    """Two linear layers with FP32 master weights and MXFP4 products."""

    def __init__(self, w1, w2, tokens):
        self.w1, self.w2 = w1.float().clone(), w2.float().clone()
        (hidden, features), vocab = w1.shape, w2.shape[0]
        need = [nv.nvfp4_w4a4_workspace_bytes(tokens, hidden, features),
                nv.nvfp4_w4a4_workspace_bytes(tokens, vocab, hidden),
                nv.nvfp4_mx_linear_backward_workspace_bytes(tokens, hidden, features),
                nv.nvfp4_mx_linear_backward_workspace_bytes(tokens, vocab, hidden)]
        self.workspace = nv.new_workspace(max(need))

    def forward(self, x):
        """Logits (bf16) and what the backward pass needs."""
        ws = self.workspace
        xq, w1 = nv.mx_quantize(x, colwise=True), nv.mx_quantize(self.w1, colwise=True)
        h = torch.tanh(nv.w4a4_gemm(xq.row, w1.row, workspace=ws))
        hq, w2 = nv.mx_quantize(h, colwise=True), nv.mx_quantize(self.w2, colwise=True)
        z = nv.w4a4_gemm(hq.row, w2.row, out_dtype=torch.bfloat16, workspace=ws)
        return z, (xq.col, w1.col, h, hq.col, w2.col)

    def backward(self, dz, saved):
        """Gradients of both master weights."""
        x_col, w1_col, h, h_col, w2_col = saved
        dh, dw2 = nv.mx_linear_backward(dz, h_col, w2_col, workspace=self.workspace)
        _, dw1 = nv.mx_linear_backward(dh * (1 - h * h), x_col, None, workspace=self.workspace)
        return dw1, dw2


def teacher_entries(x, w1, w2, k):
    """Indices and log-probabilities of the teacher's k largest logits per token."""
    logits = torch.tanh(x.float() @ w1.float().t()) @ w2.float().t()
    return tuple(reversed(torch.topk(torch.log_softmax(logits, 1), k, dim=1)))


def train(steps=30, tokens=512, features=256, hidden=512, vocab=4000, k=32, lr=0.5, seed=0):
    """Returns the mean loss of every step, on the same tokens."""
    g = torch.Generator("cuda").manual_seed(seed)
    w1 = (torch.randn(hidden, features, device="cuda", generator=g) / features ** 0.5).bfloat16()
    w2 = (torch.randn(vocab, hidden, device="cuda", generator=g) * 3 / hidden ** 0.5).bfloat16()
    x = torch.randn(tokens, features, device="cuda", generator=g).bfloat16()
    index, logp = teacher_entries(x, w1, w2, k)
    weight = (torch.rand(tokens, device="cuda", generator=g) > 0.1).float()   # answer tokens
    weight /= weight.sum()
    student = Student(w1, w2, tokens)
    losses = []
    for _ in range(steps):
        z, saved = student.forward(x)
        # the gradient takes the logits' place
        loss, dz = nv.distill_topk_loss_grad(z, index, logp, tail=True, row_weight=weight, out=z)
        dw1, dw2 = student.backward(dz, saved)
        student.w1 -= lr * dw1
        student.w2 -= lr * dw2
        losses.append(float(loss.sum()))
    return losses


if __name__ == "__main__":
    losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
    for i, value in enumerate(losses):
        print(f"step {i:3d}  distillation loss {value:.5f}")
