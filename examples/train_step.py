"""Training steps of a small model: a matrix on token embeddings, and an output head.

Each step takes the loss and its gradients through the head (``cross_entropy_grad``: the logits are
never held), the matrix's gradient by ordinary products (``matmul``), and updates the matrix by its
orthogonalised momentum (``orthogonalize``), the head by plain descent. The task is to predict a
fixed successor of each token; a quarter of the positions is masked.

    python -m examples.train_step [steps]        (from the repository's root)
"""

import sys

import torch

import dense_fp32_gemm_sgemm_gb300 as sg


class Model:
    def __init__(self, vocabulary=1000, width=192, hidden=256, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(*shape):
            return torch.randn(*shape, device="cuda", generator=gen)

        self.embedding = matrix(vocabulary, width)
        self.matrix = matrix(width, hidden) * width ** -0.5
        self.head = matrix(vocabulary, hidden) * hidden ** -0.5
        self.momentum = torch.zeros_like(self.matrix)

    def gradients(self, tokens, target):
        """(loss, gradient of the matrix, gradient of the head) in float32."""
        x = self.embedding[tokens]
        hidden = sg.matmul(x, self.matrix)
        loss, _, _, dhidden, dhead = sg.cross_entropy_grad(hidden, self.head, target)
        return loss, sg.matmul(x.T.contiguous(), dhidden), dhead

    def step(self, tokens, target, rate=0.05):
        loss, dmatrix, dhead = self.gradients(tokens, target)
        self.momentum.mul_(0.9).add_(dmatrix)
        self.matrix.sub_(sg.orthogonalize(self.momentum), alpha=rate)
        self.head.sub_(dhead, alpha=10 * rate)
        return loss


def batch(gen, vocabulary, size):
    tokens = torch.randint(vocabulary, (size,), device="cuda", generator=gen)
    masked = torch.rand(size, device="cuda", generator=gen) < 0.25
    return tokens, torch.where(masked, -100, (tokens * 7 + 3) % vocabulary)


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 20
    model = Model()
    gen = torch.Generator(device="cuda").manual_seed(1)
    losses = [model.step(*batch(gen, 1000, 512)) for _ in range(steps)]
    print([round(float(v), 3) for v in losses])


if __name__ == "__main__":
    main()
