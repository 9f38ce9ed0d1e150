"""Decoding with 4-bit weights: a few tokens a step through a small model.

The model is a stack of residual blocks (a square projection and a mixture-of-experts layer) on
token embeddings, and an output head. Its weights are quantised once. Each step is one CUDA graph
replay: products of a few rows (``q4_matmul``), the expert layers (``MoeLayer``), and the next
tokens by the largest logit. Weights are random, so what it says means nothing.

    python -m examples.decode_4bit [tokens]        (from the repository's root)
"""

import sys

import torch

import dense_fp32_gemm_sgemm_gb300 as sg


class Block:
    def __init__(self, gen, width, hidden, experts, top_k, group, dtype):
        def matrix(*shape):
            return torch.randn(*shape, device="cuda", generator=gen) * shape[-2] ** -0.5

        self.proj = sg.q4_quantize(matrix(width, width), group=group)
        gate, up, down = (sg.q4_quantize(matrix(experts, n, k), group=group)
                          for n, k in ((width, hidden), (width, hidden), (hidden, width)))
        router = matrix(width, experts).T.contiguous().to(dtype)
        self.experts = sg.MoeLayer(router, gate, up, down, top_k=top_k, dtype=dtype)

    def __call__(self, x, live):
        x = x + sg.q4_matmul(normed(x), self.proj)
        return x + self.experts(normed(x), live=live)[0]


def normed(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Model:
    def __init__(self, vocabulary=1000, width=256, hidden=192, blocks=2, experts=8, top_k=2,
                 group=64, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn(vocabulary, width, device="cuda", generator=gen).to(dtype)
        self.blocks = [Block(gen, width, hidden, experts, top_k, group, dtype)
                       for _ in range(blocks)]
        self.head = sg.q4_quantize(
            torch.randn(vocabulary, width, device="cuda", generator=gen) * width ** -0.5,
            group=group, transposed=True)

    def logits(self, tokens, live=None):
        """Logits for one token of each sequence (at most 64); those not live get zeros' logits."""
        x = self.embedding[tokens]
        for block in self.blocks:
            x = block(x, live)
        return sg.q4_matmul(normed(x), self.head)


class Decoder:
    """Steps of a fixed number of sequences, captured once."""

    def __init__(self, model, sequences):
        self.tokens = torch.zeros(sequences, dtype=torch.int64, device="cuda")
        self.live = torch.ones(sequences, dtype=torch.bool, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            model.logits(self.tokens, self.live)  # loads the kernels before the capture
        torch.cuda.current_stream().wait_stream(stream)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.logits = model.logits(self.tokens, self.live)
            following = self.logits.float().argmax(-1)
            self.tokens.copy_(torch.where(self.live, following, self.tokens))

    def run(self, tokens, steps):
        """steps more tokens after the given ones: sequences x steps."""
        self.tokens.copy_(tokens)
        out = []
        for _ in range(steps):
            self.graph.replay()
            out.append(self.tokens.clone())
        return torch.stack(out, 1)


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    decoder = Decoder(Model(), sequences=4)
    print(decoder.run(torch.arange(4, device="cuda"), steps).tolist())


if __name__ == "__main__":
    main()
