"""One decoder block as a serving loop runs it: latent attention, then the NVFP4 expert layer.

A batch of prompts goes through prefill (expanded attention, rows appended to
the paged cache), then tokens are decoded one by one (absorbed attention over
the cache).  Pages, slots and positions of each step are planned on the GPU.
The last step is compared with a prefill of the whole sequences.  `Stepper`
runs a decode step without the host: as one CUDA graph.

    python examples/decoder_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from nvfp4_block_scaled_07_gb300 import binding as B  # noqa: E402
from nvfp4_block_scaled_07_gb300 import mla  # noqa: E402

PAGE = 64


class Block:
    """x + attention(norm(x)), then x + experts(norm(x)), with random weights."""

    def __init__(self, D=512, heads=16, experts=8, k=2, inner=256, positions=4096, seed=0, **layer):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.D = D
        self.attention = mla.LatentAttention(
            w(heads * 192, D, std=D ** -0.5), w(576, D, std=D ** -0.5), w(512, std=0.1) + 1.0,
            w(heads * 256, 512, std=512 ** -0.5), w(D, heads * 128, std=(heads * 128) ** -0.5), mla.rope_table(positions))
        self.router = w(experts, D, std=D ** -0.5)
        self.experts = B.MoELayer(w(experts, 2 * inner, D, std=0.02), w(experts, D, inner, std=0.02), k, autotune=False,
                                  **layer)

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:])

    def experts_of(self, x):
        y = self.norm(x)
        return x + self.experts(y, (y @ self.router.T).float())

    def prefill(self, x, positions, slots, cache, cu):
        return self.experts_of(x + self.attention.prefill(self.norm(x), positions, slots, cache, cu))

    def decode(self, x, positions, slots, cache, tables, lens):
        return self.experts_of(x + self.attention.decode(self.norm(x), positions, slots, cache, tables, lens))


class Stepper:
    """Decode steps of a batch of sequences as one captured graph: the plan of their new tokens' pages, attention and
    experts.  A call takes the next tokens; lengths, tables and free pages stay on the GPU, and so does the result `y`,
    which the next call overwrites."""

    def __init__(self, block, cache, lens, tables, free_pages, free_count):
        n = lens.numel()
        self.block, self.cache, self.tables, self.free_pages = block, cache, tables, free_pages
        self.x = torch.zeros((n, block.D), dtype=torch.bfloat16, device="cuda")
        self.lens, self.one = lens.clone(), torch.ones_like(lens)
        self.plan = mla.alloc_token_plan(n, n, "cuda", free_count=free_count)
        state = [t.clone() for t in (self.lens, tables, free_count)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self._step()                     # an eager step first, whose effects are taken back
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.y = self._step()
        torch.cuda.current_stream().wait_stream(side)
        for t, was in zip((self.lens, tables, free_count), state):
            t.copy_(was)

    def _step(self):
        p = mla.mla_plan(self.lens, self.one, self.tables, self.free_pages, self.plan.free_count, PAGE, self.lens.numel(),
                         out=self.plan)
        y = self.block.decode(self.x, p.positions, p.slots, self.cache, self.tables, p.seq_lens)
        self.lens.copy_(p.seq_lens)
        return y

    def __call__(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def serve(lengths=(37, 130, 5), steps=4, block=None, seed=1, graph=False):
    """Prefills prompts of these lengths, decodes `steps` tokens of each.  Returns the last
    tokens' outputs by decoding and by prefilling everything, [sequences, D] each."""
    block = Block() if block is None else block
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = len(lengths)
    total = [m + steps for m in lengths]
    x = [torch.randn((m, block.D), generator=g, device="cuda").to(torch.bfloat16) for m in total]
    pages = sum(-(-m // PAGE) for m in total)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    class State:
        """An empty cache whose pages are handed out in an order of their own."""

        def __init__(self):
            self.cache = torch.zeros((pages, PAGE, mla.ROW), dtype=torch.bfloat16, device="cuda")
            self.tables = torch.full((n, -(-max(total) // PAGE)), -1, dtype=torch.int32, device="cuda")
            self.free_pages = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
            self.free_count, self.lens = ints([pages]), ints([0] * n)

        def plan(self, new):
            p = mla.mla_plan(self.lens, ints(new), self.tables, self.free_pages, self.free_count, PAGE, sum(new))
            self.lens, self.free_count = p.seq_lens, p.free_count
            return p

        def prefill(self, upto):
            p = self.plan(upto)
            y = block.prefill(torch.cat([x[b][:m] for b, m in enumerate(upto)]), p.positions, p.slots, self.cache,
                              p.cu_seqlens)
            return y[p.cu_seqlens[1:].long() - 1]

        def decode(self, tokens):
            p = self.plan([1] * n)
            return block.decode(tokens, p.positions, p.slots, self.cache, self.tables, p.seq_lens)

    s = State()
    s.prefill(list(lengths))
    decode = Stepper(block, s.cache, s.lens, s.tables, s.free_pages, s.free_count) if graph else s.decode
    for step in range(steps):
        y = decode(torch.stack([x[b][m + step] for b, m in enumerate(lengths)]))
    decoded = y.clone()
    whole = State().prefill(total).clone()
    B.sync_status()
    return decoded, whole


def main():
    B.device_check()
    decoded, whole = serve()
    off = (decoded.float() - whole.float()).norm() / whole.float().norm()
    print(f"last tokens by decoding and by prefilling: relative difference {off:.2e}")
    # groups of experts, and batches of few tokens with 16-bit activations, as one graph a step
    block = Block(n_group=4, topk_group=2, select_bias=torch.zeros(8, device="cuda"), routed_scale=2.5, few_tokens=8)
    decoded, whole = serve(block=block, graph=True)
    off = (decoded.float() - whole.float()).norm() / whole.float().norm()
    print(f"grouped routing, few tokens, as graphs: {off:.2e}")


if __name__ == "__main__":
    main()
