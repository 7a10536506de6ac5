"""One decoder block as a serving loop runs it: latent attention, then the NVFP4 expert layer.

A batch of prompts goes through prefill (expanded attention, rows appended to
the paged cache), then tokens are decoded one by one (absorbed attention over
the cache).  The last step is compared with a prefill of the whole sequences.

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

    def __init__(self, D=512, heads=16, experts=8, k=2, inner=256, positions=4096, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.D = D
        self.attention = mla.LatentAttention(
            w(heads * 192, D, std=D ** -0.5), w(576, D, std=D ** -0.5), w(512, std=0.1) + 1.0,
            w(heads * 256, 512, std=512 ** -0.5), w(D, heads * 128, std=(heads * 128) ** -0.5), mla.rope_table(positions))
        self.router = w(experts, D, std=D ** -0.5)
        self.experts = B.MoELayer(w(experts, 2 * inner, D, std=0.02), w(experts, D, inner, std=0.02), k, autotune=False)

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


def serve(lengths=(37, 130, 5), steps=4, block=None, seed=1):
    """Prefills prompts of these lengths, decodes `steps` tokens of each.  Returns the last
    tokens' outputs by decoding and by prefilling everything, [sequences, D] each."""
    block = Block() if block is None else block
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = len(lengths)
    total = [m + steps for m in lengths]
    x = [torch.randn((m, block.D), generator=g, device="cuda").to(torch.bfloat16) for m in total]
    # every sequence owns pages in an order of its own
    need = [-(-m // PAGE) for m in total]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32).split(need)
    tables = torch.full((n, max(need)), -1, dtype=torch.int32, device="cuda")
    for b, ids in enumerate(order):
        tables[b, :len(ids)] = ids

    def slots(b, positions):
        return tables[b].long()[positions // PAGE] * PAGE + positions % PAGE

    def prefill(upto, cache):
        at = [torch.arange(m, device="cuda") for m in upto]
        cu = torch.tensor([0, *upto], device="cuda").cumsum(0).to(torch.int32)
        y = block.prefill(torch.cat([x[b][:m] for b, m in enumerate(upto)]), torch.cat(at).to(torch.int32),
                          torch.cat([slots(b, p) for b, p in enumerate(at)]), cache, cu)
        return y[cu[1:].long() - 1]

    def new_cache():
        return torch.zeros((sum(need), PAGE, mla.ROW), dtype=torch.bfloat16, device="cuda")

    cache = new_cache()
    prefill(list(lengths), cache)
    for step in range(steps):
        now = torch.tensor([m + step for m in lengths], device="cuda")
        y = block.decode(torch.stack([x[b][m + step] for b, m in enumerate(lengths)]), now.to(torch.int32),
                         torch.stack([slots(b, now[b]) for b in range(n)]), cache, tables, (now + 1).to(torch.int32))
    decoded = y.clone()
    whole = prefill(total, new_cache()).clone()
    B.sync_status()
    return decoded, whole


def main():
    B.device_check()
    decoded, whole = serve()
    off = (decoded.float() - whole.float()).norm() / whole.float().norm()
    print(f"last tokens by decoding and by prefilling: relative difference {off:.2e}")


if __name__ == "__main__":
    main()
