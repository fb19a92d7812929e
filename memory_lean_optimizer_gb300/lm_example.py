"""A small language model trained with the memory-lean tail and optimizer, as they are used together:

    python -m memory_lean_optimizer_gb300.lm_example [--steps 60] [--vocab 8192] [--states u8|fp32] [--blocks 2]

An embedding feeds ``head.LMTail`` (layer norm, output matrix, cross entropy without logits), through
transformer blocks over the packed tokens if asked for (``block.TransformerBlock``); every parameter is bf16 with a Kahan residual and is stepped by AdamW with 8-bit (or fp32) moments from its
gradient hook during the backward pass (``hooks.attach_fused_adamw``), so that neither the logits nor
the gradients of the whole model nor fp32 moments exist at any time.  The data are synthetic: each
token follows from the one before it, and a part of the positions carries no target.
"""
from __future__ import annotations

import argparse

import torch

from . import block, head, hooks


def block_heads(dim: int) -> tuple[int, int]:
    """(heads, kv_heads) of a block of this width: heads of 64 elements or the next more that divide it, else of fewer, of the
    sizes that attention takes."""
    first = max(dim // 64, 1)
    for heads in (*range(first, 0, -1), *range(first + 1, dim + 1)):
        if dim % heads == 0 and dim // heads % 8 == 0 and dim // heads <= 128:
            return heads, heads // 2 if heads % 2 == 0 else heads
    raise ValueError(f"a width of {dim} does not make heads of a multiple of 8 up to 128")


class TinyLM(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, blocks: int = 0):
        super().__init__()
        heads = block_heads(dim) if blocks else (1, 1)
        self.embed = torch.nn.Embedding(vocab, dim, device="cuda", dtype=torch.bfloat16)
        self.tail = head.LMTail(dim, vocab)
        self.blocks = torch.nn.ModuleList(block.TransformerBlock(dim, *heads) for _ in range(blocks))

    def forward(self, tokens: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        x = self.embed(tokens)
        if self.blocks:                        # tokens [rows, length] as sequences side by side
            rows, length = tokens.shape
            x = x.flatten(0, 1)
            positions = torch.arange(length, device=x.device).repeat(rows)
            borders = torch.arange(rows + 1, device=x.device, dtype=torch.int32) * length
            for b in self.blocks:
                x = b(x, positions, borders)
            x = x.view(rows, length, -1)
        return self.tail(x, target)


def batch(vocab: int, rows: int, length: int, gen: torch.Generator):
    """Tokens and targets: the next token is a fixed function of the present one; one target in eight is masked."""
    tokens = torch.randint(vocab, (rows, length), generator=gen, device="cuda")
    target = (tokens * 5 + 17) % vocab
    target[torch.rand(rows, length, generator=gen, device="cuda") < 0.125] = -100
    return tokens, target


def train(steps: int = 60, vocab: int = 8192, dim: int = 256, rows: int = 16, length: int = 512, states: str = "u8",
          lr: float = 5e-3, seed: int = 0, log=None, blocks: int = 0) -> list[float]:
    """Trains the model; returns the loss of every step."""
    torch.manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = TinyLM(vocab, dim, blocks)
    stepper = hooks.attach_fused_adamw(list(model.parameters()), 2, dict(lr=lr, beta2=0.99, weight_decay=0.01), states=states)
    losses = []
    for step in range(steps):
        loss = model(*batch(vocab, rows, length, gen))
        loss.backward()                        # the groups step from the hooks, the gradients are gone after it
        losses.append(loss.detach())
        if log and step % 10 == 0:
            log(f"step {step:4d}  loss {float(loss.detach()):.4f}")
    stepper.remove()
    return [float(x) for x in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--states", choices=("u8", "fp32"), default="u8")
    ap.add_argument("--blocks", type=int, default=0)
    args = ap.parse_args()
    torch.cuda.reset_peak_memory_stats()
    losses = train(steps=args.steps, vocab=args.vocab, states=args.states, log=print, blocks=args.blocks)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; peak memory {torch.cuda.max_memory_allocated() / 2 ** 20:.0f} MiB "
          f"(fp32 logits and their gradient alone: {2 * 16 * 512 * args.vocab * 4 / 2 ** 20:.0f} MiB)")


if __name__ == "__main__":
    main()
