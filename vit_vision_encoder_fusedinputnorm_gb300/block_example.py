"""From pixels to a prompt: the front end, a tower block and the language side's attention.

    python -m vit_vision_encoder_fusedinputnorm_gb300.block_example

Two stills and a short video go through the front end (embeddings, RoPE tables, sequence
boundaries) and one encoder block, forward and backward.  Then a prompt of text and those items
gets its three-axis positions, and its queries and keys are rotated and attended, causally, first
as a whole and then its last token alone: that row has to come out the same both ways.
"""
from __future__ import annotations

import torch

from . import encoder as E
from . import synth
from .frontend import FrontEnd


def tower(hidden: int = 256, heads: int = 4, seed: int = 7):
    """(output, gradient of the input, front end, batch) of one block over the items' embeddings."""
    wl = synth.small_workload(seed, [(1, 16, 16, 1), (1, 10, 22, 1), (4, 8, 6, 8)], patch=14, hidden=hidden,
                              head_dim=hidden // heads)
    fe = FrontEnd.from_workload(wl)
    batch = fe.upload(wl.items)
    x, cos, sin = fe.embed_rope(batch, hidden // heads, wl.theta)
    cu, _ = fe.cu_seqlens(batch, 16)
    plan = E.AttentionPlan(cu, cu, batch.live_rows, batch.live_rows, heads, heads, hidden // heads)
    torch.manual_seed(seed)
    block = E.EncoderBlock(hidden, heads, 4 * hidden)
    x.requires_grad_(True)
    y = block(x, cos, sin, plan)
    y.float().square().mean().backward()
    return y.detach(), x.grad, block, fe, batch


def prompt(batch, heads: int = 8, heads_kv: int = 2, head_dim: int = 128, seed: int = 8):
    """Rotated and attended rows of a prompt over the batch's items: all at once, and the last token alone."""
    # text, the first still, text, the second, text, the video, text: one sequence
    spans = torch.tensor([[1, 5, 0, 1], [0, 9, 1, 1], [0, 3, 2, 2], [0, 12, -1, 1]], dtype=torch.int32, device="cuda")
    n_spans = torch.tensor([4], dtype=torch.int32, device="cuda")
    merged = [int(i["t"]) * int(i["h"]) * int(i["w"]) // 4 for i in batch.host_items]
    rows = 5 + 9 + 3 + 12 + sum(merged)
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    pos = E.mrope_positions(spans, n_spans, batch.items, batch.n_items, rows, merge=2, status=status)
    if status.tolist() != [0, -1]:
        raise RuntimeError(f"positions: device status {status.tolist()}")
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((rows, heads + 2 * heads_kv, head_dim), generator=g, device="cuda").to(torch.bfloat16)
    axes = E.section_axes((16, 24, 24))
    q, k = E.mrope_apply(qkv[:, :heads], qkv[:, heads:heads + heads_kv], pos, axes, theta=1e6)
    v = qkv[:, heads + heads_kv:]
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    whole = E.attention(q, k, v, E.AttentionPlan(cu, cu, rows, rows, heads, heads_kv, head_dim, causal=True))
    step = E.attention(q[-1:], k, v, E.AttentionPlan(one, cu, 1, rows, heads, heads_kv, head_dim, causal=True))
    return pos, whole, step


def main() -> None:
    y, dx, block, fe, batch = tower()
    grads = [p.grad for p in block.parameters()]
    if not all(torch.isfinite(t).all() for t in [y, dx] + grads):
        raise RuntimeError("the block's output or gradients are not finite")
    pos, whole, step = prompt(batch)
    off = float((whole[-1] - step[0]).abs().max())
    if off > 2e-2:
        raise RuntimeError(f"the last token alone differs by {off}")
    fe.close()
    print(f"tower block: {tuple(y.shape)}, prompt: {whole.shape[0]} rows up to position {int(pos.max())}, "
          f"last token alone within {off:.1e}")


if __name__ == "__main__":
    main()
