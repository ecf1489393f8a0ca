"""From token states to a trained pooling query: head norms, rotation and cross attention before the pair loss.

A tower hands on the states of every token of a batch, item after item on one tape.  This example pools them the way
the losses of this library want them:

  1. keys are normalised per head and rotated by their place in their item, and so is one learned query (position 0);
  2. the query attends to every item's states, which gives one vector per item;
  3. the vectors are normalised and scored by the sigmoid pair loss (items 2 i and 2 i + 1 belong together);
  4. the loss's gradient goes back through attention, rotation and norm to the query, its gain and the keys' gain, and
     plain gradient steps follow.

The states' heads carry a shared direction per pair of items in a few of their tokens, so there is something to find:
the loss falls as the query learns to look for those tokens.  Run it on a GPU: python examples/pool_states.py
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import contrastive_late_interaction_gb300 as cli  # noqa: E402


def batch(items, heads, dim, seed, device):
    """Keys and values [states, heads, dim] bf16 and offsets [items + 1]: noise, and in every eighth token a common key
    with the pair's own value."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    lengths = torch.randint(64, 512, (items,), generator=torch.Generator().manual_seed(seed))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), lengths.cumsum(0))).to(device)
    rows = int(lengths.sum())
    item = torch.repeat_interleave(torch.arange(items, device=device), lengths.to(device), output_size=rows)
    place = torch.arange(rows, device=device) - offsets[item]
    k = torch.randn(rows, heads, dim, generator=g, device=device)
    v = torch.randn(rows, heads, dim, generator=g, device=device)
    tell = (place % 8 == 0)[:, None, None]
    pair = torch.randn((items + 1) // 2, heads, dim, generator=g, device=device)
    k = torch.where(tell, 0.5 * k + 1.0, k)
    v = torch.where(tell, 0.5 * v + pair[item // 2], v)
    return k.bfloat16(), v.bfloat16(), offsets, place.int(), int(lengths.max())


def relations(items, device):
    """Items 2 i and 2 i + 1 attract each other."""
    other = np.arange(items, dtype=np.uint32) ^ 1
    return cli.device_edges((np.arange(items + 1, dtype=np.uint64), other), device)


def train(items=256, heads=8, dim=64, steps=30, rate=3.0, seed=0, device="cuda", say=print):
    """Runs the steps; returns the losses."""
    k, v, offsets, place, longest = batch(items, heads, dim, seed, device)
    table = cli.rotary_table(longest, dim // 2, device=device)["table"]   # half of each head is rotated
    attract = relations(items, device)
    t, b = torch.tensor([10.0], device=device), torch.tensor([-10.0], device=device)
    query = 0.2 * torch.randn(1, heads, dim, generator=torch.Generator(device=device).manual_seed(seed + 1), device=device)
    q_gain, k_gain = torch.ones(dim, device=device), torch.ones(dim, device=device)
    losses = []
    for step in range(steps):
        q = query.bfloat16()
        n = cli.norm_rotary_heads(q, table, q_gain=q_gain, k=k, k_positions=place, k_gain=k_gain)
        a = cli.cross_attention(n["q"], None, n["k"], v, offsets, max_key_rows=longest)
        pooled = a["output"].view(items, heads * dim).float()
        length = pooled.norm(dim=1, keepdim=True)
        e = pooled / length
        r = cli.pair_loss_sigmoid_fwd_bwd(e.bfloat16(), t, b, attract)
        de = r["d_embeddings"]
        d_pooled = (de - e * (de * e).sum(1, keepdim=True)) / length
        # The gradients are scaled up for bf16 on the way, and down again in the step.
        scale = items
        d = cli.cross_attention_backward(n["q"], None, n["k"], v, offsets, a["output"], a["lse"],
                                         (scale * d_pooled).view(items, heads, dim).bfloat16(), max_key_rows=longest)
        g = cli.norm_rotary_heads_backward(q, d["d_q"], table, q_gain=q_gain, k=k, d_k=d["d_k"], k_positions=place,
                                           k_gain=k_gain)
        query -= rate / scale * g["d_q"].float()
        q_gain -= rate / scale * 0.1 * g["d_q_gain"]
        k_gain -= rate / scale * 0.1 * g["d_k_gain"]
        for x, what in ((n, "norm_rotary_heads"), (a, "cross_attention"), (r, "pair_loss_sigmoid_fwd_bwd"),
                        (d, "cross_attention_backward"), (g, "norm_rotary_heads_backward")):
            cli.check_device_status(x["device_status"], what)
        losses.append(r["loss"].item())
        if step % 5 == 0 or step + 1 == steps:
            say(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--items", type=int, default=256)
    p.add_argument("--heads", type=int, default=8)
    p.add_argument("--dim", type=int, default=64)
    p.add_argument("--steps", type=int, default=30)
    a = p.parse_args()
    train(a.items, a.heads, a.dim, a.steps)
