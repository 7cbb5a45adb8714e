"""A small next-event model over user histories: the table-batched embedding
and the attention operators used together, trained and served.

Each user has a ragged history of events.  An event is a bag of item ids (the
item and its attributes), pooled by ``tbe_forward`` into one row; the rows are
projected to queries, keys and values; attention over the history (newest
``window`` events, first ``sinks`` events, learned bias by distance) gives the
state after each event, which predicts the next event's label.  One training
step runs every gradient through the library: ``tbe_attention_backward`` for
q, k, v and the bias table, ``tbe_backward_sgd`` for the item table.

Serving keeps the keys and values in a paged cache: the histories are appended
once, then each new event is appended and attends to its user's cache.

    python examples/history_model.py [--users 64] [--steps 20]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import recommender_sparse_embeddings_gb300 as tbe  # noqa: E402


class HistoryModel:
    def __init__(self, items=5000, dim=64, heads=4, kv_heads=2, head_dim=32, window=64, sinks=2, buckets=16,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device)

        self.dtype, self.heads, self.kv_heads, self.head_dim = dtype, heads, kv_heads, head_dim
        self.table = weight(items, dim, std=0.5)
        self.bags = tbe.tbe_create([self.table], "sum")
        self.w = weight(dim, (heads + 2 * kv_heads) * head_dim, std=dim ** -0.5)
        self.w_out = weight(heads * head_dim, 1, std=(heads * head_dim) ** -0.5)
        self.bias = weight(buckets, heads, std=0.1)
        self.attention = tbe.tbe_attention_create(heads, kv_heads, head_dim, dtype, window, sinks,
                                                  tbe.tbe_relative_buckets(buckets, window))

    def rows(self, ids, bag_offsets):
        """Pooled rows of the events and their q, k, v (views of one buffer)."""
        events = bag_offsets.numel() - 1
        x = tbe.tbe_forward(self.bags, ids, bag_offsets, events)
        qkv = (x @ self.w).to(self.dtype).view(events, self.heads + 2 * self.kv_heads, self.head_dim)
        h, k = self.heads, self.kv_heads
        return x, qkv[:, :h], qkv[:, h:h + k], qkv[:, h + k:]

    def step(self, ids, bag_offsets, offsets, labels, lr):
        """One training step on a batch of histories; returns the loss."""
        events = bag_offsets.numel() - 1
        x, q, k, v = self.rows(ids, bag_offsets)
        bias = self.bias.to(self.dtype)
        out, lse = tbe.tbe_attention_forward(self.attention, q, k, v, offsets, bias)
        flat = out.view(events, -1).float()
        logit = (flat @ self.w_out)[:, 0]
        loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, labels)
        d_logit = ((torch.sigmoid(logit) - labels) / events)[:, None]
        scale = float(events)  # the 16-bit gradients carry the sum, the updates divide
        d_out = (scale * d_logit @ self.w_out.t()).to(self.dtype).view_as(out)
        gq, gk, gv, gb = tbe.tbe_attention_backward(self.attention, q, k, v, offsets, out, lse, d_out, bias)
        d_qkv = torch.cat([gq, gk, gv], 1).view(events, -1).float() / scale
        d_x = (d_qkv @ self.w.t()).contiguous()
        workspace = tbe.make_workspace(self.bags, ids.numel(), events)
        self.w_out -= lr * flat.t() @ d_logit
        self.w -= lr * x.t() @ d_qkv
        self.bias -= lr * gb.float() / scale
        tbe.tbe_backward_sgd(self.bags, ids, bag_offsets, events, d_x, lr, workspace)
        return float(loss)

    def close(self):
        self.bags.close()
        self.attention.close()


class Cache:
    """A paged cache of a batch of users' keys and values."""

    def __init__(self, model, users, room, page=16, device="cuda"):
        width = (room + page - 1) // page
        shape = (users * width, page, model.kv_heads, model.head_dim)
        self.k = torch.empty(shape, dtype=model.dtype, device=device)
        self.v = torch.empty(shape, dtype=model.dtype, device=device)
        self.table = torch.randperm(users * width, device=device).to(torch.int32).view(users, width)
        self.lengths = torch.zeros(users, dtype=torch.int32, device=device)

    def append(self, model, k, v, offsets):
        tbe.tbe_attention_append(model.attention, k, v, offsets, self.lengths, self.k, self.v, self.table)
        self.lengths += (offsets[1:] - offsets[:-1]).to(torch.int32)


def make_histories(users, items, device, seed):
    """Ragged histories of 1 to 100 events, three ids an event; an event's label
    says whether its first id is even (learnable from the item table)."""
    g = torch.Generator().manual_seed(seed)
    lengths = torch.randint(1, 101, (users,), generator=g)
    events = int(lengths.sum())
    ids = torch.randint(0, items, (3 * events,), generator=g)
    labels = (ids[::3] % 2).float()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    return ids.to(device), torch.arange(0, 3 * events + 1, 3).to(device), offsets.to(device), labels.to(device)


def main(users=64, steps=20, items=500, lr=2.0, verbose=True):
    model = HistoryModel(items=items)
    ids, bags, offsets, labels = make_histories(users, items, "cuda", 1)
    losses = [model.step(ids, bags, offsets, labels, lr) for _ in range(steps)]
    if verbose:
        print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps over {offsets[-1].item()} events")

    # serving: all but each user's last event are cached, the last one arrives
    _, q, k, v = model.rows(ids, bags)
    bias = model.bias.to(model.dtype)
    want, _ = tbe.tbe_attention_forward(model.attention, q, k, v, offsets, bias)
    last = offsets[1:] - 1
    old = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    old[last] = False
    cache = Cache(model, users, 128)
    cache.append(model, k[old], v[old], offsets - torch.arange(users + 1, device="cuda"))
    cache.append(model, k[last], v[last], torch.arange(users + 1, device="cuda"))
    got = tbe.tbe_attention_decode(model.attention, q[last], cache.k, cache.v, cache.table, cache.lengths, bias)
    error = (got.float() - want[last].float()).abs().max().item()
    for h, check in ((model.bags, tbe.tbe_get_error), (model.attention, tbe.tbe_attention_get_error)):
        if check(h) != tbe.TBE_OK:
            raise RuntimeError("device error")
    if verbose:
        print(f"new events served from the cache: largest difference to the whole histories' pass {error:.2e}")
    model.close()
    return losses, error


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--users", type=int, default=64)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    main(a.users, a.steps)
