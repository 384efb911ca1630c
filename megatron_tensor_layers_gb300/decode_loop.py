"""A beam-search decode loop over the library's operators, on one GPU.

A small random model (pre-norm blocks of attention and gated MLP, no position
encoding) cut into t tensor-parallel shards generates from ragged prompts: every
step is the merged QKV projection, the append to the paged 4-bit cache, attention
over it, o_proj with the residual and norm of the sequence-parallel reduce, the MLP,
the vocab-sharded LM head, beam selection over the shards, and the fork that gives
each surviving beam its parent's pages.  Nothing of a step waits for the host.

    python -m megatron_tensor_layers_gb300.decode_loop
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

import megatron_tensor_layers_gb300 as tp
from megatron_tensor_layers_gb300 import synth


@dataclass
class Config:
    t: int = 2
    layers: int = 2
    hidden: int = 1024
    heads: int = 16
    kv_heads: int = 4
    head_dim: int = 64
    ffn: int = 2048
    vocab: int = 1000
    page_size: int = 16
    window: int = 0
    sinks: int = 0
    eos: int = 0


class Model:
    """Random weights in the layouts the entry points take, one list of t shards each."""

    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        self.cfg = c = cfg
        t, h, hd = c.t, c.hidden, c.head_dim
        make = lambda i, *shape, std=0.03: synth.normal_bf16(shape, std, seed + i, device=device)  # noqa: E731
        per_shard = (c.heads + 2 * c.kv_heads) // t * hd
        self.layers = []
        for n in range(c.layers):
            k = 100 * n + 10
            self.layers.append(dict(
                qkv=[make(k + r, per_shard, h) for r in range(t)],
                o=[make(k + 20 + r, h, c.heads // t * hd) for r in range(t)],
                gate_up=[make(k + 40 + r, 2 * c.ffn // t, h) for r in range(t)],
                down=[make(k + 60 + r, h, c.ffn // t) for r in range(t)],
                norm1=torch.ones(h, dtype=torch.bfloat16, device=device),
                norm2=torch.ones(h, dtype=torch.bfloat16, device=device)))
        per = -(-c.vocab // t)
        self.table = [make(r, max(0, min((r + 1) * per, c.vocab) - r * per), h, std=0.05) for r in range(t)]
        self.norm = torch.ones(h, dtype=torch.bfloat16, device=device)


class Cache:
    """Every layer's pools, and the page table of the running sequences."""

    def __init__(self, cfg: Config, pages: int, max_blocks: int, device="cuda"):
        self.cfg = cfg
        self.pools = [tp.tp_kv4_pool(pages, cfg.page_size, cfg.kv_heads // cfg.t, cfg.head_dim, layers=cfg.layers,
                                     device=device) for _ in range(cfg.t)]
        self.table = torch.full((0, max_blocks), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(0, dtype=torch.int32, device=device)
        self.info: Optional[torch.Tensor] = None

    def start(self, lengths: torch.Tensor) -> None:
        """Empty sequences, grown by their prompts' lengths."""
        n = lengths.numel()
        self.table = torch.full((n, self.table.shape[1]), -1, dtype=torch.int32, device=lengths.device)
        self.lens = torch.zeros(n, dtype=torch.int32, device=lengths.device)
        self.fork(torch.arange(n, dtype=torch.int32, device=lengths.device), lengths)

    def fork(self, parents: torch.Tensor, grow) -> None:
        """Row i becomes a continuation of row parents[i]; the pages nobody keeps are dealt out again."""
        self.table, self.lens, _, self.info = tp.tp_kv_fork(self.table, self.lens, parents, self.pools, grow=grow)

    def compact(self) -> None:
        self.table, _, self.info = tp.tp_kv_compact(self.table, self.lens, self.pools)


def forward(model: Model, cache: Cache, ids: torch.Tensor, cu_rows: Optional[torch.Tensor] = None,
            last: Optional[torch.Tensor] = None) -> List[torch.Tensor]:
    """Logits, as vocab shards, of the rows `ids` (the last tokens of the cache's sequences), or of the
    rows `last` among them."""
    c = model.cfg
    q_cols, kv_cols = c.heads // c.t * c.head_dim, c.kv_heads // c.t * c.head_dim
    x = tp.vocab_parallel_embed(ids, model.table, c.vocab)
    residual = torch.empty_like(x)
    partials: Sequence[torch.Tensor] = [x]
    first = True
    for n, w in enumerate(model.layers):
        # residual += what the last block gave; norm
        _, y = tp.tp_reduce_scatter_rmsnorm(partials, w["norm1"], residual=None if first else residual, residual_out=residual)
        first = False
        qkv = tp.tp_linear_col(y, w["qkv"])
        layer = [p[n] for p in cache.pools]
        tp.tp_kv4_append([s[:, q_cols:q_cols + kv_cols] for s in qkv], [s[:, q_cols + kv_cols:] for s in qkv], layer,
                         cache.table, cache.lens, cu_rows=cu_rows)
        heads = tp.tp_kv4_attention([s[:, :q_cols] for s in qkv], layer, cache.table, cache.lens, cu_rows=cu_rows,
                                    window=c.window, sinks=c.sinks)
        o = tp.tp_linear_row(heads, w["o"], reduce_results=False)
        _, y = tp.tp_reduce_scatter_rmsnorm(o, w["norm2"], residual=residual, residual_out=residual)
        partials = [tp.tp_mlp_forward(y, w["gate_up"], w["down"])]
    _, y = tp.tp_reduce_scatter_rmsnorm(partials, model.norm, residual=residual, residual_out=residual)
    if last is not None:
        y = y[last]
    return tp.lm_head_sharded(y, model.table, c.vocab, per_shard=True, out_dtype=torch.float32)


@torch.no_grad()
def generate(model: Model, prompts: Sequence[torch.Tensor], beams: int, steps: int, *, pages: int = 0,
             compact_every: int = 0):
    """Beam search from ragged prompts (1-D int32 CUDA tensors, a token each at least): (tokens [items, beams,
    steps], scores [items, beams]), best first."""
    c = model.cfg
    if not prompts or any(p.dim() != 1 or p.numel() < 1 or p.dtype != torch.int32 for p in prompts):
        raise ValueError("prompts must hold 1-D int32 tensors of a token each at least")
    if steps < 1 or beams < 1:
        raise ValueError("steps and beams must be 1 or more")
    dev, items = prompts[0].device, len(prompts)
    lengths = [int(p.numel()) for p in prompts]
    blocks = -(-(max(lengths) + steps + 1) // c.page_size)
    cache = Cache(c, pages or items * beams * blocks + items, blocks, dev)
    cache.start(torch.tensor(lengths, dtype=torch.int32, device=dev))
    ends = torch.tensor(lengths, device=dev).cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    logits = forward(model, cache, torch.cat(list(prompts)), cu_rows=cu, last=ends - 1)
    scores = torch.zeros((items, 1), device=dev)
    finished = None
    history = torch.zeros((items, 0), dtype=torch.int64, device=dev)
    for step in range(steps):
        scores, rows, tokens = tp.tp_beam_select(logits, scores, beams, finished=finished, eos=c.eos)
        parents = rows.flatten()
        keep = parents.clamp(min=0).long()
        history = torch.cat([history[keep], tokens.flatten()[:, None].long()], 1)
        finished = tokens == c.eos
        if step + 1 == steps:
            break
        cache.fork(parents, 1)
        if compact_every and step % compact_every == compact_every - 1:
            cache.compact()
        logits = forward(model, cache, tokens.flatten().clamp(min=0))
    if tp.tp_device_status() != 0:
        raise RuntimeError("a page table entry was out of range, or a wait ran out")
    return history.view(items, beams, -1), scores


def main() -> None:
    model = Model(Config())
    prompts = [synth.uniform_ids(n, model.cfg.vocab, 50 + n, device="cuda") for n in (5, 33, 130)]
    tokens, scores = generate(model, prompts, beams=4, steps=12, compact_every=4)
    for i in range(len(prompts)):
        print(f"prompt of {prompts[i].numel()} tokens: best beam {tokens[i, 0].tolist()} at {scores[i, 0].item():.3f}")


if __name__ == "__main__":
    main()
