"""One round of speculative decoding over a paged fp8 cache, on one GPU:

  1. prompts of text and image patches: queries and keys turned in place by
     three axes (time, height, width; a text token has the same position on all),
     and keys and values written to the cache;
  2. a tree of drafted tokens a request: turned, their keys and values written
     behind the context, and one attention call over the cache;
  3. the accepted branch: its rows read back, the way a program copies them to the
     places they keep.

Run `python examples/tree_decode.py` after building the library.  run() returns
the tensors, for tests.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from place_partial_rope_gb300 import binding  # noqa: E402

HEADS_Q, HEADS_K, DIM, PAGE = 16, 4, 128, 64
SECTIONS, SLICE = (16, 24, 24), (0, 128)  # pairs of each axis, lanes that turn


def prompt_positions(text: int, rows: int, cols: int) -> torch.Tensor:
    """(3, text + rows * cols): text counts up on every axis, a patch stands at
    (the image's time, its row, its column)."""
    t = torch.arange(text).expand(3, text)
    grid = torch.stack(torch.meshgrid(torch.zeros(1, dtype=torch.long), torch.arange(rows), torch.arange(cols),
                                      indexing="ij")).reshape(3, -1) + text
    return torch.cat([t, grid], 1)


def turn(x: torch.Tensor, positions: torch.Tensor) -> None:
    """x (tokens, heads, DIM) in place, positions (3, tokens)."""
    binding.rope_partial_inplace_fwd_axes(x.unsqueeze(0), positions.to(torch.int32).unsqueeze(1).contiguous(),
                                          SECTIONS, *SLICE)


def run(seed: int = 0, dtype: torch.dtype = torch.bfloat16, device: str = "cuda") -> dict:
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g).to(device=device, dtype=dtype)  # noqa: E731
    prompts = [(37, 9, 14), (5, 24, 32)]  # text tokens, then an image of rows x cols patches
    parents = [[-1, 0, 0, 1, 1, 2, 3], [-1, -1, 0, 2, 3]]  # each request's drafted tokens
    places = [prompt_positions(*p) for p in prompts]
    context, drafted = [p.shape[1] for p in places], [len(p) for p in parents]
    lens = [c + n for c, n in zip(context, drafted)]

    # pages of any order: the table says where a request's rows are
    per = [-(-n // PAGE) for n in lens]
    pages = sum(per)
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(per), max(per)), -1, dtype=torch.int32)
    for r, n in enumerate(per):
        table[r, :n] = order[sum(per[:r]):sum(per[:r]) + n]

    def slots(r: int, lo: int, hi: int) -> torch.Tensor:
        at = torch.arange(lo, hi)
        return table[r, at // PAGE].long() * PAGE + at % PAGE

    def cache_side() -> tuple[torch.Tensor, torch.Tensor]:
        rows = torch.zeros((pages, PAGE, HEADS_K, DIM), device=device).to(torch.float8_e4m3fn)
        return rows, torch.zeros((pages, PAGE, HEADS_K), device=device)

    (k, k_scale), (v, v_scale) = cache_side(), cache_side()
    cache = binding.KVCache(k, v, k_scale, v_scale)

    # 1. the prompts (their own attention is a dense pass, not shown)
    keys, values = rand(sum(context), HEADS_K, DIM), rand(sum(context), HEADS_K, DIM)
    raw_keys = keys.clone()
    turn(keys, torch.cat(places, 1).to(device))
    where = torch.cat([slots(r, 0, n) for r, n in enumerate(context)]).to(device)
    binding.rope_partial_cache_write(cache, keys, values, where)

    # 2. the drafted trees: a token's position is its depth behind the context
    depth = []
    for r, tree in enumerate(parents):
        last = int(places[r].max()) + 1
        deep: list[int] = []
        for p in tree:
            deep.append(last if p < 0 else deep[p] + 1)
        depth += deep
    at = torch.tensor(depth).expand(3, -1).to(device)
    q, new_k, new_v = rand(len(depth), HEADS_Q, DIM), rand(len(depth), HEADS_K, DIM), rand(len(depth), HEADS_K, DIM)
    turn(q, at)
    turn(new_k, at)
    fresh = torch.cat([slots(r, context[r], lens[r]) for r in range(len(lens))]).to(device)
    binding.rope_partial_cache_write(cache, new_k, new_v, fresh)
    start = torch.tensor([0] + drafted).cumsum(0).to(torch.int32).to(device)
    words = torch.cat([binding.rope_partial_tree_mask(p) for p in parents]).to(device)
    kv_len = torch.tensor(lens, dtype=torch.int32, device=device)
    out = torch.empty_like(q)
    lse = torch.empty((len(depth), HEADS_Q), device=device)
    workspace = binding.tree_attention_workspace(q, cache, max(drafted))  # kept from round to round
    binding.rope_partial_tree_attention(q, cache, start, kv_len, table.to(device), out, lse=lse, tree=words,
                                        max_q=max(drafted), workspace=workspace)

    # 3. the accepted branch of request 0 (tokens 0, 1, 3): its rows, as numbers
    branch = slots(0, context[0], lens[0])[[0, 1, 3]].to(device)
    kept_k, kept_v = (torch.empty((3, HEADS_K, DIM), dtype=dtype, device=device) for _ in range(2))
    binding.rope_partial_cache_read(cache, branch, kept_k, kept_v)
    return dict(cache=cache, raw_keys=raw_keys, keys=keys, values=values, new_k=new_k, new_v=new_v, q=q, out=out,
                lse=lse, kept_k=kept_k, kept_v=kept_v, positions=torch.cat(places, 1), parents=parents,
                context=context, drafted=drafted)


def main() -> None:
    r = run()
    torch.cuda.synchronize()
    print("out", tuple(r["out"].shape), "log-sum-exp of token 0:", [round(x, 3) for x in r["lse"][0, :4].tolist()])
    print("kept rows", tuple(r["kept_k"].shape))


if __name__ == "__main__":
    main()
