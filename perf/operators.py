"""Cases and plain forms of the rotary operators around an attention cache.

Four operators, in the order in which a decoding step uses them:

  axes   rotary positions with several axes (time, height, width), in place on
         a slice of each head, and its backward;
  write  a rotated key and a value put into a paged cache, quantised to 8 bits
         with one scale per token and head, and read back at the same slots;
  read   rows of such a cache turned back into 16-bit rows;
  tree   attention of a tree of drafted tokens (or of single tokens) over a
         paged cache, 16-bit or 8-bit.

``run`` computes them from elementary torch operations in 32 bits, or, where
``own`` is set, by the calls of ``place_partial_rope_gb300.binding``.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "fp8": torch.float8_e4m3fn, "int8": torch.int8}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1, "int8": 1}
TOP = {"fp8": 448.0, "int8": 127.0}  # the largest value that a stored byte holds
TINY = 2.0 ** -100                   # the least row maximum that a scale is made for


def listed():
    return [
        # a 16 x 16 grid of image patches of a 12-head encoder: the smallest
        # call, where latency counts (the small model's heads)
        dict(name="axes image small", op="axes", dir="fwd", type="bf16", B=1, grid="1x16x16", text=0,
             N=12, D=64, start=0, end=64, sections="0,16,16", mode="interleave", order="blocked",
             spectrum="own"),
        # frames of a video, two clips of 24960 tokens, each axis with its own spectrum
        dict(name="axes video", op="axes", dir="fwd", type="bf16", B=2, grid="16x30x52", text=0,
             N=24, D=128, start=0, end=128, sections="22,21,21", mode="interleave", order="blocked",
             spectrum="own"),
        # a prompt of text with an image inside, training step, half-split
        # pairs dealt to the axes in turn, one spectrum for all of them
        dict(name="axes text and image bwd", op="axes", dir="bwd", type="fp16", B=8, grid="1x32x40",
             text=768, N=16, D=128, start=0, end=128, sections="24,20,20", mode="half",
             order="interleaved", spectrum="shared"),
        # a slice that starts 8 bytes off, odd token count, fp32 gradients
        dict(name="axes unaligned bwd", op="axes", dir="bwd", type="fp32", B=3, grid="5x17x19", text=0,
             N=32, D=128, start=34, end=98, sections="10,11,11", mode="interleave", order="blocked",
             spectrum="shared"),
        # one decoding step: 3 requests with 11 drafted tokens each
        dict(name="write decode", op="write", type="bf16", store="fp8", T=33, H=8, dk=128, dv=128,
             start=0, end=64, mode="half", page=64, pages=128),
        # prompts being processed: 192-wide keys whose first 64 lanes turn, 128-wide values
        dict(name="write prompt", op="write", type="bf16", store="int8", T=16411, H=16, dk=192, dv=128,
             start=0, end=64, mode="interleave", page=64, pages=384),
        # the context of one short request, 64-wide heads
        dict(name="read short", op="read", type="fp16", store="int8", T=777, H=4, dk=64, dv=64,
             page=16, pages=128),
        # the context of several requests, read back for a dense pass
        dict(name="read prompt", op="read", type="bf16", store="fp8", T=65536, H=8, dk=128, dv=128,
             page=64, pages=1280),
        # one request, one token at a time
        dict(name="tree single token", op="tree", type="bf16", store="bf16", R=1, n_lo=1, n_hi=1,
             len_lo=4097, len_hi=4097, Hq=16, Hk=2, dk=128, dv=128, page=64),
        # a batch of requests with small trees over contexts of very different length
        dict(name="tree ragged batch", op="tree", type="bf16", store="fp8", R=48, n_lo=1, n_hi=13,
             len_lo=90, len_hi=12000, Hq=32, Hk=8, dk=128, dv=128, page=64),
        # wide trees at a batch: the most arithmetic per byte
        dict(name="tree wide", op="tree", type="bf16", store="bf16", R=12, n_lo=60, n_hi=64,
             len_lo=6000, len_hi=8200, Hq=32, Hk=8, dk=128, dv=128, page=16),
        # two long streams with one key head for all query heads, 64-wide heads
        dict(name="tree long stream", op="tree", type="fp16", store="int8", R=2, n_lo=24, n_hi=25,
             len_lo=130001, len_hi=131072, Hq=8, Hk=1, dk=64, dv=64, page=128),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "write", "read", "tree", "tree"])
    if op == "axes":
        D = rng.choice([64, 96, 128, 192])
        pairs = rng.choice([p for p in (16, 21, 32, 48, 64) if 2 * p <= D])
        start = rng.choice([0, 0, 2, 3, 8, D - 2 * pairs])
        start = min(start, D - 2 * pairs)
        a = rng.randint(1, pairs // 2)
        b = rng.randint(1, pairs - a - 1)
        grid = "%dx%dx%d" % (_spread(rng, 1, 16), _spread(rng, 4, 40), _spread(rng, 4, 40))
        # fp32 results are held to fp32's bound, so their positions stay those of a grid
        kind = rng.choice(["bf16", "fp16", "fp32"])
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), type=kind, B=rng.randint(1, 2), grid=grid,
                    text=0 if kind == "fp32" else rng.choice([0, _spread(rng, 1, 2000)]),
                    N=_spread(rng, 1, 24), D=D, start=start, end=start + 2 * pairs,
                    sections="%d,%d,%d" % (a, b, pairs - a - b), mode=rng.choice(["interleave", "half"]),
                    order=rng.choice(["blocked", "interleaved"]), spectrum=rng.choice(["own", "shared"]))
    if op in ("write", "read"):
        dk, dv = rng.choice([(64, 64), (128, 128), (192, 128), (96, 96), (80, 80)])
        T, page = _spread(rng, 1, 16000), rng.choice([16, 32, 48, 64, 128])
        c = dict(op=op, type=rng.choice(["bf16", "fp16"]), store=rng.choice(["fp8", "int8"]), T=T,
                 H=_spread(rng, 1, 12), dk=dk, dv=dv, page=page,
                 pages=int(T * rng.uniform(1.1, 1.6)) // page + 2)
        if op == "write":
            pairs = rng.choice([16, 32, dk // 2])
            start = rng.choice([0, 1, 2, 16, dk - 2 * pairs])
            start = min(start, dk - 2 * pairs)
            c.update(start=start, end=start + 2 * pairs, mode=rng.choice(["interleave", "half"]))
        return c
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    n_hi = _spread(rng, 1, 64)
    R = _spread(rng, 1, 64)
    # at most about what the widest listed tree computes
    room = min(60000.0, 1.2e9 / (R * n_hi * Hk * G * (dk + dv) / 2), 6e8 / (R * Hk * (dk + dv)))
    len_hi = n_hi + _spread(rng, 1, max(2, int(room)))
    kind = rng.choice(["bf16", "fp16"])
    return dict(op=op, type=kind, store=rng.choice([kind, "fp8", "int8"]), R=R, n_lo=rng.randint(1, n_hi),
                n_hi=n_hi, len_lo=n_hi + rng.randint(0, len_hi - n_hi), len_hi=len_hi, Hq=Hk * G, Hk=Hk,
                dk=dk, dv=dv, page=rng.choice([16, 32, 48, 64, 128]))


def _requests(c):
    """Drafted tokens and cache lengths of the requests of a tree case (the
    cache length counts the drafted tokens, which are its last rows)."""
    R = c["R"]
    n = [c["n_lo"] + (r * 7919) % (c["n_hi"] - c["n_lo"] + 1) for r in range(R)]
    ln = [c["len_hi"] - (c["len_hi"] - c["len_lo"]) * r // max(1, R - 1) for r in range(R)]
    return n, ln


def _sections(c):
    return [int(v) for v in c["sections"].split(",")]


def _tokens(c):
    t, h, w = (int(v) for v in c["grid"].split("x"))
    return t * h * w + c["text"]


def work(c):
    e = SIZE[c["type"]]
    if c["op"] == "axes":
        rows, L = c["B"] * _tokens(c) * c["N"], c["end"] - c["start"]
        return {"bytes": rows * L * e * 2 + 3 * c["B"] * _tokens(c) * 4, "flops": rows * L * 3}
    if c["op"] in ("write", "read"):
        rows, d = c["T"] * c["H"], c["dk"] + c["dv"]
        stored = rows * (d * SIZE[c["store"]] + 8) + c["T"] * 8
        if c["op"] == "read":
            return {"bytes": stored + rows * d * e, "flops": rows * d}
        L = c["end"] - c["start"]
        # read and stored, then read again and turned back
        return {"bytes": rows * d * e * 2 + 2 * stored + c["T"] * 2 * L * e, "flops": rows * (3 * d + 3 * L)}
    n, ln = _requests(c)
    kv = sum(ln) * c["Hk"] * ((c["dk"] + c["dv"]) * SIZE[c["store"]] + (8 if c["store"] in TOP else 0))
    qo = sum(n) * c["Hq"] * ((c["dk"] + c["dv"]) * e + 4)
    return {"bytes": kv + qo + sum(-(-v // c["page"]) for v in ln) * 4,
            "flops": 2 * c["Hq"] * (c["dk"] + c["dv"]) * sum(a * b for a, b in zip(n, ln))}


# ---------------------------------------------------------------- inputs


def _grid_positions(c):
    """(3, 1, S) positions: text counts up on all axes, then a grid of
    (time, height, width) starts where the text ends."""
    t, h, w = (int(v) for v in c["grid"].split("x"))
    g = np.stack(np.meshgrid(np.arange(t), np.arange(h), np.arange(w), indexing="ij")).reshape(3, -1)
    text = np.broadcast_to(np.arange(c["text"]), (3, c["text"]))
    return np.concatenate([text, g + c["text"]], axis=1)[:, None, :].astype(np.int32)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    kind = TYPES[c["type"]]

    def normal(*shape, like=kind):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(like)

    s = {"c": c}
    if c["op"] == "axes":
        pos = np.repeat(_grid_positions(c), c["B"], axis=1)
        if c["text"]:  # prompts that go on from an earlier turn
            pos = pos + rng.integers(0, 4000, size=(1, c["B"], 1)).astype(np.int32)
        s["x"] = normal(c["B"], _tokens(c), c["N"], c["D"])
        s["positions"] = torch.from_numpy(np.ascontiguousarray(pos)).to(DEV)
        return s

    if c["op"] in ("write", "read"):
        T, H, pages, page = c["T"], c["H"], c["pages"], c["page"]
        # whole pages in any order, as an allocator hands them out
        order = torch.randperm(pages, generator=g, device=DEV)
        s["slots"] = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:T].contiguous()
    else:
        n, ln = _requests(c)
        mix = rng.permutation(c["R"])
        n, ln = [n[i] for i in mix], [ln[i] for i in mix]
        H, page = c["Hk"], c["page"]
        per = [-(-v // page) for v in ln]
        pages = sum(per) + 3
        order = rng.permutation(pages)
        table = np.zeros((c["R"], max(per)), np.int32)
        at, bits, at_q = 0, np.zeros(sum(n), np.int64), 0
        for r in range(c["R"]):
            table[r, :per[r]] = order[at:at + per[r]]
            at += per[r]
            for i in range(n[r]):  # a random tree: each token hangs on an earlier one or on the context
                up = int(rng.integers(-1, i)) if i else -1
                seen = (int(bits[at_q + up]) & (2 ** 64 - 1) if up >= 0 else 0) | 1 << i
                bits[at_q + i] = np.array(seen, np.uint64).view(np.int64)
            at_q += n[r]
        s["q"] = normal(sum(n), c["Hq"], c["dk"])
        s["q_start"] = torch.tensor([sum(n[:r]) for r in range(c["R"] + 1)], dtype=torch.int32, device=DEV)
        s["kv_len"] = torch.tensor(ln, dtype=torch.int32, device=DEV)
        s["table"] = torch.from_numpy(table).to(DEV)
        s["tree"] = torch.from_numpy(bits[:, None]).to(DEV)
        s["out"] = torch.empty(sum(n), c["Hq"], c["dv"], dtype=kind, device=DEV)
        s["lse"] = torch.empty(sum(n), c["Hq"], dtype=torch.float32, device=DEV)

    # the cache: rows that were written before, with scales like those of unit rows
    for name, d in (("k", c["dk"]), ("v", c["dv"])):
        shape = (pages, page, H, d)
        if c["store"] == "int8":
            s["c" + name] = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
        elif c["store"] == "fp8":
            s["c" + name] = torch.empty(shape, dtype=TYPES["fp8"], device=DEV)
            s["c" + name].copy_((normal(*shape, like=torch.float16) * 120).clamp_(-448, 448))
        else:
            s["c" + name] = normal(*shape)
        s[name + "s"] = None
        if c["store"] in TOP:
            u = torch.rand(shape[:3], generator=g, device=DEV, dtype=torch.float32)
            s[name + "s"] = (2.0 + 2.0 * u) / TOP[c["store"]]
    if c["op"] == "write":
        s["k"], s["v"] = normal(c["T"], c["H"], c["dk"]), normal(c["T"], c["H"], c["dv"])
        half = (c["end"] - c["start"]) // 2
        w = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        a = torch.randint(0, 32768, (c["T"], 1), generator=g, device=DEV) * w
        a = torch.cat([a, a], -1) if c["mode"] == "half" else a.repeat_interleave(2, -1)
        s["cos"], s["sin"] = a.cos().to(kind), a.sin().to(kind)
    if c["op"] in ("write", "read"):
        s["ko"] = torch.empty(c["T"], c["H"], c["dk"], dtype=kind, device=DEV)
        s["vo"] = torch.empty(c["T"], c["H"], c["dv"], dtype=kind, device=DEV)
    if own:
        # what a serving program makes once for its cache and keeps: the
        # cache's handle and the attention's workspace
        from place_partial_rope_gb300 import binding
        s["cache"] = binding.KVCache(s["ck"], s["cv"], s["ks"], s["vs"])
        if c["op"] == "tree":
            s["workspace"] = binding.tree_attention_workspace(s["q"], s["cache"], c["n_hi"])
    return s


# ---------------------------------------------------------------- plain forms


def _axis_of_pair(c):
    """The axis and the exponent (of 1 / base) of each pair."""
    sec = _sections(c)
    pairs = sum(sec)
    if c["order"] == "blocked":
        axis = [a for a, m in enumerate(sec) for _ in range(m)]
    else:
        axis = [a for i in range(max(sec)) for a, m in enumerate(sec) if i < m]
    if c["spectrum"] == "shared":
        power = [k / pairs for k in range(pairs)]
    else:
        power = [sum(x == axis[k] for x in axis[:k]) / sec[axis[k]] for k in range(pairs)]
    return axis, power


def _split(x, mode):
    return (x[..., 0::2], x[..., 1::2]) if mode == "interleave" else x.chunk(2, -1)


def _join(a, b, mode):
    return torch.stack([a, b], -1).flatten(-2) if mode == "interleave" else torch.cat([a, b], -1)


def _axes(s):
    c = s["c"]
    axis, power = _axis_of_pair(c)
    axis = torch.tensor(axis, device=DEV)
    w = 10000.0 ** -torch.tensor(power, dtype=torch.float32, device=DEV)
    angle = s["positions"].float()[axis].permute(1, 2, 0) * w
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]
    if c["dir"] == "bwd":
        sin = -sin
    at = s["x"][..., c["start"]:c["end"]]
    a, b = _split(at.float(), c["mode"])
    at.copy_(_join(a * cos - b * sin, b * cos + a * sin, c["mode"]))
    return s["x"]


def _rows(flat, slots):
    """Rows of a flat cache, as numbers in 32 bits."""
    if flat.dtype == TYPES["fp8"]:
        return flat.view(torch.uint8)[slots].view(TYPES["fp8"]).float()
    return flat[slots].float()


def _read(s, slots):
    got = []
    for name in ("k", "v"):
        x = _rows(s["c" + name].flatten(0, 1), slots)
        if s[name + "s"] is not None:
            x = x * s[name + "s"].flatten(0, 1)[slots][..., None]
        got.append(x)
    return got


def _write(s):
    c = s["c"]
    for name in ("k", "v"):
        x = s[name].float()
        if name == "k":
            cos, sin = (_split(s[t].float()[:, None], c["mode"]) for t in ("cos", "sin"))
            a, b = _split(x[..., c["start"]:c["end"]], c["mode"])
            turned = _join(a * cos[0] - b * sin[0], b * cos[1] + a * sin[1], c["mode"])
            x = torch.cat([x[..., :c["start"]], turned, x[..., c["end"]:]], -1)
        most = x.abs().amax(-1).clamp_min(TINY)
        y = x * (TOP[c["store"]] / most)[..., None]
        if c["store"] == "int8":
            y = y.round()
        y = y.clamp(-TOP[c["store"]], TOP[c["store"]]).to(TYPES[c["store"]])
        s["c" + name].flatten(0, 1).view(torch.uint8)[s["slots"]] = y.view(torch.uint8)
        s[name + "s"].flatten(0, 1)[s["slots"]] = most / TOP[c["store"]]


def _tree(s):
    c = s["c"]
    R, most, page = c["R"], c["len_hi"], c["page"]
    j = torch.arange(most, device=DEV)
    slots = s["table"].long()[:, j // page] * page + j % page
    k, v = _read(s, slots)                                             # R, most, Hk, d
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(c["n_hi"], device=DEV)
    at = (s["q_start"][:-1].long()[:, None] + i).clamp_max(s["q"].shape[0] - 1)
    G = c["Hq"] // c["Hk"]
    q = s["q"][at].float().unflatten(2, (c["Hk"], G))                  # R, n, Hk, G, d
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = q @ k.permute(0, 2, 3, 1) * (1.0 / math.sqrt(c["dk"]))     # R, Hk, n * G, most
    draft = j - (s["kv_len"].long() - n)[:, None]                      # R, most
    bit = s["tree"][at][:, :, 0, None] >> draft.clamp(0, 63)[:, None] & 1
    seen = (draft < 0)[:, None] | ((bit == 1) & (j < s["kv_len"][:, None])[:, None])
    score = score.unflatten(2, (c["n_hi"], G)).masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.permute(0, 2, 1, 3)) / total
    lse = (top + total.log())[..., 0]
    o = o.unflatten(2, (c["n_hi"], G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.unflatten(2, (c["n_hi"], G)).permute(0, 2, 1, 3).flatten(2, 3)
    kept = i < n[:, None]
    return {"out": o[kept].to(s["q"].dtype), "lse": lse[kept]}


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["c"]
    if own:
        from place_partial_rope_gb300 import binding
        if c["op"] == "axes":
            call = (binding.rope_partial_inplace_fwd_axes if c["dir"] == "fwd"
                    else binding.rope_partial_inplace_bwd_axes)
            call(s["x"], s["positions"], _sections(c), c["start"], c["end"], mode=c["mode"],
                 order=c["order"], spectrum=c["spectrum"])
            return s["x"]
        if c["op"] == "tree":
            binding.rope_partial_tree_attention(s["q"], s["cache"], s["q_start"], s["kv_len"], s["table"],
                                                s["out"], lse=s["lse"], tree=s["tree"], max_q=c["n_hi"],
                                                workspace=s["workspace"])
            return {"out": s["out"], "lse": s["lse"]}
        if c["op"] == "write":
            binding.rope_partial_cache_write(s["cache"], s["k"], s["v"], s["slots"], s["cos"], s["sin"],
                                             c["start"], c["end"], c["mode"])
        binding.rope_partial_cache_read(s["cache"], s["slots"], s["ko"], s["vo"])
        k, v = s["ko"], s["vo"]
    elif c["op"] == "axes":
        return _axes(s)
    elif c["op"] == "tree":
        return _tree(s)
    else:
        if c["op"] == "write":
            _write(s)
        k, v = (x.to(TYPES[c["type"]]) for x in _read(s, s["slots"]))
    return {"k": k, "v": v, "k_scale": s["ks"], "v_scale": s["vs"]} if c["op"] == "write" else {"k": k, "v": v}


# ---------------------------------------------------------------- 64 bits


def _to_grid(v, store):
    """The nearest value that a byte holds, ties to even."""
    if store == "int8":
        return v.round().clamp(-127, 127)
    e = torch.frexp(v)[1].clamp_min(-5) - 4  # 3 bits after the leading one, from 2^-6 up
    step = torch.ldexp(torch.ones_like(v), e)
    return ((v / step).round() * step).clamp(-448, 448)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "axes":
        sec, L = _sections(c), c["end"] - c["start"]
        x, pos = s["x"].double(), s["positions"].double()
        left, dealt, turn = list(sec), [], 0
        while len(dealt) < L // 2:  # pairs one by one, to the axis whose turn it is
            a = turn % len(sec) if c["order"] == "interleaved" else next(i for i, m in enumerate(left) if m)
            turn += 1
            if left[a]:
                j = sec[a] - left[a]
                left[a] -= 1
                dealt.append((a, 10000.0 ** (-(2.0 * len(dealt) / L) if c["spectrum"] == "shared"
                                             else -(j / sec[a]))))
        y = x.clone()
        for k, (a, w) in enumerate(dealt):
            m = c["start"] + (2 * k if c["mode"] == "interleave" else k)
            n = m + (1 if c["mode"] == "interleave" else L // 2)
            t = (pos[a] * w)[..., None] * (1 if c["dir"] == "fwd" else -1)
            y[..., m] = x[..., m] * t.cos() - x[..., n] * t.sin()
            y[..., n] = x[..., m] * t.sin() + x[..., n] * t.cos()
        return y
    if c["op"] == "write":
        got = {}
        for name in ("k", "v"):
            x = s[name].double()
            if name == "k":
                y = x[..., c["start"]:c["end"]].clone()
                half = y.shape[-1] // 2
                for j in range(half):
                    m, n = (2 * j, 2 * j + 1) if c["mode"] == "interleave" else (j, j + half)
                    u, w = x[..., c["start"] + m], x[..., c["start"] + n]
                    co, si = s["cos"].double(), s["sin"].double()
                    y[..., m] = u * co[:, m, None] - w * si[:, m, None]
                    y[..., n] = w * co[:, n, None] + u * si[:, n, None]
                x[..., c["start"]:c["end"]] = y
            scale = x.abs().amax(-1).clamp_min(TINY) / TOP[c["store"]]
            got[name] = _to_grid(x / scale[..., None], c["store"]) * scale[..., None]
            whole = s[name + "s"].double().flatten(0, 1)
            whole[s["slots"]] = scale
            got[name + "_scale"] = whole.view(s[name + "s"].shape)
        return {"k": got["k"], "v": got["v"], "k_scale": got["k_scale"], "v_scale": got["v_scale"]}
    page = c["page"]
    flat = {}
    for name in ("k", "v"):
        def rows(slots, name=name):
            x = s["c" + name].view(torch.uint8) if c["store"] == "fp8" else s["c" + name]
            x = x.flatten(0, 1)[slots]
            x = x.view(TYPES["fp8"]).float().double() if c["store"] == "fp8" else x.double()
            return x if s[name + "s"] is None else x * s[name + "s"].flatten(0, 1)[slots].double()[..., None]
        flat[name] = rows
    if c["op"] == "read":
        return {"k": flat["k"](s["slots"]), "v": flat["v"](s["slots"])}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    starts, lens, trees = s["q_start"].tolist(), s["kv_len"].tolist(), s["tree"][:, 0].tolist()
    G = c["Hq"] // c["Hk"]
    for r in range(c["R"]):
        lo, hi, m = starts[r], starts[r + 1], lens[r]
        where = torch.arange(m, device=DEV)
        slots = s["table"][r].long()[where // page] * page + where % page
        k, v = flat["k"](slots), flat["v"](slots)
        seen = torch.ones(hi - lo, m, dtype=torch.bool)
        for i in range(hi - lo):
            for j in range(hi - lo):
                seen[i, m - (hi - lo) + j] = bool(trees[lo + i] >> j & 1)
        seen = seen.to(DEV)
        for h in range(c["Hq"]):
            z = s["q"][lo:hi, h].double() @ k[:, h // G].T / math.sqrt(c["dk"])
            z = torch.where(seen, z, -math.inf)
            lse[lo:hi, h] = torch.logsumexp(z, -1)
            out[lo:hi, h] = torch.exp(z - lse[lo:hi, h, None]) @ v[:, h // G]
    return {"out": out, "lse": lse}
