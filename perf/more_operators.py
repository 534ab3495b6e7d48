"""Cases and plain forms of the operators on either side of the paged cache.

Three families, in the order in which a model meets them:

  norm    root-mean-square norm of each query and key row and the rotation of a
          slice of it, in one pass, forward (serving and training) and backward
          with the gradients of the weights; the norm may cover a part of the
          row only (a latent row: its first lanes normed, its last ones turned);
  pages   a batch's new tokens given pages of the cache on the GPU (slots,
          positions, offsets, page table), and pages given back;
  latent  attention of drafted tokens over a paged cache of latent rows: one row a
          token for all heads, whose first lanes are also the value.

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
EPS = 1e-6


def listed():
    return [
        # a decoding step of 64 requests: rows of a fused projection, the smallest call
        dict(name="norm decode", op="norm", dir="fwd", type="bf16", weight="bf16", B=64, S=1, Nq=32, Nk=8,
             D=128, n0=0, n1=128, start=0, end=128, mode="half", fused=True, keep=False),
        # two prompts of 8192 tokens
        dict(name="norm prompt", op="norm", dir="fwd", type="bf16", weight="bf16", B=2, S=8192, Nq=32, Nk=8,
             D=128, n0=0, n1=128, start=0, end=64, mode="interleave", fused=True, keep=False),
        # the latent rows of a prompt on their way to the cache: 512 lanes normed, 64 turned
        dict(name="norm latent", op="norm", dir="fwd", type="bf16", weight="fp32", B=1, S=16411, Nq=1, Nk=0,
             D=576, n0=0, n1=512, start=512, end=576, mode="interleave", fused=False, keep=False),
        # a training step's backward pass, half-split pairs over the whole head
        dict(name="norm train bwd", op="norm", dir="bwd", type="bf16", weight="fp32", B=8, S=2048, Nq=16, Nk=4,
             D=128, n0=0, n1=128, start=0, end=128, mode="half", fused=False, keep=True),
        # fp32 gradients, a slice that starts 8 bytes off, as many keys as queries
        dict(name="norm unaligned bwd", op="norm", dir="bwd", type="fp32", weight="fp32", B=3, S=1615, Nq=12,
             Nk=12, D=128, n0=0, n1=128, start=34, end=98, mode="interleave", fused=False, keep=True),
        # a decoding step of 256 requests with up to 4 drafted tokens each
        dict(name="pages decode", op="pages", R=256, n_lo=1, n_hi=4, len_hi=12000, page=64, spare=300),
        # many prompts brought in at once
        dict(name="pages prompts", op="pages", R=512, n_lo=1, n_hi=2000, len_hi=8000, page=16, spare=40000),
        # one request, one token, a sixteenth of the heads: where latency counts
        dict(name="latent single token", op="latent", type="bf16", store="bf16", R=1, n_lo=1, n_hi=1,
             len_lo=4097, len_hi=4097, H=16, dk=576, dv=512, page=64, tree=False),
        # a serving batch over contexts of very different length, all 128 heads
        dict(name="latent ragged batch", op="latent", type="bf16", store="bf16", R=64, n_lo=1, n_hi=1,
             len_lo=90, len_hi=12000, H=128, dk=576, dv=512, page=64, tree=False),
        # small trees of drafted tokens over an 8-bit cache, heads shared out over cards
        dict(name="latent drafted", op="latent", type="bf16", store="fp8", R=32, n_lo=1, n_hi=7,
             len_lo=6000, len_hi=8200, H=32, dk=576, dv=512, page=64, tree=True),
        # two long contexts
        dict(name="latent long", op="latent", type="fp16", store="int8", R=2, n_lo=2, n_hi=2,
             len_lo=130001, len_hi=131072, H=16, dk=576, dv=512, page=128, tree=False),
        # chunks of prompts against their own earlier rows: the most arithmetic per byte
        dict(name="latent chunk", op="latent", type="fp16", store="fp16", R=3, n_lo=200, n_hi=256,
             len_lo=1031, len_hi=4099, H=64, dk=576, dv=512, page=16, tree=False),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pages", "latent", "latent"])
    if op == "norm":
        D = rng.choice([64, 72, 96, 128, 128, 192, 256, 576])
        n0, n1 = rng.choice([(0, D), (0, D), (0, D - D // 4), (D // 8, D)])
        pairs = rng.choice([p for p in (8, 16, 21, 32, 48, 64) if 2 * p <= D])
        start = min(rng.choice([0, 0, 2, 3, 8, D - 2 * pairs]), D - 2 * pairs)
        kind = rng.choice(["bf16", "fp16", "fp32"])
        Nq, Nk = _spread(rng, 1, 32), rng.choice([0, _spread(rng, 1, 12)])
        room = 8192 * 128 * 32 // (D * (Nq + Nk))
        B = _spread(rng, 1, 16)
        back = rng.choice([False, True])
        return dict(op=op, dir="bwd" if back else "fwd", type=kind, weight=rng.choice([kind, "fp32"]), B=B,
                    S=_spread(rng, 1, max(1, min(8192, room // B))), Nq=Nq, Nk=Nk, D=D, n0=n0, n1=n1,
                    start=start, end=start + 2 * pairs, mode=rng.choice(["interleave", "half"]),
                    fused=rng.choice([False, True]), keep=back or rng.choice([False, True]))
    if op == "pages":
        page = rng.choice([1, 16, 24, 64, 128])
        n_hi = _spread(rng, 1, 2000)
        R = _spread(rng, 1, min(4096, 500000 // n_hi))
        len_hi = _spread(rng, 1, min(40000, 4000000 * page // (R * 4)))
        return dict(op=op, R=R, n_lo=rng.randint(0, n_hi), n_hi=n_hi, len_hi=len_hi, page=page,
                    spare=rng.choice([R * (n_hi // page + 1), R * (n_hi // page + 1) // 3]))
    dk, dv = rng.choice([(576, 512), (576, 512), (576, 512), (288, 256), (192, 128), (320, 320)])
    H = rng.choice([1, 4, 8, 16, 20, 32, 64, 128])
    R = _spread(rng, 1, 64)
    n_hi = _spread(rng, 1, 48)
    # no more work than the largest listed cases have
    room = min(60000.0, 1.2e11 / (R * n_hi * H * (dk + dv)), 2.5e8 / (R * dk))
    len_hi = n_hi + _spread(rng, 1, max(2, int(room)))
    kind = rng.choice(["bf16", "fp16"])
    return dict(op=op, type=kind, store=rng.choice([kind, kind, "fp8", "int8"]), R=R,
                n_lo=rng.randint(1, n_hi), n_hi=n_hi, len_lo=n_hi + rng.randint(0, len_hi - n_hi),
                len_hi=len_hi, H=H, dk=dk, dv=dv, page=rng.choice([1, 16, 24, 64, 128]),
                tree=rng.choice([False, True]))


def _requests(c):
    """Drafted tokens and cache lengths of the requests of a latent case (the
    cache length counts the drafted tokens, which are its last rows)."""
    R = c["R"]
    n = [c["n_lo"] + (r * 7919) % (c["n_hi"] - c["n_lo"] + 1) for r in range(R)]
    ln = [c["len_hi"] - (c["len_hi"] - c["len_lo"]) * r // max(1, R - 1) for r in range(R)]
    return n, ln


def _batch(c):
    """New tokens and cached lengths of the requests of a pages case."""
    R = c["R"]
    n = [c["n_lo"] + (r * 7919) % (c["n_hi"] - c["n_lo"] + 1) for r in range(R)]
    ln = [(r * 104729 + 17) % (c["len_hi"] + 1) for r in range(R)]
    return n, ln


def work(c):
    if c["op"] == "norm":
        e, rows, D = SIZE[c["type"]], c["B"] * c["S"] * (c["Nq"] + c["Nk"]), c["D"]
        small = c["S"] * (c["end"] - c["start"]) * 2 * e + (2 if c["Nk"] else 1) * (c["n1"] - c["n0"]) * SIZE[c["weight"]]
        back = c["dir"] == "bwd"
        if back:
            small += (2 if c["Nk"] else 1) * (c["n1"] - c["n0"]) * 4
        return {"bytes": rows * D * e * (3 if back else 2) + (rows * 4 if c["keep"] else 0) + small,
                "flops": rows * ((c["n1"] - c["n0"]) * (9 if back else 4) + (c["end"] - c["start"]) * 3)}
    if c["op"] == "pages":
        n, ln = _batch(c)
        T, R, page = sum(n), c["R"], c["page"]
        # lengths and counts, offsets, slots and positions, the table's rows that slots
        # come from, and the pages that go over and back
        moved = sum(-(-(a + b) // page) - -(-b // page) for a, b in zip(n, ln))
        return {"bytes": R * 4 * 8 + T * 12 + min(moved, c["spare"]) * 4 * 6, "flops": T * 4}
    e = SIZE[c["type"]]
    n, ln = _requests(c)
    kv = sum(ln) * (c["dk"] * SIZE[c["store"]] + (4 if c["store"] in TOP else 0))
    qo = sum(n) * c["H"] * ((c["dk"] + c["dv"]) * e + 4)
    return {"bytes": kv + qo + sum(-(-v // c["page"]) for v in ln) * 4,
            "flops": 2 * c["H"] * (c["dk"] + c["dv"]) * sum(a * b for a, b in zip(n, ln))}


# ---------------------------------------------------------------- inputs


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, like):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(like)

    s = {"c": c}
    if c["op"] == "norm":
        kind, B, S, D = TYPES[c["type"]], c["B"], c["S"], c["D"]
        wide = c["n1"] - c["n0"]
        heads = [("q", c["Nq"])] + ([("k", c["Nk"])] if c["Nk"] else [])
        if c["fused"]:  # views of one projection's rows, with the values' heads behind them
            whole = normal(B, S, (c["Nq"] + 2 * c["Nk"]) * D, like=kind)
        at = 0
        for name, N in heads:
            if c["fused"]:
                s[name] = whole[..., at:at + N * D].unflatten(-1, (N, D))
                at += N * D
            else:
                s[name] = normal(B, S, N, D, like=kind)
            s[name + "w"] = (1.0 + 0.25 * normal(wide, like=torch.float32)).to(TYPES[c["weight"]])
            s[name + "_out"] = torch.empty(B, S, N, D, dtype=kind, device=DEV)
            if c["keep"]:
                s[name + "r"] = torch.empty(B, S, N, dtype=torch.float32, device=DEV)
            if c["dir"] == "bwd":
                s["d" + name] = normal(B, S, N, D, like=kind)
                x = s[name][..., c["n0"]:c["n1"]].float()  # what the forward pass kept
                s[name + "r"].copy_((x.square().mean(-1) + EPS).rsqrt())
                s["d" + name + "w"] = torch.empty(wide, dtype=torch.float32, device=DEV)
        half = (c["end"] - c["start"]) // 2
        w = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        if S == 1:  # requests that are at positions of their own
            a = torch.randint(0, 32768, (B, 1, 1, 1), generator=g, device=DEV) * w
        else:
            a = (torch.arange(S, device=DEV)[None, :, None, None] + int(rng.integers(0, 4000))) * w
        a = torch.cat([a, a], -1) if c["mode"] == "half" else a.repeat_interleave(2, -1)
        s["cos"], s["sin"] = a.cos().to(kind), a.sin().to(kind)
        if own and c["dir"] == "bwd":
            # what a training program makes once and keeps
            from place_partial_rope_gb300 import binding
            s["workspace"] = binding.norm_workspace(s["q"], s.get("k"), norm=(c["n0"], c["n1"]))
        return s

    if c["op"] == "pages":
        n, ln = _batch(c)
        R, page = c["R"], c["page"]
        mix = rng.permutation(R)
        n, ln = np.array(n)[mix], np.array(ln)[mix]
        held = -(-ln // page)
        room = int((-(-(ln + n) // page)).max()) + 1
        pages = int(held.sum()) + c["spare"]
        order = rng.permutation(pages).astype(np.int32)
        table = np.full((R, room), -1, np.int32)
        first = np.cumsum(held) - held
        here = np.arange(room)[None, :] < held[:, None]
        table[here] = order[(first[:, None] + np.arange(room)[None, :])[here]]
        free = np.full(pages + 1, -1, np.int32)
        free[:c["spare"]] = order[int(held.sum()):]

        def dev(x):
            return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)

        s["table"], s["free"] = dev(table), dev(free)
        s["count"] = torch.tensor([c["spare"]], dtype=torch.int32, device=DEV)
        s["kv_len"], s["back"] = dev(ln.astype(np.int32)), dev(ln.astype(np.int32))
        s["n"] = dev(n.astype(np.int32))
        T = int(n.sum()) + 5  # a batch is padded
        s["q_start"] = torch.empty(R + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(T, dtype=torch.int64, device=DEV)
        s["positions"] = torch.empty(T, dtype=torch.int32, device=DEV)
        s["granted"] = torch.empty(R, dtype=torch.int32, device=DEV)
        return s

    kind = TYPES[c["type"]]
    n, ln = _requests(c)
    mix = rng.permutation(c["R"])
    n, ln = [n[i] for i in mix], [ln[i] for i in mix]
    page = c["page"]
    per = [-(-v // page) for v in ln]
    pages = sum(per) + 3
    order = rng.permutation(pages)
    table = np.zeros((c["R"], max(per)), np.int32)
    at = 0
    for r in range(c["R"]):
        table[r, :per[r]] = order[at:at + per[r]]
        at += per[r]
    s["tree"] = None
    if c["tree"]:
        bits, at_q = np.zeros(sum(n), np.int64), 0
        for r in range(c["R"]):
            for i in range(n[r]):  # a random tree: each token hangs on an earlier one or on the context
                up = int(rng.integers(-1, i)) if i else -1
                seen = (int(bits[at_q + up]) & (2 ** 64 - 1) if up >= 0 else 0) | 1 << i
                bits[at_q + i] = np.array(seen, np.uint64).view(np.int64)
            at_q += n[r]
        s["tree"] = torch.from_numpy(bits[:, None]).to(DEV)
    s["q"] = normal(sum(n), c["H"], c["dk"], like=kind)
    s["q_start"] = torch.tensor([sum(n[:r]) for r in range(c["R"] + 1)], dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(ln, dtype=torch.int32, device=DEV)
    s["table"] = torch.from_numpy(table).to(DEV)
    s["out"] = torch.empty(sum(n), c["H"], c["dv"], dtype=kind, device=DEV)
    s["lse"] = torch.empty(sum(n), c["H"], dtype=torch.float32, device=DEV)
    # the cache: rows that were written before, with scales like those of unit rows
    shape = (pages, page, 1, c["dk"])
    if c["store"] == "int8":
        s["rows"] = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
    elif c["store"] == "fp8":
        s["rows"] = torch.empty(shape, dtype=TYPES["fp8"], device=DEV)
        s["rows"].copy_((normal(*shape, like=torch.float16) * 120).clamp_(-448, 448))
    else:
        s["rows"] = normal(*shape, like=kind)
    s["scale"] = None
    if c["store"] in TOP:
        u = torch.rand(shape[:3], generator=g, device=DEV, dtype=torch.float32)
        s["scale"] = (2.0 + 2.0 * u) / TOP[c["store"]]
    if own:
        # what a serving program makes once for its cache and keeps: the
        # cache's handle and the attention's workspace
        from place_partial_rope_gb300 import binding
        s["cache"] = binding.KVCache(s["rows"], k_scale=s["scale"])
        s["workspace"] = binding.latent_attention_workspace(s["q"], s["cache"], c["dv"], c["n_hi"])
    return s


# ---------------------------------------------------------------- plain forms


def _split(x, mode):
    return (x[..., 0::2], x[..., 1::2]) if mode == "interleave" else x.chunk(2, -1)


def _join(a, b, mode):
    return torch.stack([a, b], -1).flatten(-2) if mode == "interleave" else torch.cat([a, b], -1)


def _turn(x, s, back):
    """Lanes [start, end) turned by the rows of cos and sin, or turned back."""
    c = s["c"]
    a, b = _split(x[..., c["start"]:c["end"]], c["mode"])
    (ca, cb), (sa, sb) = (_split(s[t].float(), c["mode"]) for t in ("cos", "sin"))
    y = (a * ca + b * sb, b * cb - a * sa) if back else (a * ca - b * sa, b * cb + a * sb)
    return torch.cat([x[..., :c["start"]], _join(*y, c["mode"]), x[..., c["end"]:]], -1)


def _norm(s):
    c, got = s["c"], {}
    n0, n1 = c["n0"], c["n1"]
    for name in ("q", "k") if c["Nk"] else ("q",):
        x, w = s[name].float(), s[name + "w"].float()
        part = x[..., n0:n1]
        if c["dir"] == "fwd":
            r = (part.square().mean(-1) + EPS).rsqrt()
            y = torch.cat([x[..., :n0], part * r[..., None] * w, x[..., n1:]], -1)
            got[name] = _turn(y, s, False).to(s[name].dtype)
            if c["keep"]:
                got[name + "r"] = r
            continue
        r = s[name + "r"][..., None]
        dy = _turn(s["d" + name].float(), s, True)
        d, unit = dy[..., n0:n1], part * r
        dw = d * w
        dx = (dw - unit * (dw * unit).mean(-1, keepdim=True)) * r
        got["d" + name] = torch.cat([dy[..., :n0], dx, dy[..., n1:]], -1).to(s[name].dtype)
        got["d" + name + "w"] = (d * unit).sum((0, 1, 2))
    return got


def _pages(s):
    c = s["c"]
    page, R, room = c["page"], c["R"], s["table"].shape[1]
    n, old, count = s["n"].long(), s["kv_len"].long(), s["count"].long()
    held, want = (old + page - 1) // page, (old + n + page - 1) // page
    fits = want <= room
    need = torch.where(fits, want - held, 0)
    before = need.cumsum(0) - need
    granted = fits & ((need == 0) | (before + need <= count))
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), n.cumsum(0)])
    # pages, from the top of the stack, in the order of the requests
    col = torch.arange(room, device=DEV)
    fresh = granted[:, None] & (col >= held[:, None]) & (col < want[:, None])
    from_top = before[:, None] + col - held[:, None]
    took = s["free"][(count - 1 - from_top).clamp(0, s["free"].shape[0] - 1)]
    table = torch.where(fresh, took, s["table"])
    t = torch.arange(s["slots"].shape[0], device=DEV)
    r = torch.searchsorted(start[1:], t, right=True).clamp_max(R - 1)
    at = old[r] + t - start[r]
    inside = t < start[R]
    slot = table[r, (at // page).clamp_max(room - 1)].long() * page + at % page
    out = {"q_start": start.int(), "slots": torch.where(inside & granted[r], slot, -1),
           "positions": torch.where(inside, at, 0).int(), "granted": granted.int()}
    length = torch.where(granted, old + n, old)
    out["grown_len"], out["grown_table"] = length.int(), table
    count = count - fresh.sum()
    # and back: what lies past the kept rows goes onto the stack again
    keep = torch.minimum(s["back"].long().clamp_min(0), length)
    stay, held = (keep + page - 1) // page, (length + page - 1) // page
    gone = held - stay
    before = gone.cumsum(0) - gone
    total = gone.sum()
    out_of = (col >= stay[:, None]) & (col < held[:, None])
    place = count + total - 1 - (before[:, None] + col - stay[:, None])
    s["free"][place[out_of]] = table[out_of]
    s["table"].copy_(torch.where(out_of, -1, table))
    s["kv_len"].copy_(keep)
    s["count"].copy_(count + total)
    return {**out, "kv_len": s["kv_len"], "table": s["table"], "free": s["free"], "count": s["count"]}


def _latent(s):
    c = s["c"]
    R, most, page, H = c["R"], c["len_hi"], c["page"], c["H"]
    j = torch.arange(most, device=DEV)
    slots = s["table"].long()[:, (j // page).clamp_max(s["table"].shape[1] - 1)] * page + j % page
    flat = s["rows"].flatten(0, 1)[:, 0]
    if c["store"] == "fp8":
        x = flat.view(torch.uint8)[slots].view(TYPES["fp8"]).float()
    else:
        x = flat[slots].float()
    if s["scale"] is not None:
        x = x * s["scale"].flatten()[slots][..., None]                 # R, most, dk
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(c["n_hi"], device=DEV)
    at = (s["q_start"][:-1].long()[:, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().flatten(1, 2)                               # R, n * H, dk
    score = q @ x.transpose(1, 2) * (1.0 / math.sqrt(c["dk"]))
    draft = j - (s["kv_len"].long() - n)[:, None]                      # R, most
    if s["tree"] is None:
        bit = draft[:, None] <= i[:, None]
    else:
        bit = (s["tree"][at][:, :, 0, None] >> draft.clamp(0, 63)[:, None] & 1) == 1
    seen = (draft < 0)[:, None] | (bit & (j < s["kv_len"][:, None])[:, None])
    score = score.unflatten(1, (c["n_hi"], H)).masked_fill_(~seen[:, :, None], -math.inf).flatten(1, 2)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ x[..., :c["dv"]]) / total
    lse = (top + total.log())[..., 0]
    kept = i < n[:, None]
    return {"out": o.unflatten(1, (c["n_hi"], H))[kept].to(s["q"].dtype),
            "lse": lse.unflatten(1, (c["n_hi"], H))[kept]}


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["c"]
    if not own:
        return {"norm": _norm, "pages": _pages, "latent": _latent}[c["op"]](s)
    from place_partial_rope_gb300 import binding
    if c["op"] == "norm":
        k = s.get("k")
        if c["dir"] == "fwd":
            binding.rope_partial_norm_fwd(s["q"], k, s["qw"], s.get("kw"), s["cos"], s["sin"], c["start"], c["end"],
                                          eps=EPS, norm=(c["n0"], c["n1"]), mode=c["mode"], q_out=s["q_out"],
                                          k_out=s.get("k_out"), q_rstd=s.get("qr"), k_rstd=s.get("kr"))
            got = {"q": s["q_out"], "k": s.get("k_out"), "qr": s.get("qr"), "kr": s.get("kr")}
        else:
            binding.rope_partial_norm_bwd(s["dq"], s.get("dk"), s["q"], k, s["qw"], s.get("kw"), s["qr"],
                                          s.get("kr"), s["cos"], s["sin"], c["start"], c["end"],
                                          norm=(c["n0"], c["n1"]), mode=c["mode"], dq_out=s["q_out"],
                                          dk_out=s.get("k_out"), dq_weight=s["dqw"], dk_weight=s.get("dkw"),
                                          workspace=s["workspace"])
            got = {"dq": s["q_out"], "dk": s.get("k_out"), "dqw": s["dqw"], "dkw": s.get("dkw")}
        return {name: x for name, x in got.items() if x is not None}
    if c["op"] == "pages":
        binding.rope_partial_cache_grow(s["kv_len"], s["n"], s["table"], s["free"], s["count"], c["page"],
                                        s["q_start"], s["slots"], positions=s["positions"], granted=s["granted"])
        got = {"q_start": s["q_start"], "slots": s["slots"], "positions": s["positions"], "granted": s["granted"],
               "grown_len": s["kv_len"].clone(), "grown_table": s["table"].clone()}
        binding.rope_partial_cache_trim(s["kv_len"], s["back"], s["table"], s["free"], s["count"], c["page"])
        return {**got, "kv_len": s["kv_len"], "table": s["table"], "free": s["free"], "count": s["count"]}
    binding.rope_partial_latent_attention(s["q"], s["cache"], s["q_start"], s["kv_len"], s["table"], s["out"],
                                          lse=s["lse"], tree=s["tree"], scale=1.0 / math.sqrt(c["dk"]),
                                          max_q=c["n_hi"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        L = c["end"] - c["start"]
        other = np.arange(L) ^ 1 if c["mode"] == "interleave" else (np.arange(L) + L // 2) % L
        first = np.arange(L) % 2 == 0 if c["mode"] == "interleave" else np.arange(L) < L // 2
        other = torch.from_numpy(other).to(DEV)
        sign = torch.from_numpy(np.where(first, -1.0, 1.0)).to(DEV)
        cos, sin = s["cos"].double(), s["sin"].double()
        lanes, wide = slice(c["start"], c["end"]), slice(c["n0"], c["n1"])
        got = {}
        for name in ("q", "k") if c["Nk"] else ("q",):
            w = torch.ones(c["D"], dtype=torch.float64, device=DEV)
            w[wide] = s[name + "w"].double()
            outs, rs, dw = [], [], torch.zeros(c["n1"] - c["n0"], dtype=torch.float64, device=DEV)
            for b in range(c["B"]):
                x = s[name][b].double()
                cb, sb = (t[b if t.shape[0] > 1 else 0] for t in (cos, sin))
                if c["dir"] == "fwd":
                    r = 1.0 / torch.sqrt((x[..., wide] ** 2).mean(-1) + EPS)
                    x[..., wide] *= r[..., None]
                    x *= w
                    y = x[..., lanes]
                    x[..., lanes] = y * cb + sign * y[..., other] * sb
                    outs.append(x)
                    rs.append(r)
                else:
                    r = s[name + "r"][b].double()[..., None]
                    g = s["d" + name][b].double()
                    y = g[..., lanes]
                    g[..., lanes] = y * cb + (sign * y * sb)[..., other]  # the transposed rotation
                    unit = x[..., wide] * r
                    dw += (g[..., wide] * unit).sum((0, 1))
                    a = g[..., wide] * w[wide]
                    g[..., wide] = r * a - unit * r * (a * unit).sum(-1, keepdim=True) / (c["n1"] - c["n0"])
                    outs.append(g)
            if c["dir"] == "fwd":
                got[name] = torch.stack(outs)
                if c["keep"]:
                    got[name + "r"] = torch.stack(rs)
            else:
                got["d" + name], got["d" + name + "w"] = torch.stack(outs), dw
        return got

    if c["op"] == "pages":
        page = c["page"]
        table, free = s["table"].cpu().numpy(), s["free"].cpu().numpy()
        length, n, back = (s[t].cpu().numpy() for t in ("kv_len", "n", "back"))
        top, room, asked = c["spare"], table.shape[1], 0
        have = top
        start, granted = [0], []
        slots = np.full(s["slots"].shape[0], -1, np.int64)
        positions = np.zeros(s["slots"].shape[0], np.int32)
        for r in range(c["R"]):
            lo, hi = int(length[r]), int(length[r]) + int(n[r])
            held, want = -(-lo // page), -(-hi // page)
            ok = want <= room
            if ok and want > held:
                asked += want - held
                ok = asked <= have
            if ok:
                for p in range(held, want):
                    top -= 1
                    table[r, p] = free[top]
                length[r] = hi
                at = np.arange(lo, hi)
                slots[start[-1]:start[-1] + hi - lo] = table[r, at // page].astype(np.int64) * page + at % page
            positions[start[-1]:start[-1] + hi - lo] = np.arange(lo, hi)
            granted.append(int(ok))
            start.append(start[-1] + hi - lo)
        got = {"q_start": np.array(start, np.int32), "slots": slots, "positions": positions,
               "granted": np.array(granted, np.int32), "grown_len": length.copy(), "grown_table": table.copy()}
        for r in reversed(range(c["R"])):
            keep = min(max(int(back[r]), 0), int(length[r]))
            for p in reversed(range(-(-keep // page), -(-int(length[r]) // page))):
                free[top] = table[r, p]
                table[r, p] = -1
                top += 1
            length[r] = keep
        got.update(kv_len=length, table=table, free=free, count=np.array([top], np.int32))
        return {name: torch.from_numpy(x).to(DEV) for name, x in got.items()}

    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    page, flat = c["page"], s["rows"].flatten(0, 1)[:, 0]
    for r in range(c["R"]):
        lo, hi, m = starts[r], starts[r + 1], lens[r]
        where = torch.arange(m, device=DEV)
        slots = s["table"][r].long()[where // page] * page + where % page
        if c["store"] == "fp8":
            x = flat.view(torch.uint8)[slots].view(TYPES["fp8"]).float().double()
        else:
            x = flat[slots].double()
        if s["scale"] is not None:
            x = x * s["scale"].flatten()[slots].double()[:, None]
        seen = np.ones((hi - lo, m), bool)
        for i in range(hi - lo):
            bits = None if s["tree"] is None else int(s["tree"][lo + i, 0])
            for k in range(hi - lo):
                seen[i, m - (hi - lo) + k] = k <= i if bits is None else bool(bits >> k & 1)
        seen = torch.from_numpy(seen).to(DEV)
        for h in range(c["H"]):
            z = torch.where(seen, s["q"][lo:hi, h].double() @ x.T / math.sqrt(c["dk"]), -math.inf)
            lse[lo:hi, h] = torch.logsumexp(z, -1)
            out[lo:hi, h] = torch.exp(z - lse[lo:hi, h, None]) @ x[:, :c["dv"]]
    return {"out": out, "lse": lse}
