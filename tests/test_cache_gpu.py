"""Writing the paged cache and reading it back, on the GPU: codes and scales
bit for bit against the same fp32 steps in numpy, and values within the bounds
of an 8-bit code of the 64-bit rotation."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STORES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def make_cache(store, pages, page, heads, dk, dv, head_major=False, pad=0):
    """A cache full of a marker byte; (handle, tensors)."""
    def tensor(d, dtype):
        if head_major:
            t = torch.zeros((pages, heads, page, d + pad), dtype=dtype, device=DEV)
            t.view(torch.uint8).fill_(0x3a)
            return t[..., :d].permute(0, 2, 1, 3)
        t = torch.zeros((pages, page, heads, d + pad), dtype=dtype, device=DEV)
        t.view(torch.uint8).fill_(0x3a)
        return t[..., :d]

    k, v = tensor(dk, STORES[store]), (tensor(dv, STORES[store]) if dv else None)
    s = [torch.full((pages, page, heads), -7.0, device=DEV) if store in ref.TOP else None for _ in range(2)]
    if not dv:
        s[1] = None
    return binding.KVCache(k, v, *s), k, v, s[0], s[1]


def codes_of(t):
    """A cache tensor's codes, or 16-bit values' bits, as numpy (pages * page, heads, d)."""
    t = t.contiguous()
    t = t.view(torch.int8 if t.element_size() == 1 else torch.int16)
    return t.flatten(0, 1).cpu().numpy()


CASES = [  # T, heads, dk, dv, page, start, end, mode
    (1, 1, 64, 64, 16, 0, 64, "half"),
    (33, 8, 128, 128, 64, 0, 64, "interleave"),
    (7, 3, 192, 128, 16, 128, 192, "half"),
    (50, 2, 80, 96, 48, 16, 80, "interleave"),
    (9, 5, 64, 48, 1, 3, 41, "interleave"),     # odd start, pages of one token
    (12, 2, 72, 24, 100, 1, 59, "half"),        # odd start, odd half
    (5, 1, 576, 512, 3, 512, 576, "interleave"),
    (6, 2, 33, 17, 8, 0, 0, "half"),            # odd rows: single elements, no rotation
    (4, 2, 1024, 1024, 5, 0, 1024, "half"),
    (21, 4, 40, 0, 32, 0, 40, "interleave"),    # keys only
    (3, 2, 34, 8, 4, 2, 30, "half"),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("store", ["fp8", "int8", "bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_and_read(case, store, dtype):
    T, H, dk, dv, page, st, en, mode = CASES[case]
    pages = T // page + 3
    g = torch.Generator().manual_seed(case)
    k = torch.randn((T, H, dk), generator=g).to(TYPES[dtype])
    v = torch.randn((T, H, dv), generator=g).to(TYPES[dtype]) if dv else None
    L = en - st
    cos, sin = (torch.randn((T, L), generator=g).to(TYPES[dtype]) for _ in range(2))
    slots = torch.randperm(pages * page, generator=g)[:T].clone()
    if T > 4:
        slots[2], slots[4] = -1, pages * page  # skipped
    cache, ck, cv, ks, vs = make_cache(store, pages, page, H, dk, dv, head_major=case % 2 == 1,
                                       pad=(16 if case % 3 == 0 else 0))
    before = [None if t is None else t.clone() for t in (ck, cv, ks, vs)]
    kd, vd = k.to(DEV), None if v is None else v.to(DEV)
    rot = (cos.to(DEV), sin.to(DEV)) if L else (None, None)
    binding.rope_partial_cache_write(cache, kd, vd, slots.to(DEV), *rot, st, en, mode)
    torch.cuda.synchronize()
    assert torch.equal(kd.cpu(), k)  # the inputs stay as they are

    used = [t for t in range(T) if 0 <= slots[t] < pages * page]
    where = slots[used].numpy()
    rows = [("k", ck, ks, ref.rotate_rows_fp32(k.float().numpy(), cos.float().numpy(), sin.float().numpy(),
                                               st, en, mode) if L else k.float().numpy(), before[0], before[2])]
    if dv:
        rows.append(("v", cv, vs, v.float().numpy(), before[1], before[3]))
    for name, t, s, y, t0, s0 in rows:
        got, old = codes_of(t), codes_of(t0)
        if store in ref.TOP:
            codes, scale = ref.quantise_fp32(y[used], store)
            assert np.array_equal(got[where].view(np.uint8), codes.view(np.uint8)), name
            flat = s.flatten(0, 1).cpu().numpy()
            assert np.array_equal(flat[where], scale), name
            rest = np.setdiff1d(np.arange(pages * page), where)
            assert np.array_equal(flat[rest], s0.flatten(0, 1).cpu().numpy()[rest])
        else:
            want = torch.from_numpy(y[used]).to(STORES[store]).view(torch.int16).numpy()
            assert np.array_equal(got[where], want), name
        rest = np.setdiff1d(np.arange(pages * page), where)
        assert np.array_equal(got[rest], old[rest]), name  # every other slot untouched

    for out_dtype in ("bf16", "fp32"):
        ko = torch.full((T, H, dk), 5.0, dtype=TYPES[out_dtype], device=DEV)
        vo = torch.full((T, H, dv), 5.0, dtype=TYPES[out_dtype], device=DEV) if dv else None
        binding.rope_partial_cache_read(cache, slots.to(DEV), ko, vo)
        torch.cuda.synchronize()
        for out, t, s in ((ko, ck, ks), (vo, cv, vs)):
            if out is None:
                continue
            flat = t.contiguous().flatten(0, 1).cpu()
            want = torch.zeros(out.shape, dtype=torch.float32)
            want[used] = flat.float()[where] * (1 if s is None else s.flatten(0, 1).cpu()[where][..., None])
            assert torch.equal(out.cpu(), want.to(TYPES[out_dtype]))


@pytest.mark.parametrize("store", ["fp8", "int8"])
def test_values_within_a_code_of_the_rotation(store):
    """|value - x| is at most half a step of the code: e4m3 has 3 bits after
    the leading one (|x| 2^-4, at least half of 2^-9 of the scale), int8 half
    the scale; plus the fp32 steps (1e-6 of the row's largest)."""
    T, H, d = 300, 2, 128
    g = torch.Generator().manual_seed(5)
    k = torch.randn((T, H, d), generator=g) * torch.logspace(-20, 20, T)[:, None, None]
    th = torch.rand((T, d // 2), generator=g) * 6.28
    cos, sin = torch.cat([th.cos()] * 2, -1), torch.cat([th.sin()] * 2, -1)
    cache, ck, cv, ks, _ = make_cache(store, 20, 16, H, d, 0)
    slots = torch.arange(T, device=DEV)
    binding.rope_partial_cache_write(cache, k.to(DEV), None, slots, cos.to(DEV), sin.to(DEV), 0, d, "half")
    out = torch.empty((T, H, d), device=DEV)
    binding.rope_partial_cache_read(cache, slots, out)
    x = k.double().numpy()
    c, s = cos.double().numpy()[:, None], sin.double().numpy()[:, None]
    y = np.concatenate([x[..., :64] * c[..., :64] - x[..., 64:] * s[..., :64],
                        x[..., 64:] * c[..., 64:] + x[..., :64] * s[..., 64:]], -1)
    top = np.abs(y).max(-1, keepdims=True)
    scale = top / ref.TOP[store]
    half = np.maximum(np.abs(y) / 16, scale * 2.0 ** -10) if store == "fp8" else scale / 2
    assert np.all(np.abs(out.cpu().numpy() - y) <= half * (1 + 1e-5) + 1e-6 * top)


@pytest.mark.parametrize("store", ["fp8", "int8"])
def test_rows_of_zeros_tiny_and_not_finite(store):
    d = 64
    k = torch.zeros((6, 1, d))
    k[1] = 1e-40          # below 2^-100: stored relative to it, i.e. as zero
    k[2, 0, 3] = float("inf")
    k[3, 0, 5] = float("nan")
    k[4] = torch.linspace(-1, 1, d) * 3e38
    k[5, 0, 7] = -0.0
    cache, ck, _, ks, _ = make_cache(store, 1, 8, 1, d, 0)
    slots = torch.arange(6, device=DEV)
    binding.rope_partial_cache_write(cache, k.to(DEV), None, slots)
    out = torch.empty((6, 1, d), device=DEV)
    binding.rope_partial_cache_read(cache, slots, out)
    o, s = out.cpu().numpy()[:, 0], ks.flatten().cpu().numpy()
    least = np.float32(2.0 ** -100) / np.float32(ref.TOP[store])
    assert np.all(o[0] == 0) and np.all(o[1] == 0) and np.all(o[5] == 0)
    assert s[0] == least and s[1] == least
    assert np.isnan(o[2]).all() and np.isnan(o[3]).all() and np.isnan(s[2:4]).all()
    assert np.isfinite(o[4]).all() and abs(o[4][0] + 3e38) <= 3e38 / 16


def test_strided_inputs_and_broadcast_rotation():
    """k and v as slices of one packed tensor, one cos/sin row for all tokens,
    outputs into a packed tensor too, on another stream."""
    T, H, d = 37, 4, 64
    g = torch.Generator().manual_seed(3)
    packed = torch.randn((T, 3 * H, d), generator=g).to(torch.bfloat16)
    cos, sin = (torch.randn((1, 32), generator=g).to(torch.bfloat16) for _ in range(2))
    dev = packed.to(DEV)
    cache, ck, cv, ks, vs = make_cache("fp8", 4, 16, H, d, d)
    slots = torch.arange(T, device=DEV)
    out = torch.zeros((T, 2 * H, d), dtype=torch.bfloat16, device=DEV)
    cd, sd = cos.to(DEV), sin.to(DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    binding.rope_partial_cache_write(cache, dev[:, H:2 * H], dev[:, 2 * H:], slots, cd, sd, 32, 64, "half",
                                     stream=stream)
    binding.rope_partial_cache_read(cache, slots, out[:, :H], out[:, H:], stream=stream.cuda_stream)
    stream.synchronize()
    y = ref.rotate_rows_fp32(packed[:, H:2 * H].float().numpy(), cos.float().numpy(), sin.float().numpy(),
                             32, 64, "half")
    for i, rows in enumerate((y, packed[:, 2 * H:].float().numpy())):
        codes, scale = ref.quantise_fp32(rows, "fp8")
        want = ref.fp8_values()[codes].astype(np.float32) * scale[..., None]
        assert torch.equal(out[:, i * H:(i + 1) * H].cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_offsets_past_32_bits():
    """Slots whose rows lie more than 4 GB into the cache."""
    pages, page, H, d = 33000, 64, 16, 128  # 4.3 GB of codes
    k = torch.empty((pages, page, H, d), dtype=torch.int8, device=DEV)
    ks = torch.empty((pages, page, H), device=DEV)
    cache = binding.KVCache(k, None, ks, None)
    x = torch.randn((5, H, d), device=DEV)
    slots = torch.tensor([0, 1, pages * page - 1, pages * page - 70, pages * page // 2], device=DEV)
    binding.rope_partial_cache_write(cache, x, None, slots)
    out = torch.empty_like(x)
    binding.rope_partial_cache_read(cache, slots, out)
    codes, scale = ref.quantise_fp32(x.cpu().numpy(), "int8")
    want = codes.astype(np.float32) * scale[..., None]
    assert np.array_equal(out.cpu().numpy(), want)
    assert np.array_equal(k.flatten(0, 1)[slots].cpu().numpy(), codes)


def test_in_a_cuda_graph():
    T, H, d = 16, 2, 128
    cache, ck, cv, ks, vs = make_cache("int8", 2, 16, H, d, d)
    k, v = (torch.zeros((T, H, d), dtype=torch.float16, device=DEV) for _ in range(2))
    out = [torch.empty_like(k) for _ in range(2)]
    slots = torch.arange(T, device=DEV)

    def step():
        binding.rope_partial_cache_write(cache, k, v, slots)
        binding.rope_partial_cache_read(cache, slots, *out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        torch.manual_seed(seed)
        k.normal_()
        v.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for x, o in ((k, out[0]), (v, out[1])):
            codes, scale = ref.quantise_fp32(x.float().cpu().numpy(), "int8")
            want = torch.from_numpy(codes.astype(np.float32) * scale[..., None]).half()
            assert torch.equal(o.cpu(), want)
