"""The C ABI of include/rope_serving.h without a GPU: what a call refuses (no
CUDA call is made for a refused or empty call, so made-up device addresses
will do), the header, the host-side tree mask, and the binding's own checks."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from place_partial_rope_gb300 import binding, torch_op

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rope_serving.h")
OK, NULL, INVALID = 0, 1, 2
X, POS, K, V, KS, VS = (0x10000000 + (i << 36) for i in range(6))
A, B, C, D_, E, F, G, H = (0x7000000000000 + (i << 36) for i in range(8))
I64 = ctypes.c_int64


def i64(*v):
    return (I64 * len(v))(*v)


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def message(lib):
    return lib.rope_last_error_message().decode()


def test_header_names_are_exported_and_it_is_c(lib, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(rope_partial_[a-z_]+)\s*\(", text))
    assert names == {"rope_partial_inplace_fwd_axes", "rope_partial_inplace_bwd_axes",
                     "rope_partial_cache_write", "rope_partial_cache_read", "rope_partial_tree_attention",
                     "rope_partial_tree_attention_workspace", "rope_partial_tree_mask"}
    for n in names:
        assert hasattr(lib, n), n
    src = tmp_path / "h.c"
    src.write_text('#include "rope_serving.h"\nint main(void) { return (int)sizeof(rope_kv_cache_t); }\n')
    gcc = shutil.which("gcc")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(tmp_path / "h")], check=True)
    size = subprocess.run([str(tmp_path / "h")]).returncode
    assert size == ctypes.sizeof(binding.RopeKVCache) % 256


# ---------------------------------------------------------------- axes


def axes(lib, x=X, pos=POS, dtype=0, shape=(2, 4, 3, 16), axes=2, sections=(4, 4), pshape=(2, 2, 4),
         pstride=(8, 4, 1), order=0, spectrum=0, base=10000.0, start=0, end=16, mode=1, fn="fwd"):
    sec = None if sections is None else (ctypes.c_int32 * len(sections))(*sections)
    return getattr(lib, f"rope_partial_inplace_{fn}_axes")(
        x, pos, dtype, *shape, axes, sec, None if pshape is None else i64(*pshape),
        None if pstride is None else i64(*pstride), order, spectrum, base, start, end, mode, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=7), INVALID, "dtype"),
    (dict(mode=3), INVALID, "mode"),
    (dict(order=2), INVALID, "order"),
    (dict(spectrum=-1), INVALID, "spectrum"),
    (dict(base=0.0), INVALID, "base"),
    (dict(base=float("inf")), INVALID, "base"),
    (dict(axes=0), INVALID, "axes"),
    (dict(axes=5, sections=(2, 2, 2, 1, 1)), INVALID, "axes"),
    (dict(sections=(4, 5)), INVALID, "pairs"),
    (dict(sections=(-1, 9)), INVALID, "negative"),
    (dict(sections=None), NULL, "sections"),
    (dict(end=15), INVALID, "even"),
    (dict(end=18), INVALID, "slice"),
    (dict(shape=(2, 4, 3, 2048)), INVALID, "1024"),
    (dict(x=0), NULL, "x is null"),
    (dict(pos=0), NULL, "positions"),
    (dict(pshape=None), NULL, "pos_shape"),
    (dict(pshape=(1, 2, 4)), INVALID, "axes"),
    (dict(pshape=(2, 3, 4)), INVALID, "dim 1"),
    (dict(pshape=(2, 2, 3)), INVALID, "dim 2"),
    (dict(pstride=(8, -4, 1)), INVALID, "negative"),
    (dict(pos=POS + 2), INVALID, "aligned"),
    (dict(pos=X + 64), INVALID, "overlap"),
])
def test_axes_refusals(lib, fn, kw, status, needle):
    assert axes(lib, fn=fn, **kw) == status
    assert needle in message(lib)


def test_axes_empty_calls(lib):
    assert axes(lib, shape=(0, 4, 3, 16), pshape=(2, 0, 4), x=0, pos=0) == OK
    assert axes(lib, sections=(0, 0), start=6, end=6, x=0, pos=0) == OK
    assert message(lib) == ""


# ---------------------------------------------------------------- the cache


def cache(store=3, pages=8, page=16, heads=2, kd=64, vd=64, **kw):
    def strides(d):
        return (I64 * 3)(page * heads * d, heads * d, d)

    wide = store in (0, 1)
    c = binding.RopeKVCache(K, V if vd else None, None if wide else KS, None if wide or not vd else VS, pages, page,
                            heads, kd, vd, strides(kd), strides(vd), strides(1), strides(1), store, 0)
    for name, value in kw.items():
        setattr(c, name, value)
    return c


CACHE_FAULTS = [
    (dict(store=2), INVALID, "dtype"),
    (dict(pages=-1), INVALID, "sizes"),
    (dict(page=0), INVALID, "sizes"),
    (dict(heads=0), INVALID, "sizes"),
    (dict(kd=1025), INVALID, "1024"),
    (dict(k=None), NULL, "k is null"),
    (dict(v=None), NULL, "v must be null"),
    (dict(k_scale=None), NULL, "k_scale"),
    (dict(v_scale=VS + 2), INVALID, "4-byte"),
    (dict(store=0, k_scale=KS), INVALID, "no scales"),
    (dict(store=1, k=K + 1), INVALID, "aligned"),
    (dict(k_stride=i64(2048, 128, 63)), INVALID, "strides"),
    (dict(v_stride=i64(-2048, 128, 64)), INVALID, "strides"),
    (dict(k_scale_stride=i64(32, 2, 0)), INVALID, "scale strides"),
    (dict(pages=2 ** 40, page=2 ** 20), INVALID, "range"),
]


def write(lib, c, k=A, v=B, dtype=0, T=5, ks=(128, 64), vs=(128, 64), slots=C, cos=D_, sin=E, cst=64, sst=64, start=0,
          end=64, mode=1):
    return lib.rope_partial_cache_write(None if c is None else ctypes.byref(c), k, v, dtype, T,
                                        None if ks is None else i64(*ks), None if vs is None else i64(*vs), slots,
                                        cos, sin, cst, sst, start, end, mode, None)


@pytest.mark.parametrize("kw,status,needle", CACHE_FAULTS)
def test_cache_descriptor_refusals(lib, kw, status, needle):
    assert write(lib, cache(**kw)) == status
    assert needle in message(lib)
    assert lib.rope_partial_cache_read(ctypes.byref(cache(**kw)), C, 5, A, B, 0, i64(128, 64), i64(128, 64),
                                       None) == status


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), INVALID, "dtype"),
    (dict(mode=0), INVALID, "mode"),
    (dict(T=-1), INVALID, "T="),
    (dict(start=-2), INVALID, "slice"),
    (dict(end=66), INVALID, "slice"),
    (dict(end=63), INVALID, "even"),
    (dict(k=None), NULL, "k"),
    (dict(v=None), NULL, "v must"),
    (dict(slots=None), NULL, "slots"),
    (dict(cos=None), NULL, "cos"),
    (dict(ks=None), NULL, "strides"),
    (dict(vs=None), NULL, "v_stride"),
    (dict(ks=(-1, 64)), INVALID, "strides"),
    (dict(cst=-64), INVALID, "strides"),
    (dict(k=A + 1), INVALID, "aligned"),
    (dict(slots=C + 4), INVALID, "aligned"),
    (dict(k=K + 128), INVALID, "overlaps"),
    (dict(cos=KS), INVALID, "overlaps"),
    (dict(slots=V + 8), INVALID, "overlaps"),
])
def test_write_refusals(lib, kw, status, needle):
    assert write(lib, cache(), **kw) == status
    assert needle in message(lib)


def test_write_and_read_empty_calls(lib):
    assert write(lib, cache(), k=None, v=None, T=0, slots=None, cos=None, sin=None) == OK
    assert write(lib, cache(pages=0, k=None, v=None, k_scale=None, v_scale=None)) == OK
    assert write(lib, None) == NULL
    assert lib.rope_partial_cache_read(ctypes.byref(cache()), None, 0, A, B, 0, i64(1, 1), i64(1, 1), None) == OK
    assert lib.rope_partial_cache_read(ctypes.byref(cache()), None, 4, None, None, 0, None, None, None) == OK


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=9), INVALID, "dtype"),
    (dict(T=-1), INVALID, "T="),
    (dict(slots=None), NULL, "slots"),
    (dict(ks=None), NULL, "stride"),
    (dict(ks=(63, 64)), INVALID, "strides"),
    (dict(vs=(128, 0)), INVALID, "strides"),
    (dict(k=A + 1), INVALID, "aligned"),
    (dict(v=A), INVALID, "overlap"),
    (dict(v=A + 128, vs=(128, 64)), INVALID, "overlap"),
    (dict(k=V), INVALID, "overlap"),
    (dict(slots=A + 8), INVALID, "overlap"),
])
def test_read_refusals(lib, kw, status, needle):
    a = dict(slots=C, T=5, k=A, v=B, dtype=0, ks=(128, 64), vs=(128, 64))
    a.update(kw)
    st = lib.rope_partial_cache_read(ctypes.byref(cache()), a["slots"], a["T"], a["k"], a["v"], a["dtype"],
                                     None if a["ks"] is None else i64(*a["ks"]), i64(*a["vs"]), None)
    assert st == status
    assert needle in message(lib)


# ---------------------------------------------------------------- attention


def attend(lib, c, q=A, dtype=0, Tq=6, Hq=4, qst=(256, 64), q_start=B, kv_len=C, R=2, max_q=3, table=D_,
           max_pages=4, tst=4, tree=E, words=1, out=F, ost=(256, 64), lse=G, scale=0.125, ws=H, nbytes=1 << 40):
    return lib.rope_partial_tree_attention(
        ctypes.byref(c), q, dtype, Tq, Hq, None if qst is None else i64(*qst), q_start, kv_len, R, max_q, table,
        max_pages, tst, tree, words, out, i64(*ost), lse, scale, ws, nbytes, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), INVALID, "bf16"),
    (dict(Hq=5), INVALID, "multiple"),
    (dict(max_q=0), INVALID, "max_q"),
    (dict(Tq=-1), INVALID, "Tq"),
    (dict(R=-1), INVALID, "R="),
    (dict(max_pages=-1), INVALID, "pages"),
    (dict(max_pages=2 ** 30), INVALID, "2^31"),
    (dict(tst=3), INVALID, "page_table_stride"),
    (dict(words=0), INVALID, "tree_words"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(scale=-1.0), INVALID, "scale"),
    (dict(q=None), NULL, "q"),
    (dict(out=None), NULL, "out"),
    (dict(kv_len=None), NULL, "kv_len"),
    (dict(table=None), NULL, "page_table"),
    (dict(ws=None), NULL, "workspace"),
    (dict(q=A + 8), INVALID, "16-byte"),
    (dict(ost=(260, 64)), INVALID, "16-byte"),
    (dict(ost=(256, 0)), INVALID, "strides"),
    (dict(tree=E + 4), INVALID, "aligned"),
    (dict(lse=G + 1), INVALID, "aligned"),
    (dict(out=A), INVALID, "overlap"),
    (dict(lse=F + 64), INVALID, "overlap"),
    (dict(ws=A, nbytes=64), INVALID, "overlap"),
    (dict(out=V), INVALID, "overlap"),
    (dict(lse=B), INVALID, "overlap"),
])
def test_attention_refusals(lib, kw, status, needle):
    assert attend(lib, cache(), **kw) == status
    assert needle in message(lib)


@pytest.mark.parametrize("c,needle", [
    (dict(store=1), "type of q"),
    (dict(kd=72, vd=64), "multiples of 16"),
    (dict(kd=272, vd=64), "256"),
    (dict(kd=64, vd=128), "v_dim"),
    (dict(kd=64, vd=0), "v_dim"),
    (dict(k=K + 8), "16-byte"),
])
def test_attention_over_caches_it_does_not_take(lib, c, needle):
    assert attend(lib, cache(**c)) == INVALID
    assert needle in message(lib)


def test_attention_empty_calls(lib):
    assert attend(lib, cache(), Tq=0, q=None, out=None, ws=None) == OK
    assert attend(lib, cache(), R=0, q=None) == OK


def test_workspace_without_a_gpu(lib):
    n = I64()
    sizes = []
    for max_q in (1, 4, 8, 64, 200):
        assert lib.rope_partial_tree_attention_workspace(ctypes.byref(cache()), 0, 8, max_q, 152, ctypes.byref(n)) == OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert lib.rope_partial_tree_attention_workspace(ctypes.byref(cache()), 0, 8, 0, 152, ctypes.byref(n)) == INVALID
    assert lib.rope_partial_tree_attention_workspace(ctypes.byref(cache()), 0, 8, 1, -1, ctypes.byref(n)) == INVALID
    assert lib.rope_partial_tree_attention_workspace(ctypes.byref(cache()), 0, 8, 1, 1, None) == NULL


# ---------------------------------------------------------------- the tree mask


def test_tree_mask_against_ancestors():
    rng = np.random.default_rng(0)
    for n in (1, 2, 63, 64, 65, 200):
        parents = [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
        words = binding.rope_partial_tree_mask(parents).numpy()
        assert words.shape == (n, (n + 63) // 64)
        for i in range(n):
            want, j = set(), i
            while j >= 0:
                want.add(j)
                j = parents[j]
            got = {j for j in range(n) if int(words[i, j // 64]) >> (j % 64) & 1}
            assert got == want


def test_tree_mask_refusals(lib):
    for parents in ([0], [-1, 1], [-2], [-1, 0, 5]):
        with pytest.raises(binding.RopeError, match="parent"):
            binding.rope_partial_tree_mask(parents)
    p = (ctypes.c_int32 * 65)(*([-1] * 65))
    w = (I64 * 65)()
    assert lib.rope_partial_tree_mask(p, 65, 1, w) == INVALID
    assert lib.rope_partial_tree_mask(None, 1, 1, w) == NULL
    assert lib.rope_partial_tree_mask(None, 0, 0, None) == OK
    assert binding.rope_partial_tree_mask([]).shape == (0, 1)


# ---------------------------------------------------------------- the binding's checks (CPU tensors are refused)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 8)
    pos = torch.zeros(2, 1, 2, dtype=torch.int32)
    with pytest.raises(binding.RopeError, match="CUDA"):
        binding.rope_partial_inplace_fwd_axes(x, pos, (2, 2), 0, 8)
    with pytest.raises(binding.RopeError, match="CUDA"):
        binding.KVCache(torch.zeros(2, 4, 1, 16, dtype=torch.bfloat16))
    with pytest.raises(binding.RopeError, match="4-D"):
        binding.rope_partial_inplace_fwd_axes(x[0], pos, (2, 2), 0, 8)
    with pytest.raises(binding.RopeError, match="dtype"):
        binding.KVCache(torch.zeros(2, 4, 1, 16, dtype=torch.int16))


def test_operator_refuses_bad_arguments():
    x = torch.zeros(1, 2, 3, 8, device="meta")
    pos = torch.zeros(2, 1, 2, dtype=torch.int32, device="meta")
    torch_op.inplace_axes_rotary_mul(x, pos, (2, 2), partial_slice=[0, 8])  # the Meta kernel
    for kw, sections in ((dict(order="up"), (2, 2)), (dict(spectrum="x"), (2, 2)), (dict(rotary_mode="q"), (2, 2)),
                         (dict(partial_slice=[0]), (2, 2)), ({}, (2, 1, 1))):
        with pytest.raises(ValueError):
            torch_op.inplace_axes_rotary_mul(x, pos, sections, **kw)
    with pytest.raises(NotImplementedError):  # no CPU kernel
        torch_op.inplace_axes_rotary_mul(torch.zeros(1, 2, 3, 8), torch.zeros(2, 1, 2, dtype=torch.int32), (2, 2),
                                         partial_slice=[0, 8])
