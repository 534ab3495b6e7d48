"""The C ABI of the norm and rotation without a GPU: what a call refuses (no CUDA call
is made for it, so made-up device addresses will do), and the operator's Meta kernel."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from place_partial_rope_gb300 import binding, torch_op

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rope_step.h")
OK, NULL, INVALID = 0, 1, 2
QX, QO, QG, QW, QR, QD, KX, KO, KG, KW, KR, KD, COS, SIN, WS = (0x10000000 + (i << 36) for i in range(15))
B, S, NQ, NK, D = 2, 3, 4, 2, 64


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def message(lib):
    return lib.rope_last_error_message().decode()


def test_header_names_are_exported_and_it_is_c(lib, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(rope_partial_[a-z_]+)\s*\(", text))
    assert {"rope_partial_norm_fwd", "rope_partial_norm_bwd", "rope_partial_norm_workspace"} <= names
    for n in names:
        assert hasattr(lib, n), n
    src = tmp_path / "h.c"
    src.write_text('#include "rope_step.h"\nint main(void) { return (int)sizeof(rope_norm_rows_t); }\n')
    subprocess.run([shutil.which("gcc"), "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "h")], check=True)
    assert subprocess.run([str(tmp_path / "h")]).returncode == 128


def rows(x, out, grad, weight, rstd, dw, heads, xs=None, os_=None, gs=None, D=D, S=S):
    dense = (S * heads * D, heads * D, D)
    return binding._pack_rows(x, out, grad, weight, rstd, dw, heads, *(xs or dense), *(os_ or dense), *(gs or dense))


def call(lib, fn, q=None, k=None, dtype=0, wtype=0, B=B, S=S, D=D, n0=0, n1=None, eps=1e-6, cos=COS, sin=SIN,
         cst=(S * 64, 64), sst=(S * 64, 64), start=0, end=64, mode=1, ws=WS, wsn=1 << 40, no_k=False):
    q = {} if q is None else q
    k = {} if k is None else k
    qa = dict(x=QX, out=QO, grad=QG, weight=QW, rstd=QR, dw=QD, heads=NQ)
    ka = dict(x=KX, out=KO, grad=KG, weight=KW, rstd=KR, dw=KD, heads=NK)
    qa.update(q)
    ka.update(k)
    i2 = ctypes.c_int64 * 2
    tab = (cos, sin, None if cst is None else i2(*cst), None if sst is None else i2(*sst), start, end, mode)
    head = (rows(**qa), None if no_k else rows(**ka), dtype, wtype, B, S, D, n0, D if n1 is None else n1)
    if fn == "fwd":
        return lib.rope_partial_norm_fwd(*head, eps, *tab, None)
    return lib.rope_partial_norm_bwd(*head, *tab, ws, wsn, None)


FAULTS = [
    (dict(dtype=7), INVALID, "dtype"),
    (dict(wtype=1), INVALID, "weight_dtype"),
    (dict(mode=3), INVALID, "mode"),
    (dict(B=-1), INVALID, "sizes"),
    (dict(B=1 << 31), INVALID, "sizes"),
    (dict(B=1 << 16, S=1 << 14), INVALID, "2^31 rows"),
    (dict(D=0, end=0), INVALID, "D=0"),
    (dict(D=1025), INVALID, "D=1025"),
    (dict(n0=-1), INVALID, "normed lanes"),
    (dict(n0=8, n1=8), INVALID, "normed lanes"),
    (dict(n1=65), INVALID, "normed lanes"),
    (dict(start=-2), INVALID, "slice"),
    (dict(end=66), INVALID, "slice"),
    (dict(end=63), INVALID, "even"),
    (dict(cos=0), NULL, "cos"),
    (dict(sst=None), NULL, "strides"),
    (dict(cst=(-1, 64)), INVALID, "cos and sin"),
    (dict(cos=COS + 1), INVALID, "aligned"),
    (dict(q=dict(heads=0)), INVALID, "heads"),
    (dict(q=dict(x=0)), NULL, "q: x"),
    (dict(k=dict(out=0)), NULL, "k: x"),
    (dict(k=dict(x=KX + 1)), INVALID, "aligned"),
    (dict(q=dict(xs=(-1, 256, 64))), INVALID, "strides"),
    (dict(q=dict(os_=(768, 256, 32))), INVALID, "apart"),
    (dict(q=dict(os_=(768, 0, 64))), INVALID, "apart"),
    (dict(k=dict(out=QO + 64)), INVALID, "overlap"),
    (dict(k=dict(out=QX)), INVALID, "overlap"),
    (dict(q=dict(weight=QO + 4)), INVALID, "overlap"),
    (dict(cos=KO + 64), INVALID, "overlap"),
]


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status,needle", FAULTS)
def test_refusals(lib, fn, kw, status, needle):
    assert call(lib, fn, **kw) == status
    assert needle in message(lib)


@pytest.mark.parametrize("fn,kw,status,needle", [
    ("fwd", dict(eps=-1.0), INVALID, "eps"),
    ("fwd", dict(eps=float("nan")), INVALID, "eps"),
    ("fwd", dict(eps=1e300), INVALID, "eps"),
    ("fwd", dict(q=dict(out=QX + 2)), INVALID, "overlap"),          # x, but not as a whole
    ("fwd", dict(q=dict(out=QX, os_=(768, 256, 64), xs=(768, 256, 65))), INVALID, "overlap"),
    ("fwd", dict(q=dict(rstd=QO + 8)), INVALID, "overlap"),
    ("bwd", dict(q=dict(grad=0)), NULL, "grad"),
    ("bwd", dict(k=dict(rstd=0)), NULL, "rstd"),
    ("bwd", dict(q=dict(out=QX)), INVALID, "overlap"),              # backward: out may be grad, not x
    ("bwd", dict(q=dict(dw=QR)), INVALID, "overlap"),
    ("bwd", dict(ws=0), NULL, "workspace"),
    ("bwd", dict(ws=WS + 4), INVALID, "16-byte"),
    ("bwd", dict(ws=KO), INVALID, "overlap"),
])
def test_refusals_of_one_direction(lib, fn, kw, status, needle):
    assert call(lib, fn, **kw) == status
    assert needle in message(lib)


def test_rows_between_each_other_are_told_apart(lib):
    """Queries and keys of one projection, in place or into another: their rows do not
    meet, but one head further they do.  (An empty k grad pointer ends each call on the
    CPU: what is asked is whether an overlap is found first.)"""
    W = (NQ + 2 * NK) * D
    for batch in (S * W, (S + 5) * W):  # the second: batches that do not follow each other
        st = (batch, W, D)
        q = dict(x=QX, out=QX, xs=st, os_=st)
        for shift, hit in ((NQ * D, False), ((NQ - 1) * D, True)):
            at = QX + 2 * shift
            status = call(lib, "fwd", q=q, k=dict(x=at, out=at, xs=st, os_=st), sin=QX, start=0, end=64)
            assert status == INVALID and "overlap" in message(lib)  # (sin lies in q)
        # backward reads x and grad apart: k's grad next to q's, the outs in place
        st2 = dict(gs=st, os_=st)
        for shift, hit in ((NQ * D, False), ((NQ - 1) * D, True)):
            at = QG + 2 * shift
            status = call(lib, "bwd", q=dict(grad=QG, out=QG, **st2), k=dict(grad=at, out=at, **st2), ws=WS, wsn=8)
            assert (status == INVALID and "overlap" in message(lib)) == hit


def test_empty_calls(lib):
    assert call(lib, "fwd", B=0, q=dict(x=0, out=0), k=dict(x=0, out=0), cos=0, sin=0) == OK
    assert call(lib, "bwd", S=0, q=dict(x=0, out=0, grad=0, dw=0), k=dict(x=0, out=0, grad=0, dw=0), cos=0, sin=0,
                ws=0, wsn=0) == OK
    assert message(lib) == ""


def test_workspace_size(lib):
    n = ctypes.c_int64()
    assert lib.rope_partial_norm_workspace(128, 152, ctypes.byref(n)) == OK
    assert n.value == 128 * 4 * 2 * 152 * 8
    assert lib.rope_partial_norm_workspace(0, 152, ctypes.byref(n)) == INVALID
    assert lib.rope_partial_norm_workspace(128, -1, ctypes.byref(n)) == INVALID
    assert lib.rope_partial_norm_workspace(128, 152, None) == NULL


def test_binding_refuses():
    q = torch.empty((1, 2, 3, 8))
    with pytest.raises(binding.RopeError, match="CUDA"):
        binding.rope_partial_norm_fwd(q, None, None, None, None, None, 0, 0)
    with pytest.raises(binding.RopeError, match="4-D"):
        binding.rope_partial_norm_fwd(q[0], None, None, None, None, None, 0, 0)
    with pytest.raises(binding.RopeError, match="dtype"):
        binding.rope_partial_norm_fwd(q.double(), None, None, None, None, None, 0, 0)


def test_meta_kernel():
    torch_op.register()
    q, k = torch.empty((2, 3, 4, 8), device="meta"), torch.empty((2, 3, 1, 8), device="meta")
    out = torch_op.norm_rotary(q, k, None, None, None, None)
    assert out[0].shape == q.shape and out[1].shape == k.shape
    with pytest.raises(ValueError, match="share"):
        torch_op.norm_rotary(q, k[..., :4], None, None, None, None)
    with pytest.raises(ValueError, match="rotary_mode"):
        torch_op.norm_rotary(q, k, None, None, None, None, rotary_mode="both")
    with pytest.raises(ValueError, match="4-D"):
        torch_op.norm_rotary(q[0], None, None, None, None, None)
