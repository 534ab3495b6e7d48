"""What the calls that deal out pages refuse, without a GPU."""
import pytest
import torch

from place_partial_rope_gb300 import binding

OK, NULL, INVALID = 0, 1, 2
LEN, N, TAB, FREE, COUNT, QS, SLOTS, POS, OKS = (0x10000000 + (i << 36) for i in range(9))


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def message(lib):
    return lib.rope_last_error_message().decode()


def grow(lib, ln=LEN, n=N, R=4, tab=TAB, pages=8, stride=8, free=FREE, cap=100, count=COUNT, page=16, qs=QS,
         slots=SLOTS, pos=POS, T=50, ok=OKS):
    return lib.rope_partial_cache_grow(ln, n, R, tab, pages, stride, free, cap, count, page, qs, slots, pos, T, ok, None)


def trim(lib, ln=LEN, n=N, R=4, tab=TAB, pages=8, stride=8, free=FREE, cap=100, count=COUNT, page=16):
    return lib.rope_partial_cache_trim(ln, n, R, tab, pages, stride, free, cap, count, page, None)


BOTH = [
    (dict(R=-1), INVALID, "R=-1"),
    (dict(R=1 << 24), INVALID, "requests"),
    (dict(page=0), INVALID, "page_size"),
    (dict(pages=-1), INVALID, "pages"),
    (dict(pages=1 << 28, stride=1 << 28), INVALID, "2^31"),
    (dict(stride=7), INVALID, "page_table_stride"),
    (dict(cap=-1), INVALID, "free_capacity"),
    (dict(cap=1 << 31), INVALID, "free_capacity"),
    (dict(ln=0), NULL, "kv_len"),
    (dict(n=0), NULL, "kv_len"),
    (dict(tab=0), NULL, "page_table"),
    (dict(free=0), NULL, "free_pages"),
    (dict(count=0), NULL, "free_count"),
    (dict(ln=LEN + 2), INVALID, "aligned"),
    (dict(n=LEN), INVALID, "overlap"),
    (dict(n=TAB + 4 * (3 * 8 + 7)), INVALID, "overlap"),
    (dict(count=FREE + 4 * 99), INVALID, "overlap"),
]


@pytest.mark.parametrize("call", [grow, trim])
@pytest.mark.parametrize("kw,status,needle", BOTH)
def test_refusals(lib, call, kw, status, needle):
    assert call(lib, **kw) == status
    assert needle in message(lib)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "tokens"),
    (dict(T=1 << 31), INVALID, "tokens"),
    (dict(qs=0), NULL, "q_start"),
    (dict(slots=0), NULL, "slots"),
    (dict(slots=SLOTS + 4), INVALID, "slots"),
    (dict(pos=SLOTS + 8 * 49), INVALID, "overlap"),
    (dict(ok=QS + 16), INVALID, "overlap"),
    (dict(qs=LEN + 12), INVALID, "overlap"),
])
def test_refusals_of_grow(lib, kw, status, needle):
    assert grow(lib, **kw) == status
    assert needle in message(lib)


def test_no_requests_to_trim(lib):
    assert trim(lib, R=0, ln=0, n=0, tab=0) == OK


def test_binding_refuses():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(binding.RopeError, match="CUDA"):
        binding.rope_partial_cache_trim(i32(2), i32(2), i32(2, 3), i32(5), i32(1), 16)
    with pytest.raises(binding.RopeError, match="int32"):
        binding.rope_partial_cache_trim(i32(2).long(), i32(2), i32(2, 3), i32(5), i32(1), 16)
