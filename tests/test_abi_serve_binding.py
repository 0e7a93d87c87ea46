"""What the Python calls of a serving step's attentions refuse before the library is called (CPU tensors)."""

import pytest
import torch

from harness import lib
from position_independent_kv_stitch_gb300 import pic


@pytest.fixture(scope="module", autouse=True)
def _built():
    lib()


@pytest.fixture
def call():
    c = pic.pic_create(pic.PIC_KIND_GQA, 1, 2, 64, 64, 0, pic.PIC_PAIRING_NEOX_HALF, 16, 1e4, 4)
    cache, q = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    tables = torch.zeros(2, 2, dtype=torch.int32)
    yield {
        "tokens": lambda **kw: pic.pic_attend_tokens(c, q, 0.1, cache, cache, tables, i32(0, 1, 2), i32(0, 1), q.clone(), **kw),
        "shared": lambda n=32: pic.pic_attend_shared(c, q, 0.1, cache, cache, i32(0), i32(1), tables, i32(1, 2), n, q.clone()),
    }
    pic.pic_destroy(c)


@pytest.mark.parametrize("name", ["window", "n_first"])
@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1, 1 << 70])
def test_numbers_of_more_than_32_bits(call, name, n):
    """A window of 2^32 + 5 would be one of 5."""
    with pytest.raises(ValueError, match=f"{name}.*32 bits"):
        call["tokens"](**{name: n})


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 32])
def test_a_longest_sequence_of_more_than_32_bits(call, n):
    with pytest.raises(ValueError, match="max_seq_len.*32 bits"):
        call["shared"](n)


def test_others_come_to_the_device_check(call):
    for go in (lambda: call["tokens"](window=(1 << 31) - 1, n_first=0), lambda: call["shared"](32)):
        with pytest.raises(ValueError, match="CUDA device"):
            go()
