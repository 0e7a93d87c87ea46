"""CPU tests of the workspace sizes of a serving step's attentions."""

import pytest

from harness import lib
from position_independent_kv_stitch_gb300 import pic

MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    lib()


def _ctx(heads, d, blocks=1000, bs=16):
    return pic.pic_create(pic.PIC_KIND_GQA, 1, heads, d, d, 0, pic.PIC_PAIRING_NEOX_HALF, bs, 5e5, blocks)


@pytest.mark.parametrize("heads,hq,d", [(8, 32, 128), (8, 8, 128), (2, 16, 64), (4, 32, 256)])
@pytest.mark.parametrize("n_req", [1, 3, 256])
def test_prompts_do_not_take_a_record_per_token(heads, hq, d, n_req):
    """Records are kept for the requests' single tokens, and for tiles where their slots are split: a longer prompt,
    whose tiles fill the SMs, takes no more."""
    c = _ctx(heads, d)
    long, longer = (pic.pic_attend_tokens_workspace_bytes(c, n, n_req, hq) for n in (16384, 131072))
    assert 0 < longer <= long
    # two rounds of 256 SMs, a row block of 256 rows to each, in as many parts as fill a third; 64 ranges an SM and a row
    # for each request of the row-by-row kernel
    assert long <= 4 * 256 * 256 * (4 * d + 8) + (64 * 256 // heads + n_req) * hq * (4 * d + 8) + 8 * n_req + 4096
    pic.pic_destroy(c)


@pytest.mark.parametrize("heads,d", [(8, 128), (1, 64), (2, 256), (3, 128), (19, 64)])
@pytest.mark.parametrize("blocks", [1000, 0])
def test_a_workspace_serves_smaller_calls(heads, d, blocks):
    """Sizes never fall with more tokens, requests or query heads."""
    c = _ctx(heads, d, blocks)
    counts = list(range(1, 20)) + [31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 200, 255, 256, 257, 511, 512, 513, 1000, 4095, 4096, 4097, 70000]
    groups = [1, 2, 3, 4, 7, 8, 15, 16, 17, 32, 33, 48, 49, 64, 200]
    size = pic.pic_attend_tokens_workspace_bytes
    for group in groups:
        for n in counts:
            by_requests = [size(c, n, r, heads * group) for r in counts]
            assert by_requests == sorted(by_requests), (group, n)
        for r in counts:
            by_tokens = [size(c, n, r, heads * group) for n in counts]
            assert by_tokens == sorted(by_tokens), (group, r)
        shared = [pic.pic_attend_shared_workspace_bytes(c, r, heads * group) for r in counts]
        assert shared == sorted(shared), group
    for n in counts:
        for r in (1, 64, 256, 4096):
            by_heads = [size(c, n, r, heads * group) for group in groups]
            assert by_heads == sorted(by_heads), (n, r)
        by_heads = [pic.pic_attend_shared_workspace_bytes(c, n, heads * group) for group in groups]
        assert by_heads == sorted(by_heads), n
    pic.pic_destroy(c)


def test_of_a_cache_without_blocks_every_token_has_a_record():
    c = _ctx(2, 64, blocks=0)
    assert pic.pic_attend_tokens_workspace_bytes(c, 5000, 1, 4) >= 5000 * 4 * 64 * 4
    pic.pic_destroy(c)
