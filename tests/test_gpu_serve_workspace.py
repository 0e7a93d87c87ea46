"""One workspace, made for a loop's largest call, serves all its smaller ones, and no
call writes behind the bytes that its size asks for."""

import numpy as np
import pytest
import torch

import test_gpu_serve as serving
from position_independent_kv_stitch_gb300 import pic
from test_gpu_decode import DEV, Cache, _i32, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pic.load(build_if_missing=True)


def _attend(c, slots, hq, ws):
    counts = [len(x) for x in slots]
    q = c.normal(sum(counts), hq, c.d)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
    pic.pic_attend_tokens(c.ctx, q, c.d ** -0.5, c.k[0], c.v[0], c.d_tables[:len(slots)], _i32(np.concatenate([[0], np.cumsum(counts)])),
                          _i32([s for x in slots for s in x]), out, lse=lse, workspace=ws)
    return q, out, lse


def _shared(c, n, hq, ws):
    q = c.normal(n, hq, c.d)
    out = torch.full_like(q, 7.0)
    pic.pic_attend_shared(c.ctx, q, c.d ** -0.5, c.k[0], c.v[0], _i32(c.prefix_table), _i32([c.prefix]), c.d_tables[:n], _i32(c.lens[:n]),
                          max(c.lens), out, workspace=ws)
    return q, out


def _check(c, q, out, lse, slots, at, r):
    rows = [serving._wide_rows(x[0], c.tables[r], np.arange(c.lens[r]), c.bs) for x in (c.k, c.v)]
    seen = torch.from_numpy(np.stack([np.arange(c.lens[r]) <= s for s in slots[r]])).to(DEV)
    a = slice(at, at + len(slots[r]))
    serving._assert_rows(q[a], *rows, seen, c.d ** -0.5, out[a], lse[a], (len(slots), r))


@pytest.mark.parametrize("hq", [8, 32])
def test_tokens_of_smaller_batches(hq):
    """A workspace for 300 tokens of 40 requests: fewer tokens, fewer requests, prompts that are split and that are not."""
    c = Cache(heads=8, d=128, lens=[3000, 1200] + [50] * 38, seed=hq)
    ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, 300, 40, hq))
    heads = lambda n, m: list(range(m - n, m))  # noqa: E731
    for slots in ([heads(260, 3000)] + [[1199]] + [[49]] * 38, [heads(256, 3000)], [heads(64, 3000)], [heads(65, 3000)], [heads(17, 3000), heads(33, 1200)],
                  [[2999]], [[2999], [1199]] + [[49]] * 30, [heads(2, 3000)], [heads(129, 3000), [1199], [49]]):
        got = _attend(c, slots, hq, ws)
        _check(c, *got, slots, 0, 0)
        if len(slots) > 1:
            _check(c, *got, slots, len(slots[0]), 1)
    assert pic.pic_query_device_status(c.ctx, ws) == 0
    c.close()


def test_shared_prefixes_of_smaller_batches():
    """A workspace for 65 requests, of which some end."""
    c = serving.Shared(9001, [3 * r % 50 for r in range(65)], heads=8, d=64, seed=1)
    ws = _ws(pic.pic_attend_shared_workspace_bytes(c.ctx, 65, 32))
    clean = {n: _shared(c, n, 32, _ws(pic.pic_attend_shared_workspace_bytes(c.ctx, n, 32))) for n in (65, 64, 36, 5, 1)}
    for n, (q, want) in clean.items():
        out = torch.full_like(q, 7.0)
        pic.pic_attend_shared(c.ctx, q, c.d ** -0.5, c.k[0], c.v[0], _i32(c.prefix_table), _i32([c.prefix]), c.d_tables[:n], _i32(c.lens[:n]),
                              max(c.lens), out, workspace=ws)
        assert torch.equal(out, want), n
    assert pic.pic_query_device_status(c.ctx, ws) == 0
    c.close()


@pytest.mark.parametrize("heads,hq,d", [(8, 32, 128), (1, 3, 64), (2, 40, 256), (5, 5, 128)])
def test_nothing_is_written_behind_a_workspace(heads, hq, d):
    """The bytes asked for, followed by others that stay."""
    c = Cache(heads=heads, d=d, lens=[9000, 9000], seed=hq)

    def inside(size):
        buf = torch.full((size + (8 << 20),), 0x5a, dtype=torch.uint8, device=DEV)
        buf[:pic.PIC_STATUS_BYTES] = 0
        return buf[:size], buf[size:]

    for counts in ([1], [1, 1], [2], [20], [64], [65, 1], [150, 150], [300], [600, 3]):
        ws, behind = inside(pic.pic_attend_tokens_workspace_bytes(c.ctx, sum(counts), len(counts), hq))
        _attend(c, [list(range(9000 - n, 9000)) for n in counts], hq, ws)
        assert bool((behind == 0x5a).all()) and pic.pic_query_device_status(c.ctx, ws) == 0, counts
    c.close()
    for n in (1, 2, 20, 64, 65):
        c = serving.Shared(9000, [7] * n, heads=heads, d=d, seed=n)
        ws, behind = inside(pic.pic_attend_shared_workspace_bytes(c.ctx, n, hq))
        _shared(c, n, hq, ws)
        assert bool((behind == 0x5a).all()) and pic.pic_query_device_status(c.ctx, ws) == 0, n
        c.close()
