"""Prompts and single tokens in one call: chunks whose slots are split over several
CTAs beside many requests of a token, and captured calls whose offsets change between
replays, so that requests move from the one kernel to the other."""

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


@pytest.mark.parametrize("heads,hq,d", [(2, 8, 128), (1, 8, 64), (1, 4, 256)])
@pytest.mark.parametrize("window,n_first", [(0, 0), (9000, 100)])
def test_a_split_chunk_beside_single_tokens(heads, hq, d, window, n_first):
    """(2 KV heads, 101 requests: 206 CTAs at most, so two parts or more on 152 SMs.)"""
    rng = np.random.default_rng(hq)
    lens = rng.integers(1, 600, size=101).tolist()
    lens[40] = 20011
    c = Cache(heads=heads, d=d, lens=lens, seed=hq)
    slots = [[n - 1] if r % 9 else [] for r, n in enumerate(lens)]
    slots[40] = list(range(20011 - 70, 20011))
    slots[7] = [-1]
    serving._attend(c, slots, hq, window, n_first, pad=4, check=[40, 41, 39] + list(range(0, 101, 7)))
    c.close()


@pytest.mark.parametrize("n,n_req", [(200, 6), (6, 6)])
@pytest.mark.parametrize("window,n_first", [(0, 0), (300, 5)])
def test_captured_offsets_change(n, n_req, window, n_first):
    """One graph: a chunk of one request, then of another, then single tokens, then nothing."""
    lens = [700, 40, 9000, 1, 333, 129]
    c = Cache(heads=2, lens=lens, seed=n)
    q = c.normal(n, 8, 128)
    indptr, slot = _i32([0] * (n_req + 1)), _i32([0] * n)
    out, lse = torch.empty_like(q), torch.empty(n, 8, device=DEV)
    ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, n, n_req, 8))

    def attend():
        pic.pic_attend_tokens(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, indptr, slot, out, window=window, n_first=n_first, lse=lse,
                              workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            attend()
    torch.cuda.current_stream().wait_stream(side)
    most = n - 5
    for counts in ([1, 1, most, 1, 1, 1], [min(most, 190), 0, 0, 1, 1, 1], [1] * 6, [0] * 6, [0, 0, 0, 0, 0, 1], [0, min(n - 1, 40), 1, 0, 0, 0]):
        slots = [list(range(m - k, m)) for m, k in zip(lens, counts)]
        indptr.copy_(_i32(np.concatenate([[0], np.cumsum(counts)])))
        slot.copy_(_i32([s for x in slots for s in x] + [5] * (n - sum(counts))))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for r, x in enumerate(slots):
            a = slice(at, at + len(x))
            at += len(x)
            if not x:
                continue
            seen = np.stack([serving.serve.sees(s, np.arange(lens[r]), window, n_first) for s in x])
            rows = (serving._wide_rows(t[0], c.tables[r], np.arange(lens[r]), c.bs) for t in (c.k, c.v))
            serving._assert_rows(q[a], *rows, torch.from_numpy(seen).to(DEV), 128 ** -0.5, out[a], lse[a], (counts, r))
        assert bool((out[at:] == 7.0).all()) and bool((lse[at:] == 7.0).all())   # rows behind the last request's
    assert pic.pic_query_device_status(c.ctx, ws) == 0
    c.close()
