"""Which table entry a bad block is reported for: the request's row of the block tables and a slot in
the block, or row -1 for the table of a shared prefix."""

import numpy as np
import pytest

import test_gpu_serve as serving
from position_independent_kv_stitch_gb300 import pic
from test_gpu_decode import Cache, _i32, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pic.load(build_if_missing=True)


def _reported(c, ws, row, block):
    with pytest.raises(pic.PicError, match=rf"table row {row}[ ,]"):
        pic.pic_query_device_status(c.ctx, ws)
    status, at, slot = ws[:12].view(dtype=_i32([0]).dtype).tolist()
    assert (status, at, slot // c.bs) == (pic.PIC_DEV_BAD_BLOCK, row, block)


@pytest.mark.parametrize("counts,bad", [
    ([0, 1, 0, 1], 3),          # row by row, requests without tokens ahead
    ([0, 0, 3, 0, 0, 1], 2),    # several tokens of a request, row by row
    ([0, 5, 40], 2),            # tiles
    ([0, 40, 0, 1], 3),         # a single token beside tiles
    ([0, 0, 200], 2),
])
@pytest.mark.parametrize("block", [0, 4])
def test_tokens(counts, bad, block):
    c = Cache(heads=2, bs=16, lens=[250] * len(counts), seed=len(counts))
    tables = c.d_tables.clone()
    tables[bad, block] = c.nb
    q = c.normal(sum(counts), 8, 128)
    ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, len(q), len(counts), 8))
    pic.pic_attend_tokens(c.ctx, q, 0.1, c.k[0], c.v[0], tables, _i32(np.concatenate([[0], np.cumsum(counts)])),
                          _i32([s for n in counts for s in range(250 - n, 250)]), q.clone(), workspace=ws)
    _reported(c, ws, bad, block)
    c.close()


@pytest.mark.parametrize("columns", [10, 3000])    # row by row, and in tiles
@pytest.mark.parametrize("row", [-1, 1, 2])
def test_shared(columns, row):
    c = serving.Shared(100, [5] * 40, heads=8, seed=5)
    prefix = np.concatenate([c.prefix_table, np.zeros(columns - len(c.prefix_table), np.int32)])
    tables = c.d_tables.clone()
    if row < 0:
        prefix[2] = c.nb
    else:
        tables[row, 6] = -1
    q = c.normal(40, 32, 128)
    ws = _ws(pic.pic_attend_shared_workspace_bytes(c.ctx, 40, 32))
    pic.pic_attend_shared(c.ctx, q, 0.1, c.k[0], c.v[0], _i32(prefix), _i32([100]), tables, _i32(c.lens), max(c.lens), q.clone(), workspace=ws)
    _reported(c, ws, row, 2 if row < 0 else 6)
    c.close()
