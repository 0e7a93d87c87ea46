"""CPU tests of a serving step's entries: sizes, and refusals that come before
any launch (fake device pointers that nothing reads)."""

import ctypes
import math

import pytest

from harness import lib
from position_independent_kv_stitch_gb300 import pic
from test_abi_decode import ALIGNMENT, CAPACITY, INVALID, P, RANGE, _ctx

UNSUPPORTED = 10


@pytest.fixture(scope="module", autouse=True)
def _built():
    lib()


@pytest.fixture
def gqa():
    c = _ctx()
    yield c
    pic.pic_destroy(c)


@pytest.fixture
def mla():
    c = _ctx("mla")
    yield c
    pic.pic_destroy(c)


def _map(ctx, **over):
    t = pic.pic_token_map()
    t.n_req, t.max_blocks, t.n_tokens = 2, 4, 5
    for name, _ in pic.pic_token_map._fields_[3:]:
        setattr(t, name, P)
    ws, size = over.pop("ws", P), over.pop("ws_bytes", 256)
    for name, value in over.items():
        setattr(t, name, value)
    return pic.load().pic_map_tokens(ctx, ctypes.byref(t), ws, size, None)


@pytest.mark.parametrize("over,status", [
    (dict(n_req=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(n_tokens=-1), INVALID), (dict(d_seq_lens=None), INVALID),
    (dict(d_grow=None), INVALID), (dict(d_block_tables=None), INVALID), (dict(d_free_blocks=None), INVALID),
    (dict(d_n_free=None), INVALID), (dict(d_new_n_free=None), INVALID), (dict(d_new_lens=None), INVALID),
    (dict(d_indptr=None), INVALID), (dict(d_req=None), INVALID), (dict(d_slot=None), INVALID), (dict(ws=None), CAPACITY),
    (dict(ws_bytes=255), CAPACITY), (dict(ws=P + 8), ALIGNMENT), (dict(d_seq_lens=P + 2), ALIGNMENT), (dict(d_pos=P + 1), ALIGNMENT),
    (dict(d_shift=P + 2), ALIGNMENT), (dict(d_free_blocks=P + 1), ALIGNMENT),
])
def test_map_refusals(gqa, over, status):
    assert _map(gqa, **over) == status
    assert pic.pic_last_error(gqa)


def test_map_sizes(gqa):
    assert pic.pic_map_tokens_workspace_bytes(gqa, 1000) == pic.PIC_STATUS_BYTES
    assert pic.pic_map_tokens_workspace_bytes(gqa, -1) == 0
    assert pic.load().pic_map_tokens(gqa, None, P, 256, None) == INVALID
    assert pic.load().pic_map_tokens(None, None, P, 256, None) == INVALID


def _write(ctx, mla=False, norms=True, **over):
    t, n = pic.pic_new_tokens(), pic.pic_head_norms()
    t.n_tokens, t.num_q_heads, t.n_axes = 3, 4, 1
    t.d_pos, t.q, t.q_out, t.k, t.d_req, t.d_slot = P, P, P, P, P, P
    t.q_stride = t.q_out_stride = 4 * (1152 if mla else 256)
    t.k_stride = 1152 if mla else 512
    if not mla:
        t.v, t.v_stride = P, 512
    n.q_weight, n.k_weight, n.weight_type, n.eps, n.offset = None if mla else P, P, pic.PIC_BF16, 1e-6, 0.0
    for name, value in over.items():
        setattr(n if hasattr(n, name) else t, name, value)
    return pic.load().pic_write_normed_tokens(ctx, ctypes.byref(t), ctypes.byref(n) if norms else None, P, None if mla else P, P, 2, 4,
                                              None, 0, P, 256, None)


@pytest.mark.parametrize("over,status", [
    (dict(norms=False), INVALID), (dict(weight_type=2), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(offset=math.nan), INVALID), (dict(q_weight=P + 8), ALIGNMENT),
    (dict(k_weight=P + 2), ALIGNMENT), (dict(k_stride=496), RANGE), (dict(n_axes=0), INVALID), (dict(q=P + 8), ALIGNMENT),
])
def test_write_normed_refusals(gqa, over, status):
    assert _write(gqa, **over) == status
    assert pic.pic_last_error(gqa)


def test_write_normed_of_latent_rows(gqa, mla):
    assert _write(mla, mla=True, n_tokens=0) == 0 and _write(gqa, n_tokens=0) == 0
    assert _write(mla, mla=True, q_weight=P) == INVALID


def _attend(ctx, **over):
    a = dict(q=P, q_stride=1024, n=3, hq=4, scale=0.1, k=P, v=P, tables=P, n_req=2, max_blocks=4, indptr=P, slot=P, window=0, first=0,
             out=P, lse=P, ws=P, ws_bytes=1 << 40)
    a.update(over)
    return pic.load().pic_attend_tokens(ctx, a["q"], a["q_stride"], a["n"], a["hq"], a["scale"], a["k"], a["v"], a["tables"], a["n_req"],
                                        a["max_blocks"], a["indptr"], a["slot"], a["window"], a["first"], a["out"], a["lse"], a["ws"],
                                        a["ws_bytes"], None)


def _shared(ctx, **over):
    a = dict(q=P, q_stride=1024, n=3, hq=4, scale=0.1, k=P, v=P, prefix=P, prefix_blocks=3, prefix_len=P, tables=P, max_blocks=4, lens=P,
             max_len=64, out=P, lse=P, ws=P, ws_bytes=1 << 40)
    a.update(over)
    return pic.load().pic_attend_shared(ctx, a["q"], a["q_stride"], a["n"], a["hq"], a["scale"], a["k"], a["v"], a["prefix"],
                                        a["prefix_blocks"], a["prefix_len"], a["tables"], a["max_blocks"], a["lens"], a["max_len"],
                                        a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [_attend, _shared])
@pytest.mark.parametrize("over,status", [
    (dict(hq=3), INVALID), (dict(hq=0), INVALID), (dict(n=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(tables=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(q_stride=1008), RANGE),
    (dict(hq=1 << 17, q_stride=1 << 30), RANGE), (dict(n=2 ** 30), RANGE), (dict(q=P + 2), ALIGNMENT), (dict(q_stride=1032), ALIGNMENT),
    (dict(out=P + 8), ALIGNMENT), (dict(k=P + 8), ALIGNMENT), (dict(lse=P + 2), ALIGNMENT), (dict(tables=P + 1), ALIGNMENT),
    (dict(ws=P + 64), ALIGNMENT), (dict(ws_bytes=255), CAPACITY),
])
def test_attention_refusals(gqa, call, over, status):
    assert call(gqa, **over) == status
    assert pic.pic_last_error(gqa)


@pytest.mark.parametrize("over,status", [
    (dict(n_req=-1), INVALID), (dict(window=-1), INVALID), (dict(first=-1), INVALID), (dict(indptr=None), INVALID),
    (dict(slot=None), INVALID), (dict(indptr=P + 2), ALIGNMENT), (dict(slot=P + 1), ALIGNMENT),
])
def test_attend_tokens_refusals(gqa, over, status):
    assert _attend(gqa, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(prefix_blocks=-1), INVALID), (dict(max_len=-1), INVALID), (dict(max_len=65), RANGE), (dict(prefix=None), INVALID),
    (dict(prefix_len=None), INVALID), (dict(lens=None), INVALID), (dict(prefix=P + 2), ALIGNMENT), (dict(lens=P + 3), ALIGNMENT),
    (dict(prefix_len=P + 1), ALIGNMENT),
])
def test_attend_shared_refusals(gqa, over, status):
    assert _shared(gqa, **over) == status


def test_attention_of_nothing_and_of_latent_rows(gqa, mla):
    assert _attend(gqa, n=0) == 0 and _attend(gqa, n_req=0) == 0 and _shared(gqa, n=0) == 0
    mla_args = dict(hq=16, q_stride=16 * 1152)
    for call in (_attend, _shared):
        assert call(mla, **mla_args) == UNSUPPORTED
        assert call(None) == INVALID
    assert pic.pic_attend_tokens_workspace_bytes(mla, 4, 2, 16) == 0
    assert pic.pic_attend_shared_workspace_bytes(mla, 4, 16) == 0
    for n, hq in ((-1, 4), (4, 3), (4, 0), (2 ** 30, 4), (4, 8192)):
        assert pic.pic_attend_tokens_workspace_bytes(gqa, n, 2, hq) == 0
    assert pic.pic_attend_tokens_workspace_bytes(gqa, 4, -1, 4) == 0
    assert 256 < pic.pic_attend_tokens_workspace_bytes(gqa, 4, 2, 4) < 1 << 30


def test_more_requests_than_the_kernels_count(gqa):
    most = 1 << 30
    assert _map(gqa, n_req=most + 1) == RANGE and _attend(gqa, n_req=most + 1) == RANGE
    assert _map(gqa, n_req=2 ** 31 - 1) == RANGE and _attend(gqa, n_req=2 ** 31 - 1) == RANGE
    assert pic.pic_map_tokens_workspace_bytes(gqa, most + 1) == 0
    assert pic.pic_attend_tokens_workspace_bytes(gqa, 4, most + 1, 4) == 0
    assert pic.pic_map_tokens_workspace_bytes(gqa, most) == pic.PIC_STATUS_BYTES
    assert pic.pic_attend_tokens_workspace_bytes(gqa, 4, most, 4) > 256
