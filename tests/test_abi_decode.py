"""CPU tests of the decode-loop entries: sizes, and refusals that come before
any launch (fake device pointers that nothing reads)."""

import ctypes

import pytest

from harness import lib
from position_independent_kv_stitch_gb300 import pic

INVALID, CAPACITY, RANGE, ALIGNMENT = 1, 5, 6, 7
P = 0x10000   # a 256-byte aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def _built():
    lib()


def _ctx(kind="gqa", layers=2, heads=2, d=128, bs=16, nb=64):
    if kind == "gqa":
        return pic.pic_create(pic.PIC_KIND_GQA, layers, heads, d, d, 0, pic.PIC_PAIRING_NEOX_HALF, bs, 1e4, nb)
    return pic.pic_create(pic.PIC_KIND_MLA, layers, 1, 576, 64, 512, pic.PIC_PAIRING_INTERLEAVED, bs, 1e4, nb)


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


def _write(ctx, mla=False, **over):
    t = pic.pic_new_tokens()
    t.n_tokens, t.num_q_heads, t.n_axes = 3, 4, 1
    t.d_pos, t.q, t.q_out, t.k, t.d_req, t.d_slot = P, P, P, P, P, P
    t.q_stride = t.q_out_stride = 4 * (1152 if mla else 256)
    t.k_stride = 1152 if mla else 512
    if not mla:
        t.v, t.v_stride = P, 512
    args = dict(k_cache=P, v_cache=None if mla else P, tables=P, n_tables=2, max_blocks=4, weights=P, heads=1, ws=P,
                ws_bytes=256)
    for name, value in over.items():
        if name in args:
            args[name] = value
        else:
            setattr(t, name, value)
    return pic.load().pic_write_tokens(ctx, ctypes.byref(t), args["k_cache"], args["v_cache"], args["tables"],
                                       args["n_tables"], args["max_blocks"], args["weights"], args["heads"], args["ws"],
                                       args["ws_bytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(n_tokens=-1), INVALID), (dict(num_q_heads=-1), INVALID), (dict(n_axes=0), INVALID), (dict(n_axes=5), INVALID),
    (dict(freq_axis=bytes([0] * 63 + [1])), INVALID), (dict(ws=None), CAPACITY), (dict(ws_bytes=255), CAPACITY),
    (dict(num_q_heads=0, k=None, v=None), INVALID), (dict(d_pos=None), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(v=None), INVALID), (dict(k=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(tables=None), INVALID), (dict(d_req=None), INVALID), (dict(d_slot=None), INVALID),
    (dict(n_tables=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(heads=3), INVALID), (dict(heads=0), INVALID),
    (dict(q_stride=1008), RANGE), (dict(q_out_stride=0), RANGE), (dict(k_stride=496), RANGE), (dict(v_stride=256), RANGE),
    (dict(num_q_heads=1 << 24, q_stride=1 << 40, q_out_stride=1 << 40), RANGE),
    (dict(n_tokens=2 ** 31 - 1, num_q_heads=0, k_stride=496), RANGE), (dict(q_stride=2048), INVALID), (dict(q_out_stride=2048), INVALID),
    (dict(q=P + 8), ALIGNMENT), (dict(k_stride=520), ALIGNMENT), (dict(v_cache=P + 2), ALIGNMENT), (dict(d_slot=P + 1), ALIGNMENT),
    (dict(ws=P + 16), ALIGNMENT), (dict(weights=P + 2), ALIGNMENT),
])
def test_write_refusals(gqa, over, status):
    assert _write(gqa, **over) == status
    assert pic.pic_last_error(gqa)


def test_write_nothing_is_fine_and_mla_takes_no_values(gqa, mla):
    assert _write(gqa, n_tokens=0) == 0
    assert _write(mla, mla=True, n_tokens=0) == 0
    assert _write(mla, mla=True, v=P, v_stride=1152) == INVALID
    assert pic.load().pic_write_tokens(None, None, P, P, P, 1, 1, None, 0, P, 256, None) == INVALID


def _attend(ctx, **over):
    a = dict(q=P, q_stride=1024, n_req=2, hq=4, scale=0.1, k=P, v=P, tables=P, max_blocks=4, lens=P, max_len=64, out=P, type=0,
             lse=P, weights=None, heads=0, ws=P, ws_bytes=1 << 40)
    a.update(over)
    return pic.load().pic_attend_paged(ctx, a["q"], a["q_stride"], a["n_req"], a["hq"], a["scale"], a["k"], a["v"], a["tables"],
                                       a["max_blocks"], a["lens"], a["max_len"], a["out"], a["type"], a["lse"], a["weights"],
                                       a["heads"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(hq=3), INVALID), (dict(hq=0), INVALID), (dict(hq=-2), INVALID), (dict(n_req=-1), INVALID), (dict(max_blocks=-1), INVALID),
    (dict(max_len=-1), INVALID), (dict(type=2), INVALID), (dict(weights=P, heads=3), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(tables=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q_stride=1008), RANGE), (dict(max_len=65), RANGE),
    (dict(hq=1 << 17, q_stride=1 << 30), RANGE), (dict(q=P + 2), ALIGNMENT), (dict(q_stride=1032), ALIGNMENT),
    (dict(out=P + 4), ALIGNMENT), (dict(lens=P + 2), ALIGNMENT), (dict(ws=P + 64), ALIGNMENT), (dict(ws_bytes=1000), CAPACITY),
])
def test_attend_refusals(gqa, over, status):
    assert _attend(gqa, **over) == status
    assert pic.pic_last_error(gqa)


def test_a_cache_without_blocks_holds_no_sequence():
    c = _ctx(nb=0)
    assert _attend(c, max_len=1) == RANGE and _attend(c, max_len=0, n_req=0) == 0
    pic.pic_destroy(c)


def test_attend_sizes(gqa, mla):
    assert _attend(mla, hq=16, q_stride=16 * 1152, n_req=0, v=None) == 0
    assert _attend(mla, hq=16, q_stride=16 * 1152 - 16) == RANGE
    assert _attend(gqa, n_req=0) == 0
    bare = pic.pic_attend_paged_workspace_bytes(gqa, 2, 4, 64)
    kept = pic.pic_attend_paged_workspace_bytes(gqa, 2, 4, 64, True)
    # the scores of 2 x 64 slots under 4 heads, and their log-sum-exps
    assert 256 < bare and bare + 2 * 64 * 4 * 4 <= kept <= bare + 2 * 64 * 4 * 4 + 1024
    assert _attend(gqa, ws_bytes=bare - 1) == CAPACITY and _attend(gqa, ws_bytes=kept - 1, weights=P, heads=1) == CAPACITY
    for bad in ((gqa, -1, 4, 64), (gqa, 2, 3, 64), (gqa, 2, 4, -1), (mla, 2, 0, 64), (None, 2, 4, 64)):
        assert pic.load().pic_attend_paged_workspace_bytes(*bad, 0) == 0


def _evict(ctx, **over):
    a = dict(layers=2, k=P, v=P, cls=64 * 16 * 512, weights=P, wls=64 * 16 * 8, heads=2, tables=P, n_req=2, max_blocks=4, lens=P,
             budget=8, first=1, recent=2, renumber=0, kept=P, new=P, ws=P, ws_bytes=1 << 40)
    a.update(over)
    return pic.load().pic_evict_tokens(ctx, a["layers"], a["k"], a["v"], a["cls"], a["weights"], a["wls"], a["heads"], a["tables"],
                                       a["n_req"], a["max_blocks"], a["lens"], a["budget"], a["first"], a["recent"],
                                       a["renumber"], a["kept"], a["new"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(n_req=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(layers=0), RANGE), (dict(layers=3), RANGE),
    (dict(heads=3), INVALID), (dict(budget=0), INVALID), (dict(first=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(first=4, recent=5), INVALID), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(weights=None), INVALID), (dict(tables=None), INVALID), (dict(lens=None), INVALID),
    (dict(kept=None), INVALID), (dict(new=None), INVALID), (dict(ws=None), INVALID), (dict(cls=64 * 16 * 512 - 16), RANGE),
    (dict(wls=64 * 16 * 8 - 4), RANGE), (dict(k=P + 8), ALIGNMENT), (dict(cls=64 * 16 * 512 + 8), ALIGNMENT),
    (dict(wls=64 * 16 * 8 + 2), ALIGNMENT), (dict(kept=P + 2), ALIGNMENT), (dict(ws=P + 32), ALIGNMENT), (dict(ws_bytes=256), CAPACITY),
])
def test_evict_refusals(gqa, over, status):
    assert _evict(gqa, **over) == status
    assert pic.pic_last_error(gqa)


def test_evict_sizes(gqa, mla):
    assert _evict(gqa, n_req=0) == 0
    assert _evict(mla, n_req=0, v=None, heads=1, cls=64 * 16 * 1152) == 0
    need = pic.pic_evict_workspace_bytes(gqa, 2, 3, 2)
    assert need >= 256 + 3 * 4 + 2 * 3 * 2 * 8
    assert _evict(gqa, n_req=3, ws_bytes=need - 1) == CAPACITY
    for bad in ((None, 2, 3, 2), (gqa, 0, 3, 2), (gqa, 2, -1, 2), (gqa, 2, 3, 3)):
        assert pic.load().pic_evict_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors_and_foreign_shapes(gqa):
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(64, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pic.pic_write_tokens(gqa, i, cache[0, :2], cache[0, :2], i, i, i.view(1, 2), cache, cache)
    with pytest.raises(ValueError):
        pic.pic_write_tokens(gqa, i, None, None, None, None, None, None, None, q=cache[0, :2])
    with pytest.raises(ValueError):
        pic.pic_write_tokens(gqa, i, cache[0, :2], cache[0, :2], None, i, i.view(1, 2), cache, cache)
    with pytest.raises(ValueError):
        pic.pic_attend_paged(gqa, cache[0, :2], 1.0, cache, cache, i.view(2, 1), i, 16, torch.empty(2, 2, 128))
    with pytest.raises(ValueError):
        pic.pic_evict_tokens(gqa, cache[None], cache[None], torch.zeros(1, 64, 2, 16), i.view(2, 1), i, 4, i, i)
    for bad in (cache[:63], cache.float(), cache[:, :8], cache.transpose(0, 1), cache[0]):
        with pytest.raises(ValueError):
            pic._check_caches(gqa, bad, None, 4)
        with pytest.raises(ValueError):
            pic._check_caches(gqa, cache, bad, 4)
    pic._check_caches(gqa, cache, cache, 4)
    with pytest.raises(ValueError):
        pic._weight_heads(torch.zeros(64, 2, 8), cache.shape)
    with pytest.raises(ValueError):
        pic._token_rows(cache.transpose(1, 2)[0], "q", (2, 16, 128))


def test_binding_wants_latent_outputs_whether_or_not_a_value_cache_is_given(mla):
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(64, 16, 1, 576, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 576, dtype=torch.bfloat16)
    for v in (None, cache):
        with pytest.raises(ValueError, match="out must be"):
            pic.pic_attend_paged(mla, q, 1.0, cache, v, i.view(2, 1), i, 16, torch.empty(2, 4, 576))
        with pytest.raises(ValueError, match="CUDA device"):
            pic.pic_attend_paged(mla, q, 1.0, cache, v, i.view(2, 1), i, 16, torch.empty(2, 4, 512))


def test_empty_batches_need_no_buffers_of_their_own(gqa, mla):
    """What an empty tensor gives as its address is null: no tokens and no requests are no error."""
    none = dict(d_pos=None, q=None, q_out=None, k=None, v=None, d_req=None, d_slot=None)
    for ctx in (gqa, mla):
        for heads in (0, 4):
            assert _write(ctx, mla=ctx is mla, n_tokens=0, num_q_heads=heads, **none) == 0
    assert _write(gqa, n_tokens=0, n_tables=0, tables=None, **none) == 0
    none = dict(n_req=0, q=None, lens=None, out=None, lse=None)
    assert _attend(gqa, **none) == 0 and _attend(gqa, tables=None, **none) == 0
    assert _attend(gqa, weights=P, heads=1, **none) == 0
    assert _attend(mla, hq=16, q_stride=16 * 1152, v=None, **none) == 0
    none = dict(n_req=0, lens=None, kept=None, new=None)
    assert _evict(gqa, **none) == 0 and _evict(gqa, tables=None, **none) == 0
    assert _evict(mla, heads=1, v=None, cls=64 * 16 * 1152, **none) == 0
    # what has nothing to do with the batch is still looked at
    assert _write(gqa, n_tokens=0, n_axes=0) == INVALID and _write(gqa, n_tokens=0, ws=None) == CAPACITY
    assert _attend(gqa, n_req=0, hq=3) == INVALID and _attend(gqa, n_req=0, ws=None) == INVALID
    assert _evict(gqa, n_req=0, budget=0) == INVALID and _evict(gqa, n_req=0, k=None) == INVALID


def test_host_calls_need_no_torch():
    """Registry, plans and windows run where torch cannot be imported; only the calls that take tensors want it."""
    import subprocess
    import sys
    code = """
import sys
sys.modules["torch"] = None
from position_independent_kv_stitch_gb300 import pic
ctx = pic.pic_create(pic.PIC_KIND_GQA, 2, 2, 128, 128, 0, pic.PIC_PAIRING_NEOX_HALF, 16, 1e4, 64)
chunk = pic.pic_register_chunk(ctx, b"a" * 32, 0, 40)[0]
plan, table = pic.pic_build_block_table(ctx, [chunk], 8)
assert len(table) == 8 and pic.pic_evict_workspace_bytes(ctx, 2, 3, 2) > 0
pic.pic_free_request(ctx, plan)
try:
    pic.pic_write_tokens(ctx, None, None, None, None, None, None, None, None)
except ImportError:
    print("wants torch")
pic.pic_destroy(ctx)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=pic._build.ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "wants torch", r.stderr


def _axes_passed(monkeypatch, ctx, freq_axis):
    """The frequency axes that the library would be given."""
    import torch
    seen = []
    monkeypatch.setattr(pic, "_launch", lambda ctx, fn, device, stream, args: seen.append(
        ctypes.string_at(pic._NEW_TOKENS.unpack(args[0])[3], 64)))
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    pic.pic_write_tokens(ctx, torch.zeros(4, 2, dtype=torch.int32), None, None, None, None, None, None, None, q=q, q_out=q,
                         freq_axis=freq_axis)
    return list(seen[0])


def test_frequency_axes_of_any_integers(gqa, monkeypatch):
    """Lists, tuples, bytes, and arrays and tensors of any integer type name the same axes."""
    import array

    import numpy as np
    import torch
    axes = [f * 4 // 64 for f in range(64)]
    for x in (axes, tuple(axes), bytes(axes), bytearray(axes), array.array("i", axes), torch.tensor(axes), torch.tensor(axes, dtype=torch.uint8),
              *(np.array(axes, dtype=t) for t in (np.int64, np.int32, np.uint8, np.uint16)), np.array(axes * 2)[:64][::1]):
        assert _axes_passed(monkeypatch, gqa, x) == axes, type(x)
    for bad in (axes[:-1], axes + [0]):
        with pytest.raises(ValueError, match="frequencies"):
            _axes_passed(monkeypatch, gqa, bad)
    for bad in ([-1] + axes[1:], [256] + axes[1:], np.array([-1] + axes[1:])):
        with pytest.raises(ValueError):
            _axes_passed(monkeypatch, gqa, bad)
    with pytest.raises(TypeError):
        _axes_passed(monkeypatch, gqa, np.array(axes, dtype=np.float32))


def test_frequency_axes_are_not_kept(gqa, monkeypatch):
    """However many different lists are passed, the binding holds no more than the last one."""
    import gc
    import weakref
    made, array_of = [], ctypes.create_string_buffer

    class Kept:   # a buffer whose end can be seen
        def __init__(self, *a):
            self.buffer = array_of(*a)

    def buffer(*a):
        k = Kept(*a)
        made.append(weakref.ref(k))
        return k

    monkeypatch.setattr(ctypes, "create_string_buffer", buffer)
    monkeypatch.setattr(ctypes, "addressof", lambda k, _f=ctypes.addressof: _f(k.buffer))
    for i in range(20):
        axes = [(f >> (i % 5)) % 4 for f in range(64)]
        axes[i] = 3 - axes[i]
        assert _axes_passed(monkeypatch, gqa, axes) == axes
    gc.collect()
    assert len(made) == 20 and sum(r() is not None for r in made) <= 1


def test_lengths_near_the_integer_limit_are_refused():
    """A table that repeats its blocks may hold more slots than 31 bits count: what kernels add to a slot (steps
    looked up ahead, whole steps behind the end) must not pass the limit."""
    c = _ctx("mla", bs=256)
    blocks, cap = 1 << 23, 2 ** 31 - 1 - 8192
    for n, status in ((cap, CAPACITY), (cap + 1, RANGE), (2 ** 31 - 33, RANGE), (2 ** 31 - 1, RANGE)):
        assert _attend(c, hq=16, q_stride=16 * 1152, v=None, max_blocks=blocks, max_len=n, ws_bytes=0) == status, n
    pic.pic_destroy(c)

def test_workspace_sizes_of_what_the_calls_refuse_are_zero(gqa, mla):
    """No size wraps around: what is more than a call takes has no workspace."""
    size = pic.load().pic_attend_paged_workspace_bytes
    assert size(gqa, 1, 4096, 64, 1) > 0 and size(gqa, 1, 4098, 64, 1) == 0
    longest = 2 ** 31 - 1 - 8192
    assert size(gqa, 1 << 18, 4096, longest, 1) == 0 and size(gqa, 1, 4, longest + 1, 0) == 0
    assert size(gqa, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 1, 1) == 0
    assert size(mla, (1 << 18) - 1, 4096, longest, 1) > 2 ** 60
    size = pic.load().pic_evict_workspace_bytes
    assert size(gqa, 2, 1000, 2) > 0 and size(gqa, 3, 1000, 2) == 0
    assert size(gqa, 2, 2 ** 31 - 1, 2) == 0
