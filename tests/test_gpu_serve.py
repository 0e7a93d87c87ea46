"""GPU parity of a serving step's operators against the fp64 oracle: blocks and
slots from request lengths, token writes with head norms, attention of many
tokens per request (windows, first tokens, recompute lists), attention over a
shared prefix, and the four run together.

Tolerances.  A normed and rotated bf16 element: half a step of its value (2^-8
relative), the angle and the rotation as for plain writes (2^-19 of its pair's length),
and the norm: a sum of D squares of fp32 FMAs ((D + 8) 2^-24 relative, halved by the
root), the reciprocal root (2^-22) and two products (2^-23), below 2^-16 of
the pair's length up to D = 512.  Attention: a score of D fp32-accumulated products is off by
(D + 8) 2^-23 sum |q k| (tensor cores may truncate); a probability by twice the
largest score error, 2^-20 for the exponential, 2^-8 where P is rounded to bf16 for the value product, and T 2^-23 for
a sum over T, all relative to sum p |v|; outputs add half a step of bf16.  Log-sum-exps: the
score error, 2^-20 + T 2^-23, and 2^-22 of their value.  Integers and
untouched rows are compared exactly."""

import math

import numpy as np
import pytest
import torch

import oracle
from gpu_util import bits
from oracle import serve
from position_independent_kv_stitch_gb300 import pic
from test_gpu_decode import DEV, Cache, _f64, _i32, _pair_length, _status, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pic.load(build_if_missing=True)


# ------------------------------------------------------------- blocks and slots

class Pool:
    """A context over `blocks` blocks, requests holding some of them, the rest on the pile."""

    def __init__(self, lens, cols, blocks, bs, seed=0):
        rng = np.random.default_rng(seed)
        order = rng.permutation(blocks).astype(np.int32)
        self.bs, self.lens, self.blocks = bs, list(lens), blocks
        self.tables = np.full((len(lens), cols), -3, np.int32)
        at = 0
        for r, n in enumerate(lens):
            have = -(-max(0, n) // bs)
            self.tables[r, :have] = order[at:at + have]
            at += have
        self.n_free = blocks - at
        self.free = np.concatenate([order[at:], np.full(at, -9, np.int32)])
        self.ctx = pic.pic_create(pic.PIC_KIND_GQA, 1, 1, 64, 64, 0, pic.PIC_PAIRING_NEOX_HALF, bs, 1e4, blocks)

    def check(self, grow, n_tokens, shift=None, in_place=False, n_free=None, ws=None):
        n_free = self.n_free if n_free is None else n_free
        want = serve.map_tokens(self.lens, grow, self.tables, self.free, n_free, self.bs, n_tokens, shift)
        n = len(self.lens)
        d_lens, d_tables, d_free, d_n_free = _i32(self.lens), _i32(self.tables), _i32(self.free), _i32([n_free])
        new_lens, new_free = (d_lens, d_n_free) if in_place else (_i32([77] * n), _i32([77]))
        indptr, req, slot, pos = (_i32([77] * k) for k in (n + 1, n_tokens, n_tokens, n_tokens))
        ws = _ws() if ws is None else ws
        pic.pic_map_tokens(self.ctx, d_lens, _i32(grow), d_tables, d_free, d_n_free, new_lens, new_free, indptr, req, slot,
                           positions=pos, shift=None if shift is None else _i32(shift), workspace=ws)
        assert pic.pic_query_device_status(self.ctx, ws, raise_on_device_error=False) == want[8]
        for got, w, what in zip((new_lens, d_tables, d_free, new_free, indptr, req, slot, pos),
                                want[:3] + ([want[3]],) + want[4:8], ("lens", "tables", "free", "n_free", "indptr", "req", "slot", "pos")):
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(w, np.int64).reshape(got.shape), err_msg=what)
        ws.zero_()
        return want


@pytest.mark.parametrize("n_req", [1, 2, 33, 1024, 1025, 3000])
@pytest.mark.parametrize("bs", [1, 16, 100])
@pytest.mark.parametrize("in_place", [False, True])
def test_map_tokens(n_req, bs, in_place):
    rng = np.random.default_rng(n_req + bs)
    cols = max(2, 300 // bs)
    lens = rng.integers(0, cols * bs // 2 + 1, size=n_req).tolist()
    grow = [int(rng.integers(-n, cols * bs // 2 + 1)) if rng.random() < 0.7 else 1 for n in lens]
    total = sum(max(0, g) for g in grow)
    p = Pool(lens, cols, sum(-(-n // bs) for n in lens) + sum(-(-max(0, g) // bs) + 1 for g in grow), bs, seed=n_req)
    p.check(grow, total, rng.integers(0, 1000, size=n_req).tolist(), in_place)
    p.check(grow, total + 9000, None, in_place)
    p.check([1] * n_req, n_req, in_place=in_place)
    # too few blocks, too few rows
    p.check(grow, total, None, in_place, n_free=p.n_free // 8)
    p.check(grow, total // 2, None, in_place)
    pic.pic_destroy(p.ctx)


def test_map_tokens_long_prompts_in_many_parts():
    """Token rows for many CTAs: the state is written once, and the workspace serves the next call."""
    p = Pool([0, 5, 70000, 3, 31], 9000, 30000, 16, seed=1)
    ws = _ws()
    for in_place in (False, True, False):
        p.check([50000, 65536, -69999, 1, 16], 50000 + 65536 + 17 + 11, [0, 7, 0, 1, 2], in_place, ws=ws)
        p.check([0] * 5, 100000, None, in_place, ws=ws)
    pic.pic_destroy(p.ctx)


@pytest.mark.parametrize("n_tokens", [12, 20000])
def test_map_tokens_refusals(n_tokens):
    p = Pool([-1, 30, 64, 10, 10, 16], 4, 40, 16)
    p.check([4, 40, 0, -11, 2 ** 31 - 1, -16], n_tokens)
    p.check([-2 ** 31, 5, 1, 5, 0, 0], n_tokens)
    for n_free in (-1, 41, 2 ** 31 - 1):
        p.check([0, 3, 0, 1, 1, 20], n_tokens, n_free=n_free)
    p.check([0, -30, 0, -10, -10, -16], n_tokens, n_free=37)      # the pile holds three more, seven blocks come back
    p.tables[3, 0] = 99                                           # blocks outside the cache are moved, and raised
    p.free[p.n_free - 1] = -5
    p.check([0, 0, 0, -10, 30, 0], n_tokens)
    pic.pic_destroy(p.ctx)


def test_map_tokens_of_nothing():
    p = Pool([], 3, 5, 16)
    p.check([], 0)
    p.check([], 7)
    pic.pic_destroy(p.ctx)
    p = Pool([0, 0], 3, 0, 16)                                    # a cache without blocks
    p.check([0, 1], 4)
    pic.pic_destroy(p.ctx)


# ------------------------------------------------------------- normed writes

def _write_normed(c, n_tok, hq, q_norm=True, k_norm=True, dtype=torch.bfloat16, offset=0.0, eps=1e-6, axes=1, in_place=False, pad=0,
                  scale=2.0, weights=True):
    gqa, half = c.kind == "gqa", c.m.rope_dim // 2
    dims = c.d if gqa else 512
    fx = [f % axes for f in range(half)]
    pos = c.rng.integers(0, 40000, size=(axes, n_tok))
    places = [(r, s) for r, n in enumerate(c.lens) for s in range(n, c.tables.shape[1] * c.bs)]
    pick = c.rng.permutation(len(places))[:n_tok]
    req, slot = np.array([places[i][0] for i in pick]), np.array([places[i][1] for i in pick])
    slot[:pad] = -1
    rows = c.normal(n_tok, hq + 2 * c.heads, c.d) * scale
    q, k, v = rows[:, :hq], rows[:, hq:hq + c.heads], rows[:, hq + c.heads:] if gqa else None
    qn = c.normal(dims).to(dtype) if q_norm and gqa else None
    kn = (c.normal(dims) + 0.25).to(dtype) if k_norm else None
    want = serve.write_normed(_f64(q), _f64(k), None if qn is None else _f64(qn), None if kn is None else _f64(kn), eps, offset, pos, fx,
                              c.theta, c.pairing, c.m.rope_offset, c.m.rope_dim)
    kb, vb, wb = c.k[0].clone(), None if v is None else c.v[0].clone(), c.w[0].clone()
    q_out = q if in_place else torch.full((n_tok, hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _ws()
    pic.pic_write_normed_tokens(c.ctx, _i32(pos if axes > 1 else pos[0]), k, v, _i32(req), _i32(slot), c.d_tables, c.k[0],
                                None if v is None else c.v[0], q_norm=qn, k_norm=kn, eps=eps, offset=offset, q=q, q_out=q_out,
                                freq_axis=fx, weights=c.w[0] if weights else None, workspace=ws)
    assert _status(c, ws) == 0
    live = np.nonzero(slot >= 0)[0]
    page, row = c.tables[req[live], slot[live] // c.bs], slot[live] % c.bs
    for got, w, what in ((_f64(q_out), want[0], "q"), (_f64(c.k[0])[page, row], want[1][live], "k")):
        lim = 2.0 ** -8 * np.abs(w) * (1 + 2.0 ** -9) + (2.0 ** -19 + 2.0 ** -16) * np.maximum(np.abs(w), _pair_length(w, c)) + 1e-38
        assert np.all(np.abs(got - w) <= lim), (what, (np.abs(got - w) / lim).max())
    kb[page, row] = c.k[0][page, row]
    assert torch.equal(c.k[0], kb)                                  # rows nobody wrote
    if v is not None:
        vb[page, row] = v[torch.from_numpy(live).to(DEV)]
        assert torch.equal(c.v[0], vb)
    if weights:
        wb[page, :, row] = 0.0
    assert torch.equal(c.w[0], wb)


@pytest.mark.parametrize("heads,hq,d,bs,pairing", [(2, 8, 128, 16, "neox"), (8, 32, 128, 16, "interleaved"), (1, 7, 64, 1, "neox"),
                                                   (3, 15, 64, 17, "interleaved"), (5, 5, 256, 256, "neox"),
                                                   (4, 4, 256, 7, "interleaved"), (16, 48, 64, 64, "neox"), (1, 1, 128, 16, "neox")])
@pytest.mark.parametrize("n_tok,axes,dtype", [(1, 1, torch.bfloat16), (37, 3, torch.float32), (200, 1, torch.bfloat16)])
def test_write_normed(heads, hq, d, bs, pairing, n_tok, axes, dtype):
    c = Cache(heads=heads, d=d, bs=bs, pairing=pairing, lens=[5, 0, 31], room=-(-n_tok // 3) + bs, seed=heads + n_tok)
    _write_normed(c, n_tok, hq, dtype=dtype, axes=axes, offset=1.0 if axes > 1 else 0.0)
    c.close()


@pytest.mark.parametrize("kw", [dict(q_norm=False), dict(k_norm=False), dict(q_norm=False, k_norm=False), dict(in_place=True),
                                dict(pad=9), dict(eps=0.0), dict(eps=10.0), dict(scale=1e-12), dict(scale=1e15), dict(weights=False)])
def test_write_normed_forms(kw):
    c = Cache(heads=4, lens=[20, 3], room=90, seed=5)
    _write_normed(c, 70, 12, **kw)
    c.close()


@pytest.mark.parametrize("pairing", ["neox", "interleaved"])
@pytest.mark.parametrize("in_place,dtype", [(False, torch.bfloat16), (True, torch.float32)])
@pytest.mark.parametrize("n_tok,hq,k_norm", [(1, 16, True), (33, 3, True), (7, 128, True), (9, 16, False)])
def test_write_normed_latents(pairing, in_place, dtype, n_tok, hq, k_norm):
    c = Cache("mla", bs=16, pairing=pairing, lens=[5, 9], room=60, seed=n_tok, weight_heads=1)
    _write_normed(c, n_tok, hq, k_norm=k_norm, dtype=dtype, in_place=in_place, axes=2, pad=min(2, n_tok - 1))
    c.close()


def test_write_normed_zero_rows_and_bad_tokens():
    """A head of zeros stays zeros; tokens with bad places or positions are left out, queries by position alone."""
    c = Cache(heads=2, lens=[16, 16], room=16, seed=4)
    c.d_tables[1, 1] = c.nb
    q, k, v = c.normal(5, 4, 128), c.normal(5, 2, 128), c.normal(5, 2, 128)
    q[0], k[0] = 0, 0
    req, slot, pos = [0, 1, 2, 0, 0], [16, 16, 3, 32, 17], [3, 4, 5, 7, 1 << 24]
    w = c.normal(128)
    q_out, ws, kb = torch.full_like(q, 9.0), _ws(), c.k[0].clone()
    pic.pic_write_normed_tokens(c.ctx, _i32(pos), k, v, _i32(req), _i32(slot), c.d_tables, c.k[0], c.v[0], q_norm=w, k_norm=w, q=q,
                                q_out=q_out, workspace=ws)
    assert _status(c, ws) == pic.PIC_DEV_BAD_BLOCK | pic.PIC_DEV_BAD_POS
    page = int(c.tables[0][1])
    assert bool((c.k[0][page, 0] == 0).all()) and bool((q_out[0] == 0).all()) and bool((q_out[4] == 9.0).all())
    assert not bool((q_out[1:4] == 9.0).all())
    kb[page, 0] = c.k[0][page, 0]
    assert torch.equal(c.k[0], kb)
    c.close()


# ---------------------------------------------------------- attention of tokens

def _wide_rows(cache, table, slots, bs):
    """Rows [heads][T][dim] in 64 bits, on the device."""
    s = torch.as_tensor(np.asarray(slots), device=DEV, dtype=torch.long)
    t = torch.as_tensor(np.asarray(table), device=DEV, dtype=torch.long)
    return cache[t[s // bs], s % bs].double().transpose(0, 1)


def _assert_rows(q, k, v, seen, scale, out, lse, what):
    """q [n][Hq][D] and its outputs against softmax attention in 64 bits over rows k, v [Hk][T][D], seen [n][T]."""
    hk, t, d = k.shape
    n, hq = q.shape[0], q.shape[1]
    qd = q.double().reshape(n, hk, hq // hk, d)
    x = torch.einsum("nhgd,htd->nhgt", qd, k) * scale
    mag = torch.einsum("nhgd,htd->nhgt", qd.abs(), k.abs()) * abs(scale)
    mask = seen[:, None, None]
    x = x.masked_fill(~mask, -math.inf)
    s_err = mag.masked_fill(~mask, 0.0).amax(-1) * (d + 8) * 2.0 ** -23 if t else torch.zeros(n, hk, hq // hk, device=DEV)
    want_lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(want_lse.isinf(), 0.0, want_lse)[..., None])
    want = torch.einsum("nhgt,htd->nhgd", p, v)
    spread = torch.einsum("nhgt,htd->nhgd", p, v.abs())
    count = seen.sum(-1)[:, None, None]
    rel = 2 * s_err + 2.0 ** -20 + count * 2.0 ** -23
    lim = (rel + 2.0 ** -8)[..., None] * spread + 2.0 ** -8 * want.abs() * (1 + rel + 2.0 ** -8)[..., None] + 1e-38
    err = (out.double().reshape(want.shape) - want).abs()
    assert bool((err <= lim).all()), (what, "out", float((err / lim).max()), float(err.max()))
    got = lse.double().reshape(want_lse.shape)
    none = (count == 0).expand_as(got)
    assert bool((got[none] == -math.inf).all()), what
    bad = ((got - want_lse).abs() > s_err + rel + 2.0 ** -22 * want_lse.abs())[~none]
    assert not bool(bad.any()), (what, "lse")


def _attend(c, slots, hq, window=0, n_first=0, scale=None, pad=0, q=None, layer=0, tables=None, status=0, check=None, pitch=0):
    """slots: per request, its tokens' slots."""
    scale = 1.0 / math.sqrt(c.d) if scale is None else scale
    counts = [len(x) for x in slots]
    indptr = np.concatenate([[0], np.cumsum(counts)])
    n = int(indptr[-1]) + pad
    if q is None:
        q = c.normal(n, hq + pitch, c.d)[:, :hq] * 1.5 if not pitch else c.normal(n, hq + pitch, c.d)[:, :hq]
    slot = _i32([x for xs in slots for x in xs] + [3] * pad)
    out = torch.full((n, hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, n, len(slots), hq))
    pic.pic_attend_tokens(c.ctx, q, scale, c.k[layer], c.v[layer], c.d_tables if tables is None else tables, _i32(indptr), slot, out,
                          window=window, n_first=n_first, lse=lse, workspace=ws)
    assert _status(c, ws) == status
    if pad:
        assert bool((out[n - pad:] == 7.0).all()) and bool((lse[n - pad:] == 7.0).all())
    for r, xs in enumerate(slots):
        if (check is not None and r not in check) or not xs:
            continue
        a = slice(int(indptr[r]), int(indptr[r + 1]))
        seen = np.stack([serve.sees(s, np.arange(max(xs) + 1), window, n_first) for s in xs])
        used = np.nonzero(seen.any(0))[0]
        k, v = (_wide_rows(x[layer], c.tables[r], used, c.bs) for x in (c.k, c.v))
        _assert_rows(q[a], k, v, torch.from_numpy(seen[:, used]).to(DEV), scale, out[a], lse[a], (r, window, n_first))
    return out, lse, q


SHAPES = [(2, 8, 128, 16), (8, 32, 128, 16), (1, 1, 64, 1), (3, 15, 64, 17), (2, 14, 128, 5), (2, 16, 256, 64), (1, 12, 128, 48),
          (2, 32, 64, 32), (1, 16, 256, 16), (1, 40, 128, 256), (5, 5, 256, 3), (9, 9, 64, 16), (1, 200, 128, 16), (1, 3, 256, 100)]


@pytest.mark.parametrize("heads,hq,d,bs", SHAPES)
@pytest.mark.parametrize("window,n_first", [(0, 0), (70, 4)])
def test_attend_tokens(heads, hq, d, bs, window, n_first):
    """Prompts, chunked prompts, single tokens, an idle request and padding rows together."""
    lens = [300, 1, 0, 77, 260, 129]
    c = Cache(heads=heads, d=d, bs=bs, lens=lens, seed=hq)
    slots = [list(range(300)), [0], [], [76], list(range(100, 260)), [-1, 128]]
    _attend(c, slots, hq, window, n_first, pad=3)
    c.close()


@pytest.mark.parametrize("heads,hq,d,bs", SHAPES)
@pytest.mark.parametrize("window,n_first", [(0, 0), (1, 0), (33, 0), (64, 130), (2 ** 31 - 1, 5)])
def test_attend_single_tokens(heads, hq, d, bs, window, n_first):
    """The decode form: a token per request, lengths around the tiles."""
    lens = [1, 77, 16, 200, 15, 17, 129, 500]
    c = Cache(heads=heads, d=d, bs=bs, lens=lens, seed=hq)
    _attend(c, [[n - 1] for n in lens], hq, window, n_first)
    c.close()


@pytest.mark.parametrize("window,n_first", [(0, 0), (1, 1), (2, 0), (16, 3), (127, 0), (128, 128), (129, 1), (1000, 4), (333, 700)])
def test_attend_tokens_windows(window, n_first):
    c = Cache(heads=2, lens=[1500, 900], seed=window)
    _attend(c, [list(range(1500)), list(range(890, 900))], 8, window, n_first)
    c.close()


def test_attend_tokens_in_any_order():
    """A recompute list: chunk heads and the end, twice the same slot, descending, far apart."""
    c = Cache(heads=2, lens=[3000, 2000], seed=9)
    slots = [[5, 5, 2999, 0, 1000, 1001, 1002, 17, 2500], list(range(1999, 1600, -3)) + list(range(0, 64)) + [-1, -1]]
    for window, n_first in ((0, 0), (100, 2), (1500, 64)):
        _attend(c, slots, 8, window, n_first, pad=1)
    c.close()


@pytest.mark.parametrize("d,group", [(128, 4), (64, 8), (256, 2)])
def test_attend_tokens_long(d, group):
    """Long contexts under few rows: the work of a tile is split over its slots."""
    c = Cache(heads=2, d=d, lens=[20011, 9000], seed=1)
    _attend(c, [list(range(20011 - 70, 20011)), [8999]], 2 * group)
    _attend(c, [list(range(20011 - 5, 20011)), [8999, 17]], 2 * group, window=15000, n_first=100)
    c.close()


@pytest.mark.parametrize("heads,hq,d,bs", [(8, 16, 128, 16), (8, 32, 64, 16), (19, 19, 128, 1), (10, 30, 64, 4), (8, 8, 128, 128), (8, 24, 64, 5)])
@pytest.mark.parametrize("window,n_first", [(0, 0), (70, 4), (333, 200)])
def test_attend_tokens_in_two_tiles(heads, hq, d, bs, window, n_first):
    """More requests' rows than SMs, of which some fill a tile, two, more, or a part of one."""
    rng = np.random.default_rng(hq)
    counts = [1, 7, 64, 128, 200, 0, 300] + rng.integers(2, 150, size=14).tolist()
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 300, size=len(counts)))]
    c = Cache(heads=heads, d=d, bs=bs, lens=lens, seed=hq)
    _attend(c, [list(range(n - k, n)) for n, k in zip(lens, counts)], hq, window, n_first, pad=2)
    c.close()


@pytest.mark.parametrize("window,n_first", [(0, 0), (40, 3)])
def test_attend_tokens_in_two_tiles_ignores_what_no_token_sees(window, n_first):
    """As below with more rows: junk where nobody sees, blocks given back there, and a bad block in one request."""
    lens = [150 + 11 * r for r in range(24)]
    c = Cache(heads=8, bs=16, lens=lens, room=40, seed=6)
    q = c.normal(24 * 50, 16, 128)
    slots = [list(range(n - 50, n)) for n in lens]
    clean, clean_lse, _ = _attend(c, slots, 16, window, n_first, q=q, check=range(0, 24, 5))
    for r, n in enumerate(lens):
        seen = np.zeros(c.tables.shape[1] * 16, bool)
        seen[max(0, n - 49 - window) if window else 0:n] = True
        seen[:n_first] = True
        for s in np.nonzero(~seen)[0]:
            c.k[0, int(c.tables[r][s // 16]), s % 16] = float("nan") if s % 2 else float("inf")
            c.v[0, int(c.tables[r][s // 16]), s % 16] = float("inf") if s % 3 else float("nan")
        for b in range(c.tables.shape[1]):
            if not seen[b * 16:(b + 1) * 16].any():
                c.d_tables[r, b] = -1 if b % 2 else 2 ** 31 - 1
    out, lse, _ = _attend(c, slots, 16, window, n_first, q=q, check=())
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    bad = (lens[3] - 20) // 16   # seen by the last tokens of request 3
    c.d_tables[3, bad] = c.nb
    out, lse, _ = _attend(c, slots, 16, window, n_first, q=q, status=pic.PIC_DEV_BAD_BLOCK, check=())
    a = slice(150, 200)
    others = torch.ones(len(out), dtype=torch.bool, device=DEV)
    others[a] = False
    assert torch.equal(out[others], clean[others]) and torch.equal(lse[others], clean_lse[others])
    keep = np.array([s for s in range(lens[3]) if s // 16 != bad and (window == 0 or s >= lens[3] - 49 - window or s < n_first)])
    seen = torch.from_numpy(np.stack([serve.sees(s, keep, window, n_first) for s in slots[3]])).to(DEV)
    _assert_rows(q[a], *(_wide_rows(x[0], c.tables[3], keep, 16) for x in (c.k, c.v)), seen, 128 ** -0.5, out[a], lse[a], "bad block")
    c.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,context", [(31, 3000), (33, 3000), (128, 16384), (400, 4500), (512, 512), (608, 4600)])
def test_attend_tokens_of_one_request(d, tokens, context):
    """Row blocks of one tile and of two, whole and in parts."""
    c = Cache(heads=8, d=d, lens=[context], seed=tokens)
    q = c.normal(tokens, 32, d)
    out, lse, _ = _attend(c, [list(range(context - tokens, context))], 32, q=q, check=())
    k, v = (_wide_rows(x[0], c.tables[0], np.arange(context), c.bs) for x in (c.k, c.v))
    for a in range(0, tokens, 32):
        rows = slice(a, min(tokens, a + 32))
        at = torch.arange(context - tokens + a, context - tokens + rows.stop, device=DEV)
        seen = torch.arange(context, device=DEV)[None] <= at[:, None]
        _assert_rows(q[rows], k, v, seen, d ** -0.5, out[rows], lse[rows], a)
    c.close()


def test_attend_tokens_many_requests():
    """Hundreds of requests of a few tokens, empty ones among them."""
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 90, size=700).tolist()
    c = Cache(heads=1, d=64, lens=lens, seed=2)
    slots = [list(range(max(0, n - int(rng.integers(0, 6))), n)) for n in lens]
    _attend(c, slots, 4, check=range(0, 700, 7))
    _attend(c, [[n - 1] for n in lens], 4, window=20, n_first=2, check=range(0, 700, 7))
    c.close()


@pytest.mark.parametrize("tokens", [1, 60])
@pytest.mark.parametrize("window,n_first", [(0, 0), (40, 3)])
def test_attend_tokens_ignores_what_no_token_sees(tokens, window, n_first):
    """NaN and infinities behind the sequence, before the window and behind the first tokens; blocks given back there."""
    c = Cache(heads=2, bs=16, lens=[400, 170], room=40, seed=6)
    q = c.normal(2 * tokens, 8, 128)
    slots = [list(range(n - tokens, n)) for n in c.lens]
    clean, clean_lse, _ = _attend(c, slots, 8, window, n_first, q=q)
    for r, n in enumerate(c.lens):
        seen = np.zeros(c.tables.shape[1] * 16, bool)
        lo = max(0, n - tokens + 1 - window) if window else 0
        seen[lo:n] = True
        seen[:min(n_first, n)] = True
        for s in np.nonzero(~seen)[0]:
            c.k[0, int(c.tables[r][s // 16]), s % 16] = float("nan") if s % 2 else float("inf")
            c.v[0, int(c.tables[r][s // 16]), s % 16] = float("inf") if s % 3 else float("nan")
        for b in range(c.tables.shape[1]):
            if not seen[b * 16:(b + 1) * 16].any():
                c.d_tables[r, b] = -1 if b % 2 else 2 ** 31 - 1
    out, lse, _ = _attend(c, slots, 8, window, n_first, q=q, check=())
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    c.close()


@pytest.mark.parametrize("tokens", [1, 50])
def test_attend_tokens_bad_blocks_and_slots(tokens):
    """Slots in a block outside the cache are left out; a slot past the table sees nothing; the others are as without."""
    c = Cache(heads=2, bs=16, lens=[100, 100, 100, 100], seed=8)
    q = c.normal(4 * tokens, 8, 128)
    slots = [list(range(100 - tokens, 100)) for _ in range(4)]
    clean, clean_lse, _ = _attend(c, slots, 8, q=q)
    tables = c.d_tables.clone()
    tables[1, 2], tables[3, :] = c.nb, -1
    out, lse, _ = _attend(c, slots, 8, q=q, tables=tables, status=pic.PIC_DEV_BAD_BLOCK, check=())
    for r in (0, 2):
        a = slice(r * tokens, (r + 1) * tokens)
        assert torch.equal(out[a], clean[a]) and torch.equal(lse[a], clean_lse[a])
    assert bool((out[3 * tokens:] == 0).all()) and bool((lse[3 * tokens:] == -math.inf).all())
    keep = np.array([s for s in range(100) if s // 16 != 2])
    seen = torch.from_numpy(np.stack([keep <= s for s in slots[1]])).to(DEV)
    a = slice(tokens, 2 * tokens)
    _assert_rows(q[a], *(_wide_rows(x[0], c.tables[1], keep, 16) for x in (c.k, c.v)), seen, 128 ** -0.5, out[a], lse[a], "bad block")
    slots[0][0], slots[2][-1] = 2 ** 31 - 1, c.tables.shape[1] * 16
    out, lse, _ = _attend(c, slots, 8, q=q, status=pic.PIC_DEV_BAD_LENGTH, check=())
    for i in (0, 3 * tokens - 1):
        assert bool((out[i] == 0).all()) and bool((lse[i] == -math.inf).all())
    # (how a request's work is split, and with it the last bit, may follow from the others' slots)
    seen = torch.from_numpy(np.stack([np.arange(100) <= s for s in slots[1]])).to(DEV)
    _assert_rows(q[a], *(_wide_rows(x[0], c.tables[1], np.arange(100), 16) for x in (c.k, c.v)), seen, 128 ** -0.5, out[a], lse[a], "good")
    c.close()


@pytest.mark.parametrize("indptr", [[-5, 3, 6], [0, 100, 6], [4, 2, 6], [0, 3, 2 ** 31 - 1], [2, 2, 2], [-3, -2, -1], [7, 8, 9]])
@pytest.mark.parametrize("n", [2, 6, 40])
def test_attend_tokens_bad_offsets(indptr, n):
    """Offsets outside the rows: nothing beyond the buffers is touched, and they are raised."""
    c = Cache(heads=1, d=64, lens=[50, 50], seed=1)
    big = torch.full((n + 20, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out, q = big[:n], c.normal(n, 4, 64)
    ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, n, 2, 4))
    pic.pic_attend_tokens(c.ctx, q, 0.1, c.k[0], c.v[0], c.d_tables, _i32(indptr), _i32(np.arange(n) % 50), out, workspace=ws)
    ok = 0 <= indptr[0] <= indptr[1] <= indptr[2] <= n
    assert _status(c, ws) == (0 if ok else pic.PIC_DEV_BAD_LENGTH)
    assert bool((big[n:] == 7.0).all())
    c.close()


@pytest.mark.parametrize("tokens", [1, 9])
def test_attention_over_a_cache_without_blocks(tokens):
    """No slot exists: every row but padding raises and sees nothing; an empty prefix and empty requests are fine."""
    ctx = pic.pic_create(pic.PIC_KIND_GQA, 1, 2, 64, 64, 0, pic.PIC_PAIRING_NEOX_HALF, 16, 1e4, 0)
    cache, q = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16, device=DEV), torch.ones(tokens, 4, 64, dtype=torch.bfloat16, device=DEV)
    tables, out = _i32(np.zeros((1, 3))), torch.full_like(q, 7.0)
    ws = _ws(max(pic.pic_attend_tokens_workspace_bytes(ctx, tokens, 1, 4), pic.pic_attend_shared_workspace_bytes(ctx, 1, 4)))
    pic.pic_attend_tokens(ctx, q, 0.1, cache, cache, tables, _i32([0, tokens]), _i32(np.arange(tokens) - 1), out, workspace=ws)
    want = 0 if tokens == 1 else pic.PIC_DEV_BAD_LENGTH
    assert pic.pic_query_device_status(ctx, ws, raise_on_device_error=False) == want and bool((out == 0).all())
    ws.zero_()
    out.fill_(7.0)
    pic.pic_attend_shared(ctx, q[:1], 0.1, cache, cache, tables[0], _i32([0]), tables, _i32([0]), 0, out[:1], workspace=ws)
    assert pic.pic_query_device_status(ctx, ws) == 0 and bool((out[:1] == 0).all())
    pic.pic_destroy(ctx)


def test_attend_tokens_forms():
    """Query rows apart, a negative and a zero scale, another layer, no lse, dense caches of many layers."""
    c = Cache(heads=2, layers=3, lens=[200, 33], seed=4)
    slots = [list(range(150, 200)), [32]]
    _attend(c, slots, 8, pitch=4)
    for scale in (-0.05, 0.0, 1.0):
        _attend(c, slots, 8, scale=scale, layer=2)
        _attend(c, [[199], [32]], 8, scale=scale, layer=1)
    q = c.normal(51, 8, 128)
    out, _, _ = _attend(c, slots, 8, q=q)
    again, ws = torch.empty_like(out), _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, 51, 2, 8))
    pic.pic_attend_tokens(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, _i32([0, 50, 51]), _i32(slots[0] + slots[1]), again,
                          workspace=ws)
    assert torch.equal(out, again)
    c.close()


def test_offsets_beyond_32_bits():
    """Layers of 6.6 GB, blocks at both ends; query rows 5 MB apart; maps, writes and both attentions."""
    nb, bs, heads, d, hq = 201_000, 16, 8, 128, 16
    ctx = pic.pic_create(pic.PIC_KIND_GQA, 1, heads, d, d, 0, pic.PIC_PAIRING_NEOX_HALF, bs, 5e5, nb)
    k_cache, v_cache = (torch.zeros(nb, bs, heads, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(3)
    free = np.arange(nb)
    free[-20:] = [200_999, 0, 131_072, 131_071, 65_536, 200_998, 1, 196_608, 2, 131_073] + list(range(200_900, 200_910))
    tables, lens, n_free = _i32(np.full((2, 10), -1)), _i32([0, 0]), _i32([nb])
    n, pitch = 150, 5 * (1 << 20) // 256
    indptr, req, slot, pos = _i32([0] * 3), _i32([0] * n), _i32([0] * n), _i32([0] * n)
    ws = _ws(max(pic.pic_attend_tokens_workspace_bytes(ctx, n, 2, hq), pic.pic_attend_shared_workspace_bytes(ctx, 2, hq)))
    pic.pic_map_tokens(ctx, lens, _i32([100, 50]), tables, _i32(free), n_free, lens, n_free, indptr, req, slot, positions=pos, workspace=ws)
    host = tables.cpu().numpy()
    assert host[0, :7].tolist() == free[-1:-8:-1].tolist()
    wide = torch.zeros(n, pitch, d, dtype=torch.bfloat16, device=DEV)
    wide[:, :hq + 2 * heads] = torch.randn((n, hq + 2 * heads, d), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = wide[:, :hq], wide[:, hq:hq + heads], wide[:, hq + heads:hq + 2 * heads]
    w = torch.ones(d, device=DEV)
    pic.pic_write_normed_tokens(ctx, pos, k, v, req, slot, tables, k_cache, v_cache, q_norm=w, k_norm=w, q=q, q_out=q, workspace=ws)
    out, lse = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(n, hq, device=DEV)
    pic.pic_attend_tokens(ctx, q, d ** -0.5, k_cache, v_cache, tables, indptr, slot, out, lse=lse, workspace=ws)
    for r, (a, b) in enumerate(((0, 100), (100, 150))):
        assert torch.equal(v_cache[tables[r].long()[torch.arange(b - a, device=DEV) // bs], torch.arange(b - a, device=DEV) % bs], v[a:b])
        rows = [_wide_rows(x, host[r], np.arange(b - a), bs) for x in (k_cache, v_cache)]
        seen = torch.tril(torch.ones(b - a, b - a, dtype=torch.bool, device=DEV))
        _assert_rows(q[a:b], *rows, seen, d ** -0.5, out[a:b], lse[a:b], r)
    dec, dec_lse = torch.empty(2, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(2, hq, device=DEV)
    pic.pic_attend_shared(ctx, q[:2], d ** -0.5, k_cache, v_cache, tables[0, :4], _i32([60]), tables, _i32([100, 60]), 160, dec, lse=dec_lse,
                          workspace=ws)
    rows = [_wide_rows(x, host[0], np.arange(100), bs) for x in (k_cache, v_cache)]
    for r, m in enumerate((100, 60)):
        _assert_rows(q[r:r + 1], *(x[:, :m] for x in rows), torch.ones(1, m, dtype=torch.bool, device=DEV), d ** -0.5, dec[r:r + 1],
                     dec_lse[r:r + 1], r)
    assert pic.pic_query_device_status(ctx, ws) == 0
    pic.pic_destroy(ctx)


def test_attend_tokens_extreme_scores():
    """Scores far apart and rising along the sequence: the running maximum moves, sums stay exact."""
    c = Cache(heads=1, lens=[700], seed=5)
    ramp = torch.linspace(0.0, 6.0, 700, device=DEV).to(torch.bfloat16)
    for s in range(700):
        c.k[0, int(c.tables[0][s // 16]), s % 16] = ramp[s]
    for sign in (1.0, -1.0):
        q = torch.full((300, 4, 128), sign, dtype=torch.bfloat16, device=DEV)
        _attend(c, [list(range(400, 700))], 4, q=q, scale=0.5)
        _attend(c, [[699]], 4, q=q[:1], scale=0.5)
    c.close()


# ------------------------------------------------------------- a shared prefix

class Shared(Cache):
    """Requests over one prefix; the blocks that hold nothing else are in every table."""

    def __init__(self, prefix, own, **kw):
        kw.setdefault("bs", 16)
        super().__init__(lens=[prefix + n if n is not None else 0 for n in own], room=1, **kw)
        whole = prefix // self.bs
        spare = -(-prefix // self.bs)
        rows = self.tables[0][:spare].copy()
        self.prefix = prefix
        if prefix % self.bs:               # the prefix's last block: a spare one
            used = set(self.tables.flatten().tolist())
            rows[-1] = next(b for b in range(self.nb) if b not in used)
        self.prefix_table = rows
        self.tables[:, :whole] = rows[:whole]
        self.d_tables = _i32(self.tables)


def _shared(c, hq, q=None, lens=None, prefix=None, scale=None, tables=None, prefix_table=None, status=0, check=True, max_len=None):
    lens, prefix = c.lens if lens is None else lens, c.prefix if prefix is None else prefix
    scale = 1.0 / math.sqrt(c.d) if scale is None else scale
    n = len(lens)
    q = c.normal(n, hq, c.d) * 1.5 if q is None else q
    out, lse = torch.full((n, hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((n, hq), 7.0, device=DEV)
    ws = _ws(pic.pic_attend_shared_workspace_bytes(c.ctx, n, hq))
    pic.pic_attend_shared(c.ctx, q, scale, c.k[0], c.v[0], _i32(c.prefix_table if prefix_table is None else prefix_table), _i32([prefix]),
                          c.d_tables if tables is None else tables, _i32(lens), max(lens) if max_len is None else max_len, out, lse=lse,
                          workspace=ws)
    assert _status(c, ws) == status
    if check:
        for r, length in enumerate(lens):
            head, tail = np.arange(min(prefix, length)), np.arange(prefix, max(prefix, length))
            k, v = (torch.cat([_wide_rows(x[0], c.prefix_table, head, c.bs), _wide_rows(x[0], c.tables[r], tail, c.bs)], 1)
                    for x in (c.k, c.v))
            seen = torch.ones(1, k.shape[1], dtype=torch.bool, device=DEV)
            _assert_rows(q[r:r + 1], k, v, seen, scale, out[r:r + 1], lse[r:r + 1], ("request", r))
    return out, lse, q


@pytest.mark.parametrize("heads,hq,d,bs", SHAPES)
@pytest.mark.parametrize("prefix", [1, 100, 515])
def test_attend_shared(heads, hq, d, bs, prefix):
    c = Shared(prefix, [1, 0, 77, 16, None, 40], heads=heads, d=d, bs=bs, seed=hq)
    _shared(c, hq)
    c.close()


@pytest.mark.parametrize("n_req", [1, 2, 31, 64, 65, 200])
def test_attend_shared_batches(n_req):
    rng = np.random.default_rng(n_req)
    c = Shared(2003, rng.integers(0, 200, size=n_req).tolist(), heads=2, seed=n_req)
    _shared(c, 8)
    c.close()


def test_attend_shared_long_prefix():
    c = Shared(30011, [3, 900, None, 17], heads=2, seed=2)
    _shared(c, 8)
    _shared(c, 32)
    c.close()


@pytest.mark.parametrize("d,n_req,prefix", [(128, 5, 33000), (128, 36, 33000), (64, 36, 40003), (128, 64, 8200), (64, 70, 9001)])
def test_attend_shared_tile_forms(d, n_req, prefix):
    """Prefixes in row blocks of one tile and of two."""
    c = Shared(prefix, [3 * r % 50 for r in range(n_req)], heads=8, d=d, seed=n_req)
    _shared(c, 32)
    c.close()


def test_attend_shared_short_requests_and_no_prefix():
    """Requests that end inside the prefix; a prefix of length 0 is plain paged attention."""
    c = Shared(200, [5, 60, 9], heads=2, seed=3)
    _shared(c, 8, lens=[205, 63, 1])
    _shared(c, 8, lens=[200, 0, 199])
    _shared(c, 8, lens=[0, 0, 0], max_len=10)
    _shared(c, 8, prefix=0, lens=[150, 0, 199])
    c.close()


def test_attend_shared_ignores_what_no_request_sees():
    """The prefix's last block behind it, tables' entries in the prefix, and rows behind the ends hold anything."""
    c = Shared(205, [5, 60, 0], heads=2, seed=4)
    clean, clean_lse, q = _shared(c, 8)
    page = int(c.prefix_table[-1])
    c.k[0, page, 205 % 16:], c.v[0, page, 205 % 16:] = float("nan"), float("inf")
    tables = c.d_tables.clone()
    tables[:, :205 // 16] = -1
    for r, n in enumerate(c.lens):
        c.k[0, int(c.tables[r][n // 16]), n % 16:], c.v[0, int(c.tables[r][n // 16]), n % 16:] = float("inf"), float("nan")
        own = int(c.tables[r][205 // 16])
        c.k[0, own, :205 % 16], c.v[0, own, :205 % 16] = float("nan"), float("nan")
    out, lse, _ = _shared(c, 8, q=q, tables=tables, check=False)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    c.close()


def test_attend_shared_bad_lengths_and_blocks():
    c = Shared(100, [5, 60, 9], heads=2, seed=5)
    q = c.normal(3, 8, 128)
    for lens, prefix in (([105, -1, 109], 100), ([105, 161, 109], 100)):
        out, lse, _ = _shared(c, 8, q=q, lens=lens, prefix=prefix, status=pic.PIC_DEV_BAD_LENGTH, check=False, max_len=160)
        assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
        want, want_lse, _ = _shared(c, 8, q=q, lens=[105, 0, 109], max_len=160)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    for prefix in (-1, len(c.prefix_table) * 16 + 1):      # counts as 0: the tables alone
        out, lse, _ = _shared(c, 8, q=q, lens=[105, 160, 109], prefix=prefix, status=pic.PIC_DEV_BAD_LENGTH, check=False)
        want, want_lse, _ = _shared(c, 8, q=q, lens=[105, 160, 109], prefix=0, check=False)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    bad = c.prefix_table.copy()
    bad[2] = c.nb
    out, lse, _ = _shared(c, 8, q=q, prefix_table=bad, status=pic.PIC_DEV_BAD_BLOCK, check=False)
    for r, n in enumerate(c.lens):
        head, tail = np.array([s for s in range(100) if s // 16 != 2]), np.arange(100, n)
        k, v = (torch.cat([_wide_rows(x[0], c.prefix_table, head, 16), _wide_rows(x[0], c.tables[r], tail, 16)], 1) for x in (c.k, c.v))
        _assert_rows(q[r:r + 1], k, v, torch.ones(1, k.shape[1], dtype=torch.bool, device=DEV), 128 ** -0.5, out[r:r + 1], lse[r:r + 1], r)
    c.close()


# ------------------------------------------------------- captured, side by side

def test_captured_steps_follow_the_device_arrays():
    """A graph of the four calls, replayed while lengths, slots and the prefix change, on a stream of its own."""
    heads, hq, d, bs = 2, 8, 128, 16
    c = Cache(heads=heads, d=d, bs=bs, lens=[200, 90, 333], room=60, seed=11)
    lens, grow, n_free = _i32([150, 60, 300]), _i32([3, 0, 5]), _i32([2])
    free = _i32([c.nb - 1, c.nb - 2] + [0] * (c.nb - 2))
    new_lens, new_free, indptr = torch.empty_like(lens), torch.empty_like(n_free), _i32([0] * 4)
    n = 12
    req, slot, pos = (_i32([0] * n) for _ in range(3))
    rows, w = c.normal(n, hq + 2 * heads, d), c.normal(d)
    q, k, v = rows[:, :hq], rows[:, hq:hq + heads], rows[:, hq + heads:]
    q_out, out, lse = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n, hq, d, dtype=torch.bfloat16, device=DEV), \
        torch.zeros(n, hq, device=DEV)
    dec, dec_lse = torch.zeros(3, hq, d, dtype=torch.bfloat16, device=DEV), torch.zeros(3, hq, device=DEV)
    prefix_len = _i32([40])
    ws = _ws(max(pic.pic_attend_tokens_workspace_bytes(c.ctx, n, 3, hq), pic.pic_attend_shared_workspace_bytes(c.ctx, 3, hq)))

    def step(stream=None):
        pic.pic_map_tokens(c.ctx, lens, grow, c.d_tables, free, n_free, new_lens, new_free, indptr, req, slot, positions=pos,
                           workspace=ws)
        pic.pic_write_normed_tokens(c.ctx, pos, k, v, req, slot, c.d_tables, c.k[0], c.v[0], q_norm=w, k_norm=w, q=q, q_out=q_out,
                                    workspace=ws)
        pic.pic_attend_tokens(c.ctx, q_out, 0.09, c.k[0], c.v[0], c.d_tables, indptr, slot, out, window=64, n_first=4, lse=lse,
                              workspace=ws)
        pic.pic_attend_shared(c.ctx, q_out[:3], 0.09, c.k[0], c.v[0], c.d_tables[0], prefix_len, c.d_tables, new_lens,
                              c.tables.shape[1] * bs, dec, lse=dec_lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for new, more, prefix in (([150, 60, 300], [3, 0, 5], 40), ([10, 200, 31], [1, 9, 2], 11), ([0, 0, 7], [12, 0, 0], 0)):
        lens.copy_(_i32(new))
        grow.copy_(_i32(more))
        prefix_len.copy_(_i32([prefix]))
        before_k, before_v = c.k.clone(), c.v.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, lse, dec, dec_lse, q_out, new_lens, indptr, slot, c.k, c.v)]
        c.k.copy_(before_k)
        c.v.copy_(before_v)
        for x in (out, lse, dec, dec_lse, q_out):
            x.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, lse, dec, dec_lse, q_out, new_lens, indptr, slot, c.k, c.v)):
            # (rows of padding keep what they held)
            rows_used = sum(more)
            a, b = (a[:rows_used], b[:rows_used]) if a.shape[:1] == (n,) and a is not got[7] else (a, b)
            assert torch.equal(a, b)
        _assert_step(c, new, more, q_out, out, lse)
    assert _status(c, ws) == 0
    c.close()


def _assert_step(c, lens, grow, q, out, lse):
    at = 0
    for r, (n, g) in enumerate(zip(lens, grow)):
        if g == 0:
            continue
        table = c.d_tables[r].cpu().numpy()
        slots = list(range(n, n + g))
        seen = np.stack([serve.sees(s, np.arange(n + g), 64, 4) for s in slots])
        k, v = (_wide_rows(x[0], table, np.arange(n + g), c.bs) for x in (c.k, c.v))
        _assert_rows(q[at:at + g], k, v, torch.from_numpy(seen).to(DEV), 0.09, out[at:at + g], lse[at:at + g], ("step", r))
        at += g


def test_two_loops_at_once():
    """Calls on two streams with workspaces of their own: the results of each are those it gives alone."""
    c = Cache(heads=4, lens=[4000, 3000], seed=12)
    sides, jobs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        slots = [list(range(3000 + 300 * i, 3400 + 300 * i)), [2999 - i]]
        n = 401
        q = c.normal(n, 16, 128)
        ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, n, 2, 16))
        jobs.append((q, _i32([0, 400, 401]), _i32(slots[0] + slots[1]), ws))

    def attend(job, out, lse):
        q, indptr, slot, ws = job
        pic.pic_attend_tokens(c.ctx, q, 0.088, c.k[0], c.v[0], c.d_tables, indptr, slot, out, window=2000, n_first=4, lse=lse, workspace=ws)

    alone = []
    for job in jobs:
        out, lse = torch.empty_like(job[0]), torch.empty(401, 16, device=DEV)
        attend(job, out, lse)
        alone.append((out, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(torch.empty_like(job[0]), torch.empty(401, 16, device=DEV)) for job in jobs]
        torch.cuda.synchronize()
        for side, job, (out, lse) in zip(sides, jobs, got):
            with torch.cuda.stream(side):
                attend(job, out, lse)
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(alone, got):
            assert torch.equal(a, x) and torch.equal(b, y)
    c.close()


def test_binding_refuses_wrong_tensors():
    c = Cache(heads=2, lens=[40], seed=1)
    q, out = c.normal(4, 8, 128), torch.empty(4, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = _ws(pic.pic_attend_tokens_workspace_bytes(c.ctx, 4, 1, 8))
    good = dict(q=q, softmax_scale=0.1, k_cache=c.k[0], v_cache=c.v[0], block_tables=c.d_tables, indptr=_i32([0, 4]), slot=_i32([1, 2, 3, 4]),
                out=out, workspace=ws)
    pic.pic_attend_tokens(c.ctx, **good)
    for name, bad in (("out", out.float()), ("out", out[:3]), ("slot", _i32([1])), ("indptr", _i32([])), ("slot", _i32([1, 2, 3, 4]).long()),
                      ("q", q.float()), ("block_tables", c.d_tables.long()), ("k_cache", c.k)):
        with pytest.raises((ValueError, pic.PicError)):
            pic.pic_attend_tokens(c.ctx, **{**good, name: bad})
    for name, bad in (("q", q.cpu()), ("slot", _i32([1, 2, 3, 4]).cpu()), ("out", out.cpu()), ("workspace", ws[:100])):
        with pytest.raises((ValueError, pic.PicError)):
            pic.pic_attend_tokens(c.ctx, **{**good, name: bad})
    k = c.normal(1, 2, 128)
    for bad in (c.normal(64), c.normal(128).half(), c.normal(2, 128)):
        with pytest.raises(ValueError):
            pic.pic_write_normed_tokens(c.ctx, _i32([0]), k, k, _i32([0]), _i32([0]), c.d_tables, c.k[0], c.v[0], k_norm=bad, workspace=ws)
    c.close()


# ------------------------------------------------------------------ together

def test_a_serving_step_end_to_end():
    """Prompts over a shared prefix, then decode steps, blocks from the pile: every attention against the rows that
    the cache holds, and the rows against the oracle's norm and rotation."""
    heads, hq, d, bs, blocks, cols = 2, 8, 128, 16, 80, 20
    m = Cache(heads=heads, d=d, bs=bs, lens=[1], seed=21)
    ctx = pic.pic_create(pic.PIC_KIND_GQA, 1, heads, d, d, 0, pic.PIC_PAIRING_NEOX_HALF, bs, 5e5, blocks)
    k_cache = torch.full((blocks, bs, heads, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    v_cache = torch.full_like(k_cache, float("inf"))
    tables, free = _i32(np.full((3, cols), -1)), _i32(np.random.default_rng(0).permutation(blocks))
    n_free, lens = _i32([blocks]), _i32([0, 0, 0])
    w = [m.normal(d) + 1.0 for _ in range(2)]
    ws = _ws(max(pic.pic_attend_tokens_workspace_bytes(ctx, 300, 3, hq), pic.pic_attend_shared_workspace_bytes(ctx, 3, hq)))

    def step(grow, n):
        indptr, req, slot, pos = _i32([0] * 4), _i32([0] * n), _i32([0] * n), _i32([0] * n)
        pic.pic_map_tokens(ctx, lens, _i32(grow), tables, free, n_free, lens, n_free, indptr, req, slot, positions=pos, workspace=ws)
        rows = m.normal(n, hq + 2 * heads, d)
        q, k, v = rows[:, :hq], rows[:, hq:hq + heads], rows[:, hq + heads:]
        q_out = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        pic.pic_write_normed_tokens(ctx, pos, k, v, req, slot, tables, k_cache, v_cache, q_norm=w[0], k_norm=w[1], q=q, q_out=q_out,
                                    workspace=ws)
        return indptr, slot, q_out, k, pos

    # the prefix: 100 tokens of request 0, whose whole blocks the others then share
    indptr, slot, q, k, pos = step([100, 0, 0], 103)
    want = serve.write_normed(_f64(q), _f64(k), None, _f64(w[1]), 1e-6, 0.0, pos.cpu().numpy()[None], [0] * (d // 2), m.theta, m.pairing,
                              0, d)[1][:100]
    t0 = tables[0].cpu().numpy()
    got = _f64(k_cache)[t0[np.arange(100) // bs], np.arange(100) % bs]
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -9) + 2.0 ** -15 * _pair_length(want, m))
    whole = 96
    tables[1:, :whole // bs] = tables[0, :whole // bs]
    lens[1:] = whole
    prefix_table, prefix_len = tables[0, :whole // bs].clone(), _i32([whole])
    # a question each, with a window; then decode steps
    indptr, slot, q, *_ = step([7, 30, 17], 60)
    out, lse = torch.zeros(60, hq, d, dtype=torch.bfloat16, device=DEV), torch.zeros(60, hq, device=DEV)
    pic.pic_attend_tokens(ctx, q, d ** -0.5, k_cache, v_cache, tables, indptr, slot, out, window=50, n_first=4, lse=lse, workspace=ws)
    at = indptr.cpu().tolist()
    host, now = tables.cpu().numpy(), lens.cpu().tolist()
    assert now == [107, 126, 113]
    for r in range(3):
        a = slice(at[r], at[r + 1])
        slots = slot[a].cpu().tolist()
        seen = torch.from_numpy(np.stack([serve.sees(s, np.arange(now[r]), 50, 4) for s in slots])).to(DEV)
        k, v = (_wide_rows(x, host[r], np.arange(now[r]), bs) for x in (k_cache, v_cache))
        _assert_rows(q[a], k, v, seen, d ** -0.5, out[a], lse[a], ("question", r))
    for _ in range(20):
        indptr, slot, q, *_ = step([1, 1, 1], 3)
        out, lse = torch.empty(3, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(3, hq, device=DEV)
        pic.pic_attend_shared(ctx, q, d ** -0.5, k_cache, v_cache, prefix_table, prefix_len, tables, lens, cols * bs, out, lse=lse,
                              workspace=ws)
    host, now = tables.cpu().numpy(), lens.cpu().tolist()
    assert now == [127, 146, 133]
    for r in range(3):
        k, v = (_wide_rows(x, host[r], np.arange(now[r]), bs) for x in (k_cache, v_cache))
        _assert_rows(q[r:r + 1], k, v, torch.ones(1, now[r], dtype=torch.bool, device=DEV), d ** -0.5, out[r:r + 1], lse[r:r + 1], r)
    # two requests end: every block is in one place again (the prefix's stay with request 0)
    lens[1:] -= whole
    tables[1:, :cols - whole // bs] = tables[1:, whole // bs:].clone()
    before = sorted(set(host[0][:-(-127 // bs)].tolist()))
    step([0, -50, -37], 1)
    assert lens.cpu().tolist() == [127, 0, 0] and pic.pic_query_device_status(ctx, ws) == 0
    assert sorted(free[:int(n_free)].cpu().tolist() + before) == list(range(blocks))
    pic.pic_destroy(ctx)
    m.close()
