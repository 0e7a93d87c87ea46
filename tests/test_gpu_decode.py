"""GPU parity of the decode loop over a paged cache against the fp64 oracle:
token writes at positions of one or several axes, paged attention of one new
token with its accumulated weights, eviction by weight, and the three run
together after a stitch.

Tolerances.  A rotated bf16 element: half a step of its value (2^-8 relative)
plus fp32 arithmetic and the angle, 2^-19 of its pair's length.  Attention: a
score of D fp32-accumulated products is off by (D + 8) 2^-23 sum |q k|
(tensor cores may truncate, hence 2^-23); a probability by twice that largest
score error plus 2^-20 for the exponentials and P's split, and a sum over T of
them by another T 2^-23 at most, all relative to sum p |v| (1 for the weights);
bf16 outputs add half a step.  Indices, values, weights moved and untouched
rows are compared bit for bit."""

import math

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_util import Stitched, bits, pairing_of, theta_of
from position_independent_kv_stitch_gb300 import pic

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pic.load(build_if_missing=True)


class Cache:
    """A context with random caches, weights and shuffled block tables; lens[r] slots in use."""

    def __init__(self, kind="gqa", heads=2, d=128, bs=16, layers=1, lens=(40,), room=0, pairing="neox", weight_heads=None, seed=0,
                 theta=5e5):
        self.m = W.Model("dec", "gqa", layers, heads, d, d, 0, pairing, theta, bs) if kind == "gqa" else \
            W.Model("dec", "mla", layers, 1, 576, 64, 512, pairing, theta, bs)
        self.kind, self.bs, self.layers, self.lens = kind, bs, layers, list(lens)
        self.heads, self.d = self.m.num_kv_heads, self.m.head_dim
        self.wh = self.heads if weight_heads is None else weight_heads
        per = max(1, -(-(max(lens) + room) // bs))
        self.nb = per * len(lens) + 3
        rng = np.random.default_rng(seed)
        order = rng.permutation(self.nb)
        self.tables = order[:per * len(lens)].reshape(len(lens), per).astype(np.int32)
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.rng = rng
        shape = (layers, self.nb, bs, self.heads, self.d)
        self.k, self.v = self.normal(*shape), self.normal(*shape) if kind == "gqa" else None
        self.w = torch.rand((layers, self.nb, self.wh, bs), generator=self.g, device=DEV)
        self.d_tables = torch.from_numpy(self.tables).to(DEV)
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.ctx = pic.create_from_spec(pic.model_spec_from(self.m), self.nb)
        self.theta, self.pairing = theta_of(self.m), pairing_of(self.m)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV).to(torch.bfloat16)

    def host(self, layer=0):
        return (self.k[layer].double().cpu().numpy(), None if self.v is None else self.v[layer].double().cpu().numpy(),
                self.w[layer].double().cpu().numpy())

    def close(self):
        pic.pic_destroy(self.ctx)


def _ws(n=pic.PIC_STATUS_BYTES):
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


def _status(c, ws):
    return pic.pic_query_device_status(c.ctx, ws, raise_on_device_error=False)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV).contiguous()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _pair_length(rows, c):
    """Length of each element's pair (0 outside the rope slice)."""
    a, b = oracle.rope_pairs(c.m.rope_dim, c.pairing)
    off = c.m.rope_offset
    out = np.zeros_like(rows)
    n = np.hypot(rows[..., off + np.asarray(a)], rows[..., off + np.asarray(b)])
    out[..., off + np.asarray(a)] = n
    out[..., off + np.asarray(b)] = n
    return out


def _assert_rotated(got, want, c, what):
    err = np.abs(got - want) - 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -9) - 2.0 ** -19 * _pair_length(want, c)
    assert err.max() <= 0, f"{what}: {(err > 0).sum()} of {err.size} off, worst by {err.max():.2e}"


# ------------------------------------------------------------------- writes

def _write(c, n_tok, axes, hq, layer=0, fused=False, in_place=False, pad=0, weights=True, far=False, freq_axis="cycle"):
    half = c.m.rope_dim // 2
    fx = None if freq_axis is None else [f % axes for f in range(half)]
    pos = c.rng.integers(-(1 << 24) + 1, 1 << 24, size=(axes, n_tok)) if far else c.rng.integers(0, 40000, size=(axes, n_tok))
    # distinct free places behind the sequences
    places = [(r, s) for r, n in enumerate(c.lens) for s in range(n, c.tables.shape[1] * c.bs)]
    pick = c.rng.permutation(len(places))[:n_tok]
    req, slot = np.array([places[i][0] for i in pick]), np.array([places[i][1] for i in pick])
    if pad:
        slot[:pad] = -1
        req[:pad] = 12345
    gqa = c.kind == "gqa"
    if fused:
        all_rows = c.normal(n_tok, hq + 2 * c.heads, c.d)
        q, k, v = all_rows[:, :hq], all_rows[:, hq:hq + c.heads], all_rows[:, hq + c.heads:]
    else:
        q, k, v = c.normal(n_tok, hq, c.d), c.normal(n_tok, c.heads, c.d), c.normal(n_tok, c.heads, c.d)
    v = v if gqa else None
    kh, vh, wh = c.host(layer)
    want = oracle.write_tokens(_f64(q), _f64(k), None if v is None else _f64(v), pos, fx or [0] * half, c.theta, c.pairing,
                               c.m.rope_offset, c.m.rope_dim, req, slot, c.tables, c.bs, kh, vh, wh)
    q_out = q if in_place else torch.full((n_tok, hq, c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _ws()
    pic.pic_write_tokens(c.ctx, _i32(pos if axes > 1 else pos[0]), k, v, _i32(req), _i32(slot), c.d_tables, c.k[layer],
                         None if v is None else c.v[layer], q=q, q_out=q_out, freq_axis=fx,
                         weights=c.w[layer] if weights else None, workspace=ws)
    assert _status(c, ws) == 0
    _assert_rotated(_f64(q_out), want[0], c, "q")
    got_k = _f64(c.k[layer])
    _assert_rotated(got_k, want[1], c, "k")
    mask = np.ones(got_k.shape[:2], bool)
    for r, s in zip(req, slot):
        if s >= 0:
            mask[c.tables[r][s // c.bs], s % c.bs] = False
    np.testing.assert_array_equal(got_k[mask], kh[mask])        # rows nobody wrote
    lat = c.m.rope_offset
    np.testing.assert_array_equal(got_k[..., :lat], want[1][..., :lat])
    if v is not None:
        np.testing.assert_array_equal(_f64(c.v[layer]), want[2])
    np.testing.assert_array_equal(_f64(c.w[layer]), want[3] if weights else wh)


@pytest.mark.parametrize("heads,hq,d,bs,pairing", [(2, 8, 128, 16, "neox"), (8, 32, 128, 16, "interleaved"), (1, 7, 64, 1, "neox"),
                                                   (3, 15, 64, 17, "interleaved"), (5, 5, 256, 256, "neox"),
                                                   (4, 4, 256, 7, "interleaved"), (16, 48, 64, 64, "neox")])
@pytest.mark.parametrize("n_tok,axes", [(1, 1), (37, 3), (200, 4)])
def test_write_tokens(heads, hq, d, bs, pairing, n_tok, axes):
    c = Cache(heads=heads, d=d, bs=bs, pairing=pairing, lens=[5, 0, 31], room=-(-n_tok // 3) + bs, seed=heads + n_tok)
    _write(c, n_tok, axes, hq)
    c.close()


@pytest.mark.parametrize("pairing", ["neox", "interleaved"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_tok,hq", [(1, 16), (33, 3), (7, 128)])
def test_write_tokens_mla(pairing, in_place, n_tok, hq):
    c = Cache("mla", bs=16, pairing=pairing, lens=[5, 9], room=60, seed=n_tok)
    _write(c, n_tok, 2, hq, in_place=in_place)
    c.close()


@pytest.mark.parametrize("kw", [dict(fused=True), dict(in_place=True), dict(fused=True, in_place=True), dict(pad=6), dict(far=True),
                                dict(weights=False), dict(freq_axis=None, axes=1), dict(layer=2)])
def test_write_tokens_forms(kw):
    kw = dict(kw)
    c = Cache(heads=4, d=128, layers=3, lens=[20, 3], room=90, weight_heads=1 if kw.get("pad") else None, seed=5)
    _write(c, 70, kw.pop("axes", 3), 12, **kw)
    c.close()


def test_write_queries_only_and_the_inverse():
    """Without keys nothing but q is written; negated positions turn back (the rotation's gradient)."""
    c = Cache(heads=2, lens=[4], seed=3)
    q = c.normal(9, 6, 128)
    pos = c.rng.integers(0, 1 << 20, size=(3, 9))
    fx = [f % 3 for f in range(64)]
    out, back, ws = torch.empty_like(q), torch.empty_like(q), _ws()
    before = bits(c.k)
    pic.pic_write_tokens(c.ctx, _i32(pos), None, None, None, None, None, None, None, q=q, q_out=out, freq_axis=fx, workspace=ws)
    pic.pic_write_tokens(c.ctx, _i32(-pos), None, None, None, None, None, None, None, q=out, q_out=back, freq_axis=fx, workspace=ws)
    assert _status(c, ws) == 0
    want = np.stack([oracle.rotate_axes(_f64(q)[i], pos[:, i], fx, c.theta, c.pairing, 0, 128) for i in range(9)])
    _assert_rotated(_f64(out), want, c, "q")
    # turned twice, each time rounded: half a step of two pair lengths
    lim = 2 * 2.0 ** -8 * _pair_length(_f64(q), c) + 2.0 ** -17
    assert np.all(np.abs(_f64(back) - _f64(q)) <= lim)
    np.testing.assert_array_equal(bits(c.k), before)
    c.close()


def test_write_bad_tokens_are_left_out():
    c = Cache(heads=2, lens=[16, 16], room=16, seed=4)
    c.d_tables[1, 1] = c.nb          # a block outside the cache
    k, v, q = c.normal(6, 2, 128), c.normal(6, 2, 128), c.normal(6, 4, 128)
    req, slot = [0, 1, 2, -1, 0, 0], [16, 16, 3, 3, 32, 17]   # good, bad block, bad rows twice, past the table, far position
    pos = [3, 4, 5, 6, 7, 1 << 24]
    q_out, ws = torch.full_like(q, 9.0), _ws()
    kb, vb = c.k[0].clone(), c.v[0].clone()
    pic.pic_write_tokens(c.ctx, _i32(pos), k, v, _i32(req), _i32(slot), c.d_tables, c.k[0], c.v[0], q=q, q_out=q_out, workspace=ws)
    assert _status(c, ws) == pic.PIC_DEV_BAD_BLOCK | pic.PIC_DEV_BAD_POS
    page = int(c.tables[0][1])
    np.testing.assert_array_equal(bits(c.v[0][page, 0]), bits(v[0]))
    kb[page, 0], vb[page, 0] = c.k[0][page, 0], c.v[0][page, 0]
    assert torch.equal(c.k[0], kb) and torch.equal(c.v[0], vb)
    want = np.stack([oracle.rotate(_f64(q)[i], pos[i], c.theta, c.pairing) for i in range(5)])
    _assert_rotated(_f64(q_out[:5]), want, c, "q")
    assert bool((q_out[5] == 9.0).all())
    c.close()


@pytest.mark.parametrize("bs", [1, 2, 3, 7, 48, 100, 255, 256])
def test_write_tokens_finds_every_slot(bs):
    """Slots over a long table, the first and last of its blocks among them: the values lie where slot // bs says."""
    c = Cache(heads=1, d=64, bs=bs, lens=[70000], seed=bs)
    per = c.tables.shape[1]
    edge = np.arange(0, per, max(1, per // 300))
    slots = np.unique(np.concatenate([edge * bs, edge * bs + bs - 1, c.rng.integers(0, per * bs, size=400)]))
    n = len(slots)
    k, v = c.normal(n, 1, 64), c.normal(n, 1, 64)
    ws = _ws()
    pic.pic_write_tokens(c.ctx, _i32(np.zeros(n)), k, v, _i32(np.zeros(n)), _i32(slots), c.d_tables, c.k[0], c.v[0], workspace=ws)
    assert _status(c, ws) == 0
    rows = torch.from_numpy(c.tables[0][slots // bs].astype(np.int64)).to(DEV), torch.from_numpy(slots % bs).to(DEV)
    assert torch.equal(c.v[0][rows], v) and torch.equal(c.k[0][rows], k)
    c.close()


# ---------------------------------------------------------------- attention

def _attend(c, hq, out_type, layer=0, weights=True, scale=None, q=None):
    n = len(c.lens)
    scale = 1.0 / math.sqrt(c.d) if scale is None else scale
    q = c.normal(n, hq, c.d) * 2 if q is None else q
    kh, vh, wh = c.host(layer)
    vh = kh[..., :512] if vh is None else vh
    want = oracle.attend_paged(_f64(q), kh, vh, c.tables, c.lens, c.bs, scale, wh)
    max_len = max(1, max(c.lens))
    out = torch.full((n, hq, vh.shape[-1]), 7.0, dtype=out_type, device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    ws = _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, n, hq, max_len, weights))
    pic.pic_attend_paged(c.ctx, q, scale, c.k[layer], None if c.v is None else c.v[layer], c.d_tables, c.d_lens, max_len, out, lse=lse,
                         weights=c.w[layer] if weights else None, workspace=ws)
    assert _status(c, ws) == 0
    _check_attend(c, q, kh, vh, wh, want, out, lse, scale, c.w[layer] if weights else None)
    return out, lse


def _check_attend(c, q, kh, vh, wh, want, out, lse, scale, w):
    qh, T = _f64(q), max(1, max(c.lens))
    hq = qh.shape[1]
    group = hq // c.heads
    got_out, got_lse = _f64(out), _f64(lse)
    w_tol = np.full(wh.shape, 0.0)
    for r, n in enumerate(c.lens):
        if n == 0:
            assert np.all(got_out[r] == 0) and np.all(np.isneginf(got_lse[r]))
            continue
        at = [(c.tables[r][s // c.bs], s % c.bs) for s in range(n)]
        for h in range(hq):
            keys = np.stack([kh[b, i, h // group] for b, i in at])
            vals = np.stack([vh[b, i, h // group] for b, i in at])
            s_err = scale * (np.abs(keys) @ np.abs(qh[r, h])).max() * (c.d + 8) * 2.0 ** -23
            rel = 2 * s_err + 2.0 ** -20 + T * 2.0 ** -23
            if out.dtype == torch.bfloat16:
                rel += 2.0 ** -16    # P in two bf16 parts
            p = np.exp(scale * (keys @ qh[r, h]) - want[1][r, h])
            lim = rel * (p @ np.abs(vals)) + (2.0 ** -8 * np.abs(want[0][r, h]) * (1 + rel) if out.dtype == torch.bfloat16 else 0)
            err = np.abs(got_out[r, h] - want[0][r, h])
            assert np.all(err <= lim), (r, h, err.max(), lim.min())
            assert abs(got_lse[r, h] - want[1][r, h]) <= s_err + rel + 2.0 ** -22 * abs(want[1][r, h])
            for t, (b, i) in enumerate(at):
                w_tol[b, h // (hq // wh.shape[1]), i] += rel * p[t]
    if w is not None:
        err = np.abs(_f64(w) - want[2])
        assert np.all(err <= w_tol + np.where(w_tol > 0, 2.0 ** -22 * want[2], 0)), err.max()


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,hq,d,bs", [(2, 8, 128, 16), (8, 32, 128, 16), (1, 1, 64, 1), (3, 15, 64, 17), (2, 14, 128, 5),
                                           (2, 16, 256, 64), (1, 12, 128, 16), (2, 32, 64, 32), (1, 16, 256, 16), (1, 40, 128, 256),
                                           (5, 5, 256, 3), (9, 9, 64, 16)])
def test_attend_paged(heads, hq, d, bs, out_type):
    lens = [1, 0, 77, 16, 200, 15, 17, 129]
    c = Cache(heads=heads, d=d, bs=bs, lens=lens, seed=hq, weight_heads=1 if hq % 3 == 0 else heads)
    _attend(c, hq, out_type)
    c.close()


@pytest.mark.parametrize("lens", [[1], [0], [0, 0], [16], [3000], [0, 1, 0], [0, 2500, 0, 0, 33]])
@pytest.mark.parametrize("weights", [False, True])
def test_attend_paged_lengths(lens, weights):
    c = Cache(heads=2, d=128, bs=16, lens=lens, seed=len(lens))
    _attend(c, 8, torch.float32, weights=weights)
    c.close()


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,bs", [(1, 16), (16, 16), (20, 7), (32, 64), (64, 16), (128, 1), (100, 256)])
def test_attend_paged_mla(hq, bs, out_type):
    """Latent rows: 1 to 128 query heads over lengths around the 64-slot steps."""
    c = Cache("mla", bs=bs, lens=[1, 0, 63, 64, 65, 200, 17, 130], seed=hq)
    _attend(c, hq, out_type, scale=0.03)
    c.close()


@pytest.mark.parametrize("lens", [[3000], [0], [5000, 0, 16, 700], [40] * 200])
def test_attend_paged_mla_lengths(lens):
    c = Cache("mla", lens=lens, seed=len(lens))
    _attend(c, 16, torch.float32, scale=0.03)
    c.close()


def test_attend_paged_mla_junk_and_bad_blocks():
    """Rows behind the end hold NaN; a block outside the cache is left out."""
    c = Cache("mla", lens=[70, 33, 100], seed=3)
    q = c.normal(3, 32, 576)
    clean, _ = _attend(c, 32, torch.float32, scale=0.03, weights=False, q=q)
    for r, n in enumerate(c.lens):
        for s in range(n, c.tables.shape[1] * 16):
            c.k[0, int(c.tables[r][s // 16]), s % 16] = float("nan")
    tables = c.d_tables.clone()
    tables[1, 1] = c.nb
    out, ws = torch.empty(3, 32, 512, device=DEV), _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 3, 32, 100))
    pic.pic_attend_paged(c.ctx, q, 0.03, c.k[0], None, tables, c.d_lens, 100, out, workspace=ws)
    assert _status(c, ws) == pic.PIC_DEV_BAD_BLOCK
    assert torch.equal(out[[0, 2]], clean[[0, 2]])
    kh = c.host()[0]
    rows = np.stack([kh[c.tables[1][s // 16], s % 16] for s in range(33) if s // 16 != 1])
    want, _ = oracle.attention_decode(_f64(q[1]), rows, rows[..., :512], 0.03)
    np.testing.assert_allclose(_f64(out[1]), want, atol=1e-4)
    c.close()


def test_attend_paged_many_short_requests():
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 40, size=300)]
    c = Cache(heads=4, d=64, bs=8, lens=lens, seed=1)
    _attend(c, 8, torch.float32)
    c.close()


def test_attend_paged_thousands_of_requests():
    """3,000 requests, half of them empty: what a join needs of the list does not depend on how many came before."""
    rng = np.random.default_rng(5)
    lens = [int(x) * (i % 2) for i, x in enumerate(rng.integers(1, 50, size=3000))]
    c = Cache(heads=1, d=64, bs=16, lens=lens, seed=2)
    q = c.normal(3000, 4, 64)
    out, lse, ws = torch.empty(3000, 4, 64, device=DEV), torch.empty(3000, 4, device=DEV), \
        _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 3000, 4, 64, True))
    w = c.w[0].clone()
    pic.pic_attend_paged(c.ctx, q, 0.125, c.k[0], c.v[0], c.d_tables, c.d_lens, 64, out, lse=lse, weights=w, workspace=ws)
    assert _status(c, ws) == 0
    k = c.k[0][c.d_tables.long()].reshape(3000, 64, 64).double()
    v = c.v[0][c.d_tables.long()].reshape(3000, 64, 64).double()
    x = torch.einsum("rhd,rtd->rht", q.double(), k) * 0.125
    x.masked_fill_(torch.arange(64, device=DEV)[None, None] >= c.d_lens[:, None, None], float("-inf"))
    p = torch.softmax(x, -1).nan_to_num(0.0)
    torch.testing.assert_close(out.double(), torch.einsum("rht,rtd->rhd", p, v), rtol=1e-4, atol=1e-5)
    live = c.d_lens > 0
    torch.testing.assert_close(lse[live].double(), torch.logsumexp(x, -1)[live], rtol=1e-5, atol=1e-5)
    want = c.w[0].double()
    want[c.d_tables.long().flatten(), 0] += p.sum(1).reshape(-1, 16)
    torch.testing.assert_close(w.double(), want, rtol=1e-4, atol=1e-5)
    c.close()


@pytest.mark.parametrize("n", [1, 17, 1000, 40000, 100000, 200000])
def test_attend_paged_weights_of_many_heads(n):
    """32 query heads a weight: a warp's runs from one tile (its lanes share the heads) to more than it holds at once."""
    c = Cache(heads=2, d=64, bs=16, lens=[n], seed=n)
    q = c.normal(1, 64, 64)
    out, ws = torch.empty(1, 64, 64, device=DEV), _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 1, 64, n, True))
    w = c.w[0].clone()
    pic.pic_attend_paged(c.ctx, q, 0.125, c.k[0], c.v[0], c.d_tables, c.d_lens, n, out, weights=w, workspace=ws)
    assert _status(c, ws) == 0
    rows = c.k[0][c.d_tables[0].long()].reshape(-1, 2, 64)[:n].double()
    heads = q[0].double().reshape(2, 32, 64)
    p = torch.softmax(torch.einsum("ghd,tgd->ght", heads, rows) * 0.125, -1).sum(1)
    s_err = 0.125 * torch.einsum("ghd,tgd->ght", heads.abs(), rows.abs()).max().item() * (64 + 8) * 2.0 ** -23
    rel = 2 * s_err + 2.0 ** -20 + n * 2.0 ** -23
    slots = torch.arange(n, device=DEV)
    at = c.d_tables[0].long()[slots // 16]
    got = w[at, :, slots % 16].T.double()
    old = c.w[0][at, :, slots % 16].T.double()
    assert bool(((got - old - p).abs() <= rel * p + 2.0 ** -22 * (old + p)).all())
    want = c.w[0].clone()
    want[at, :, slots % 16] = w[at, :, slots % 16]
    assert torch.equal(w, want)      # no other place
    c.close()


def test_attend_paged_ignores_what_lies_behind_the_end():
    lens = [33, 0, 50, 16]
    c = Cache(heads=2, d=128, bs=16, lens=lens, room=16, seed=2)
    for r, n in enumerate(lens):
        for s in range(n, c.tables.shape[1] * c.bs):
            b, i = int(c.tables[r][s // c.bs]), s % c.bs
            c.k[0, b, i] = float("nan") if s % 2 else float("inf")
            c.v[0, b, i] = float("-inf") if s % 3 else float("nan")
            c.w[0, b, :, i] = float("nan")
    before = c.w.clone()
    kh, vh, wh = c.host()
    q = c.normal(4, 8, 128)
    clean = Cache(heads=2, d=128, bs=16, lens=lens, room=16, seed=2)   # the same rows without the junk
    out, _ = _attend(clean, 8, torch.float32, q=q)
    got, lse, ws = torch.empty(4, 8, 128, device=DEV), torch.empty(4, 8, device=DEV), \
        _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 4, 8, 50, True))
    pic.pic_attend_paged(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, c.d_lens, 50, got, lse=lse, weights=c.w[0], workspace=ws)
    assert _status(c, ws) == 0
    assert torch.equal(got, out)
    behind = torch.isnan(before)
    assert torch.equal(torch.isnan(c.w), behind)
    assert torch.equal(c.w[~behind], clean.w[~behind])
    c.close()
    clean.close()


def test_attend_paged_peaked_and_flat_scores():
    """One key that takes all the weight, late in the sequence, and all scores equal."""
    c = Cache(heads=2, d=128, bs=16, lens=[300, 200], seed=6)
    q = torch.ones(2, 4, 128, device=DEV, dtype=torch.bfloat16)
    c.k.zero_()
    b, i = int(c.tables[0][280 // 16]), 280 % 16
    c.k[0, b, i] = 100.0
    out, lse = _attend(c, 4, torch.float32, q=q)
    for h in range(4):
        np.testing.assert_array_equal(_f64(out[0, h]), _f64(c.v[0, b, i, h // 2]))
    np.testing.assert_allclose(_f64(lse[1]), math.log(200), rtol=2.0 ** -22)
    c.close()


def test_attend_paged_bad_lengths_and_blocks():
    c = Cache(heads=2, d=128, bs=16, lens=[40, 48, 33], seed=7)
    q = c.normal(3, 8, 128)
    ref, _ = _attend(c, 8, torch.float32, weights=False, q=q)
    for bad in (-1, 49, 2 ** 31 - 1, -2 ** 31):
        lens = c.d_lens.clone()
        lens[1] = bad
        out, ws = torch.empty_like(ref), _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 3, 8, 48))
        pic.pic_attend_paged(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, lens, 48, out, workspace=ws)
        assert _status(c, ws) == pic.PIC_DEV_BAD_LENGTH
        assert bool((out[1] == 0).all())
        torch.testing.assert_close(out[[0, 2]], ref[[0, 2]], rtol=1e-5, atol=1e-6)
        # the status stays until it is cleared
        pic.pic_attend_paged(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, c.d_lens, 48, out, workspace=ws)
        assert _status(c, ws) == pic.PIC_DEV_BAD_LENGTH
    # a block outside the cache: its slots are left out, their weights untouched
    for bad in (-1, c.nb, 2 ** 31 - 1, -2 ** 31):
        c2 = Cache(heads=2, d=128, bs=16, lens=[40, 48, 33], seed=7)
        tables = c2.d_tables.clone()
        tables[1, 1] = bad
        before = c2.w.clone()
        out, ws = torch.empty_like(ref), _ws(pic.pic_attend_paged_workspace_bytes(c2.ctx, 3, 8, 48, True))
        pic.pic_attend_paged(c2.ctx, q, 128 ** -0.5, c2.k[0], c2.v[0], tables, c2.d_lens, 48, out, weights=c2.w[0], workspace=ws)
        assert _status(c2, ws) == pic.PIC_DEV_BAD_BLOCK
        kh, vh, _ = c2.host()
        rows = [(c2.tables[1][s // 16], s % 16) for s in range(48) if s // 16 != 1]
        want, _ = oracle.attention_decode(_f64(q[1]), np.stack([kh[a] for a in rows]), np.stack([vh[a] for a in rows]), 128 ** -0.5)
        np.testing.assert_allclose(_f64(out[1]), want, atol=1e-4)
        lost = int(c2.tables[1][1])
        assert torch.equal(c2.w[0, lost], before[0, lost])
        torch.testing.assert_close(out[[0, 2]], ref[[0, 2]], rtol=1e-5, atol=1e-6)
        c2.close()
    c.close()


def test_attend_paged_nothing_attended():
    """A request all of whose blocks are bad, and one whose scores are all -inf: out 0, lse -inf, no weight added."""
    c = Cache(heads=2, d=128, bs=16, lens=[40, 33, 20], seed=17)
    q = c.normal(3, 8, 128)
    q[1] = 1.0
    c.k[0, torch.from_numpy(c.tables[1]).long().to(DEV)] = float("-inf")
    tables = c.d_tables.clone()
    tables[0] = -1
    before = c.w.clone()
    out, lse, ws = torch.full((3, 8, 128), 7.0, device=DEV), torch.full((3, 8), 7.0, device=DEV), \
        _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 3, 8, 48, True))
    pic.pic_attend_paged(c.ctx, q, 0.1, c.k[0], c.v[0], tables, c.d_lens, 48, out, lse=lse, weights=c.w[0], workspace=ws)
    assert _status(c, ws) == pic.PIC_DEV_BAD_BLOCK
    assert bool((out[:2] == 0).all()) and bool(torch.isneginf(lse[:2]).all()) and bool(torch.isfinite(out[2]).all())
    for r in (0, 1):
        mine = torch.from_numpy(c.tables[r]).long().to(DEV)
        assert torch.equal(c.w[0, mine], before[0, mine])
    c.close()


def test_attend_paged_infinite_and_nan_scores():
    """A +inf score or a NaN in a key makes its request's heads NaN, as the definition does, and touches no other."""
    c = Cache(heads=2, d=128, bs=16, lens=[40, 33, 20], seed=18)
    q = torch.ones(3, 8, 128, device=DEV, dtype=torch.bfloat16)
    clean, _ = _attend(c, 8, torch.float32, weights=False, q=q)
    for r, bad in ((0, float("inf")), (1, float("nan"))):
        c.k[0, int(c.tables[r][1]), 3, 0] = bad
    out, ws = torch.empty(3, 8, 128, device=DEV), _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 3, 8, 40))
    pic.pic_attend_paged(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, c.d_lens, 40, out, workspace=ws)
    assert bool(torch.isnan(out[:2, :4]).all())
    assert torch.equal(out[:2, 4:], clean[:2, 4:]) and torch.equal(out[2], clean[2])
    c.close()


def test_attend_paged_shared_prefix_blocks():
    """Requests that share their first blocks (no weights kept)."""
    c = Cache(heads=2, d=128, bs=16, lens=[64, 80, 70], seed=8)
    c.tables[1, :3] = c.tables[0, :3]
    c.tables[2, :3] = c.tables[0, :3]
    c.d_tables = torch.from_numpy(c.tables).to(DEV)
    _attend(c, 8, torch.float32, weights=False)
    c.close()


def test_attend_paged_query_stride_streams_and_repeatability():
    c = Cache(heads=4, d=128, bs=16, lens=[700, 31, 1200], seed=9)
    qkv = c.normal(3, 24, 128)
    q = qkv[:, 4:20]
    side = torch.cuda.Stream()
    kh, vh, wh = c.host()
    want = oracle.attend_paged(_f64(q), kh, vh, c.tables, c.lens, c.bs, 0.1, wh)
    outs = []
    for k in range(3):
        w = c.w.clone()
        out, lse = torch.empty(3, 16, 128, device=DEV), torch.empty(3, 16, device=DEV)
        ws = _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 3, 16, 1200, True))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pic.pic_attend_paged(c.ctx, q, 0.1, c.k[0], c.v[0], c.d_tables, c.d_lens, 1200, out, lse=lse, weights=w[0], workspace=ws)
        side.synchronize()
        outs.append((out, lse, w))
    _check_attend(c, q, kh, vh, wh, want, outs[0][0], outs[0][1], 0.1, outs[0][2][0])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    c.close()


# ----------------------------------------------------------------- eviction

def _evict(c, budget, first, recent, renumber, alias_lens=False):
    n = len(c.lens)
    host = [c.host(l) for l in range(c.layers)]
    want = [oracle.evict_tokens(*host[l], c.tables, np.array(c.lens), c.bs, budget, first, recent, renumber, c.theta, c.pairing,
                                c.m.rope_offset, c.m.rope_dim) for l in range(c.layers)]
    kept = torch.full((c.layers, n, c.wh, budget), -7, dtype=torch.int32, device=DEV)
    new = c.d_lens if alias_lens else torch.full((n,), -7, dtype=torch.int32, device=DEV)
    ws = _ws(pic.pic_evict_workspace_bytes(c.ctx, c.layers, n, c.wh))
    pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, c.d_lens, budget, kept, new, n_first=first, n_recent=recent,
                         renumber=renumber, workspace=ws)
    assert _status(c, ws) == 0
    for l in range(c.layers):
        kn, vn, wn, keep, lens = want[l]
        np.testing.assert_array_equal(kept[l].cpu().numpy(), keep)
        np.testing.assert_array_equal(new.cpu().numpy(), lens)
        np.testing.assert_array_equal(_f64(c.w[l]), wn)
        if vn is not None:
            np.testing.assert_array_equal(_f64(c.v[l]), vn)
        got = _f64(c.k[l])
        if renumber:
            _assert_rotated(got, kn, c, "k")
            same = kn == host[l][0]     # rows that stayed, and whatever lies outside
            np.testing.assert_array_equal(got[same], kn[same])
        else:
            np.testing.assert_array_equal(got, kn)


@pytest.mark.parametrize("renumber", [False, True])
@pytest.mark.parametrize("heads,d,bs,wh,pairing", [(2, 128, 16, 2, "neox"), (2, 128, 16, 1, "interleaved"), (8, 64, 7, 8, "neox"),
                                                   (3, 256, 1, 3, "interleaved"), (4, 64, 256, 1, "neox"), (1, 128, 32, 1, "neox")])
@pytest.mark.parametrize("budget,first,recent", [(50, 4, 10), (1, 0, 0), (1, 1, 0), (64, 0, 64), (33, 16, 17), (128, 3, 5)])
def test_evict_tokens(heads, d, bs, wh, pairing, budget, first, recent, renumber):
    c = Cache(heads=heads, d=d, bs=bs, layers=2, lens=[200, 0, 50, 51, 1, 129], weight_heads=wh, pairing=pairing, seed=budget)
    _evict(c, budget, first, recent, renumber)
    c.close()


@pytest.mark.parametrize("renumber", [False, True])
@pytest.mark.parametrize("pairing", ["neox", "interleaved"])
def test_evict_tokens_mla(renumber, pairing):
    c = Cache("mla", layers=2, bs=16, lens=[300, 90, 100], pairing=pairing, seed=11)
    _evict(c, 91, 4, 20, renumber)
    c.close()


@pytest.mark.parametrize("kind", ["ties", "zeros", "specials", "rising", "falling", "tiny"])
def test_evict_tokens_weights(kind):
    """Equal weights, infinities, NaN, negative and subnormal weights, and orders in which nothing or everything moves."""
    c = Cache(heads=2, d=64, bs=16, lens=[1500, 700], seed=12)
    n = c.w.numel()
    if kind == "ties":
        c.w = torch.randint(0, 3, c.w.shape, generator=c.g, device=DEV).float()
    elif kind == "zeros":
        c.w = torch.where(c.w < 0.5, 0.0, -0.0)
    elif kind == "specials":
        special = torch.tensor([math.inf, -math.inf, math.nan, -1.0, 0.0, -0.0, 1e-42, 3.0], device=DEV)
        c.w = special[torch.randint(0, 8, c.w.shape, generator=c.g, device=DEV)]
    elif kind == "tiny":
        c.w = c.w * 1e-39
    else:
        seq = torch.arange(n, device=DEV).float().reshape(c.w.shape)
        order = torch.empty(c.nb, dtype=torch.long, device=DEV)
        order[torch.from_numpy(c.tables.reshape(-1)).long().to(DEV)] = torch.arange(c.tables.size, device=DEV)
        by_slot = (order[:, None, None] * c.bs + torch.arange(c.bs, device=DEV)).expand(-1, 2, -1).float()
        c.w = (by_slot if kind == "rising" else -by_slot)[None].contiguous() + 0 * seq
    _evict(c, 600, 5, 30, True, alias_lens=True)
    c.close()


def test_evict_longer_than_many_tiles():
    c = Cache(heads=2, d=128, bs=16, lens=[9001, 5000], seed=13)
    _evict(c, 4099, 4, 300, True)
    c.close()


def test_evict_bad_requests_are_left_alone():
    c = Cache(heads=2, d=128, bs=16, layers=2, lens=[60, 60, 60], seed=14)
    for change, flag in ((lambda t, n: t.__setitem__((1, 2), c.nb), pic.PIC_DEV_BAD_BLOCK),
                         (lambda t, n: t.__setitem__((1, 0), -1), pic.PIC_DEV_BAD_BLOCK),
                         (lambda t, n: n.__setitem__(1, 65), pic.PIC_DEV_BAD_LENGTH),
                         (lambda t, n: n.__setitem__(1, -3), pic.PIC_DEV_BAD_LENGTH)):
        tables, lens = c.d_tables.clone(), c.d_lens.clone()
        change(tables, lens)
        k, v, w = c.k.clone(), c.v.clone(), c.w.clone()
        kept, ws = torch.empty(2, 3, 2, 20, dtype=torch.int32, device=DEV), _ws(pic.pic_evict_workspace_bytes(c.ctx, 2, 3, 2))
        length = int(lens[1])
        pic.pic_evict_tokens(c.ctx, k, v, w, tables, lens, 20, kept, lens, workspace=ws)
        assert _status(c, ws) == flag
        assert lens.tolist() == [20, length, 20]
        assert bool((kept[:, 1] == -1).all()) and bool((kept[:, [0, 2]] >= 0).all())
        mine = torch.from_numpy(c.tables[1]).long().to(DEV)
        assert torch.equal(k[:, mine], c.k[:, mine]) and torch.equal(v[:, mine], c.v[:, mine]) and torch.equal(w[:, mine], c.w[:, mine])
    c.close()


# ------------------------------------------------------------- run together

def _decode_steps(c, steps, budget, slack, hq, renumber, graph):
    """A decode loop on every layer of a cache: write, attend with weights, and
    evict when a sequence has outgrown budget + slack; checked per step
    against the oracle run from the device's own cache."""
    n, half = len(c.lens), c.m.rope_dim // 2
    limit = c.tables.shape[1] * c.bs
    fx = [f % 3 for f in range(half)]
    qkv = torch.empty(n, hq + 2 * c.heads, c.d, dtype=torch.bfloat16, device=DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + c.heads], qkv[:, hq + c.heads:]
    q_out = torch.empty(n, hq, c.d, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty(n, hq, c.d, device=DEV), torch.empty(n, hq, device=DEV)
    pos = torch.empty(3, n, dtype=torch.int32, device=DEV)
    req, slot = _i32(range(n)), torch.empty(n, dtype=torch.int32, device=DEV)
    lens = c.d_lens
    ws_w, ws_a = _ws(), _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, n, hq, limit, True))
    ws_e = _ws(pic.pic_evict_workspace_bytes(c.ctx, c.layers, n, c.wh))
    kept = torch.empty(c.layers, n, c.wh, budget, dtype=torch.int32, device=DEV)
    scale = c.d ** -0.5

    def step(layer):
        pic.pic_write_tokens(c.ctx, pos, k, v, req, slot, c.d_tables, c.k[layer], c.v[layer], q=q, q_out=q_out, freq_axis=fx,
                             weights=c.w[layer], workspace=ws_w)
        pic.pic_attend_paged(c.ctx, q_out, scale, c.k[layer], c.v[layer], c.d_tables, lens, limit, out, lse=lse,
                             weights=c.w[layer], workspace=ws_a)

    graphs = {}
    if graph:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for layer in range(c.layers):
                graphs[layer] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graphs[layer], stream=stream):
                    step(layer)
        torch.cuda.synchronize()
    position = list(c.lens)
    for _ in range(steps):
        slot.copy_(lens)
        lens.add_(1)
        c.lens = lens.tolist()
        pos.copy_(torch.tensor([[p, p // 2, p % 50] for p in position], dtype=torch.int32).T)
        for layer in range(c.layers):
            qkv.normal_(generator=c.g)
            kh, vh, wh = c.host(layer)
            want = oracle.write_tokens(_f64(q), _f64(k), _f64(v), pos.cpu().numpy(), fx, c.theta, c.pairing, 0, c.d, range(n),
                                       slot.tolist(), c.tables, c.bs, kh, vh, wh)
            graphs[layer].replay() if graph else step(layer)
            torch.cuda.synchronize()
            _assert_rotated(_f64(q_out), want[0], c, "q")
            kn, vn, _ = c.host(layer)
            _assert_rotated(kn, want[1], c, "k")
            np.testing.assert_array_equal(vn, want[2])
            att = oracle.attend_paged(_f64(q_out), kn, vn, c.tables, c.lens, c.bs, scale, want[3])
            _check_attend(c, q_out, kn, vn, want[3], att, out, lse, scale, c.w[layer])
        position = [p + 1 for p in position]
        if max(c.lens) > budget + slack:
            host = [c.host(l) for l in range(c.layers)]
            pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, lens, budget, kept, lens, n_first=2, n_recent=8,
                                 renumber=renumber, workspace=ws_e)
            torch.cuda.synchronize()
            for l in range(c.layers):
                kn, vn, wn, keep, new = oracle.evict_tokens(*host[l], c.tables, np.array(c.lens), c.bs, budget, 2, 8, renumber,
                                                            c.theta, c.pairing, 0, c.d)
                np.testing.assert_array_equal(kept[l].cpu().numpy(), keep)
                np.testing.assert_array_equal(_f64(c.w[l]), wn)
                np.testing.assert_array_equal(_f64(c.v[l]), vn)
                _assert_rotated(_f64(c.k[l]), kn, c, "k after eviction")
            assert lens.tolist() == new.tolist()
            if renumber:
                position = lens.tolist()
    for ws in (ws_w, ws_a, ws_e):
        assert _status(c, ws) == 0
    assert max(lens.tolist()) <= budget + slack + 1


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("renumber", [False, True])
def test_decode_loop(renumber, graph):
    c = Cache(heads=2, d=64, bs=8, layers=2, lens=[30, 12, 44], room=30, seed=20 + renumber)
    c.w.zero_()
    _decode_steps(c, 14, 36, 5, 6, renumber, graph)
    c.close()


def test_decode_loop_mla():
    """Write, attend and evict over latent rows, step by step against the oracle."""
    c = Cache("mla", bs=16, lens=[20, 33], room=30, seed=50)
    c.w.zero_()
    hq, budget, scale = 16, 36, 0.03
    q_out, out = torch.empty(2, hq, 576, dtype=torch.bfloat16, device=DEV), torch.empty(2, hq, 512, device=DEV)
    lse, lens, ws = torch.empty(2, hq, device=DEV), c.d_lens, _ws(1 << 25)
    kept = torch.empty(1, 2, 1, budget, dtype=torch.int32, device=DEV)
    for step in range(8):
        slot = lens.clone()
        lens.add_(1)
        c.lens = lens.tolist()
        q, k = c.normal(2, hq, 576), c.normal(2, 1, 576)
        kh, _, wh = c.host()
        want = oracle.write_tokens(_f64(q), _f64(k), None, slot.cpu().numpy()[None], [0] * 32, c.theta, c.pairing, 512, 64, [0, 1],
                                   slot.tolist(), c.tables, c.bs, kh, None, wh)
        pic.pic_write_tokens(c.ctx, slot, k, None, _i32([0, 1]), slot, c.d_tables, c.k[0], None, q=q, q_out=q_out, weights=c.w[0],
                             workspace=ws)
        pic.pic_attend_paged(c.ctx, q_out, scale, c.k[0], None, c.d_tables, lens, c.tables.shape[1] * 16, out, lse=lse,
                             weights=c.w[0], workspace=ws)
        _assert_rotated(_f64(q_out), want[0], c, "q")
        kn = c.host()[0]
        _assert_rotated(kn, want[1], c, "k")
        att = oracle.attend_paged(_f64(q_out), kn, kn[..., :512], c.tables, c.lens, c.bs, scale, want[3])
        _check_attend(c, q_out, kn, kn[..., :512], want[3], att, out, lse, scale, c.w[0])
        if max(c.lens) > budget + 3:
            host = c.host()
            pic.pic_evict_tokens(c.ctx, c.k, None, c.w, c.d_tables, lens, budget, kept, lens, n_first=1, n_recent=4, renumber=True,
                                 workspace=ws)
            kn, _, wn, keep, new = oracle.evict_tokens(*host, c.tables, np.array(c.lens), c.bs, budget, 1, 4, True, c.theta, c.pairing,
                                                       512, 64)
            np.testing.assert_array_equal(kept[0].cpu().numpy(), keep)
            np.testing.assert_array_equal(_f64(c.w[0]), wn)
            _assert_rotated(_f64(c.k[0]), kn, c, "k after eviction")
            assert lens.tolist() == new.tolist()
    assert _status(c, ws) == 0
    c.close()


def test_evict_captured_and_replayed():
    """An eviction in a graph, replayed: the second replay finds sequences within the budget and leaves them."""
    c = Cache(heads=2, d=64, bs=16, layers=2, lens=[200, 90, 61], seed=41)
    k, v, w, lens = c.k.clone(), c.v.clone(), c.w.clone(), c.d_lens.clone()
    kept = torch.empty(2, 3, 2, 70, dtype=torch.int32, device=DEV)
    ws = _ws(pic.pic_evict_workspace_bytes(c.ctx, 2, 3, 2))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            pic.pic_evict_tokens(c.ctx, k, v, w, c.d_tables, lens, 70, kept, lens, n_first=2, n_recent=9, renumber=True, workspace=ws)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [70, 70, 61]
    once = k.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(k, once) and kept[0, 0, 0].tolist() == list(range(70))
    d = c.d_lens.clone()
    pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, d, 70, kept, d, n_first=2, n_recent=9, renumber=True, workspace=ws)
    assert _status(c, ws) == 0
    assert torch.equal(c.k, once) and torch.equal(c.v, v) and torch.equal(c.w, w)
    c.close()


def test_offsets_beyond_32_bits():
    """A layer of 6.6 GB: rows, weights and pages at its far end."""
    bs, heads, d, nb = 16, 8, 128, 200_000
    m = W.Model("far", "gqa", 1, heads, d, d, 0, "neox", 5e5, bs)
    ctx = pic.create_from_spec(pic.model_spec_from(m), nb)
    k, v = (torch.empty(1, nb, bs, heads, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    w = torch.empty(1, nb, heads, bs, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    pages = [nb - 1, 7, nb - 3, nb - 2, 150_001]
    for p in pages:
        k[0, p].normal_(generator=g)
        v[0, p].normal_(generator=g)
        w[0, p].uniform_(generator=g)
    tables = _i32([pages])
    new = [torch.randn((2, h, d), generator=g, device=DEV).to(torch.bfloat16) for h in (16, heads, heads)]
    small = Cache(heads=heads, d=d, bs=bs, lens=[70], room=10, seed=1)   # the same pages in a small cache
    small.tables = np.arange(5, dtype=np.int32)[None]
    small.d_tables = torch.from_numpy(small.tables).to(DEV)
    small.k[0, :5], small.v[0, :5], small.w[0, :5] = k[0, pages], v[0, pages], w[0, pages]
    for c, kk, vv, ww, tt in ((ctx, k, v, w, tables), (small.ctx, small.k, small.v, small.w, small.d_tables)):
        q_out, lens = torch.empty_like(new[0]), _i32([72])
        ws = _ws(1 << 25)
        pic.pic_write_tokens(c, _i32([70, 71]), new[1], new[2], _i32([0, 0]), _i32([70, 71]), tt, kk[0], vv[0], q=new[0], q_out=q_out,
                             weights=ww[0], workspace=ws)
        out = torch.empty(1, 16, d, device=DEV)
        pic.pic_attend_paged(c, q_out[1:], 0.1, kk[0], vv[0], tt, lens, 72, out, weights=ww[0], workspace=ws)
        kept = torch.empty(1, 1, heads, 33, dtype=torch.int32, device=DEV)
        pic.pic_evict_tokens(c, kk, vv, ww, tt, lens, 33, kept, lens, n_first=1, n_recent=4, renumber=True, workspace=ws)
        assert pic.pic_query_device_status(c, ws) == 0
        if c is ctx:
            want = (out, kept)
    assert torch.equal(out, want[0]) and torch.equal(kept, want[1])
    assert torch.equal(small.k[0, :5], k[0, pages]) and torch.equal(small.v[0, :5], v[0, pages])
    assert torch.equal(small.w[0, :5], w[0, pages])
    pic.pic_destroy(ctx)
    small.close()


def test_decode_loop_after_a_stitch():
    """The prompt comes from pic_stitch; the loop goes on in its blocks and agrees
    with pic_attend_decode over the stitched cache before anything is added."""
    wl = W.tiny_gqa()
    s = Stitched(wl, spare_blocks=0).run()
    m, n = wl.model, len(wl.requests)
    total = wl.request_tokens[0]
    hq = 2 * m.num_kv_heads
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn((n, hq, m.head_dim), generator=g, device=DEV).to(torch.bfloat16)
    scale = m.head_dim ** -0.5
    out, want = torch.empty(n, hq, m.head_dim, device=DEV), torch.empty(1, n, hq, m.head_dim, device=DEV)
    weights = torch.zeros(s.nb, m.num_kv_heads, s.bs, device=DEV)
    lens = _i32(wl.request_tokens)
    ws = _ws(pic.pic_attend_paged_workspace_bytes(s.ctx, n, hq, total, True))
    pic.pic_attend_paged(s.ctx, q, scale, s.k_cache[0], s.v_cache[0], s.d_bt, lens, max(wl.request_tokens), out, weights=weights,
                         workspace=ws)
    aws = torch.empty(pic.pic_attend_workspace_bytes(s.ctx, s.plans, hq, 1), dtype=torch.uint8, device=DEV)
    pic.pic_attend_decode(s.ctx, s.plans, pic.PIC_ATTEND_CACHE, q[None], scale, s.k_pool, s.v_pool, s.k_cache, s.v_cache, want,
                          workspace=aws)
    assert pic.pic_query_device_status(s.ctx, ws) == 0 and pic.pic_query_device_status(s.ctx, aws) == 0
    torch.testing.assert_close(out, want[0], rtol=2e-5, atol=2e-5)
    assert abs(float(weights.sum()) - n * hq) < 1e-3 * n * hq
    budget = total // 3
    kept, ews = torch.empty(1, n, m.num_kv_heads, budget, dtype=torch.int32, device=DEV), \
        _ws(pic.pic_evict_workspace_bytes(s.ctx, 1, n, m.num_kv_heads))
    before = s.v_cache.clone()
    pic.pic_evict_tokens(s.ctx, s.k_cache, s.v_cache, weights[None], s.d_bt, lens, budget, kept, lens, n_first=4, n_recent=16,
                         renumber=True, workspace=ews)
    assert pic.pic_query_device_status(s.ctx, ews) == 0 and lens.tolist() == [budget] * n
    kh = kept.cpu().numpy()
    for h in range(m.num_kv_heads):
        for j in (0, 3, 4, budget // 2, budget - 1):
            src = int(kh[0, 0, h, j])
            a, b = s.tables[0][j // s.bs], s.tables[0][src // s.bs]
            assert torch.equal(s.v_cache[0, a, j % s.bs, h], before[0, b, src % s.bs, h])
    s.close()


def test_attend_paged_more_heads_than_warps():
    """1,500 KV heads: every warp of the launch serves more than one."""
    c = Cache(heads=1500, d=64, bs=4, lens=[9, 3], seed=30)
    _attend(c, 1500, torch.bfloat16)
    c.close()


@pytest.mark.parametrize("n", [4099, 60000])
@pytest.mark.parametrize("kind", ["one digit", "many ties", "spread"])
def test_evict_selection_borders(kind, n):
    """Long sequences (beyond the weights that shared memory holds, too) whose
    weights share their top bits, or are equal, or are spread: the kept list."""
    c = Cache(heads=1, d=64, bs=16, lens=[n], seed=n)
    if kind == "one digit":
        c.w = 1.0 + c.w / 1024.0
    elif kind == "many ties":
        c.w = torch.floor(c.w * 3.0) * 0.5
    kept, new = torch.empty(1, 1, 1, n // 3, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    w = c.w.clone()
    ws = _ws(pic.pic_evict_workspace_bytes(c.ctx, 1, 1, 1))
    pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, c.d_lens, n // 3, kept, new, n_first=3, n_recent=50, workspace=ws)
    assert _status(c, ws) == 0
    s = np.arange(n)
    by_slot = w[0, torch.from_numpy(c.tables[0][s // 16]).long().to(DEV), 0, torch.from_numpy(s % 16).to(DEV)].double().cpu().numpy()
    want = oracle.kept_slots(by_slot, n, n // 3, 3, 50)
    assert kept[0, 0, 0].tolist() == want
    got = c.w[0, torch.from_numpy(c.tables[0][np.arange(n // 3) // 16]).long().to(DEV), 0, torch.from_numpy(np.arange(n // 3) % 16).to(DEV)]
    np.testing.assert_array_equal(got.double().cpu().numpy(), by_slot[want])
    c.close()


def _assert_small_angles(got, x, angle):
    """got = x sin(angle), |angle| < pi / 4, an element that is small beside its partner x: its own half step of bf16, and 2^-20
    for fp32 (the angle in turns, its sine and the product are each within a few 2^-24 of themselves), relative all of them."""
    want = x * np.sin(angle)
    err = np.abs(got - want) - (2.0 ** -8 + 2.0 ** -20) * np.abs(want)
    assert err.max() <= 0, f"{(err > 0).sum()} of {err.size} off, worst by {(np.abs(got - want) / np.abs(want)).max():.2e} of the value"


@pytest.mark.parametrize("pairing", ["neox", "interleaved"])
@pytest.mark.parametrize("kind", ["gqa", "mla"])
def test_small_angles_keep_their_relative_precision(kind, pairing):
    """Pairs (x, 0) turned by small angles, in a write and in a renumbering eviction: the second element is right
    to bf16's precision of itself, not of x."""
    c = Cache(kind, heads=2, d=128, bs=16, lens=[40], room=16, pairing=pairing, seed=60)
    n_rope, off = c.m.rope_dim, c.m.rope_offset
    a, b = (off + np.asarray(i) for i in oracle.rope_pairs(n_rope, c.pairing))
    theta, second = np.asarray(c.theta), torch.as_tensor(b, device=DEV)
    pos = np.array([1, 2, 7, 40, 1000, -3])
    n = len(pos)
    q, k = c.normal(n, 4, c.d), c.normal(n, c.heads, c.d)
    q[..., second], k[..., second] = 0.0, 0.0
    v = c.normal(n, c.heads, c.d) if kind == "gqa" else None
    slot = np.arange(40, 40 + n)
    q_out, ws = torch.empty_like(q), _ws(1 << 16)
    pic.pic_write_tokens(c.ctx, _i32(pos), k, v, _i32(np.zeros(n)), _i32(slot), c.d_tables, c.k[0], None if v is None else c.v[0],
                         q=q, q_out=q_out, workspace=ws)
    rows = np.stack([_f64(c.k[0])[c.tables[0][s // 16], s % 16] for s in slot])
    angle = pos[:, None] * theta
    near = np.broadcast_to((np.abs(angle) < math.pi / 4)[:, None], q.shape[:2] + angle.shape[1:])
    assert near.mean() > 0.3
    for got, x in ((_f64(q_out), _f64(q)), (rows, _f64(k))):
        m = near[:, :x.shape[1]]
        _assert_small_angles(got[..., b][m], x[..., a][m], np.broadcast_to(angle[:, None], m.shape)[m])
    # an eviction that keeps the first and the last tokens turns the last by the budget less the length
    c.k[..., second] = 0.0
    before, budget = c.host()[0], 37
    kept, new = torch.empty(1, 1, c.wh, budget, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, c.d_lens, budget, kept, new, n_first=10, n_recent=budget - 10,
                         renumber=True, workspace=ws)
    assert _status(c, ws) == 0
    after = c.host()[0]
    m = np.abs(3 * theta) < math.pi / 4
    for j in range(10, budget):
        x = before[c.tables[0][(j + 3) // 16], (j + 3) % 16][:, a][:, m]
        got = after[c.tables[0][j // 16], j % 16][:, b][:, m]
        _assert_small_angles(got, x, np.broadcast_to(-3.0 * theta[m], x.shape))
    c.close()


@pytest.mark.parametrize("n,budget", [(700, 300), (4099, 1000), (60000, 30000)])
@pytest.mark.parametrize("heads,bs", [(2, 16), (1, 7)])
def test_evict_moves_weights_bit_for_bit(n, budget, heads, bs):
    """Signed zeros and NaNs with payloads arrive as they were, in short sequences and in ones whose weights
    shared memory does not hold; slots behind the budget keep theirs."""
    c = Cache(heads=heads, d=64, bs=bs, lens=[n, 0, n // 2], seed=n + heads)
    raw = c.w.view(torch.int32)
    pick = torch.randint(0, 8, raw.shape, generator=c.g, device=DEV)
    odd = torch.tensor([-2 ** 31, 0x7fc00001, 0x7f800123, -4194000, 0, 0x7fffffff], dtype=torch.int32, device=DEV)   # -0, NaNs, 0
    c.w = torch.where(pick < 6, odd[pick.clamp(max=5)], raw).view(torch.float32)
    before = c.w.clone()
    kept, new = torch.empty(1, 3, heads, budget, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    ws = _ws(pic.pic_evict_workspace_bytes(c.ctx, 1, 3, heads))
    pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, c.d_lens, budget, kept, new, n_first=2, n_recent=60, workspace=ws)
    assert _status(c, ws) == 0
    bits32 = lambda t: t.view(torch.int32).cpu().numpy()  # noqa: E731
    want, old = bits32(before), bits32(before)
    for r, length in enumerate(c.lens):
        if length <= budget:
            continue
        page, row = c.tables[r].astype(np.int64)[np.arange(length) // bs], np.arange(length) % bs
        for h in range(heads):
            w = before[0, torch.from_numpy(page).to(DEV), h, torch.from_numpy(row).to(DEV)].double().cpu().numpy()
            src = kept[0, r, h].cpu().numpy()
            assert src.tolist() == oracle.kept_slots(w, length, budget, 2, 60)
            want[0, page[:budget], h, row[:budget]] = old[0, page[src], h, row[src]]
    np.testing.assert_array_equal(bits32(c.w), want)
    c.close()


@pytest.mark.parametrize("kind", ["gqa", "mla"])
def test_empty_batches(kind):
    """No token and no request, as a serving loop without a live request calls: nothing happens."""
    c = Cache(kind, heads=2, d=128, lens=[20], seed=70)
    hq, dv, before = 4, c.d if kind == "gqa" else 512, (c.k.clone(), c.w.clone())
    i0, q0 = torch.empty(0, dtype=torch.int32, device=DEV), c.normal(3, hq, c.d)[:0]
    k0, v = c.normal(3, c.heads, c.d)[:0], None if c.v is None else c.v[0]
    v0 = None if c.v is None else k0
    ws = _ws(1 << 25)
    for tables in (c.d_tables[:0], c.d_tables):
        for q in (None, q0):
            pic.pic_write_tokens(c.ctx, i0, k0, v0, i0, i0, tables, c.k[0], v, q=q, q_out=q, weights=c.w[0], workspace=ws)
        pic.pic_write_tokens(c.ctx, i0.view(2, 0), None, None, None, None, None, None, None, q=q0, q_out=q0, workspace=ws,
                             freq_axis=[0, 1] * (c.m.rope_dim // 4))
        for w in (None, c.w[0]):
            pic.pic_attend_paged(c.ctx, q0, 0.1, c.k[0], v, tables, i0, 20, torch.empty(0, hq, dv, device=DEV),
                                 lse=torch.empty(0, hq, device=DEV), weights=w, workspace=ws)
        pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, tables, i0, 7, torch.empty(1, 0, c.wh, 7, dtype=torch.int32, device=DEV), i0,
                             n_first=1, n_recent=2, workspace=ws)
    assert _status(c, ws) == 0 and torch.equal(c.k, before[0]) and torch.equal(c.w, before[1])
    c.close()


def test_requests_without_blocks():
    """Tables of no blocks and sequences of no slots: outputs 0, nothing kept, keys without a place raise."""
    c = Cache(heads=2, d=128, lens=[20], seed=71)
    tables, lens = torch.empty(2, 0, dtype=torch.int32, device=DEV), _i32([0, 0])
    q, ws = c.normal(2, 4, 128), _ws(1 << 25)
    out, lse = torch.full((2, 4, 128), 7.0, device=DEV), torch.empty(2, 4, device=DEV)
    before = c.k.clone()
    pic.pic_attend_paged(c.ctx, q, 0.1, c.k[0], c.v[0], tables, lens, 0, out, lse=lse, weights=c.w[0], workspace=ws)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    kept, new = torch.empty(1, 2, 2, 3, dtype=torch.int32, device=DEV), torch.full((2,), 7, dtype=torch.int32, device=DEV)
    pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, tables, lens, 3, kept, new, workspace=ws)
    assert bool((kept == -1).all()) and new.tolist() == [0, 0] and _status(c, ws) == 0
    pic.pic_write_tokens(c.ctx, lens, c.normal(2, 2, 128), c.normal(2, 2, 128), _i32([0, 1]), _i32([-1, 0]), tables, c.k[0], c.v[0],
                         workspace=ws)
    assert _status(c, ws) == pic.PIC_DEV_BAD_BLOCK and torch.equal(c.k, before)
    c.close()


@pytest.mark.parametrize("kind,heads,hq,d,pairing,n_tok", [("gqa", 8, 32, 128, "neox", 5000), ("gqa", 4, 9, 256, "interleaved", 5001),
                                                           ("gqa", 2, 61, 64, "neox", 4999), ("mla", 1, 64, 576, "interleaved", 2500)])
def test_write_tokens_prompts(kind, heads, hq, d, pairing, n_tok):
    """As many tokens as make a warp take all heads of its token, in several rounds of its two row buffers."""
    c = Cache(kind, heads=heads, d=d, pairing=pairing, lens=[3, 40], room=-(-n_tok // 2) + 16, seed=hq)
    _write(c, n_tok, 3, hq)
    c.close()


@pytest.mark.parametrize("kind", ["gqa", "mla"])
@pytest.mark.parametrize("renumber", [False, True])
def test_evict_layers_apart(kind, renumber):
    """Caches and weights whose layers are slices of larger tensors: nothing between the layers is touched."""
    c = Cache(kind, heads=2, d=64, layers=3, lens=[150, 61, 90], seed=80)
    joint = c.normal(3, 2, *c.k.shape[1:])
    weights = torch.rand((3, 5, *c.w.shape[1:]), generator=c.g, device=DEV)
    joint[:, 0], weights[:, 2] = c.k, c.w
    if kind == "gqa":
        joint[:, 1] = c.v
        c.v = joint[:, 1]
    between = weights.clone(), joint[:, 1].clone()
    c.k, c.w = joint[:, 0], weights[:, 2]
    assert not c.k.is_contiguous() and not c.w.is_contiguous()
    _evict(c, 60, 3, 20, renumber)
    assert all(torch.equal(weights[:, i], between[0][:, i]) for i in (0, 1, 3, 4))
    if kind == "mla":
        assert torch.equal(joint[:, 1], between[1])
    c.close()


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq", [5, 16, 33])
def test_attend_paged_mla_steps(hq, out_type):
    """Lengths around one and two 16-slot tiles, which make up a 32-slot step, weights kept."""
    c = Cache("mla", bs=16, lens=[15, 16, 17, 31, 32, 33, 47, 48, 49, 1, 63, 64, 65, 0, 80], seed=hq)
    _attend(c, hq, out_type, scale=0.03)
    c.close()


def test_attend_paged_mla_ranges_of_several_steps():
    """Hundreds of requests of one to seven tiles: ranges hold several requests and steps, and end within a step."""
    lens = [int(x) for x in np.random.default_rng(9).integers(0, 112, size=240)] + [31, 32, 33, 47, 48, 49]
    c = Cache("mla", bs=16, lens=lens, seed=81)
    hq, n, scale = 20, len(lens), 0.03
    q = c.normal(n, hq, 576) * 2
    out, lse = torch.empty(n, hq, 512, device=DEV), torch.empty(n, hq, device=DEV)
    ws, w = _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, n, hq, max(lens), True)), c.w[0].clone()
    pic.pic_attend_paged(c.ctx, q, scale, c.k[0], None, c.d_tables, c.d_lens, max(lens), out, lse=lse, weights=w, workspace=ws)
    assert _status(c, ws) == 0
    _check_batch(c, q, c.k[0], c.k[0][..., :512], scale, out, lse, w)
    c.close()


def _check_batch(c, q, k, v, scale, out, lse, w):
    """_check_attend's bounds for a batch at once, in 64 bits on the device (the largest score error serves all)."""
    n, hq, T = len(c.lens), q.shape[1], max(c.lens)
    pages, heads = c.d_tables.long(), k.shape[2]
    rows = k[pages].flatten(1, 2).double()                                    # [request, slot, head, dim]
    live = torch.arange(rows.shape[1], device=DEV)[None] < c.d_lens[:, None]
    qg = q.double().reshape(n, heads, hq // heads, -1)
    x = scale * torch.einsum("rhgd,rthd->rhgt", qg, rows)
    s_err = scale * torch.einsum("rhgd,rthd->rhgt", qg.abs(), rows.abs()).max().item() * (q.shape[2] + 8) * 2.0 ** -23
    del rows
    x.masked_fill_(~live[:, None, None], -math.inf)
    want_lse = torch.logsumexp(x, -1).reshape(n, hq)
    p = torch.softmax(x, -1).nan_to_num(0.0)
    vals = v[pages].flatten(1, 2).double() * live[..., None, None]
    want = torch.einsum("rhgt,rthd->rhgd", p, vals).reshape(n, hq, -1)
    size = torch.einsum("rhgt,rthd->rhgd", p, vals.abs()).reshape(n, hq, -1)
    rel = 2 * s_err + 2.0 ** -20 + T * 2.0 ** -23
    bf16 = out.dtype == torch.bfloat16
    lim = (rel + (2.0 ** -16 if bf16 else 0)) * size + (2.0 ** -8 * want.abs() * (1 + rel) if bf16 else 0)
    assert bool(((out.double() - want).abs() <= lim).all())
    some = c.d_lens > 0
    assert bool(((lse.double() - want_lse).abs() <= s_err + rel + 2.0 ** -22 * want_lse.abs())[some].all())
    assert bool(torch.isneginf(lse[~some]).all())
    if w is not None:
        share = p.reshape(n, w.shape[1], -1, p.shape[-1]).sum(2)              # [request, weight head, slot]
        share = share.reshape(n, w.shape[1], -1, c.bs).transpose(1, 2)        # [request, page, weight head, row]
        at = c.w[0].double()
        add = torch.zeros_like(at)
        add[pages.flatten()] = share.flatten(0, 1)
        assert bool(((w.double() - at - add).abs() <= rel * add + 2.0 ** -22 * torch.where(add > 0, at + add, 0)).all())


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,group,d,weights", [(2, 16, 128, True), (1, 9, 64, True), (1, 24, 128, True), (2, 12, 256, False),
                                                   (1, 40, 256, True), (3, 17, 64, False)])
def test_attend_paged_wide_groups_over_long_sequences(heads, group, d, weights, out_type):
    """9 and more query heads per KV head over ranges of many tiles: the ring goes round, scores leave many times,
    and requests end within a range."""
    c = Cache(heads=heads, d=d, bs=16, lens=[9001, 40, 0, 20000, 333, 4097], seed=group, weight_heads=1 if group == 24 else heads)
    n, hq, T, scale = len(c.lens), heads * group, max(c.lens), d ** -0.5
    q = c.normal(n, hq, d) * 2
    out, lse = torch.empty(n, hq, d, dtype=out_type, device=DEV), torch.empty(n, hq, device=DEV)
    ws, w = _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, n, hq, T, weights)), c.w[0].clone() if weights else None
    pic.pic_attend_paged(c.ctx, q, scale, c.k[0], c.v[0], c.d_tables, c.d_lens, T, out, lse=lse, weights=w, workspace=ws)
    assert _status(c, ws) == 0
    _check_batch(c, q, c.k[0], c.v[0], scale, out, lse, w)
    c.close()


def test_attend_paged_infinite_values_stay_in_their_dimension():
    """An infinite value leaves its dimension of the heads that read it without a number, and changes nothing else."""
    c = Cache(heads=2, d=128, bs=16, lens=[100, 50], seed=82)
    q = c.normal(2, 8, 128)
    clean, lse = _attend(c, 8, torch.float32, weights=False, q=q)
    c.v[0, int(c.tables[0][2]), 5, 1, 77] = float("inf")
    out, got, ws = torch.empty_like(clean), torch.empty_like(lse), _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, 2, 8, 100))
    pic.pic_attend_paged(c.ctx, q, 128 ** -0.5, c.k[0], c.v[0], c.d_tables, c.d_lens, 100, out, lse=got, workspace=ws)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 4:, 77] = True
    assert not bool(torch.isfinite(out[hit]).any()) and torch.equal(out[~hit], clean[~hit]) and torch.equal(got, lse)
    c.close()


def test_attend_captured_many_requests_and_other_lengths():
    """A graph of an attention over more requests than the joins walk, replayed for other lengths, none among them."""
    n, longest = 300, 90
    c = Cache(heads=2, d=64, bs=16, lens=[longest] * n, seed=90)
    q = c.normal(n, 8, 64) * 2
    out, lse = torch.empty(n, 8, 64, device=DEV), torch.empty(n, 8, device=DEV)
    ws, w, lens = _ws(pic.pic_attend_paged_workspace_bytes(c.ctx, n, 8, longest, True)), c.w[0].clone(), c.d_lens.clone()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            pic.pic_attend_paged(c.ctx, q, 0.125, c.k[0], c.v[0], c.d_tables, lens, longest, out, lse=lse, weights=w, workspace=ws)
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    for new in (np.full(n, longest), rng.integers(0, longest + 1, n), np.zeros(n, int), np.arange(n) % 2, (np.arange(n) == 299) * 17):
        c.lens, c.d_lens = [int(x) for x in new], _i32(new)
        lens.copy_(c.d_lens)
        w.copy_(c.w[0])
        graph.replay()
        torch.cuda.synchronize()
        if max(c.lens) == 0:
            assert bool((out == 0).all()) and bool(torch.isneginf(lse).all()) and torch.equal(w, c.w[0])
        else:
            _check_batch(c, q, c.k[0], c.v[0], 0.125, out, lse, w)
    assert _status(c, ws) == 0
    c.close()


@pytest.mark.parametrize("kind", ["gqa", "mla"])
def test_two_loops_at_once(kind):
    """Two streams write, attend and evict at the same time, each on caches and a workspace of its own: what they
    leave is what each leaves alone, whichever way the stream is named."""
    hq, budget = 8, 200

    def prepare(c, stream, how):
        g = torch.Generator(device=DEV).manual_seed(5)
        n, dv = len(c.lens), 512 if kind == "mla" else c.d
        lens, ws = c.d_lens.clone(), _ws(1 << 26)
        out, kept = torch.empty(n, hq, dv, device=DEV), torch.empty(1, n, c.wh, budget, dtype=torch.int32, device=DEV)
        rows = torch.randn((6, n, hq + 2 * c.heads, c.d), generator=g, device=DEV).to(torch.bfloat16)
        q_out, req, v_cache = torch.empty(n, hq, c.d, dtype=torch.bfloat16, device=DEV), _i32(range(n)), None if c.v is None else c.v[0]
        longest, slot = c.tables.shape[1] * c.bs, torch.empty_like(lens)
        s = dict(stream=None if how == "current" else stream if how == "object" else stream.cuda_stream)

        def step(x):
            with torch.cuda.stream(stream):
                slot.copy_(lens)
                lens.add_(1)
                v = x[:, hq + c.heads:] if kind == "gqa" else None
                pic.pic_write_tokens(c.ctx, slot, x[:, hq:hq + c.heads], v, req, slot, c.d_tables, c.k[0], v_cache, q=x[:, :hq],
                                     q_out=q_out, weights=c.w[0], workspace=ws, **s)
                pic.pic_attend_paged(c.ctx, q_out, 0.05, c.k[0], v_cache, c.d_tables, lens, longest, out, weights=c.w[0],
                                     workspace=ws, **s)
                pic.pic_evict_tokens(c.ctx, c.k, c.v, c.w, c.d_tables, lens, budget, kept, lens, n_first=4, n_recent=20,
                                     renumber=True, workspace=ws, **s)
        return [lambda x=x: step(x) for x in rows], (out, kept, lens, c.k, c.v, c.w, ws)

    def caches():
        return [Cache(kind, heads=2, d=128, lens=[900, 300, 2000 + i, 190], room=16, seed=91 + i) for i in range(2)]

    streams = torch.cuda.Stream(), torch.cuda.Stream()
    alone, together = caches(), caches()
    want, got = [], []
    for c, stream in zip(alone, streams):
        steps, left = prepare(c, stream, "current")
        torch.cuda.synchronize()
        for step in steps:
            step()
        torch.cuda.synchronize()
        want.append(left)
    both = [prepare(c, stream, how) for c, stream, how in zip(together, streams, ("object", "handle"))]
    got = [left for _, left in both]
    torch.cuda.synchronize()
    for one, other in zip(both[0][0], both[1][0]):
        one()
        other()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, together):
        assert _status(c, b[-1]) == 0
        assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(a[:-1], b[:-1]))
    for c in alone + together:
        c.close()
