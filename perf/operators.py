"""The decode-loop operators over a paged cache, as measured: writing new tokens
at positions of one or several axes, attending one new token per request, and
evicting tokens by accumulated attention weight.

`run` computes them in their plain form (torch operations, 32 bits) where `own`
is false, and through the library's calls where it is true.  `exact` restates
each definition in 64 bits.  Sizes follow this repository's workloads (8 KV
heads of 128 dims under 32 query heads, blocks of 16 tokens, 576-wide latent
rows, contexts of 16k to 128k) and generic variations of them.
"""

import math
import random

import torch

own = False

THETA = 5.0e5
LATENT, ROPE = 512, 64


# ------------------------------------------------------------------ the cases

def listed():
    gqa = dict(kind="gqa", kv_heads=8, q_heads=32, head_dim=128, pairing="neox", block=16)
    mla = dict(kind="mla", kv_heads=1, q_heads=16, head_dim=576, pairing="interleaved", block=16)
    return [
        # one user, one new token after a stitched prompt: the smallest call, all latency
        dict(gqa, name="write_one", op="write", reqs=1, per_req=1, axes=1, context=4096, fused=False, weights=False, pad=0),
        # a decode batch of 64 requests (three of its rows are padding) out of a fused q/k/v projection,
        # three position axes, the eviction weights of the new slots cleared
        dict(gqa, name="write_batch", op="write", reqs=64, per_req=1, axes=3, context=1024, fused=True, weights=True, pad=3),
        # the prefill of one video: 16k tokens with time, height and width positions
        dict(gqa, name="write_video", op="write", reqs=1, per_req=16384, axes=3, context=300, fused=True, weights=False, pad=0),
        # recomputed chunk heads of a latent-cache model: 512 tokens in each of 4 requests, 16 query heads
        dict(mla, name="write_latent", op="write", reqs=4, per_req=512, axes=1, context=2048, fused=False, weights=True, pad=0),
        # one user, a short chat: latency again
        dict(gqa, name="attend_short", op="attend", reqs=1, low=777, high=777, weights=False, out="f32", lens_seed=1),
        # a ragged decode batch with weights kept for eviction, one idle slot of length 0
        dict(gqa, name="attend_batch", op="attend", reqs=64, low=1, high=8192, weights=True, out="bf16", lens_seed=2),
        # one user at the end of a 128k window, weights kept: the cache's length has to be split
        dict(gqa, name="attend_long", op="attend", reqs=1, low=131071, high=131071, weights=True, out="bf16", lens_seed=3),
        # 64 requests of 16k tokens: the largest read of a cache
        dict(gqa, name="attend_stress", op="attend", reqs=64, low=16384, high=16384, weights=False, out="f32", lens_seed=4),
        # one layer of one request a little over its budget, as after every few steps
        dict(gqa, name="evict_step", op="evict", layers=1, reqs=1, low=2064, high=2064, budget=2048, first=4, recent=256,
             shared=False, renumber=False, lens_seed=5),
        # a 32k prompt cut to 4k once, in half of a model's layers, keys re-rotated to their new places
        dict(gqa, name="evict_prompt", op="evict", layers=16, reqs=1, low=32768, high=32768, budget=4096, first=4, recent=512,
             shared=False, renumber=True, lens_seed=6),
        # a ragged batch of which some are below the budget; all heads of a token kept or dropped together
        dict(gqa, name="evict_batch", op="evict", layers=8, reqs=16, low=1500, high=6000, budget=2048, first=4, recent=256,
             shared=True, renumber=False, lens_seed=7),
        # latent rows: only the rope slice is rotated
        dict(mla, name="evict_latent", op="evict", layers=16, reqs=4, low=12001, high=16384, budget=8190, first=32, recent=512,
             shared=True, renumber=True, lens_seed=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "evict"])
    mla = op != "attend" and rng.random() < 0.3
    block = rng.choice([16, 16, 32, 64, _log_int(rng, 1, 256)])
    if mla:
        c = dict(kind="mla", kv_heads=1, q_heads=rng.choice([16, 32, 128]), head_dim=576)
    else:
        kv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        c = dict(kind="gqa", kv_heads=kv, q_heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), head_dim=rng.choice([64, 128, 128, 256]))
    c.update(op=op, pairing=rng.choice(["neox", "interleaved"]), block=block)
    row = c["kv_heads"] * c["head_dim"]            # elements of a token in K
    if op == "write":
        reqs = _log_int(rng, 1, 64)
        wide = row * 2 + c["q_heads"] * c["head_dim"]
        per = _log_int(rng, 1, max(1, min(8192, 40_000_000 // (wide * reqs))))
        c.update(reqs=reqs, per_req=per, axes=rng.choice([1, 2, 3, 4]), context=_log_int(rng, 1, max(2, 60_000_000 // (row * reqs) - per)),
                 fused=rng.random() < 0.5, weights=rng.random() < 0.5, pad=rng.choice([0, 0, 1, 5]))
    elif op == "attend":
        reqs = _log_int(rng, 1, 64)
        high = _log_int(rng, 1, max(1, min(131072, 250_000_000 // (row * reqs))))
        low = rng.choice([high, max(1, high // 2), 1])
        c.update(reqs=reqs, low=low, high=high, weights=rng.random() < 0.5, out=rng.choice(["f32", "bf16"]), lens_seed=rng.randrange(1 << 30))
    else:
        layers, reqs = _log_int(rng, 1, 16), _log_int(rng, 1, 16)
        high = _log_int(rng, 2, max(2, min(65536, 200_000_000 // (row * layers * reqs))))
        budget = rng.randint(1, high)
        first = rng.randint(0, min(32, budget // 2))
        c.update(layers=layers, reqs=reqs, low=max(1, high // rng.choice([1, 2, 8])), high=high, budget=budget, first=first,
                 recent=rng.randint(0, budget - first), shared=mla or rng.random() < 0.4, renumber=rng.random() < 0.5,
                 lens_seed=rng.randrange(1 << 30))
    return c


def _lens(case):
    """Cached tokens of each request (the last of a ragged batch is an idle slot)."""
    rng = random.Random(case["lens_seed"])
    lens = [rng.randint(case["low"], case["high"]) for _ in range(case["reqs"])]
    lens[0] = case["high"]
    if case["reqs"] > 2 and case["low"] < case["high"]:
        lens[-1] = 0
    return lens


def _written(case):
    """Tokens of a write that land in the cache."""
    return case["reqs"] * case["per_req"] - min(case["pad"], case["reqs"] * case["per_req"] - 1)


def work(case):
    row = case["kv_heads"] * case["head_dim"] * 2                      # bytes of a token in one cache tensor
    tensors = 2 if case["kind"] == "gqa" else 1
    rope = case["head_dim"] if case["kind"] == "gqa" else ROPE
    if case["op"] == "write":
        n, w = case["reqs"] * case["per_req"], _written(case)
        q = case["q_heads"] * case["head_dim"] * 2
        return {"bytes": 2 * n * q + w * row * tensors * 2 + 4 * n * (case["axes"] + 2) + (4 * w * _weight_heads(case) if case["weights"] else 0),
                "flops": 3 * rope * (n * case["q_heads"] + w * case["kv_heads"])}
    lens = _lens(case)
    if case["op"] == "attend":
        out = case["q_heads"] * case["head_dim"] * len(lens)
        return {"bytes": sum(lens) * (2 * row + (8 * case["kv_heads"] if case["weights"] else 0)) + out * (2 + (4 if case["out"] == "f32" else 2)),
                "flops": 4 * sum(lens) * case["q_heads"] * case["head_dim"]}
    hw = _weight_heads(case)
    over = [n for n in lens if n > case["budget"]]
    moved = sum(case["budget"] - case["first"] for _ in over) * case["layers"]
    read = sum(over) * case["layers"] * hw * 4
    listing = 4 * case["layers"] * len(lens) * hw * case["budget"]
    return {"bytes": read + listing + moved * (row * tensors * 2 + hw * 8),
            "flops": 3 * moved * case["kv_heads"] * rope if case["renumber"] else moved}


def _weight_heads(case):
    return 1 if case.get("shared") else case["kv_heads"]


# ----------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, scale, generator=g)


def _tables(g, reqs, per, spare):
    """Block tables [reqs][per] over shuffled blocks, and the number of blocks."""
    n = reqs * per + spare
    order = torch.randperm(n, device="cuda", generator=g).to(torch.int32)
    return order[:reqs * per].reshape(reqs, per).contiguous(), n


def _axis_of_freq(case):
    """The position axis of each frequency: the first quarter (at least one) on axis 0, the rest dealt out."""
    half = (case["head_dim"] if case["kind"] == "gqa" else ROPE) // 2
    axes = case["axes"]
    if axes == 1:
        return [0] * half
    head = half // 4
    return [0 if f < head else 1 + (f - head) * (axes - 1) // (half - head) for f in range(half)]


def _inputs(case, seed):
    g = _generator(seed)
    bs, hk, hq, d = case["block"], case["kv_heads"], case["q_heads"], case["head_dim"]
    gqa = case["kind"] == "gqa"
    s = {}
    if case["op"] == "write":
        reqs, per = case["reqs"], case["per_req"]
        n = reqs * per
        s["tables"], blocks = _tables(g, reqs, -(-(case["context"] + per) // bs), 2)
        s["k_cache"] = _normal(g, blocks, bs, hk, d)
        s["v_cache"] = _normal(g, blocks, bs, hk, d) if gqa else None
        if case["fused"] and gqa:   # slices of one projection's output: rows apart, heads dense
            qkv = _normal(g, n, hq + 2 * hk, d)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            s["q"], s["k"], s["v"] = _normal(g, n, hq, d), _normal(g, n, hk, d), _normal(g, n, hk, d) if gqa else None
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        i = torch.arange(n, device="cuda", dtype=torch.int32)
        s["req"], s["slot"] = i // per, case["context"] + i % per
        side = max(1, int(per ** (1 / 3)))      # a video's grid: frames of side x side patches
        t = i % per
        grid = [t // (side * side), t // side % side, t % side, t % 7]
        s["pos"] = torch.stack([case["context"] + (t if case["axes"] == 1 else grid[a]) for a in range(case["axes"])]).to(torch.int32)
        if n > _written(case):                  # rows that fill up a padded batch
            s["slot"][_written(case):] = -1
        s["axis_of_freq"] = _axis_of_freq(case)
        s["weights"] = torch.rand(blocks, _weight_heads(case), bs, device="cuda", generator=g) if case["weights"] else None
        return s
    lens = _lens(case)
    reqs = len(lens)
    s["tables"], blocks = _tables(g, reqs, max(1, -(-max(lens) // bs)), 3)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        s["k_cache"], s["v_cache"] = _normal(g, blocks, bs, hk, d), _normal(g, blocks, bs, hk, d)
        s["q"] = _normal(g, reqs, hq, d, scale=2.0)
        for r in (0, reqs - 1):                 # what pages hold behind a sequence's end is anything
            cut = lens[r] % bs
            if cut or lens[r] == 0:
                page = int(s["tables"][r, lens[r] // bs])
                s["k_cache"][page, cut:] = math.nan
                s["v_cache"][page, cut:] = math.inf
        s["weights"] = torch.rand(blocks, _weight_heads(case), bs, device="cuda", generator=g) if case["weights"] else None
        s["out"] = torch.empty(reqs, hq, d, device="cuda", dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
        s["lse"] = torch.empty(reqs, hq, device="cuda")
        return s
    layers, hw = case["layers"], _weight_heads(case)
    s["k_cache"] = _normal(g, layers, blocks, bs, hk, d)
    s["v_cache"] = _normal(g, layers, blocks, bs, hk, d) if gqa else None
    # sums of attention weights: a few heavy tokens, a long tail, and some never attended (equal, at 0)
    w = torch.rand(layers, blocks, hw, bs, device="cuda", generator=g)
    s["weights"] = torch.where(w < 0.1, torch.zeros_like(w), w ** 8 * 30)
    s["kept"] = torch.empty(layers, reqs, hw, case["budget"], dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.empty(reqs, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.load()
        gqa = case["kind"] == "gqa"
        d = case["head_dim"]
        s["ctx"] = pic.pic_create(pic.PIC_KIND_GQA if gqa else pic.PIC_KIND_MLA, case.get("layers", 1), case["kv_heads"], d,
                                  d if gqa else ROPE, 0 if gqa else LATENT,
                                  pic.PIC_PAIRING_NEOX_HALF if case["pairing"] == "neox" else pic.PIC_PAIRING_INTERLEAVED,
                                  case["block"], THETA, s["k_cache"].shape[-4])
        if case["op"] == "write":
            size = pic.PIC_STATUS_BYTES
        elif case["op"] == "attend":
            size = pic.pic_attend_paged_workspace_bytes(s["ctx"], case["reqs"], case["q_heads"], max(1, max(_lens(case))), case["weights"])
        else:
            size = pic.pic_evict_workspace_bytes(s["ctx"], case["layers"], case["reqs"], _weight_heads(case))
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        s["max_len"] = max(1, max(_lens(case))) if case["op"] == "attend" else 0
    return s


# ------------------------------------------------------------- the operators

def run(s):
    return {"write": _run_write, "attend": _run_attend, "evict": _run_evict}[s["case"]["op"]](s)


def _rope_theta(case):
    n = case["head_dim"] if case["kind"] == "gqa" else ROPE
    return torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"),
                     -torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / n)


def _rotate(case, x, angle):
    """x: [..., head_dim] in 32 bits; angle: 64-bit, one per frequency, broadcast over the heads."""
    c, s = angle.cos().float(), angle.sin().float()
    rope = x if case["kind"] == "gqa" else x[..., LATENT:]
    if case["pairing"] == "neox":
        half = rope.shape[-1] // 2
        a, b = rope[..., :half], rope[..., half:]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = rope[..., 0::2], rope[..., 1::2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return turned if case["kind"] == "gqa" else torch.cat([x[..., :LATENT], turned], -1)


def _run_write(s):
    case = s["case"]
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_write_tokens(s["ctx"], s["pos"], s["k"], s["v"], s["req"], s["slot"], s["tables"], s["k_cache"], s["v_cache"],
                             q=s["q"], q_out=s["q_out"], freq_axis=s["axis_of_freq"], weights=s["weights"], workspace=s["ws"])
    else:
        axis = torch.tensor(s["axis_of_freq"], device="cuda")
        angle = (s["pos"].double()[axis].T * _rope_theta(case))[:, None]          # [token, 1, frequency]
        s["q_out"].copy_(_rotate(case, s["q"].float(), angle))
        k = _rotate(case, s["k"].float(), angle).to(torch.bfloat16)
        live = s["slot"] >= 0
        slot, req = s["slot"][live].long(), s["req"][live].long()
        page, row = s["tables"][req, slot // case["block"]].long(), slot % case["block"]
        s["k_cache"][page, row] = k[live]
        if s["v"] is not None:
            s["v_cache"][page, row] = s["v"][live]
        if s["weights"] is not None:
            s["weights"][page, :, row] = 0.0
    return [s["q_out"], s["k_cache"], s["v_cache"], s["weights"]]


def _run_attend(s):
    case = s["case"]
    scale = case["head_dim"] ** -0.5
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_attend_paged(s["ctx"], s["q"], scale, s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["max_len"], s["out"],
                             lse=s["lse"], weights=s["weights"], workspace=s["ws"])
        return [s["out"], s["lse"], s["weights"]]
    bs, hk, d = case["block"], case["kv_heads"], case["head_dim"]
    reqs, longest = s["tables"].shape[0], s["tables"].shape[1] * bs
    live = torch.arange(longest, device="cuda")[None] < s["lens"][:, None]        # [request, slot]
    pages = s["tables"].long()
    k = s["k_cache"][pages].reshape(reqs, longest, hk, d).permute(0, 2, 3, 1).float()
    q = s["q"].float().reshape(reqs, hk, -1, d)
    x = (torch.matmul(q, k) * scale).masked_fill(~live[:, None, None], -math.inf)
    del k
    top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)      # an idle slot has nothing to attend
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    v = s["v_cache"][pages].reshape(reqs, longest, hk, d).float().masked_fill(~live[:, :, None, None], 0.0)
    s["out"].copy_(torch.matmul(p, v.transpose(1, 2)).reshape(s["out"].shape))
    s["lse"].copy_((top + total.log()).reshape(s["lse"].shape))
    if s["weights"] is not None:
        share = p.sum(2).reshape(reqs, hk, -1, bs).transpose(1, 2)                 # [request, page, head, row]
        s["weights"].index_add_(0, pages.flatten(), share.reshape(-1, hk, bs))
    return [s["out"], s["lse"], s["weights"]]


def _run_evict(s):
    case = s["case"]
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_evict_tokens(s["ctx"], s["k_cache"], s["v_cache"], s["weights"], s["tables"], s["lens"], case["budget"], s["kept"],
                             s["new_lens"], n_first=case["first"], n_recent=case["recent"], renumber=case["renumber"],
                             workspace=s["ws"])
        return [s["k_cache"], s["v_cache"], s["weights"], s["kept"], s["new_lens"]]
    bs, budget = case["block"], case["budget"]
    layers, hw, hk = case["layers"], _weight_heads(case), case["kv_heads"]
    reqs, longest = s["tables"].shape[0], s["tables"].shape[1] * bs
    w = s["weights"][:, s["tables"].long()].permute(0, 1, 3, 2, 4).reshape(layers, reqs, hw, longest)
    slot = torch.arange(longest, device="cuda")
    n = s["lens"].long()[:, None, None]
    # protected slots before everything, then by weight, then what lies behind the end
    rank = torch.where((slot < case["first"]) | (slot >= n - case["recent"]), math.inf, w)
    rank = torch.where(slot < n, rank, -math.inf)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    best = torch.where(best < n, best, longest).sort(-1).values                    # ascending, nothing behind the end
    if best.shape[-1] < budget:
        best = torch.cat([best, best.new_full((layers, reqs, hw, budget - best.shape[-1]), longest)], -1)
    kept = torch.where(best < longest, best, -1)
    s["kept"].copy_(kept)
    s["new_lens"].copy_(s["lens"].clamp(max=budget))
    l, r, h, j = (kept >= 0).nonzero(as_tuple=True)
    src = kept[l, r, h, j]
    tables = s["tables"].long()
    from_page, from_row, to_page, to_row = tables[r, src // bs], src % bs, tables[r, j // bs], j % bs
    s["weights"][l, to_page, h, to_row] = s["weights"][l, from_page, h, from_row]
    if s["v_cache"] is not None:
        if hw == hk:
            s["v_cache"][l, to_page, to_row, h] = s["v_cache"][l, from_page, from_row, h]
        else:
            s["v_cache"][l, to_page, to_row] = s["v_cache"][l, from_page, from_row]
    k = s["k_cache"][l, from_page, from_row, h] if hw == hk else s["k_cache"][l, from_page, from_row]
    if case["renumber"]:
        angle = (j - src).double()[:, None] * _rope_theta(case)
        k = _rotate(case, k.float(), angle if hw == hk else angle[:, None]).to(torch.bfloat16)
    if hw == hk:
        s["k_cache"][l, to_page, to_row, h] = k
    else:
        s["k_cache"][l, to_page, to_row] = k
    return [s["k_cache"], s["v_cache"], s["weights"], s["kept"], s["new_lens"]]


# ---------------------------------------------- the definitions, in 64 bits

def _turn(case, rows, pos, axis=None):
    """Rows [n][heads][head_dim] in 64 bits, each frequency's pair as a complex number times exp(i pos theta)."""
    n = case["head_dim"] if case["kind"] == "gqa" else ROPE
    theta = torch.tensor([THETA ** (-2.0 * i / n) for i in range(n // 2)], dtype=torch.float64, device="cuda")
    pos = pos.double()
    angle = pos[:, None] * theta if axis is None else torch.stack([pos[a] * t for a, t in zip(axis, theta)], -1)
    off = 0 if case["kind"] == "gqa" else LATENT
    if case["pairing"] == "neox":
        first, second = slice(off, off + n // 2), slice(off + n // 2, off + n)
    else:
        first, second = slice(off, off + n, 2), slice(off + 1, off + n, 2)
    z = torch.complex(rows[..., first], rows[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    rows = rows.clone()
    rows[..., first], rows[..., second] = z.real, z.imag
    return rows


def exact(case, seed):
    s = _inputs(case, seed)
    bs = case["block"]
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "write":
        q = _turn(case, s["q"].double(), s["pos"], s["axis_of_freq"])
        k = _turn(case, s["k"].double(), s["pos"], s["axis_of_freq"])
        kc, vc, w = wide(s["k_cache"]), wide(s["v_cache"]), wide(s["weights"])
        for r in range(case["reqs"]):
            i = ((s["req"] == r) & (s["slot"] >= 0)).nonzero().flatten()
            at = s["slot"][i].long()
            rows = s["tables"][r].long()[at // bs] * bs + at % bs
            kc.view(-1, *kc.shape[2:])[rows] = k[i]
            if vc is not None:
                vc.view(-1, *vc.shape[2:])[rows] = s["v"].double()[i]
            if w is not None:
                w.transpose(1, 2)[rows // bs, rows % bs] = 0.0
        return [q, kc, vc, w]
    lens = _lens(case)
    if case["op"] == "attend":
        d, group = case["head_dim"], case["q_heads"] // case["kv_heads"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        w = wide(s["weights"])
        for r, n in enumerate(lens):
            if n == 0:
                continue
            i = torch.arange(n, device="cuda")
            page, row = s["tables"][r].long()[i // bs], i % bs
            for h in range(case["kv_heads"]):
                k, v = s["k_cache"][page, row, h].double(), s["v_cache"][page, row, h].double()
                heads = slice(h * group, (h + 1) * group)
                x = s["q"][r, heads].double() @ k.T / math.sqrt(d)
                lse[r, heads] = torch.logsumexp(x, -1)
                p = torch.softmax(x, -1)
                out[r, heads] = p @ v
                if w is not None:
                    w[page, h, row] += p.sum(0)
        return [out, lse, w]
    kc, vc, w = wide(s["k_cache"]), wide(s["v_cache"]), wide(s["weights"])
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int32, device="cuda")
    hw, budget = _weight_heads(case), case["budget"]
    heads_of = lambda h: slice(h, h + 1) if hw == case["kv_heads"] else slice(None)  # noqa: E731
    tables = s["tables"].cpu()
    for l in range(case["layers"]):
        for r, n in enumerate(lens):
            i = torch.arange(n)
            rows = (tables[r].long()[i // bs] * bs + i % bs).cuda()
            for h in range(hw):
                mine = s["weights"][l, rows // bs, h, rows % bs]
                if n <= budget:
                    take = torch.arange(n, device="cuda")
                else:
                    a, b = case["first"], n - case["recent"]
                    order = torch.sort(-mine[a:b], stable=True).indices[:budget - case["first"] - case["recent"]] + a
                    ends = torch.cat([torch.arange(a), torch.arange(b, n)]).cuda()
                    take = torch.cat([ends, order]).sort().values
                kept[l, r, h, :len(take)] = take.int()
                to, hs = rows[:len(take)], heads_of(h)
                flat = kc[l].view(-1, *kc.shape[3:])
                moved = flat[rows[take], hs]
                flat[to, hs] = _turn(case, moved, torch.arange(len(take), device="cuda") - take) if case["renumber"] else moved
                if vc is not None:
                    flat = vc[l].view(-1, *vc.shape[3:])
                    flat[to, hs] = flat[rows[take], hs]
                w[l, to // bs, h, to % bs] = mine[take].double()
    return [kc, vc, w, kept, torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device="cuda")]
