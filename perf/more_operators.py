"""A serving step's operators over a paged cache, as measured: block tables and
slot lists built from request lengths, new tokens written with the norms of
their heads applied, attention of any number of new tokens per request (all
slots before them, or a sliding window with a few first tokens that stay
visible), and decode attention of a batch whose requests share a long prefix.

`run` computes them in their plain form (torch operations, 32 bits) where `own`
is false, and through the library's calls where it is true.  `exact` restates
each definition in 64 bits.  Sizes follow this repository's workloads (8 KV
heads of 128 dims under 32 query heads, blocks of 16 tokens, 576-wide latent
rows, contexts of 16k to 32k) and generic variations of them.
"""

import math
import random

import torch

own = False

THETA = 5.0e5
EPS = 1.0e-6
LATENT, ROPE = 512, 64

# what a drawn case costs at most: scores of the plain form, their products, and the cache rows it gathers
MOST_SCORES, MOST_ROWS = 8192 * 8192 * 32, 64 * 16384 * 1024


# ------------------------------------------------------------------ the cases

def listed():
    gqa = dict(kind="gqa", kv_heads=8, q_heads=32, head_dim=128, pairing="neox", block=16)
    mla = dict(kind="mla", kv_heads=1, q_heads=16, head_dim=576, pairing="interleaved", block=16)
    return [
        # a decode step of 64 requests: a token each, a few requests end and give their blocks back
        dict(name="map_step", op="map", block=16, reqs=64, low=1, high=8192, grow_low=1, grow_high=1, ends=4, pad=0, short=False,
             lens_seed=1),
        # prompts and decode tokens of 256 requests scheduled together, the token rows padded; the pool of free
        # blocks runs out for the last of them
        dict(name="map_prompts", op="map", block=16, reqs=256, low=0, high=4096, grow_low=1, grow_high=1000, ends=16, pad=77,
             short=True, lens_seed=2),
        # one user, one new token: the smallest write, all latency
        dict(gqa, name="norm_one", op="norm", reqs=1, per_req=1, context=4096, fused=True, pad=0),
        # a 16k prompt out of a fused q/k/v projection, heads normalised
        dict(gqa, name="norm_prompt", op="norm", reqs=1, per_req=16384, context=300, fused=True, pad=0),
        # latent rows of 4 requests, the latent normalised on its way into the cache
        dict(mla, name="norm_latent", op="norm", reqs=4, per_req=512, context=2048, fused=False, pad=2),
        # one user, one new token in a short chat, a window of 512: latency again
        dict(gqa, name="attend_one", op="attend", reqs=1, per_req=1, low=777, high=777, window=512, first=4, scattered=False, pad=0,
             lens_seed=4),
        # a ragged decode batch with a window of 4k, one idle row; the pages out of the windows have been given back
        dict(gqa, name="attend_step", op="attend", reqs=64, per_req=1, low=1, high=16384, window=4096, first=4, scattered=False,
             pad=0, lens_seed=5),
        # an 8k prompt in a layer with a window of 4k
        dict(gqa, name="attend_prompt", op="attend", reqs=1, per_req=8192, low=8192, high=8192, window=4096, first=4, scattered=False,
             pad=0, lens_seed=6),
        # after a stitch: recomputed chunk heads and the question of 4 requests, every slot before them visible
        dict(gqa, name="attend_heads", op="attend", reqs=4, per_req=500, low=14000, high=16384, window=0, first=0, scattered=True,
             pad=5, lens_seed=7),
        # 4 samples of one prompt, shortly after it
        dict(gqa, name="shared_samples", op="shared", reqs=4, prefix=1031, low=1, high=64, lens_seed=8),
        # 64 requests over one 32k document
        dict(gqa, name="shared_document", op="shared", reqs=64, prefix=32768, low=1, high=2048, lens_seed=9),
        # many short chats under one system prompt, whose end is inside a block
        dict(gqa, name="shared_chats", op="shared", reqs=256, prefix=2003, low=100, high=1000, lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["map", "norm", "attend", "attend", "shared"])
    block = rng.choice([16, 16, 32, 64, _log_int(rng, 1, 256)])
    seed = rng.randrange(1 << 30)
    if op == "map":
        reqs = _log_int(rng, 1, 2048)
        high = _log_int(rng, 1, min(16384, 8_000_000 // reqs))
        grow = rng.choice([1, _log_int(rng, 1, max(1, min(4096, 250_000 // reqs)))])
        return dict(op=op, block=block, reqs=reqs, low=rng.choice([0, high // 2]), high=high, grow_low=rng.choice([1, grow]), grow_high=grow,
                    ends=rng.randint(0, reqs // 2), pad=rng.choice([0, 0, 1, 100]), short=rng.random() < 0.3, lens_seed=seed)
    if op == "norm" and rng.random() < 0.3:
        c = dict(kind="mla", kv_heads=1, q_heads=rng.choice([16, 32, 128]), head_dim=576)
    else:
        kv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        c = dict(kind="gqa", kv_heads=kv, q_heads=kv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16]), head_dim=rng.choice([64, 128, 128, 256]))
    c.update(op=op, pairing=rng.choice(["neox", "interleaved"]), block=block)
    row = c["kv_heads"] * c["head_dim"]            # elements of a token in K
    scores = MOST_SCORES // c["q_heads"] * 128 // max(128, c["head_dim"])
    if op == "norm":
        reqs = _log_int(rng, 1, 64)
        wide = row * 2 + c["q_heads"] * c["head_dim"]
        per = _log_int(rng, 1, max(1, min(8192, 40_000_000 // (wide * reqs))))
        c.update(reqs=reqs, per_req=per, context=_log_int(rng, 1, max(2, 60_000_000 // (row * reqs) - per)), fused=rng.random() < 0.5,
                 pad=rng.choice([0, 0, 1, 5]))
    elif op == "attend":
        reqs = _log_int(rng, 1, 64)
        high = _log_int(rng, 1, max(1, min(65536, MOST_ROWS // (row * reqs))))
        per = rng.choice([1, _log_int(rng, 1, max(1, min(high, 8192, scores // (reqs * high))))])
        window = rng.choice([0, _log_int(rng, 1, 8192)])
        c.update(reqs=reqs, per_req=per, low=rng.choice([high, (high + per) // 2, per]), high=high, window=window,
                 first=rng.choice([0, 4, _log_int(rng, 1, 256)]) if window else 0, scattered=rng.random() < 0.3,
                 pad=rng.choice([0, 0, 3]), lens_seed=seed)
    else:
        reqs = _log_int(rng, 2, 256)
        high = _log_int(rng, 1, max(1, min(8192, MOST_ROWS // 2 // (row * reqs))))
        prefix = _log_int(rng, 16, max(16, min(65536, MOST_SCORES // 4 // (reqs * c["q_heads"]), MOST_ROWS // 2 // row)))
        c.update(reqs=reqs, prefix=prefix, low=rng.choice([1, high]), high=high, lens_seed=seed)
    return c


def _tokens(case):
    """Of an attention: per request its sequence's length and its new tokens' slots, ascending (the last of a
    ragged batch is an idle row: one token with slot -1)."""
    rng = random.Random(case["lens_seed"])
    out = []
    for r in range(case["reqs"]):
        n = case["per_req"] if r == 0 or case["per_req"] == 1 else rng.randint(1, case["per_req"])
        length = case["high"] if r == 0 else rng.randint(max(n, case["low"]), max(n, case["high"]))
        slots = list(range(length - n, length))
        if case["scattered"] and n > 1:            # half of them the first 16 tokens of chunks, half the sequence's end
            heads = n // 2
            chunks = -(-heads // 16)
            stride = (length - n) // chunks
            if stride >= 16:
                slots = [j // 16 * stride + j % 16 for j in range(heads)] + slots[heads:]
        out.append((length, slots))
    if case["reqs"] > 2 and case["low"] < case["high"]:
        out[-1] = (0, [-1])
    return out


def _seen(case, slots):
    """Slots that some of a request's tokens see, as merged intervals; and how many each sees, summed."""
    runs, pairs, w = [], 0, case["window"]
    for s in slots:
        if s < 0:
            continue
        lo = max(0, s + 1 - w) if w else 0
        pairs += s + 1 - lo + min(case["first"], lo)
        for a, b in ((0, min(case["first"], lo)), (lo, s + 1)):
            if a < b:
                runs.append((a, b))
    merged = []
    for a, b in sorted(runs):
        if merged and a <= merged[-1][1]:
            merged[-1][1] = max(merged[-1][1], b)
        else:
            merged.append([a, b])
    return merged, pairs


def _shared_lens(case):
    rng = random.Random(case["lens_seed"])
    lens = [case["prefix"] + (case["high"] if r == 0 else rng.randint(case["low"], case["high"])) for r in range(case["reqs"])]
    if case["reqs"] > 4 and case["low"] < case["high"]:
        lens[-1] = 0                                # an idle row
    return lens


def _map_lens(case):
    """Lengths and growths (below 0: a request that ends) of a map."""
    rng = random.Random(case["lens_seed"])
    lens = [rng.randint(case["low"], case["high"]) for _ in range(case["reqs"])]
    grow = [rng.randint(case["grow_low"], case["grow_high"]) for _ in range(case["reqs"])]
    for r in rng.sample(range(case["reqs"]), case["ends"]):
        grow[r] = -lens[r]
    return lens, grow


def _map_sizes(case):
    """Blocks the map gives back and takes (were there enough), free blocks before it, and its token rows."""
    lens, grow = _map_lens(case)
    up = lambda n: -(-n // case["block"])  # noqa: E731
    back = sum(up(n) - up(n + g) for n, g in zip(lens, grow) if g < 0)
    need = sum(up(n + g) - up(n) for n, g in zip(lens, grow) if g > 0)
    spare = max(0, need * 2 // 3 - back) if case["short"] else need + 3
    return back, need, spare, sum(g for g in grow if g > 0) + case["pad"]


def work(case):
    if case["op"] == "map":
        back, need, spare, n = _map_sizes(case)
        return {"bytes": 4 * (case["reqs"] * 4 + 3 + 2 * back + 2 * min(need, back + spare) + 3 * n), "flops": 3 * n + 8 * case["reqs"]}
    row = case["kv_heads"] * case["head_dim"] * 2                      # bytes of a token in one cache tensor
    token = case["q_heads"] * case["head_dim"] * 2
    if case["op"] == "norm":
        tensors = 2 if case["kind"] == "gqa" else 1
        n = case["reqs"] * case["per_req"]
        w = n - min(case["pad"], n - 1)
        heads = n * case["q_heads"] + w * case["kv_heads"] if case["kind"] == "gqa" else w
        rope = case["head_dim"] if case["kind"] == "gqa" else ROPE
        return {"bytes": 2 * n * token + w * row * tensors * 2 + 12 * n,
                "flops": 4 * heads * (case["head_dim"] if case["kind"] == "gqa" else LATENT) +
                         3 * rope * (n * case["q_heads"] + w * case["kv_heads"])}
    if case["op"] == "attend":
        rows = pairs = tokens = 0
        for _, slots in _tokens(case):
            runs, p = _seen(case, slots)
            rows += sum(b - a for a, b in runs)
            pairs += p
            tokens += len(slots)
        return {"bytes": 2 * rows * row + tokens * (2 * token + 4 + 4 * case["q_heads"]), "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}
    lens = _shared_lens(case)
    rows = case["prefix"] + sum(max(0, n - case["prefix"]) for n in lens)
    return {"bytes": 2 * rows * row + len(lens) * (2 * token + 4 * case["q_heads"]), "flops": 4 * sum(lens) * case["q_heads"] * case["head_dim"]}


# ----------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, scale, generator=g)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _shuffled(g, n):
    return torch.randperm(n, device="cuda", generator=g).to(torch.int32)


def _map_inputs(case, g):
    lens, grow = _map_lens(case)
    back, need, spare, n = _map_sizes(case)
    have = [-(-x // case["block"]) for x in lens]
    per = max(1, max(-(-max(x, x + y) // case["block"]) for x, y in zip(lens, grow)))
    blocks = sum(have) + spare + 1
    order = _shuffled(g, blocks)
    s = {"lens": _i32(lens), "grow": _i32(grow), "blocks": blocks}
    tables = torch.full((len(lens), per), -1, dtype=torch.int32, device="cuda")
    tables[torch.arange(per, device="cuda")[None] < _i32(have)[:, None]] = order[:sum(have)]
    s["tables"] = tables
    s["free"] = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    s["free"][:spare] = order[sum(have):sum(have) + spare]
    s["n_free"] = _i32([spare])
    s["shift"] = torch.randint(0, 100, (len(lens),), generator=g, device="cuda").to(torch.int32)   # tokens evicted before
    s["new_lens"], s["new_n_free"] = torch.empty_like(s["lens"]), torch.empty_like(s["n_free"])
    s["indptr"] = torch.empty(len(lens) + 1, dtype=torch.int32, device="cuda")
    s["req"], s["slot"], s["pos"] = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3))
    return s


def _inputs(case, seed):
    g = _generator(seed)
    if case["op"] == "map":
        return _map_inputs(case, g)
    s = {}
    bs, hk, hq, d = case["block"], case["kv_heads"], case["q_heads"], case["head_dim"]
    if case["op"] == "norm":
        gqa = case["kind"] == "gqa"
        reqs, per = case["reqs"], case["per_req"]
        n = reqs * per
        pages = -(-(case["context"] + per) // bs)
        s["blocks"] = reqs * pages + 2
        s["tables"] = _shuffled(g, s["blocks"])[:reqs * pages].reshape(reqs, pages).contiguous()
        s["k_cache"] = _normal(g, s["blocks"], bs, hk, d)
        s["v_cache"] = _normal(g, s["blocks"], bs, hk, d) if gqa else None
        if case["fused"] and gqa:   # slices of one projection's output: rows apart, heads dense
            qkv = _normal(g, n, hq + 2 * hk, d, scale=2.0)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            s["q"], s["k"] = _normal(g, n, hq, d), _normal(g, n, hk, d, scale=3.0)
            s["v"] = _normal(g, n, hk, d) if gqa else None
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        # learned weights: around 1, a few channels far larger
        w = [1.0 + 0.3 * _normal(g, d if gqa else LATENT).float() for _ in range(2)]
        for x in w:
            x[::61] *= 6.0
        s["q_norm"], s["k_norm"] = w[0].to(torch.bfloat16) if gqa else None, w[1].to(torch.bfloat16)
        i = torch.arange(n, device="cuda", dtype=torch.int32)
        s["req"], s["slot"] = i // per, case["context"] + i % per
        s["pos"] = s["slot"].clone()
        if case["pad"] and n > 1:               # rows that fill up a padded batch
            s["slot"][n - min(case["pad"], n - 1):] = -1
        return s
    if case["op"] == "attend":
        tokens = _tokens(case)
        reqs, n = len(tokens), sum(len(x) for _, x in tokens)
        pages = max(1, -(-max(x for x, _ in tokens) // bs))
        s["blocks"] = reqs * pages + 3
        s["tables"] = _shuffled(g, s["blocks"])[:reqs * pages].reshape(reqs, pages).contiguous()
        s["indptr"] = _i32([0] + torch.tensor([len(x) for _, x in tokens]).cumsum(0).tolist())
        s["slot"] = _i32([x for _, xs in tokens for x in xs] + [-1] * case["pad"])
        s["k_cache"], s["v_cache"] = _normal(g, s["blocks"], bs, hk, d), _normal(g, s["blocks"], bs, hk, d)
        n += case["pad"]
        for r in {0, reqs - 1}:                 # what pages hold behind a sequence's end is anything
            length = tokens[r][0]
            if length % bs or length == 0:
                page = int(s["tables"][r, length // bs])
                s["k_cache"][page, length % bs:] = math.nan
                s["v_cache"][page, length % bs:] = math.inf
        if case["window"]:                      # pages that no token sees have been given back
            for r, (_, slots) in enumerate(tokens):
                runs, _ = _seen(case, slots)
                used = torch.zeros(pages, dtype=torch.bool)
                lo, hi = (max(0, min(x for x in slots)), max(slots) + 1) if runs else (0, 0)
                if runs:
                    used[max(0, lo + 1 - case["window"]) // bs:-(-hi // bs)] = True
                    used[:-(-min(case["first"], hi) // bs)] = True
                s["tables"][r, ~used.cuda()] = -1
        s["q"] = _normal(g, n, hq, d, scale=2.0)
        s["out"] = torch.zeros(n, hq, d, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros(n, hq, device="cuda")
        return s
    lens, prefix = _shared_lens(case), case["prefix"]
    reqs, whole = len(lens), prefix // bs       # blocks that hold nothing but the prefix
    pages = -(-max(lens) // bs)
    mine = pages - whole
    s["blocks"] = -(-prefix // bs) + reqs * mine + 3
    order = _shuffled(g, s["blocks"])
    s["prefix_table"] = order[:-(-prefix // bs)].contiguous()
    s["tables"] = torch.cat([s["prefix_table"][:whole].expand(reqs, whole),
                             order[len(s["prefix_table"]):len(s["prefix_table"]) + reqs * mine].reshape(reqs, mine)], 1).contiguous()
    s["prefix_len"], s["lens"] = _i32([prefix]), _i32(lens)
    s["k_cache"], s["v_cache"] = _normal(g, s["blocks"], bs, hk, d), _normal(g, s["blocks"], bs, hk, d)
    if prefix % bs:                             # what follows the prefix in its last block is anything
        s["k_cache"][int(s["prefix_table"][-1]), prefix % bs:] = math.nan
        s["v_cache"][int(s["prefix_table"][-1]), prefix % bs:] = math.inf
    s["q"] = _normal(g, reqs, hq, d, scale=2.0)
    s["out"] = torch.zeros(reqs, hq, d, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.zeros(reqs, hq, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.load()
        if case["op"] == "map":
            s["ctx"] = pic.pic_create(pic.PIC_KIND_GQA, 1, 1, 128, 128, 0, pic.PIC_PAIRING_NEOX_HALF, case["block"], THETA, s["blocks"])
            size = pic.pic_map_tokens_workspace_bytes(s["ctx"], case["reqs"])
        else:
            gqa = case["kind"] == "gqa"
            d = case["head_dim"]
            s["ctx"] = pic.pic_create(pic.PIC_KIND_GQA if gqa else pic.PIC_KIND_MLA, 1, case["kv_heads"], d, d if gqa else ROPE,
                                      0 if gqa else LATENT,
                                      pic.PIC_PAIRING_NEOX_HALF if case["pairing"] == "neox" else pic.PIC_PAIRING_INTERLEAVED,
                                      case["block"], THETA, s["blocks"])
            size = pic.PIC_STATUS_BYTES
            if case["op"] == "attend":
                size = pic.pic_attend_tokens_workspace_bytes(s["ctx"], len(s["slot"]), case["reqs"], case["q_heads"])
            elif case["op"] == "shared":
                size = pic.pic_attend_shared_workspace_bytes(s["ctx"], case["reqs"], case["q_heads"])
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    if case["op"] == "shared":
        s["max_len"] = max(_shared_lens(case))
    return s


# ------------------------------------------------------------- the operators

def run(s):
    return {"map": _run_map, "norm": _run_norm, "attend": _run_attend, "shared": _run_shared}[s["case"]["op"]](s)


def _run_map(s):
    outputs = [s[x] for x in ("new_lens", "tables", "free", "new_n_free", "indptr", "req", "slot", "pos")]
    bs = s["case"]["block"]
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_map_tokens(s["ctx"], s["lens"], s["grow"], s["tables"], s["free"], s["n_free"], s["new_lens"], s["new_n_free"],
                           s["indptr"], s["req"], s["slot"], positions=s["pos"], shift=s["shift"], workspace=s["ws"])
        return outputs
    lens, grow = s["lens"].long(), s["grow"].long()
    have, want = (lens + bs - 1) // bs, (lens + grow + bs - 1) // bs
    column = torch.arange(s["tables"].shape[1], device="cuda")
    # requests that shrink put their last blocks on the pile of free ones, in order
    back = s["tables"][(column >= want[:, None]) & (column < have[:, None])]
    pile = s["n_free"].long() + back.numel()
    s["free"][s["n_free"].long() + torch.arange(back.numel(), device="cuda")] = back
    # those that grow take theirs from its top, in order, while it lasts
    need = (want - have).clamp(min=0)
    granted = (need == 0) | (need.cumsum(0) <= pile)
    takes = (column >= have[:, None]) & (column < want[:, None]) & granted[:, None]
    rank = (takes.flatten().cumsum(0) - 1).reshape(takes.shape)
    s["tables"].copy_(torch.where(takes, s["free"][(pile - 1 - rank).clamp(0, len(s["free"]) - 1)], s["tables"]))
    s["new_n_free"].copy_(pile - takes.sum())
    s["new_lens"].copy_(torch.where(granted, lens + grow, lens))
    s["indptr"][0] = 0
    s["indptr"][1:] = grow.clamp(min=0).cumsum(0)
    row = torch.arange(len(s["slot"]), device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["indptr"][1:].contiguous(), row, right=True)
    live = req < len(lens)                      # rows behind the last request's are padding
    req = torch.where(live, req, 0)
    slot = torch.where(live & granted[req], lens[req] + row - s["indptr"][req], -1)
    s["req"].copy_(req)
    s["slot"].copy_(slot)
    s["pos"].copy_(torch.where(slot >= 0, slot + s["shift"][req], 0))
    return outputs


def _rope_theta(case):
    n = case["head_dim"] if case["kind"] == "gqa" else ROPE
    return torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"),
                     -torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / n)


def _rotate(case, x, angle):
    """x: [..., rope dims] in 32 bits; angle: 64-bit, one per frequency, broadcast over the heads."""
    c, s = angle.cos().float(), angle.sin().float()
    if case["pairing"] == "neox":
        half = x.shape[-1] // 2
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _run_norm(s):
    case = s["case"]
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_write_normed_tokens(s["ctx"], s["pos"], s["k"], s["v"], s["req"], s["slot"], s["tables"], s["k_cache"], s["v_cache"],
                                    q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, q=s["q"], q_out=s["q_out"], workspace=s["ws"])
    else:
        angle = (s["pos"].double()[:, None] * _rope_theta(case))[:, None]         # [token, 1, frequency]
        q, k = s["q"].float(), s["k"].float()
        if case["kind"] == "gqa":
            q, k = _rotate(case, _norm(q, s["q_norm"]), angle), _rotate(case, _norm(k, s["k_norm"]), angle)
        else:
            q = torch.cat([q[..., :LATENT], _rotate(case, q[..., LATENT:], angle)], -1)
            k = torch.cat([_norm(k[..., :LATENT], s["k_norm"]), _rotate(case, k[..., LATENT:], angle)], -1)
        s["q_out"].copy_(q)
        live = s["slot"] >= 0
        slot, req = s["slot"][live].long(), s["req"][live].long()
        page, row = s["tables"][req, slot // case["block"]].long(), slot % case["block"]
        s["k_cache"][page, row] = k.to(torch.bfloat16)[live]
        if s["v"] is not None:
            s["v_cache"][page, row] = s["v"][live]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _softmax_parts(x, seen):
    """exp(x - max), their sum, and the log-sum-exp over the last axis, where seen; nothing seen: 0, 0, -inf."""
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    return e, total, top + total.log()


def _run_attend(s):
    case = s["case"]
    scale = case["head_dim"] ** -0.5
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_attend_tokens(s["ctx"], s["q"], scale, s["k_cache"], s["v_cache"], s["tables"], s["indptr"], s["slot"], s["out"],
                              window=case["window"], n_first=case["first"], lse=s["lse"], workspace=s["ws"])
        return [s["out"], s["lse"]]
    bs, hk, d = case["block"], case["kv_heads"], case["head_dim"]
    group = case["q_heads"] // hk
    reqs, longest = s["tables"].shape[0], s["tables"].shape[1] * bs
    count = s["indptr"][1:] - s["indptr"][:-1]
    i = torch.arange(case["per_req"], device="cuda")
    mine = i < count[:, None]                                                      # [request, token]
    token = torch.where(mine, s["indptr"][:-1, None] + i, 0).long()
    slot = torch.where(mine, s["slot"][token], -1)[..., None]
    t = torch.arange(longest, device="cuda")
    seen = t <= slot                                                               # [request, token, slot]
    if case["window"]:
        seen &= (t > slot - case["window"]) | (t < case["first"])
    some = seen.any(1)[:, :, None, None]
    pages = s["tables"].long().clamp(min=0)
    k = s["k_cache"][pages].reshape(reqs, longest, hk, d).float().masked_fill_(~some, 0.0).permute(0, 2, 3, 1)
    q = s["q"][token].float().reshape(reqs, -1, hk, group, d).permute(0, 2, 3, 1, 4).reshape(reqs, hk, -1, d)
    x = (torch.matmul(q, k) * scale).reshape(reqs, hk, group, -1, longest)
    del k
    e, total, lse = _softmax_parts(x, seen[:, None, None])
    v = s["v_cache"][pages].reshape(reqs, longest, hk, d).float().masked_fill_(~some, 0.0).transpose(1, 2)
    o = torch.matmul(e.reshape(reqs, hk, -1, longest), v).reshape(reqs, hk, group, -1, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(reqs, -1, hk * group, d)
    s["out"][token[mine]] = o[mine].to(torch.bfloat16)
    s["lse"][token[mine]] = lse[..., 0].permute(0, 3, 1, 2).reshape(reqs, -1, hk * group)[mine]
    return [s["out"], s["lse"]]


def _run_shared(s):
    case = s["case"]
    scale = case["head_dim"] ** -0.5
    if own:
        from position_independent_kv_stitch_gb300 import pic
        pic.pic_attend_shared(s["ctx"], s["q"], scale, s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_len"], s["tables"],
                              s["lens"], s["max_len"], s["out"], lse=s["lse"], workspace=s["ws"])
        return [s["out"], s["lse"]]
    bs, hk, d, prefix = case["block"], case["kv_heads"], case["head_dim"], case["prefix"]
    group, reqs = case["q_heads"] // hk, len(s["lens"])
    q = s["q"].float().reshape(reqs, hk, group, d)
    # the prefix once, for all requests' queries
    k = s["k_cache"][s["prefix_table"].long()].reshape(-1, hk, d)[:prefix].float()
    x = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, -1, d), k.permute(1, 2, 0)).reshape(hk, reqs, group, prefix).transpose(0, 1)
    # each request's own slots
    skip = prefix // bs
    pages = s["tables"][:, skip:].long()
    t = skip * bs + torch.arange(pages.shape[1] * bs, device="cuda")
    seen = (t >= prefix) & (t < s["lens"][:, None])
    k = s["k_cache"][pages].reshape(reqs, -1, hk, d).float().masked_fill_(~seen[:, :, None, None], 0.0).permute(0, 2, 3, 1)
    x = torch.cat([x, torch.matmul(q, k)], -1) * scale
    del k
    seen = torch.cat([torch.arange(prefix, device="cuda") < s["lens"][:, None], seen], -1)
    e, total, lse = _softmax_parts(x, seen[:, None, None])
    v = s["v_cache"][s["prefix_table"].long()].reshape(-1, hk, d)[:prefix].float()
    o = torch.matmul(e[..., :prefix].transpose(0, 1).reshape(hk, -1, prefix), v.transpose(0, 1)).reshape(hk, reqs, group, d).transpose(0, 1)
    v = s["v_cache"][pages].reshape(reqs, -1, hk, d).float().masked_fill_(~seen[:, prefix:, None, None], 0.0)
    o = o + torch.matmul(e[..., prefix:], v.transpose(1, 2))
    s["out"].copy_(torch.where(total > 0, o / total, torch.zeros_like(o)).reshape(s["out"].shape))
    s["lse"].copy_(lse.reshape(s["lse"].shape))
    return [s["out"], s["lse"]]


# ---------------------------------------------- the definitions, in 64 bits

def _turn(case, rows, pos):
    """Rows [n][heads][rope dims] in 64 bits, each frequency's pair as a complex number times exp(i pos theta)."""
    n = rows.shape[-1]
    theta = torch.tensor([THETA ** (-2.0 * i / n) for i in range(n // 2)], dtype=torch.float64, device="cuda")
    angle = (pos.double()[:, None] * theta)[:, None]
    first, second = (slice(0, n // 2), slice(n // 2, n)) if case["pairing"] == "neox" else (slice(0, n, 2), slice(1, n, 2))
    z = torch.complex(rows[..., first], rows[..., second]) * torch.polar(torch.ones_like(angle), angle)
    rows = rows.clone()
    rows[..., first], rows[..., second] = z.real, z.imag
    return rows


def _exact_norm(case, s):
    unit = lambda x, w: w.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)  # noqa: E731
    q, k = s["q"].double(), s["k"].double()
    if case["kind"] == "gqa":
        q, k = _turn(case, unit(q, s["q_norm"]), s["pos"]), _turn(case, unit(k, s["k_norm"]), s["pos"])
    else:
        k[..., :LATENT] = unit(k[..., :LATENT], s["k_norm"])
        for x in (q, k):
            x[..., LATENT:] = _turn(case, x[..., LATENT:], s["pos"])
    kc, vc, bs = s["k_cache"].double(), None if s["v"] is None else s["v_cache"].double(), case["block"]
    for r in range(case["reqs"]):
        i = ((s["req"] == r) & (s["slot"] >= 0)).nonzero().flatten()
        at = s["slot"][i].long()
        rows = s["tables"][r].long()[at // bs] * bs + at % bs
        kc.view(-1, *kc.shape[2:])[rows] = k[i]
        if vc is not None:
            vc.view(-1, *vc.shape[2:])[rows] = s["v"].double()[i]
    return [q, kc, vc]


def _one_attention(q, k, v, seen):
    """q [tokens][heads][dim], k and v [slots][dim] of their KV head, seen [tokens][slots]; (out, log-sum-exp)."""
    x = torch.einsum("nhd,td->nht", q, k) / math.sqrt(q.shape[-1])
    x = torch.where(seen[:, None], x, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None])
    return torch.einsum("nht,td->nhd", p, v), lse


def _exact_attend(case, s):
    out, lse = s["out"].double(), s["lse"].double()
    bs, group, at = case["block"], case["q_heads"] // case["kv_heads"], 0
    for r, (_, slots) in enumerate(_tokens(case)):
        rows = slice(at, at + len(slots))
        at += len(slots)
        runs, _ = _seen(case, slots)
        i = torch.cat([torch.arange(a, b) for a, b in runs]).cuda() if runs else torch.zeros(0, dtype=torch.long, device="cuda")
        if not len(i):
            out[rows], lse[rows] = 0.0, -math.inf
            continue
        mine = torch.tensor(slots, device="cuda")[:, None]
        seen = i[None] <= mine
        if case["window"]:
            seen &= (mine - i[None] < case["window"]) | (i[None] < case["first"])
        page, row = s["tables"][r].long()[i // bs], i % bs
        for h in range(case["kv_heads"]):
            heads = slice(h * group, (h + 1) * group)
            out[rows, heads], lse[rows, heads] = _one_attention(s["q"][rows, heads].double(), s["k_cache"][page, row, h].double(),
                                                                s["v_cache"][page, row, h].double(), seen)
    return [out, lse]


def _exact_shared(case, s):
    out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), s["lse"].double()
    bs, group = case["block"], case["q_heads"] // case["kv_heads"]
    for r, n in enumerate(_shared_lens(case)):
        i = torch.arange(n, device="cuda")
        page = torch.cat([s["prefix_table"].long()[i[:case["prefix"]] // bs], s["tables"][r].long()[i[case["prefix"]:] // bs]])
        if n == 0:
            lse[r] = -math.inf
            continue
        seen = torch.ones(1, n, dtype=torch.bool, device="cuda")
        for h in range(case["kv_heads"]):
            heads = slice(h * group, (h + 1) * group)
            out[r:r + 1, heads], lse[r:r + 1, heads] = _one_attention(
                s["q"][r:r + 1, heads].double(), s["k_cache"][page, i % bs, h].double(), s["v_cache"][page, i % bs, h].double(), seen)
    return [out, lse]


def _exact_map(case, s):
    lens, grow = _map_lens(case)
    tables, free, count = s["tables"].tolist(), s["free"].tolist(), int(s["n_free"])
    bs, at = case["block"], count
    up = lambda n: -(-n // bs)  # noqa: E731
    for r, (n, g) in enumerate(zip(lens, grow)):
        for b in range(up(n + g), up(n)):
            free[at] = tables[r][b]
            at += 1
    top, asked, new, ends, req, slot = at, 0, [], [0], [], []
    for r, (n, g) in enumerate(zip(lens, grow)):
        need = max(0, up(n + g) - up(n))
        asked += need
        ok = need == 0 or asked <= at
        for b in range(up(n), up(n) + need if ok else 0):
            top -= 1
            tables[r][b] = free[top]
        new.append(n + g if ok else n)
        ends.append(ends[-1] + max(0, g))
        req += [r] * max(0, g)
        slot += [n + j if ok else -1 for j in range(max(0, g))]
    req, slot = req + [0] * case["pad"], slot + [-1] * case["pad"]
    shift = s["shift"].tolist()
    pos = [x + shift[r] if x >= 0 else 0 for r, x in zip(req, slot)]
    return [_i32(x) for x in (new, tables, free, [top], ends, req, slot, pos)]


def exact(case, seed):
    return {"map": _exact_map, "norm": _exact_norm, "attend": _exact_attend, "shared": _exact_shared}[case["op"]](case, _inputs(case, seed))
