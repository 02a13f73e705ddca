"""What is measured of the decode that accumulates attention weight, the choice of tokens by it, and the decode of a shared prefix.

Three operators of the library (include/oscar.h):

- ``weights``  oscar_decode_attn_weights: one query token per sequence over sink + stored history + recent window, and each
  token's attention weight, summed over the query heads, added to a running score;
- ``select``   oscar_history_select: the history tokens that stay under a budget, by that score, as the list that
  oscar_history_gather takes;
- ``shared``   oscar_decode_attn_shared: the decode of a batch in which groups of sequences share the first pages of their
  histories, the shared pages attended once for all.

The history is stored in 2 or 4 bits.  A block of a (page, KV head) holds 64 tokens, ng = 128 / g (scale, zero) pairs per vector:
2 bits: K codes (byte 32 t + j: positions j, 32 + j, 64 + j, 96 + j from the low bits), V codes at 2048 (byte 64 j + t: the same
positions of token t), K pairs at 4096, V pairs behind them.  4 bits: K codes (byte 64 t + 16 a + 4 k + i: positions
32 k + 8 a + 2 i, low nibble, and the next one), K pairs, then at 4096 + 256 ng V codes (byte 64 j + t: positions 2 j and 2 j + 1)
and V pairs.  Value = s * code + z in the rotated domain; stored position p is output bitrev7(p) of x . U . Hadamard.
"""
import math

import torch

own = False
D, PAGE, SINK, RECENT = 128, 64, 64, 256
NSLOT = SINK + RECENT


def listed():
    return [
        # one sequence, one KV head, context 1024: the smallest step, where latency counts
        {"name": "weights-1x1k", "op": "weights", "bits": 4, "batch": 1, "hq": 4, "hk": 1, "group": 32, "lo": 705, "hi": 705, "std": 3.67,
         "slots": True, "decay": 1.0, "bf16": False},
        # batch 64, context 4K to 32K: one layer of a decode step that scores its tokens
        {"name": "weights-64x4k-32k", "op": "weights", "bits": 4, "batch": 64, "hq": 32, "hk": 8, "group": 32, "lo": 3777, "hi": 32449,
         "std": 3.67, "slots": True, "decay": 1.0, "bf16": True},
        # batch 8 at 32K in 2 bits, older weight fading
        {"name": "weights-8x32k-2bit", "op": "weights", "bits": 2, "batch": 8, "hq": 32, "hk": 8, "group": 32, "lo": 32449, "hi": 32449,
         "std": 3.67, "slots": True, "decay": 0.97, "bf16": True},
        # eight query heads per KV head, ragged from one token on, keys without outlier channels (a flat softmax)
        {"name": "weights-32x8k-g8-2bit", "op": "weights", "bits": 2, "batch": 32, "hq": 64, "hk": 8, "group": 128, "lo": 1, "hi": 8129,
         "std": 1.0, "slots": False, "decay": 1.0, "bf16": False},
        # two thirds of a short history
        {"name": "select-1x705", "op": "select", "batch": 1, "lo": 705, "hi": 705, "keep": 0.67, "protect": 64, "ties": False},
        # half of eight 32K histories
        {"name": "select-8x32k", "op": "select", "batch": 8, "lo": 32449, "hi": 32449, "keep": 0.5, "protect": 256, "ties": False},
        # a batch of 64 held under one budget, scores of few distinct values
        {"name": "select-64x4k-32k", "op": "select", "batch": 64, "lo": 3777, "hi": 32449, "keep": 0.25, "protect": 256, "ties": True},
        # one long context cut to a tenth
        {"name": "select-1x100k", "op": "select", "batch": 1, "lo": 100033, "hi": 100033, "keep": 0.1, "protect": 1024, "ties": False},
        # four samples of one short prompt
        {"name": "shared-4x1k-2bit", "op": "shared", "bits": 2, "batch": 4, "hq": 4, "hk": 1, "group": 32, "groups": 1, "alone": 0,
         "prefix": 704, "lo": 1, "hi": 64, "short": False, "std": 3.67, "bf16": False},
        # 64 requests behind one 28K document
        {"name": "shared-64x28k", "op": "shared", "bits": 4, "batch": 64, "hq": 32, "hk": 8, "group": 32, "groups": 1, "alone": 0,
         "prefix": 28672, "lo": 64, "hi": 3777, "short": False, "std": 3.67, "bf16": True},
        # 256 sequences, half of them behind an 8K prefix, in 2 bits
        {"name": "shared-256x8k-2bit", "op": "shared", "bits": 2, "batch": 256, "hq": 32, "hk": 8, "group": 32, "groups": 1, "alone": 128,
         "prefix": 8192, "lo": 705, "hi": 4033, "short": False, "std": 3.67, "bf16": True},
        # three prompts with several samples each and some sequences of their own; eight query heads per KV head, fp32 output
        {"name": "shared-32x16k-g8", "op": "shared", "bits": 4, "batch": 32, "hq": 64, "hk": 8, "group": 128, "groups": 3, "alone": 8,
         "prefix": 16384, "lo": 0, "hi": 1025, "short": True, "std": 1.0, "bf16": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "select", "shared", "shared"])
    hk, g, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([32, 64, 128])
    bits, std, bf16 = rng.choice([2, 4]), rng.choice([1.0, 3.67]), rng.random() < 0.5
    if op == "weights":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, min(100000, 700000 // batch))
        return {"op": op, "bits": bits, "batch": batch, "hq": hk * g, "hk": hk, "group": group, "lo": rng.randint(0, hi), "hi": hi, "std": std,
                "slots": rng.random() < 0.7, "decay": rng.choice([1.0, 1.0, 0.9, 0.0]), "bf16": bf16}
    if op == "select":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, min(131072, 2000000 // batch))
        return {"op": op, "batch": batch, "lo": rng.randint(0, hi), "hi": hi, "keep": rng.choice([0.02, 0.1, 0.25, 0.5, 0.9, 1.0]),
                "protect": rng.choice([0, 1, 64, 256]), "ties": rng.random() < 0.4}
    batch = _log(rng, 2, 128)
    groups = rng.choice([1, 1, 1, 2, 3])
    prefix = PAGE * _log(rng, 1, min(1000, 14000 // batch))
    hi = _log(rng, 1, min(8192, 450000 // batch))
    return {"op": op, "bits": bits, "batch": batch, "hq": hk * g, "hk": hk, "group": group, "groups": groups, "alone": rng.randint(0, batch // 2),
            "prefix": prefix, "lo": rng.randint(0, hi), "hi": hi, "short": rng.random() < 0.2, "std": std, "bf16": bf16}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _block(bits, group):
    return (4096 if bits == 2 else 8192) + 512 * (D // group)


def _pairs_at(bits, group):
    """Byte offsets of the K and the V (scale, zero) pairs inside a block."""
    ng = D // group
    return (4096, 4096 + 256 * ng) if bits == 2 else (4096, 4096 + 256 * ng + 4096)


def _pool(gen, pages, hk, bits, group, std):
    """Blocks of codes with the pairs of groups of normal values of this deviation."""
    ng, top = D // group, 3 if bits == 2 else 15
    pool = torch.randint(0, 256, (max(pages, 1), hk, _block(bits, group)), dtype=torch.uint8, device="cuda", generator=gen)
    half = math.sqrt(2 * math.log(group)) * 0.8 * std     # about the largest of `group` normal values
    for at in _pairs_at(bits, group):
        r = torch.rand(pool.shape[0], hk, PAGE * ng, 2, device="cuda", generator=gen)
        lo, hi = -half * (0.8 + 0.4 * r[..., 0]), half * (0.8 + 0.4 * r[..., 1])
        sz = torch.stack([(hi - lo) / top, lo], -1).half()
        pool[:, :, at:at + 256 * ng] = sz.view(torch.uint8).reshape(pool.shape[0], hk, 256 * ng)
    return pool


def _rotation(gen, hk):
    """Orthogonal U [hk][2][d][d], as an offline calibration gives it."""
    q, _ = torch.linalg.qr(torch.randn(hk * 2, D, D, device="cuda", generator=gen))
    return q.reshape(hk, 2, D, D).contiguous()


def _lengths(gen, lo, hi, batch):
    n = torch.randint(lo, hi + 1, (batch,), generator=gen, device="cuda").int()
    n[-1] = hi
    return n


def _scores(gen, shape):
    """Accumulated attention weight: a few tokens hold most of it."""
    return torch.exp(2.0 * torch.randn(shape, device="cuda", generator=gen) - 4.0)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    op, batch = case["op"], case["batch"]
    if op == "select":
        s["hist"] = _lengths(gen, case["lo"], case["hi"], batch)
        width = (case["hi"] + PAGE - 1) // PAGE * PAGE
        s["weight"] = _scores(gen, (batch, width))
        if case["ties"]:
            s["weight"] = (s["weight"] * 64).round() / 64
        s["budget"] = (s["hist"] * case["keep"]).int()
        s["keep_list"] = torch.full((batch, max(1, int(s["budget"].max()))), -1, dtype=torch.int32, device="cuda")
        s["n_keep"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros_like(s["weight"])
        if own:
            from bit_kv_cache_evict_gb300 import oscar as O
            s["O"] = O
        return s
    hq, hk, bits, group = case["hq"], case["hk"], case["bits"], case["group"]
    if op == "weights":
        s["hist"] = _lengths(gen, case["lo"], case["hi"], batch)
        need = [(h + PAGE - 1) // PAGE for h in s["hist"].tolist()]
        most, pages = max(1, max(need)), sum(need)
        ids = torch.randperm(pages, generator=gen, device="cuda").int()
        s["table"] = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            s["table"][b, :n] = ids[at:at + n]
            at += n
        s["weight"] = _scores(gen, (batch, most * PAGE))
        s["slot_weight"] = _scores(gen, (batch, NSLOT)) if case["slots"] else None
    else:
        # the first batch - alone sequences belong to a group each, in a seeded order; every history is its group's
        # prefix (if any) and tokens of its own; `short`: one member's history ends inside the prefix
        order = torch.randperm(batch, generator=gen, device="cuda")
        group_of = torch.where(order < batch - case["alone"], order % case["groups"], -1).int()
        shared = case["prefix"] // PAGE
        hist = _lengths(gen, case["lo"], case["hi"], batch) + torch.where(group_of >= 0, case["prefix"], 0).int()
        if case["short"]:
            hist[0] = torch.clamp(hist[0], max=case["prefix"] // 2 + 1)
        s["hist"], s["group_of"] = hist, group_of
        s["group_pages"] = torch.full((case["groups"],), shared, dtype=torch.int32, device="cuda")
        need = [(h + PAGE - 1) // PAGE for h in hist.tolist()]
        first = [min(n, shared) if g >= 0 else 0 for n, g in zip(need, group_of.tolist())]
        most = max(1, max(need))
        pages = case["groups"] * shared + sum(need) - sum(first)
        ids = torch.randperm(pages, generator=gen, device="cuda").int()
        s["table"] = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
        at = case["groups"] * shared
        for b, (n, f, g) in enumerate(zip(need, first, group_of.tolist())):
            s["table"][b, :f] = ids[g * shared:g * shared + f] if f else ids[:0]
            s["table"][b, f:n] = ids[at:at + n - f]
            at += n - f
    s["num_pages"] = pages
    s["pool"] = _pool(gen, pages, hk, bits, group, case["std"])
    s["U"] = _rotation(gen, hk)
    s["kv"] = (torch.randn(batch, NSLOT, hk, 2, D, device="cuda", generator=gen) * case["std"]).bfloat16()
    # a context without history may have a part of its windows only
    part = torch.randint(1, NSLOT + 1, (batch,), generator=gen, device="cuda").int()
    s["len"] = torch.where(s["hist"] > 0, torch.full_like(part, NSLOT), part)
    s["q"] = torch.randn(batch, hq, D, device="cuda", generator=gen).bfloat16()
    s["out"] = torch.empty(batch, hq, D, dtype=torch.bfloat16 if case["bf16"] else torch.float32, device="cuda")
    if own:
        from bit_kv_cache_evict_gb300 import oscar as O
        s["O"] = O
        s["shape"] = O.make_shape(hq, hk, quant_group=group)
        if op == "weights":
            size = O.oscar_decode_workspace_bytes_weights(s["shape"], bits, batch, most)
        else:
            size = O.oscar_decode_workspace_bytes_shared(s["shape"], bits, batch, most, case["groups"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        O = s["O"]
        if op == "weights":
            O.oscar_decode_attn_weights(s["shape"], s["bits"], s["q"], s["kv"], s["len"], s["pool"], s["table"], s["table"].shape[1], s["num_pages"],
                                        s["hist"], s["U"], 1 / math.sqrt(D), s["out"], s["weight"], s["ws"], slot_weight=s["slot_weight"],
                                        decay=s["decay"])
            return [s["out"], s["weight"]] + ([s["slot_weight"]] if s["slots"] else [])
        if op == "select":
            O.oscar_history_select(s["weight"], s["hist"], s["budget"], s["keep_list"], s["n_keep"], protect=s["protect"], kept_weight=s["kept"])
            return s["keep_list"], s["n_keep"], s["kept"]
        O.oscar_decode_attn_shared(s["shape"], s["bits"], s["q"], s["kv"], s["len"], s["pool"], s["table"], s["table"].shape[1], s["num_pages"],
                                   s["hist"], s["group_of"], s["group_pages"], s["U"], 1 / math.sqrt(D), s["out"], s["ws"])
        return s["out"]
    if op == "select":
        return _plain_select(s)
    out, ph, pb, total = _plain_decode(s)
    if op == "shared":
        return out
    ph, pb = (ph / total).sum((1, 2)), (pb / total).sum((1, 2))
    inside = torch.arange(ph.shape[1], device="cuda") < s["hist"][:, None]
    s["weight"].copy_(torch.where(inside, s["decay"] * s["weight"] + ph, s["weight"]))
    if not s["slots"]:
        return [out, s["weight"]]
    inside = torch.arange(NSLOT, device="cuda") < s["len"][:, None]
    s["slot_weight"].copy_(torch.where(inside, s["decay"] * s["slot_weight"] + pb, s["slot_weight"]))
    return [out, s["weight"], s["slot_weight"]]


def _bitrev():
    i = torch.arange(D, device="cuda")
    return sum(((i >> k) & 1) << (6 - k) for k in range(7))


def _hadamard(dtype):
    """Sylvester order, orthonormal, its columns in stored order."""
    i = torch.arange(D, device="cuda")
    bits = (i[:, None] & i[None, :])
    odd = sum((bits >> k) & 1 for k in range(7)) & 1
    h = (1 - 2 * odd).to(dtype) / math.sqrt(D)
    return h[:, _bitrev()]


def _plain_values(pool, bits, group):
    """K and V values fp32 [pages][hk][64][d] in stored order."""
    n, hk = pool.shape[:2]
    ng = D // group
    at = _pairs_at(bits, group)
    sz = [pool[:, :, a:a + 256 * ng].contiguous().view(torch.float16).reshape(n, hk, PAGE, ng, 2).float() for a in at]
    if bits == 2:
        k = torch.stack([(pool[:, :, :2048].reshape(n, hk, PAGE, 32) >> (2 * i)) & 3 for i in range(4)], 3)
        v = torch.stack([(pool[:, :, 2048:4096].reshape(n, hk, 32, PAGE).transpose(2, 3) >> (2 * i)) & 3 for i in range(4)], 3)
    else:
        b = pool[:, :, :4096].reshape(n, hk, PAGE, 4, 4, 4).transpose(3, 4)
        k = torch.stack([b & 15, b >> 4], -1)
        h = at[0] + 256 * ng
        b = pool[:, :, h:h + 4096].reshape(n, hk, 64, PAGE).transpose(2, 3)
        v = torch.stack([b & 15, b >> 4], -1)
    return [(c.reshape(n, hk, PAGE, ng, group).float() * p[..., :1] + p[..., 1:]).reshape(n, hk, PAGE, D) for c, p in zip((k, v), sz)]


def _plain_decode(s):
    """The output, the numerators of the weights of history and windows, and their sum."""
    batch, hq, hk = s["batch"], s["hq"], s["hk"]
    g = hq // hk
    rot = s["U"] @ _hadamard(torch.float32)                    # [hk][2][d][d]
    q = s["q"].float().reshape(batch, hk, g, D)
    k, v = _plain_values(s["pool"], s["bits"], s["group"])
    page = s["table"].long().clamp(min=0)
    most = page.shape[1] * PAGE
    inside = (torch.arange(most, device="cuda") < s["hist"][:, None])[:, None, None]
    k = k[page].permute(0, 2, 1, 3, 4).reshape(batch, hk, most, D)
    lh = torch.matmul(torch.einsum("bhgd,hde->bhge", q, rot[:, 0]), k.transpose(2, 3)) / math.sqrt(D)
    del k
    lh = lh.masked_fill(~inside, -math.inf)
    kv = s["kv"].float().permute(0, 2, 3, 1, 4)                # [batch][hk][2][slots][d]
    lb = torch.matmul(q, kv[:, :, 0].transpose(2, 3)) / math.sqrt(D)
    lb = lb.masked_fill(torch.arange(NSLOT, device="cuda") >= s["len"][:, None, None, None], -math.inf)
    top = torch.maximum(lh.amax(-1, keepdim=True), lb.amax(-1, keepdim=True))
    ph, pb = torch.exp(lh - top), torch.exp(lb - top)
    v = v[page].permute(0, 2, 1, 3, 4).reshape(batch, hk, most, D)
    o = torch.einsum("bhge,hde->bhgd", torch.matmul(ph, v), rot[:, 1]) + torch.matmul(pb, kv[:, :, 1])
    total = ph.sum(-1, keepdim=True) + pb.sum(-1, keepdim=True)
    return (o / total).reshape(batch, hq, D).to(s["out"].dtype), ph, pb, total


def _plain_select(s):
    """The newest `protect` tokens first, then the others by score (ties to the lower position), as many as the budget has."""
    hist, at = s["hist"][:, None], torch.arange(s["weight"].shape[1], device="cuda")
    m = torch.minimum(s["budget"], s["hist"])[:, None]
    w = torch.where(at < hist - s["protect"], s["weight"], math.inf)   # (scores are finite)
    w = torch.where(at < hist, w, -math.inf)
    # protected tokens are taken from the newest on where the budget has no room for all
    newest = torch.where((at < hist) & (at >= hist - s["protect"]), at, 0)
    order = torch.argsort(newest, dim=1, descending=True, stable=True)
    order = torch.gather(order, 1, torch.argsort(torch.gather(w, 1, order), dim=1, descending=True, stable=True))
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(1, order, at < m)
    place = kept.long().cumsum(1) - 1
    b, pos = kept.nonzero(as_tuple=True)
    to = place[b, pos]
    s["keep_list"][b, to] = pos.int()
    s["kept"][b, to] = s["weight"][b, pos]
    s["n_keep"].copy_(m[:, 0])
    return s["keep_list"], s["n_keep"], s["kept"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, batch = case["op"], case["batch"]
    mean = batch * (case["lo"] + case["hi"]) / 2
    if op == "select":
        # a score read per token, a position and a score written per kept one
        return {"bytes": mean * 4 + mean * case["keep"] * 8, "flops": mean}
    hk, hq = case["hk"], case["hq"]
    stored = (2 * 32 if case["bits"] == 2 else 2 * 64) + 8 * (D // case["group"])   # bytes of a token and KV head, K and V
    slots = batch * NSLOT
    fixed = slots * hk * 512 + batch * hq * D * (2 + (2 if case["bf16"] else 4)) + hk * 2 * D * D * 4
    if op == "weights":
        scores = (mean + (slots if case["slots"] else 0)) * (8 if case["decay"] else 4)
        return {"bytes": mean * hk * stored + fixed + scores, "flops": (mean + slots) * hq * (4 * D + 2)}
    once = case["groups"] * case["prefix"]
    return {"bytes": (mean + once) * hk * stored + fixed,
            "flops": (mean + (batch - case["alone"]) * case["prefix"] + slots) * hq * 4 * D}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _matrix(U):
    """R = U . Hadamard . bit-reversal of one KV head's K or V, 64 bits."""
    h = torch.ones(1, 1, dtype=torch.float64, device=U.device)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    order = [int(format(p, "07b")[::-1], 2) for p in range(D)]
    return (U.double() @ (h / h[0].norm()))[:, order]


def _stored(pool, page, slot, which, bits, group):
    """64-bit values [tokens][d] of one KV head's K or V: `pool` [pages][block], in stored order."""
    ng = D // group
    p = torch.arange(D, device=pool.device)
    slot = slot[:, None]
    if bits == 2:
        byte, shift = (slot * 32 + p % 32 if which == 0 else 2048 + (p % 32) * 64 + slot), 2 * (p // 32)
        pairs = 4096 + which * 256 * ng
    else:
        half = 4096 + 256 * ng
        byte = slot * 64 + 16 * ((p % 32) // 8) + 4 * (p // 32) + (p % 8) // 2 if which == 0 else half + (p // 2) * 64 + slot
        shift = 4 * (p % 2)
        pairs = which * half + 4096
    code = (pool[page[:, None], byte].long() >> shift) & (3 if bits == 2 else 15)
    words = pool[:, pairs:pairs + 256 * ng].contiguous().view(torch.float16)
    at = (slot * ng + p // group) * 2
    return words[page[:, None], at].double() * code + words[page[:, None], at + 1].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return None
    g = case["hq"] // case["hk"]
    out = torch.zeros(case["batch"], case["hq"], D, dtype=torch.float64, device="cuda")
    scored = case["op"] == "weights"
    if scored:
        weight = s["weight"].double()
        slot_weight = s["slot_weight"].double() if case["slots"] else None
    mats = [[_matrix(s["U"][h, w]) for w in (0, 1)] for h in range(case["hk"])]
    for b in range(case["batch"]):
        n, m = int(s["hist"][b]), int(s["len"][b])
        at = torch.arange(n, device="cuda")
        page, slot = s["table"][b].long()[at // PAGE], at % PAGE
        step = torch.zeros(n + m, dtype=torch.float64, device="cuda")
        for h in range(case["hk"]):
            keys, vals = (torch.cat([_stored(s["pool"][:, h], page, slot, w, case["bits"], case["group"]) @ mats[h][w].T, s["kv"][b, :m, h, w].double()])
                          for w in (0, 1))
            p = torch.softmax(s["q"][b, h * g:(h + 1) * g].double() @ keys.T / math.sqrt(D), -1)
            out[b, h * g:(h + 1) * g] = p @ vals
            step += p.sum(0)
        if scored:
            weight[b, :n] = case["decay"] * weight[b, :n] + step[:n]
            if case["slots"]:
                slot_weight[b, :m] = case["decay"] * slot_weight[b, :m] + step[n:]
    if not scored:
        return out
    return [out, weight] + ([slot_weight] if case["slots"] else [])
