"""What is measured of the 4-bit history and of the calls that move, gather and read stored tokens.

Five operators of the library (include/oscar.h):

- ``evict``   oscar_evict_quantize_int4: token rows into the 4-bit history, read back with oscar_history_read (the
  stored codes are returned as the values they stand for);
- ``decode``  oscar_decode_attn_int4: one query token per sequence over sink + 4-bit history + recent window;
- ``read``    oscar_history_read: stored tokens back as rows, in the rotated domain;
- ``copy``    oscar_pages_copy_device: pages copied in every layer's pool by one launch;
- ``gather``  oscar_history_gather: the kept tokens of each history moved into fresh pages.

A 4-bit block of a (page, KV head), ng = 128 / g (scale, zero) pairs per vector, half = 4096 + 256 ng bytes:
K codes (byte 64 t + 16 a + 4 k + i: stored positions 32 k + 8 a + 2 i, low nibble, and the next one), K pairs (4 ng
bytes per token, fp16 s then fp16 z), then at ``half`` V codes (byte 64 j + t: positions 2 j and 2 j + 1 of token t)
and V pairs.  Value = s * code + z in the rotated domain; stored position p is output bitrev7(p) of x . U . Hadamard.
"""
import math

import torch

own = False
D, PAGE, SINK, RECENT = 128, 64, 64, 256
NSLOT = SINK + RECENT
LAYERS = 36


def listed():
    return [
        # a decode step's eviction of 64 sequences (the batch of the 36-layer workload), ring append included
        {"name": "evict-step-64", "op": "evict", "batch": 64, "hk": 8, "group": 32, "per_seq": 1, "append": True},
        # the history of four 4096-token prompts, quantised in one call
        {"name": "evict-prompt-4x3776", "op": "evict", "batch": 4, "hk": 8, "group": 32, "per_seq": 3776, "append": False},
        # one sequence, one KV head, context 1024: the smallest step, where latency counts
        {"name": "decode-1x1k", "op": "decode", "batch": 1, "hq": 4, "hk": 1, "group": 32, "lo": 705, "hi": 705, "std": 3.67,
         "shuffled": False, "bf16": False},
        # batch 8 at 32K, 32 query and 8 KV heads, contiguous pages
        {"name": "decode-8x32k", "op": "decode", "batch": 8, "hq": 32, "hk": 8, "group": 32, "lo": 32449, "hi": 32449, "std": 3.67,
         "shuffled": False, "bf16": True},
        # batch 64, context 4K to 32K, shuffled pages: one layer of the 36-layer workload
        {"name": "decode-64x4k-32k", "op": "decode", "batch": 64, "hq": 32, "hk": 8, "group": 32, "lo": 3777, "hi": 32449,
         "std": 3.67, "shuffled": True, "bf16": True},
        # eight query heads per KV head, one scale per vector; keys without outlier channels (a flat softmax)
        {"name": "decode-32x32k-g8", "op": "decode", "batch": 32, "hq": 64, "hk": 8, "group": 128, "lo": 32449, "hi": 32449,
         "std": 1.0, "shuffled": True, "bf16": False},
        # a short 2-bit history restored for a prompt that continues it
        {"name": "read-2bit-705", "op": "read", "bits": 2, "hk": 8, "group": 64, "tokens": 705, "bf16": True},
        # a 32K 4-bit history restored
        {"name": "read-4bit-32448", "op": "read", "bits": 4, "hk": 8, "group": 32, "tokens": 32448, "bf16": True},
        # three sequences fork inside a page: three pages copied in each of 36 layers
        {"name": "copy-3x36", "op": "copy", "bits": 4, "hk": 8, "group": 32, "pages": 3, "pools": LAYERS},
        # 2048 pages of one pool moved (a pool made dense again)
        {"name": "copy-2048", "op": "copy", "bits": 4, "hk": 8, "group": 32, "pages": 2048, "pools": 1},
        # a third of a short 2-bit history dropped
        {"name": "gather-2bit-705", "op": "gather", "bits": 2, "batch": 1, "hk": 1, "group": 32, "hist": 705, "keep": 0.67},
        # half of eight 32K histories kept (tokens chosen by a score)
        {"name": "gather-8x32k", "op": "gather", "bits": 4, "batch": 8, "hk": 8, "group": 32, "hist": 32448, "keep": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["evict", "decode", "decode", "read", "copy", "gather"])
    group = rng.choice([32, 64, 128])
    if op == "evict":
        if rng.random() < 0.5:
            return {"op": op, "batch": _log(rng, 1, 256), "hk": rng.choice([1, 2, 4, 8]), "group": group, "per_seq": 1, "append": True}
        return {"op": op, "batch": rng.randint(1, 4), "hk": rng.choice([1, 2, 4, 8]), "group": group, "per_seq": _log(rng, 2, 3776),
                "append": False}
    if op == "decode":
        hk, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 64)
        top = max(2, 700000 // batch)
        hi = _log(rng, 1, min(100000, top))
        return {"op": op, "batch": batch, "hq": hk * g, "hk": hk, "group": group, "lo": rng.randint(0, hi), "hi": hi,
                "std": rng.choice([1.0, 3.67]), "shuffled": rng.random() < 0.5, "bf16": rng.random() < 0.5}
    if op == "read":
        return {"op": op, "bits": rng.choice([2, 4]), "hk": rng.choice([1, 2, 4, 8]), "group": group, "tokens": _log(rng, 1, 32448),
                "bf16": rng.random() < 0.7}
    if op == "copy":
        pools = rng.choice([1, 1, 4, LAYERS])
        return {"op": op, "bits": rng.choice([2, 4]), "hk": rng.choice([1, 2, 4, 8]), "group": group,
                "pages": _log(rng, 1, 2048 // pools), "pools": pools}
    return {"op": op, "bits": rng.choice([2, 4]), "batch": rng.randint(1, 8), "hk": rng.choice([1, 2, 4, 8]), "group": group,
            "hist": _log(rng, 1, 32448), "keep": rng.choice([0.1, 0.5, 0.67, 0.95, 1.0])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _block(bits, group):
    return (4096 if bits == 2 else 8192) + 512 * (D // group)


def _pairs_at(bits, group):
    """Byte offsets of the K and the V (scale, zero) pairs inside a block."""
    ng = D // group
    return (4096, 4096 + 256 * ng) if bits == 2 else (4096, 4096 + 256 * ng + 4096)


def _table(gen, batch, need, shuffled, extra=0):
    """int32 [batch][max] page ids (-1 unused) for need[b] pages each, and the number of pages."""
    most, total = max(1, max(need)), sum(need)
    ids = torch.randperm(total + extra, generator=gen, device="cuda") if shuffled else torch.arange(total + extra, device="cuda")
    table = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n].int()
        at += n
    return table, ids[total:].int(), total + extra


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


def _rows(gen, shape, hk, n_outlier=4):
    """K/V rows of normal values with a few channels of 20 times the size, per KV head and K/V."""
    at = torch.randint(0, D, (hk, 2, n_outlier), device="cuda", generator=gen)
    scale = torch.ones(hk, 2, D, device="cuda").scatter_(-1, at, 20.0)
    x = torch.randn(*shape, hk, 2, D, device="cuda", generator=gen) * scale
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    op, hk, group = case["op"], case["hk"], case["group"]
    if op == "evict":
        batch, per = case["batch"], case["per_seq"]
        # a step's tokens go behind histories of any length; a prompt's tokens fill the pages from the start
        start = torch.randint(0, 500, (batch,), generator=gen, device="cuda").int() if per == 1 else torch.zeros(batch, dtype=torch.int32, device="cuda")
        s["table"], _, s["num_pages"] = _table(gen, batch, [(int(h) + per + PAGE - 1) // PAGE for h in start.tolist()], True)
        s["pool"] = torch.zeros(s["num_pages"], hk, _block(4, group), dtype=torch.uint8, device="cuda")
        s["seq"] = torch.arange(batch, device="cuda").int().repeat_interleave(per)
        s["pos"] = (start[:, None] + torch.arange(per, device="cuda")).int().reshape(-1)
        s["U"], s["clip"] = _rotation(gen, hk), 0.9 + 0.1 * torch.rand(hk, 2, device="cuda", generator=gen)
        if case["append"]:
            s["kv"] = _rows(gen, (batch * NSLOT,), hk)
            s["row"] = (torch.arange(batch, device="cuda") * NSLOT + SINK + torch.randint(0, RECENT, (batch,), generator=gen, device="cuda")).int()
            s["new"] = _rows(gen, (batch,), hk)
        else:
            s["kv"], s["row"], s["new"] = _rows(gen, (batch * per,), hk), None, None
        s["out"] = torch.empty(batch * per, hk, 2, D, dtype=torch.bfloat16, device="cuda")
    elif op == "decode":
        batch, hq = case["batch"], case["hq"]
        hist = torch.randint(case["lo"], case["hi"] + 1, (batch,), generator=gen, device="cuda").int()
        hist[-1] = case["hi"]
        need = [(h + PAGE - 1) // PAGE for h in hist.tolist()]
        s["table"], _, s["num_pages"] = _table(gen, batch, need, case["shuffled"])
        s["pool"] = _pool(gen, s["num_pages"], hk, 4, group, case["std"])
        s["hist"] = hist
        s["U"] = _rotation(gen, hk)
        s["kv"] = (torch.randn(batch, NSLOT, hk, 2, D, device="cuda", generator=gen) * case["std"]).bfloat16()
        # a context without history may have a part of its windows only
        part = torch.randint(1, NSLOT + 1, (batch,), generator=gen, device="cuda").int()
        s["len"] = torch.where(hist > 0, torch.full_like(part, NSLOT), part)
        s["q"] = torch.randn(batch, hq, D, device="cuda", generator=gen).bfloat16()
        s["out"] = torch.empty(batch, hq, D, dtype=torch.bfloat16 if case["bf16"] else torch.float32, device="cuda")
    elif op == "read":
        n = case["tokens"]
        s["table"], _, s["num_pages"] = _table(gen, 1, [(n + PAGE - 1) // PAGE], True)
        s["pool"] = _pool(gen, s["num_pages"], hk, case["bits"], group, 3.67)
        s["seq"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["pos"] = torch.arange(n, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(n, hk, 2, D, dtype=torch.bfloat16 if case["bf16"] else torch.float32, device="cuda")
    elif op == "copy":
        n = case["pages"]
        s["num_pages"] = 2 * n + 1
        ids = torch.randperm(2 * n, generator=gen, device="cuda").int()
        s["src"], s["dst"] = ids[:n].contiguous(), ids[n:].contiguous()
        s["pools"] = [torch.randint(0, 256, (s["num_pages"], hk, _block(case["bits"], group)), dtype=torch.uint8, device="cuda", generator=gen)
                      for _ in range(case["pools"])]
    else:
        batch, hist = case["batch"], case["hist"]
        need = [(hist + PAGE - 1) // PAGE] * batch
        most = max(1, int(hist * case["keep"]))
        n_keep = torch.tensor([max(1, most - 3 * b) for b in range(batch)], device="cuda")   # each sequence keeps its own number
        best = torch.rand(batch, hist, device="cuda", generator=gen).argsort(1)[:, :most]
        best = torch.where(torch.arange(most, device="cuda") < n_keep[:, None], best, hist)  # behind the last: past the history
        s["keep"] = best.sort(1).values.int().contiguous()
        s["n_keep"] = n_keep.int()
        fresh = [(int(k) + PAGE - 1) // PAGE for k in n_keep.tolist()]
        s["table"], spare, s["num_pages"] = _table(gen, batch, need, True, extra=sum(fresh))
        s["dst_table"] = torch.full((batch, max(fresh)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, f in enumerate(fresh):
            s["dst_table"][b, :f] = spare[at:at + f]
            at += f
        s["pool"] = _pool(gen, s["num_pages"], hk, case["bits"], group, 3.67)
    if own:
        from bit_kv_cache_evict_gb300 import oscar as O
        s["O"] = O
        s["shape"] = O.make_shape(case.get("hq", hk), hk, quant_group=group)
        if op == "decode":
            s["ws"] = torch.empty(O.oscar_decode_workspace_bytes_int4(s["shape"], case["batch"], s["table"].shape[1]), dtype=torch.uint8,
                                  device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        O, sh = s["O"], s["shape"]
        if op == "evict":
            batch, most = s["table"].shape
            O.oscar_evict_quantize_int4(sh, s["kv"], s["seq"], s["pos"], s["U"], s["clip"], s["pool"], s["table"], batch, most, s["num_pages"],
                                        src_row=s["row"], new_kv=s["new"])
            O.oscar_history_read(sh, 4, s["seq"], s["pos"], s["pool"], s["table"], batch, most, s["num_pages"], s["out"])
            return s["out"], s["kv"]
        if op == "decode":
            O.oscar_decode_attn_int4(sh, s["q"], s["kv"], s["len"], s["pool"], s["table"], s["table"].shape[1], s["num_pages"], s["hist"], s["U"],
                                     1 / math.sqrt(D), s["out"], s["ws"])
            return s["out"]
        if op == "read":
            O.oscar_history_read(sh, s["bits"], s["seq"], s["pos"], s["pool"], s["table"], 1, s["table"].shape[1], s["num_pages"], s["out"])
            return s["out"]
        if op == "copy":
            O.oscar_pages_copy_device(s["pools"][0][0].numel(), s["src"], s["dst"], s["pools"], s["num_pages"])
            return s["pools"]
        O.oscar_history_gather(sh, s["bits"], s["pool"], s["table"], s["dst_table"], s["keep"], s["n_keep"], s["num_pages"])
        return s["pool"]
    if op == "evict":
        return _plain_evict(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "read":
        page = s["table"][s["seq"].long(), s["pos"].long() // PAGE].long()
        k, v = _plain_values(s["pool"], s["bits"], s["group"])
        rows = torch.stack([k, v], 3)                          # [pages][hk][64][2][d]
        return rows[page, :, s["pos"].long() % PAGE].to(s["out"].dtype)
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        return [p.index_copy_(0, dst, p[src]) for p in s["pools"]]
    return _plain_gather(s)


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


def _half(x):
    """64-bit values rounded to fp16 once, to nearest even."""
    e = torch.frexp(x)[1].clamp(min=-13)
    ulp = torch.ldexp(torch.ones_like(x), e - 11)
    return (torch.round(x / ulp) * ulp).half()


def _plain_evict(s):
    hk, group, pool = s["hk"], s["group"], s["pool"]
    row = s["row"].long() if s["row"] is not None else slice(None)
    x = s["kv"][row].double()                                  # codes lie next to borders: 64 bits
    y = torch.einsum("nhwd,hwde->nhwe", x, s["U"].double()) @ _hadamard(torch.float64)
    y = y.reshape(*y.shape[:3], D // group, group)
    c = s["clip"].double()[None, :, :, None, None]
    t = torch.where(c < 1, c * y.abs().amax(-1, keepdim=True), math.inf)
    y = torch.minimum(torch.maximum(y, -t), t)
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    sc, z = _half((hi - lo) / 15), _half(lo)
    code = torch.where(sc > 0, torch.round((y - z.double()) / torch.where(sc > 0, sc.double(), 1)).clamp(0, 15), 0)
    page, slot = s["table"][s["seq"].long(), s["pos"].long() // PAGE].long(), s["pos"].long() % PAGE
    n, ng = page.numel(), D // group
    at = _pairs_at(4, group)
    sz = torch.cat([sc, z], -1).view(torch.uint8).reshape(n, hk, 2, 4 * ng)
    both = code.to(torch.uint8).reshape(n, hk, 2, 64, 2)
    both = both[..., 0] | (both[..., 1] << 4)                  # byte j: positions 2j, 2j + 1
    kc = both[:, :, 0].reshape(n, hk, 4, 4, 4).transpose(2, 3).reshape(n, hk, 64)
    pool[:, :, :4096].unflatten(2, (PAGE, 64))[page, :, slot] = kc
    pool[:, :, at[0]:at[0] + 256 * ng].unflatten(2, (PAGE, 4 * ng))[page, :, slot] = sz[:, :, 0]
    h = at[0] + 256 * ng
    pool[:, :, h:h + 4096].unflatten(2, (64, PAGE)).transpose(2, 3)[page, :, slot] = both[:, :, 1]
    pool[:, :, at[1]:at[1] + 256 * ng].unflatten(2, (PAGE, 4 * ng))[page, :, slot] = sz[:, :, 1]
    if s["new"] is not None:
        s["kv"][row] = s["new"]
    values = (code.reshape(n, hk, 2, ng, group).float() * sc.float() + z.float()).reshape(n, hk, 2, D)
    return values.bfloat16(), s["kv"]


def _plain_decode(s):
    batch, hq, hk = s["batch"], s["hq"], s["hk"]
    g = hq // hk
    h = _hadamard(torch.float32)
    rot = s["U"] @ h                                           # [hk][2][d][d]
    q = s["q"].float().reshape(batch, hk, g, D)
    k, v = _plain_values(s["pool"], 4, s["group"])
    page = s["table"].long().clamp(min=0)
    most = page.shape[1] * PAGE
    k, v = (x[page].permute(0, 2, 1, 3, 4).reshape(batch, hk, most, D) for x in (k, v))
    lh = torch.matmul(torch.einsum("bhgd,hde->bhge", q, rot[:, 0]), k.transpose(2, 3)) / math.sqrt(D)
    lh = lh.masked_fill(torch.arange(most, device="cuda") >= s["hist"][:, None, None, None], -math.inf)
    kv = s["kv"].float().permute(0, 2, 3, 1, 4)                # [batch][hk][2][slots][d]
    lb = torch.matmul(q, kv[:, :, 0].transpose(2, 3)) / math.sqrt(D)
    lb = lb.masked_fill(torch.arange(NSLOT, device="cuda") >= s["len"][:, None, None, None], -math.inf)
    top = torch.maximum(lh.amax(-1, keepdim=True), lb.amax(-1, keepdim=True))
    ph, pb = torch.exp(lh - top), torch.exp(lb - top)
    o = torch.einsum("bhge,hde->bhgd", torch.matmul(ph, v), rot[:, 1]) + torch.matmul(pb, kv[:, :, 1])
    return (o / (ph.sum(-1, keepdim=True) + pb.sum(-1, keepdim=True))).reshape(batch, hq, D).to(s["out"].dtype)


def _plain_gather(s):
    pool, bits, ng = s["pool"], s["bits"], D // s["group"]
    b, i = (torch.arange(s["keep"].shape[1], device="cuda") < s["n_keep"][:, None]).nonzero(as_tuple=True)
    at = s["keep"][b, i].long()
    sp, ss = s["table"][b, at // PAGE].long(), at % PAGE
    dp, ds = s["dst_table"][b, i // PAGE].long(), i % PAGE
    pairs, code = _pairs_at(bits, s["group"]), 2048 if bits == 2 else 4096
    for a, n in ((0, code), (pairs[0], 256 * ng), (pairs[1], 256 * ng)):
        part = pool[:, :, a:a + n].unflatten(2, (PAGE, n // PAGE))
        part[dp, :, ds] = part[sp, :, ss]
    a = 2048 if bits == 2 else pairs[0] + 256 * ng
    part = pool[:, :, a:a + code].unflatten(2, (code // PAGE, PAGE)).transpose(2, 3)
    part[dp, :, ds] = part[sp, :, ss]
    return pool


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, hk = case["op"], case["hk"]
    ng = D // case["group"]
    stored = (2 * 32 if case.get("bits", 4) == 2 else 2 * 64) + 8 * ng   # bytes of a token and KV head, K and V
    if op == "evict":
        n = case["batch"] * case["per_seq"] * hk
        moved = n * (512 + stored) + hk * 2 * D * D * 4 + (n * 2 * 512 if case["append"] else 0)
        return {"bytes": moved + n * (stored + 512), "flops": n * 2 * (2 * D * D + 7 * D + 8 * D)}
    if op == "decode":
        n = case["batch"] * (case["lo"] + case["hi"]) / 2 * hk
        slots = case["batch"] * NSLOT * hk
        qo = case["batch"] * case["hq"] * D * (2 + (2 if case["bf16"] else 4))
        return {"bytes": n * stored + slots * 512 + qo + hk * 2 * D * D * 4, "flops": (n + slots) * (case["hq"] // hk) * 4 * D}
    if op == "read":
        n = case["tokens"] * hk
        return {"bytes": n * (stored + 2 * D * (2 if case["bf16"] else 4)), "flops": n * 2 * 2 * D}
    if op == "copy":
        return {"bytes": 2 * case["pages"] * case["pools"] * hk * _block(case["bits"], case["group"]), "flops": 0}
    n = case["batch"] * max(1, case["hist"] * case["keep"]) * hk
    return {"bytes": 2 * n * stored, "flops": 0}


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
    op = case["op"]
    if op in ("copy", "gather"):
        return None
    if op == "read":
        page, slot = s["table"][0].long()[s["pos"].long() // PAGE], s["pos"].long() % PAGE
        return torch.stack([torch.stack([_stored(s["pool"][:, h], page, slot, w, case["bits"], case["group"]) for w in (0, 1)], 1)
                            for h in range(case["hk"])], 1)
    if op == "evict":
        import numpy as np
        rows = s["kv"] if s["row"] is None else s["kv"][s["row"].long()]
        out = torch.empty(rows.shape, dtype=torch.float64, device="cuda")
        for h in range(case["hk"]):
            for w in (0, 1):
                y = (rows[:, h, w].double() @ _matrix(s["U"][h, w])).reshape(-1, case["group"])
                c = float(s["clip"][h, w])
                t = c * y.abs().max(1, keepdim=True).values if c < 1 else torch.full((y.shape[0], 1), math.inf, dtype=y.dtype, device=y.device)
                y = torch.where(y > t, t, torch.where(y < -t, -t, y))
                low, high = (f(y, 1).values for f in (torch.min, torch.max))
                scale, zero = (torch.from_numpy(a.cpu().numpy().astype(np.float16).astype(np.float64)).cuda()[:, None]
                               for a in ((high - low) / 15, low))
                u = torch.where(scale == 0, torch.zeros_like(y), (y - zero) / scale)
                down = torch.floor(u)
                code = down + ((u - down > 0.5) | ((u - down == 0.5) & (down % 2 == 1)))
                out[:, h, w] = (zero + scale * code.clamp(0, 15)).reshape(-1, D)
        kept = s["kv"].double()
        if s["new"] is not None:
            kept[s["row"].long()] = s["new"].double()
        return out, kept
    g = case["hq"] // case["hk"]
    out = torch.zeros(case["batch"], case["hq"], D, dtype=torch.float64, device="cuda")
    mats = [[_matrix(s["U"][h, w]) for w in (0, 1)] for h in range(case["hk"])]
    for b in range(case["batch"]):
        n, m = int(s["hist"][b]), int(s["len"][b])
        at = torch.arange(n, device="cuda")
        page, slot = s["table"][b].long()[at // PAGE], at % PAGE
        for h in range(case["hk"]):
            keys, vals = (torch.cat([_stored(s["pool"][:, h], page, slot, w, 4, case["group"]) @ mats[h][w].T, s["kv"][b, :m, h, w].double()])
                          for w in (0, 1))
            p = torch.softmax(s["q"][b, h * g:(h + 1) * g].double() @ keys.T / math.sqrt(D), -1)
            out[b, h * g:(h + 1) * g] = p @ vals
    return out
