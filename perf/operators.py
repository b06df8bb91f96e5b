"""Workloads of the decode-serving operators: rotary positions, the paged key-value cache's append,
attention of one new token per sequence over that cache, and the cache's page operations.

`run` computes a workload either with the library (`own` true) or in plain torch operations in 32
bits (64 for angles); `exact` restates it in 64 bits.  Sizes are the attention shape the library
benchmarks (32 query heads of 128, up to 8192 to 131072 cached tokens, grouped key-value heads)
and generic ones around it.

A cache is two planes [layers, pages, heads, page, d] (keys and values) of fp16, bf16 or E4M3 with
one UE8M0 scale per 32 elements ([..., d / 32] bytes, rows padded to 4 bytes).  A sequence's tokens
lie in the pages its row of the table names.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32
DEV = "cuda"


def listed():
    return [
        # one decode step's queries and keys of 8 sequences (32 + 8 heads): latency
        rope_case(8, 40, 128, 128, "f16", False, "none", False, name="rope_decode_8"),
        # a long-context prefill chunk, interleaved pairs, frequencies scaled by parts
        rope_case(8192, 40, 128, 128, "bf16", True, "by_parts", False, name="rope_prefill_8192"),
        # backward of a rotation over part of an odd head, odd token count
        rope_case(30011, 12, 96, 48, "f16", False, "linear", True, name="rope_inverse_odd"),
        # one decode step's append to a quantised cache: latency
        append_case(64, 1, 32, 8, 128, 64, "f16", True, True, "none", name="append_decode_e4m3"),
        # a prefill chunk of 8 sequences into a 16-bit cache, interleaved pairs
        append_case(8, 2048, 32, 8, 128, 64, "bf16", False, True, "by_parts", name="append_prefill_bf16"),
        # a prefill chunk of odd length into a quantised cache, pages that end inside it
        append_case(3, 5003, 28, 4, 128, 24, "f16", True, False, "linear", name="append_prefill_e4m3_odd"),
        # one user, short context: latency
        attend_case(1, 32, 8, 128, 700, False, 16, "f16", False, 0, name="attend_1x700"),
        # a serving batch with lengths from empty to 8192, small pages
        attend_case(64, 32, 8, 128, 8192, True, 16, "f16", False, 0, name="attend_ragged_64x8192"),
        # a few users with very long contexts: the split over the cache's length
        attend_case(4, 32, 8, 128, 131072, False, 128, "bf16", False, 0, name="attend_long_4x131072"),
        # a large batch over a block-scaled 8-bit cache
        attend_case(128, 64, 8, 128, 8192, True, 64, "f16", True, 0, name="attend_e4m3_128x8192"),
        # a beam step: 8 hypotheses from 2, pages of 16 tokens in 32 layers
        fork_case(32, 512, 8, 16, 128, "f16", False, 16, 8, 600, name="fork_beam_8"),
        # compaction after many sequences ended: a third of the pages move
        compact_case(8, 1024, 8, 64, 128, "f16", True, 48, 16, 4, 256, name="compact_256_pages"),
    ]


def rope_case(tokens, heads, d, rot, dtype, interleaved, scaling, inverse, **more):
    return dict(more, op="rope", tokens=tokens, heads=heads, d=d, rot=rot, dtype=dtype, interleaved=interleaved,
                scaling=scaling, inverse=inverse)


def append_case(seqs, new, hq, hkv, d, page, dtype, e4m3, interleaved, scaling, **more):
    """`new` tokens for each of `seqs` sequences, which hold earlier ones already."""
    return dict(more, op="append", seqs=seqs, new=new, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, e4m3=e4m3,
                interleaved=interleaved, scaling=scaling)


def attend_case(batch, hq, hkv, d, length, ragged, page, dtype, e4m3, window, **more):
    return dict(more, op="attend", batch=batch, hq=hq, hkv=hkv, d=d, length=length, ragged=ragged, page=page, dtype=dtype,
                e4m3=e4m3, window=window)


def fork_case(layers, pages, heads, page, d, dtype, e4m3, slots, children, length, **more):
    """`children` sequences become copies of the first quarter of them; `length`: the parents' tokens."""
    return dict(more, op="fork", layers=layers, pages=pages, heads=heads, page=page, d=d, dtype=dtype, e4m3=e4m3,
                slots=slots, children=children, length=length)


def compact_case(layers, pages, heads, page, d, dtype, e4m3, slots, each, shared, moved, **more):
    """`slots` sequences of `each` pages, the first `shared` of them common to all; `moved` pages lie too high."""
    return dict(more, op="compact", layers=layers, pages=pages, heads=heads, page=page, d=d, dtype=dtype, e4m3=e4m3,
                slots=slots, each=each, shared=shared, moved=moved)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "append", "attend", "attend", "fork", "compact"])
    dtype = rng.choice(["f16", "bf16"])
    scaling = rng.choice(["none", "linear", "by_parts"])
    flip = rng.random() < 0.5
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 256])
        return rope_case(log(1, 16384), rng.randint(1, 48), d, rng.choice([d, d // 2, 2 * (d // 5)]), dtype, flip, scaling,
                         rng.random() < 0.3)
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 24, 32, 64, 100, 128])
    e4m3 = rng.random() < 0.5
    if op == "append":
        seqs = log(1, 128)
        return append_case(seqs, 1 if flip else log(1, max(1, 16384 // seqs)), hq, hkv, d, page, dtype, e4m3,
                           rng.random() < 0.5, scaling)
    if op == "attend":
        batch = log(1, 128)
        length = log(1, min(131072, 4 * 2 ** 20 // (batch * hkv)))
        return attend_case(batch, hq, hkv, d, length, batch > 2 and rng.random() < 0.7, page, dtype, e4m3,
                           0 if rng.random() < 0.7 else log(1, length + 1))
    layers = log(2, 16)
    if op == "fork":
        children = log(1, 32)
        length = log(1, 100) * page + rng.randint(0, page - 1)
        pages = children * (-(-length // page) + 2) + rng.randint(0, 64)
        return fork_case(fitting(layers, pages * page * hkv * d), pages, hkv, page, d, dtype, e4m3, 2 * children, children, length)
    slots, each = log(2, 32), log(2, 16)
    shared = rng.randint(0, each - 1)
    used = slots * each - (slots - 1) * shared
    moved = rng.randint(1, used)
    pages = used + moved + rng.randint(0, 64)
    return compact_case(fitting(layers, pages * page * hkv * d), pages, hkv, page, d, dtype, e4m3, slots, each, shared, moved)


def fitting(layers, plane):
    """At most `layers` layers of `plane` values: a plane of at most 2^29 in all."""
    return max(1, min(layers, 2 ** 29 // plane))


# ------------------------------------------------------------------------------- sizes of a case

def lengths(c):
    """The tokens each sequence holds: all `length`, or from none, one and two up to it, most of them short."""
    if not c["ragged"]:
        return [c["length"]] * c["batch"]
    n = c["batch"]
    got = [int(c["length"] * ((i + 1) / n) ** 2) for i in range(n)]
    return [min(i, got[i]) for i in range(min(3, n - 1))] + got[min(3, n - 1):]


def fork_lengths(c):
    return [max(1, c["length"] - 3 * i) for i in range(parents_of(c))]


def parents_of(c):
    return max(1, c["children"] // 4)


def token_bytes(c):
    """Bytes of one token of one head in one layer: a key and a value."""
    return 2 * (c["d"] + c["d"] // BLOCK if c["e4m3"] else 2 * c["d"])


def work(c):
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"]
        return {"bytes": 2 * n * c["d"] * 2 + 4 * c["tokens"], "flops": 3 * n * c["rot"]}
    if c["op"] == "append":
        t = c["seqs"] * c["new"]
        return {"bytes": t * ((2 * c["hq"] + 2 * c["hkv"]) * c["d"] * 2 + c["hkv"] * token_bytes(c) + 12),
                "flops": 3 * t * (c["hq"] + c["hkv"]) * c["d"]}
    if c["op"] == "attend":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in lengths(c))
        pages = sum(-(-n // c["page"]) for n in lengths(c))
        return {"bytes": seen * c["hkv"] * token_bytes(c) + 4 * pages + c["batch"] * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * seen * c["hq"] * c["d"]}
    if c["op"] == "fork":
        lens = fork_lengths(c)
        lens = [lens[i % len(lens)] for i in range(c["children"])]
        tails = sum(n % c["page"] for n in lens)
        return {"bytes": 2 * tails * c["layers"] * c["heads"] * token_bytes(c) + sum(12 * (n // c["page"]) for n in lens) + 16 * len(lens),
                "flops": 0}
    return {"bytes": 2 * c["moved"] * c["page"] * c["layers"] * c["heads"] * token_bytes(c) + 8 * c["slots"] * c["each"] + 4 * c["pages"],
            "flops": 0}


# ------------------------------------------------------------------------------------ inputs

def quantised(x):
    """(codes, scale bytes) of x with one power of two per 32 elements, in 32 bits; small inputs' blocks stop at 2^-15."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - 8, torch.zeros_like(amax, dtype=torch.int32))
    e = e.clamp(-15 if x.dtype == torch.float16 else -127, 127)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


def padded(s):
    """Scale rows in their 4 bytes."""
    room = torch.zeros(*s.shape[:-1], 4 * -(-s.shape[-1] // 4), dtype=torch.uint8, device=s.device)
    room[..., :s.shape[-1]] = s
    return room


def cache_of(c, layers, pages, heads, g):
    """The planes of a cache full of earlier tokens: keys of larger norm than values, a few strong channels."""
    shape = (layers, pages, heads, c["page"], c["d"])
    strong = 1 + 3 * (torch.rand(heads, 1, c["d"], generator=g, device=DEV) < 0.03).float()
    planes = {}
    for name, size in (("k", 1.0), ("v", 0.5)):
        x = torch.randn(shape, generator=g, device=DEV, dtype=TYPES[c["dtype"]])
        x *= (size * strong).to(x.dtype)
        if c["e4m3"]:
            codes, s = zip(*(quantised(x[i]) for i in range(layers)))
            planes[name], planes[name + "s"] = torch.stack(codes), padded(torch.stack(s))
        else:
            planes[name] = x
    return planes


def handle(s):
    """The library's view of the planes (made once, as a program does)."""
    import block_scaled_quantized_tcgen05_gb300 as q
    return q.qgemm_create_kv_cache(s["k"], s["v"], s.get("ks"), s.get("vs"))


def table_of(lens, slots, most, pages, page, g):
    """A table whose sequences lie in pages of a random order."""
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((slots, most), -1, dtype=torch.int32)
    at = 0
    order = order.cpu()
    for i, n in enumerate(lens):
        k = -(-n // page)
        table[i, :k] = order[at:at + k]
        at += k
    return table.to(DEV)


def frequencies(rot, scaling, dtype=torch.float64):
    """Radians a position turns each pair, in 64 bits."""
    w = 10000.0 ** (-torch.arange(0, rot, 2, dtype=dtype, device=DEV) / rot)
    if scaling == "linear":
        w = w / FACTOR
    if scaling == "by_parts":
        turns = ORIGINAL * w / (2 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        w = w * (keep + (1 - keep) / FACTOR)
    return w


FACTOR, ORIGINAL, LOW, HIGH, MSCALE = 8.0, 8192, 1.0, 4.0, 1.2


def rotation(c, rot):
    if not own:
        return None
    import block_scaled_quantized_tcgen05_gb300 as q
    if c["scaling"] == "none":
        return q.qgemm_create_rope(rot, interleaved=c["interleaved"])
    if c["scaling"] == "linear":
        return q.qgemm_create_rope(rot, interleaved=c["interleaved"], scaling="linear", factor=FACTOR)
    return q.qgemm_create_rope(rot, interleaved=c["interleaved"], scaling="by_parts", factor=FACTOR, original_len=ORIGINAL,
                               low_turns=LOW, high_turns=HIGH, mscale=MSCALE)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"rope": prepare_rope, "append": prepare_append, "attend": prepare_attend, "fork": prepare_fork,
            "compact": prepare_compact}[c["op"]](dict(c), g)


def prepare_rope(c, g):
    x = torch.randn(c["tokens"], c["heads"], c["d"], generator=g, device=DEV, dtype=TYPES[c["dtype"]])
    start = torch.randint(0, 120000, (1,), generator=g, device=DEV, dtype=torch.int32)
    pos = start + torch.arange(c["tokens"], dtype=torch.int32, device=DEV)
    return {"c": c, "x": x, "pos": pos, "y": torch.empty_like(x), "rope": rotation(c, c["rot"]), "rot": c["rot"]}


def prepare_append(c, g):
    dt, t = TYPES[c["dtype"]], c["seqs"] * c["new"]
    before = [(37 * i + 11) % 300 for i in range(c["seqs"])]
    lens = [n + c["new"] for n in before]
    most = max(-(-n // c["page"]) for n in lens)
    pages = sum(-(-n // c["page"]) for n in lens) + 3
    s = {"c": c, "rot": c["d"], **cache_of(c, 2, pages, c["hkv"], g)}
    s["table"] = table_of(lens, c["seqs"], most, pages, c["page"], g)
    s["seqs"] = torch.arange(c["seqs"], dtype=torch.int32, device=DEV).repeat_interleave(c["new"])
    first = torch.tensor(before, dtype=torch.int32, device=DEV).repeat_interleave(c["new"])
    s["pos"] = first + torch.arange(c["new"], dtype=torch.int32, device=DEV).repeat(c["seqs"])
    qkv = torch.randn(t, c["hq"] + 2 * c["hkv"], c["d"], generator=g, device=DEV, dtype=dt)  # as a fused projection leaves it
    s["q"], s["kn"], s["vn"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
    s["qo"] = torch.empty(t, c["hq"], c["d"], dtype=dt, device=DEV)
    s["rope"] = rotation(c, c["d"])
    if own:
        s["kv"] = handle(s)
    return s


def prepare_attend(c, g):
    lens = lengths(c)
    order = torch.randperm(len(lens), generator=torch.Generator().manual_seed(g.initial_seed())).tolist()
    lens = [lens[i] for i in order]
    pages = sum(-(-n // c["page"]) for n in lens) + 3
    s = {"c": c, **cache_of(c, 1, pages, c["hkv"], g)}
    most = max(1, max(-(-n // c["page"]) for n in lens))
    s["table"] = table_of(lens, len(lens), most, pages, c["page"], g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["q"] = 1.5 * torch.randn(c["batch"], c["hq"], c["d"], generator=g, device=DEV, dtype=TYPES[c["dtype"]])
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(c["batch"], c["hq"], dtype=torch.float32, device=DEV)
    if own:
        import block_scaled_quantized_tcgen05_gb300 as q
        s["kv"] = handle(s)
        s["workspace"] = q.qgemm_paged_attention_workspace(s["kv"], c["batch"], c["hq"])
    return s


def meta_of(slots, most, pages, dev=DEV):
    """One buffer with the table, the lengths and the pages' reference counts, and its three parts."""
    meta = torch.zeros(slots * most + slots + pages, dtype=torch.int32, device=dev)
    table, lens, refs = meta.split([slots * most, slots, pages])
    table.fill_(-1)
    return meta, table.view(slots, most), lens, refs


def prepare_fork(c, g):
    s = {"c": c, **cache_of(c, c["layers"], c["pages"], c["heads"], g)}
    plens, n, p = fork_lengths(c), c["children"], parents_of(c)
    most = -(-c["length"] // c["page"])
    s["meta"], s["table"], s["lens"], s["refs"] = meta_of(c["slots"], most, c["pages"])
    slot = torch.randperm(c["slots"], generator=g, device=DEV).to(torch.int32)
    held = table_of(plens, p, most, c["pages"], c["page"], g)
    s["table"][slot[:p].long()] = held
    s["lens"][slot[:p].long()] = torch.tensor(plens, dtype=torch.int32, device=DEV)
    s["refs"][held[held >= 0].long()] = 1
    if p + n > c["slots"]:
        raise ValueError("slots")
    s["parents"] = slot[:p].repeat(-(-n // p))[:n].contiguous()
    s["children"] = slot[p:p + n].contiguous()
    if own:
        s["kv"] = handle(s)
    return s


def prepare_compact(c, g):
    s = {"c": c, **cache_of(c, c["layers"], c["pages"], c["heads"], g)}
    n, each, shared, moved = c["slots"], c["each"], c["shared"], c["moved"]
    used = n * each - (n - 1) * shared
    low = torch.randperm(used, generator=g, device=DEV)[:used - moved]
    high = used + torch.randperm(c["pages"] - used, generator=g, device=DEV)[:moved]
    pages = torch.cat([low, high])
    pages = pages[torch.randperm(used, generator=g, device=DEV)].to(torch.int32)
    meta0, table, lens, refs = meta_of(n, each, c["pages"])
    table[:, :shared] = pages[:shared]
    table[:, shared:] = pages[shared:].view(n, each - shared)
    lens.copy_(each * c["page"] - torch.randint(0, c["page"], (n,), generator=g, device=DEV, dtype=torch.int32))
    refs[pages[:shared].long()] = n
    refs[pages[shared:].long()] = 1
    s["meta0"] = meta0.clone()
    s["meta"], s["table"], s["lens"], s["refs"] = meta0, table, lens, refs
    if own:
        s["kv"] = handle(s)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["c"]["op"]
    if own:
        return {"rope": own_rope, "append": own_append, "attend": own_attend, "fork": own_fork, "compact": own_compact}[op](s)
    return {"rope": plain_rope, "append": plain_append, "attend": plain_attend, "fork": plain_fork, "compact": plain_compact}[op](s)


def planes(s):
    """The cache as the values it stands for: 8-bit planes and their scales as the numbers they are."""
    if "ks" in s:
        n = s["c"]["d"] // BLOCK
        return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
                "ks": s["ks"][..., :n].view(torch.float8_e8m0fnu), "vs": s["vs"][..., :n].view(torch.float8_e8m0fnu)}
    return {"k": s["k"], "v": s["v"]}


def own_rope(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    return q.qgemm_rope(s["x"], s["pos"], s["rope"], out=s["y"], inverse=s["c"]["inverse"])


def own_append(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    q.qgemm_kv_append(s["kv"], 1, s["kn"], s["vn"], s["seqs"], s["pos"], s["table"], rope=s["rope"], Q=s["q"], Q_out=s["qo"])
    return dict(planes(s), q=s["qo"])


def own_attend(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    q.qgemm_paged_attention(s["q"], s["kv"], 0, s["table"], s["lens"], s["o"], lse=s["lse"], window=s["c"]["window"],
                            workspace=s["workspace"])
    return {"o": s["o"], "lse": s["lse"]}


def own_fork(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    q.qgemm_kv_fork(s["kv"], s["table"], s["lens"], s["refs"], s["parents"], s["children"])
    return dict(planes(s), table=s["table"], lens=s["lens"], refs=s["refs"])


def own_compact(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    s["meta"].copy_(s["meta0"])  # the pages lie as before compaction again
    q.qgemm_kv_compact(s["kv"], s["table"], s["lens"], s["refs"])
    return dict(planes(s), table=s["table"], lens=s["lens"], refs=s["refs"])


def rotated(x, pos, rot, interleaved, scaling, inverse=False):
    """x [tokens, heads, d] turned by its positions, in 32 bits (the angles in 64)."""
    angle = pos.double()[:, None] * frequencies(rot, scaling)
    m = MSCALE if scaling == "by_parts" else 1.0
    cos, sin = (m * angle.cos()).float()[:, None], (m * angle.sin()).float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def plain_rope(s):
    c = s["c"]
    s["y"].copy_(rotated(s["x"], s["pos"], c["rot"], c["interleaved"], c["scaling"], c["inverse"]))
    return s["y"]


def plain_append(s):
    c = s["c"]
    s["qo"].copy_(rotated(s["q"], s["pos"], s["rot"], c["interleaved"], c["scaling"]))
    k = rotated(s["kn"], s["pos"], s["rot"], c["interleaved"], c["scaling"])
    pos = s["pos"].long()
    page, off = s["table"][s["seqs"].long(), pos // c["page"]].long(), pos % c["page"]
    for name, x in (("k", k), ("v", s["vn"])):
        if c["e4m3"]:
            b = x.float().unflatten(-1, (-1, BLOCK))
            amax = b.abs().amax(-1, keepdim=True)
            e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, 0).clamp(-15 if c["dtype"] == "f16" else -127, 127)
            s[name][1, page, :, off] = torch.ldexp(b, -e).clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "s"][1, page, :, off, :c["d"] // BLOCK] = (e + 127).squeeze(-1).to(torch.uint8)
        else:
            s[name][1, page, :, off] = x.to(s[name].dtype)
    return dict(planes(s), q=s["qo"])


def plain_attend(s):
    c = s["c"]
    g, d = c["hq"] // c["hkv"], c["d"]
    at = s["table"].clamp(min=0).long()
    token = torch.arange(at.shape[1] * c["page"], device=DEV)
    n = s["lens"][:, None]
    seen = token < n
    if c["window"]:
        seen &= token >= n - c["window"]
    kv = []
    for name in ("k", "v"):
        x = s[name][0][at]  # [batch, pages, heads, page, d]
        if c["e4m3"]:
            scale = s[name + "s"][0][at][..., :d // BLOCK, None]
            x = x.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLOCK)) * torch.exp2(scale.float() - 127)
            x = x.flatten(-2)
        kv.append(x.float().transpose(2, 3).flatten(1, 2).transpose(1, 2).masked_fill(~seen[:, None, :, None], 0))
    q = s["q"].float().unflatten(1, (c["hkv"], g))
    score = (q @ kv[0].transpose(-1, -2) * d ** -0.5).masked_fill(~seen[:, None, None], -math.inf)
    most = score.amax(-1, keepdim=True)
    p = torch.exp(score - most.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    s["o"].copy_((p @ kv[1] / total.clamp(min=1e-30)).flatten(1, 2))
    s["lse"].copy_((torch.log(total) + most).flatten(1))
    return {"o": s["o"], "lse": s["lse"]}


def plain_fork(s):
    c, table, lens, refs = s["c"], s["table"], s["lens"], s["refs"]
    parents, children = s["parents"].long(), s["children"].long()
    column = torch.arange(table.shape[1], device=DEV)
    # the children's slots give back what they hold
    held = column < -(-lens[children] // c["page"])[:, None]
    refs.index_add_(0, table[children].clamp(min=0).flatten().long(), -held.flatten().int())
    # whole pages are shared, a page that ends early is copied into the lowest free ones in the children's order
    n = lens[parents]
    full, tail = n // c["page"], n % c["page"]
    share = column < full[:, None]
    rows = table[parents]
    free = torch.sort((refs > 0).int(), stable=True)[1][:len(parents)]
    need = (tail > 0).int()
    place = torch.where(tail > 0, need.cumsum(0) - 1, need.sum() + (1 - need).cumsum(0) - 1)
    new = free[place]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), share.flatten().int())
    refs.index_add_(0, new, need)
    source = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0].clamp(min=0).long()
    early = torch.arange(c["page"], device=DEV) < tail[:, None]
    for name in ("k", "v", "ks", "vs"):
        if name in s:
            s[name][:, new] = torch.where(early[None, :, None, :, None], s[name][:, source], s[name][:, new])
    row = torch.where(share, rows, -1)
    table[children] = torch.where((column == full[:, None]) & (tail > 0)[:, None], new[:, None].int(), row)
    lens[children] = n
    return dict(planes(s), table=table, lens=lens, refs=refs)


def plain_compact(s):
    s["meta"].copy_(s["meta0"])
    c, table, lens, refs = s["c"], s["table"], s["lens"], s["refs"]
    used = refs > 0
    index = torch.arange(len(refs), device=DEV)
    high = index >= used.sum()
    source, target = torch.nonzero(used & high)[:, 0], torch.nonzero(~used & ~high)[:, 0]
    moved = index.int().index_copy(0, source, target.int())
    held = torch.arange(table.shape[1], device=DEV) < -(-lens // c["page"])[:, None]
    table.copy_(torch.where(held, moved[table.clamp(min=0).long()], table))
    refs[target] = refs[source]
    refs[source] = 0
    for name in ("k", "v", "ks", "vs"):
        if name in s:
            s[name][:, target] = s[name][:, source]
    return dict(planes(s), table=table, lens=lens, refs=refs)


# ------------------------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    return {"rope": exact_rope, "append": exact_append, "attend": exact_attend, "fork": exact_pages,
            "compact": exact_pages}[c["op"]](c, prepare(c, seed))


def turn(x, pos, rot, interleaved, scaling, sign):
    """Rotation as a product of complex numbers."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    w = torch.exp(-2 * i / rot * math.log(10000.0))
    size = 1.0
    if scaling == "linear":
        w = w / 8
    elif scaling == "by_parts":
        rounds = 8192 / (2 * math.pi / w)
        part = (rounds - 1) / 3
        w = torch.where(part <= 0, w / 8, torch.where(part >= 1, w, part * w + (1 - part) * w / 8))
        size = 1.2
    z = torch.polar(torch.full((len(pos), 1, rot // 2), size, dtype=torch.float64, device=DEV),
                    sign * (pos.double()[:, None] * w)[:, None])
    x = x.double()
    if interleaved:
        y = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    else:
        y = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * z
        y = torch.cat([y.real, y.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def exact_rope(c, s):
    return turn(s["x"], s["pos"], c["rot"], c["interleaved"], c["scaling"], -1 if c["inverse"] else 1)


def wide(s):
    return {name: x.double() for name, x in planes(s).items()}


def exact_append(c, s):
    q, k = (turn(s[x], s["pos"], c["d"], c["interleaved"], c["scaling"], 1) for x in ("q", "kn"))
    got = dict(wide(s), q=q)
    pos = s["pos"].tolist()
    table = s["table"].tolist()
    at = torch.tensor([[table[b][p // c["page"]], p % c["page"]] for b, p in zip(s["seqs"].tolist(), pos)], device=DEV)
    for name, x in (("k", k), ("v", s["vn"].double())):
        if not c["e4m3"]:
            got[name][1][at[:, 0], :, at[:, 1]] = x
            continue
        blocks = x.reshape(*x.shape[:-1], c["d"] // BLOCK, BLOCK)
        top = blocks.abs().max(-1)[0]
        e = torch.floor(torch.log2(torch.where(top > 0, top, 256.0))) - 8
        e = e.clamp(min=-15.0 if c["dtype"] == "f16" else -127.0)
        unit = torch.exp2(e)[..., None]
        r = (blocks / unit).clamp(-448, 448)
        step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
        got[name][1][at[:, 0], :, at[:, 1]] = (torch.round(r / step) * step).reshape(x.shape)
        got[name + "s"][1][at[:, 0], :, at[:, 1]] = torch.exp2(e)
    return got


def exact_attend(c, s):
    d, g = c["d"], c["hq"] // c["hkv"]
    o = torch.zeros(c["batch"], c["hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((c["batch"], c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        rows = s["table"][b, lo // c["page"]:-(-n // c["page"])].long()
        first = lo // c["page"] * c["page"]
        kv = []
        for name in ("k", "v"):
            x = s[name][0, rows]
            if c["e4m3"]:
                x = x.view(torch.float8_e4m3fn).double()
                x = x * torch.exp2(s[name + "s"][0, rows][..., :d // BLOCK].double() - 127).repeat_interleave(BLOCK, -1)
            x = x.double().permute(1, 0, 2, 3).reshape(c["hkv"], -1, d)
            kv.append(x[:, lo - first:n - first])
        z = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(c["hkv"], g, d), kv[0]) / math.sqrt(d)
        lse[b] = torch.logsumexp(z, -1).view(-1)
        o[b] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), kv[1]).view(c["hq"], d)
    return {"o": o, "lse": lse}


def exact_pages(c, s):
    """The page operations, sequence by sequence on the host."""
    data = planes(s)
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    size = c["page"]
    pairs = []
    if c["op"] == "fork":
        children, parents = s["children"].tolist(), s["parents"].tolist()
        for ch in children:
            for j in range(-(-lens[ch] // size)):
                refs[table[ch][j]] -= 1
        for ch, p in zip(children, parents):
            full, tail = divmod(lens[p], size)
            row = [-1] * len(table[ch])
            row[:full] = table[p][:full]
            for page in row[:full]:
                refs[page] += 1
            if tail:
                row[full] = refs.index(0)
                refs[row[full]] = 1
                pairs.append((table[p][full], row[full], tail))
            table[ch], lens[ch] = row, lens[p]
    else:
        count = sum(r > 0 for r in refs)
        for page in range(count, len(refs)):
            if refs[page]:
                to = refs.index(0)
                refs[to], refs[page] = refs[page], 0
                pairs.append((page, to, size))
                for row in table:
                    row[:] = [to if x == page else x for x in row]
    got = {}
    for name, x in data.items():
        y = x.view(torch.uint8) if name in ("k", "v") and "ks" in data or name in ("ks", "vs") else x
        y = y.clone()
        for a, b, n in pairs:
            y[:, b, :, :n] = y[:, a, :, :n]
        got[name] = (y.view(x.dtype) if y.dtype != x.dtype else y).double()
    return dict(got, table=torch.tensor(table, dtype=torch.int32), lens=torch.tensor(lens, dtype=torch.int32),
                refs=torch.tensor(refs, dtype=torch.int32))
