"""Cases of what stands around the 4-bit key/value cache's attention when a decoder serves many requests: norms and
rotation of queries and keys on their way into the cache, attention of sequences that share a prefix, and low-rank
adapters beside a projection.

"rotate": rows of a fused QKV product; each head of q and k is normed (or not) and rotated by its token's position
(one axis, or several for images and video), q goes to 16 bits, k and v to 4 bits in the cache, from which they are
read back.  "shared": runs of sequences whose first pages are the same; otherwise causal attention over the cache.
"adapt": y + scale * B (A x) for segments of rows, each with an adapter of its own or none.

A page of the cache holds 64 tokens; a block is one head of one page: the codes of K and of V (nibble = code + 8),
then the fp32 scales of both.
"""
import math

import torch

own = False

PAGE = 64
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _rotate(name, dtype, batch, rows, kv, q_heads, kv_heads, dim, group, rot, norm, paired, axes=1, cycle=False,
            ragged=False):
    c = dict(op="rotate", dtype=dtype, batch=batch, rows=rows, kv=kv, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
             group=group, rot=rot, norm=norm, paired=paired, axes=axes, cycle=cycle, ragged=ragged)
    return {**c, "name": name} if name else c


def _shared(name, dtype, batch, groups, prefix, rows, tail, q_heads, kv_heads, dim, group, ragged=False):
    c = dict(op="shared", dtype=dtype, batch=batch, groups=groups, prefix=prefix, rows=rows, tail=tail,
             q_heads=q_heads, kv_heads=kv_heads, dim=dim, group=group, ragged=ragged)
    return {**c, "name": name} if name else c


def _adapt(name, dtype, segments, rows, slots, rank, inputs, ends, ragged=False):
    c = dict(op="adapt", dtype=dtype, segments=segments, rows=rows, slots=slots, rank=rank, inputs=inputs, ends=ends,
             ragged=ragged)
    return {**c, "name": name} if name else c


def listed():
    return [
        # One token of one conversation, 32 query and 8 key/value heads of 128, rotated whole.  All latency.
        _rotate("rotate_one_token", "f16", 1, 1, 1001, 32, 8, 128, 64, 128, False, False),
        # The ordinary serving step of a model with q and k norms: a token of each of 64 conversations.
        _rotate("rotate_batch", "bf16", 64, 1, 8192, 32, 8, 128, 64, 128, True, False, ragged=True),
        # Prompts of different lengths entering the cache at once, with norms.
        _rotate("rotate_prompts", "bf16", 6, 4096, 4096, 32, 8, 128, 128, 128, True, False, ragged=True),
        # A prompt with a video: time, height and width by turns over the pairs, small heads, a part of them rotated,
        # neighbouring elements as pairs.
        _rotate("rotate_video", "f16", 1, 5003, 6003, 28, 4, 64, 64, 48, True, True, 3, True),
        # Samples of one short question: few columns, latency.
        _shared("shared_samples", "f16", 4, 1, 1000, 1, 131, 32, 8, 128, 64),
        # The ordinary step of 64 conversations behind one system prompt, one of them a padded slot.
        _shared("shared_batch", "bf16", 64, 1, 8192, 1, 1024, 32, 8, 128, 64, ragged=True),
        # Three system prompts of one length or another, a few drafted tokens each, small heads.
        _shared("shared_drafts", "f16", 30, 3, 6000, 4, 700, 28, 4, 64, 64, ragged=True),
        # Questions about one long document: their prompts over it.
        _shared("shared_document", "bf16", 16, 1, 65536, 64, 64, 32, 8, 128, 128),
        # One token with an adapter beside the O product.
        _adapt("adapt_one_token", "f16", 1, 1, 8, 16, 4096, "4096"),
        # The ordinary step: 64 conversations with 24 adapters among them, beside the fused QKV product.
        _adapt("adapt_batch", "bf16", 64, 1, 24, 16, 4096, "4096,5120,6144"),
        # Prompts of different lengths beside QKV.
        _adapt("adapt_prompts", "bf16", 6, 2048, 8, 16, 4096, "4096,5120,6144", ragged=True),
        # A chunk of a prompt beside the fused gate and up product, at a high rank.
        _adapt("adapt_chunk", "f16", 1, 2000, 4, 64, 4096, "12288,24576"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotate", "shared", "adapt"])
    dtype = rng.choice(["f16", "bf16"])
    ragged = rng.random() < 0.6
    if op == "adapt":
        inputs = 64 * _spread(rng, 8, 192)
        slices = rng.choice([1, 1, 2, 3])
        ends = [64 * _spread(rng, 4, 128)]
        for _ in range(slices - 1):
            ends.append(ends[-1] + 64 * _spread(rng, 4, 64))
        rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
        if rng.random() < 0.5:
            segments, rows = _spread(rng, 1, 128), rng.choice([1, 1, 2, 5])
        else:
            segments = _spread(rng, 1, 8)
            rows = _spread(rng, 9, 4096 // segments)
        return _adapt(None, dtype, segments, rows, _spread(rng, 1, 32), rank, inputs, ",".join(map(str, ends)),
                      ragged and segments > 1)
    dim = rng.choice([64, 128, 128])
    group = 64 if dim == 64 else rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    if op == "rotate":
        batch = _spread(rng, 1, 32)
        rows = _spread(rng, 1, 8192 // batch)
        kv = rows if rng.random() < 0.5 else rows + _spread(rng, 1, 4000)
        axes = rng.choice([1, 1, 2, 3])
        rot = dim if rng.random() < 0.6 else 16 * rng.randint(1, dim // 16)
        return _rotate(None, dtype, batch, rows, kv, q_heads, kv_heads, dim, group, rot, rng.random() < 0.6,
                       rng.random() < 0.4, axes, rng.random() < 0.5, ragged and batch > 1)
    batch = _spread(rng, 2, 64)
    rows = rng.choice([1, 1, 1, 2, 5]) if rng.random() < 0.7 else _spread(rng, 1, 1024 // batch)
    tail = rows + _spread(rng, 1, 1500)
    prefix = _spread(rng, 64, min(65536, 300000 // batch))
    return _shared(None, dtype, batch, min(batch, rng.choice([1, 1, 2, 3])), prefix, rows, tail, q_heads, kv_heads,
                   dim, group, ragged)


def _part(b):
    return 1.0 - 0.85 * ((b * 0.6180339887) % 1.0)


def _lengths(case):
    """(rows, cached tokens) of each sequence.  Ragged batches spread both; their third sequence is a slot that the
    program padded its batch with: one row, nothing cached."""
    out = []
    for b in range(case["batch"]):
        n, part = case["rows"], _part(b) if case["ragged"] else 1.0
        if n > 8:
            n = max(1, int(n * part))
        if case["op"] == "rotate":
            kv = n + int((case["kv"] - case["rows"]) * part)
        else:
            kv = _prefix(case, _group(case, b)) + n + int((case["tail"] - case["rows"]) * part)
        out.append((1, 0) if case["ragged"] and b == 2 else (n, kv))
    return out


def _group(case, b):
    return b * case["groups"] // case["batch"]


def _prefix(case, g):
    return case["prefix"] if not case["ragged"] else max(1, case["prefix"] - g * case["prefix"] // 4)


def _rows_of_segments(case):
    return [max(1, int(case["rows"] * _part(b))) if case["ragged"] else case["rows"] for b in range(case["segments"])]


def _slots_of_segments(case):
    """Every seventh segment has no adapter; the others take the slots by turns, some more often."""
    return [-1 if b % 7 == 6 else (b * b + b // 2) % case["slots"] for b in range(case["segments"])]


def _ends(case):
    return [int(e) for e in case["ends"].split(",")]


def work(case):
    if case["op"] == "adapt":
        n, k, r, slices = _ends(case)[-1], case["inputs"], case["rank"], len(_ends(case))
        rows, slots = _rows_of_segments(case), _slots_of_segments(case)
        used = sum(m for m, s in zip(rows, slots) if s >= 0)
        weights = r * (slices * k + n) * len({s for s in slots if s >= 0})
        return {"bytes": 2 * (used * k + 2 * sum(rows) * n + weights), "flops": 2 * used * r * (slices * k + n)}
    dim, hk, hq = case["dim"], case["kv_heads"], case["q_heads"]
    lens = _lengths(case)
    rows = sum(n for n, _ in lens)
    stored = dim + 8 * (dim // case["group"])  # one token's K and V of one head in the cache
    if case["op"] == "rotate":
        # q, k, v and the table's entries in, q and the codes out, k and v back in 16 bits
        there = sum(min(n, kv) for n, kv in lens)
        return {"bytes": there * (4 * hq * dim + hk * (2 * stored + 8 * dim) + 4 * case["rot"]),
                "flops": there * (hq + 2 * hk) * dim * 10}
    # every page of a prefix once, every token behind it once
    whole = [_prefix(case, g) // PAGE * PAGE for g in range(case["groups"])]
    tokens = sum(whole) + sum(max(0, kv - whole[_group(case, b)]) for b, (_, kv) in enumerate(lens))
    pairs = sum(n * kv - n * (n - 1) // 2 for n, kv in lens if kv)
    return {"bytes": tokens * hk * stored + 4 * rows * hq * dim, "flops": 4 * dim * hq * pairs}


# ---------------------------------------------------------------- inputs

def _quantise(x, group):
    """(codes -8 .. 7, fp32 scales) of fp32 rows [..., dim]: scale = max|x| / 7 of each group, code = rint(x / scale)."""
    g = x.float().unflatten(-1, (-1, group))
    top = g.abs().amax(-1)
    s = top / torch.full_like(top, 7)  # a tensor's division rounds correctly; a number's may be a product
    q = torch.where(s[..., None] == 0, torch.zeros_like(g), torch.round(g / s[..., None]).clamp(-8, 7))
    return q.flatten(-2), s


def _nibbles(bytes_):
    return torch.stack([bytes_ & 15, bytes_ >> 4], -1).flatten(-2)


def _bytes(nibbles):
    n = nibbles.unflatten(-1, (-1, 2))
    return n[..., 0] | (n[..., 1] << 4)


def _to_blocks(qk, sk, qv, sv):
    """Codes [P, 64, H, dim] and scales [P, 64, H, dim/group] of K and V as cache blocks uint8 [P, H, block]."""
    P, _, H, D = qk.shape
    k = (qk.permute(0, 2, 1, 3) + 8).to(torch.uint8).unflatten(-1, (D // 32, 4, 8)).transpose(-2, -3)
    v = (qv.permute(0, 2, 1, 3) + 8).to(torch.uint8)  # P H t d
    v = v.reshape(P, H, 2, 2, 4, 4, D // 64, 4, 16)   # P H B b j i g x c
    v = v.permute(0, 1, 2, 6, 4, 8, 7, 3, 5)          # P H B g j c x b i
    codes = [_bytes(a.reshape(P, H, 64 * D)) for a in (k, v)]
    scales = [a.permute(0, 2, 3, 1).contiguous().view(torch.uint8).reshape(P, H, -1) for a in (sk, sv)]
    return torch.cat(codes + scales, -1)


def _from_blocks(blocks, D, group):
    """The inverse: codes as small integers and fp32 scales, both with tokens before heads."""
    P, H, _ = blocks.shape
    n, m = 32 * D, 256 * (D // group)
    k = _nibbles(blocks[..., :n]).reshape(P, H, 64, 4, D // 32, 8).transpose(-2, -3).reshape(P, H, 64, D)
    v = _nibbles(blocks[..., n:2 * n]).reshape(P, H, 2, D // 64, 4, 16, 4, 2, 4)  # B g j c x b i
    v = v.permute(0, 1, 2, 7, 4, 8, 3, 6, 5).reshape(P, H, 64, D)
    sk, sv = (blocks[..., 2 * n + i * m:2 * n + (i + 1) * m].contiguous().view(torch.float32).reshape(P, H, -1, 64)
              for i in (0, 1))
    return (k.transpose(1, 2).to(torch.int8) - 8, sk.permute(0, 3, 1, 2),
            v.transpose(1, 2).to(torch.int8) - 8, sv.permute(0, 3, 1, 2))


def _values(q, s, group):
    return (q.float().unflatten(-1, (-1, group)) * s[..., None]).flatten(-2)


def _random_kv(gen, shape, dtype):
    """Keys with a few strong channels, as rotary models have them, and plain values, each token of its own size."""
    k = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    k = k * (1 + 4 * (torch.rand(shape[-2:], generator=gen, device="cuda") < 0.05))
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    v = v * (0.25 + torch.rand(shape[:-1], generator=gen, device="cuda"))[..., None]
    return k.to(dtype), v.to(dtype)


def _cache_inputs(case, gen):
    """The batch: rows of the fused projection, the pool of pages and the page table.  Sequences of one run hold the
    same pages for the whole pages of its prefix."""
    dev, dt = "cuda", DTYPES[case["dtype"]]
    D, H, HQ, group = case["dim"], case["kv_heads"], case["q_heads"], case["group"]
    lens = _lengths(case)
    shared = case["op"] == "shared"
    common = [_prefix(case, _group(case, b)) // PAGE if shared else 0 for b in range(len(lens))]
    need = [-(-kv // PAGE) for _, kv in lens]
    most = max(max(need), max(common), 1)
    total = sum(_prefix(case, g) // PAGE for g in range(case["groups"])) if shared else 0
    total += sum(max(0, n - c) for n, c in zip(need, common))
    num = total + 3  # a pool has free pages too
    order = torch.randperm(num, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.zeros((len(lens), most), dtype=torch.int32)
    filled = torch.zeros((num, PAGE), dtype=torch.bool)
    at, of_group = 0, {}
    for b, (n, kv) in enumerate(lens):
        c = common[b]
        if shared and _group(case, b) not in of_group:
            of_group[_group(case, b)] = order[at:at + c]
            filled[order[at:at + c].long()] = True
            at += c
        if shared:
            table[b, :c] = of_group[_group(case, b)]
        mine = order[at:at + max(0, need[b] - c)]
        at += len(mine)
        table[b, c:c + len(mine)] = mine
        held = kv if shared else max(0, kv - n)
        filled[mine.long()] = (torch.arange(c * PAGE, (c + len(mine)) * PAGE) < held).view(-1, PAGE)
    rows = sum(n for n, _ in lens)
    # the fused projection's output rows: queries, keys, values side by side
    qkv = torch.randn((rows, (HQ + 2 * H) * D), generator=gen, device=dev, dtype=torch.float32)
    qkv[:, :HQ * D] *= 1.5
    k, v = _random_kv(gen, (rows, H, D), dt)
    qkv = qkv.to(dt)
    qkv[:, HQ * D:(HQ + H) * D] = k.reshape(rows, -1)
    qkv[:, (HQ + H) * D:] = v.reshape(rows, -1)
    # what the pool's pages hold where no token has been written is anything: NaN scales here
    k, v = _random_kv(gen, (num, PAGE, H, D), dt)
    (qk, sk), (qv, sv) = _quantise(k, group), _quantise(v, group)
    free = ~filled.to(dev)[..., None, None]
    cache = _to_blocks(qk, sk.masked_fill(free, math.nan), qv, sv.masked_fill(free, math.nan))
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    i32 = dict(dtype=torch.int32, device=dev)
    return {"qkv": qkv, "cache": cache, "pages": table.to(dev), "row_start": torch.tensor(starts, **i32),
            "kv_len": torch.tensor([kv for _, kv in lens], **i32), "rows": rows, "num_pages": num, "max_pages": most}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    dt, i32 = DTYPES[case["dtype"]], dict(dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    if case["op"] == "adapt":
        K, R, ends = case["inputs"], case["rank"], _ends(case)
        N, segments = ends[-1], _rows_of_segments(case)
        rows = sum(segments)
        x = normal(rows, K) * (1 + 9 * (torch.rand((K,), generator=gen, device="cuda") < 0.01))
        s = {"x": x.to(dt), "a": (normal(case["slots"], len(ends) * R, K) / math.sqrt(K)).to(dt),
             "b": (normal(case["slots"], N, R) / math.sqrt(R)).to(dt), "y_in": normal(rows, N).to(dt), "rows": rows,
             "scale": 0.25 + torch.rand((case["slots"],), generator=gen, device="cuda")}
        starts = [0]
        for n in segments:
            starts.append(starts[-1] + n)
        s["seg_start"] = torch.tensor(starts, **i32)
        s["slot"] = torch.tensor(_slots_of_segments(case), **i32)
        return s
    s = _cache_inputs(case, gen)
    if case["op"] == "shared":
        firsts = [next(b for b in range(case["batch"]) if _group(case, b) >= g) for g in range(case["groups"])]
        s["group_start"] = torch.tensor(firsts + [case["batch"]], **i32)
        s["shared_len"] = torch.tensor([_prefix(case, g) for g in range(case["groups"])], **i32)
        counts = torch.tensor([n for n, _ in _lengths(case)])
        s["group_rows"] = max(int(counts[a:b].sum()) for a, b in zip(firsts, firsts[1:] + [case["batch"]]))
        return s
    pairs = case["rot"] // 2
    length = case["kv"] + 1
    angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
    s["table"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    s["table_len"] = length
    s["axis_of_pair"] = bytes(i % case["axes"] if case["cycle"] else i * case["axes"] // pairs for i in range(pairs))
    s["positions"] = None
    if case["axes"] > 1:  # text, then frames: time stands still over a frame, height and width run within it
        b, pos = _places(s)
        pos = pos.clamp(min=0)
        grid = [pos // 256, pos // 16 % 16, pos % 16]
        early = pos < 100
        s["positions"] = torch.stack([torch.where(early, pos, 100 + g).clamp(max=length - 1)
                                      for g in grid[:case["axes"]]]).to(torch.int32).contiguous()
    D = case["dim"]
    s["q_weight"], s["k_weight"] = ((0.5 + torch.rand((D,), generator=gen, device="cuda") for _ in range(2))
                                    if case["norm"] else (None, None))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "adapt":
        s["y"] = torch.empty_like(s["y_in"])
        # room for the products with A: fp32, split over the inputs
        s["workspace"] = torch.empty(max(64 << 20, s["rows"] * case["rank"] * len(_ends(case)) * 64), dtype=torch.uint8,
                                     device="cuda")
        return s
    D, H, HQ, dt = case["dim"], case["kv_heads"], case["q_heads"], DTYPES[case["dtype"]]
    rows = s["rows"]
    s["q"] = s["qkv"][:, :HQ * D]
    s["k"] = s["qkv"][:, HQ * D:(HQ + H) * D]
    s["v"] = s["qkv"][:, (HQ + H) * D:]
    half = dict(dtype=dt, device="cuda")
    if case["op"] == "shared":
        s["y"] = torch.empty((rows, HQ * D), **half)
        s["workspace"] = torch.empty(max(256 << 20, rows * HQ * 40 * (D + 2) * 4), dtype=torch.uint8, device="cuda")
    else:
        s["q_out"] = torch.empty((rows, HQ * D), **half)
        s["k_out"], s["v_out"] = (torch.empty((rows, H * D), **half) for _ in range(2))
    return s


# ---------------------------------------------------------------- plain forms

def _places(s):
    """Of every row: its sequence and its position (below 0: the row is not there)."""
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["row_start"][1:].contiguous(), r, right=True)
    n = s["row_start"][1:] - s["row_start"][:-1]
    return b, (s["kv_len"] - n)[b] + r - s["row_start"][b]


def _plain_turn(s, x, weight, places):
    """Heads x [rows, heads, D] (fp32 or fp64) normed and rotated."""
    c = s["case"]
    if weight is not None:
        x = x * weight / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    axis = torch.tensor(list(s["axis_of_pair"]), device="cuda")
    at = places[None] if s["positions"] is None else s["positions"].long()
    at = at[axis if s["positions"] is not None else torch.zeros_like(axis)].T  # rows, pairs
    cs = s["table"][at, torch.arange(len(axis), device="cuda")].to(x.dtype)[:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    turned, kept = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["paired"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned.chunk(2, -1)
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, kept], -1)


def _plain_rotate(s):
    c = s["case"]
    D, H, HQ, group = c["dim"], c["kv_heads"], c["q_heads"], c["group"]
    b, pos = _places(s)
    there = pos >= 0
    at = pos.clamp(min=0)
    dt = s["qkv"].dtype
    q = _plain_turn(s, s["q"].float().unflatten(-1, (HQ, D)), s["q_weight"], at)
    q = torch.where(there[:, None, None], q, 0.0).flatten(1).to(dt)
    # keys in 64 bits: a code's rounding border is no place for 32
    k = _plain_turn(s, s["k"].double().unflatten(-1, (H, D)), s["k_weight"], at)
    new = _quantise(k.float(), group) + _quantise(s["v"].unflatten(-1, (H, D)), group)
    # into the blocks of the pages that they touch
    n = s["row_start"][1:] - s["row_start"][:-1]
    first = (s["kv_len"] - n).clamp(min=0) // PAGE
    near = first[:, None] + torch.arange(-(-c["rows"] // PAGE) + 1, device="cuda")
    holds = near * PAGE < s["kv_len"][:, None]
    phys = torch.where(holds, s["pages"].gather(1, near.clamp(max=s["max_pages"] - 1)), 0).flatten().long()
    held = list(_from_blocks(s["cache"][phys], D, group))
    at = b * near.shape[1] * PAGE + at - first[b] * PAGE
    held = [old.flatten(0, 1).index_put((at[there],), x[there].to(old.dtype)).unflatten(0, (-1, PAGE))
            for old, x in zip(held, new)]
    keep = holds.flatten()
    s["cache"][phys[keep]] = _to_blocks(*held)[keep]
    # and back
    qk, sk, qv, sv = (x.flatten(0, 1) for x in _from_blocks(s["cache"][phys], D, group))
    out = [torch.where(there[:, None, None], _values(y[at], t[at], group), 0.0) for y, t in ((qk, sk), (qv, sv))]
    return [q] + [x.flatten(1).to(dt) for x in out]


def _plain_shared(s):
    c = s["case"]
    D, H, HQ, group = c["dim"], c["kv_heads"], c["q_heads"], c["group"]
    B, R, G, P = c["batch"], c["rows"], HQ // H, s["max_pages"]
    qk, sk, qv, sv = _from_blocks(s["cache"], D, group)
    k, v = (_values(q, x, group).permute(0, 2, 1, 3) for q, x in ((qk, sk), (qv, sv)))  # pages, heads, tokens, dim
    b, pos = _places(s)
    i = torch.arange(s["rows"], device="cuda") - s["row_start"][b]
    q = torch.zeros((B, R, HQ, D), device="cuda").index_put((b, i), s["q"].float().unflatten(-1, (HQ, D)))
    q = q.view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    at = torch.full((B, R), -1, device="cuda").index_put((b, i), pos)
    t = torch.arange(P * PAGE, device="cuda")
    seen = t <= at[..., None]
    ids = s["pages"].flatten().long()
    keys = k[ids].unflatten(0, (B, P)).permute(0, 2, 4, 1, 3).reshape(B, H, D, P * PAGE)
    x = torch.matmul(q, keys.nan_to_num_(0.0)) * (1 / math.sqrt(D))
    del keys
    x = x.view(B, H, R, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = (x - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    x /= torch.where(total == 0, 1.0, total)
    values = v[ids].unflatten(0, (B, P)).permute(0, 2, 1, 3, 4).reshape(B, H, P * PAGE, D)
    y = torch.matmul(x.view(B, H, R * G, -1), values.nan_to_num_(0.0))
    y = y.view(B, H, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, HQ * D)
    return y[b, i].to(s["q"].dtype)


def _plain_adapt(s):
    """Each row's slot; then every adapter's two products for all rows, of which a row keeps its own adapter's."""
    c = s["case"]
    R, ends = c["rank"], _ends(c)
    r = torch.arange(s["rows"], device="cuda")
    slot = s["slot"].long()[torch.searchsorted(s["seg_start"][1:].contiguous(), r, right=True)]
    mine = slot[:, None] == torch.arange(c["slots"], device="cuda")  # rows, slots
    t = s["x"].float() @ s["a"].float().flatten(0, 1).T.contiguous()
    t = t.unflatten(-1, (c["slots"], len(ends), R)) * (mine * s["scale"])[:, :, None, None]
    widths = [b - a for a, b in zip([0] + ends, ends)]
    parts = [t[:, :, i].flatten(1) @ w.float().transpose(1, 2).flatten(0, 1).contiguous()
             for i, w in enumerate(s["b"].split(widths, 1))]
    return (s["y_in"].float() + torch.cat(parts, 1)).to(s["x"].dtype)


# ---------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rotate": _plain_rotate, "shared": _plain_shared, "adapt": _plain_adapt}[c["op"]](s)
    import w4a8_quantized_linear_amd as cider
    dtype = cider.CIDER_DTYPE_F16 if c["dtype"] == "f16" else cider.CIDER_DTYPE_BF16
    if c["op"] == "adapt":
        ends = _ends(c)
        w = cider.cider_lora(s["a"], s["b"], s["scale"], c["slots"], c["rank"], c["inputs"], ends)
        cider.cider_lora_add(w, s["seg_start"], s["slot"], c["segments"], s["rows"], c["rows"], s["x"], dtype,
                             c["inputs"], s["y_in"], ends[-1], s["workspace"], s["workspace"].numel(), s["y"], ends[-1])
        return s["y"]
    D, H, HQ = c["dim"], c["kv_heads"], c["q_heads"]
    batch = cider.cider_kv4_batch(s["cache"], s["pages"], s["row_start"], s["kv_len"], c["batch"], s["rows"],
                                  c["rows"], s["max_pages"] * PAGE, s["max_pages"], s["num_pages"], H, D, c["group"])
    ld = (HQ + 2 * H) * D
    if c["op"] == "shared":
        runs = cider.cider_kv4_runs(s["group_start"], s["shared_len"], c["groups"], s["group_rows"], c["prefix"])
        cider.cider_kv4_attention_shared(batch, runs, s["q"], dtype, ld, HQ, 1 / math.sqrt(D), s["workspace"],
                                         s["workspace"].numel(), s["y"], dtype, HQ * D)
        return s["y"]
    turn = cider.cider_rotation(s["table"], s["table_len"], c["rot"], c["paired"], s["positions"], c["axes"],
                                s["axis_of_pair"], s["q_weight"], s["k_weight"], EPS)
    cider.cider_kv4_append_rotated(batch, turn, s["q"], s["k"], s["v"], dtype, ld, ld, ld, HQ, s["q_out"], HQ * D)
    cider.cider_kv4_read(batch, s["k_out"], s["v_out"], dtype, H * D, H * D)
    return [s["q_out"], s["k_out"], s["v_out"]]


# ---------------------------------------------------------------- in 64 bits

def _exact_codes(x, group):
    """What the cache gives back of 64-bit rows: rows, scale and quotient are fp32 numbers by definition."""
    g = x.float().double().unflatten(-1, (-1, group))
    top = g.abs().amax(-1, keepdim=True)
    s = (top / torch.full_like(top, 7)).float().double()
    quotient = (g / torch.where(s == 0, 1.0, s)).float().double()
    return (torch.round(quotient).clamp(-8, 7) * (s != 0) * s).flatten(-2)


def _exact_turn(s, case, x, weight, pos):
    """By complex numbers: x [rows, heads, D] in 64 bits."""
    if weight is not None:
        x = x * weight.double() * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS)
    pairs = case["rot"] // 2
    z = torch.view_as_complex(s["table"].double())
    cols = []
    for i, axis in enumerate(s["axis_of_pair"]):
        cols.append(z[pos if s["positions"] is None else s["positions"][axis].long(), i])
    w = torch.stack(cols, -1)[:, None]
    i = torch.arange(pairs, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["paired"] else (i, i + pairs)
    y = torch.complex(x[..., first], x[..., second]) * w
    out = x.clone()
    out[..., first], out[..., second] = y.real, y.imag
    return out


def _exact_cached(blocks, D, group):
    """K and V [H, 64 * pages, dim] in 64 bits of a run of blocks [pages, H, block], each code found by its address."""
    P, H, _ = blocks.shape
    t = torch.arange(PAGE, device="cuda")[:, None]
    d = torch.arange(D, device="cuda")[None, :]
    k_at = t * (D // 2) + ((d // 8) % 4) * (D // 8) + (d // 32) * 4 + (d % 8) // 2
    k_high = (d % 2).expand_as(k_at)
    place = (((t // 32) * (D // 64) + d // 64) * 4 + (t // 4) % 4) * 64 + (d % 16) * 4 + (d // 16) % 4
    nib = ((t // 16) % 2) * 4 + t % 4
    v_at = 32 * D + place * 4 + nib // 2
    v_high = (nib % 2).expand_as(v_at)
    out = []
    for at, high, s0 in ((k_at, k_high, 64 * D), (v_at, v_high, 64 * D + 256 * (D // group))):
        byte = blocks[:, :, at].to(torch.int32)
        code = ((byte >> (4 * high)) & 15) - 8
        scale = blocks[:, :, s0:s0 + 256 * (D // group)].contiguous().view(torch.float32).double()
        scale = scale.view(P, H, D // group, PAGE).transpose(-1, -2).repeat_interleave(group, -1)
        out.append((code * scale).transpose(0, 1).reshape(H, P * PAGE, D))
    return out


def _exact_shared(case, s):
    D, H, HQ, group = case["dim"], case["kv_heads"], case["q_heads"], case["group"]
    G, lo, ys = HQ // H, 0, []
    for b, (n, have) in enumerate(_lengths(case)):
        q = s["qkv"][lo:lo + n, :HQ * D].double().view(n, H, G, D)
        lo += n
        y = torch.zeros((n, H, G, D), dtype=torch.float64, device="cuda")
        if have:
            ids = s["pages"][b, :-(-have // PAGE)].long()
            k, v = (x[:, :have] for x in _exact_cached(s["cache"][ids], D, group))
            hidden = torch.arange(have, device="cuda") > torch.arange(have - n, have, device="cuda")[:, None]
            for h in range(H):
                x = (q[:, h].reshape(-1, D) @ k[h].T.contiguous()).view(n, G, have) / math.sqrt(D)
                x = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
                y[:, h] = (x.view(-1, have) @ v[h].contiguous()).view(n, G, D)
        ys.append(y.flatten(1))
    return torch.cat(ys)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "shared":
        return _exact_shared(case, s)
    if case["op"] == "adapt":
        y, lo, R = s["y_in"].double(), 0, case["rank"]
        for n, a in zip(_rows_of_segments(case), _slots_of_segments(case)):
            if a >= 0:
                t = s["x"][lo:lo + n].double() @ s["a"][a].double().T.contiguous() * s["scale"][a].double()
                for i, (e0, e1) in enumerate(zip([0] + _ends(case), _ends(case))):
                    y[lo:lo + n, e0:e1] += t[:, i * R:(i + 1) * R] @ s["b"][a, e0:e1].double().T.contiguous()
            lo += n
        return y
    D, H, HQ, group = case["dim"], case["kv_heads"], case["q_heads"], case["group"]
    x = s["qkv"].double().unflatten(-1, (HQ + 2 * H, D))
    pos = torch.cat([torch.arange(kv - n, kv, device="cuda") for n, kv in _lengths(case)])
    at = pos.clamp(min=0)
    q = _exact_turn(s, case, x[:, :HQ], s["q_weight"], at)
    k = _exact_codes(_exact_turn(s, case, x[:, HQ:HQ + H], s["k_weight"], at), group)
    v = _exact_codes(x[:, HQ + H:], group)
    gone = (pos < 0)[:, None, None]
    return [y.masked_fill(gone, 0.0).flatten(1) for y in (q, k, v)]
