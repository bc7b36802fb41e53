"""Cases of the 4-bit key/value cache: writing and reading it back, and the attention over it.

Every case is a batch of sequences that share one paged cache.  Sequence b brings n_b rows (tokens) to the call and
holds kv_b tokens in the cache once they are in it, so its row i stands at position kv_b - n_b + i.  A page holds 64
tokens; a block is one head of one page: the codes of K and of V (nibble = code + 8), then the fp32 scales of both.
"""
import math

import torch

own = False

PAGE = 64
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# Scratch that a serving program keeps for the attention's partial results.
WORKSPACE_BYTES = 64 << 20


# ---------------------------------------------------------------- cases

def _case(name, op, dtype, batch, rows, kv, q_heads, kv_heads, dim, group, window=0, sinks=0, ragged=False):
    c = dict(op=op, dtype=dtype, batch=batch, rows=rows, kv=kv, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
             group=group, window=window, sinks=sinks, ragged=ragged)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One token of one conversation: 32 query and 8 key/value heads of 128, as the decoder stack's fused
        # QKV product (6144 outputs) gives them.  All latency.
        _case("write_one_token", "write", "f16", 1, 1, 1001, 32, 8, 128, 64),
        # A batch of prompts of different lengths entering the cache at once.
        _case("write_prompts", "write", "bf16", 6, 4096, 4096, 32, 8, 128, 128, ragged=True),
        # The prefix of one conversation, read back for a program that attends in 16 bits.
        _case("read_prefix", "read", "f16", 1, 777, 777, 32, 8, 128, 64),
        # A whole batch's caches read back (moved to another format).
        _case("read_batch", "read", "bf16", 8, 8192, 8192, 32, 8, 128, 64, ragged=True),
        # Single tokens: one short conversation, where launches and latency count.
        _case("attend_one_short", "attend", "f16", 1, 1, 1001, 32, 8, 128, 64),
        # The ordinary serving step: a batch of conversations of all lengths, one of them a padded slot.
        _case("attend_batch", "attend", "bf16", 64, 1, 8192, 32, 8, 128, 64, ragged=True),
        # One very long document: the axis has to be split.
        _case("attend_one_long", "attend", "f16", 1, 1, 131072, 32, 8, 128, 128),
        # A batch under a sliding window with the first four tokens kept.
        _case("attend_window_batch", "attend", "bf16", 32, 1, 20000, 32, 8, 128, 64, window=4096, sinks=4, ragged=True),
        # A few drafted tokens verified at once, small heads, seven query heads to a key/value head.
        _case("attend_drafts", "attend", "f16", 16, 5, 3001, 28, 4, 64, 64, ragged=True),
        # A chunk of a long prompt over what is cached already.
        _case("attend_chunk", "attend", "f16", 1, 2048, 16384, 32, 8, 128, 64),
        # Whole prompts of different lengths, causal.
        _case("attend_prompts", "attend", "bf16", 4, 4096, 4096, 32, 8, 128, 128, ragged=True),
        # A prompt under a sliding window with sinks.
        _case("attend_window_prompt", "attend", "f16", 1, 8000, 8000, 32, 8, 128, 64, window=1024, sinks=4),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128])
    group = 64 if dim == 64 else rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    dtype = rng.choice(["f16", "bf16"])
    ragged = rng.random() < 0.6
    if op != "attend":
        batch = _spread(rng, 1, 32)
        rows = _spread(rng, 1, (16384 if op == "write" else 32768) // batch)
        kv = rows if op == "read" or rng.random() < 0.5 else rows + _spread(rng, 1, 4000)
        return _case(None, op, dtype, batch, rows, kv, q_heads, kv_heads, dim, group, ragged=ragged and batch > 1)
    window, sinks = 0, 0
    if rng.random() < 0.4:
        window, sinks = _spread(rng, 1, 8192), rng.choice([0, 1, 4, 4, 70])
    if rng.random() < 0.6:
        batch, rows = _spread(rng, 1, 64), rng.choice([1, 1, 1, 2, 5, 8])
        kv = _spread(rng, rows, min(131072, 200000 // batch))
    else:
        batch = _spread(rng, 1, 4)
        rows = _spread(rng, 9, 4096 // batch)
        kv = rows + (0 if rng.random() < 0.5 else _spread(rng, 1, 12288))
        while q_heads * batch * rows * (kv - rows / 2) > 32 * 2048 * 15360:  # the listed chunk's work
            rows, kv = rows // 2 + 1, kv - rows + rows // 2 + 1
    return _case(None, op, dtype, batch, rows, kv, q_heads, kv_heads, dim, group, window, sinks, ragged and batch > 1)


def _lengths(case):
    """(rows, cached tokens) of each sequence.  Ragged batches spread both; their third sequence is a slot that the
    program padded its batch with: one row, nothing cached."""
    out = []
    for b in range(case["batch"]):
        n, kv = case["rows"], case["kv"]
        if case["ragged"]:
            part = 1.0 - 0.85 * ((b * 0.6180339887) % 1.0)
            before = int((kv - n) * part)
            if n > 8:
                n = max(1, int(n * part))
            kv = n + before
            if b == 2 and case["op"] != "read":
                n, kv = 1, 0
        out.append((n, kv))
    return out


def _visible(n, kv, window, sinks):
    """(pairs, tokens): how many (row, token) pairs a sequence has, and how many tokens any row sees."""
    pairs, tokens = 0, 0
    first = max(0, kv - n)
    for p in range(first, kv):
        seen = p + 1
        if window and seen > window:
            seen = window + min(sinks, seen - window)
        pairs += seen
    if kv > 0:
        tokens = kv
        if window and first + 1 > window:
            tokens = kv - (first + 1 - window) + min(sinks, first + 1 - window)
    return pairs, tokens


def work(case):
    dim, hk, hq = case["dim"], case["kv_heads"], case["q_heads"]
    lens = _lengths(case)
    rows = sum(n for n, _ in lens)
    stored = dim + 8 * (dim // case["group"])  # one token's K and V of one head in the cache
    plain = 4 * dim                            # the same in 16 bits
    if case["op"] == "write":  # 16-bit rows in, codes and scales out, and back
        there = sum(min(n, kv) for n, kv in lens)
        return {"bytes": 2 * there * hk * (stored + plain), "flops": there * hk * dim * 12}
    if case["op"] == "read":
        return {"bytes": rows * hk * (stored + plain), "flops": rows * hk * dim * 4}
    seen = [_visible(n, kv, case["window"], case["sinks"]) for n, kv in lens]
    return {"bytes": sum(t for _, t in seen) * hk * stored + 4 * rows * hq * dim,
            "flops": 4 * dim * hq * sum(p for p, _ in seen)}


# ---------------------------------------------------------------- inputs

def _quantise(x, group):
    """(codes -8 .. 7, fp32 scales) of rows [..., dim]: scale = max|x| / 7 of each group, code = rint(x / scale)."""
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
    D = shape[-1]
    k = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    k = k * (1 + 4 * (torch.rand(shape[-2:], generator=gen, device="cuda") < 0.05))
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    v = v * (0.25 + torch.rand(shape[:-1], generator=gen, device="cuda"))[..., None]
    return k.to(dtype), v.to(dtype)


def _inputs(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)
    D, H, HQ, group = case["dim"], case["kv_heads"], case["q_heads"], case["group"]
    lens = _lengths(case)
    need = [-(-kv // PAGE) for _, kv in lens]
    most = max(max(need), 1)
    total = sum(need)
    num = total + 3  # a pool has free pages too
    order = torch.randperm(num, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), most), dtype=torch.int32)
    at, filled = 0, torch.zeros((num, PAGE), dtype=torch.bool)
    order_host = order.cpu()
    for b, (n, kv) in enumerate(lens):
        table[b, :need[b]] = order_host[at:at + need[b]]
        held = max(0, kv - n) if case["op"] == "write" else kv
        mask = (torch.arange(need[b] * PAGE) < held).view(-1, PAGE)
        filled[order_host[at:at + need[b]].long()] = mask
        at += need[b]
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


def prepare(case, seed):
    s = _inputs(case, seed)
    D, H, HQ, dt = case["dim"], case["kv_heads"], case["q_heads"], DTYPES[case["dtype"]]
    rows, dev = s["rows"], "cuda"
    s["case"] = case
    s["q"] = s["qkv"][:, :HQ * D]
    s["k"] = s["qkv"][:, HQ * D:(HQ + H) * D]
    s["v"] = s["qkv"][:, (HQ + H) * D:]
    if case["op"] == "attend":
        s["y"] = torch.empty((rows, HQ * D), dtype=dt, device=dev)
        s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    else:
        s["k_out"] = torch.empty((rows, H * D), dtype=dt, device=dev)
        s["v_out"] = torch.empty((rows, H * D), dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------- plain forms

def _places(s):
    """Of every row: its sequence and its position (below 0: the row is not there)."""
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["row_start"][1:].contiguous(), r, right=True)
    n = s["row_start"][1:] - s["row_start"][:-1]
    return b, (s["kv_len"] - n)[b] + r - s["row_start"][b]


def _plain_write(s):
    """Quantises the rows into the blocks of the pages that they touch."""
    c = s["case"]
    D, H, group = c["dim"], c["kv_heads"], c["group"]
    b, pos = _places(s)
    n = s["row_start"][1:] - s["row_start"][:-1]
    first = (s["kv_len"] - n).clamp(min=0) // PAGE
    near = first[:, None] + torch.arange(-(-c["rows"] // PAGE) + 1, device="cuda")
    there = near * PAGE < s["kv_len"][:, None]
    phys = torch.where(there, s["pages"].gather(1, near.clamp(max=s["max_pages"] - 1)), 0).flatten().long()
    held = list(_from_blocks(s["cache"][phys], D, group))
    at = (b * near.shape[1] * PAGE + pos - first[b] * PAGE)[pos >= 0]
    new = _quantise(s["k"].unflatten(-1, (H, D)), group) + _quantise(s["v"].unflatten(-1, (H, D)), group)
    held = [old.flatten(0, 1).index_put((at,), x[pos >= 0].to(old.dtype)).unflatten(0, (-1, PAGE))
            for old, x in zip(held, new)]
    blocks = _to_blocks(*held)
    keep = there.flatten()
    s["cache"][phys[keep]] = blocks[keep]


def _plain_read(s):
    c = s["case"]
    D, group = c["dim"], c["group"]
    b, pos = _places(s)
    at = pos.clamp(min=0)
    n = s["row_start"][1:] - s["row_start"][:-1]
    first = (s["kv_len"] - n).clamp(min=0) // PAGE
    near = first[:, None] + torch.arange(-(-c["rows"] // PAGE) + 1, device="cuda")
    phys = s["pages"].gather(1, near.clamp(max=s["max_pages"] - 1)).flatten().long()
    qk, sk, qv, sv = (x.flatten(0, 1) for x in _from_blocks(s["cache"][phys], D, group))
    at = b * near.shape[1] * PAGE + at - first[b] * PAGE
    out = [torch.where(pos[:, None, None] >= 0, _values(q[at], t[at], group), 0.0) for q, t in ((qk, sk), (qv, sv))]
    return [x.flatten(1).to(s["qkv"].dtype) for x in out]


def _plain_attend(s):
    c = s["case"]
    D, H, HQ, group = c["dim"], c["kv_heads"], c["q_heads"], c["group"]
    B, R, G = c["batch"], c["rows"], HQ // H
    P = s["max_pages"]
    qk, sk, qv, sv = _from_blocks(s["cache"][s["pages"].flatten().long()], D, group)
    t = torch.arange(P * PAGE, device="cuda")
    held = (t < s["kv_len"][:, None])[:, :, None, None]
    k, v = (torch.where(held, _values(q, x, group).reshape(B, P * PAGE, H, D), 0.0).permute(0, 2, 1, 3)
            for q, x in ((qk, sk), (qv, sv)))
    b, pos = _places(s)
    i = torch.arange(s["rows"], device="cuda") - s["row_start"][b]
    q = torch.zeros((B, R, HQ, D), device="cuda").index_put((b, i), s["q"].float().unflatten(-1, (HQ, D)))
    q = q.view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    at = torch.full((B, R), -1, device="cuda").index_put((b, i), pos)
    seen = t <= at[..., None]
    if c["window"]:
        seen &= (t > at[..., None] - c["window"]) | (t < c["sinks"])
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()) * (1 / math.sqrt(D))
    x = x.view(B, H, R, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = (x - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    x /= torch.where(total == 0, 1.0, total)
    y = torch.matmul(x.view(B, H, R * G, -1), v.contiguous())
    y = y.view(B, H, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, HQ * D)
    return y[b, i].to(s["q"].dtype)


# ---------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "attend":
            return _plain_attend(s)
        if c["op"] == "write":
            _plain_write(s)
        return _plain_read(s)
    import w4a8_quantized_linear_amd as cider
    dtype = cider.CIDER_DTYPE_F16 if c["dtype"] == "f16" else cider.CIDER_DTYPE_BF16
    D, H, HQ = c["dim"], c["kv_heads"], c["q_heads"]
    batch = cider.cider_kv4_batch(s["cache"], s["pages"], s["row_start"], s["kv_len"], c["batch"], s["rows"],
                                  c["rows"], s["max_pages"] * PAGE, s["max_pages"], s["num_pages"], H, D, c["group"])
    ld = (HQ + 2 * H) * D
    if c["op"] == "attend":
        cider.cider_kv4_attention(batch, s["q"], dtype, ld, HQ, 1 / math.sqrt(D), c["window"], c["sinks"],
                                  s["workspace"], WORKSPACE_BYTES, s["y"], dtype, HQ * D)
        return s["y"]
    if c["op"] == "write":
        cider.cider_kv4_append(batch, s["k"], s["v"], dtype, ld, ld)
    cider.cider_kv4_read(batch, s["k_out"], s["v_out"], dtype, H * D, H * D)
    return [s["k_out"], s["v_out"]]


# ---------------------------------------------------------------- in 64 bits

def _exact_codes(x, group):
    """Codes and scales of rows in 64 bits; the scale and the quotient are fp32 numbers by definition."""
    g = x.double().unflatten(-1, (-1, group))
    top = g.abs().amax(-1, keepdim=True)
    s = (top / torch.full_like(top, 7)).float().double()
    quotient = (g / torch.where(s == 0, 1.0, s)).float().double()
    return (torch.round(quotient).clamp(-8, 7) * (s != 0) * s).flatten(-2)


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


def exact(case, seed):
    s = _inputs(case, seed)
    D, H, HQ, group = case["dim"], case["kv_heads"], case["q_heads"], case["group"]
    lens = _lengths(case)
    G, lo = HQ // H, 0
    if case["op"] == "write":
        kv = s["qkv"][:, HQ * D:].unflatten(-1, (2, H, D))
        back = _exact_codes(kv, group)
        for n, have in lens:
            back[lo:lo + max(0, n - have)] = 0
            lo += n
        return [back[:, 0].flatten(1), back[:, 1].flatten(1)]
    ys = []
    for b, (n, have) in enumerate(lens):
        q = s["qkv"][lo:lo + n, :HQ * D].double().view(n, H, G, D)
        lo += n
        if have == 0:
            ys.append(torch.zeros((n, HQ * D), dtype=torch.float64, device="cuda"))
            continue
        ids = s["pages"][b, :-(-have // PAGE)].long()
        k, v = (x[:, :have] for x in _exact_cached(s["cache"][ids], D, group))
        if case["op"] == "read":
            ys.append(torch.stack([k[:, have - n:], v[:, have - n:]]).transpose(1, 2).flatten(2))
            continue
        y = torch.zeros((n, H, G, D), dtype=torch.float64, device="cuda")
        t = torch.arange(have, device="cuda")
        step = max(1, (1 << 28) // (H * G * have))
        for r in range(0, n, step):
            p = torch.arange(r, min(n, r + step), device="cuda") + have - n
            seen = t <= p[:, None]
            if case["window"]:
                seen &= (t > p[:, None] - case["window"]) | (t < case["sinks"])
            for h in range(H):
                x = (q[r:r + step, h].reshape(-1, D) @ k[h].T.contiguous()).view(len(p), G, have) / math.sqrt(D)
                x = torch.softmax(x.masked_fill(~seen[:, None], -math.inf), -1).nan_to_num(0.0)
                y[r:r + step, h] = (x.view(-1, have) @ v[h].contiguous()).view(len(p), G, D)
        ys.append(y.flatten(1))
    if case["op"] == "read":
        both = torch.cat(ys, 1)
        return [both[0], both[1]]
    return torch.cat(ys)
