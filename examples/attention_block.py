"""One decoder attention block served from quantized weights and a 4-bit
key/value cache:  x -> QKV product -> append -> attention -> O product -> x,
a batch of prompts first, then decoding steps replayed from a HIP graph.

    python examples/attention_block.py [--batch 8] [--prompt 1000] [--steps 32]
                                       [--bits 4] [--window 0] [--sinks 4]
                                       [--rotate] [--adapters 0] [--shared 0]

Sizes are those of the benchmark's decoder stack (hidden 4096, 32 query heads
and 8 key/value heads of 128: QKV 6144 x 4096, O 4096 x 4096); weights are
random.  --rotate: q and k are normed for each head and turned by their positions
on the way into the cache (without it positions are not encoded).  --adapters n:
the sequences take n low-rank adapters by turns, beside both products.  --shared
n: the prompts begin with the same n tokens, whose whole pages are in the cache
once and attended to once for all sequences.  Prints the time of the prompt pass
and of a decoding step, and how far the block's attention is from 16-bit attention
over the same keys and values (what 4 bits cost)."""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import w4a8_quantized_linear_amd as cider  # noqa: E402

F16 = cider.CIDER_DTYPE_F16
PAGE = cider.KV4_PAGE_TOKENS


class Linear:
    """y = x W^T with int8 or packed int4 weights, quantized once."""

    def __init__(self, out_features, in_features, bits, generator):
        w = torch.randn((out_features, in_features), device="cuda", generator=generator) / math.sqrt(in_features)
        self.N, self.K, self.bits = out_features, in_features, bits
        self.wq = torch.empty((self.N, self.K * bits // 8), dtype=torch.uint8, device="cuda")
        self.scale = torch.empty(self.N, dtype=torch.float32, device="cuda")
        cider.cider_quantize_weight(w.half(), self.N, self.K, bits, 0, self.wq, self.scale)

    def __call__(self, x, rows, ldx, y, workspace):
        cider.cider_linear_ex(x, F16, rows, self.K, ldx, None, self.wq, self.scale, self.N, self.bits, 0, F16,
                              workspace, workspace.numel(), y)


class Adapters:
    """Low-rank corrections of a product, `slots` of them, and the segments of rows that take them."""

    def __init__(self, ends, in_features, slots, rank, generator):
        half = dict(device="cuda", generator=generator, dtype=torch.float32)
        self.ends, self.rank, self.K, self.slots = ends, rank, in_features, slots
        self.a = (torch.randn((slots, len(ends) * rank, in_features), **half) / math.sqrt(in_features)).half()
        self.b = (torch.randn((slots, ends[-1], rank), **half) * (0.1 / math.sqrt(rank))).half()
        self.lora = cider.cider_lora(self.a, self.b, None, slots, rank, in_features, ends)

    def __call__(self, x, rows, ldx, starts, slot, max_rows, y, workspace):
        """Adds them to y in place."""
        cider.cider_lora_add(self.lora, starts, slot, slot.numel(), rows, max_rows, x, F16, ldx, y, self.ends[-1],
                             workspace, workspace.numel(), y, self.ends[-1])


class AttentionBlock:
    def __init__(self, batch, capacity, bits=4, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, group_size=64,
                 window=0, sinks=0, seed=0, rotate=False, adapters=0, shared=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.HQ, self.H, self.D, self.gs, self.hidden = q_heads, kv_heads, head_dim, group_size, hidden
        self.window, self.sinks, self.batch = window, sinks, batch
        self.width = (q_heads + 2 * kv_heads) * head_dim
        self.qkv = Linear(self.width, hidden, bits, g)
        self.o = Linear(hidden, q_heads * head_dim, bits, g)
        self.per_seq = -(-capacity // PAGE)
        self.num_pages = batch * self.per_seq
        nbytes = cider.cider_kv4_cache_bytes(self.num_pages, kv_heads, head_dim, group_size)
        self.cache = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        # any assignment of pages will do; a server hands them out as sequences grow
        self.pages = torch.randperm(self.num_pages, device="cuda", generator=g).int().view(batch, self.per_seq)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.rotation = self.table = None
        if rotate:
            angle = torch.arange(capacity, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
                -torch.arange(head_dim // 2, device="cuda", dtype=torch.float64) / (head_dim // 2))
            self.table = torch.stack([angle.cos(), angle.sin()], -1).float()
            self.norm = 0.5 + torch.rand(head_dim, device="cuda", generator=g)
            self.rotation = cider.cider_rotation(self.table, capacity, head_dim, q_weight=self.norm, k_weight=self.norm)
        self.adapters = None
        if adapters:
            ends = [q_heads * head_dim, (q_heads + kv_heads) * head_dim, self.width]
            self.adapters = (Adapters(ends, hidden, adapters, 16, g), Adapters([hidden], q_heads * head_dim, adapters, 16, g))
            # keys and values of a shared prefix are those of one adapter
            self.slot = torch.arange(batch, dtype=torch.int32, device="cuda") % (1 if shared else adapters)
        self.shared = shared // PAGE * PAGE
        if self.shared:
            self.pages[:, :self.shared // PAGE] = self.pages[0, :self.shared // PAGE].clone()
            self.group = torch.tensor([0, batch], dtype=torch.int32, device="cuda")
            self.shared_len = torch.tensor([self.shared], dtype=torch.int32, device="cuda")

    def runs(self, rows):
        return cider.cider_kv4_runs(self.group, self.shared_len, 1, rows, self.shared)

    def buffers(self, rows, max_rows):
        """What a pass over `rows` rows writes, and its scratch."""
        half = dict(dtype=torch.float16, device="cuda")
        b = {"qkv": torch.empty((rows, self.width), **half), "att": torch.empty((rows, self.HQ * self.D), **half),
             "y": torch.empty((rows, self.hidden), **half)}
        linear = max(cider.cider_linear_workspace_bytes_ex(rows, l.N, l.K, l.bits, 0) for l in (self.qkv, self.o))
        b["linear"] = torch.empty(linear, dtype=torch.uint8, device="cuda")
        seqs = self._batch(rows, max_rows, self.kv_len)
        if self.shared:
            need = cider.cider_kv4_attention_shared_workspace_bytes(seqs, self.runs(rows), self.HQ)
        else:
            need = cider.cider_kv4_attention_workspace_bytes(seqs, self.HQ, self.window, self.sinks)
        if self.adapters:
            lora = max(cider.cider_lora_workspace_bytes(x.lora, self.batch, rows, max_rows) for x in self.adapters)
            b["lora"] = torch.empty(lora, dtype=torch.uint8, device="cuda")
        b["attention"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        return b

    def _batch(self, rows, max_rows, row_start):
        return cider.cider_kv4_batch(self.cache, self.pages, row_start, self.kv_len, self.batch, rows, max_rows,
                                     self.per_seq * PAGE, self.per_seq, self.num_pages, self.H, self.D, self.gs)

    def forward(self, x, row_start, max_rows, b):
        """x [rows, hidden]; kv_len already counts the rows.  Every call is asynchronous on the current stream."""
        rows, ld = x.shape[0], self.width
        seqs = self._batch(rows, max_rows, row_start)
        self.qkv(x, rows, self.hidden, b["qkv"], b["linear"])
        if self.adapters:
            self.adapters[0](x, rows, self.hidden, row_start, self.slot, max_rows, b["qkv"], b["lora"])
        k = b["qkv"][:, self.HQ * self.D:]
        v = b["qkv"][:, (self.HQ + self.H) * self.D:]
        if self.rotation:  # q is turned in place
            cider.cider_kv4_append_rotated(seqs, self.rotation, b["qkv"], k, v, F16, ld, ld, ld, self.HQ, b["qkv"], ld)
        else:
            cider.cider_kv4_append(seqs, k, v, F16, ld, ld)
        if self.shared:
            cider.cider_kv4_attention_shared(seqs, self.runs(rows), b["qkv"], F16, ld, self.HQ, 1 / math.sqrt(self.D),
                                             b["attention"], b["attention"].numel(), b["att"], F16, self.HQ * self.D)
        else:
            cider.cider_kv4_attention(seqs, b["qkv"], F16, ld, self.HQ, 1 / math.sqrt(self.D), self.window, self.sinks,
                                      b["attention"], b["attention"].numel(), b["att"], F16, self.HQ * self.D)
        self.o(b["att"], rows, self.HQ * self.D, b["y"], b["linear"])
        if self.adapters:
            self.adapters[1](b["att"], rows, self.HQ * self.D, row_start, self.slot, max_rows, b["y"], b["lora"])
        return b["y"]


def turned(block, x):
    """Heads [n, heads, D] of the positions 0 .. n - 1, normed and rotated."""
    if block.rotation is None:
        return x
    x = x * block.norm * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    c, s = block.table[:x.shape[0], None].unbind(-1)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def attention_in_16_bits(block, qkv, lengths):
    """The same rows' attention over their own unquantized keys and values (whole prompts, window 0).  Behind a shared
    prefix a sequence but the first brings only what it has of its own; q is turned already, k is not."""
    out, lo = [], 0
    for b, n in enumerate(lengths):
        own = qkv[lo:lo + n - (block.shared if b else 0)]
        lo += len(own)
        rows = own if len(own) == n else torch.cat([qkv[:n - len(own)], own])
        q, k, v = (rows.float()[:, a * block.D:b * block.D].view(n, -1, block.D)
                   for a, b in ((0, block.HQ), (block.HQ, block.HQ + block.H), (block.HQ + block.H, block.HQ + 2 * block.H)))
        q, k, v = (t.transpose(0, 1).contiguous() for t in (q, turned(block, k), v))
        k, v = (t.repeat_interleave(block.HQ // block.H, 0) for t in (k, v))
        s = q @ k.transpose(1, 2).contiguous() / math.sqrt(block.D)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        out.append((torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, -1)[n - len(own):])
    return torch.cat(out)


def timed(f, n):
    f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n * 1e3


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=1000, help="tokens of the longest prompt; others are shorter")
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--bits", type=int, default=4, choices=(4, 8))
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=4)
    p.add_argument("--rotate", action="store_true")
    p.add_argument("--adapters", type=int, default=0)
    p.add_argument("--shared", type=int, default=0, help="first tokens that all prompts have in common")
    a = p.parse_args(argv)
    if a.shared and (a.window or a.shared >= a.prompt // 2):
        p.error("--shared goes with no window and prompts of more than twice as many tokens")
    if not cider.cider_is_available():
        raise SystemExit("no usable gfx950 device")
    block = AttentionBlock(a.batch, a.prompt + a.steps, a.bits, window=a.window, sinks=a.sinks, rotate=a.rotate,
                           adapters=a.adapters, shared=a.shared)
    lengths = [max(1, a.prompt - b * a.prompt // (2 * a.batch)) for b in range(a.batch)]
    counts = [n - (block.shared if b else 0) for b, n in enumerate(lengths)]
    rows = sum(counts)
    i32 = dict(dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), **i32)
    x = torch.randn((rows, block.hidden), device="cuda").half()

    block.kv_len.copy_(torch.tensor(lengths, **i32))
    b = block.buffers(rows, max(counts))
    prompt_us = timed(lambda: block.forward(x, starts, max(counts), b), 3)
    result = {"prompt_us": prompt_us, "rows": rows}
    if a.window == 0:
        want = attention_in_16_bits(block, b["qkv"], lengths)
        result["error"] = ((b["att"].float() - want).norm() / want.norm()).item()

    # one token per sequence and step: the graph appends and attends at whatever lengths kv_len holds
    b = block.buffers(a.batch, 1)
    x = torch.randn((a.batch, block.hidden), device="cuda").half()
    one_each = torch.arange(a.batch + 1, **i32)
    block.kv_len += 1
    block.forward(x, one_each, 1, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, one_each, 1, b)
        x.copy_(b["y"])
        block.kv_len += 1
    result["step_us"] = timed(graph.replay, max(1, a.steps - 2))
    result["finite"] = bool(b["y"].isfinite().all().item())
    print("prompts: %d tokens in %.0f us; decoding: batch %d, %.1f us a step; W%dA8, 4-bit cache%s" % (
        rows, prompt_us, a.batch, result["step_us"], a.bits,
        "" if "error" not in result else "; attention off by %.3f of its norm against 16-bit keys and values"
        % result["error"]))
    return result


if __name__ == "__main__":
    main()
