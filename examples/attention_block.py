"""One decoder attention block served from quantized weights and a 4-bit
key/value cache:  x -> QKV product -> append -> attention -> O product -> x,
a batch of prompts first, then decoding steps replayed from a HIP graph.

    python examples/attention_block.py [--batch 8] [--prompt 1000] [--steps 32]
                                       [--bits 4] [--window 0] [--sinks 4]

Sizes are those of the benchmark's decoder stack (hidden 4096, 32 query heads
and 8 key/value heads of 128: QKV 6144 x 4096, O 4096 x 4096); weights are
random.  Positions are not encoded: a model that rotates q and k does so with an
operation of its own between the product and the append.  Prints the time of the prompt pass and of a decoding step, and how far
the block's attention is from 16-bit attention over the same keys and values
(what 4 bits cost)."""
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


class AttentionBlock:
    def __init__(self, batch, capacity, bits=4, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, group_size=64,
                 window=0, sinks=0, seed=0):
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

    def buffers(self, rows, max_rows):
        """What a pass over `rows` rows writes, and its scratch."""
        half = dict(dtype=torch.float16, device="cuda")
        b = {"qkv": torch.empty((rows, self.width), **half), "att": torch.empty((rows, self.HQ * self.D), **half),
             "y": torch.empty((rows, self.hidden), **half)}
        linear = max(cider.cider_linear_workspace_bytes_ex(rows, l.N, l.K, l.bits, 0) for l in (self.qkv, self.o))
        b["linear"] = torch.empty(linear, dtype=torch.uint8, device="cuda")
        need = cider.cider_kv4_attention_workspace_bytes(self._batch(rows, max_rows, self.kv_len), self.HQ,
                                                         self.window, self.sinks)
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
        k = b["qkv"][:, self.HQ * self.D:]
        v = b["qkv"][:, (self.HQ + self.H) * self.D:]
        cider.cider_kv4_append(seqs, k, v, F16, ld, ld)
        cider.cider_kv4_attention(seqs, b["qkv"], F16, ld, self.HQ, 1 / math.sqrt(self.D), self.window, self.sinks,
                                  b["attention"], b["attention"].numel(), b["att"], F16, self.HQ * self.D)
        self.o(b["att"], rows, self.HQ * self.D, b["y"], b["linear"])
        return b["y"]


def attention_in_16_bits(block, qkv, lengths):
    """The same rows' attention over their own unquantized keys and values (whole prompts, window 0)."""
    out, lo = [], 0
    for n in lengths:
        q, k, v = (qkv[lo:lo + n].float()[:, a * block.D:b * block.D].view(n, -1, block.D).transpose(0, 1).contiguous()
                   for a, b in ((0, block.HQ), (block.HQ, block.HQ + block.H), (block.HQ + block.H, block.HQ + 2 * block.H)))
        k, v = (t.repeat_interleave(block.HQ // block.H, 0) for t in (k, v))
        s = q @ k.transpose(1, 2).contiguous() / math.sqrt(block.D)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        out.append((torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, -1))
        lo += n
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
    a = p.parse_args(argv)
    if not cider.cider_is_available():
        raise SystemExit("no usable gfx950 device")
    block = AttentionBlock(a.batch, a.prompt + a.steps, a.bits, window=a.window, sinks=a.sinks)
    lengths = [max(1, a.prompt - b * a.prompt // (2 * a.batch)) for b in range(a.batch)]
    rows = sum(lengths)
    i32 = dict(dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), **i32)
    x = torch.randn((rows, block.hidden), device="cuda").half()

    block.kv_len.copy_(torch.tensor(lengths, **i32))
    b = block.buffers(rows, max(lengths))
    prompt_us = timed(lambda: block.forward(x, starts, max(lengths), b), 3)
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
