"""Norm and rotation of heads (include/cider.h, cider_rotation) in 64 bits by index formulas in numpy, and the bound of
what 32 bits may be off by."""
import numpy as np

from tests import kv4_reference as ref


class Rotation:
    """table float32 [length, rot / 2, 2] (or None), positions int [axes, rows] or None, weights float32 [D] or None."""

    def __init__(self, table=None, interleaved=False, positions=None, pair_axis=None, q_weight=None, k_weight=None,
                 eps=1e-6):
        self.table, self.interleaved, self.positions, self.pair_axis = table, interleaved, positions, pair_axis
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        self.rot = 0 if table is None else 2 * table.shape[1]

    def turns(self, row, p):
        """(cos, sin) float64 [rot / 2] of a row at position p."""
        pairs = np.arange(self.rot // 2)
        if self.positions is None:
            at = np.full(len(pairs), p)
        elif len(self.positions) == 1:
            at = np.full(len(pairs), self.positions[0][row])
        else:
            at = np.asarray(self.positions)[np.asarray(self.pair_axis), row]
        cs = self.table[np.clip(at, 0, len(self.table) - 1), pairs].astype(np.float64)
        return cs[:, 0], cs[:, 1]

    def apply(self, x, weight, row, p):
        """x float64 [heads, D] -> (turned, bound of a 32-bit evaluation without the output's rounding).

        The bound: the mean's root is rounded to 32 bits, then two products, two more and a sum of a pair (or fewer,
        fused): at most six roundings of 2^-24 of |a c| + |b s|, here 2^-21."""
        n = x.copy()
        if weight is not None:
            with np.errstate(over="ignore"):
                n = x * weight.astype(np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(self.eps)))
        out, size = n.copy(), np.abs(n)
        if self.rot:
            c, s = self.turns(row, p)
            i = np.arange(self.rot // 2)
            a, b = (2 * i, 2 * i + 1) if self.interleaved else (i, i + self.rot // 2)
            out[:, a] = n[:, a] * c - n[:, b] * s
            out[:, b] = n[:, b] * c + n[:, a] * s
            size[:, a] = np.abs(n[:, a] * c) + np.abs(n[:, b] * s)
            size[:, b] = np.abs(n[:, b] * c) + np.abs(n[:, a] * s)
        return out, 2.0 ** -21 * size


def half_step(dtype, x):
    """What rounding a value to fp16 (0) or bf16 (1) may be off by, subnormal results included."""
    return np.maximum(np.abs(x) * 2.0 ** (-8 if dtype else -11), 2.0 ** (-134 if dtype else -25))


def put_keys(cache, table, lens, counts, k, v, rotation, gs):
    """Appends the rows' k (turned) and v, float64 [rows, H, D], into a reference cache."""
    row = 0
    for b, (kv, n) in enumerate(zip(lens, counts)):
        for i in range(n):
            p = kv - n + i
            if p >= 0:
                page = table[b][p // 64]
                if 0 <= page < len(cache.data):
                    turned, _ = rotation.apply(k[row], rotation.k_weight, row, p)
                    cache.put(page, p % 64, 0, *ref.quantize(turned, gs))
                    cache.put(page, p % 64, 1, *ref.quantize(v[row], gs))
            row += 1
