"""Plain oracle of the 8-bit key/value cache: quantiser, code order, attention.

Independent of the GPU code (numpy, element by element where it matters).
Quantiser in IEEE fp32 rounded after every operation, per block and head:
a = max |finite x| of the call's new tokens, s = a / 127 (the larger of that
and the block's scale where the block goes on), code = clamp(rint(x / s),
-127, 127), 0 for s == 0 or NaN; earlier codes of a block whose scale grew
become rint((code * old) / s).  Attention in fp64 from code * scale.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


def code_of(x, s):
    x = np.asarray(x, F32)
    if not s > 0:
        return np.zeros(x.shape, np.int32)
    with np.errstate(invalid="ignore", over="ignore"):
        t = np.clip(np.rint(x / F32(s)), F32(-127), F32(127))
    return np.where(np.isnan(x), F32(0), t).astype(np.int32)


def key_byte(t, d, D):
    """Byte of slot t, dim d inside the codes of one (block, head) of the keys."""
    return 16 * D * (t // 16) + 1024 * (d // 64) + 16 * ((t % 16) + 16 * ((d // 16) % 4)) + d % 16


def value_byte(t, d, D):
    return (32 * D * (t // 32) + 1024 * (d // 32) + 16 * ((d % 16) + 16 * ((t % 16) // 4))
            + 8 * ((d // 16) % 2) + 4 * ((t // 16) % 2) + t % 4)


class Cache:
    """codes [num_blocks][kv_heads][block_tokens][head_dim] and scales, keys and values."""

    def __init__(self, num_blocks, kv_heads, head_dim, block_tokens):
        shape = (num_blocks, kv_heads, block_tokens, head_dim)
        self.P, self.D = block_tokens, head_dim
        self.codes = {"k": np.zeros(shape, np.int32), "v": np.zeros(shape, np.int32)}
        self.scale = {"k": np.zeros(shape[:2], F32), "v": np.zeros(shape[:2], F32)}
        self.written = np.zeros((num_blocks, block_tokens), bool)

    def write(self, k, v, table, first, offset):
        for b, f in enumerate(first):
            n = offset[b + 1] - offset[b]
            if f < 0:
                continue
            for e in range(f // self.P, (f + n + self.P - 1) // self.P if n else 0):
                if e >= table.shape[1] or not 0 <= table[b, e] < len(self.written):
                    continue
                lo, hi = max(f, e * self.P), min(f + n, (e + 1) * self.P)
                if lo >= hi:
                    continue
                rows = slice(offset[b] + lo - f, offset[b] + hi - f)
                for name, x in (("k", k[rows]), ("v", v[rows])):
                    self._fill(name, table[b, e], lo - e * self.P, np.asarray(x, F32))
                self.written[table[b, e], lo - e * self.P:hi - e * self.P] = True

    def _fill(self, name, blk, slot, x):
        for h in range(x.shape[1]):
            y = x[:, h]
            fin = np.abs(y[np.isfinite(y)])
            a = F32(fin.max()) if fin.size else F32(0)
            s = F32(a / F32(127))
            if slot > 0:
                old = self.scale[name][blk, h]
                if s > old:
                    q = self.codes[name][blk, h, :slot]
                    self.codes[name][blk, h, :slot] = code_of(q.astype(F32) * old, s)
                s = max(s, old)
            self.scale[name][blk, h] = s
            self.codes[name][blk, h, slot:slot + len(y)] = code_of(y, s)

    def values(self, name, table_row, lo, hi):
        """code * scale (fp32) of positions lo .. hi - 1: [tokens][kv_heads][head_dim]."""
        t = np.arange(lo, hi)
        blk = table_row[t // self.P]
        return (self.codes[name][blk, :, t % self.P].astype(F32)
                * self.scale[name][blk][:, :, None].astype(F32))


def sees(length, n, causal=True, window=0):
    """[n][length] which positions each query row sees."""
    p = np.arange(length)[None, :]
    if not causal:
        return np.ones((n, length), bool)
    at = (length - n + np.arange(n))[:, None]
    m = p <= at
    return m & (p > at - window) if window else m


def attention(q, k, v, mask, scale, step=None):
    """One sequence in fp64.  q [n][Hq][D], k, v [L][H][D], mask [n][L], step [L][H] the value
    scales.  Returns out, lse and, for error bounds, (sum_t p_t |v_t|) [n][Hq][D],
    max_t sum_d |q_d k_td| * scale [n][Hq] and max_t p_t step_t [n][Hq]."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    q, k, v = (a.astype(np.float64) for a in (q, k, v))
    out, absum = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, size, big = np.full((n, Hq), -np.inf), np.zeros((n, Hq)), np.zeros((n, Hq))
    some = mask.any(1)
    for h in range(Hq):
        if not some.any():
            break
        x = np.where(mask, q[:, h] @ k[:, h // G].T * scale, -np.inf)[some]
        top = x.max(1, keepdims=True)
        w = np.exp(x - top)
        z = w.sum(1, keepdims=True)
        out[some, h] = w @ v[:, h // G] / z
        absum[some, h] = w @ np.abs(v[:, h // G]) / z
        lse[some, h] = (top + np.log(z))[:, 0]
        if step is not None:
            big[some, h] = (w / z * step[:, h // G].astype(np.float64)).max(1)
        size[some, h] = np.where(mask[some], np.abs(q[some, h]) @ np.abs(k[:, h // G]).T, 0).max(1) * scale
    return out, lse, absum, size, big
