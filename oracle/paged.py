"""The paged 4-bit cache, the position rotation and causal packed attention.

Test infrastructure only (see oracle/__init__.py).

* Pages: the byte layout of include/tq.h (tq_paged_cache), written from its
  prose, one (token, channel) at a time.
* Codec: the min/max group quantization of ``quant.encode_values`` at 4 bits
  for keys and values alike ("turboquant/audit_claims.py", AUDIT 1).
* Rotation: pair (a, b) of a head row turns by its position's angle; float64
  products and sum, rounded to float32 (the stored codes are of that value).
* Attention: float64 softmax over the cached (dequantized) or given K and V.
"""

from __future__ import annotations

import numpy as np

from . import quant

CELL, GROUP = 16, 32


class PagedSpec:
    """Layout of a pool: d, h_kv, page_tokens, num_pages."""

    def __init__(self, d: int, h_kv: int, page_tokens: int, num_pages: int):
        self.d, self.h_kv, self.page, self.pages = d, h_kv, page_tokens, num_pages
        self.groups = d // GROUP
        self.cell_bytes = 20 * d
        self.cells = page_tokens // CELL
        self.page_bytes = h_kv * self.cells * self.cell_bytes
        P = min(self.groups, 4)
        n = np.arange(CELL)[:, None]
        c = np.arange(d)[None, :]
        j, r = c // 32, c % 32
        s, t, e = n // 8, n % 8 // 2, n % 2
        self.key_byte = (j // P) * 256 * P + n * 16 * P + (r // 8) * 4 * P + (j % P) * 4 + (r % 8) // 2
        self.val_byte = 8 * d + (j // P) * 256 * P + s * 128 * P + ((r // 4) * 4 + t) * 4 * P + (j % P) * 4 + 2 * e + (r % 4) // 2
        self.shift = np.broadcast_to(4 * (r % 2), (CELL, d))
        g = np.arange(self.groups)[None, :]
        G = self.groups
        half = t * 4 * G + g * 4 + s * 2 + e
        sect = 32 * G
        self.key_scale = 16 * d + 2 * half
        self.key_zero = 16 * d + sect + 2 * (n * G + g)
        self.val_scale = 16 * d + 2 * sect + 2 * half
        self.val_zero = 16 * d + 3 * sect + 2 * half

    def nbytes(self) -> int:
        return self.pages * self.page_bytes

    def cell(self, buf: np.ndarray, page: int, h: int, pos: int) -> np.ndarray:
        """The bytes (a view) of the cell of position pos."""
        at = page * self.page_bytes + (h * self.cells + pos % self.page // CELL) * self.cell_bytes
        return buf[at : at + self.cell_bytes]

    def write(self, buf, page: int, h: int, pos: int, key: dict, val: dict, i: int) -> None:
        """Store encoded token i (quant.encode_values of keys and of values) at position pos."""
        cell, n = self.cell(buf, page, h, pos), pos % CELL
        for rec, at in ((key, self.key_byte), (val, self.val_byte)):
            for c in range(self.d):
                k, sh = at[n, c], int(self.shift[n, c])
                cell[k] = (int(cell[k]) & (0xF0 >> sh)) | (int(rec["codes"][i, c]) << sh)
        for x, at in ((key["scale16"], self.key_scale), (key["zero16"], self.key_zero), (val["scale16"], self.val_scale),
                      (val["zero16"], self.val_zero)):
            for g in range(self.groups):
                cell[at[n, g] : at[n, g] + 2] = np.frombuffer(np.float16(x[i, g]).tobytes(), np.uint8)

    def write_sequence(self, buf, table_row, h: int, start: int, key: dict, val: dict) -> None:
        """All encoded tokens, from position start on."""
        for i in range(len(key["codes"])):
            pos = start + i
            self.write(buf, int(table_row[pos // self.page]), h, pos, key, val, i)

    def read(self, buf, table_row, h: int, start: int, count: int):
        """(keys, values) [count, d] float64 that the pages stand for."""
        k, v = np.zeros((count, self.d)), np.zeros((count, self.d))
        for i in range(count):
            pos = start + i
            cell, n = self.cell(buf, int(table_row[pos // self.page]), h, pos), pos % CELL

            def f16(at):
                return np.array([cell[a : a + 2].view(np.float16)[0] for a in at], np.float64).repeat(GROUP)

            k[i] = ((cell[self.key_byte[n]] >> self.shift[n]) & 15) * f16(self.key_scale[n]) + f16(self.key_zero[n])
            v[i] = ((cell[self.val_byte[n]] >> self.shift[n]) & 15) * f16(self.val_scale[n]) + f16(self.val_zero[n])
        return k, v


def rotate(x: np.ndarray, table, positions, interleaved: bool) -> np.ndarray:
    """Rows x [n, heads, d] turned by their positions' angles, rounded to float32 (returned as float64)."""
    y = np.array(x, np.float64)
    if table is None:
        return y
    rot = table.shape[1]
    half = rot // 2
    ang = np.asarray(table, np.float64)[positions][:, None, :]
    z = np.arange(half)
    a, b = (2 * z, 2 * z + 1) if interleaved else (z, z + half)
    w = (y[..., a] + 1j * y[..., b]) * (ang[..., :half] + 1j * ang[..., half:])
    y[..., a], y[..., b] = w.real, w.imag
    return y.astype(np.float32).astype(np.float64)


def encode(x: np.ndarray) -> dict:
    return quant.encode_values(x, 4, GROUP)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, seen: int, scale: float):
    """One query row [d] over the first ``seen`` rows of k and v: (output, sum of p |v| / l, largest sum of |q k| scale)."""
    d = q.shape[0]
    if seen <= 0:
        return np.zeros(d), np.zeros(d), 0.0
    k, v = k[:seen], v[:seen]
    s = k @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * abs(scale))
