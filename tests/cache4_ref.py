"""Plain 64-bit forms of the norm and rotation, and of a cache held in 4 bits, for
tests/test_gpu_rope*.py and tests/test_gpu_cache4*.py."""
import numpy as np
import torch

from tests import target_ref as ref

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
NAN = 255


def turn(x, pos, rope, rot, interleaved, w=None, eps=1e-6):
    """x [rows][heads][D] float64, rope [n][rot]; returns the turned heads, and for bounds the sum of
    the sizes that each is added up from."""
    x = x.copy()
    D = x.shape[-1]
    if w is not None:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps) * w
    size = np.abs(x)
    if rope is None:
        return x, size
    h = rot // 2
    c, s = rope[pos][:, None, :h].astype(np.float64), rope[pos][:, None, h:].astype(np.float64)
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, size


def turn_tol(y, size, bf16):
    """Bounds of the float kernel's error, u = 2^-24.  The sum of squares takes at most 8 additions in
    a lane and 5 across lanes, each product rounded with its addition, so mean + eps is off by at most
    16 u of itself, its square root by 9 u, the reciprocal by 10 u, and x f w by 12 u; a product with
    the cosine or sine adds u, the sum another of the result: 14 u of the sizes added up.  One rounding
    to bf16 is 2^-9 of what it rounds, below 2^-8 of the exact value."""
    tol = 14 * 2.0 ** -24 * size
    return tol + (2.0 ** -8 * np.abs(y) if bf16 else 0) + 1e-37


def rope_table(n, rot, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def quantise(x):
    """Codes and bytes of float64 values [.., D], by the definition: powers tried from the smallest
    on, every code's distance looked at."""
    y = x.reshape(-1, 32)
    codes, byte = np.zeros(y.shape, np.uint8), np.zeros(len(y), np.uint8)
    for g, row in enumerate(y):
        if not np.isfinite(row).all():
            byte[g] = NAN
            continue
        top, e = np.abs(row).max(), -120
        while e < 125 and top > 7 * 2.0 ** e:
            e += 1
        byte[g] = e + 127
        far = np.abs(np.abs(row)[:, None] / 2.0 ** e - GRID)
        best = far == far.min(1, keepdims=True)
        lo, hi = best.argmax(1), 7 - best[:, ::-1].argmax(1)
        codes[g] = np.where(lo % 2 == 0, lo, hi) + 8 * np.signbit(row)
    codes = codes.reshape(x.shape)
    return codes[..., 0::2] | codes[..., 1::2] << 4, byte.reshape(*x.shape[:-1], -1)


def values(codes, byte):
    """float64 values of codes [.., D/2] and bytes [.., D/32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    p = np.where(byte == NAN, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return v * np.repeat(p, 32, -1)


class Cache4(ref.Cache):
    """A paged 4-bit cache of random contents: codes kc, vc and scales sc (numpy, [P][Hkv][page]..),
    and k, v, the values they stand for, as ref.Cache has them.  fill: a byte for the scales of
    every token that belongs to nobody."""

    def __init__(self, seed, ctx, n, Hkv, D, page, layout="phtd", spare=2, fill=None, held_extra=0):
        super().__init__(seed, ctx, n, Hkv, D, page, torch.float32, "phtd", spare, None, held_extra)
        g = np.random.default_rng(seed + 1)
        shape = (self.P, Hkv, page)
        self.kc = g.integers(0, 256, (*shape, D // 2), dtype=np.uint8)
        self.vc = g.integers(0, 256, (*shape, D // 2), dtype=np.uint8)
        self.sc = g.integers(122, 128, (*shape, 2, D // 32), dtype=np.uint8)
        if fill is not None:
            used = np.zeros((self.P, page), bool)
            for q, (c, m) in enumerate(zip(ctx, n)):
                for t in range(c + m):
                    used[self.table[q, t // page], t % page] = True
            self.sc.swapaxes(1, 2)[~used] = fill
        self.way = layout
        self.renew()

    def renew(self):
        self.k = torch.from_numpy(values(self.kc, self.sc[..., 0, :]))
        self.v = torch.from_numpy(values(self.vc, self.sc[..., 1, :]))

    def dev4(self):
        """k_cache, v_cache, scales on the device, in the layout asked for."""
        out = []
        for x in (self.kc, self.vc, self.sc):
            t = torch.from_numpy(x)
            if self.way == "pthd":
                t = t.transpose(1, 2).contiguous().to("cuda:0").transpose(1, 2)
            out.append(t.to("cuda:0"))
        return out
