"""Plain 64-bit forms of the target-side operators (a request, a row, a head at a time), and
builders of paged caches, for tests/test_gpu_target_*.py."""
import math

import numpy as np
import torch


def cdiv(a, b):
    return -(-a // b)


# ----------------------------------------------------------------------------------------
# plan and commit on lists
# ----------------------------------------------------------------------------------------
def plan(lens, ctx, held, table, free, n_free, page, rows, extra, parent=None):
    """The plan by its definition; table (a list of lists) is updated.  Returns row_off, per-row
    lists and the faults' bits."""
    LEN, PAGE, TREE = 4, 8, 16
    R, W = len(lens), len(table[0])
    bits = 0
    cum_n = cum_need = out = 0
    off, req, pos, slot, anc = [0], [], [], [], []
    new_held = list(held)
    for q in range(R):
        n = lens[q] + extra
        most = 2 ** 31 if parent is None else min(len(parent[q]), 65)
        if n < 0 or ctx[q] < 0 or not 0 <= held[q] <= W or ctx[q] + n > W * page or n > most:
            bits |= LEN
            n = 0
        cum_n += n
        if n and cum_n > rows:
            bits |= LEN
        need = 0
        if cum_n <= rows and n:
            need = max(0, cdiv(ctx[q] + n, page) - held[q])
        before, cum_need = cum_need, cum_need + need
        if n and cum_n <= rows and need and cum_need > n_free:
            bits |= PAGE
            n = 0
        elif cum_n > rows:
            n = 0
        if n:
            for i in range(need):
                table[q][held[q] + i] = free[n_free - 1 - (before + i)]
            out += need
            new_held[q] += need
        paths = []
        for i in range(n):
            up = i - 1
            if parent is not None and i:
                up = parent[q][i]
                if not 0 <= up < i:
                    bits |= TREE
                    up = i - 1
            paths.append((paths[up] if i else []) + ([i] if i else []))
            t = ctx[q] + i
            p = table[q][t // page]
            if p < 0 or (p + 1) * page > 2 ** 31:
                bits |= PAGE
                slot.append(-1)
            else:
                slot.append(p * page + t % page)
            req.append(q)
            pos.append(ctx[q] + len(paths[i]))
            anc.append(sum(1 << (j - 1) for j in paths[i]))
        off.append(off[-1] + n)
    return dict(row_off=off, req=req, position=pos, slot=slot,
                anc=[a - 2 ** 64 if a >= 2 ** 63 else a for a in anc], held=new_held,
                n_free=n_free - out), bits


# ----------------------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------------------
def sees(n, anc=None):
    """[n][n] truth: node i sees node j of its block (anc: the rows' masks, or None)."""
    m = np.tril(np.ones((n, n), bool))
    if anc is not None:
        for i in range(n):
            for j in range(1, n):
                m[i, j] = bool((int(anc[i]) >> (j - 1)) & 1)
            m[i, 0] = True
    return m


def attention(q, K, V, ctx, scale, see):
    """q [n][Hq][D], K and V [ctx + n][Hkv][D], see [n][n]; float64 throughout, over the tokens
    a row sees only.  Returns o [n][Hq][D], lse [n][Hq], and bounds: A = sum_t p_t |V_t| (what
    a relative error of the weights does to o) and S = max_t scale sum_d |q_d K_td| (what the
    products' rounding does to a score)."""
    n, Hq, D = q.shape
    G = Hq // K.shape[1]
    o, A = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, S = np.zeros((n, Hq)), np.zeros((n, Hq))
    for i in range(n):
        idx = np.concatenate([np.arange(ctx), ctx + np.flatnonzero(see[i])])
        for a in range(Hq):
            k, v = K[idx, a // G], V[idx, a // G]
            s = scale * (k @ q[i, a])
            top = s.max()
            p = np.exp(s - top)
            z = p.sum()
            o[i, a] = (p / z) @ v
            A[i, a] = (p / z) @ np.abs(v)
            lse[i, a] = top + math.log(z)
            S[i, a] = scale * (np.abs(k) @ np.abs(q[i, a])).max()
    return o, lse, A, S


def attention_tol(o, lse, A, S, L, D, bf16):
    """Bounds of the kernel's error.  A score is a sum of D products, each step rounded in float:
    off by at most (D + 4) 2^-24 S (the scale's product and the exponent's argument included),
    which moves its weight by that, relatively, and the normaliser again.  Sums over L tokens
    add L 2^-24 each (weights times V, and the weights), and the hardware's exponential and the
    rescalings 32 2^-24.  bf16: each weight and each output rounded, at most 2^-8 of it."""
    u = 2.0 ** -24
    d = (D + 4) * u * S
    rel = 2 * d + (2 * L + 32) * u
    tol = A * rel[..., None] + 1e-30
    if bf16:
        tol = tol + 2.0 ** -8 * (A + np.abs(o))
    return tol, d + (L + 32) * u + 4 * u * np.abs(lse)


class Cache:
    """A paged cache of random contents, its block tables, and the tokens in it as arrays."""

    def __init__(self, seed, ctx, n, Hkv, D, page, dtype, layout="phtd", spare=2, fill=None,
                 held_extra=0):
        import torch
        g = np.random.default_rng(seed)
        held = [cdiv(c + m, page) + held_extra for c, m in zip(ctx, n)]
        P = sum(held) + spare
        order = g.permutation(P)
        W = max(held) + 1
        self.table = np.full((len(ctx), W), -1, np.int32)
        at = 0
        for q, h in enumerate(held):
            self.table[q, :h] = order[at:at + h]
            at += h
        self.held, self.free, self.page, self.P = held, order[at:], page, P
        shape = (P, Hkv, page, D) if layout == "phtd" else (P, page, Hkv, D)
        k, v = (torch.from_numpy(g.standard_normal(shape, np.float32)).to(dtype) for _ in range(2))
        if fill is not None:  # every token that belongs to nobody
            used = np.zeros((P, page), bool)
            for q, (c, m) in enumerate(zip(ctx, n)):
                for t in range(c + m):
                    used[self.table[q, t // page], t % page] = True
            dead = torch.from_numpy(~used)
            for x in (k, v):
                y = x if layout == "pthd" else x.transpose(1, 2)
                y[dead] = fill
        self.layout = layout
        self.k, self.v = k, v

    def dev(self, x):
        x = x.to("cuda:0")
        return x if self.layout == "phtd" else x.transpose(1, 2)

    def tokens(self, x, q, count):
        """[count][Hkv][D] float64 of request q's first tokens."""
        y = (x if self.layout == "phtd" else x.transpose(1, 2)).double().numpy()
        return np.stack([y[self.table[q, t // self.page], :, t % self.page] for t in range(count)])


# ----------------------------------------------------------------------------------------
# logits
# ----------------------------------------------------------------------------------------
def logits(rows, x, hist, prompt, rep, pres, freq, bias, masks):
    """One request: rows [L+1][V] (float64 of the stored values), x drafted tokens, hist its
    tokens with `prompt` of them the prompt's, bias a list of (id, value), masks a list of
    allowed arrays or None.  Returns [L+1][V] and the size of what was added up (for bounds)."""
    V = rows.shape[1]
    out, size = np.empty(rows.shape), np.empty(rows.shape)
    add = dict(bias)
    for j in range(rows.shape[0]):
        gen = list(hist[prompt:]) + list(x[:j])
        cnt = np.bincount(np.asarray(gen, int), minlength=V).astype(float)
        seen = cnt > 0
        seen[np.asarray(hist, int)] = True
        l = rows[j].copy()
        l = np.where(seen, np.where(l > 0, l / rep, l * rep), l)
        size[j] = np.abs(l) + np.abs(freq) * cnt + np.abs(pres)
        l = l - freq * cnt - pres * (cnt > 0)
        for v, b in add.items():
            l[v] += b
            size[j, v] += abs(b)
        if masks[j] is not None:
            l = np.where(masks[j], l, -np.inf)
        out[j] = l
    return out, size
