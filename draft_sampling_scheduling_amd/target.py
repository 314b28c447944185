"""The target's side of a decode cycle: binding of include/dspark_target.h.

  cache_plan      rows, pages and cache slots of a step, from lengths on the device
  qk_rope         norms of queries and keys for each head, and the position rotation
  rope_append     the same on the way into the paged cache
  cache_append    the step's keys and values into the paged cache
  tree_attention  the step's rows (a chain, a tree, a piece of a prompt) over the cache
  target_logits   penalties, biases and grammar masks, into the layout verify() reads
  cache_commit    after verify(): accepted path moved, lengths advanced, pages given back
  cache_read      tokens back out of a cache of 4 bits

verify() takes the plan's row_off, so that requests the plan could not serve are left out.
As in the other calls, tensors are device tensors, work goes to the current stream (of the
tensors' device), bad shapes and types raise before anything is enqueued, and faults in the
data set bits of `status` ([1] int32, nullable).  A cache is [n_pages][Hkv][page_size][D]
with any strides over contiguous rows of D: transpose(1, 2) of [n_pages][page_size][Hkv][D]
serves too.  One of 4 bits is k_cache and v_cache [n_pages][Hkv][page_size][D // 2] uint8 (two
elements a byte) with scales [n_pages][Hkv][page_size][2][D // 32] uint8 (a power of two for 32
elements of the keys, then of the values), which the calls take as scales=.
"""
from __future__ import annotations

import ctypes as C

import torch

FAULT_PAGE, FAULT_TREE, FAULT_PARAM = 8, 16, 32
MAX_TREE_NODES = 65
TARGET_EXPORTS = ("dspark_cache_plan_workspace_bytes", "dspark_cache_plan",
                  "dspark_cache_append", "dspark_qk_rope", "dspark_rope_append",
                  "dspark_cache4_append", "dspark_cache4_read",
                  "dspark_tree_attention_workspace_bytes",
                  "dspark_tree_attention", "dspark_tree_attention4_workspace_bytes",
                  "dspark_tree_attention4", "dspark_target_logits",
                  "dspark_target_logits_tree", "dspark_verify_rows",
                  "dspark_cache_commit_workspace_bytes", "dspark_cache_commit", "dspark_cache4_commit")

_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
_U8 = torch.uint8


def set_argtypes(L):
    """ctypes signatures of the library's target-side entry points."""
    i, i64, sz, vp, f = C.c_int, C.c_int64, C.c_size_t, C.c_void_p, C.c_float
    u64 = C.c_uint64
    L.dspark_cache_plan_workspace_bytes.argtypes = [i] * 3
    L.dspark_cache_plan_workspace_bytes.restype = sz
    L.dspark_cache_plan.argtypes = ([i] * 6 + [vp] * 7 + [i] + [vp] * 7 + [sz, vp])
    L.dspark_cache_append.argtypes = ([i] * 6 + [vp] * 2 + [i64] * 2 + [vp] * 4 + [i64] * 3 +
                                      [vp] * 2)
    d = C.c_double
    rope = [vp, vp, i, vp, vp, d, vp]  # position, rope, n_pos, the norms, eps, n_rows
    L.dspark_qk_rope.argtypes = [i] * 7 + [vp, i64] * 2 + rope + [vp, i64] * 2 + [vp] * 2
    L.dspark_rope_append.argtypes = ([i] * 9 + [vp, i64] * 3 + [vp] + rope + [vp, i64] + [vp] * 2 +
                                     [i64] * 3 + [vp] * 2)
    L.dspark_cache4_append.argtypes = ([i] * 9 + [vp, i64] * 3 + [vp] + rope + [vp, i64] + [vp] * 2 +
                                       [i64] * 3 + [vp] + [i64] * 3 + [vp] * 2)
    L.dspark_cache4_read.argtypes = ([i] * 7 + [vp] * 4 + [i64] * 4 + [vp] + [i64] * 4 + [vp] * 4)
    L.dspark_tree_attention_workspace_bytes.argtypes = [i] * 6
    L.dspark_tree_attention_workspace_bytes.restype = sz
    L.dspark_tree_attention.argtypes = ([i] * 9 + [vp, i64] + [vp] * 2 + [i64] * 3 + [vp] * 4 +
                                        [f] + [vp] * 4 + [sz, vp])
    L.dspark_tree_attention4_workspace_bytes.argtypes = [i] * 6
    L.dspark_tree_attention4_workspace_bytes.restype = sz
    L.dspark_tree_attention4.argtypes = ([i] * 9 + [vp, i64] + [vp] * 2 + [i64] * 3 + [vp] + [i64] * 3 +
                                         [vp] * 4 + [f] + [vp] * 4 + [sz, vp])
    L.dspark_target_logits.argtypes = ([i] * 4 + [vp, i64, i] + [vp] * 4 + [i] + [vp] * 7 +
                                       [i, vp, i, i] + [vp] * 4)
    L.dspark_target_logits_tree.argtypes = ([i] * 4 + [vp, i64, i] + [vp] * 5 + [i] + [vp] * 7 +
                                            [i, vp, i, i] + [vp] * 4)
    L.dspark_verify_rows.argtypes = ([i] * 5 + [vp] * 4 + [i] + [vp] * 6 + [u64] * 2 + [vp] * 6 +
                                     [sz, vp])
    L.dspark_cache_commit_workspace_bytes.argtypes = [i] * 3
    L.dspark_cache_commit_workspace_bytes.restype = sz
    L.dspark_cache_commit.argtypes = ([i] * 5 + [vp] * 9 + [i] * 5 + [vp] * 2 + [i64] * 4 +
                                      [vp] * 2 + [sz, vp])
    L.dspark_cache4_commit.argtypes = ([i] * 5 + [vp] * 9 + [i] * 4 + [vp] * 2 + [i64] * 4 + [vp] +
                                       [i64] * 4 + [vp] * 2 + [sz, vp])
    for name in TARGET_EXPORTS:
        if not name.endswith("_bytes"):
            getattr(L, name).restype = i


# ----------------------------------------------------------------------------------------
# checks and calls (a decode step makes many of them, so the passing case costs little: about
# 0.4 us a tensor; what is wrong with one is found out only once something is)
# ----------------------------------------------------------------------------------------
try:  # (there are device tensors by then, so the device's state exists)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
    from torch._C import _cuda_getDevice as _current_device
except ImportError:
    _current_device = torch.cuda.current_device

    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


# (get_device(): a tensor's device index, -1 on the host, at half the cost of its device)
def _dims(t, name, n):
    """Sizes of a tensor of n dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {n}")
    return t.shape


def _refuse(t, name, dev, shape, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _chk(t, name, dev, shape, dtype):
    """One tensor argument; returns its address."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.get_device() == dev.index and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dev, shape, dtype)


def _opt(t, name, dev, shape, dtype):
    """_chk of an argument that may be None (written out: a call less)."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.get_device() == dev.index and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dev, shape, dtype)


def _dt(t, name):
    if t.dtype is _BF16:
        return 1
    if t.dtype is _F32:
        return 0
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _strides(t, last):
    """Strides of the leading dimensions (0 for a dimension of size 1, whose stride is never
    used) of a tensor whose last `last` dimensions are dense; None where they are not."""
    shape, st = t.shape, t.stride()
    n, dense = len(shape) - last, 1
    for k in range(len(shape) - 1, n - 1, -1):
        if st[k] != dense and shape[k] != 1:
            return None
        dense *= shape[k]
    return [s if m != 1 else 0 for s, m in zip(st[:n], shape)]


def _rows(t, name, dev, shape, dtype):
    """A tensor of rows [rows][heads][D], each dense; returns its address and row stride."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or
            t.get_device() != dev.index):
        _refuse(t, name, dev, shape, dtype)
    st = t.stride()
    if st[2] == 1 and st[1] == shape[2] and shape[0] != 1:
        return t.data_ptr(), st[0]
    st = _strides(t, 2)
    if st is None:
        raise ValueError(f"{name} must be dense within a row")
    return t.data_ptr(), st[0]


def _cache(k_cache, v_cache, dev, dims):
    """Addresses, shape and strides of a pair of caches (`dims`: 4, or 5 with a leading layer)."""
    shape = _dims(k_cache, "k_cache", dims)
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if (not isinstance(t, torch.Tensor) or t.get_device() != dev.index or
                t.dtype is not k_cache.dtype or t.shape != shape):
            _refuse(t, name, dev, shape, k_cache.dtype)
    st = k_cache.stride()
    if 1 in shape or st[-1] != 1 or v_cache.stride() != st:
        st = _strides(k_cache, 1)
        if st is None or _strides(v_cache, 1) is None:
            raise ValueError("the caches' last dimension must be contiguous")
        if st != _strides(v_cache, 1):
            raise ValueError("k_cache and v_cache differ in strides")
    return k_cache.data_ptr(), v_cache.data_ptr(), shape, st[:dims - 1]


def _cache4(k_cache, v_cache, scales, dev, dims):
    """_cache of a 4-bit cache and its scales: addresses, shape (with D), strides."""
    Tensor, i = torch.Tensor, dev.index
    if (isinstance(k_cache, Tensor) and isinstance(v_cache, Tensor) and isinstance(scales, Tensor) and
            k_cache.dtype is _U8 and v_cache.dtype is _U8 and scales.dtype is _U8):
        shape, st, vst, sst = k_cache.shape, k_cache.stride(), v_cache.stride(), scales.stride()
        *lead, half = shape
        g = half // 16
        if 1 in lead:  # a dimension of size 1, whose stride is never used
            st, vst, sst = [[0 if n == 1 else a for a, n in zip(x, (*lead, 2, 2))] for x in (st, vst, sst)]
        if (len(lead) == dims - 1 and (g == 2 or g == 4) and st[-1] == 1 and
                v_cache.shape == shape and vst == st and scales.shape == (*lead, 2, g) and
                sst[-1] == 1 and sst[-2] == g and half == 16 * g and k_cache.get_device() == i and
                v_cache.get_device() == i and scales.get_device() == i):
            return (k_cache.data_ptr(), v_cache.data_ptr(), (*lead, 2 * half), st[:-1],
                    scales.data_ptr(), sst[:-2])
    # what is wrong
    kp, vp, shape, st = _cache(k_cache, v_cache, dev, dims)
    if k_cache.dtype is not _U8:
        raise TypeError(f"k_cache must be uint8 beside scales, got {k_cache.dtype}")
    shape = (*shape[:-1], 2 * shape[-1])
    if shape[-1] not in (64, 128):
        raise ValueError(f"a 4-bit cache has heads of 64 or 128 elements, got {shape[-1]}")
    want = (*shape[:-1], 2, shape[-1] // 32)
    if (not isinstance(scales, Tensor) or scales.dtype is not _U8 or scales.shape != want or
            scales.get_device() != i):
        _refuse(scales, "scales", dev, want, _U8)
    sst = _strides(scales, 2)
    if sst is None:
        raise ValueError("a token's scales must be dense")
    return kp, vp, shape, st, scales.data_ptr(), sst


_fns = {}


def _fn(name):
    """The library's function."""
    f = _fns.get(name)
    if f is None:
        from . import lib
        f = _fns[name] = getattr(lib(), name)
    return f


def _call(dev, name, *args):
    """The library's `name`(*args, stream) on `dev`; raises on a refusal."""
    f = _fn(name)
    index = dev.index
    if _current_device() == index:
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(index))
    if rc != 0:
        from . import EWORKSPACE, DsparkError
        if rc == EWORKSPACE:
            raise ValueError("workspace too small")
        raise DsparkError(name, rc)


def _workspace(nbytes, dev):
    """A workspace of its own for one call."""
    if nbytes == 0:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws, ws.data_ptr(), nbytes


def _given(ws, dev):
    """The caller's workspace (the library looks at its size)."""
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a torch.Tensor")
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def cache_plan_workspace_bytes(R, rows, width=0) -> int:
    return _fn("dspark_cache_plan_workspace_bytes")(R, rows, width)


def cache_plan(lens, ctx, held, table, free_pages, n_free, page_size, *, rows, extra=0,
               parent=None, out=None, ws=None, status=None):
    """Rows, pages and slots of a step in which request q brings lens[q] + extra rows behind
    its ctx[q] committed tokens (extra=1: lens is the scheduler's ell, the anchor comes on
    top).  Pages that the rows lack are taken from the end of free_pages[:n_free], in place:
    table [R][max_pages], held [R] and n_free [1] are updated.  parent [R][width]: drafted
    trees (parent[q][i] < i is the node above node i >= 1).  `rows` bounds the step's rows.
    Returns dict(row_off [R+1], req, position, slot [rows], and with parent anc [rows] int64);
    a caller-supplied `out` may leave "req" and "position" out.  Rows behind row_off[-1] are
    left as they were."""
    dev = _device(lens, "lens")
    per = R, = _dims(lens, "lens", 1)
    W, F = _dims(table, "table", 2)[1], _dims(free_pages, "free_pages", 1)[0]
    width = 0 if parent is None else _dims(parent, "parent", 2)[1]
    a = [_chk(lens, "lens", dev, per, _I32), _chk(ctx, "ctx", dev, per, _I32),
         _chk(held, "held", dev, per, _I32), _chk(table, "table", dev, (R, W), _I32),
         _chk(free_pages, "free_pages", dev, (F,), _I32),
         _chk(n_free, "n_free", dev, (1,), _I32),
         _opt(parent, "parent", dev, (R, width), _I32)]
    if out is None:
        out = dict(row_off=torch.empty(R + 1, dtype=_I32, device=dev))
        for k in ("req", "position", "slot"):
            out[k] = torch.empty(rows, dtype=_I32, device=dev)
        if parent is not None:
            out["anc"] = torch.empty(rows, dtype=_I64, device=dev)
    b = [_chk(out["row_off"], "row_off", dev, (R + 1,), _I32),
         _opt(out.get("req"), "req", dev, (rows,), _I32),
         _opt(out.get("position"), "position", dev, (rows,), _I32),
         _chk(out["slot"], "slot", dev, (rows,), _I32),
         None if parent is None else _chk(out["anc"], "anc", dev, (rows,), _I64),
         _opt(status, "status", dev, (1,), _I32)]
    if R == 0:
        out["row_off"].zero_()
        return out
    if ws is None:
        ws, wp, wb = _workspace(cache_plan_workspace_bytes(R, rows, width), dev)
    else:
        ws, wp, wb = _given(ws, dev)
    _call(dev, "dspark_cache_plan", R, rows, page_size, W, F, extra, *a, width, *b, wp, wb)
    return out


def cache_append(k, v, k_cache, v_cache, slot, *, scales=None, n_rows=None, status=None):
    """Row i's keys and values (k, v [rows][Hkv][D], rows any stride apart, as slices of a
    fused projection are) into cache slot slot[i] (-1: skipped).  n_rows: a device int32 [1];
    rows at and behind it are skipped (a plan's row_off[-1:]).  scales: the cache's, if it is one
    of 4 bits."""
    if scales is not None:
        rope_append(None, k, v, k_cache, v_cache, slot, None, None, scales=scales, n_rows=n_rows,
                    status=status)
        return
    dev = _device(k, "k")
    kp, vp, (P, Hkv, page, D), st = _cache(k_cache, v_cache, dev, 4)
    rows = _dims(k, "k", 3)[0]
    dt = _dt(k_cache, "k_cache")
    a, ks = _rows(k, "k", dev, (rows, Hkv, D), k_cache.dtype)
    b, vs = _rows(v, "v", dev, (rows, Hkv, D), k_cache.dtype)
    _call(dev, "dspark_cache_append", rows, Hkv, D, dt, page, P, a, b, ks, vs,
          _chk(slot, "slot", dev, (rows,), _I32), _opt(n_rows, "n_rows", dev, (1,), _I32), kp, vp,
          *st, _opt(status, "status", dev, (1,), _I32))


def _rope_args(dev, rows, D, dtype, position, rope, q_norm, k_norm, eps, n_rows):
    """rot, and the arguments from position to n_rows."""
    n_pos = rot = 0
    pp = tp = None
    if rope is not None:
        n_pos, rot = _dims(rope, "rope", 2)
        pp, tp = _chk(position, "position", dev, (rows,), _I32), _chk(rope, "rope", dev, (n_pos, rot), _F32)
    return rot, (pp, tp, n_pos, None if q_norm is None else _chk(q_norm, "q_norm", dev, (D,), dtype),
                 None if k_norm is None else _chk(k_norm, "k_norm", dev, (D,), dtype), eps,
                 None if n_rows is None else _chk(n_rows, "n_rows", dev, (1,), _I32))


def qk_rope(q, k, position, rope, *, q_norm=None, k_norm=None, eps=1e-6, interleaved=False,
            n_rows=None, out=None, status=None):
    """Queries q [rows][Hq][D] and keys k [rows][Hkv][D] (either may be None; rows any stride apart,
    as slices of a fused projection are), each head divided by its root mean square and multiplied
    by q_norm, k_norm [D] where given, then its pairs (i, i + rot // 2), or with interleaved
    (2 i, 2 i + 1), turned by row position[i] of rope [n_pos][rot] float32 (rot // 2 cosines, then the
    sines; None: nothing turns).  Rows at and behind n_rows (a device int32 [1]), and those whose
    position is not in the table (FAULT_PARAM), are left alone.
    Returns dict(q, k); a caller-supplied `out` may hold q and k themselves."""
    some, name = (k, "k") if q is None else (q, "q")
    dev = _device(some, name)
    rows, _, D = _dims(some, name, 3)
    dtype, dt = some.dtype, _dt(some, name)
    Hq = 0 if q is None else some.shape[1]
    Hkv = 0 if k is None else _dims(k, "k", 3)[1]
    qp, qs = (None, 0) if q is None else _rows(q, "q", dev, (rows, Hq, D), dtype)
    kp, ks = (None, 0) if k is None else _rows(k, "k", dev, (rows, Hkv, D), dtype)
    rot, a = _rope_args(dev, rows, D, dtype, position, rope, q_norm, k_norm, eps, n_rows)
    if out is None:
        out = dict(q=None if q is None else torch.empty((rows, Hq, D), dtype=dtype, device=dev),
                   k=None if k is None else torch.empty((rows, Hkv, D), dtype=dtype, device=dev))
    qo, qos = (None, 0) if q is None else _rows(out["q"], "out['q']", dev, (rows, Hq, D), dtype)
    ko, kos = (None, 0) if k is None else _rows(out["k"], "out['k']", dev, (rows, Hkv, D), dtype)
    sp = None if status is None else _chk(status, "status", dev, (1,), _I32)
    if rows == 0:
        return out
    _call(dev, "dspark_qk_rope", rows, Hq, Hkv, D, rot, interleaved, dt, qp, qs, kp, ks, *a, qo, qos, ko, kos,
          sp)
    return out


def rope_append(q, k, v, k_cache, v_cache, slot, position, rope, *, scales=None, q_norm=None,
                k_norm=None, eps=1e-6, interleaved=False, n_rows=None, out=None, status=None):
    """qk_rope on the way into the cache: row i's keys, normed and turned, and its values as they are
    into cache slot slot[i] (-1: skipped), its queries to `out` [rows][Hq][D] (default: a new tensor;
    may be q itself), which is returned (None without q).  scales: the cache's, if it is one of
    4 bits."""
    dev = _device(k, "k")
    rows, Hkv, D = shape = _dims(k, "k", 3)
    dtype, dt = k.dtype, _dt(k, "k")
    if scales is None:
        kc, vc, (P, heads, page, size), st = _cache(k_cache, v_cache, dev, 4)
        name, more = "dspark_rope_append", ()
        if k_cache.dtype is not dtype:
            raise TypeError(f"k_cache has dtype {k_cache.dtype}, expected {dtype}")
    else:
        kc, vc, (P, heads, page, size), st, scp, sst = _cache4(k_cache, v_cache, scales, dev, 4)
        name, more = "dspark_cache4_append", (scp, *sst)
    if heads != Hkv or size != D:
        raise ValueError(f"k has {Hkv} heads of {D}, the cache {heads} of {size}")
    kp, ks = _rows(k, "k", dev, shape, dtype)
    vp, vs = _rows(v, "v", dev, shape, dtype)
    rot, a = _rope_args(dev, rows, D, dtype, position, rope, q_norm, k_norm, eps, n_rows)
    sl = _chk(slot, "slot", dev, (rows,), _I32)
    if q is None:
        Hq, qp, qs, out, qo, qos = 0, None, 0, None, None, 0
    else:
        Hq = _dims(q, "q", 3)[1]
        qp, qs = _rows(q, "q", dev, (rows, Hq, D), dtype)
        if out is None:
            out = torch.empty((rows, Hq, D), dtype=dtype, device=dev)
        qo, qos = _rows(out, "out", dev, (rows, Hq, D), dtype)
    sp = None if status is None else _chk(status, "status", dev, (1,), _I32)
    _call(dev, name, rows, Hq, Hkv, D, rot, interleaved, dt, page, P, qp, qs, kp, ks, vp, vs, sl, *a, qo, qos,
          kc, vc, *st, *more, sp)
    return out


def cache_read(k_cache, v_cache, scales, slot, *, dtype=_BF16, n_rows=None, out=None, status=None):
    """Tokens of a 4-bit cache as the values they stand for: dict(k, v), [rows][Hkv][D] each for slots
    slot [rows] (of caches with a leading layer dimension [layers][rows][Hkv][D]), in bfloat16 or
    float32 (exact in both).  Rows of slot -1, and at and behind n_rows (a device int32 [1]), are
    left as they were."""
    dev = _device(k_cache, "k_cache")
    if k_cache.dim() == 5:
        kc, vc, (layers, P, Hkv, page, D), st, scp, sst = _cache4(k_cache, v_cache, scales, dev, 5)
        rows, = _dims(slot, "slot", 1)
        want = (layers, rows, Hkv, D)
    else:
        kc, vc, (P, Hkv, page, D), st, scp, sst = _cache4(k_cache, v_cache, scales, dev, 4)
        rows, = _dims(slot, "slot", 1)
        layers, st, sst, want = 1, (0, *st), (0, *sst), (rows, Hkv, D)
    if out is None:
        out = dict(k=torch.empty(want, dtype=dtype, device=dev), v=torch.empty(want, dtype=dtype, device=dev))
    k, v = out["k"], out["v"]
    dt = _dt(k, "out['k']") if isinstance(k, torch.Tensor) else _refuse(k, "out['k']", dev, want, dtype)
    ko, vo = _chk(k, "out['k']", dev, want, k.dtype), _chk(v, "out['v']", dev, want, k.dtype)
    sl = _chk(slot, "slot", dev, (rows,), _I32)
    np = None if n_rows is None else _chk(n_rows, "n_rows", dev, (1,), _I32)
    sp = None if status is None else _chk(status, "status", dev, (1,), _I32)
    _call(dev, "dspark_cache4_read", layers, rows, Hkv, D, dt, page, P, sl, np, kc, vc, *st, scp, *sst, ko, vo,
          sp)
    return out


def tree_attention_workspace_bytes(R, rows, Hq, Hkv, D, dt, four=False) -> int:
    """four: over a cache of 4 bits.  The size for one request with the most rows of any step (R = 1)
    serves all of them."""
    name = "dspark_tree_attention4_workspace_bytes" if four else "dspark_tree_attention_workspace_bytes"
    return _fn(name)(R, rows, Hq, Hkv, D, dt)


def _attention_bytes(name, dev, *sizes):
    """The workspace of a call of these sizes on `dev`, whose compute units it goes by."""
    f = _fn(name + "_workspace_bytes")
    if _current_device() == dev.index:
        nbytes = f(*sizes)
    else:
        with torch.cuda.device(dev):
            nbytes = f(*sizes)
    if nbytes == 0:
        from . import EINVAL, DsparkError
        raise DsparkError(name + "_workspace_bytes", EINVAL)
    return nbytes


def tree_attention(q, k_cache, v_cache, table, ctx, row_off, *, scales=None, anc=None, scale=None, out=None,
                   ws=None, status=None):
    """Attention of a step's packed rows q [rows][Hq][D] over the paged cache, their own keys
    and values appended: every row sees its request's ctx tokens, the anchor (node 0), and of
    the block's further nodes those up to its own (anc=None), or those whose bit is set in
    anc [rows] int64 (a plan's).  scales: the cache's, if it is one of 4 bits (q bfloat16 or float32).
    scale: of the scores, default D ** -0.5.
    Returns dict(o [rows][Hq][D], lse [rows][Hq] float32); a caller-supplied `out` may leave
    "lse" out.  Rows behind row_off[-1] are left as they were."""
    dev = _device(q, "q")
    dt = _dt(q, "q")
    if scales is None:
        kp, vp, (P, Hkv, page, D), st = _cache(k_cache, v_cache, dev, 4)
        name, kind = "dspark_tree_attention", k_cache.dtype
    else:
        kp, vp, (P, Hkv, page, D), st, scp, sst = _cache4(k_cache, v_cache, scales, dev, 4)
        name, kind, st = "dspark_tree_attention4", q.dtype, (*st, scp, *sst)
    rows, Hq, _ = _dims(q, "q", 3)
    qp, qs = _rows(q, "q", dev, (rows, Hq, D), kind)
    R, W = _dims(table, "table", 2)
    a = [_chk(table, "table", dev, (R, W), _I32), _chk(ctx, "ctx", dev, (R,), _I32),
         _chk(row_off, "row_off", dev, (R + 1,), _I32),
         None if anc is None else _chk(anc, "anc", dev, (rows,), _I64)]
    if out is None:
        out = dict(o=torch.empty((rows, Hq, D), dtype=q.dtype, device=dev),
                   lse=torch.empty((rows, Hq), dtype=_F32, device=dev))
    b = [_chk(out["o"], "o", dev, (rows, Hq, D), q.dtype),
         _opt(out.get("lse"), "lse", dev, (rows, Hq), _F32),
         None if status is None else _chk(status, "status", dev, (1,), _I32)]
    if R == 0 or rows == 0:
        return out
    if ws is None:
        ws, wp, wb = _workspace(_attention_bytes(name, dev, R, rows, Hq, Hkv, D, dt), dev)
    else:
        ws, wp, wb = _given(ws, dev)
    _call(dev, name, R, rows, Hq, Hkv, D, dt, page, W, P, qp, qs, kp, vp, *st,
          *a, D ** -0.5 if scale is None else scale, *b, wp, wb)
    return out


def target_logits(logits, ell, x, *, row_off=None, anc=None, hist=None, hist_len=None, prompt_len=None,
                  rep=None, pres=None, freq=None, bias_id=None, bias=None, mask=None,
                  mask_idx=None, out=None, status=None):
    """The target's logits with each request's penalties, biases and grammar masks, in the
    layout verify() takes: out [R][gamma+1][V], row j = 0..ell[q] following the anchor and
    x[q][:j] (x [R][gamma]: the drafted tokens).
    logits: packed [rows][V] with row_off [R+1] (a plan's), or [R][gamma+1][V] without; `out`
    may be logits itself in the latter form.  Rows that row_off does not give a request (one
    that the plan did not serve, say) are left as they were and set FAULT_LEN.
    anc [rows] int64 (a plan's): a tree, row j follows the anchor and the tokens x[q][i-1] of the
    nodes i in its mask.
    hist [R][n] with hist_len [R], prompt_len [R]: each request's tokens, prompt first, anchor
    included; rep divides positive and multiplies other logits of seen ids; pres and freq (times
    the count) are taken off generated ids; bias_id, bias [R][nbias] (-1: unused; the last
    entry for an id counts); mask [n][words] int32: bit v % 32 of word v // 32 allows id v, of
    the mask mask_idx [R][gamma+1] names (-1: none; without mask_idx: mask q * (gamma + 1) + j);
    other ids become -inf."""
    dev = _device(logits, "logits")
    dt = _dt(logits, "logits")
    R, gamma = _dims(x, "x", 2)
    xp = _chk(x, "x", dev, (R, gamma), _I32)
    V = logits.shape[-1]
    if row_off is None:
        lp = _chk(logits, "logits", dev, (R, gamma + 1, V), logits.dtype)
        rows, stride = R * (gamma + 1), V
    else:
        rows = _dims(logits, "logits", 2)[0]
        st = _strides(logits, 1)
        if st is None:
            raise ValueError("rows of logits must be contiguous")
        lp, stride = logits.data_ptr(), st[0] if rows > 1 else V
    if out is None:
        out = torch.empty((R, gamma + 1, V), dtype=logits.dtype, device=dev)
    op = _chk(out, "out", dev, (R, gamma + 1, V), logits.dtype)
    n_hist = nb = n_mask = words = 0
    histp = None
    if hist is not None:
        if hist_len is None:
            raise ValueError("hist needs hist_len")
        n_hist = _dims(hist, "hist", 2)[1]
        histp = _chk(hist, "hist", dev, (R, n_hist), _I32)
        if n_hist == 0:  # (a tensor of no elements has no address)
            histp = xp
    if (bias is None) != (bias_id is None):
        raise ValueError("bias and bias_id come together")
    if bias is not None:
        nb = _dims(bias, "bias", 2)[1]
    if mask is not None:
        n_mask, words = _dims(mask, "mask", 2)
        if mask_idx is None and n_mask < R * (gamma + 1):
            raise ValueError("without mask_idx there is a mask for every row")
    per = (R,)
    name, masks = "dspark_target_logits", ()
    if anc is not None:
        name, masks = "dspark_target_logits_tree", (_chk(anc, "anc", dev, (rows,), _I64),)
    _call(dev, name, R, gamma, V, dt, lp, stride, rows,
          _opt(row_off, "row_off", dev, (R + 1,), _I32), _chk(ell, "ell", dev, per, _I32), xp,
          *masks, histp, n_hist,
          _opt(hist_len, "hist_len", dev, per, _I32),
          _opt(prompt_len, "prompt_len", dev, per, _I32), _opt(rep, "rep", dev, per, _F32),
          _opt(pres, "pres", dev, per, _F32), _opt(freq, "freq", dev, per, _F32),
          _opt(bias_id, "bias_id", dev, (R, nb), _I32), _opt(bias, "bias", dev, (R, nb), _F32), nb,
          _opt(mask, "mask", dev, (n_mask, words), _I32), n_mask, words,
          _opt(mask_idx, "mask_idx", dev, (R, gamma + 1), _I32), op,
          _opt(status, "status", dev, (1,), _I32))
    return out


def cache_commit_workspace_bytes(R, max_pages, moves_in_place=False) -> int:
    return _fn("dspark_cache_commit_workspace_bytes")(R, max_pages, moves_in_place)


def cache_commit(n_acc, ctx, held, table, free_pages, n_free, page_size, *, path=None, done=None,
                 k_cache=None, v_cache=None, scales=None, out=None, ws=None, status=None):
    """After verification: the lengths with the anchor and the n_acc accepted nodes of each
    request committed ([R] int32; `out` may be ctx itself).  path [R][gamma] (trees): the
    accepted nodes, ascending; their keys and values move to the places behind the anchor, in
    the caches ([n_pages][Hkv][page_size][D], or with a leading layer dimension; scales: theirs, if
    they are of 4 bits).  done [R]: finished requests (nonzero) give their pages back: free_pages
    and n_free grow, held and the length become 0."""
    dev = _device(n_acc, "n_acc")
    per = R, = _dims(n_acc, "n_acc", 1)
    W, F = _dims(table, "table", 2)[1], _dims(free_pages, "free_pages", 1)[0]
    gamma = 0 if path is None else _dims(path, "path", 2)[1]
    a = [_chk(n_acc, "n_acc", dev, per, _I32), _opt(path, "path", dev, (R, gamma), _I32),
         _opt(done, "done", dev, per, _I32), _chk(ctx, "ctx", dev, per, _I32)]
    if out is None:
        out = torch.empty(R, dtype=_I32, device=dev)
    b = [_chk(out, "out", dev, per, _I32), _chk(held, "held", dev, per, _I32),
         _chk(table, "table", dev, (R, W), _I32), _chk(free_pages, "free_pages", dev, (F,), _I32),
         _chk(n_free, "n_free", dev, (1,), _I32)]
    name, c = "dspark_cache_commit", [0, 0, 0, 0, 0, None, None, 0, 0, 0, 0]
    if path is not None:
        if k_cache is None or v_cache is None:
            raise ValueError("a path needs the caches")
        if gamma == 0:
            raise ValueError("path has no places")
        dims = 5 if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 5 else 4
        if scales is None:
            kp, vp, shape, st = _cache(k_cache, v_cache, dev, dims)
        else:
            kp, vp, shape, st, scp, sst = _cache4(k_cache, v_cache, scales, dev, dims)
        if dims == 4:
            shape, st = (1, *shape), [0, *st]
        if shape[3] != page_size:
            raise ValueError(f"the caches have pages of {shape[3]} tokens, expected {page_size}")
        if scales is None:
            c = [shape[0], shape[2], shape[4], _dt(k_cache, "k_cache"), shape[1], kp, vp, *st]
        else:
            name = "dspark_cache4_commit"
            c = [shape[0], shape[2], shape[4], shape[1], kp, vp, *st, scp, *([0] if dims == 4 else []), *sst]
    sp = _opt(status, "status", dev, (1,), _I32)
    if R == 0:
        return out
    if ws is None:
        ws, wp, wb = _workspace(
            cache_commit_workspace_bytes(R, W, path is not None and a[3] == b[0]), dev)
    else:
        ws, wp, wb = _given(ws, dev)
    _call(dev, name, R, gamma, page_size, W, F, *a, *b, *c, sp, wp, wb)
    return out
