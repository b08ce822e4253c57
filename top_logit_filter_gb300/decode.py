"""Decoding with several hypotheses at once: beams and drafted tokens.

Python face of include/topkp_decode.h, next to the logit filter and with its
manner: CUDA tensors in, the calling thread's current stream, no CPU path.

    score, parent, token = beam_select(logits, scores, n, finished=None, pad_token=0)
    states = beam_reorder(states, parent, lengths=None, out=None)
    cache_write(k, v, slots, k_cache, v_cache, k_exp=None, v_exp=None)
    k, v = cache_read(slots, k_cache, v_cache, k_exp=None, v_exp=None, dtype=None)
    out = tree_attention(q, k_cache, v_cache, context, pages=None, tree=None, ...)

and, for several continuations of one prompt and for drafted tokens:

    out = shared_attention(q, k_cache, v_cache, context, pages, shared, tree=None, ...)
    count, path, token = draft_verify(target, tokens, uniform=None, race=None, draft=None, parent=None, ...)
    states = cache_compact(states, start, keep, kept, pages=None)
    pages, refs, missing = cache_fork(states, pages, lengths, source, refs, grow=0)

A cache is [pages, page_size, heads, dim] with a block table, or
[requests, capacity, heads, dim] without one; its elements are of the rows'
type, or ``torch.float8_e4m3fn`` with a uint8 exponent for each (page, token,
head).  Every call runs forward only: none records a gradient.
"""
from __future__ import annotations

import struct

from . import TopKPError, _lib, _workspace

torch = None    # imported by the first call, as the package itself does
_CODES = {}     # torch dtype -> topkp_dtype
_E4M3 = None    # torch.float8_e4m3fn

# The C structures, packed straight from Python values: a ctypes.Structure
# takes several times as long to fill, which is most of a small call's time.
_CACHE = struct.Struct("=QQi4x6q")
_STATE = struct.Struct("=QQ7q")
_ATTENTION = struct.Struct("=QQQ" + 2 * "QQi4x6q" + "QQQQQQ16qif")
_VERIFY = struct.Struct("=11Q8qif")
_FORK = struct.Struct("=11Q9q")
assert _CACHE.size == _lib.ctypes.sizeof(_lib.Cache) and _STATE.size == _lib.ctypes.sizeof(_lib.State)
assert _ATTENTION.size == _lib.ctypes.sizeof(_lib.TreeAttentionArgs)
assert _VERIFY.size == _lib.ctypes.sizeof(_lib.DraftVerifyArgs)
assert struct.calcsize("=Q4q") == _lib.ctypes.sizeof(_lib.Pages) and _FORK.size == _lib.ctypes.sizeof(_lib.CacheForkArgs)


def _ready():
    """The loaded library; imports torch once."""
    global torch, _E4M3
    if torch is None:
        import torch as module
        _E4M3 = module.float8_e4m3fn
        _CODES.update({module.float32: _lib.TOPKP_F32, module.float16: _lib.TOPKP_F16, module.bfloat16: _lib.TOPKP_BF16})
        torch = module
    return _lib._lib or _lib.load()


def _dtype_code(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32, float16 or bfloat16)")
    return code


def _ptr(t):
    # a present but empty tensor may have no address: any one will do, since empty problems return before it is used
    return 0 if t is None else t.data_ptr() or (16 if t.numel() == 0 else 0)


def _cuda(t, name, dim=None, dtype=None, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (dim is not None and t.dim() != dim):
        raise ValueError(f"{name} must be a {'' if dim is None else str(dim) + '-D '}CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t


def _vec(t, n, dtype, name, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        t = torch.as_tensor(t, dtype=dtype, device=device)
    if t.device != device or t.dtype != dtype or t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be a 1-D {dtype} tensor of length {n} on {device}")
    return t.contiguous()


def _launch(device, call, *args):
    """call(*args, the current stream of device) with that device current."""
    index = device.index
    if index == torch.cuda.current_device():  # the usual case, without the guard's cost
        status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != _lib.TOPKP_SUCCESS:
        raise TopKPError(status, _lib.last_error())


def beam_select(logits, scores, n: int, finished=None, pad_token: int = 0, workspace=None):
    """One step of beam search (topkp_beam_select).

    logits: [B * K, V] CUDA tensor (float32, float16 or bfloat16); scores:
    [B, K] float32, the beams' summed log-probabilities (-inf: no beam);
    finished: [B, K] bool or uint8, beams that go on with ``pad_token`` only,
    at their score.  Returns (score [B, n] float32 descending, parent [B, n]
    int32, token [B, n] int32); a slot without a candidate holds -inf, its
    index mod K and -1.  ``workspace``: a uint8 tensor of at least
    ``beam_select_workspace_size`` bytes (allocated when None)."""
    lib = _ready()
    _cuda(logits, "logits", 2)
    dt, dev = _dtype_code(logits), logits.device
    _cuda(scores, "scores", 2, torch.float32, dev)
    B, K = scores.shape
    R, V = logits.shape
    if R != B * K:
        raise ValueError(f"logits has {R} rows; scores has {B} x {K}")
    if logits.stride(1) != 1 and V > 1:
        logits = logits.contiguous()
    scores = scores.contiguous()
    if finished is not None:
        _cuda(finished, "finished", 2, None, dev)
        if finished.shape != (B, K) or finished.dtype not in (torch.bool, torch.uint8):
            raise ValueError("finished must be a bool or uint8 tensor shaped like scores")
        finished = finished.contiguous()
    n = int(n)
    need = int(lib.topkp_beam_select_workspace_size(B, K, V, dt, n))
    workspace = _workspace(workspace, need, dev)
    score = torch.empty((B, max(n, 0)), dtype=torch.float32, device=dev)
    parent = torch.empty((B, max(n, 0)), dtype=torch.int32, device=dev)
    token = torch.empty((B, max(n, 0)), dtype=torch.int32, device=dev)
    _launch(dev, lib.topkp_beam_select, _ptr(logits), B, K, V, logits.stride(0) if R > 1 else V, dt, _ptr(scores),
            _ptr(finished), int(pad_token), n, _ptr(score), _ptr(parent), _ptr(token), _ptr(workspace),
            workspace.numel())
    return score, parent, token


def beam_select_workspace_size(B: int, K: int, V: int, dtype, n: int) -> int:
    """Bytes of workspace ``beam_select`` needs."""
    return int(_ready().topkp_beam_select_workspace_size(B, K, V, _CODES[dtype], n))


def _layout(t, time_dim, name):
    """(row stride, block stride, blocks, entries, entry bytes) of a state in bytes."""
    es = t.element_size()
    if time_dim == 1 and t.dim() > 1 and t.numel() and t.is_contiguous():  # the usual case
        row = t.numel() // t.shape[0] * es
        return row, row, 1, t.shape[1], row // t.shape[1]
    shape, stride = list(t.shape), list(t.stride())
    if not 1 <= time_dim < max(t.dim(), 2):
        raise ValueError(f"time_dim {time_dim} of a {t.dim()}-D {name}")

    def run(dims):  # (elements, stride of the innermost step) of dimensions that lie densely in each other
        count, step = 1, None
        for d in reversed(dims):
            if shape[d] == 1:
                continue
            if step is None:
                step = stride[d]
            elif stride[d] != step * count:
                raise ValueError(f"{name} must be dense within a row (shape {tuple(shape)}, strides {tuple(stride)})")
            count *= shape[d]
        return count, step

    inner = list(range(time_dim, t.dim()))
    total, step = run(inner)
    if total > 1 and step != 1:
        raise ValueError(f"{name} must be dense within a row (shape {tuple(shape)}, strides {tuple(stride)})")
    entries = shape[time_dim] if t.dim() > 1 else 1
    blocks, block_step = run(list(range(1, time_dim)))
    if 0 in shape:
        return 0, 0, 0, 0, 0
    row = stride[0] if shape[0] > 1 else max(total, (blocks - 1) * (block_step or 0) + total)
    return row * es, (block_step if blocks > 1 else total) * es, blocks, entries, total // entries * es


def beam_reorder(states, parent, lengths=None, time_dim: int = 1, out=None):
    """The beams' states follow their parents (topkp_beam_reorder).

    states: one tensor or a sequence of them, each [B * K, ...] and dense
    within a row, of any dtype; parent: [B, K] int32.  Row b * K + j becomes
    row b * K + parent[b, j], in place, or in ``out`` (tensors like
    ``states``).  lengths: [B, K] int32, how many entries along ``time_dim``
    of each row are live: only they move, and the rest of a destination row
    keeps what it held.  Returns the reordered tensors."""
    lib = _ready()
    single = torch.is_tensor(states)
    src = [states] if single else list(states)
    dst = src if out is None else [out] if torch.is_tensor(out) else list(out)
    if len(dst) != len(src):
        raise ValueError(f"{len(src)} states and {len(dst)} outputs")
    if not torch.is_tensor(parent) or not parent.is_cuda or parent.dim() != 2 or parent.dtype != torch.int32:
        raise ValueError("parent must be a 2-D int32 CUDA tensor")
    dev = parent.device
    B, K = parent.shape
    parent = parent.contiguous()
    if lengths is not None:
        _cuda(lengths, "lengths", 2, torch.int32, dev)
        if lengths.shape != (B, K):
            raise ValueError("lengths must be shaped like parent")
        lengths = lengths.contiguous()
    rows, table = B * K, []
    for i, (s, d) in enumerate(zip(src, dst)):
        shape = s.shape
        for t in (s,) if d is s else (s, d):
            if not isinstance(t, torch.Tensor) or t.device != dev:
                raise ValueError(f"states[{i}] must be a CUDA tensor on {dev}")
            if len(shape) < 1 or shape[0] != rows or t.shape != shape or t.dtype != s.dtype:
                raise ValueError(f"states[{i}] must have {B} x {K} rows, and its output its shape and dtype")
        if len(shape) == 4 and time_dim == 1 and s.is_contiguous() and s.numel():
            # [rows, time, heads, dim], the usual cache
            size = shape[2] * shape[3] * s.element_size()
            row = blk = shape[1] * size
            blocks, entries = 1, shape[1]
        else:
            row, blk, blocks, entries, size = _layout(s, time_dim if len(shape) > 1 else 1, "a state")
        drow, dblk = (row, blk) if d is s or d.stride() == s.stride() else _layout(d, time_dim if len(shape) > 1 else 1, "an output")[:2]
        table.append(_STATE.pack(_ptr(s), _ptr(d), row, drow, blk, dblk, blocks, entries, size))
    _launch(dev, lib.topkp_beam_reorder, b"".join(table), len(src), B, K, _ptr(parent), _ptr(lengths))
    return dst[0] if single else dst


def _cache(t, exp, name, device, row_dtype):
    """The fields of a topkp_cache."""
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_cuda or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-D CUDA tensor on {device}")
    dtype, shape = t.dtype, t.shape
    p0, p1, p2, p3 = t.stride()
    if p3 != 1 and shape[3] > 1:
        raise ValueError(f"{name}: a head's elements must be contiguous")
    if dtype != _E4M3:
        if dtype != row_dtype:
            raise TypeError(f"{name} must be {row_dtype} or torch.float8_e4m3fn, not {dtype}")
        if exp is not None:
            raise ValueError(f"{name}: exponents go with torch.float8_e4m3fn, and only with it")
        return _ptr(t), 0, _CODES[dtype], p0, p1, p2, 0, 0, 0
    if exp is None:
        raise ValueError(f"{name}: exponents go with torch.float8_e4m3fn, and only with it")
    if not isinstance(exp, torch.Tensor) or exp.dtype != torch.uint8 or exp.device != device:
        raise ValueError(f"{name}'s exponents must be a uint8 tensor on {device}")
    if exp.shape != shape[:3]:
        raise ValueError(f"{name}'s exponents must be {tuple(shape[:3])}, not {tuple(exp.shape)}")
    return _ptr(t), _ptr(exp), _lib.TOPKP_E4M3, p0, p1, p2, *exp.stride()


def _pair(k_cache, v_cache):
    if k_cache.shape != v_cache.shape:
        raise ValueError(f"k_cache is {tuple(k_cache.shape)} and v_cache {tuple(v_cache.shape)}")


def cache_write(k, v, slots, k_cache, v_cache, k_exp=None, v_exp=None):
    """Rows of keys and values into a cache (topkp_cache_write).

    k, v: [N, H, D] CUDA tensors (float32, float16 or bfloat16; heads and
    tokens may be strided); slots: [N] int64, page * page_size + place, -1 to
    skip a row; k_cache, v_cache: [pages, page_size, H, D], of the rows'
    dtype, or float8_e4m3fn with k_exp, v_exp [pages, page_size, H] uint8,
    quantised as they are written.  v and v_cache may both be None."""
    lib = _ready()
    _cuda(k, "k", 3)
    dt, dev = _dtype_code(k), k.device
    N, H, D = k.shape
    rows = [k] if v is None else [k, v]
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    for i, t in enumerate(rows):
        _cuda(t, "kv"[i], 3, k.dtype, dev)
        if t.shape != k.shape:
            raise ValueError(f"v is {tuple(t.shape)} and k {tuple(k.shape)}")
        if t.stride(2) != 1 and D > 1:
            rows[i] = t.contiguous()
    _cuda(slots, "slots", 1, torch.int64, dev)
    if slots.shape[0] != N:
        raise ValueError(f"{N} rows and {slots.shape[0]} slots")
    slots = slots.contiguous()
    kc = _cache(k_cache, k_exp, "k_cache", dev, k.dtype)
    vc = None
    if v is not None:
        vc = _cache(v_cache, v_exp, "v_cache", dev, k.dtype)
        _pair(k_cache, v_cache)
    if tuple(k_cache.shape[2:]) != (H, D):
        raise ValueError(f"rows are {H} x {D} and the cache's {tuple(k_cache.shape[2:])}")
    last = rows[-1]
    _launch(dev, lib.topkp_cache_write, _ptr(rows[0]), _ptr(last) if v is not None else None, N, H, D,
            *rows[0].stride()[:2], *last.stride()[:2], dt, _ptr(slots), _CACHE.pack(*kc),
            None if vc is None else _CACHE.pack(*vc), *k_cache.shape[:2])


def cache_read(slots, k_cache, v_cache, k_exp=None, v_exp=None, dtype=None):
    """The cache's entries as dense rows (topkp_cache_read): (k, v), each
    [N, H, D] of ``dtype`` (the cache's own, or any of the three for an e4m3
    cache, bfloat16 when None).  A slot outside the cache gives zeros.
    v_cache may be None; v is then None."""
    lib = _ready()
    _cuda(slots, "slots", 1, torch.int64)
    dev = slots.device
    slots = slots.contiguous()
    _cuda(k_cache, "k_cache", 4, None, dev)
    if dtype is None:
        dtype = torch.bfloat16 if k_cache.dtype == torch.float8_e4m3fn else k_cache.dtype
    kc = _cache(k_cache, k_exp, "k_cache", dev, dtype)
    vc = None
    if v_cache is not None:
        vc = _cache(v_cache, v_exp, "v_cache", dev, dtype)
        _pair(k_cache, v_cache)
    N, (H, D) = slots.shape[0], k_cache.shape[2:]
    k = torch.empty((N, H, D), dtype=dtype, device=dev)
    v = torch.empty((N, H, D), dtype=dtype, device=dev) if vc is not None else None
    _launch(dev, lib.topkp_cache_read, _ptr(slots), N, H, D, _CACHE.pack(*kc),
            None if vc is None else _CACHE.pack(*vc), *k_cache.shape[:2], _dtype_code(k), _ptr(k), _ptr(v))
    return k, v


def _attention_shape(q, k_cache, pages, max_context):
    """An argument block that holds shapes and dtypes only."""
    pool, page_size, Hkv, D = k_cache.shape
    B, T, Hq = q.shape[:3]
    max_pages = 1 if pages is None else pages.shape[1]
    cache = (0, 0, _lib.TOPKP_E4M3 if k_cache.dtype == _E4M3 else _CODES[k_cache.dtype], 0, 0, 0, 0, 0, 0)
    shape = (B, T, Hq, Hkv, D, pool, page_size, max_pages, max_pages,
             max_pages * page_size if max_context is None else int(max_context), 0, 0, 0, 0, 0, 0, _dtype_code(q), 0.0)
    return _ATTENTION.pack(0, 0, 0, *cache, *cache, 0, 0, 0, 0, 0, 0, *shape)


def tree_attention_workspace_size(q, k_cache, pages=None, max_context=None) -> int:
    """Bytes of workspace ``tree_attention`` needs for tensors of these shapes
    and dtypes (their values are not read)."""
    lib = _ready()
    return int(lib.topkp_tree_attention_workspace_size(_attention_shape(q, k_cache, pages, max_context)))


def shared_attention_workspace_size(q, k_cache, pages, groups: int, max_context=None, max_shared=None) -> int:
    """Bytes of workspace ``shared_attention`` needs for tensors of these
    shapes and dtypes (their values are not read) and that many groups."""
    lib = _ready()
    most = pages.shape[1] * k_cache.shape[1] if max_shared is None else int(max_shared)
    return int(lib.topkp_shared_attention_workspace_size(_attention_shape(q, k_cache, pages, max_context), int(groups), most))


def tree_attention(q, k_cache, v_cache, context, pages=None, tree=None, nodes=None, k_exp=None, v_exp=None,
                   scale=None, max_context=None, out=None, want_lse: bool = False, workspace=None):
    """Attention of drafted nodes over a cache and each other (topkp_tree_attention).

    q: [B, T, Hq, D] (float16 or bfloat16); k_cache, v_cache:
    [pages, page_size, Hkv, D] with ``pages`` [B, max_pages] int32 (the block
    table), or [B, capacity, Hkv, D] without; context: [B] int32, tokens in
    the cache before the drafted ones, which stand at context[b] + i.  tree:
    [B, T] int64, bit j of tree[b, i] set where node i sees node j (T <= 64);
    None is a chain, and T = 1 ordinary decoding.  nodes: [B] int32, how many
    of the T nodes a request has.  scale: D ** -0.5 when None.  max_context:
    a bound of ``context`` known on the host, which plans the work (the
    capacity when None).  ``workspace``: a uint8 tensor of at least
    ``tree_attention_workspace_size`` bytes (allocated when None).  Returns
    out ([B, T, Hq, D]), or (out, lse) with lse [B, T, Hq] float32."""
    lib = _ready()
    return _attention(q, k_cache, v_cache, context, pages, tree, nodes, k_exp, v_exp, scale, max_context, out, want_lse, workspace,
                      lib.topkp_tree_attention_workspace_size, lib.topkp_tree_attention, ())


def shared_attention(q, k_cache, v_cache, context, pages, shared, tree=None, nodes=None, k_exp=None, v_exp=None, scale=None,
                     max_context=None, max_shared=None, out=None, want_lse: bool = False, workspace=None):
    """``tree_attention`` of requests that share a prefix, whose keys and
    values are read once for all of them (topkp_shared_attention).

    shared: [groups] int32; the B requests are that many runs of as many
    consecutive ones, and the first shared[g] tokens of group g's requests are
    the same: the same pages (as ``cache_fork`` leaves them) or equal ones.
    max_shared: a bound of ``shared`` known on the host, which plans the work
    (the capacity when None: give it where far less is shared, since what it
    leaves of max_context is planned as the requests' own).  ``workspace``: a uint8 tensor of at least
    ``shared_attention_workspace_size`` bytes (allocated when None).
    Everything else as for ``tree_attention``; the result differs from its by
    the order of the sums only."""
    lib = _ready()
    _cuda(q, "q", 4)
    _cuda(shared, "shared", 1, torch.int32, q.device)
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2:
        raise ValueError("pages must be a 2-D CUDA tensor")
    shared = shared.contiguous()
    groups = shared.shape[0]
    if groups < 1 or q.shape[0] % groups:
        raise ValueError(f"{q.shape[0]} requests do not make {groups} groups")
    most = pages.shape[1] * k_cache.shape[1] if max_shared is None else int(max_shared)
    return _attention(q, k_cache, v_cache, context, pages, tree, nodes, k_exp, v_exp, scale, max_context, out, want_lse, workspace,
                      lambda args: lib.topkp_shared_attention_workspace_size(args, groups, most), lib.topkp_shared_attention,
                      (_ptr(shared), groups, most))


def _attention(q, k_cache, v_cache, context, pages, tree, nodes, k_exp, v_exp, scale, max_context, out, want_lse, workspace, size,
               call, more):
    _cuda(q, "q", 4)
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q must be float16 or bfloat16, not {q.dtype}")
    dev = q.device
    B, T, Hq, D = q.shape
    if D > 1 and q.stride(3) != 1:
        q = q.contiguous()
    kc = _cache(k_cache, k_exp, "k_cache", dev, q.dtype)
    vc = _cache(v_cache, v_exp, "v_cache", dev, q.dtype)
    _pair(k_cache, v_cache)
    pool, page_size, Hkv, Dc = k_cache.shape
    if Dc != D:
        raise ValueError(f"head dimension {D} of q and {Dc} of the cache")
    context = _vec(context, B, torch.int32, "context", dev)
    nodes = _vec(nodes, B, torch.int32, "nodes", dev)
    if pages is not None:
        _cuda(pages, "pages", 2, torch.int32, dev)
        if pages.shape[0] != B:
            raise ValueError(f"pages has {pages.shape[0]} rows and q {B} requests")
        if pages.shape[1] > 1 and pages.stride(1) != 1 or B > 1 and pages.stride(0) < pages.shape[1]:
            pages = pages.contiguous()
    elif pool != B:
        raise ValueError(f"without a block table the cache holds one entry a request ({B}), not {pool}")
    if tree is not None:
        _cuda(tree, "tree", 2, torch.int64, dev)
        if tree.shape != (B, T):
            raise ValueError(f"tree must be {(B, T)}, not {tuple(tree.shape)}")
        tree = tree.contiguous()
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=q.dtype, device=dev)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != dev or (D > 1 and out.stride(3) != 1):
        raise ValueError("out must match q in shape, dtype and device, with its last dimension contiguous")
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    max_pages = 1 if pages is None else pages.shape[1]
    q0, q1, q2, _ = q.stride()
    o0, o1, o2, _ = out.stride()
    shape = (B, T, Hq, Hkv, D, pool, page_size, max_pages,
             0 if pages is None else pages.stride(0) if B > 1 else max_pages,
             max_pages * page_size if max_context is None else int(max_context), q0, q1, q2, o0, o1, o2, _CODES[q.dtype],
             float(D) ** -0.5 if scale is None else float(scale))
    front = (_ptr(q), _ptr(out), _ptr(lse), *kc, *vc, _ptr(pages), _ptr(context), _ptr(nodes), _ptr(tree))
    args = _ATTENTION.pack(*front, 0, 0, *shape)
    need = size(args)
    if need:
        workspace = _workspace(workspace, need, dev)
        args = _ATTENTION.pack(*front, _ptr(workspace), workspace.numel(), *shape)
    _launch(dev, call, args, *more)
    return (out, lse) if want_lse else out


def draft_verify(target, tokens, uniform=None, race=None, draft=None, parent=None, nodes=None, eps: float = 1e-10,
                 want_logprob: bool = False):
    """Which drafted tokens the target accepts, and the token to go on with (topkp_draft_verify).

    target: [B, T, V] CUDA tensor (float32, float16 or bfloat16), the
    target's logits after each node, filtered or not; tokens: [B, T] int32,
    the nodes' tokens (node 0 is the last accepted one); parent: [B, T]
    int32, each node's parent, an earlier node, or None for a chain; draft:
    like target, the logits that the children of a node were drawn from, or
    None where they were not drawn (the best ones, say).  uniform: [B, T]
    float32 of [0, 1), and race: [B, V] float32 of Exp(1), the random numbers
    of acceptance and of the draw; both None is greedy decoding.  nodes: [B]
    int32, how many of the T nodes a request has.

    Returns count [B] int32 (nodes of the accepted path, node 0 included),
    path [B, T] int32 (those nodes, then -1) and token [B] int32, and with
    ``want_logprob`` logprob [B, T] float32: log-probabilities of the
    path's tokens behind node 0's, then of the drawn one."""
    lib = _ready()
    if not isinstance(target, torch.Tensor) or not target.is_cuda or target.dim() != 3:
        raise ValueError("target must be a 3-D CUDA tensor")
    dt, dev = _CODES.get(target.dtype), target.device
    if dt is None:
        raise TypeError(f"unsupported dtype {target.dtype} (float32, float16 or bfloat16)")
    B, T, V = target.shape
    ts = target.stride()
    if ts[2] != 1 and V > 1 or ts[1] < V and T > 1:
        target = target.contiguous()
        ts = target.stride()
    ds = (0, 0)
    if draft is not None:
        _cuda(draft, "draft", 3, target.dtype, dev)
        if draft.shape != target.shape:
            raise ValueError(f"draft is {tuple(draft.shape)} and target {tuple(target.shape)}")
        ds = draft.stride()
        if ds[2] != 1 and V > 1 or ds[1] < V and T > 1:
            draft = draft.contiguous()
            ds = draft.stride()
    if (uniform is None) != (race is None):
        raise ValueError("uniform and race go together")
    if uniform is None and draft is not None:
        raise ValueError("draft goes with uniform and race")
    tokens = _of_nodes(tokens, torch.int32, "tokens", B, T, dev)
    if parent is not None:
        parent = _of_nodes(parent, torch.int32, "parent", B, T, dev)
    ld = V
    if race is not None:
        uniform = _of_nodes(uniform, torch.float32, "uniform", B, T, dev)
        _cuda(race, "race", 2, torch.float32, dev)
        if race.shape != (B, V):
            raise ValueError(f"race must be {(B, V)}, not {tuple(race.shape)}")
        ld, one = race.stride()
        if V > 1 and one != 1 or B > 1 and ld < V:
            race = race.contiguous()
            ld = V
        if B <= 1:
            ld = V
    if nodes is not None:
        nodes = _vec(nodes, B, torch.int32, "nodes", dev)
    count, token = torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    path = torch.empty((B, T), dtype=torch.int32, device=dev)
    logprob = torch.empty((B, T), dtype=torch.float32, device=dev) if want_logprob else None
    args = _VERIFY.pack(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(parent), _ptr(nodes), _ptr(uniform), _ptr(race), _ptr(count),
                        _ptr(path), _ptr(token), _ptr(logprob), B, T, V, ts[0], ts[1] if T > 1 else V, ds[0], ds[1] if T > 1 else V,
                        ld, dt, eps)
    _launch(dev, lib.topkp_draft_verify, args)
    return (count, path, token, logprob) if want_logprob else (count, path, token)


def _of_nodes(t, dtype, name, B, T, device):
    """A tensor with an entry for each node of each request."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.shape != (B, T):
        raise ValueError(f"{name} must be a {(B, T)} tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t.contiguous()


_PACKERS = {}   # by the number of states: their descriptors in one piece


def _page_states(states, time_dim, dev):
    """(tensors, packed descriptors, pages, page size) of a sequence of tensors of pages."""
    many = [states] if isinstance(states, torch.Tensor) else list(states)
    values, like, pages, page_size = [], None, None, None
    for i, t in enumerate(many):
        if not isinstance(t, torch.Tensor) or t.device != dev:
            raise ValueError(f"states[{i}] must be a CUDA tensor on {dev}")
        shape = t.shape
        # layers of one shape lie alike
        if shape != like or t.dtype is not kind or not t.is_contiguous():
            if len(shape) < 2 or not 1 <= time_dim < len(shape):
                raise ValueError(f"states[{i}] must be [pages, page_size, ...] with its tokens along dimension {time_dim}")
            if pages is None:
                pages, page_size = shape[0], shape[time_dim]
            if shape[0] != pages or shape[time_dim] != page_size:
                raise ValueError(f"states[{i}] has {shape[0]} pages of {shape[time_dim]} tokens, others {pages} of {page_size}")
            row, blk, blocks, _, size = _layout(t, time_dim, "a state")
            like, kind = (shape, t.dtype) if t.is_contiguous() else (None, None)
        values += (t.data_ptr() or 16, row, blk, blocks, size)
    n = len(many)
    pack = _PACKERS.get(n) or _PACKERS.setdefault(n, struct.Struct("=" + "Q4q" * n).pack)
    return many, pack(*values), pages, page_size


def cache_fork(states, pages, lengths, source, refs, grow=0, time_dim: int = 1, out=None, refs_out=None, workspace=None):
    """Block tables and pages follow the requests that go on (topkp_cache_fork).

    states: one tensor or a sequence of them, each [pages, page_size, ...] and
    dense within a page, of any dtype (keys, values and exponents of every
    layer); pages: [R, max_pages] int32, the block table; lengths: [R] int32,
    live tokens of its rows; source: [N] int32, the row that each new row goes
    on from (-1: an empty one); refs: [pool] int32, holders of each page; grow:
    tokens that every new row shall have room for besides, or [N] int32.

    Whole pages are shared, a partly filled last one is copied for all but one
    of its rows, what nobody goes on with is freed, and new pages are the free
    ones of the lowest numbers.  Returns (pages [N, max_pages], refs, missing
    [1] int32): with too few free pages nothing happens but that ``missing``
    says how many lack and the new table is all -1.  The new row n holds
    ``lengths[source[n]]`` tokens.  ``out``: where the new table goes;
    ``refs_out``: where the new counts go (``refs`` itself to update it)."""
    lib = _ready()
    _cuda(pages, "pages", 2, torch.int32)
    dev = pages.device
    R, M = pages.shape
    ld, one = pages.stride()
    if M > 1 and one != 1 or R > 1 and ld < M:
        pages = pages.contiguous()
        ld = M
    lengths = _vec(lengths, R, torch.int32, "lengths", dev)
    _cuda(source, "source", 1, torch.int32, dev)
    N = source.shape[0]
    source = source.contiguous()
    _cuda(refs, "refs", 1, torch.int32, dev)
    pool = refs.shape[0]
    if refs_out is None:
        refs = refs.contiguous()
        refs_out = torch.empty(pool, dtype=torch.int32, device=dev)
    else:
        _cuda(refs_out, "refs_out", 1, torch.int32, dev)
        if refs_out.shape != refs.shape or not refs_out.is_contiguous():
            raise ValueError("refs_out must be contiguous and shaped like refs")
        refs = refs.contiguous()
    many, packed, pool_, page_size = _page_states(states, time_dim, dev)
    if not many:
        raise ValueError("no states: the page size is theirs")
    if pool_ != pool:
        raise ValueError(f"refs counts {pool} pages and the states have {pool_}")
    grow_all = 0
    if isinstance(grow, torch.Tensor):
        grow = _vec(grow, N, torch.int32, "grow", dev)
    else:
        grow, grow_all = None, int(grow)
    if out is None:
        out, ld_out = torch.empty((N, M), dtype=torch.int32, device=dev), M
    elif out.shape != (N, M) or out.dtype != torch.int32 or out.device != dev or (M > 1 and out.stride(1) != 1) or (N > 1 and out.stride(0) < M):
        raise ValueError(f"out must be a {(N, M)} int32 tensor on {dev} with contiguous rows")
    else:
        ld_out = out.stride(0) if N > 1 else M
    missing = torch.empty(1, dtype=torch.int32, device=dev)
    workspace = _workspace(workspace, lib.topkp_cache_fork_workspace_size(N, pool), dev)
    held = _lib.ctypes.c_char_p(packed)  # keeps the descriptors where the call reads them
    args = _FORK.pack(_lib.ctypes.cast(held, _lib.ctypes.c_void_p).value, _ptr(pages), _ptr(lengths), _ptr(source), _ptr(grow),
                      _ptr(refs), _ptr(out), _ptr(refs_out), _ptr(missing), _ptr(workspace), workspace.numel(), len(many), R, N, M,
                      ld if R > 1 else M, ld_out, pool, page_size, grow_all)
    _launch(dev, lib.topkp_cache_fork, args)
    return out, refs_out, missing


def cache_fork_workspace_size(N: int, pool: int) -> int:
    """Bytes of workspace ``cache_fork`` needs for N new rows and a pool of that many pages."""
    return int(_ready().topkp_cache_fork_workspace_size(N, pool))


def cache_compact(states, start, keep, kept, pages=None, time_dim: int = 1):
    """The kept tokens of each request move up, in place (topkp_cache_compact).

    states: one tensor or a sequence of them, each [pages, page_size, ...] and
    dense within a page, with ``pages`` [B, max_pages] int32 (the block
    table), or [B, capacity, ...] without; start: [B] int32; keep: [B, W]
    int32, W <= 64; kept: [B] int32.  The token at start[b] + keep[b, j] moves
    to start[b] + j, j < kept[b], where keep[b, j] > j: after ``draft_verify``
    start is the context, keep the path and kept its count.  Returns states."""
    lib = _ready()
    _cuda(keep, "keep", 2, torch.int32)
    dev = keep.device
    B, W = keep.shape
    keep = keep.contiguous()
    start, kept = _vec(start, B, torch.int32, "start", dev), _vec(kept, B, torch.int32, "kept", dev)
    many, packed, pool, page_size = _page_states(states, time_dim, dev)
    if not many:
        return states
    M, ld = 1, 1
    if pages is not None:
        _cuda(pages, "pages", 2, torch.int32, dev)
        if pages.shape[0] != B:
            raise ValueError(f"pages has {pages.shape[0]} rows and keep {B}")
        M = pages.shape[1]
        if M > 1 and pages.stride(1) != 1 or B > 1 and pages.stride(0) < M:
            pages = pages.contiguous()
        ld = pages.stride(0) if B > 1 else M
    elif pool != B:
        raise ValueError(f"without a block table a state holds one entry a request ({B}), not {pool}")
    _launch(dev, lib.topkp_cache_compact, packed, len(many), B, W, _ptr(pages), ld, M, pool, page_size, _ptr(start), _ptr(keep),
            _ptr(kept))
    return states
