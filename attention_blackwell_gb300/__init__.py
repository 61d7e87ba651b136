"""GB300-native fused exact attention: a thin ctypes binding over libfa.so.

Every step of the computation runs in the library's CUDA kernels; this module
only marshals arguments (torch tensors -> device pointers, the current CUDA
stream) and turns status codes into exceptions.  It never falls back to any
other implementation: if ``lib/libfa.so`` is missing, every call raises.

Build the library with ``python -m attention_blackwell_gb300.build``.
"""
import ctypes
import os

import torch

__all__ = ["fwd", "set_fwd_kernel", "fwd_pairs_resident", "set_bwd_kernel", "bwd_pairs_resident", "set_schedule_order", "bwd", "bwd_workspace", "page_plan", "page_pool", "kv_store", "prefix_fwd", "prefix_workspace", "exp2_emu", "selftest_timeout", "set_tuning", "set_debug_counters", "device_status", "num_sms", "FAError", "library_path", "lib"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "lib", "libfa.so")
_lib = None

HEAD_DIM = 128


class FAError(RuntimeError):
    """A libfa call returned a non-zero status."""

    def __init__(self, code, what):
        self.code = code
        super().__init__("%s: %s (%d)" % (what, _status_string(code), code))


def library_path():
    return _LIB_PATH


def lib():
    """The loaded libfa.so (ctypes.CDLL); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libfa.so is not built (%s); run `python -m attention_blackwell_gb300.build`"
                               % _LIB_PATH)
        L = ctypes.CDLL(_LIB_PATH)
        vp, i, f, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_status_string.argtypes = [i]
        L.fa_num_sms.restype = i
        L.fa_num_sms.argtypes = []
        L.fa_set_tuning.restype = i
        L.fa_set_tuning.argtypes = [i, f]
        L.fa_set_fwd_kernel.restype = i
        L.fa_set_fwd_kernel.argtypes = [i]
        L.fa_fwd_pairs_resident.restype = i
        L.fa_fwd_pairs_resident.argtypes = []
        L.fa_set_bwd_kernel.restype = i
        L.fa_set_bwd_kernel.argtypes = [i]
        L.fa_bwd_pairs_resident.restype = i
        L.fa_bwd_pairs_resident.argtypes = []
        L.fa_set_schedule_order.restype = i
        L.fa_set_schedule_order.argtypes = [i]
        L.fa_fwd.restype = i
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp]
        sz = ctypes.c_size_t
        L.fa_bwd_workspace_size.restype = sz
        L.fa_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
        L.fa_bwd_stages.restype = i
        L.fa_bwd_stages.argtypes = [i] + [vp] * 9 + [i, i, i, i, i, f, i, vp, i, i, vp, sz, vp]
        L.fa_bwd.restype = i
        L.fa_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, f, i, vp, i, i, vp, sz, vp]
        L.fa_get_device_status.restype = i
        L.fa_get_device_status.argtypes = [vp, vp]
        L.fa_page_plan.restype = i
        L.fa_page_plan.argtypes = [vp, vp, i, i, vp, i, vp, i, vp, vp, vp, vp, vp, i, vp]
        L.fa_kv_store.restype = i
        L.fa_kv_store.argtypes = [vp, vp, i64, i64, vp, i, i, i, vp, vp, i, i, vp]
        L.fa_prefix_workspace_size.restype = sz
        L.fa_prefix_workspace_size.argtypes = [i] * 6
        L.fa_prefix_fwd.restype = i
        L.fa_prefix_fwd.argtypes = [vp, i64, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, i, vp, vp, i, vp, i, vp, sz, vp]
        L.fa_exp2_emu.restype = i
        L.fa_exp2_emu.argtypes = [vp, vp, i64, vp]
        L.fa_selftest_timeout.restype = i
        L.fa_selftest_timeout.argtypes = [vp]
        L.fa_set_debug_counters.restype = i
        L.fa_set_debug_counters.argtypes = [vp, vp, vp]
        _lib = L
    return _lib


def _status_string(code):
    try:
        return lib().fa_status_string(int(code)).decode()
    except Exception:  # library missing while formatting an error
        return "status"


def _check(rc, what):
    if rc != 0:
        raise FAError(rc, what)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def set_bwd_kernel(kernel=0):
    """Backward main kernel for later calls: 0 one CTA per 128-key tile (the
    default), 1 CTA pairs per 256-key block (fixed length, d = 128)."""
    _check(lib().fa_set_bwd_kernel(int(kernel)), "fa_set_bwd_kernel")


def set_schedule_order(order=0):
    """Order of the work units for later calls: 0 the cost-ordered schedule
    (the default), 1 plain enumeration (for testing the scheduler)."""
    _check(lib().fa_set_schedule_order(int(order)), "fa_set_schedule_order")


def bwd_pairs_resident():
    """CTA pairs backward kernel 1 keeps resident (0 before its first launch)."""
    return int(lib().fa_bwd_pairs_resident())


def fwd_pairs_resident():
    """CTA pairs forward kernel 2 keeps resident (0 before its first launch)."""
    return int(lib().fa_fwd_pairs_resident())


def num_sms():
    n = lib().fa_num_sms()
    if n < 0:
        raise FAError(n, "fa_num_sms")
    return n


def set_tuning(exp2_emu_sixteenths=0, tau=8.0):
    """Process-wide forward tuning (sixteenths of exp2 on the FMA pipe, 0-4;
    rescale threshold tau)."""
    _check(lib().fa_set_tuning(int(exp2_emu_sixteenths), float(tau)), "fa_set_tuning")


def set_fwd_kernel(kernel=2):
    """Forward kernel for later calls: 0 ping-pong 128x128 tiles, 2 CTA pairs
    with 256-key blocks (the default)."""
    _check(lib().fa_set_fwd_kernel(int(kernel)), "fa_set_fwd_kernel")


def fwd(q, k, v, causal=False, alpha=None, cu_seqlens=None, max_seqlen=None, out=None, lse=None, stream=None):
    """Forward attention.  Returns (o, lse).

    Fixed length: q [B,N,Hq,d], k/v [B,N,Hkv,d] bf16 -> o like q,
    lse float32 [B,Hq,N].  Varlen: q [T,Hq,d], k/v [T,Hkv,d],
    cu_seqlens int32 [B+1] on the device, max_seqlen -> o [T,Hq,d],
    lse [Hq,T].  d = 128, 64 or 256.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16)
    varlen = cu_seqlens is not None
    if varlen:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        if q.dim() != 3:
            raise ValueError("varlen q must be [T, Hq, d]")
        T, Hq, d = q.shape
        Hkv = k.shape[1]
        B, N = cu_seqlens.numel() - 1, T
        if max_seqlen is None:
            raise ValueError("varlen needs max_seqlen")
        lse_shape = (Hq, T)
    else:
        if q.dim() != 4:
            raise ValueError("q must be [B, N, Hq, d]")
        B, N, Hq, d = q.shape
        Hkv = k.shape[2]
        max_seqlen = N
        lse_shape = (B, Hq, N)
    if k.shape != v.shape or k.shape[:-2] != q.shape[:-2]:
        raise ValueError("k and v must match q's leading shape")
    if alpha is None:
        alpha = 1.0 / (d ** 0.5)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    _need(out, "out", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    rc = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d, float(alpha),
                      1 if causal else 0, _ptr(cu_seqlens), int(max_seqlen), _stream(stream))
    _check(rc, "fa_fwd")
    return out, lse


def _shapes(q, k, cu_seqlens, max_seqlen):
    if cu_seqlens is not None:
        T, Hq, d = q.shape
        return cu_seqlens.numel() - 1, T, Hq, k.shape[1], d, max_seqlen
    B, N, Hq, d = q.shape
    return B, N, Hq, k.shape[2], d, N


def bwd_workspace(B, Hq, N, deterministic=False, varlen=False, device=None, d=HEAD_DIM):
    """A uint8 CUDA tensor large enough for fa_bwd (N = total tokens if varlen)."""
    n = lib().fa_bwd_workspace_size(int(B), int(Hq), int(N), int(d), int(bool(deterministic)), int(bool(varlen)))
    if n == 0:
        raise ValueError("invalid sizes for the backward workspace")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def bwd(q, k, v, o, lse, do, causal=False, alpha=None, cu_seqlens=None, max_seqlen=None, deterministic=False,
        workspace=None, dq=None, dk=None, dv=None, stages=7, stream=None):
    """Backward attention.  Returns (dq, dk, dv); layouts as in fwd, d = 128,
    64 or 256.

    ``stages`` selects the launches (1 preprocess, 2 main, 4 postprocess);
    the default runs all three.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _need(t, n, torch.bfloat16)
    _need(lse, "lse", torch.float32)
    varlen = cu_seqlens is not None
    if varlen:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        if max_seqlen is None:
            raise ValueError("varlen needs max_seqlen")
    B, N, Hq, Hkv, d, ms = _shapes(q, k, cu_seqlens, max_seqlen)
    if alpha is None:
        alpha = 1.0 / (d ** 0.5)
    if workspace is None:
        workspace = bwd_workspace(B, Hq, N, deterministic, varlen, device=q.device, d=d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, n, torch.bfloat16)
    rc = lib().fa_bwd_stages(int(stages), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                             _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, float(alpha), 1 if causal else 0,
                             _ptr(cu_seqlens), int(ms), int(bool(deterministic)), _ptr(workspace),
                             workspace.numel(), _stream(stream))
    _check(rc, "fa_bwd")
    return dq, dk, dv


# A serving step is a few short kernels, so what a call costs on the host counts:
# one expression checks all tensors of a kind and hands over to _need for the
# message, pointers and the stream go to ctypes as plain integers, and only a
# call for another device or stream goes through _elsewhere.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _current_raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _current_raw_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(stream, tensors, call):
    """call() with the tensors' device current and, on it, the given stream or
    that device's current one, which is then where call() allocates.  Tensors
    that the caching allocator holds for another stream are marked as used on
    this one."""
    tensors = [t for t in tensors if t is not None]
    dev = tensors[0].get_device()
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    with torch.cuda.device(dev):
        if stream is None:
            return call()
        if stream.device.index != dev:
            raise ValueError("the stream must be on the tensors' device")
        if stream != torch.cuda.current_stream():
            for t in tensors:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call()


def _one_device(dev, tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")


def _all_int32(**tensors):
    for n, t in tensors.items():
        _need(t, n, torch.int32)


def _rows(t, name):
    """Elements between the tokens of a bf16 [T, H, d] tensor that is dense
    within a token (rows may be cut from a wider projection)."""
    if t.dtype is not torch.bfloat16:
        raise ValueError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must have 3 dimensions" % name)
    T, H, d = shape
    st, sh, sd = t.stride()
    if d > 1 and sd != 1 or H > 1 and sh != d:
        raise ValueError("%s must be contiguous within a token" % name)
    return st if T > 1 else H * d


def _pages(k_pages, v_pages):
    if (k_pages.dtype is not torch.bfloat16 or v_pages.dtype is not torch.bfloat16
            or not k_pages.is_contiguous() or not v_pages.is_contiguous()):
        _need(k_pages, "k_pages", torch.bfloat16)
        _need(v_pages, "v_pages", torch.bfloat16)
    shape = k_pages.shape
    if len(shape) != 4 or shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, d]")
    return shape


def page_pool(num_pages, device=None):
    """(ring, pool) of a cache whose num_pages pages are all free: int32
    [num_pages] and int64 [3], as page_plan takes them."""
    dev = device or "cuda"
    return (torch.arange(num_pages, dtype=torch.int32, device=dev),
            torch.tensor([0, num_pages, 0], dtype=torch.int64, device=dev))


def page_plan(ctx_lens, new_lens, block_table, ring, pool, page_size, num_slots=None, cu_new=None, kv_lens=None,
              slots=None, pool_out=None, stream=None):
    """Pages and slots for a step's new tokens.  Returns (cu_new, kv_lens,
    slots, pool_out); block_table and ring are updated in place.

    ctx_lens, new_lens int32 [B] (new_lens < 0: the request leaves),
    block_table int32 [B, W], ring int32 [num_pages], pool int64 [3] = head,
    tail, missing (see page_pool; missing: pages that could not be given, free
    ones that are no pages included).  -> cu_new int32 [B+1], kv_lens int32 [B],
    slots int32 [num_slots] (-1: none), pool_out int64 [3].  num_slots is needed
    when slots is not given.  No tensor that is written may overlap another:
    kv_lens is another tensor than ctx_lens, pool_out than pool.
    """
    dev, i32 = ctx_lens.get_device(), torch.int32
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(stream, (ctx_lens, new_lens, block_table, ring, pool, cu_new, kv_lens, slots, pool_out),
                          lambda: page_plan(ctx_lens, new_lens, block_table, ring, pool, page_size, num_slots, cu_new,
                                            kv_lens, slots, pool_out))
    B = ctx_lens.numel()
    if slots is None:
        if num_slots is None:
            raise ValueError("page_plan needs num_slots or slots")
        slots = torch.empty(num_slots, dtype=i32, device=ctx_lens.device)
    if cu_new is None:
        cu_new = torch.empty(B + 1, dtype=i32, device=ctx_lens.device)
    if kv_lens is None:
        kv_lens = torch.empty(B, dtype=i32, device=ctx_lens.device)
    if pool_out is None:
        pool_out = torch.empty(3, dtype=torch.int64, device=ctx_lens.device)
    if (ctx_lens.dtype is not i32 or new_lens.dtype is not i32 or block_table.dtype is not i32 or ring.dtype is not i32
            or cu_new.dtype is not i32 or kv_lens.dtype is not i32 or slots.dtype is not i32
            or pool.dtype is not torch.int64 or pool_out.dtype is not torch.int64
            or not ctx_lens.is_contiguous() or not new_lens.is_contiguous() or not block_table.is_contiguous()
            or not ring.is_contiguous() or not cu_new.is_contiguous() or not kv_lens.is_contiguous()
            or not slots.is_contiguous() or not pool.is_contiguous() or not pool_out.is_contiguous()):
        _all_int32(ctx_lens=ctx_lens, new_lens=new_lens, block_table=block_table, ring=ring, cu_new=cu_new,
                   kv_lens=kv_lens, slots=slots)
        _need(pool, "pool", torch.int64)
        _need(pool_out, "pool_out", torch.int64)
    if not (new_lens.get_device() == block_table.get_device() == ring.get_device() == pool.get_device()
            == cu_new.get_device() == kv_lens.get_device() == slots.get_device() == pool_out.get_device() == dev):
        raise ValueError("all tensors must be on one device")
    table = block_table.shape
    if new_lens.numel() != B or len(table) != 2 or table[0] != B:
        raise ValueError("ctx_lens, new_lens and block_table must have one entry or row a request")
    if pool.numel() != 3 or cu_new.numel() != B + 1 or kv_lens.numel() != B or pool_out.numel() != 3:
        raise ValueError("pool and pool_out must have 3 elements, cu_new B + 1 and kv_lens B")
    rc = (_lib or lib()).fa_page_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), B, int(page_size), block_table.data_ptr(),
                                      table[1], ring.data_ptr(), ring.numel(), pool.data_ptr(), pool_out.data_ptr(),
                                      cu_new.data_ptr(), kv_lens.data_ptr(), slots.data_ptr(), slots.numel(),
                                      _current_raw_stream(dev))
    if rc:
        _check(rc, "fa_page_plan")
    return cu_new, kv_lens, slots, pool_out


def kv_store(k, v, slots, k_pages, v_pages, stream=None):
    """Write rows of k and v ([T, Hkv, d] bf16, tokens may be strided) into the
    cache at slots (int32 [T], distinct; negative: skipped).  k_pages and v_pages
    must not overlap (one tensor for both takes one k and v).  Returns (k_pages,
    v_pages)."""
    dev = k_pages.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(stream, (k_pages, v_pages, k, v, slots), lambda: kv_store(k, v, slots, k_pages, v_pages))
    P, Hkv, page, d = _pages(k_pages, v_pages)
    ks, vs = _rows(k, "k"), _rows(v, "v")
    if slots.dtype is not torch.int32 or not slots.is_contiguous():
        _need(slots, "slots", torch.int32)
    if not (v_pages.get_device() == k.get_device() == v.get_device() == slots.get_device() == dev):
        raise ValueError("all tensors must be on one device")
    shape = k.shape
    T = shape[0]
    if shape[1] != Hkv or shape[2] != d or shape != v.shape:
        raise ValueError("k and v must be [T, Hkv, d] with the pages' Hkv and d")
    if slots.numel() != T:
        raise ValueError("slots must have one element a token")
    if T == 0:
        return k_pages, v_pages
    rc = (_lib or lib()).fa_kv_store(k.data_ptr(), v.data_ptr(), ks, vs, slots.data_ptr(), T, Hkv, d, k_pages.data_ptr(),
                                     v_pages.data_ptr(), P, page, _current_raw_stream(dev))
    if rc:
        _check(rc, "fa_kv_store")
    return k_pages, v_pages


def prefix_workspace(B, Hq, Hkv, T, max_seqlen=1, d=HEAD_DIM, device=None):
    """A uint8 CUDA tensor large enough for prefix_fwd of T rows of B requests
    with at most max_seqlen rows each."""
    dev = torch.device(device or "cuda")
    with torch.cuda.device(dev):
        n = lib().fa_prefix_workspace_size(int(T), int(B), int(Hq), int(Hkv), int(d), min(int(max_seqlen), max(int(T), 1)))
        if n == 0:
            raise ValueError("invalid sizes for the prefix workspace")
        return torch.empty(n, dtype=torch.uint8, device=dev)


def prefix_fwd(q, k_pages, v_pages, block_table, kv_lens, cu_seqlens=None, max_seqlen=None, prefix_table=None,
               prefix_len=0, alpha=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens over a prefix that all requests share and each
    request's own paged keys.  Returns (o, lse).

    q [T, Hq, d] bf16 (tokens may be strided), k_pages / v_pages [num_pages,
    Hkv, page_size, d], block_table int32 [B, W], kv_lens int32 [B] (new tokens
    included), prefix_table int32 pages of the prefix's prefix_len tokens ->
    o [T, Hq, d], lse float32 [Hq, T].  Without cu_seqlens (int32 [B+1]) every
    request has one row; with it max_seqlen bounds a request's rows.  out, lse
    and the workspace must not overlap q, the pages or the tables.
    """
    dev, i32 = q.get_device(), torch.int32
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(stream, (q, k_pages, v_pages, block_table, kv_lens, cu_seqlens, prefix_table, out, lse, workspace),
                          lambda: prefix_fwd(q, k_pages, v_pages, block_table, kv_lens, cu_seqlens, max_seqlen,
                                             prefix_table, prefix_len, alpha, out, lse, workspace))
    P, Hkv, page, d = _pages(k_pages, v_pages)
    qs = _rows(q, "q")
    if (block_table.dtype is not i32 or kv_lens.dtype is not i32 or not block_table.is_contiguous()
            or not kv_lens.is_contiguous()):
        _all_int32(block_table=block_table, kv_lens=kv_lens)
    T, Hq, dq = q.shape
    B = kv_lens.numel()
    if dq != d:
        raise ValueError("q and the pages must have one head dim")
    table = block_table.shape
    if len(table) != 2 or table[0] != B:
        raise ValueError("block_table must be [B, W] with kv_lens' B")
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not i32 or not cu_seqlens.is_contiguous():
            _all_int32(cu_seqlens=cu_seqlens)
        if cu_seqlens.numel() != B + 1:
            raise ValueError("cu_seqlens must have B + 1 elements")
        if max_seqlen is None:
            raise ValueError("cu_seqlens needs max_seqlen")
    elif T != B:
        raise ValueError("without cu_seqlens q must have one row a request")
    else:
        max_seqlen = 1
    max_seqlen, prefix_len = min(int(max_seqlen), max(T, 1)), int(prefix_len)
    if prefix_len > 0:
        if prefix_table is None:
            raise ValueError("prefix_len needs prefix_table")
        if prefix_table.dtype is not i32 or not prefix_table.is_contiguous():
            _all_int32(prefix_table=prefix_table)
        if prefix_table.numel() * page < prefix_len:
            raise ValueError("prefix_table is too short for prefix_len")
    else:
        prefix_table = None
    if alpha is None:
        alpha = 1.0 / (d ** 0.5)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    if (out.dtype is not torch.bfloat16 or lse.dtype is not torch.float32 or not out.is_contiguous()
            or not lse.is_contiguous()):
        _need(out, "out", torch.bfloat16)
        _need(lse, "lse", torch.float32)
    if out.shape != (T, Hq, d) or lse.shape != (Hq, T):
        raise ValueError("out must be [T, Hq, d] and lse [Hq, T]")
    if T == 0:
        return out, lse
    if workspace is None:
        workspace = prefix_workspace(B, Hq, Hkv, T, max_seqlen, d, device=q.device)
    if not (k_pages.get_device() == v_pages.get_device() == block_table.get_device() == kv_lens.get_device()
            == out.get_device() == lse.get_device() == workspace.get_device() == dev):
        raise ValueError("all tensors must be on one device")
    _one_device(dev, (cu_seqlens, prefix_table))
    rc = (_lib or lib()).fa_prefix_fwd(q.data_ptr(), qs, k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       T, B, Hq, Hkv, d, alpha, P, page, block_table.data_ptr(), table[1],
                                       kv_lens.data_ptr(), cu_seqlens.data_ptr() if cu_seqlens is not None else None,
                                       max_seqlen, prefix_table.data_ptr() if prefix_table is not None else None,
                                       prefix_len, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                       _current_raw_stream(dev))
    if rc:
        _check(rc, "fa_prefix_fwd")
    return out, lse


def set_debug_counters(visits=None, inner=None, rescales=None):
    """Arm (tensors) or disarm (None) the kernels' debug counters: int32
    visits / inner and int64 rescales[2] CUDA tensors the caller zeroes."""
    for t, n, dt in ((visits, "visits", torch.int32), (inner, "inner", torch.int32), (rescales, "rescales", torch.int64)):
        if t is not None:
            _need(t, n, dt)
    _check(lib().fa_set_debug_counters(_ptr(visits), _ptr(inner), _ptr(rescales)), "fa_set_debug_counters")


def device_status(workspace=None, stream=None):
    """Synchronise the stream and return (and clear) the device status code."""
    return lib().fa_get_device_status(_ptr(workspace), _stream(stream))


def exp2_emu(x, stream=None):
    """The forward kernel's FMA-pipe 2^x on a float32 CUDA tensor."""
    _need(x, "x", torch.float32)
    y = torch.empty_like(x)
    _check(lib().fa_exp2_emu(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "fa_exp2_emu")
    return y


def selftest_timeout(stream=None):
    """Enqueue the failure-detection diagnostic (a bounded wait on a barrier
    nothing arrives at); device_status() afterwards reports the timeout."""
    _check(lib().fa_selftest_timeout(_stream(stream)), "fa_selftest_timeout")
