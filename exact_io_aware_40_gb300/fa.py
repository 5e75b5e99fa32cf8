"""ctypes binding of the C ABI in include/fa.h and include/fa_kv4.h (libfa_sm103.so).

Argument marshalling only: every step of attention runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (PyTorch provides device memory and
streams); the library is loaded from this package directory and is never
replaced by another implementation -- if it is missing or cannot load, calls
raise.
"""
import ctypes
import math
import os

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa_sm103.so")
_lib = None


class FAError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s returned %s" % (where, status_string(status)))


def load_library():
    """Load libfa_sm103.so (built by build.py); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("%s is not built; run exact_io_aware_40_gb300/build.py "
                           "(or __graft_entry__.build())" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_kvlen.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp]
    lib.fa_fwd_masked.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp, vp]
    u64 = ctypes.c_uint64
    lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp, f, u64, vp]
    lib.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i,
                                   vp, f, u64, vp, sz, vp]
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_bytes.restype = sz
    lib.fa_fwd_fp8_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_fwd_fp8_workspace_bytes.restype = sz
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, f, f, f, i, vp, vp, sz, vp]
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.fa_bwd_masked.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp,
                                  vp, sz, vp]
    lib.fa_bwd_prepare.argtypes = [vp, vp, i, i, i, i, vp, sz, vp]
    lib.fa_bwd_dkdv.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.fa_bwd_dq.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp]
    lib.fa_bwd_noalloc.restype = ctypes.c_int
    lib.fa_selftest_stalled_wait.argtypes = [ctypes.c_uint64, vp]
    lib.fa_check_error.argtypes = [vp]
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_kv4_page_bytes.argtypes = [i, i, i]
    lib.fa_kv4_page_bytes.restype = sz
    lib.fa_kv4_plan.argtypes = [vp, vp, i, i, i, vp, i, vp, vp, i, vp, vp, vp, vp, vp]
    lib.fa_kv4_append.argtypes = [vp, vp, i, i, i, i, i, i, i, vp, vp, i, i, i, vp]
    lib.fa_kv4_gather.argtypes = [vp, vp, i, i, i, i, i, i, vp, vp, vp]
    lib.fa_kv4_attn_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_kv4_attn_workspace_bytes.restype = sz
    lib.fa_kv4_attn_call_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i, i]
    lib.fa_kv4_attn_call_workspace_bytes.restype = sz
    lib.fa_kv4_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, i, i, i, f,
                                i, i, vp, sz, vp]
    for fn in ("fa_kv4_plan", "fa_kv4_append", "fa_kv4_gather", "fa_kv4_attn",
               "fa_fwd", "fa_fwd_kvlen", "fa_fwd_masked", "fa_bwd", "fa_bwd_masked",
               "fa_fwd_dropout", "fa_bwd_dropout", "fa_fwd_fp8",
               "fa_bwd_prepare", "fa_bwd_dkdv",
               "fa_bwd_dq", "fa_check_error", "fa_selftest_stalled_wait"):
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status):
    return load_library().fa_status_string(int(status)).decode()


fa_status_string = status_string


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, ref):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(ref.device).cuda_stream)


def _check(status, where):
    if status != FA_OK:
        raise FAError(status, where)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    return tuple(int(x) for x in q.shape)


def _expect(t, name, dtype, shape):
    if t is None:
        raise ValueError("%s is required" % name)
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError("%s must be a contiguous CUDA %s tensor of shape %s" % (name, dtype, shape))


# ------------------------------------------------------------------ raw ABI

def fa_fwd(q, k, v, o, L, scale, causal, stream=None):
    """fa_fwd on torch tensors (bf16 [B,H,N,d] q/k/v/o, fp32 [B,H,N] L)."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d,
                                 float(scale), int(bool(causal)), _stream(stream, q)), "fa_fwd")


def fa_fwd_kvlen(q, k, v, o, L, scale, causal, kv_len, stream=None):
    """fa_fwd_kvlen on torch tensors; kv_len is a CUDA int32 [B] tensor or None."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_fwd_kvlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d,
                                       float(scale), int(bool(causal)), _ptr(kv_len),
                                       _stream(stream, q)), "fa_fwd_kvlen")


def fa_fwd_masked(q, k, v, o, L, scale, causal, kv_len, window, block_mask, stream=None):
    """fa_fwd_masked; window is an int (-1: none), block_mask a CUDA uint8
    [ceil(N/128), ceil(N/128)] tensor or None."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d,
                                        float(scale), int(bool(causal)), _ptr(kv_len), int(window),
                                        _ptr(block_mask), _stream(stream, q)), "fa_fwd_masked")


def fa_fwd_dropout(q, k, v, o, L, scale, causal, kv_len, window, block_mask, dropout_p, seed,
                   stream=None):
    """fa_fwd_dropout: the masked forward with dropout (p in [0, 1), 64-bit seed)."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(L), B, H, N, d,
                                         float(scale), int(bool(causal)), _ptr(kv_len),
                                         int(window), _ptr(block_mask), float(dropout_p),
                                         int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream, q)),
           "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, window, block_mask,
                   dropout_p, seed, workspace, stream=None):
    """fa_bwd_dropout on torch tensors (same masks, p and seed as the forward)."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(L),
                                         _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                         int(bool(causal)), _ptr(kv_len), int(window),
                                         _ptr(block_mask), float(dropout_p),
                                         int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(workspace),
                                         workspace.numel(), _stream(stream, q)), "fa_bwd_dropout")


def fa_fwd_fp8_workspace_bytes(B, H, N, d):
    return int(load_library().fa_fwd_fp8_workspace_bytes(B, H, N, d))


def fa_fwd_fp8(q8, k8, v8, o, L, scale, descale_q, descale_k, descale_v, causal, kv_len,
               workspace, stream=None):
    """fa_fwd_fp8: q8/k8/v8 are CUDA uint8 tensors of e4m3 codes [B,H,N,d]; O bf16."""
    B, H, N, d = _shape(q8)
    _check(load_library().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(o), _ptr(L), B, H, N, d,
                                     float(scale), float(descale_q), float(descale_k),
                                     float(descale_v), int(bool(causal)), _ptr(kv_len),
                                     _ptr(workspace), workspace.numel(), _stream(stream, q8)),
           "fa_fwd_fp8")


def fa_bwd_workspace_bytes(B, H, N, d):
    return int(load_library().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, workspace, stream=None):
    """fa_bwd on torch tensors; workspace is a CUDA byte tensor."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(L), _ptr(dq),
                                 _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                                 _ptr(kv_len), _ptr(workspace), workspace.numel(),
                                 _stream(stream, q)), "fa_bwd")


def fa_bwd_masked(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, window, block_mask,
                  workspace, stream=None):
    """fa_bwd_masked on torch tensors (masks as in fa_fwd_masked)."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(L),
                                        _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                        int(bool(causal)), _ptr(kv_len), int(window),
                                        _ptr(block_mask), _ptr(workspace), workspace.numel(),
                                        _stream(stream, q)), "fa_bwd_masked")


def fa_bwd_prepare(o, do, workspace, stream=None):
    """fa_bwd_prepare: D = rowsum(dO * O) into the workspace."""
    B, H, N, d = _shape(o)
    _check(load_library().fa_bwd_prepare(_ptr(o), _ptr(do), B, H, N, d, _ptr(workspace),
                                         workspace.numel(), _stream(stream, o)), "fa_bwd_prepare")


def fa_bwd_dkdv(q, k, v, do, L, dk, dv, scale, causal, kv_len, workspace, stream=None):
    """fa_bwd_dkdv: dK and dV from a prepared workspace."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(L), _ptr(dk),
                                      _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                                      _ptr(kv_len), _ptr(workspace), workspace.numel(),
                                      _stream(stream, q)), "fa_bwd_dkdv")


def fa_bwd_dq(q, k, v, do, L, dq, scale, causal, kv_len, workspace, stream=None):
    """fa_bwd_dq: dQ from a prepared workspace."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(L), _ptr(dq),
                                    B, H, N, d, float(scale), int(bool(causal)), _ptr(kv_len),
                                    _ptr(workspace), workspace.numel(), _stream(stream, q)),
           "fa_bwd_dq")


def fa_bwd_noalloc(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, stream=None):
    """fa_bwd_noalloc: the backward pass with the library's fixed scratch as the
    workspace, for callers that cannot allocate device memory (see fa.h)."""
    B, H, N, d = _shape(q)
    _check(load_library().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(L),
                                         _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                         int(bool(causal)), _ptr(kv_len), _stream(stream, q)),
           "fa_bwd_noalloc")


def fa_selftest_stalled_wait(limit_ns, stream=None):
    """Enqueue the stalled-wait self test; fa_check_error then reports FA_ERR_TIMEOUT."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    _check(load_library().fa_selftest_stalled_wait(int(limit_ns), ctypes.c_void_p(int(stream))),
           "fa_selftest_stalled_wait")


def fa_check_error(stream=None, device=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    _check(load_library().fa_check_error(ctypes.c_void_p(int(stream))), "fa_check_error")


# ------------------------------------------------------------------ convenience

MASK_BLOCK = 128  # block size of block_mask (FA_MASK_BLOCK)


def _same_device(*ts):
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        raise ValueError("all tensors must be on one CUDA device, got %s" % sorted(map(str, devs)))


def _expect_mask(block_mask, N):
    import torch
    if block_mask is not None:
        nb = (N + MASK_BLOCK - 1) // MASK_BLOCK
        _expect(block_mask, "block_mask", torch.uint8, (nb, nb))


def attention_fwd(q, k, v, causal=False, scale=None, kv_len=None, out=None, lse=None, stream=None,
                  window=-1, block_mask=None, dropout_p=0.0, seed=0):
    """Exact attention forward.  Returns (O bf16 [B,H,N,d], L fp32 [B,H,N]).

    window (int, -1 = none) and block_mask (CUDA uint8 [ceil(N/128)]^2 or None)
    select the sliding-window and block-sparse mask terms of fa_fwd_masked."""
    import torch
    B, H, N, d = _shape(q)
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _expect(t, nm, torch.bfloat16, (B, H, N, d))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _expect(out, "out", torch.bfloat16, (B, H, N, d))
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _expect(lse, "lse", torch.float32, (B, H, N))
    if kv_len is not None:
        _expect(kv_len, "kv_len", torch.int32, (B,))
    _same_device(q, k, v, out, lse, kv_len, block_mask)
    with torch.cuda.device(q.device):
        if dropout_p > 0.0:
            _expect_mask(block_mask, N)
            fa_fwd_dropout(q, k, v, out, lse, scale, causal, kv_len, window, block_mask,
                           dropout_p, seed, stream)
        elif window >= 0 or block_mask is not None:
            _expect_mask(block_mask, N)
            fa_fwd_masked(q, k, v, out, lse, scale, causal, kv_len, window, block_mask, stream)
        else:
            fa_fwd_kvlen(q, k, v, out, lse, scale, causal, kv_len, stream)
    return out, lse


def attention_bwd(q, k, v, o, do, L, causal=False, scale=None, kv_len=None, workspace=None,
                  stream=None, window=-1, block_mask=None, dropout_p=0.0, seed=0):
    """Exact attention backward.  Returns (dQ, dK, dV), bf16 [B,H,N,d]."""
    import torch
    B, H, N, d = _shape(q)
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _expect(t, nm, torch.bfloat16, (B, H, N, d))
    _expect(L, "L", torch.float32, (B, H, N))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if kv_len is not None:
        _expect(kv_len, "kv_len", torch.int32, (B,))
    need = fa_bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _expect(workspace, "workspace", torch.uint8, (workspace.numel(),))
    _same_device(q, k, v, o, do, L, kv_len, block_mask, workspace)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    with torch.cuda.device(q.device):
        if dropout_p > 0.0:
            _expect_mask(block_mask, N)
            fa_bwd_dropout(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, window,
                           block_mask, dropout_p, seed, workspace, stream)
        elif window >= 0 or block_mask is not None:
            _expect_mask(block_mask, N)
            fa_bwd_masked(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, window,
                          block_mask, workspace, stream)
        else:
            fa_bwd(q, k, v, o, do, L, dq, dk, dv, scale, causal, kv_len, workspace, stream)
    return dq, dk, dv


# ------------------------------------------------------------------ paged 4-bit cache
#
# A decode step's kernels take a few microseconds, so these calls check their
# arguments with few attribute reads and hand ctypes plain integers.

_KV4_RECORD = {}  # (d, page_size, group) -> bytes of a page of one head


def kv4_page_bytes(d, page_size, group=32):
    """Bytes of one page of one K/V head; raises for an unsupported geometry."""
    n = _KV4_RECORD.get((d, page_size, group))
    if n is None:
        n = int(load_library().fa_kv4_page_bytes(d, page_size, group))
        if n == 0:
            raise ValueError("d must be 64, 128 or 256, page_size 16, 32, 64 or 128 and group 32 "
                             "or 64, got %s, %s, %s" % (d, page_size, group))
        _KV4_RECORD[d, page_size, group] = n
    return n


def kv4_cache(num_pages, kv_heads, page_size, d, group=32, device="cuda"):
    """A cache of num_pages pages: uint8 [num_pages, kv_heads, page bytes], uninitialised
    (rows that were not appended are never used)."""
    import torch
    return torch.empty(num_pages, kv_heads, kv4_page_bytes(d, page_size, group), dtype=torch.uint8,
                       device=device)


def _need(t, name, dtype, shape, dev):
    """Checks a contiguous tensor on CUDA device number `dev`."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _expect(t, name, dtype, tuple(shape))
        raise ValueError("all tensors must be on one CUDA device, %s is on cuda:%d and not cuda:%d"
                         % (name, t.get_device(), dev))


def _need_rows(t, name, dtype, shape, dev):
    """Checks a [tokens, heads, d] tensor of any strides the kernels take; returns its token
    and head strides."""
    ts, hs, cs = t.stride()
    if t.dtype != dtype or t.shape != shape or cs != 1 or t.get_device() != dev:
        raise ValueError("%s must be a %s tensor of shape %s with contiguous channels on the CUDA "
                         "device of the others" % (name, dtype, tuple(shape)))
    if (ts | hs) & 7 or ts > 0x7fffffff or hs > 0x7fffffff or t.data_ptr() & 15:
        ts, hs = ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0  # unused strides are free
        if (ts | hs) & 7 or ts > 0x7fffffff or hs > 0x7fffffff or t.data_ptr() & 15:
            raise ValueError("%s: strides must be multiples of 8 elements (below 2^31) and the "
                             "data 16-byte aligned" % name)
    return ts, hs


def _need_cache(cache, dtype, page_size, d, group):
    """Checks a cache tensor against its geometry; returns (num_pages, kv_heads, device)."""
    if cache.dim() != 3:
        raise ValueError("expected a [num_pages, kv_heads, page bytes] cache")
    pages, heads, record = cache.shape
    dev = cache.get_device()
    want = _KV4_RECORD.get((d, page_size, group)) or kv4_page_bytes(d, page_size, group)
    if record != want or cache.dtype != dtype or dev < 0 or not cache.is_contiguous():
        _expect(cache, "cache", dtype, (pages, heads, want))
    return pages, heads, dev


def _elsewhere(dev, stream, call, *args, **kwargs):
    """call(*args) with device number `dev` current, and `stream` (a raw stream) if one is
    given: what the call allocates then belongs to the stream that uses it."""
    import torch
    if stream is None:
        with torch.cuda.device(dev):
            return call(*args, **kwargs)
    with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=dev)):
        return call(*args, **kwargs)


def kv4_plan(past_len, new_len, block_table, free_list, free_state, page_size, max_tokens,
             num_pages=None, stream=None):
    """One step's pages and slots from the requests' lengths, on the GPU (fa_kv4_plan).

    past_len, new_len: CUDA int32 [B] (new_len -1: the request is finished); block_table int32
    [B, max_pages] and free_list int32 [num_pages] are updated in place; free_state int32 [>= 2]
    (first free entry, number): the state an earlier call returned.  Returns (kv_len [B],
    cu_q [B + 1], slots [max_tokens], state [4])."""
    import torch
    if block_table.dim() != 2:
        raise ValueError("expected a [B, max_pages] block_table")
    B, max_pages = block_table.shape
    n, state_n = free_list.numel(), free_state.numel()
    dev, i32 = past_len.get_device(), torch.int32
    if dev < 0:
        raise ValueError("past_len must be a CUDA tensor")
    _need(past_len, "past_len", i32, (B,), dev)
    _need(new_len, "new_len", i32, (B,), dev)
    _need(block_table, "block_table", i32, (B, max_pages), dev)
    _need(free_list, "free_list", i32, (n,), dev)
    _need(free_state, "free_state", i32, (state_n,), dev)
    if state_n < 2 or not 1 <= max_tokens <= 0x7fffffff or (num_pages is not None and num_pages != n):
        raise ValueError("free_state must hold the first free entry and their number, free_list "
                         "num_pages entries, and max_tokens be positive")
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, kv4_plan, past_len, new_len, block_table, free_list,
                          free_state, page_size, max_tokens)
    at = past_len.device
    kv_len = torch.empty(B, dtype=i32, device=at)
    cu_q = torch.empty(B + 1, dtype=i32, device=at)
    slots = torch.empty(max_tokens, dtype=i32, device=at)
    state = torch.empty(4, dtype=i32, device=at)
    status = load_library().fa_kv4_plan(
        past_len.data_ptr(), new_len.data_ptr(), B, page_size, n, block_table.data_ptr(), max_pages,
        free_list.data_ptr(), free_state.data_ptr(), max_tokens, kv_len.data_ptr(), cu_q.data_ptr(),
        slots.data_ptr(), state.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise FAError(status, "fa_kv4_plan")
    return kv_len, cu_q, slots, state


def kv4_append(k, v, slots, cache, page_size, group=32, stream=None):
    """Quantises k, v (bf16 [T, kv_heads, d], views of a packed projection allowed) and writes
    them to their slots (CUDA int32 [T], -1 skips) in the cache (fa_kv4_append)."""
    import torch
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("expected [T, kv_heads, d] keys and values")
    shape, bf16 = k.shape, torch.bfloat16
    T, heads, d = shape
    pages, cache_heads, dev = _need_cache(cache, torch.uint8, page_size, d, group)
    if heads != cache_heads:
        raise ValueError("k has %d heads, the cache %d" % (heads, cache_heads))
    k_ts, k_hs = _need_rows(k, "k", bf16, shape, dev)
    v_ts, v_hs = _need_rows(v, "v", bf16, shape, dev)
    _need(slots, "slots", torch.int32, (T,), dev)
    if T == 0:
        return
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, kv4_append, k, v, slots, cache, page_size, group)
    status = load_library().fa_kv4_append(
        k.data_ptr(), v.data_ptr(), T, heads, d, k_ts, k_hs, v_ts, v_hs, slots.data_ptr(),
        cache.data_ptr(), pages, page_size, group, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise FAError(status, "fa_kv4_append")


def kv4_gather(slots, cache, page_size, d, group=32, out_k=None, out_v=None, stream=None):
    """The values the cache holds at `slots` (CUDA int32 [T]): bf16 (K, V), each
    [T, kv_heads, d].  Rows whose slot is -1 are not written (fa_kv4_gather)."""
    import torch
    pages, heads, dev = _need_cache(cache, torch.uint8, page_size, d, group)
    T = slots.numel()
    bf16, shape = torch.bfloat16, (T, heads, d)
    _need(slots, "slots", torch.int32, (T,), dev)
    if out_k is not None:
        _need(out_k, "out_k", bf16, shape, dev)
    if out_v is not None:
        _need(out_v, "out_v", bf16, shape, dev)
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, kv4_gather, slots, cache, page_size, d, group, out_k, out_v)
    if out_k is None:
        out_k = torch.empty(shape, dtype=bf16, device=cache.device)
    if out_v is None:
        out_v = torch.empty(shape, dtype=bf16, device=cache.device)
    if T:
        status = load_library().fa_kv4_gather(
            slots.data_ptr(), cache.data_ptr(), pages, page_size, group, T, heads, d,
            out_k.data_ptr(), out_v.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
        if status:
            raise FAError(status, "fa_kv4_gather")
    return out_k, out_v


def kv4_attention_workspace_bytes(q_heads, kv_heads, d, max_q):
    return int(load_library().fa_kv4_attn_workspace_bytes(q_heads, kv_heads, d, max_q))


def kv4_attention(q, cache, block_table, cu_q, kv_len, max_q, page_size, group=32, causal=True,
                  scale=None, window=-1, out=None, lse=None, workspace=None, stream=None):
    """Exact attention of new tokens over the cache (fa_kv4_attn).

    q: bf16 [total_q, q_heads, d], the requests' new tokens one after the other (views of a
    packed projection allowed); block_table int32 [B, max_pages]; cu_q int32 [B + 1] (request b
    has rows cu_q[b] .. cu_q[b + 1] - 1, at most max_q of them, its last tokens); kv_len int32
    [B], new tokens included.  Query heads h * q_heads / kv_heads .. share K/V head h.  Returns
    (O bf16 [total_q, q_heads, d], L fp32 [total_q, q_heads]); rows behind the last request are
    not written.  A workspace (uint8, kv4_attention_workspace_bytes) must not be shared by
    calls that may overlap."""
    import torch
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("expected [total_q, q_heads, d] queries and a [B, max_pages] block_table")
    shape, bf16, i32 = q.shape, torch.bfloat16, torch.int32
    total, q_heads, d = shape
    pages, kv_heads, dev = _need_cache(cache, torch.uint8, page_size, d, group)
    B, max_pages = block_table.shape
    q_ts, q_hs = _need_rows(q, "q", bf16, shape, dev)
    if q_heads % kv_heads:
        raise ValueError("%d query heads do not divide into %d K/V heads" % (q_heads, kv_heads))
    if not 1 <= max_q <= 0x7fffffff or not -1 <= window <= 0x7fffffff or total > 0x7fffffff:
        raise ValueError("max_q must be positive, window at least -1, and sizes below 2^31")
    _need(block_table, "block_table", i32, (B, max_pages), dev)
    _need(cu_q, "cu_q", i32, (B + 1,), dev)
    _need(kv_len, "kv_len", i32, (B,), dev)
    if out is not None:
        _need(out, "out", bf16, shape, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (total, q_heads), dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _elsewhere(dev, stream, kv4_attention, q, cache, block_table, cu_q, kv_len, max_q,
                          page_size, group, causal, scale, window, out, lse, workspace)
    at = q.device
    if out is None:
        out = torch.empty(shape, dtype=bf16, device=at)
    if lse is None:
        lse = torch.empty((total, q_heads), dtype=torch.float32, device=at)
    if total == 0 or B == 0:
        return out, lse
    lib = load_library()
    space = None  # the workspace's address
    if workspace is None:
        size = lib.fa_kv4_attn_call_workspace_bytes(B, total, max_q, q_heads, kv_heads, d, max_pages,
                                                    page_size, window)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=at)
            space = workspace.data_ptr()
    else:
        space, size = workspace.data_ptr(), workspace.numel()
    status = lib.fa_kv4_attn(
        q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(),
        out.data_ptr(), lse.data_ptr(), B, total, max_q, q_heads, kv_heads, d, q_ts, q_hs, pages,
        max_pages, page_size, group, 1.0 / math.sqrt(d) if scale is None else float(scale),
        1 if causal else 0, window, space, size,
        torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise FAError(status, "fa_kv4_attn")
    return out, lse


# ------------------------------------------------------------------ autograd

_FLASH_FN = None


def _flash_function():
    """The torch.autograd.Function over attention_fwd / attention_bwd (built on
    first use so that importing this module does not import torch)."""
    global _FLASH_FN
    if _FLASH_FN is None:
        import torch

        class FlashAttnFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, causal, scale, kv_len, window, block_mask, dropout_p, seed):
                o, L = attention_fwd(q, k, v, causal=causal, scale=scale, kv_len=kv_len,
                                     window=window, block_mask=block_mask,
                                     dropout_p=dropout_p, seed=seed)
                ctx.save_for_backward(q, k, v, o, L)
                ctx.rest = (causal, scale, kv_len, window, block_mask, dropout_p, seed)
                ctx.mark_non_differentiable(L)
                return o, L

            @staticmethod
            def backward(ctx, do, _dL):
                q, k, v, o, L = ctx.saved_tensors
                causal, scale, kv_len, window, block_mask, dropout_p, seed = ctx.rest
                dq, dk, dv = attention_bwd(q, k, v, o, do.contiguous(), L, causal=causal,
                                           scale=scale, kv_len=kv_len, window=window,
                                           block_mask=block_mask, dropout_p=dropout_p, seed=seed)
                return dq, dk, dv, None, None, None, None, None, None, None

        _FLASH_FN = FlashAttnFunction
    return _FLASH_FN


def flash_attn_func(q, k, v, causal=False, softmax_scale=None, kv_len=None, window=-1,
                    block_mask=None, dropout_p=0.0, seed=0, return_lse=False):
    """Exact attention as a differentiable op: O = softmax(scale * Q K^T + mask) V.

    The drop-in form of the method's interface (bxzpzcl.cn article, section
    "5分钟快速部署指南", basic usage example: Q, K, V and a causal flag in, the
    attention output out) with torch autograd: the backward runs
    attention_bwd, recomputing P from the saved logsumexp L.  Tensors are
    contiguous bf16 CUDA [B, H, N, d] (heads before tokens); softmax_scale
    defaults to 1/sqrt(d); the mask and dropout arguments are those of
    attention_fwd.  Returns O, or (O, L) with return_lse (L is not
    differentiable)."""
    d = q.shape[-1]
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    o, L = _flash_function().apply(q, k, v, bool(causal), scale, kv_len, int(window), block_mask,
                                   float(dropout_p), int(seed))
    return (o, L) if return_lse else o
