"""One rank's shard of a paged key-value cache: append, decode attention, accumulated attention
weights and eviction (include/dcp_paged.h).

A decode step of one rank:

    dcp_kv_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc, shard=r, num_shards=N)
    send = paged_attention_pack(q, k_cache, v_cache, block_table, seq_lens, N, shard=r, num_shards=N, logits=logits)
    ...                                                 # exchange of the send buffers
    out, lse = unpack_combine(recv, return_lse=True)    # this rank's heads, LSE over all shards
    dcp_kv_weights(logits, all_heads_lse, seq_lens, weights, shard=r, num_shards=N)

and, when the local cache is over its budget,

    kept, new_lens, weights = kv_evict(weights, k_cache, v_cache, block_table, seq_lens, new_block_table, keep, recent,
                                       shard=r, num_shards=N)

after which new_lens are this rank's lengths (num_shards = 1).  A token that follows goes to the rank
that owns its position p in the request, (p // interleave) % N, and only there: that rank's length grows by one,
and in dcp_kv_append a length of 0 leaves out the token of a request.  On the device, with `lens` this
rank's lengths and `total` the requests' lengths with the new token:

    own = (total - 1) // interleave % N == r
    lens += own
    dcp_kv_append(k_new, v_new, k_cache, v_cache, block_table, torch.where(own, lens, 0), query_start_loc)
    send = paged_attention_pack(q, k_cache, v_cache, block_table, lens, N, logits=logits)

The cache is any pair of [pages, page_size, heads, D] views whose last dimension is contiguous
(permute a [pages, heads, page_size, D] pool); local position p of request b is slot p % page_size
of page block_table[b, p // page_size].  Lengths and tables stay on the device, so a call can be
captured into a CUDA graph and replayed with other lengths.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import threading
import warnings

import torch

# the package defines these before it imports this module
from . import DCPError, _build, _code, _cuda, _stream, dcp_last_error, dcp_lse_pack_dim, library

_i32, _i64, _ptr, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class _PagedKV(ctypes.Structure):
    """dcp_paged_kv of include/dcp_paged.h."""
    _fields_ = [("k", _ptr), ("v", _ptr), ("block_table", _ptr), ("num_pages", _i64),
                ("k_stride_page", _i64), ("k_stride_slot", _i64), ("k_stride_head", _i64),
                ("v_stride_page", _i64), ("v_stride_slot", _i64), ("v_stride_head", _i64),
                ("table_stride", _i64), ("max_pages", _i64),
                ("page_size", _i32), ("heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the paged calls of libdcpcombine.so."""
    kv = ctypes.POINTER(_PagedKV)
    lib.dcp_paged_attention_workspace.argtypes = [_i64, _i32, _i32, _i32]
    lib.dcp_paged_attention_workspace.restype = _i64
    lib.dcp_paged_attention.argtypes = [kv, _ptr, _ptr, _ptr, _ptr, _ptr, _i64, _i64, _i64, _i64, _i64, _i64, _i64,
                                        _f32, _i32, _i32, _i32, _i32, _ptr, _i64, _ptr]
    lib.dcp_paged_attention.restype = _i32
    lib.dcp_paged_attention_pack.argtypes = [kv, _ptr, _ptr, _ptr, _ptr, _i64, _i64, _i32, _i64, _i64, _i64, _i64,
                                             _i64, _f32, _i32, _i32, _i32, _i32, _ptr, _i64, _ptr]
    lib.dcp_paged_attention_pack.restype = _i32
    lib.dcp_testing_paged_attention_stalled.argtypes = [kv, _ptr, _ptr, _ptr, _ptr, _i64, _i64, _i64, _i64, _f32, _ptr,
                                                        _i64, _ptr]
    lib.dcp_testing_paged_attention_stalled.restype = _i32
    lib.dcp_testing_paged_attention_resident.argtypes = [_i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32)]
    lib.dcp_testing_paged_attention_resident.restype = _i32
    lib.dcp_testing_rows_overlap.argtypes = [_i64] * 7
    lib.dcp_testing_rows_overlap.restype = _i32
    lib.dcp_kv_append.argtypes = [kv, _ptr, _ptr, _ptr, _ptr, _i64, _i32, _i64, _i64, _i64, _i64, _i32, _i32, _i32,
                                  _ptr]
    lib.dcp_kv_append.restype = _i32
    lib.dcp_kv_weights.argtypes = [_ptr, _ptr, _ptr, _ptr, *[_i64] * 10, _i32, _i32, _i32, _i32, _ptr]
    lib.dcp_kv_weights.restype = _i32
    lib.dcp_kv_evict.argtypes = [kv, kv, _ptr, _ptr, _ptr, _ptr, _ptr, *[_i64] * 9, _i32, _i32, _i32, _ptr]
    lib.dcp_kv_evict.restype = _i32


_native = None
_lock = threading.Lock()


class _NoBinding:
    """In the place of a binding that could not be built: leaves every call to the code here."""
    attend = append = weigh = evict = staticmethod(lambda *args: None)


def _load_binding():
    spec = importlib.util.spec_from_file_location(f"{__package__}._paged_binding", _build.build_binding())
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_library(_build.build())
    return module


def _binding():
    """The compiled binding (built first if it is missing or older than its source).  Its functions
    make the calls below in the usual case and return None in every other one, where the code here
    makes the call or says what is wrong with it.  Without a compiler, or a directory to build in, the code
    here makes all of them."""
    global _native
    if _native is None:
        library()
        with _lock:
            if _native is None:
                try:
                    _native = _load_binding()
                except (RuntimeError, OSError, ImportError) as e:
                    warnings.warn(f"the compiled binding of the paged calls is not available, their host side takes "
                                  f"10 to 20 us longer per call: {e}", RuntimeWarning, stacklevel=3)
                    _native = _NoBinding
    return _native


def _done(status) -> bool:
    """Whether the binding made the call; raises where the library refused it."""
    if type(status) is int:
        raise DCPError(status, dcp_last_error())
    return status is not None


def _check_ints(bits: int = 32, **values) -> None:
    """Arguments that the C ABI takes as integers of so many bits (ctypes would cut them)."""
    for what, n in values.items():
        if not -(1 << bits - 1) <= n < 1 << bits - 1:
            raise ValueError(f"{what}={n} is outside the range of {bits}-bit integers")


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, requests: int,
           what: str = "") -> _PagedKV:
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError(f"{what}k_cache and v_cache must be [pages, page_size, heads, D] of one shape, got "
                         f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    if v_cache.dtype != k_cache.dtype:
        raise ValueError(f"{what}k_cache and v_cache differ in dtype")
    pages, page_size, heads, D = k_cache.shape
    kp, ks, kh, kd = k_cache.stride()
    vp, vs, vh, vd = v_cache.stride()
    if D > 1 and (kd != 1 or vd != 1):
        raise ValueError(f"{what}k_cache and v_cache must be contiguous in their last dimension")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != requests:
        raise ValueError(f"{what}block_table must be int32 [{requests}, max_pages], got {block_table.dtype} "
                         f"{tuple(block_table.shape)}")
    _check_ints(page_size=page_size, heads=heads, D=D)
    width, (tb, te) = block_table.shape[1], block_table.stride()
    if width > 1 and te != 1:
        raise ValueError(f"{what}block_table must be contiguous in its last dimension")
    return _PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), pages, kp, ks, kh, vp, vs, vh, tb,
                    width, page_size, heads, D, _code(k_cache.dtype))


def _lens(seq_lens: torch.Tensor, requests: int) -> None:
    if seq_lens.dtype != torch.int32 or seq_lens.shape != (requests,) or not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens must be a contiguous int32 tensor of {requests} entries, got {seq_lens.dtype} "
                         f"{tuple(seq_lens.shape)}")


def _rows(t: torch.Tensor, shape, what: str) -> tuple[int, int]:
    """Strides of the first two dimensions of an fp32 tensor of ``shape`` (None: any size) that is
    contiguous in its last one."""
    if t.dtype != torch.float32 or t.dim() != 3 or any(n is not None and t.shape[i] != n
                                                       for i, n in enumerate(shape)):
        raise ValueError(f"{what} must be fp32 {list(shape)}, got {t.dtype} {tuple(t.shape)}")
    s = t.stride()
    if t.shape[2] > 1 and s[2] != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    return s[0], s[1]


_workspace_bytes: dict = {}
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _call(device: torch.device, fn, *args) -> None:
    """One library call with ``device`` current (a decode step makes several calls of a few
    microseconds each, so the switch is made only where it is one)."""
    if device.index == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status:
        raise DCPError(status, dcp_last_error())


def _raw_stream(device: torch.device, stream) -> int:
    return _current_stream(device.index) if stream is None else _stream(device, stream)


def paged_attention_workspace(q: torch.Tensor, k_cache: torch.Tensor) -> int:
    """Bytes of workspace that attention of ``q`` [B, H, D] over ``k_cache`` needs on their device
    (whatever B and the lengths are)."""
    key = (q.shape[1], k_cache.shape[2], k_cache.shape[3], k_cache.dtype, k_cache.get_device())
    n = _workspace_bytes.get(key)
    if n is None:
        with torch.cuda.device(k_cache.device):
            n = library().dcp_paged_attention_workspace(key[0], key[1], key[2], _code(key[3]))
        if n < 0:
            return 0  # sizes that the call itself refuses, with the reason
        _workspace_bytes[key] = n
    return n


def _scratch(like: torch.Tensor, nbytes: int, stream) -> torch.Tensor | None:
    """Workspace for one call, in the order of the stream that the call runs on."""
    if nbytes == 0:
        return None
    n = -(-nbytes // like.element_size())
    if stream is None:
        return like.new_empty(n)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(n)


def _attend(q, k_cache, v_cache, block_table, seq_lens, out, lse, world_size, scale, shard, num_shards, interleave,
            logits, is_lse_base_on_e, workspace, stream) -> None:
    dev = _cuda(q, k_cache, v_cache, block_table, seq_lens, out, lse, logits, workspace)
    _check_ints(shard=shard, num_shards=num_shards, interleave=interleave)
    B, H, D = q.shape
    kv = _cache(k_cache, v_cache, block_table, B)
    _lens(seq_lens, B)
    if D != kv.head_dim or q.dtype != k_cache.dtype:
        raise ValueError(f"q {q.dtype} {tuple(q.shape)} does not match the cache {k_cache.dtype} "
                         f"{tuple(k_cache.shape)}")
    qb, qh, qd = q.stride()
    if D > 1 and qd != 1:
        raise ValueError("q must be contiguous in its last dimension")
    lg, lb, lh, cap = None, 0, 0, 0
    if logits is not None:
        lb, lh = _rows(logits, (B, H, None), "logits")
        lg, cap = logits.data_ptr(), logits.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D) if D else 1.0
    if workspace is None:
        workspace = _scratch(q, paged_attention_workspace(q, k_cache), stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    ws, wsb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    tail = (qb, qh, lb, lh, cap, scale, shard, num_shards, interleave, 1 if is_lse_base_on_e else 0, ws, wsb,
            _raw_stream(dev, stream))
    lib = library()
    if world_size is None:
        _call(dev, lib.dcp_paged_attention, kv, q.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), lg,
              B, H, *tail)
    else:
        _call(dev, lib.dcp_paged_attention_pack, kv, q.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lg, B, H,
              world_size, *tail)


def dcp_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, result: torch.Tensor, lse: torch.Tensor, scale: float | None = None,
                        shard: int = 0, num_shards: int = 1, interleave: int = 1,
                        logits: torch.Tensor | None = None, is_lse_base_on_e: bool = True,
                        workspace: torch.Tensor | None = None, stream=None) -> None:
    """Attention of one new token per request, q [B, H, D], over this rank's shard of the cache ->
    result [B, H, D] and lse [B, H] fp32 (a request without held positions: 0 and -inf).

    seq_lens [B] int32 are the lengths over all shards (num_shards = 1: this rank's own); scale
    defaults to 1/sqrt(D).  logits [B, H, cap] fp32, if given, receives scale * (q . k_p) at the
    held positions p < cap.  workspace (paged_attention_workspace bytes) is allocated per call
    unless given; calls that may run at the same time need one each."""
    if workspace is None and stream is None and _done(_binding().attend(
            q, k_cache, v_cache, block_table, seq_lens, 0, scale, shard, num_shards, interleave, logits,
            is_lse_base_on_e, result, lse)):
        return
    B, H, D = q.shape
    if tuple(result.shape) != (B, H, D) or result.dtype != q.dtype or not result.is_contiguous():
        raise ValueError(f"result must be a contiguous [{B}, {H}, {D}] tensor of q's dtype")
    if tuple(lse.shape) != (B, H) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 [{B}, {H}] tensor")
    _attend(q, k_cache, v_cache, block_table, seq_lens, result, lse, None, scale, shard, num_shards, interleave,
            logits, is_lse_base_on_e, workspace, stream)


def dcp_paged_attention_pack(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                             seq_lens: torch.Tensor, send_buf: torch.Tensor, world_size: int,
                             scale: float | None = None, shard: int = 0, num_shards: int = 1, interleave: int = 1,
                             logits: torch.Tensor | None = None, is_lse_base_on_e: bool = True,
                             workspace: torch.Tensor | None = None, stream=None) -> None:
    """dcp_paged_attention with its rows and LSEs written as dcp_pack would: send_buf [world_size, B,
    H/world_size, D + P]."""
    if workspace is None and stream is None and world_size != 0 and _done(_binding().attend(
            q, k_cache, v_cache, block_table, seq_lens, world_size, scale, shard, num_shards, interleave, logits,
            is_lse_base_on_e, send_buf, None)):
        return
    B, H, D = q.shape
    if world_size < 1 or H % world_size:
        raise ValueError(f"H={H} heads do not split over world_size={world_size}")
    want = (world_size, B, H // world_size, D + dcp_lse_pack_dim(q.dtype))
    if tuple(send_buf.shape) != want or send_buf.dtype != q.dtype or not send_buf.is_contiguous():
        raise ValueError(f"send_buf must be a contiguous {want} tensor of q's dtype")
    _attend(q, k_cache, v_cache, block_table, seq_lens, send_buf, None, int(world_size), scale, shard, num_shards,
            interleave, logits, is_lse_base_on_e, workspace, stream)


def dcp_kv_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_table: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor, shard: int = 0,
                  num_shards: int = 1, interleave: int = 1, stream=None) -> None:
    """Writes the rows of new tokens, k_new and v_new [T, heads, D], into the cache, in place.

    Tokens query_start_loc[r] <= t < query_start_loc[r + 1] are the last ones of request r's
    seq_lens[r] positions (new tokens included).  Only the positions that this rank holds are
    written; tokens outside every request are skipped.  Two tokens that land in the same slot (requests
    that share the page they append to) leave a mixture of their rows there."""
    if stream is None and _done(_binding().append(k_new, v_new, k_cache, v_cache, block_table, seq_lens,
                                                  query_start_loc, shard, num_shards, interleave)):
        return
    dev = _cuda(k_new, v_new, k_cache, v_cache, block_table, seq_lens, query_start_loc)
    _check_ints(shard=shard, num_shards=num_shards, interleave=interleave)
    R = seq_lens.numel()
    _lens(seq_lens, R)
    kv = _cache(k_cache, v_cache, block_table, R)
    heads, D = k_cache.shape[2:]
    for t, what in ((k_new, "k_new"), (v_new, "v_new")):
        if t.dim() != 3 or t.shape[0] != k_new.shape[0] or t.shape[1:] != k_cache.shape[2:] \
                or t.dtype != k_cache.dtype:
            raise ValueError(f"{what} must be [T, {heads}, {D}] of the cache's dtype, got {t.dtype} {tuple(t.shape)}")
        if D > 1 and t.stride(2) != 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
    if query_start_loc.dtype != torch.int32 or query_start_loc.shape != (R + 1,) \
            or not query_start_loc.is_contiguous():
        raise ValueError(f"query_start_loc must be a contiguous int32 tensor of {R + 1} entries")
    ks, vs = k_new.stride(), v_new.stride()
    _call(dev, library().dcp_kv_append, kv, k_new.data_ptr(), v_new.data_ptr(), seq_lens.data_ptr(),
          query_start_loc.data_ptr(), k_new.shape[0], R, ks[0], ks[1], vs[0], vs[1], shard, num_shards, interleave,
          _raw_stream(dev, stream))


def dcp_kv_weights(logits: torch.Tensor, global_lse: torch.Tensor, seq_lens: torch.Tensor, weights: torch.Tensor,
                   shard: int = 0, num_shards: int = 1, interleave: int = 1, is_lse_base_on_e: bool = True,
                   stream=None) -> None:
    """weights [B, heads, cap] fp32 += the attention weights of this step, in place: exp(logits
    [B, H, cap] - global_lse [B, H]) at the held positions, summed over the H / heads query heads of
    each key head.  global_lse is the LSE over all shards (the combine's); logits are
    paged_attention's."""
    if stream is None and _done(_binding().weigh(logits, global_lse, seq_lens, weights, shard, num_shards, interleave,
                                                 is_lse_base_on_e)):
        return
    dev = _cuda(logits, global_lse, seq_lens, weights)
    _check_ints(shard=shard, num_shards=num_shards, interleave=interleave)
    if weights.dim() != 3 or logits.dim() != 3:
        raise ValueError("logits must be [B, H, cap] and weights [B, heads, cap]")
    B, H = logits.shape[:2]
    heads, cap = weights.shape[1], min(logits.shape[2], weights.shape[2])
    ls, ws = _rows(logits, (B, H, None), "logits"), _rows(weights, (B, heads, None), "weights")
    if global_lse.shape != (B, H) or global_lse.dtype != torch.float32:
        raise ValueError(f"global_lse must be fp32 [{B}, {H}], got {global_lse.dtype} {tuple(global_lse.shape)}")
    _lens(seq_lens, B)
    _call(dev, library().dcp_kv_weights, logits.data_ptr(), global_lse.data_ptr(), seq_lens.data_ptr(),
          weights.data_ptr(), B, H, heads, cap, *ls, *global_lse.stride(), *ws, shard, num_shards, interleave,
          1 if is_lse_base_on_e else 0, _raw_stream(dev, stream))


def dcp_kv_evict(weights: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, new_block_table: torch.Tensor,
                 keep: int, recent: int, kept: torch.Tensor, new_lens: torch.Tensor, new_weights: torch.Tensor,
                 shard: int = 0, num_shards: int = 1, interleave: int = 1, stream=None) -> None:
    """Keeps, per request and key head, the `keep` positions of largest weights [B, heads, cap] (the
    last `recent` always among them) and moves their rows, in order, into the pages of
    new_block_table [B, max_pages] in k_out / v_out (which may be the same pools).  Writes kept
    [B, heads, keep] int32 (positions, then -1), new_lens [B] int32 and new_weights [B, heads,
    new_cap >= keep] (the kept weights, then 0)."""
    dev = _cuda(weights, k_cache, v_cache, block_table, seq_lens, k_out, v_out, new_block_table, kept, new_lens,
                new_weights)
    _check_ints(shard=shard, num_shards=num_shards, interleave=interleave)
    _check_ints(64, keep=keep, recent=recent)
    B = seq_lens.numel()
    _lens(seq_lens, B)
    src = _cache(k_cache, v_cache, block_table, B)
    dst = _cache(k_out, v_out, new_block_table, B, "new ")
    heads = k_cache.shape[2]
    ws = _rows(weights, (B, heads, None), "weights")
    ns = _rows(new_weights, (B, heads, None), "new_weights")
    if tuple(kept.shape) != (B, heads, keep) or kept.dtype != torch.int32 or not kept.is_contiguous():
        raise ValueError(f"kept must be a contiguous int32 [{B}, {heads}, {keep}] tensor")
    if tuple(new_lens.shape) != (B,) or new_lens.dtype != torch.int32 or not new_lens.is_contiguous():
        raise ValueError(f"new_lens must be a contiguous int32 [{B}] tensor")
    _call(dev, library().dcp_kv_evict, src, dst, seq_lens.data_ptr(), weights.data_ptr(), new_weights.data_ptr(),
          kept.data_ptr(), new_lens.data_ptr(), B, weights.shape[2], new_weights.shape[2], *ws, *ns, keep, recent,
          shard, num_shards, interleave, _raw_stream(dev, stream))


# ---- allocating helpers ------------------------------------------------------------------
def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, scale: float | None = None, shard: int = 0, num_shards: int = 1,
                    interleave: int = 1, logits: torch.Tensor | None = None, is_lse_base_on_e: bool = True):
    """Attention of q [B, H, D] over this rank's shard: (result [B, H, D], lse [B, H] fp32), the
    partial pair that pack() or lse_weighted_combine() takes.  See dcp_paged_attention."""
    out = _binding().attend(q, k_cache, v_cache, block_table, seq_lens, 0, scale, shard, num_shards, interleave, logits,
                            is_lse_base_on_e, None, None)
    if _done(out):
        return out
    result = q.new_empty(q.shape)
    lse = q.new_empty(q.shape[:2], dtype=torch.float32)
    dcp_paged_attention(q, k_cache, v_cache, block_table, seq_lens, result, lse, scale, shard, num_shards, interleave,
                        logits, is_lse_base_on_e)
    return result, lse


def paged_attention_pack(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, world_size: int, scale: float | None = None, shard: int = 0,
                         num_shards: int = 1, interleave: int = 1, logits: torch.Tensor | None = None,
                         is_lse_base_on_e: bool = True) -> torch.Tensor:
    """The packed send buffer [world_size, B, H/world_size, D + P] of paged_attention's result, in
    one step.  See dcp_paged_attention_pack."""
    if world_size != 0:
        out = _binding().attend(q, k_cache, v_cache, block_table, seq_lens, world_size, scale, shard, num_shards,
                                interleave, logits, is_lse_base_on_e, None, None)
        if _done(out):
            return out
    B, H, D = q.shape
    if world_size < 1 or H % world_size:
        raise ValueError(f"H={H} heads do not split over world_size={world_size}")
    send = q.new_empty((world_size, B, H // world_size, D + dcp_lse_pack_dim(q.dtype)))
    dcp_paged_attention_pack(q, k_cache, v_cache, block_table, seq_lens, send, world_size, scale, shard, num_shards,
                             interleave, logits, is_lse_base_on_e)
    return send


def kv_evict(weights: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
             seq_lens: torch.Tensor, new_block_table: torch.Tensor, keep: int, recent: int = 0,
             k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, shard: int = 0,
             num_shards: int = 1, interleave: int = 1):
    """Eviction into the pages of new_block_table, in the same pools unless k_out and v_out are
    given: (kept [B, heads, keep] int32, new_lens [B] int32, new_weights of weights' shape, at least
    `keep` long).  See dcp_kv_evict."""
    if keep < 1:
        raise DCPError(1, f"kv_evict: keep={keep} is less than 1")
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        k_out, v_out = k_cache, v_cache
    out = _binding().evict(weights, k_cache, v_cache, block_table, seq_lens, k_out, v_out, new_block_table, keep, recent,
                           shard, num_shards, interleave)
    if _done(out):
        return out
    B, heads, cap = weights.shape
    kept = weights.new_empty((B, heads, keep), dtype=torch.int32)
    new_lens = weights.new_empty(B, dtype=torch.int32)
    new_weights = weights.new_empty((B, heads, max(cap, keep)), dtype=torch.float32)
    dcp_kv_evict(weights, k_cache, v_cache, block_table, seq_lens, k_out, v_out, new_block_table, keep, recent, kept,
                 new_lens, new_weights, shard, num_shards, interleave)
    return kept, new_lens, new_weights
