"""Python binding of libcsa2 (the CSA2 sparse-attention decode step on B200).

Argument marshalling only: every call forwards torch tensors' device pointers
to the C ABI declared in ``include/csa2.h`` and raises on a non-OK status.
Importing this package loads ``libcsa2.so`` from this directory, building it
with nvcc first when it is missing or older than its sources, and fails
loudly when it can be neither built nor found; there is no other code path.
"""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

LATENT, CODE_BYTES, SCALE_BYTES, KEY_DIM, IDX_HEADS = 512, 256, 32, 128, 32
BLOCK, MAX_BLOCKS, POOL, TOPK, SWA = 8, 2048, 16384, 512, 128
PAGE_ENTRIES, PAGE_BYTES, SWA_BYTES, PENDING_STRIDE = 64, 27648, 66048, 656
PAGE_CODES_BYTES, PAGE_SCALES_BYTES, PAGE_KEYS_BYTES, PAGE_SUMM_BYTES = 16384, 2048, 8192, 1024


def plane_offsets(n_pages: int):
    """Byte offsets of the codes / scales / keys / summaries planes of a pool."""
    return 0, n_pages * 16384, n_pages * 18432, n_pages * 26624
SWA_CODES_OFF, SWA_SCALE_OFF = 0, 65536
INDEX_FLAT, INDEX_FULL, INDEX_REINDEX = 0, 1, 2

EXPORTS = ("csa2_page_bytes", "csa2_swa_bytes", "csa2_workspace_bytes", "csa2_prefill", "csa2_append",
           "csa2_index", "csa2_attend", "csa2_get_device_error", "csa2_status_string", "csa2_set_profile_events",
           "csa2_launch_count", "csa2_attend_noalloc", "csa2_topk", "csa2_shard_blocks", "csa2_shard_pool",
           "csa2_shard_rescore", "csa2_shard_topk", "csa2_attend_partial", "csa2_combine",
           "csa2_selftest_wait_timeout", "csa2_verify", "csa2_plan_tokens", "csa2_norm_rope",
           "csa2_prompt_attend", "csa2_prompt_workspace_bytes")
MAX_SHARDS = 8
ATTEND_NOALLOC_MAX_ROWS = 512
MAX_DRAFT, PLAN_MAX_BATCH = 31, 4096
ROPE_HALVES, ROPE_INVERSE, ROPE_NO_NORM = 1, 2, 4
PROMPT_WORKSPACE_MAX = 38951424
KERNEL_BLOCK_SCORE, KERNEL_FLAT_SCORE, KERNEL_POOL_SCORE, KERNEL_SELECT, KERNEL_ATTEND, KERNEL_COMBINE = range(6)


class CSA2Error(RuntimeError):
    def __init__(self, call: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{call} failed: {status_string(status)} ({status}){detail}")


class csa2_cache(C.Structure):
    _fields_ = [("pool", C.c_void_p), ("n_pages", C.c_int32), ("page_table", C.c_void_p),
                ("max_pages", C.c_int32), ("n_tokens", C.c_void_p), ("m", C.c_void_p), ("swa", C.c_void_p),
                ("pending", C.c_void_p), ("error", C.c_void_p), ("batch", C.c_int32)]


def _load():
    from . import build as _build
    if not _build.up_to_date():
        try:
            _build.build()
        except (OSError, subprocess.CalledProcessError) as e:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"libcsa2.so is not built at {LIB_PATH} and building it failed: {e}") from e
    L = C.CDLL(LIB_PATH)
    P, I32, SZ = C.c_void_p, C.c_int32, C.c_size_t
    sig = {
        "csa2_page_bytes": (SZ, []),
        "csa2_swa_bytes": (SZ, []),
        "csa2_workspace_bytes": (SZ, [I32, I32]),
        "csa2_prefill": (C.c_int, [P, I32, I32, I32, I32, I32, P, P, P, P]),
        "csa2_append": (C.c_int, [P, P, P, P, P, P]),
        "csa2_index": (C.c_int, [P, C.c_int, P, P, P, P, P, P, SZ, P]),
        "csa2_attend": (C.c_int, [P, I32, P, P, C.c_float, P, I32, C.c_uint32, P, SZ, P]),
        "csa2_get_device_error": (C.c_int, [P, C.POINTER(C.c_int32), P]),
        "csa2_status_string": (C.c_char_p, [C.c_int]),
        "csa2_set_profile_events": (C.c_int, [I32, P, P]),
        "csa2_attend_noalloc": (C.c_int, [P, I32, P, P, C.c_float, P, I32, P]),
        "csa2_launch_count": (C.c_uint64, []),
        "csa2_topk": (C.c_int, [P, C.c_int64, P, I32, I32, P, P]),
        "csa2_shard_blocks": (C.c_int, [P, P, P, P, P, P, P, SZ, P]),
        "csa2_shard_pool": (C.c_int, [P, P, I32, P, P, P, P, P]),
        "csa2_shard_rescore": (C.c_int, [P, P, P, P, P, P, P, P, P]),
        "csa2_shard_topk": (C.c_int, [P, P, I32, P, P, P, P]),
        "csa2_attend_partial": (C.c_int, [P, I32, P, P, C.c_float, I32, P, P, C.c_uint32, P]),
        "csa2_combine": (C.c_int, [I32, P, P, I32, I32, P, I32, P]),
        "csa2_selftest_wait_timeout": (C.c_int, [P, C.c_uint32, P]),
        "csa2_verify": (C.c_int, [I32, I32, I32, P, P, P, P, P, P, P, P, P]),
        "csa2_plan_tokens": (C.c_int, [I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, P, P, P, P]),
        "csa2_norm_rope": (C.c_int, [I32, I32, I32, P, C.c_int64, P, P, I32, P, C.c_int64, P, P, P, P, P, I32,
                                     C.c_float, C.c_uint32, P, P]),
        "csa2_prompt_workspace_bytes": (SZ, [I32, I32, I32]),
        "csa2_prompt_attend": (C.c_int, [I32, P, P, I32, I32, I32, P, P, C.c_int64, I32, C.c_float, P, I32, P, P, P,
                                         SZ, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


lib = _load()


def status_string(status: int) -> str:
    return lib.csa2_status_string(status).decode()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libcsa2 takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libcsa2 takes contiguous tensors")
    return C.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object (3 us of a call's host time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return C.c_void_p(_raw_stream(torch.cuda.current_device()))
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(name, st):
    if st != 0:
        raise CSA2Error(name, st)


class Cache:
    """Device storage of a batch of requests' CSA2 caches (allocated by torch)
    plus the matching C struct."""

    def __init__(self, page_table: torch.Tensor, n_pages: int, m, device="cuda"):
        self.device = torch.device(device)
        self.batch = int(page_table.shape[0])
        self.max_pages = int(page_table.shape[1])
        self.n_pages = int(n_pages)
        self.pool = torch.zeros(self.n_pages * PAGE_BYTES, dtype=torch.uint8, device=self.device)
        self.page_table = page_table.to(self.device, torch.int32).contiguous()
        self.n_tokens = torch.zeros(self.batch, dtype=torch.int32, device=self.device)
        self.m = torch.as_tensor(m, dtype=torch.int32).to(self.device).contiguous()
        self.m_host = [int(x) for x in torch.as_tensor(m)]
        self.swa = torch.zeros(self.batch * SWA_BYTES, dtype=torch.uint8, device=self.device)
        self.pending = torch.zeros(self.batch * PENDING_STRIDE, dtype=torch.float32, device=self.device)
        self.error = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.c = csa2_cache(self.pool.data_ptr(), self.n_pages, self.page_table.data_ptr(), self.max_pages,
                            self.n_tokens.data_ptr(), self.m.data_ptr(), self.swa.data_ptr(),
                            self.pending.data_ptr(), self.error.data_ptr(), self.batch)

    @property
    def ref(self):
        return C.byref(self.c)

    @property
    def max_entries(self) -> int:
        return self.max_pages * PAGE_ENTRIES

    # Views of the packed bytes (for tests and inspection).
    def page_view(self) -> torch.Tensor:
        return self.pool.view(self.n_pages, PAGE_BYTES)

    def swa_view(self) -> torch.Tensor:
        return self.swa.view(self.batch, SWA_BYTES)


def csa2_page_bytes() -> int:
    return int(lib.csa2_page_bytes())


def csa2_swa_bytes() -> int:
    return int(lib.csa2_swa_bytes())


def csa2_workspace_bytes(batch: int, max_entries: int) -> int:
    return int(lib.csa2_workspace_bytes(batch, max_entries))


def workspace(cache: Cache) -> torch.Tensor:
    n = csa2_workspace_bytes(cache.batch, cache.max_entries)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def csa2_prefill(cache: Cache, req: int, tok_begin: int, n_tok_final: int, lat, key, gate, stream=None):
    n = int(key.shape[0])
    _check("csa2_prefill", lib.csa2_prefill(cache.ref, req, cache.m_host[req], tok_begin, n, n_tok_final,
                                            _ptr(lat), _ptr(key), _ptr(gate), _stream(stream)))


def csa2_append(cache: Cache, lat, key, gate, n_new, stream=None):
    _check("csa2_append", lib.csa2_append(cache.ref, _ptr(lat), _ptr(key), _ptr(gate), _ptr(n_new),
                                          _stream(stream)))


def csa2_index(cache: Cache, mode: int, q_idx, w, pool, pool_len, topk, ws, stream=None):
    qi = q_idx.view(torch.int16) if q_idx.dtype == torch.bfloat16 else q_idx
    _check("csa2_index", lib.csa2_index(cache.ref, mode, _ptr(qi), _ptr(w), _ptr(pool), _ptr(pool_len),
                                        _ptr(topk), _ptr(ws), ws.numel(), _stream(stream)))


def csa2_topk(scores, n, k: int, out, stream=None):
    """Top-k of each row of scores [batch, stride] (f32), first n[b] elements
    (n int32 [batch]); out int32 [batch, k] gets ascending indices, -1 padded."""
    assert scores.dtype == torch.float32 and scores.stride(1) == 1 and n.dtype == torch.int32
    assert out.dtype == torch.int32 and out.is_contiguous() and tuple(out.shape) == (scores.shape[0], k)
    _check("csa2_topk", lib.csa2_topk(_ptr(scores), scores.stride(0), _ptr(n), int(scores.shape[0]), int(k),
                                      _ptr(out), _stream(stream)))


ATTEND_INPUTS_SETTLED = 1


def csa2_attend(cache: Cache, q, topk, scale: float, out, ws, stream=None, flags: int = 0):
    heads = int(q.shape[1])
    qq = q.view(torch.int16) if q.dtype == torch.bfloat16 else q
    fp32 = 1 if out.dtype == torch.float32 else 0
    _check("csa2_attend", lib.csa2_attend(cache.ref, heads, _ptr(qq), _ptr(topk), float(scale), _ptr(out), fp32,
                                          flags, _ptr(ws), ws.numel(), _stream(stream)))


def csa2_get_device_error(cache: Cache, stream=None) -> int:
    code = C.c_int32(0)
    st = lib.csa2_get_device_error(cache.ref, C.byref(code), _stream(stream))
    if st not in (0, 4):
        raise CSA2Error("csa2_get_device_error", st)
    return int(code.value)


def csa2_set_profile_events(kernel: int, start=None, stop=None):
    """Bracket every later launch of `kernel` with torch.cuda.Event pair
    (start, stop) recorded on the launching stream; None/None turns it off."""
    a = C.c_void_p(start.cuda_event) if start is not None else None
    b = C.c_void_p(stop.cuda_event) if stop is not None else None
    _check("csa2_set_profile_events", lib.csa2_set_profile_events(kernel, a, b))


def csa2_launch_count() -> int:
    return int(lib.csa2_launch_count())


def csa2_attend_noalloc(cache: Cache, q, topk, scale: float, out, stream=None) -> int:
    """csa2_attend without a workspace, for callers that cannot allocate
    device memory: the library keeps the split partials in its own fixed
    array (batch * heads <= ATTEND_NOALLOC_MAX_ROWS).  Returns the C status;
    raises on anything but OK or CSA2_ERR_UNSUPPORTED (size over the limit)."""
    heads = int(q.shape[1])
    qq = q.view(torch.int16) if q.dtype == torch.bfloat16 else q
    fp32 = 1 if out.dtype == torch.float32 else 0
    st = lib.csa2_attend_noalloc(cache.ref, heads, _ptr(qq), _ptr(topk), float(scale), _ptr(out), fp32,
                                 _stream(stream))
    if st not in (0, 2):
        raise CSA2Error("csa2_attend_noalloc", st)
    return int(st)


# ---------------------------------------------------------------- sequence shards
def _ptrs(ts):
    """Host array of the device pointers of tensors ts (kept alive by the caller)."""
    if not 1 <= len(ts) <= MAX_SHARDS:
        raise ValueError(f"1..{MAX_SHARDS} shards, got {len(ts)}")
    arr = (C.c_void_p * len(ts))(*[_ptr(t).value for t in ts])
    return C.cast(arr, C.c_void_p), arr


def _bits16(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def csa2_shard_blocks(cache, entry_offset, q_idx, w, block_ids, block_scores, ws, stream=None):
    _check("csa2_shard_blocks", lib.csa2_shard_blocks(cache.ref, _ptr(entry_offset), _ptr(_bits16(q_idx)), _ptr(w),
                                                      _ptr(block_ids), _ptr(block_scores), _ptr(ws), ws.numel(),
                                                      _stream(stream)))


def csa2_shard_pool(cache, entry_offset, cand_ids, cand_scores, pool, pool_len, stream=None):
    pi, ki = _ptrs(cand_ids)
    ps, ks = _ptrs(cand_scores)
    _check("csa2_shard_pool", lib.csa2_shard_pool(cache.ref, _ptr(entry_offset), len(cand_ids), pi, ps, _ptr(pool),
                                                  _ptr(pool_len), _stream(stream)))
    del ki, ks


def csa2_shard_rescore(cache, entry_offset, q_idx, w, pool, pool_len, ids, scores, stream=None):
    _check("csa2_shard_rescore", lib.csa2_shard_rescore(cache.ref, _ptr(entry_offset), _ptr(_bits16(q_idx)), _ptr(w),
                                                        _ptr(pool), _ptr(pool_len), _ptr(ids), _ptr(scores),
                                                        _stream(stream)))


def csa2_shard_topk(cache, entry_offset, cand_ids, cand_scores, topk, stream=None):
    pi, ki = _ptrs(cand_ids)
    ps, ks = _ptrs(cand_scores)
    _check("csa2_shard_topk", lib.csa2_shard_topk(cache.ref, _ptr(entry_offset), len(cand_ids), pi, ps, _ptr(topk),
                                                  _stream(stream)))
    del ki, ks


def csa2_attend_partial(cache, q, topk, scale: float, with_window: bool, o, lse, stream=None, flags: int = 0):
    assert o.dtype == torch.float32 and lse.dtype == torch.float32
    _check("csa2_attend_partial", lib.csa2_attend_partial(cache.ref, int(q.shape[1]), _ptr(_bits16(q)), _ptr(topk),
                                                          float(scale), 1 if with_window else 0, _ptr(o), _ptr(lse),
                                                          flags, _stream(stream)))


def csa2_combine(o_parts, lse_parts, out, stream=None):
    """out [batch, heads, 512] (bf16 or f32) = log-sum-exp merge of the
    partial results o_parts[s] [batch, heads, 512] f32 with lse_parts[s]
    [batch, heads] f32."""
    if len(o_parts) != len(lse_parts):
        raise ValueError("one lse per partial output")
    po, ko = _ptrs(o_parts)
    pl, kl = _ptrs(lse_parts)
    fp32 = 1 if out.dtype == torch.float32 else 0
    _check("csa2_combine", lib.csa2_combine(len(o_parts), po, pl, int(out.shape[0]), int(out.shape[1]), _ptr(out),
                                            fp32, _stream(stream)))
    del ko, kl


def csa2_selftest_wait_timeout(error_word, polls: int = 1024, stream=None):
    """Run the bounded-wait self-test: error_word (int32 device tensor of one
    element) receives CSA2_DEV_TIMEOUT once the probe's wait runs out."""
    _check("csa2_selftest_wait_timeout", lib.csa2_selftest_wait_timeout(_ptr(error_word), int(polls), _stream(stream)))


# ---------------------------------------------------------------- around the layers
# A step of a serving program makes these calls eagerly with small tensors,
# where the host's time is the call's: one pass of cheap checks per argument.
_F32, _I32, _B16 = torch.float32, torch.int32, torch.bfloat16


def _typed(name, t, dtype, shape, dev):
    """The device pointer of t after its type, shape and device are checked (None passes)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError("libcsa2 takes contiguous tensors")
    return _here(t, dev)


def _here(t, dev):
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("libcsa2 takes device tensors")
        raise ValueError("libcsa2 takes tensors of the current device")
    return t.data_ptr()


def _device():
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2      # -1 is the host


def _stream_on(stream, dev):
    if stream is None and _raw_stream is not None and dev >= 0:
        return _raw_stream(dev)
    return _stream(stream)


def csa2_verify(target, probs, draft, n_draft, u, n_accepted, tokens, error, stream=None):
    """Accept drafted tokens draft [batch, k] against target [batch, k+1,
    vocab] f32 and the drafter's probs [batch, k, vocab] f32 (None: it named
    its tokens for certain) with random numbers u [batch, k+1]; n_accepted
    [batch] and tokens [batch, k+1] (kept drafts, drawn token, -1) receive the
    outcome."""
    B, k1, V = target.shape
    dev = _device()
    st = lib.csa2_verify(
        B, k1 - 1, V, _typed("target", target, _F32, (B, k1, V), dev),
        _typed("probs", probs, _F32, (B, k1 - 1, V), dev), _typed("draft", draft, _I32, (B, k1 - 1), dev),
        _typed("n_draft", n_draft, _I32, (B,), dev), _typed("u", u, _F32, (B, k1), dev),
        _typed("n_accepted", n_accepted, _I32, (B,), dev), _typed("tokens", tokens, _I32, (B, k1), dev),
        _typed("error", error, _I32, (1,), dev), _stream_on(stream, dev))
    if st:
        raise CSA2Error("csa2_verify", st)


def csa2_plan_tokens(n_tokens, n_new, m, page_table, free_pages, n_free, n_free_out, cu_new, token_req, token_pos,
                     token_slot, error, stream=None):
    """Pages and slots of a step's new tokens (int32 tensors throughout):
    n_tokens, n_new, m [batch]; page_table [batch, max_pages] and free_pages
    [n_pages] are updated; n_free, n_free_out [1]; cu_new [batch+1];
    token_req, token_pos, token_slot [max_new].  Dropped tokens that were in
    the cache: csa2_prefill writes the window of those that stay again."""
    B, width = page_table.shape
    one, per, rows, dev = (1,), (B,), token_req.shape, _device()
    n_pages = free_pages.shape[0]
    st = lib.csa2_plan_tokens(
        B, width, n_pages, rows[0], _typed("n_tokens", n_tokens, _I32, per, dev), _typed("n_new", n_new, _I32, per, dev),
        _typed("m", m, _I32, per, dev), _typed("page_table", page_table, _I32, (B, width), dev),
        _typed("free_pages", free_pages, _I32, (n_pages,), dev), _typed("n_free", n_free, _I32, one, dev),
        _typed("n_free_out", n_free_out, _I32, one, dev), _typed("cu_new", cu_new, _I32, (B + 1,), dev),
        _typed("token_req", token_req, _I32, (rows[0],), dev), _typed("token_pos", token_pos, _I32, rows, dev),
        _typed("token_slot", token_slot, _I32, rows, dev), _typed("error", error, _I32, one, dev),
        _stream_on(stream, dev))
    if st:
        raise CSA2Error("csa2_plan_tokens", st)


def _heads(name, t, dev):
    """(pointer, heads, dim, token stride) of a bf16 [n, heads, dim] tensor whose
    tokens may lie apart (a slice of a wider projection)."""
    if t.dtype is not _B16 or t.dim() != 3:
        raise ValueError(f"{name}: bfloat16 [n, heads, dim] expected, got {t.dtype} {tuple(t.shape)}")
    n, h, d = t.shape
    apart, head, chan = t.stride()
    if chan != 1 or (h > 1 and head != d):
        if t.numel():
            raise ValueError(f"{name}: the heads of a token must be contiguous")
    return _here(t, dev), h, d, apart if n > 1 else h * d


def csa2_norm_rope(q, k, pos, inv_freq, q_weight, k_weight, eps: float, q_out, k_out, k_out_f32=None, n_valid=None,
                   flags: int = 0, stream=None):
    """Normalise (times weight [dim] f32) and rotate the heads of q [n, heads,
    dim] and k [n, kv_heads, dim] (bf16; either may be None): q_out and k_out
    bf16, k_out_f32 f32 (one k output may be None).  pos [n] i32; inv_freq
    [rot_dim / 2] f32 or None; n_valid: device int32 [1] or None; flags:
    ROPE_HALVES | ROPE_INVERSE | ROPE_NO_NORM."""
    dev = _device()
    qp, h, dq, qs = (None, 0, 0, 0) if q is None else _heads("q", q, dev)
    kp, g, dk, ks = (None, 0, 0, 0) if k is None else _heads("k", k, dev)
    if q is None and k is None:
        raise ValueError("csa2_norm_rope needs q or k")
    n, d = (k if q is None else q).shape[0], dq or dk
    if q is not None and k is not None and (dq != dk or k.shape[0] != n):
        raise ValueError("q and k differ in tokens or channels")
    half = 0 if inv_freq is None else inv_freq.shape[0]
    st = lib.csa2_norm_rope(
        n, d, h, qp, qs, _typed("q_weight", q_weight, _F32, (d,), dev), _typed("q_out", q_out, _B16, (n, h, d), dev),
        g, kp, ks, _typed("k_weight", k_weight, _F32, (d,), dev), _typed("k_out", k_out, _B16, (n, g, d), dev),
        _typed("k_out_f32", k_out_f32, _F32, (n, g, d), dev), _typed("pos", pos, _I32, (n,), dev),
        _typed("inv_freq", inv_freq, _F32, (half,), dev), 2 * half, eps, flags,
        _typed("n_valid", n_valid, _I32, (1,), dev), _stream_on(stream, dev))
    if st:
        raise CSA2Error("csa2_norm_rope", st)


def csa2_prompt_workspace_bytes(n_q: int, heads: int, n_k: int) -> int:
    """Workspace of one call of this shape.  Smaller shapes may need more:
    PROMPT_WORKSPACE_MAX is enough for calls of any shape."""
    return int(lib.csa2_prompt_workspace_bytes(n_q, heads, n_k))


def csa2_prompt_attend(q, lat, cu_q, cu_k, window: int, scale: float, out, lse, error, ws, stream=None):
    """Causal attention of packed prompts q [n_q, heads, 512] over latents lat
    [n_k, 512] (bf16; rows may lie apart), request b holding tokens
    cu_q[b]..cu_q[b+1] and latents cu_k[b]..cu_k[b+1]; window 0 sees
    everything.  out like q, bf16 or f32; lse [n_q, heads] f32 or None; ws:
    uint8, csa2_prompt_workspace_bytes(n_q, heads, n_k), or PROMPT_WORKSPACE_MAX
    where one workspace serves calls of different shapes."""
    n_q, heads = q.shape[:2]
    dev = _device()
    if lat.dtype is not _B16 or lat.dim() != 2 or lat.shape[1] != LATENT or (lat.stride(1) != 1 and lat.numel()):
        raise ValueError(f"lat: rows of {LATENT} bfloat16 expected, got {lat.dtype} {tuple(lat.shape)}")
    n_k, cu, rows = lat.shape[0], cu_q.shape, (n_q, heads, LATENT)
    fp32 = out.dtype is _F32
    n_ws = ws.numel()
    st = lib.csa2_prompt_attend(
        cu[0] - 1, _typed("cu_q", cu_q, _I32, (cu[0],), dev), _typed("cu_k", cu_k, _I32, cu, dev), n_q, n_k, heads,
        _typed("q", q, _B16, rows, dev), _here(lat, dev), lat.stride(0) if n_k > 1 else LATENT, window, scale,
        _typed("out", out, _F32 if fp32 else _B16, rows, dev), fp32, _typed("lse", lse, _F32, (n_q, heads), dev),
        _typed("error", error, _I32, (1,), dev), _typed("ws", ws, torch.uint8, (n_ws,), dev), n_ws,
        _stream_on(stream, dev))
    if st:
        raise CSA2Error("csa2_prompt_attend", st)
