"""Python binding of libfastar, the FAST-AR per-chunk attention library.

Argument marshalling only: every function reads shapes from torch tensors,
passes their device pointers and the current CUDA stream to the C ABI of
include/fastar.h, and raises FastarError on a non-zero status.  All work
runs in the library's CUDA kernels; there is no fallback.  If the library
has not been built, loading it raises (build it with
`python -m merged_attention_autoregressive_gb300.build`).
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfastar.so")

BF16, F32 = 0, 1
OP_HASH, OP_MERGE, OP_PRUNE, OP_ANNCA, OP_ANNSA, OP_ANNSA_PARTS = 0, 1, 2, 3, 4, 5
REP_LAST, REP_MEAN = 0, 1
REPS = {"last": REP_LAST, "mean": REP_MEAN}
SEARCH_PREV, SEARCH_LSH, SEARCH_QUANT = 0, 1, 2
OP_QUANT = 6
OP_BRANCH = 7
ROPE_MAX_AXES, ROPE_MAX_PAIRS = 4, 64
PAIRINGS = {"adjacent": 0, "halves": 1}


def search_code(search: str) -> int:
    """"prev", "lsh" or "quant<bits>" (e.g. "quant8") as the C ABI's search value."""
    if search == "prev":
        return SEARCH_PREV
    if search == "lsh":
        return SEARCH_LSH
    if search.startswith("quant"):
        bits = int(search[5:])
        return SEARCH_QUANT | (bits << 8)
    raise ValueError(f"unknown search {search!r}")
STATUS = {0: "FASTAR_OK", 1: "FASTAR_ERR_ARG", 2: "FASTAR_ERR_UNSUPPORTED", 3: "FASTAR_ERR_CUDA",
          4: "FASTAR_ERR_WORKSPACE", 16: "FASTAR_ERR_CAPACITY", 17: "FASTAR_ERR_TIMEOUT",
          18: "FASTAR_ERR_DEVICE_ARG"}
EXPORTS = ["fastar_status_string", "fastar_version", "fastar_launch_count",
           "fastar_timing_begin", "fastar_timing_end", "fastar_timing_name",
           "fastar_workspace_size", "fastar_hash", "fastar_hash_many", "fastar_bucket_csr",
           "fastar_tempcache_merge", "fastar_tempcache_merge_ev", "fastar_annca_prune", "fastar_annca_attention",
           "fastar_annsa_attention", "fastar_check_bounded_wait", "fastar_tempcache_merge_rep",
           "fastar_annsa_attention_part", "fastar_annsa_combine", "fastar_tempcache_merge_search",
           "fastar_annsa_quant_attention", "fastar_annca_quant_attention",
           "fastar_rope_plan_init", "fastar_rope", "fastar_page_append", "fastar_branch_attention"]


class FastarError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)} ({lib().fastar_status_string(code).decode()})")
        self.code = code


class CacheStruct(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("D", ctypes.c_int), ("C", ctypes.c_int),
                ("T", ctypes.c_int), ("B", ctypes.c_int), ("dt", ctypes.c_int),
                ("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("last_frame", ctypes.c_void_p),
                ("size", ctypes.c_void_p), ("inserted", ctypes.c_void_p),
                ("evicted", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p)]


class RopePlanStruct(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int), ("axes", ctypes.c_int), ("pairs", ctypes.c_int),
                ("pairing", ctypes.c_int), ("turn", ctypes.c_uint64 * ROPE_MAX_PAIRS),
                ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS)]


class PagesStruct(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("D", ctypes.c_int), ("page", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("B", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("dt", ctypes.c_int), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("len", ctypes.c_void_p)]


class PrefixStruct(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("C", ctypes.c_int), ("D", ctypes.c_int), ("dt", ctypes.c_int),
                ("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("size", ctypes.c_void_p)]


_lib = None
_VP, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_I64 = ctypes.c_int64
MAX_HASH_JOBS = 4


class HashJob(ctypes.Structure):
    """fastar_hash_job: one input of fastar_hash_many."""
    _fields_ = [("x", _VP), ("N", _I), ("codes", _VP), ("perm", _VP), ("offsets", _VP)]


def lib() -> ctypes.CDLL:
    """Load the in-tree libfastar.so (raises OSError when it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{LIB_PATH} is missing: build it with "
                          "`python -m merged_attention_autoregressive_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.fastar_status_string.restype = ctypes.c_char_p
        L.fastar_status_string.argtypes = [_I]
        L.fastar_version.restype = _I
        L.fastar_launch_count.restype = ctypes.c_uint64
        L.fastar_timing_begin.argtypes = [_VP, _I]
        L.fastar_timing_begin.restype = _I
        L.fastar_timing_end.restype = _I
        L.fastar_timing_name.argtypes = [_I]
        L.fastar_timing_name.restype = ctypes.c_char_p
        L.fastar_workspace_size.restype = _SZ
        L.fastar_workspace_size.argtypes = [_I] * 7
        L.fastar_hash.argtypes = [_I, _VP, _I, _I, _I, _VP, _I, _I, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]
        L.fastar_bucket_csr.argtypes = [_VP, _I, _I, _I, _VP, _VP, _VP, _VP]
        L.fastar_hash_many.argtypes = [_I, _I, ctypes.POINTER(HashJob), _I, _I, _VP, _I, _I, _VP, _SZ,
                                       _VP, _VP]
        L.fastar_tempcache_merge.argtypes = [ctypes.POINTER(CacheStruct), _VP, _VP, _VP, _I, _I,
                                             ctypes.c_int32, _F, _VP, _VP, _SZ, _VP, _VP]
        L.fastar_tempcache_merge_ev.argtypes = [ctypes.POINTER(CacheStruct), _VP, _VP, _VP, _I, _I,
                                                ctypes.c_int32, _F, _VP, _VP, _SZ, _VP, _VP, _VP]
        L.fastar_annca_prune.argtypes = [_VP, _VP, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _SZ, _VP, _VP]
        L.fastar_annca_attention.argtypes = [_I, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F,
                                             _VP, _VP, _SZ, _VP, _VP]
        L.fastar_annsa_attention.argtypes = [_I, _VP, _VP, _VP, _VP, _I, ctypes.POINTER(CacheStruct),
                                             _F, _VP, _VP, _VP, _SZ, _VP, _VP]
        L.fastar_check_bounded_wait.argtypes = [_I, _VP, _VP]
        L.fastar_annsa_attention_part.argtypes = [_I, _VP, _VP, _VP, _VP, _I, ctypes.POINTER(CacheStruct),
                                                  _F, _I, _I, _VP, _SZ, _VP, _VP]
        L.fastar_annsa_combine.argtypes = [_I, _I, _I, _I, _VP, _SZ, _VP, _VP, _VP, _VP]
        L.fastar_tempcache_merge_rep.argtypes = [ctypes.POINTER(CacheStruct), _VP, _VP, _VP, _I, _I,
                                                 ctypes.c_int32, _F, _I, _VP, _VP, _VP, _SZ, _VP, _VP, _VP]
        L.fastar_tempcache_merge_search.argtypes = [ctypes.POINTER(CacheStruct), _VP, _VP, _VP, _I, _I,
                                                    ctypes.c_int32, _F, _I, _VP, _VP, _SZ, _VP, _VP, _VP]
        L.fastar_annsa_quant_attention.argtypes = [_I, _VP, _I, ctypes.POINTER(CacheStruct), _F, _I, _I, _VP, _VP,
                                                   _VP, _VP, _SZ, _VP, _VP]
        L.fastar_annca_quant_attention.argtypes = [_I, _VP, _VP, _VP, _I, _I, _I, _I, _F, _I, _I, _VP, _VP, _VP,
                                                   _SZ, _VP, _VP]
        L.fastar_rope_plan_init.argtypes = [_VP, _I, _I, ctypes.POINTER(_I), _I, ctypes.POINTER(ctypes.c_double)]
        L.fastar_rope.argtypes = [_I, _VP, _I64, _I64, _I, _I, _I, _VP, _VP, _I, _VP, _I64, _I64, _VP, _VP]
        L.fastar_page_append.argtypes = [_VP, _VP, _I64, _I64, _VP, _I64, _I64, _I, _VP, _VP, _VP, _VP, _I64, _I64,
                                         _I, _VP, _VP, _VP]
        L.fastar_branch_attention.argtypes = [_I, _VP, _I, _I, _VP, _VP, _VP, _F, _I, _VP, _VP, _VP, _SZ, _VP, _VP]
        for name in EXPORTS[7:]:
            getattr(L, name).restype = _I
        _lib = L
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str):
    if rc != 0:
        raise FastarError(rc, where)


def fastar_check_bounded_wait(polls, status, stream=None):
    """Run the library's bounded-wait error path once (see the C header):
    afterwards `status` holds FASTAR_ERR_TIMEOUT (17) unless it already held
    an error."""
    _check(lib().fastar_check_bounded_wait(int(polls), _p(status), _stream(stream)),
           "fastar_check_bounded_wait")


def fastar_launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().fastar_launch_count())


class LaunchTimer:
    """Per-kernel device durations of the library's launches (diagnostic).

    Usage: t = LaunchTimer(n); t.begin(); <calls on the current stream>;
    t.end() -> [(kernel name, ms), ...] in launch order.
    """

    def __init__(self, capacity: int):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        for e in self.events:          # create the underlying CUDA events now
            e.record()
        self.start = torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        self._handles = (ctypes.c_void_p * capacity)(*[e.cuda_event for e in self.events])

    def begin(self):
        self.start.record()
        _check(lib().fastar_timing_begin(ctypes.cast(self._handles, ctypes.c_void_p), len(self.events)),
               "fastar_timing_begin")

    def end(self):
        n = int(lib().fastar_timing_end())
        names = [lib().fastar_timing_name(i).decode() for i in range(n)]
        torch.cuda.synchronize()
        out, prev = [], self.start
        for i in range(n):
            out.append((names[i], prev.elapsed_time(self.events[i])))
            prev = self.events[i]
        return out


def fastar_workspace_size(op: int, H: int, N: int, D: int, T: int, B: int, C: int) -> int:
    return int(lib().fastar_workspace_size(op, H, N, D, T, B, C))


def _ws(op, H, N, D, T, B, C, ws, device):
    need = fastar_workspace_size(op, H, N, D, T, B, C)
    if need == 0:
        return None, 0
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def fastar_hash(x, planes, T, B, codes, perm=None, offsets=None, status=None, stream=None):
    """codes [H][T][N] (and optional CSR perm/offsets) of x [H][N][D]."""
    H, N, D = x.shape
    _check(lib().fastar_hash(_dt(x), _p(x), H, N, D, _p(planes), T, B, _p(codes), _p(perm),
                             _p(offsets), None, 0, _p(status), _stream(stream)), "fastar_hash")


def fastar_bucket_csr(codes, B, perm, offsets, status=None, stream=None):
    """perm / offsets of codes [..., N] (leading dims flattened into groups)."""
    N = codes.shape[-1]
    G = codes.numel() // max(N, 1)
    _check(lib().fastar_bucket_csr(_p(codes), G, N, B, _p(perm), _p(offsets), _p(status),
                                   _stream(stream)), "fastar_bucket_csr")


def fastar_hash_many(jobs, planes, T, B, status=None, stream=None):
    """One pass over up to MAX_HASH_JOBS inputs that share H and D.

    jobs: list of (x [H][N][D], codes [H][T][N], perm or None, offsets or
    None); the result equals one fastar_hash call per job."""
    if not 1 <= len(jobs) <= MAX_HASH_JOBS:
        raise ValueError(f"1 to {MAX_HASH_JOBS} jobs")
    arr = (HashJob * len(jobs))()
    H, _, D = jobs[0][0].shape
    for j, (x, codes, perm, offsets) in enumerate(jobs):
        if x.shape[0] != H or x.shape[2] != D or x.dtype != jobs[0][0].dtype:
            raise ValueError("jobs must share H, D and the dtype")
        arr[j] = HashJob(_p(x), x.shape[1], _p(codes), _p(perm), _p(offsets))
    _check(lib().fastar_hash_many(_dt(jobs[0][0]), len(jobs), arr, H, D, _p(planes), T, B, None, 0,
                                  _p(status), _stream(stream)), "fastar_hash_many")


class Cache:
    """Device buffers of one layer's merged cache (allocated once, torch-owned)."""

    def __init__(self, H, C, D, T, B, dtype=torch.bfloat16, device="cuda"):
        self.H, self.C, self.D, self.T, self.B, self.dtype = H, C, D, T, B, dtype
        dev = torch.device(device)
        self.K = torch.zeros(H, C, D, dtype=dtype, device=dev)
        self.V = torch.zeros(H, C, D, dtype=dtype, device=dev)
        self.m = torch.zeros(H, C, dtype=torch.int32, device=dev)
        self.codes = torch.zeros(H, T, C, dtype=torch.int32, device=dev)
        self.last_frame = torch.full((H, C), -1, dtype=torch.int32, device=dev)
        self.size = torch.zeros(H, dtype=torch.int32, device=dev)
        self.inserted = torch.zeros(H, dtype=torch.int64, device=dev)
        self.evicted = torch.zeros(H, dtype=torch.int64, device=dev)
        self.perm = torch.zeros(H, T, C, dtype=torch.int32, device=dev)
        self.offsets = torch.zeros(H, T, (1 << B) + 1, dtype=torch.int32, device=dev)

    BUFFERS = ("K", "V", "m", "codes", "last_frame", "size", "inserted", "evicted", "perm", "offsets")

    @classmethod
    def view(cls, T, B, **buffers):
        """A cache description over existing tensors (nothing is allocated):
        K, V [H][C][D], m, last_frame [H][C], codes, perm [H][T][C], size [H],
        inserted, evicted [H] and offsets [H][T][2^B+1], all given."""
        c = cls.__new__(cls)
        c.H, c.C, c.D = buffers["K"].shape
        c.T, c.B, c.dtype = T, B, buffers["K"].dtype
        for n in cls.BUFFERS:
            setattr(c, n, buffers[n])
        return c

    def struct(self) -> CacheStruct:
        return CacheStruct(self.H, self.D, self.C, self.T, self.B,
                           BF16 if self.dtype == torch.bfloat16 else F32,
                           *[getattr(self, n).data_ptr() for n in self.BUFFERS])

    def snapshot(self) -> dict:
        return {n: getattr(self, n).clone() for n in self.BUFFERS}

    def restore(self, snap: dict):
        for n in self.BUFFERS:
            getattr(self, n).copy_(snap[n], non_blocking=True)

    def save(self, path: str):
        """Write a checkpoint of the cache (every buffer and its shape
        parameters) to `path` with torch.save; a rollout resumed from it
        continues bit for bit as if it had not stopped."""
        torch.save({"shape": (self.H, self.C, self.D, self.T, self.B, str(self.dtype)),
                    "buffers": {n: getattr(self, n).detach().cpu() for n in self.BUFFERS}}, path)

    def load(self, path: str):
        """Restore a checkpoint written by `save` into this cache's buffers
        (same H, C, D, T, B and dtype, or ValueError)."""
        ck = torch.load(path, map_location="cpu")
        if tuple(ck["shape"]) != (self.H, self.C, self.D, self.T, self.B, str(self.dtype)):
            raise ValueError(f"checkpoint of shape {ck['shape']} does not fit this cache")
        for n in self.BUFFERS:
            getattr(self, n).copy_(ck["buffers"][n])

    def nbytes(self) -> int:
        return sum(getattr(self, n).numel() * getattr(self, n).element_size() for n in self.BUFFERS)


def fastar_tempcache_merge(cache: Cache, k_new, v_new, codes_new, F, n_f, first_frame, tau,
                           match_out=None, ws=None, status=None, stream=None, codes_ready=None,
                           rep="last", planes=None, search="prev"):
    """Merge the F frames of a chunk (k_new/v_new [H][F*n_f][D]) into `cache`.

    codes_ready: a torch.cuda.Event after which codes_new and v_new are
    final (fastar_tempcache_merge_ev); None: they are ready on `stream`.
    rep: "last" (the method's representative) or "mean" (the mean-key
    ablation, fastar_tempcache_merge_rep; needs the hash `planes`).
    search: "prev" (the previous frame's groups, the method), "lsh" (every
    earlier group sharing a bucket) or "quant<bits>" (the previous frame's
    groups ranked by their b-bit quantised keys), fastar_tempcache_merge_search."""
    ws, nbytes = _ws(OP_MERGE, cache.H, n_f, cache.D, cache.T, cache.B, cache.C, ws, k_new.device)
    cs = cache.struct()
    if search != "prev":
        if rep != "last":
            raise ValueError("the search over every earlier frame keeps the last key")
        _check(lib().fastar_tempcache_merge_search(
            ctypes.byref(cs), _p(k_new), _p(v_new), _p(codes_new), F, n_f, first_frame, tau, search_code(search),
            _p(match_out), _p(ws), nbytes, _p(status), _stream(stream),
            None if codes_ready is None else codes_ready.cuda_event), "fastar_tempcache_merge_search")
        return
    if rep != "last":
        _check(lib().fastar_tempcache_merge_rep(
            ctypes.byref(cs), _p(k_new), _p(v_new), _p(codes_new), F, n_f, first_frame, tau, REPS[rep],
            _p(planes), _p(match_out), _p(ws), nbytes, _p(status), _stream(stream),
            None if codes_ready is None else codes_ready.cuda_event), "fastar_tempcache_merge_rep")
        return
    args = (ctypes.byref(cs), _p(k_new), _p(v_new), _p(codes_new), F, n_f, first_frame, tau,
            _p(match_out), _p(ws), nbytes, _p(status), _stream(stream))
    if codes_ready is None:
        _check(lib().fastar_tempcache_merge(*args), "fastar_tempcache_merge")
    else:
        _check(lib().fastar_tempcache_merge_ev(*args, codes_ready.cuda_event),
               "fastar_tempcache_merge_ev")


def fastar_annca_prune(q_codes, p_codes, F, n_f, B, kept_idx, kept_cnt, status=None, stream=None):
    """kept_idx [H][F][P] / kept_cnt [H][F] of the prompt tokens per frame."""
    H, T, _ = q_codes.shape
    P = p_codes.shape[2]
    _check(lib().fastar_annca_prune(_p(q_codes), _p(p_codes), H, F, n_f, P, T, B, _p(kept_idx),
                                    _p(kept_cnt), None, 0, _p(status), _stream(stream)),
           "fastar_annca_prune")


def fastar_annca_attention(q, k_p, v_p, kept_idx, kept_cnt, F, n_f, scale, out, ws=None,
                           status=None, stream=None):
    """out [H][F*n_f][D]: cross-attention of each frame over its kept tokens.

    ws: a uint8 device tensor of at least
    fastar_workspace_size(OP_ANNCA, H, F, D, 0, 0, P) bytes; one is allocated
    for the call when it is None."""
    H, Nq, D = q.shape
    P = k_p.shape[1]
    ws, nbytes = _ws(OP_ANNCA, H, F, D, 0, 0, P, ws, q.device)
    _check(lib().fastar_annca_attention(_dt(q), _p(q), _p(k_p), _p(v_p), _p(kept_idx),
                                        _p(kept_cnt), H, F, n_f, P, D, scale, _p(out), _p(ws), nbytes,
                                        _p(status), _stream(stream)), "fastar_annca_attention")


def fastar_annsa_attention_part(q, q_codes, q_perm, q_offsets, cache: Cache, scale, part_base, part_total, ws,
                                status=None, stream=None):
    """Per-table partials of AnnSA over `cache` into slots part_base.. of ws."""
    H, Nq, D = q.shape
    nbytes = ws.numel() * ws.element_size()
    cs = cache.struct()
    _check(lib().fastar_annsa_attention_part(_dt(q), _p(q), _p(q_codes), _p(q_perm), _p(q_offsets), Nq,
                                             ctypes.byref(cs), scale, part_base, part_total, _p(ws), nbytes,
                                             _p(status), _stream(stream)), "fastar_annsa_attention_part")


def fastar_annsa_combine(part_total, ws, out, lse=None, status=None, stream=None):
    """out [H][Nq][D] (and lse) from the part_total partials in ws."""
    H, Nq, D = out.shape
    _check(lib().fastar_annsa_combine(H, Nq, D, part_total, _p(ws), ws.numel() * ws.element_size(), _p(out),
                                      _p(lse), _p(status), _stream(stream)), "fastar_annsa_combine")


def fastar_annsa_attention(q, q_codes, q_perm, q_offsets, cache: Cache, scale, out, lse=None,
                           ws=None, status=None, stream=None):
    """out [H][Nq][D] (and lse [H][Nq]): bucket-restricted attention over `cache`."""
    H, Nq, D = q.shape
    ws, nbytes = _ws(OP_ANNSA, cache.H, Nq, cache.D, cache.T, cache.B, cache.C, ws, q.device)
    cs = cache.struct()
    _check(lib().fastar_annsa_attention(_dt(q), _p(q), _p(q_codes), _p(q_perm), _p(q_offsets), Nq,
                                        ctypes.byref(cs), scale, _p(out), _p(lse), _p(ws), nbytes,
                                        _p(status), _stream(stream)), "fastar_annsa_attention")


def fastar_annsa_quant_attention(q, cache: Cache, scale, topk, bits, out, lse=None, sel_mask=None, ws=None,
                                 status=None, stream=None):
    """out [H][Nq][D]: each query attends its topk live slots of largest
    approximate score under bits-bit quantised keys (sel_mask optional
    [H][Nq][ceil(C/32)] int32 receives the kept slots as bits)."""
    H, Nq, D = q.shape
    ws, nbytes = _ws(OP_QUANT, cache.H, Nq, cache.D, bits, 0, cache.C, ws, q.device)
    cs = cache.struct()
    _check(lib().fastar_annsa_quant_attention(_dt(q), _p(q), Nq, ctypes.byref(cs), scale, topk, bits, _p(out),
                                              _p(lse), _p(sel_mask), _p(ws), nbytes, _p(status), _stream(stream)),
           "fastar_annsa_quant_attention")


def fastar_annca_quant_attention(q, k_p, v_p, scale, topk, bits, out, sel_mask=None, ws=None, status=None,
                                 stream=None):
    """out [H][Nq][D]: each query attends its topk prompt tokens of largest
    approximate score under bits-bit quantised prompt keys."""
    H, Nq, D = q.shape
    P = k_p.shape[1]
    ws, nbytes = _ws(OP_QUANT, H, Nq, D, bits, 0, P, ws, q.device)
    _check(lib().fastar_annca_quant_attention(_dt(q), _p(q), _p(k_p), _p(v_p), H, Nq, P, D, scale, topk, bits,
                                              _p(out), _p(sel_mask), _p(ws), nbytes, _p(status), _stream(stream)),
           "fastar_annca_quant_attention")


# ---- branched rollouts: rotary positions, pages, attention over a shared prefix

class RopePlan:
    """Rotary positions with several axes: dims[a] channels turn by axis a
    (e.g. (44, 42, 42) for time, height and width of a 128-channel head), the
    channels behind their sum are copied.

    pairing: "adjacent" (channels 2p, 2p+1) or "halves" (channels p, p + sum/2);
    freqs: radians per position of each of the sum/2 pairs; by default pair i
    of axis a has base**(-2 i / dims[a])."""

    def __init__(self, D, dims, base=10000.0, pairing="adjacent", freqs=None):
        dims = [int(d) for d in dims]
        if pairing not in PAIRINGS:
            raise ValueError(f"unknown pairing {pairing!r}")
        if freqs is None:
            freqs = [float(base) ** (-2.0 * i / d) for d in dims for i in range(d // 2)]
        freqs = [float(f) for f in freqs]
        if len(freqs) != sum(dims) // 2:
            raise ValueError(f"{len(freqs)} frequencies for {sum(dims) // 2} pairs")
        self.D, self.dims, self.pairing, self.axes = D, tuple(dims), pairing, len(dims)
        self.struct = RopePlanStruct()
        self.addr = ctypes.addressof(self.struct)
        _check(lib().fastar_rope_plan_init(self.addr, D, len(dims), (_I * len(dims))(*dims), PAIRINGS[pairing],
                                           (ctypes.c_double * len(freqs))(*freqs)), "fastar_rope_plan_init")


def _at(t, dev):
    """Pointer of a contiguous tensor of GPU `dev` (None: NULL)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _rows(t, dev, what):
    """Pointer and (head, token) strides of rows [H][N][D] on GPU `dev`."""
    if t.get_device() != dev:
        raise ValueError("tensors must be on one GPU")
    st = t.stride()
    if len(st) != 3 or st[2] != 1:
        raise ValueError(f"{what} must be [heads][tokens][D] with contiguous rows")
    return t.data_ptr(), st[0], st[1]


def _positions(pos, N, plan, dev):
    if pos is None:
        return None
    if pos.dtype is not torch.int32 or pos.shape != (N, plan.axes):
        raise ValueError(f"positions must be int32 [{N}][{plan.axes}]")
    return _at(pos, dev)


def _int32(t, n, dev, what):
    if t.dtype is not torch.int32 or t.numel() != n:
        raise ValueError(f"{what} must be int32 with {n} entries")
    return _at(t, dev)


def _gpu(t):
    """The GPU that holds t."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    return dev


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_gpu = getattr(torch._C, "_cuda_getDevice", None)


def _on(dev, stream, call, *args):
    """call(*args, stream) on GPU `dev`: on its current stream by default."""
    stream = _raw_stream(dev) if stream is None else _stream(stream)
    if dev == _current_gpu():
        return call(*args, stream)
    with torch.cuda.device(dev):
        return call(*args, stream)


def fastar_rope(x, pos, plan: RopePlan, out, inverse=False, status=None, stream=None):
    """out = the rows of x [H][N][D] rotated by pos [N][axes] (int32).

    x and out may have any head and token strides (the transpose of a
    projection's [N][H][D] output, for one); out may be x itself.
    inverse: turn back, which is also the gradient of the forward rotation."""
    shape = H, N, D = x.shape
    dt, dev = x.dtype, x.get_device()
    if out.shape != shape or out.dtype is not dt or D != plan.D:
        raise ValueError("x, out and the plan must agree in shape and dtype")
    xs, os = x.stride(), out.stride()
    if dev < 0 or out.get_device() != dev or xs[2] != 1 or os[2] != 1:
        _gpu(x), _rows(x, dev, "x"), _rows(out, dev, "out")  # says which
    args = (BF16 if dt is torch.bfloat16 else _dt(x), x.data_ptr(), xs[0], xs[1], H, N, D, _positions(pos, N, plan, dev),
            plan.addr, 1 if inverse else 0, out.data_ptr(), os[0], os[1], _at(status, dev))
    if stream is None and dev == _current_gpu():
        rc = (_lib or lib()).fastar_rope(*args, _raw_stream(dev))
    else:
        rc = _on(dev, stream, lib().fastar_rope, *args)
    if rc:
        raise FastarError(rc, "fastar_rope")


class _Bound:
    """Holds the tensors that a call's struct points at.  Assigning one of them
    drops the struct and what follows from the shapes; the next use takes them
    from the tensors that are there then."""
    _tensors = _derived = ()

    def __setattr__(self, name, value):
        if name in self._tensors:
            for d in self._derived:
                self.__dict__.pop(d, None)
        object.__setattr__(self, name, value)

    def __getattr__(self, name):
        if name not in self._derived:
            raise AttributeError(f"{type(self).__name__!r} object has no attribute {name!r}")
        self._bind()
        return self.__dict__[name]


class PagedKV(_Bound):
    """Keys and values of a layer's branches in pages (torch-owned):
    K, V [n_pages][H][page][D], table [B][max_pages] int32 page ids, len [B]
    int32 positions of each branch, the new tokens of a call included.  The
    caller hands out the pages (table) and counts the positions (len): in
    place, or by assigning another tensor (a tensor whose own storage is
    replaced, as by resize_, has to be assigned again)."""
    _tensors = ("K", "V", "table", "len")
    _derived = ("n_pages", "H", "page", "D", "B", "max_pages", "dtype", "device", "struct", "addr")

    def __init__(self, H, D, page, n_pages, B, max_pages, dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        self._set(torch.zeros(n_pages, H, page, D, dtype=dtype, device=dev),
                  torch.zeros(n_pages, H, page, D, dtype=dtype, device=dev),
                  torch.zeros(B, max_pages, dtype=torch.int32, device=dev),
                  torch.zeros(B, dtype=torch.int32, device=dev))

    @classmethod
    def view(cls, K, V, table, length):
        """Pages over existing tensors (nothing is allocated)."""
        p = cls.__new__(cls)
        p._set(K, V, table, length)
        return p

    def _set(self, K, V, table, length):
        self.K, self.V, self.table, self.len = K, V, table, length
        self._bind()

    def _bind(self):
        K, V, table, length = self.K, self.V, self.table, self.len
        if K.shape != V.shape or K.dtype != V.dtype or K.dim() != 4 or table.dim() != 2:
            raise ValueError("K and V are [n_pages][H][page][D], the table [B][max_pages]")
        n_pages, H, page, D = K.shape
        B, max_pages = table.shape
        dev = _gpu(K)
        struct = PagesStruct(H, D, page, n_pages, B, max_pages, _dt(K), _at(K, dev), _at(V, dev),
                             _int32(table, table.numel(), dev, "the table"), _int32(length, B, dev, "the lengths"))
        self.n_pages, self.H, self.page, self.D, self.B, self.max_pages = n_pages, H, page, D, B, max_pages
        self.dtype, self.device, self.struct, self.addr = K.dtype, dev, struct, ctypes.addressof(struct)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.K, self.V, self.table, self.len))


class Prefix(_Bound):
    """The rows that every branch attends: K, V [H][C][D], optional counts m
    [H][C] int32 (+ ln m) and live rows size [H] int32.  They change in place
    or by assigning other tensors."""
    _tensors = ("K", "V", "m", "size")
    _derived = ("device", "struct", "addr")

    def __init__(self, K, V, m=None, size=None):
        self.K, self.V, self.m, self.size = K, V, m, size
        self._bind()

    def _bind(self):
        K, V, m, size = self.K, self.V, self.m, self.size
        if K.shape != V.shape or K.dtype != V.dtype or K.dim() != 3:
            raise ValueError("K and V are [H][C][D]")
        H, C, D = K.shape
        dev = _gpu(K)
        struct = PrefixStruct(H, C, D, _dt(K), _at(K, dev), _at(V, dev),
                              None if m is None else _int32(m, H * C, dev, "m"),
                              None if size is None else _int32(size, H, dev, "size"))
        self.device, self.struct, self.addr = dev, struct, ctypes.addressof(struct)

    @classmethod
    def of(cls, cache: Cache):
        """The live groups of a merged cache, each with its + ln m."""
        return cls(cache.K, cache.V, m=cache.m, size=cache.size)


def fastar_page_append(pages: PagedKV, k, v, cu, pos=None, plan: RopePlan | None = None, q=None, q_out=None,
                       status=None, stream=None):
    """Put the keys and values of new tokens k, v [H][N][D] (any head and
    token strides) into the pages: token cu[b] + i of branch b becomes
    position len[b] - n_b + i.  The keys are rotated by pos and plan (none:
    stored as they are); optional queries q [Hq][N][D] are rotated into q_out
    [Hq][N][D] in the same pass."""
    shape = H, N, D = k.shape
    dt, dev = pages.dtype, pages.device
    if v.shape != shape or H != pages.H or D != pages.D or k.dtype is not dt or v.dtype is not dt:
        raise ValueError("k and v do not fit the pages")
    if (plan is None) != (pos is None):
        raise ValueError("positions and their plan come together")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if plan is not None and plan.D != D:
        raise ValueError("the plan has another head dimension")
    ks, vs = k.stride(), v.stride()
    if k.get_device() != dev or v.get_device() != dev or ks[2] != 1 or vs[2] != 1:
        _rows(k, dev, "k"), _rows(v, dev, "v")  # says which
    qa, Hq, qs = None, 0, (0, 0)
    if q is not None:
        Hq, n, d = q.shape
        if q_out.shape != (Hq, n, d) or n != N or d != D or q.dtype is not dt or q_out.dtype is not dt:
            raise ValueError("q and q_out do not fit k")
        qa, *qs = _rows(q, dev, "q")
    args = (pages.addr, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], N,
            _int32(cu, pages.B + 1, dev, "cu"), _positions(pos, N, plan, dev), None if plan is None else plan.addr,
            qa, qs[0], qs[1], Hq, _at(q_out, dev), _at(status, dev))
    if stream is None and dev == _current_gpu():
        rc = (_lib or lib()).fastar_page_append(*args, _raw_stream(dev))
    else:
        rc = _on(dev, stream, lib().fastar_page_append, *args)
    if rc:
        raise FastarError(rc, "fastar_page_append")


def branch_workspace_size(Hq: int, H: int, N: int, D: int) -> int:
    """Bytes of workspace of fastar_branch_attention for N tokens."""
    return fastar_workspace_size(OP_BRANCH, Hq, N, D, H, 0, 0)


def fastar_branch_attention(q, cu, prefix: Prefix | None, pages: PagedKV, scale, out, lse=None, block=0, ws=None,
                            status=None, stream=None):
    """out [Hq][N][D] (and lse [Hq][N]): every branch's tokens over the shared
    prefix and the branch's own pages.

    cu [B + 1] int32: token cu[b] + i of q is new token i of branch b, whose
    keys are already in the pages (fastar_page_append).  block 0: a token sees
    every position of its branch; n: those of its own and earlier blocks of n
    positions (1: causal).  ws: a uint8 device tensor of at least
    branch_workspace_size(Hq, H, N, D) bytes; one is allocated for the call
    when it is None."""
    Hq, N, D = q.shape
    if out.shape != q.shape or not out.dtype == q.dtype == pages.dtype or D != pages.D:
        raise ValueError("q, out and the pages must agree in shape and dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() != Hq * N):
        raise ValueError("lse must be float32 [Hq][N]")
    dev = pages.device
    if prefix is not None and prefix.device != dev:
        raise ValueError("tensors must be on one GPU")
    if ws is None:
        # from the pool of the call's stream: a free block of another stream's may
        # still be in use there
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(_stream(stream)), device=q.device)
        with torch.cuda.stream(stream):
            ws = torch.empty(max(1, branch_workspace_size(Hq, pages.H, N, D)), dtype=torch.uint8, device=q.device)
    rc = _on(dev, stream, (_lib or lib()).fastar_branch_attention, pages.struct.dt, _at(q, dev), Hq, N,
             _int32(cu, pages.B + 1, dev, "cu"), None if prefix is None else prefix.addr, pages.addr, scale, block,
             _at(out, dev), _at(lse, dev), _at(ws, dev), ws.numel() * ws.element_size(), _at(status, dev))
    if rc:
        raise FastarError(rc, "fastar_branch_attention")
