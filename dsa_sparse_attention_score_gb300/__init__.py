"""Python binding of the GB300 DSA hot-path library (libdsa_gb300.so).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  The
functions carry the C-ABI names and raise DsaError on any non-OK status.
There is no fallback: if the compiled library is missing, loading raises.

Tensor conventions (all CUDA, contiguous):
  fp16 tensors are torch.float16, bf16 tensors torch.bfloat16,
  positions torch.int32, offsets torch.int64, scores/outputs torch.float32.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdsa_gb300.so")

DSA_OK = 0
DSA_ERR_INVALID_ARGUMENT = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_MISALIGNED = 3
DSA_ERR_WORKSPACE_TOO_SMALL = 4
DSA_ERR_CUDA = 5
DSA_ERR_DEVICE = 6

DSA_DEV_BAD_POSITION = 1
DSA_DEV_BAD_INDEX = 2
DSA_DEV_TIMEOUT = 4
DSA_DEV_SMEM_LAYOUT = 8

DSA_KEY_F32 = 0
DSA_KEY_F16 = 1

DSA_DT_F32 = 0
DSA_DT_F16 = 1
DSA_DT_BF16 = 2

DSA_ROPE_NONE = 0
DSA_ROPE_LINEAR = 1
DSA_ROPE_NTK = 2
DSA_ROPE_YARN = 3

DSA_OP_K_APPEND = 0
DSA_OP_INDEXER_SCORE = 1
DSA_OP_TOPK = 2
DSA_OP_SPARSE_ATTN = 3
DSA_OP_DECODE = 4
DSA_OP_KPOOL = 5
DSA_OP_MLA_ATTN = 6

KPOOL = 4            # positions per pool of the kpool indexer
KPOOL_ROW = 257      # fp16 values per packed indexer row: k | gate | valid
Q8_ROW = 640         # codes per row of the 8-bit latent cache (512 without a tail)

# Every symbol the header declares, with (restype, argtypes).
_P = C.c_void_p
_I = C.c_int
_I64 = C.c_int64
_SZ = C.c_size_t
_F = C.c_float


class dsa_batch_t(C.Structure):
    _fields_ = [("batch", C.c_int32), ("total_q", C.c_int32), ("max_q_per_seq", C.c_int32),
                ("max_kv", C.c_int32), ("cache_rows", C.c_int64), ("cu_q", _P), ("q_pos", _P),
                ("kv_off", _P)]


_BP = C.POINTER(dsa_batch_t)
SIGNATURES = {
    "dsa_indexer_k_append": (_I, [_P, _I, _BP, _P, _I, _P, _SZ, _P]),
    "dsa_indexer_score": (_I, [_P, _P, _P, _BP, _I, _I, _P, _I64, _P, _SZ, _P]),
    "dsa_topk": (_I, [_P, _I64, _BP, _I, _P, _P, _SZ, _P]),
    "dsa_topk_sink": (_I, [_P, _I64, _BP, _I, _I, _P, _P, _P, _SZ, _P]),
    "dsa_sparse_mla_attn": (_I, [_P, _P, _P, _BP, _P, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "dsa_sparse_mla_attn_nope": (_I, [_P, _P, _BP, _P, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "dsa_decode": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _BP, _I, _I, _I, _F, _I, _P, _P, _P, _P, _SZ, _P]),
    "dsa_decode_sink": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _BP, _I, _I, _I, _F, _I, _I, _P, _P, _P, _P, _P,
                             _SZ, _P]),
    "dsa_decode_paged": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _BP, C.c_void_p, _I, _I, _I, _F, _I, _P, _P, _P, _P,
                              _SZ, _P]),
    "dsa_decode_noalloc": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _BP, _I, _I, _I, _F, _I, _P, _P, _P, _P]),
    "dsa_workspace_size": (_I, [_I, _BP, _I, _I, _I, C.POINTER(C.c_size_t)]),
    "dsa_workspace_init": (_I, [_P, _SZ, _P]),
    "dsa_decode_launches": (_I, [_BP, _I, _I, _I, C.POINTER(C.c_int)]),
    "dsa_read_device_status": (_I, [_P, _P, C.POINTER(C.c_uint32)]),
    "dsa_status_string": (C.c_char_p, [_I]),
    "dsa_set_trace_events": (_I, [_P, _I]),
    "dsa_set_timeline": (_I, [_P]),
    "dsa_set_test_faults": (_I, [C.c_uint64, _I]),
    "dsa_kpool_append": (_I, [_P, _P, _P, _BP, _P, _P, _I64, _P, _SZ, _P]),
    "dsa_kpool_select": (_I, [_P, _P, _P, _P, _I64, _BP, _I, _I, _P, _P, _SZ, _P]),
    "dsa_decode_kpool": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _BP, _I, _I, _I, _F, _P, _P, _P, _P, _SZ,
                              _P]),
    "dsa_rope_frequencies": (_I, [_I, C.c_double, _I, C.c_double, _I, C.c_double, C.c_double, _P, _P]),
    "dsa_rope": (_I, [_P, _I64, _I64, _P, _I64, _I64, _I, _I, _I, _I, _I, _P, _P, _I, _P]),
    "dsa_kv_append": (_I, [_P, _I64, _P, _I64, _I, _BP, _P, _P, _P, _P, _SZ, _P]),
    "dsa_kv_append_q8": (_I, [_P, _I64, _P, _I64, _I, _BP, _P, _P, _P, _P, _P, _SZ, _P]),
    "dsa_kv_read_q8": (_I, [_P, _P, _I, _BP, _P, _P, _I, _I64, _P, _SZ, _P]),
    "dsa_sparse_mla_attn_q8": (_I, [_P, _P, _P, _P, _BP, _P, _P, _I, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "dsa_rms_norm": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I, _F, _P, _I64, _I, _I, _I, _P]),
    "dsa_rms_norm_q8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I, _F, _P, _P, _I, _I, _I, _I, _P]),
    "dsa_mla_attn": (_I, [_P, _P, _P, _BP, _P, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "dsa_mla_attn_window": (_I, [_P, _P, _P, _BP, _P, _I, _I, _I, _P, _F, _P, _I, _P, _P, _SZ, _P]),
    "dsa_version": (_I, []),
}

_LIB = None


class DsaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lib().dsa_status_string(code).decode()} (code {code})")


def lib():
    """The loaded CUDA library.  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run dsa_sparse_attention_score_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(code: int, what: str):
    if code != DSA_OK:
        raise DsaError(code, what)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


# Fixed innermost extents of the tensors the calls take (include/dsa.h).
_WIDTH = {"k_new": 128, "gate_new": 128, "ape": 128, "q_idx": 128, "k_cache": 128, "q_lat": 512, "q_rope": 64, "kv_cache": 576,
          "kv_latent": 512, "out": 512}


def _req(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    if name in _WIDTH and (t.dim() < 2 or t.shape[-1] != _WIDTH[name]):
        raise TypeError(f"{name}: expected rows of {_WIDTH[name]} elements, got shape {tuple(t.shape)}")


@dataclass
class Batch:
    """Device batch description plus its host bounds."""
    cu_q: object           # int32 [B+1]
    q_pos: object          # int32 [T]
    kv_off: object         # int64 [B]
    max_q_per_seq: int
    max_kv: int
    cache_rows: int

    @classmethod
    def from_host(cls, cu_q, q_pos, kv_off, cache_rows: int, device="cuda",
                  max_q_per_seq: int | None = None, max_kv: int | None = None):
        import torch
        cu = torch.as_tensor(list(cu_q), dtype=torch.int32)
        qp = torch.as_tensor(list(q_pos), dtype=torch.int32)
        ko = torch.as_tensor(list(kv_off), dtype=torch.int64)
        mq = max_q_per_seq if max_q_per_seq is not None else int((cu[1:] - cu[:-1]).max())
        mk = max_kv if max_kv is not None else int(qp.max()) + 1
        return cls(cu.to(device), qp.to(device), ko.to(device), mq, mk, int(cache_rows))

    @property
    def B(self) -> int:
        return self.cu_q.numel() - 1

    @property
    def T(self) -> int:
        return self.q_pos.numel()

    def desc(self) -> dsa_batch_t:
        import torch
        _req(self.cu_q, torch.int32, "cu_q")
        _req(self.q_pos, torch.int32, "q_pos")
        _req(self.kv_off, torch.int64, "kv_off")
        return dsa_batch_t(self.B, self.T, self.max_q_per_seq, self.max_kv, self.cache_rows,
                           self.cu_q.data_ptr(), self.q_pos.data_ptr(), self.kv_off.data_ptr())


def dsa_workspace_size(op: int, batch: Batch, H_I: int, H: int, k: int) -> int:
    n = C.c_size_t(0)
    d = dsa_batch_t(batch.B, batch.T, batch.max_q_per_seq, batch.max_kv, batch.cache_rows, None, None, None)
    _check(lib().dsa_workspace_size(op, C.byref(d), H_I, H, k, C.byref(n)), "dsa_workspace_size")
    return n.value


def dsa_decode_launches(batch: Batch, H_I: int, H: int, k: int) -> int:
    n = C.c_int(0)
    d = dsa_batch_t(batch.B, batch.T, batch.max_q_per_seq, batch.max_kv, batch.cache_rows, None, None, None)
    _check(lib().dsa_decode_launches(C.byref(d), H_I, H, k, C.byref(n)), "dsa_decode_launches")
    return n.value


def dsa_workspace_init(ws, stream=None):
    _check(lib().dsa_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "dsa_workspace_init")


def workspace(op: int, batch: Batch, H_I: int = 1, H: int = 1, k: int = 1, device="cuda"):
    """Allocate (with torch) and initialise a workspace for `op`."""
    import torch
    n = dsa_workspace_size(op, batch, H_I, H, k)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    dsa_workspace_init(ws)
    return ws


def dsa_read_device_status(ws, stream=None) -> int:
    """Synchronises the stream; returns and clears the DSA_DEV_* bits."""
    f = C.c_uint32(0)
    code = lib().dsa_read_device_status(_ptr(ws), _stream(stream), C.byref(f))
    if code not in (DSA_OK, DSA_ERR_DEVICE):
        raise DsaError(code, "dsa_read_device_status")
    return f.value


def dsa_indexer_k_append(k_new, batch: Batch, k_cache, hadamard: bool, ws, stream=None):
    import torch
    kd = DSA_KEY_F16 if k_new.dtype == torch.float16 else DSA_KEY_F32
    _req(k_new, torch.float16 if kd == DSA_KEY_F16 else torch.float32, "k_new")
    _req(k_cache, torch.float16, "k_cache")
    d = batch.desc()
    _check(lib().dsa_indexer_k_append(_ptr(k_new), kd, C.byref(d), _ptr(k_cache), int(hadamard),
                                      _ptr(ws), ws.numel(), _stream(stream)), "dsa_indexer_k_append")


def dsa_indexer_score(q_idx, w, k_cache, batch: Batch, hadamard_q: bool, scores, ws, stream=None):
    import torch
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req(k_cache, torch.float16, "k_cache")
    _req(scores, torch.float32, "scores")
    d = batch.desc()
    _check(lib().dsa_indexer_score(_ptr(q_idx), _ptr(w), _ptr(k_cache), C.byref(d), q_idx.shape[1],
                                   int(hadamard_q), _ptr(scores), scores.shape[1], _ptr(ws), ws.numel(),
                                   _stream(stream)), "dsa_indexer_score")


def dsa_topk(scores, batch: Batch, k: int, idx, ws, stream=None):
    import torch
    _req(scores, torch.float32, "scores")
    _req(idx, torch.int32, "idx")
    d = batch.desc()
    _check(lib().dsa_topk(_ptr(scores), scores.shape[1], C.byref(d), k, _ptr(idx), _ptr(ws), ws.numel(),
                          _stream(stream)), "dsa_topk")


def dsa_topk_sink(scores, batch: Batch, k: int, n_sink: int, sink_pos0, idx, ws, stream=None):
    """dsa_topk with the first n_sink positions of each sequence (from
    sink_pos0[b], an int32 CUDA tensor [B], or 0 when None) forced in."""
    import torch
    _req(scores, torch.float32, "scores")
    _req(idx, torch.int32, "idx")
    _req(sink_pos0, torch.int32, "sink_pos0")
    d = batch.desc()
    _check(lib().dsa_topk_sink(_ptr(scores), scores.shape[1], C.byref(d), k, n_sink, _ptr(sink_pos0), _ptr(idx),
                               _ptr(ws), ws.numel(), _stream(stream)), "dsa_topk_sink")


def dsa_sparse_mla_attn(q_lat, q_rope, kv_cache, batch: Batch, idx, sm_scale: float, out, lse, ws,
                        stream=None):
    import torch
    _req(q_lat, torch.bfloat16, "q_lat")
    _req(q_rope, torch.bfloat16, "q_rope")
    _req(kv_cache, torch.bfloat16, "kv_cache")
    _req(idx, torch.int32, "idx")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    d = batch.desc()
    _check(lib().dsa_sparse_mla_attn(_ptr(q_lat), _ptr(q_rope), _ptr(kv_cache), C.byref(d), _ptr(idx),
                                     idx.shape[1], q_lat.shape[1], sm_scale, _ptr(out), _ptr(lse),
                                     _ptr(ws), ws.numel(), _stream(stream)), "dsa_sparse_mla_attn")


def dsa_sparse_mla_attn_nope(q_lat, kv_latent, batch: Batch, idx, sm_scale: float, out, lse, ws, stream=None):
    """MLA-NoPE: q_lat [T,H,512] against latent rows kv_latent [rows,512] (no rope tail)."""
    import torch
    _req(q_lat, torch.bfloat16, "q_lat")
    _req(kv_latent, torch.bfloat16, "kv_latent")
    _req(idx, torch.int32, "idx")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    d = batch.desc()
    _check(lib().dsa_sparse_mla_attn_nope(_ptr(q_lat), _ptr(kv_latent), C.byref(d), _ptr(idx), idx.shape[1],
                                          q_lat.shape[1], sm_scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                          _stream(stream)), "dsa_sparse_mla_attn_nope")


def dsa_decode(k_new, q_idx, w, q_lat, q_rope, k_cache, kv_cache, batch: Batch, k: int, sm_scale: float,
               hadamard: bool, out, lse, idx_out, ws, stream=None):
    import torch
    kd = DSA_KEY_F16 if k_new.dtype == torch.float16 else DSA_KEY_F32
    _req(k_new, torch.float16 if kd == DSA_KEY_F16 else torch.float32, "k_new")
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req(q_lat, torch.bfloat16, "q_lat")
    _req(q_rope, torch.bfloat16, "q_rope")
    _req(k_cache, torch.float16, "k_cache")
    _req(kv_cache, torch.bfloat16, "kv_cache")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    _req(idx_out, torch.int32, "idx_out")
    d = batch.desc()
    _check(lib().dsa_decode(_ptr(k_new), kd, _ptr(q_idx), _ptr(w), _ptr(q_lat), _ptr(q_rope), _ptr(k_cache),
                            _ptr(kv_cache), C.byref(d), q_idx.shape[1], q_lat.shape[1], k, sm_scale,
                            int(hadamard), _ptr(out), _ptr(lse), _ptr(idx_out), _ptr(ws), ws.numel(),
                            _stream(stream)), "dsa_decode")


class dsa_paging_t(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("max_blocks", C.c_int32), ("block_size", C.c_int32)]


def dsa_decode_paged(k_new, q_idx, w, q_lat, q_rope, k_cache, kv_cache, batch: Batch, block_table,
                     block_size: int, k: int, sm_scale: float, hadamard: bool, out, lse, idx_out, ws,
                     stream=None):
    """dsa_decode over paged caches: block_table is an int32 CUDA tensor
    [B, max_blocks]; position pos of sequence b lives at cache row
    block_table[b, pos // block_size] * block_size + pos % block_size."""
    import torch
    kd = DSA_KEY_F16 if k_new.dtype == torch.float16 else DSA_KEY_F32
    _req(k_new, torch.float16 if kd == DSA_KEY_F16 else torch.float32, "k_new")
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req(q_lat, torch.bfloat16, "q_lat")
    _req(q_rope, torch.bfloat16, "q_rope")
    _req(k_cache, torch.float16, "k_cache")
    _req(kv_cache, torch.bfloat16, "kv_cache")
    _req(block_table, torch.int32, "block_table")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    _req(idx_out, torch.int32, "idx_out")
    d = batch.desc()
    pg = dsa_paging_t(block_table.data_ptr(), block_table.shape[1], block_size)
    _check(lib().dsa_decode_paged(_ptr(k_new), kd, _ptr(q_idx), _ptr(w), _ptr(q_lat), _ptr(q_rope), _ptr(k_cache),
                                  _ptr(kv_cache), C.byref(d), C.byref(pg), q_idx.shape[1], q_lat.shape[1], k,
                                  sm_scale, int(hadamard), _ptr(out), _ptr(lse), _ptr(idx_out), _ptr(ws),
                                  ws.numel(), _stream(stream)), "dsa_decode_paged")


def dsa_decode_sink(k_new, q_idx, w, q_lat, q_rope, k_cache, kv_cache, batch: Batch, k: int, sm_scale: float,
                    hadamard: bool, n_sink: int, sink_pos0, out, lse, idx_out, ws, stream=None):
    """dsa_decode with the attention sink forced into every selection (see
    dsa_topk_sink)."""
    import torch
    kd = DSA_KEY_F16 if k_new.dtype == torch.float16 else DSA_KEY_F32
    _req(k_new, torch.float16 if kd == DSA_KEY_F16 else torch.float32, "k_new")
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req(q_lat, torch.bfloat16, "q_lat")
    _req(q_rope, torch.bfloat16, "q_rope")
    _req(k_cache, torch.float16, "k_cache")
    _req(kv_cache, torch.bfloat16, "kv_cache")
    _req(sink_pos0, torch.int32, "sink_pos0")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    _req(idx_out, torch.int32, "idx_out")
    d = batch.desc()
    _check(lib().dsa_decode_sink(_ptr(k_new), kd, _ptr(q_idx), _ptr(w), _ptr(q_lat), _ptr(q_rope), _ptr(k_cache),
                                 _ptr(kv_cache), C.byref(d), q_idx.shape[1], q_lat.shape[1], k, sm_scale,
                                 int(hadamard), n_sink, _ptr(sink_pos0), _ptr(out), _ptr(lse), _ptr(idx_out),
                                 _ptr(ws), ws.numel(), _stream(stream)), "dsa_decode_sink")


def dsa_decode_noalloc(k_new, q_idx, w, q_lat, q_rope, k_cache, kv_cache, batch: Batch, k: int,
                       sm_scale: float, hadamard: bool, out, lse, idx_out, stream=None):
    """dsa_decode with the library's static scratch instead of a workspace
    (for callers that cannot allocate device memory)."""
    import torch
    kd = DSA_KEY_F16 if k_new.dtype == torch.float16 else DSA_KEY_F32
    _req(k_new, torch.float16 if kd == DSA_KEY_F16 else torch.float32, "k_new")
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req(q_lat, torch.bfloat16, "q_lat")
    _req(q_rope, torch.bfloat16, "q_rope")
    _req(k_cache, torch.float16, "k_cache")
    _req(kv_cache, torch.bfloat16, "kv_cache")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    _req(idx_out, torch.int32, "idx_out")
    d = batch.desc()
    _check(lib().dsa_decode_noalloc(_ptr(k_new), kd, _ptr(q_idx), _ptr(w), _ptr(q_lat), _ptr(q_rope),
                                    _ptr(k_cache), _ptr(kv_cache), C.byref(d), q_idx.shape[1], q_lat.shape[1], k,
                                    sm_scale, int(hadamard), _ptr(out), _ptr(lse), _ptr(idx_out),
                                    _stream(stream)), "dsa_decode_noalloc")


def kpool_width(top_k: int) -> int:
    """Positions per token of a kpool selection: 4 * floor(top_k / 4) + 3."""
    return (top_k // KPOOL) * KPOOL + KPOOL - 1


def _req_rows(rows):
    import torch
    if not rows.is_cuda or rows.dtype != torch.float16 or not rows.is_contiguous() or rows.dim() != 2 \
            or rows.shape[1] != KPOOL_ROW:
        raise TypeError(f"idx_rows: expected a contiguous CUDA float16 [rows, {KPOOL_ROW}] tensor")


def dsa_kpool_append(k_new, gate_new, ape, batch: Batch, idx_rows, pool_keys, ws, stream=None):
    """Packed rows k|gate|1.0 of the new tokens and the pooled key of every
    pool they complete (GLM-5.3-Flash kpool indexer)."""
    import torch
    _req(k_new, torch.float16, "k_new")
    _req(gate_new, torch.float16, "gate_new")
    _req(ape, torch.float32, "ape")
    _req_rows(idx_rows)
    _req(pool_keys, torch.float16, "k_cache")
    d = batch.desc()
    _check(lib().dsa_kpool_append(_ptr(k_new), _ptr(gate_new), _ptr(ape), C.byref(d), _ptr(idx_rows),
                                  _ptr(pool_keys), pool_keys.shape[0], _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_kpool_append")


def dsa_kpool_select(q_idx, w, idx_rows, pool_keys, batch: Batch, top_k: int, idx, ws, stream=None):
    """Positions [T, kpool_width(top_k)] of the best top_k/4 pools and the tail."""
    import torch
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req_rows(idx_rows)
    _req(pool_keys, torch.float16, "k_cache")
    _req(idx, torch.int32, "idx")
    d = batch.desc()
    _check(lib().dsa_kpool_select(_ptr(q_idx), _ptr(w), _ptr(idx_rows), _ptr(pool_keys), pool_keys.shape[0],
                                  C.byref(d), q_idx.shape[1], top_k, _ptr(idx), _ptr(ws), ws.numel(),
                                  _stream(stream)), "dsa_kpool_select")


def dsa_decode_kpool(k_new, gate_new, ape, q_idx, w, q_lat, idx_rows, pool_keys, kv_latent, batch: Batch, top_k: int,
                     sm_scale: float, out, lse, idx_out, ws, stream=None):
    """The fused GLM-5.3-Flash DSA step: kpool append, selection, MLA-NoPE attention."""
    import torch
    _req(k_new, torch.float16, "k_new")
    _req(gate_new, torch.float16, "gate_new")
    _req(ape, torch.float32, "ape")
    _req(q_idx, torch.float16, "q_idx")
    _req(w, torch.float32, "w")
    _req(q_lat, torch.bfloat16, "q_lat")
    _req_rows(idx_rows)
    _req(pool_keys, torch.float16, "k_cache")
    _req(kv_latent, torch.bfloat16, "kv_latent")
    _req(out, torch.float32, "out")
    _req(lse, torch.float32, "lse")
    _req(idx_out, torch.int32, "idx_out")
    d = batch.desc()
    _check(lib().dsa_decode_kpool(_ptr(k_new), _ptr(gate_new), _ptr(ape), _ptr(q_idx), _ptr(w), _ptr(q_lat),
                                  _ptr(idx_rows), _ptr(pool_keys), pool_keys.shape[0], _ptr(kv_latent), C.byref(d),
                                  q_idx.shape[1], q_lat.shape[1], top_k, sm_scale, _ptr(out), _ptr(lse),
                                  _ptr(idx_out), _ptr(ws), ws.numel(), _stream(stream)), "dsa_decode_kpool")


class dsa_rope_t(C.Structure):
    _fields_ = [("inv_freq", _P), ("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("scale", C.c_float)]


_ROPE_SCALING = {"none": DSA_ROPE_NONE, "linear": DSA_ROPE_LINEAR, "ntk": DSA_ROPE_NTK, "yarn": DSA_ROPE_YARN}


@dataclass
class Rope:
    """A rotation (dsa_rope_t): pair j of a token at position p turns by
    p * inv_freq[j] and is multiplied by scale."""
    inv_freq: object       # float64 CUDA [rot_dim / 2], radians per position
    interleaved: bool      # pairs (2j, 2j+1), else (j, j + rot_dim / 2)
    scale: float = 1.0

    @classmethod
    def make(cls, rot_dim: int, base: float = 10000.0, interleaved: bool = True, scaling: str = "none",
             factor: float = 1.0, trained_ctx: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
             device="cuda"):
        """Frequencies of dsa_rope_frequencies; scaling none, linear, ntk or yarn."""
        import torch
        f, scale = dsa_rope_frequencies(rot_dim, base, scaling, factor, trained_ctx, beta_fast, beta_slow)
        return cls(torch.tensor(f, dtype=torch.float64).to(device), interleaved, scale)

    @property
    def rot_dim(self) -> int:
        return 2 * self.inv_freq.numel()

    def desc(self) -> dsa_rope_t:
        if not _DT:
            _bind()
        f = self.inv_freq
        n = f.numel()
        _shaped(f, "inv_freq", _t_f64, (n,), _cuda(f, "inv_freq"))
        return dsa_rope_t(f.data_ptr(), 2 * n, 1 if self.interleaved else 0, self.scale)


def dsa_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                         trained_ctx: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(list of rot_dim / 2 float64 frequencies, scale) on the host."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling: expected one of {sorted(_ROPE_SCALING)}, got {scaling!r}")
    f = (C.c_double * max(1, rot_dim // 2))()
    scale = C.c_float(0.0)
    _check(lib().dsa_rope_frequencies(rot_dim, base, _ROPE_SCALING[scaling], factor, trained_ctx, beta_fast,
                                      beta_slow, f, C.byref(scale)), "dsa_rope_frequencies")
    return list(f), scale.value


# The calls below take microseconds on the device, so their checks are kept to
# a few attribute reads per tensor, on names bound by the first call.
_DT = {}
_ANY_FLOAT = (DSA_DT_F32, DSA_DT_F16, DSA_DT_BF16)
_OUT_FLOAT = (DSA_DT_F32, DSA_DT_BF16)


def _bind():
    global _DT, _t_u8, _t_i32, _t_i64, _t_f32, _t_f64, _t_bf16, _get_device, _raw_stream, _on_device
    import torch
    _t_u8, _t_i32, _t_i64 = torch.uint8, torch.int32, torch.int64
    _t_f32, _t_f64, _t_bf16 = torch.float32, torch.float64, torch.bfloat16
    _get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _on_device = torch.cuda.device
    _DT = {torch.float32: DSA_DT_F32, torch.float16: DSA_DT_F16, torch.bfloat16: DSA_DT_BF16}


def _cuda(t, name):
    """The CUDA index of t's device."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return dev


def _dt(t, name, allowed=_ANY_FLOAT):
    d = _DT.get(t.dtype)
    if d not in allowed:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return d


def _shaped(t, name, dtype, shape, dev):
    """A contiguous tensor of that dtype and shape on device `dev` (a CUDA index)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}, "
                        f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, name, dtype, shape, dev):
    """A matrix of contiguous rows any stride apart; returns that stride."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or t.stride(1) != 1:
        raise TypeError(f"{name}: expected {dtype} rows {tuple(shape)} on cuda:{dev}, "
                        f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.stride(0)


def _q8_cache(codes, scale, tail: bool, batch: Batch, dev):
    rows = codes.shape[0]
    _shaped(codes, "codes", _t_u8, (rows, Q8_ROW if tail else 512), dev)
    _shaped(scale, "scale", _t_f32, (rows,), dev)
    if rows < batch.cache_rows:
        raise TypeError(f"codes: {rows} rows, the batch names {batch.cache_rows}")


def _batch_desc(batch: Batch, dev) -> dsa_batch_t:
    """Batch.desc with its tensors' device checked as well."""
    cu, pos, off = batch.cu_q, batch.q_pos, batch.kv_off
    B, T = cu.numel() - 1, pos.numel()
    _shaped(cu, "cu_q", _t_i32, (B + 1,), dev)
    _shaped(pos, "q_pos", _t_i32, (T,), dev)
    _shaped(off, "kv_off", _t_i64, (B,), dev)
    return dsa_batch_t(B, T, batch.max_q_per_seq, batch.max_kv, batch.cache_rows, cu.data_ptr(), pos.data_ptr(),
                       off.data_ptr())


def _paging(block_table, block_size: int, batch: Batch, dev):
    """(dsa_paging_t pointer or None) of an optional block table [B, max_blocks]."""
    if block_table is None:
        return None
    blocks = block_table.shape[-1]
    _shaped(block_table, "block_table", _t_i32, (batch.B, blocks), dev)
    return C.byref(dsa_paging_t(block_table.data_ptr(), blocks, block_size))


def _call(name, dev, stream, fn, *args):
    """fn(*args, stream) on device dev; the current stream of dev unless one is given."""
    if _get_device() != dev:
        with _on_device(dev):
            return _call(name, dev, stream, fn, *args)
    code = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if code != DSA_OK:
        raise DsaError(code, name)


def dsa_rope(x, pos, rope: Rope, out, rot_off: int = 0, inverse: bool = False, stream=None):
    """out = x with rope.rot_dim values of each head, from rot_off on, turned at
    the tokens' positions.  x, out: [T, heads, dim] of one dtype (float32,
    float16, bfloat16), any token and head strides, contiguous heads; out may
    be x.  pos: int32 [T].  inverse: the gradient's direction."""
    if not _DT:
        _bind()
    dt, dev, shape = _dt(x, "x"), _cuda(x, "x"), x.shape
    xs, ys = x.stride(), out.stride()
    if len(shape) != 3 or out.shape != shape or out.dtype is not x.dtype or out.get_device() != dev \
            or (shape[2] > 1 and (xs[2] != 1 or ys[2] != 1)):
        raise TypeError(f"x, out: expected CUDA tensors [T, heads, dim] of one shape and dtype with contiguous heads, "
                        f"got {x.dtype} {tuple(shape)} on {x.device} and {out.dtype} {tuple(out.shape)} on {out.device}")
    T, heads, dim = shape
    _shaped(pos, "pos", _t_i32, (T,), dev)
    r = rope.desc()
    if rope.inv_freq.get_device() != dev:
        raise TypeError(f"inv_freq: on {rope.inv_freq.device}, x on {x.device}")
    _call("dsa_rope", dev, stream, lib().dsa_rope, x.data_ptr(), xs[0], xs[1], out.data_ptr(), ys[0], ys[1], dt, T,
          heads, dim, rot_off, pos.data_ptr(), C.byref(r), 1 if inverse else 0)


def _append_args(c_new, r_new, batch: Batch, rope, block_table, block_size, dev):
    """The arguments the two append calls share, up to the cache."""
    T, dt, kind = batch.q_pos.numel(), _dt(c_new, "c_new"), c_new.dtype
    cs = _rows(c_new, "c_new", kind, (T, 512), dev)
    rp, rs, turn = None, 0, None
    if r_new is not None:
        rs = _rows(r_new, "r_new", kind, (T, 64), dev)
        rp = r_new.data_ptr()
    if rope is not None:
        turn = C.byref(rope.desc())
        if rope.inv_freq.get_device() != dev:
            raise TypeError(f"inv_freq: on {rope.inv_freq.device}, c_new on {c_new.device}")
    return (c_new.data_ptr(), cs, rp, rs, dt, C.byref(_batch_desc(batch, dev)),
            _paging(block_table, block_size, batch, dev), turn)


def _workspace_arg(ws, dev):
    if ws.get_device() != dev:
        raise TypeError(f"ws: expected on cuda:{dev}, got {ws.device}")
    return ws.data_ptr(), ws.nbytes


def dsa_kv_append(c_new, r_new, batch: Batch, rope, kv_cache, ws, block_table=None, block_size: int = 0, stream=None):
    """One bf16 latent row per token into kv_cache [rows, 576] ([rows, 512]
    with r_new None).  c_new [T, 512] and r_new [T, 64] may be column slices;
    the tail is turned at the token's position when rope (a Rope) is given."""
    if not _DT:
        _bind()
    dev, rows = _cuda(c_new, "c_new"), kv_cache.shape[0]
    args = _append_args(c_new, r_new, batch, rope, block_table, block_size, dev)
    _shaped(kv_cache, "kv_cache", _t_bf16, (rows, 512 if r_new is None else 576), dev)
    if rows < batch.cache_rows:
        raise TypeError(f"kv_cache: {rows} rows, the batch names {batch.cache_rows}")
    _call("dsa_kv_append", dev, stream, lib().dsa_kv_append, *args, kv_cache.data_ptr(), *_workspace_arg(ws, dev))


def q8_cache(rows: int, tail: bool = True, device="cuda"):
    """(codes, scale) of an 8-bit latent cache of `rows` rows, all zero."""
    import torch
    return (torch.zeros(rows, Q8_ROW if tail else 512, dtype=torch.uint8, device=device),
            torch.zeros(rows, device=device))


def dsa_kv_append_q8(c_new, r_new, batch: Batch, rope, codes, scale, ws, block_table=None, block_size: int = 0,
                     stream=None):
    """dsa_kv_append into an 8-bit cache: codes uint8 [rows, 640] ([rows, 512]
    with r_new None), scale float32 [rows]."""
    if not _DT:
        _bind()
    dev = _cuda(c_new, "c_new")
    args = _append_args(c_new, r_new, batch, rope, block_table, block_size, dev)
    _q8_cache(codes, scale, r_new is not None, batch, dev)
    _call("dsa_kv_append_q8", dev, stream, lib().dsa_kv_append_q8, *args, codes.data_ptr(), scale.data_ptr(),
          *_workspace_arg(ws, dev))


def dsa_kv_read_q8(codes, scale, batch: Batch, out, ws, block_table=None, block_size: int = 0, stream=None):
    """The tokens' rows of an 8-bit cache as out [T, 576] ([T, 512] for codes
    of 512), bfloat16 or float32; out may be a column slice of wider rows."""
    if not _DT:
        _bind()
    dev, T = _cuda(codes, "codes"), batch.q_pos.numel()
    tail = codes.shape[-1] == Q8_ROW
    _q8_cache(codes, scale, tail, batch, dev)
    dt, width = _dt(out, "out", _OUT_FLOAT), 576 if tail else 512
    stride = _rows(out, "out", out.dtype, (T, width), dev)
    _call("dsa_kv_read_q8", dev, stream, lib().dsa_kv_read_q8, codes.data_ptr(), scale.data_ptr(), 1 if tail else 0,
          C.byref(_batch_desc(batch, dev)), _paging(block_table, block_size, batch, dev), out.data_ptr(), dt,
          stride if T > 1 else width, *_workspace_arg(ws, dev))


def dsa_sparse_mla_attn_q8(q_lat, q_rope, codes, scale, batch: Batch, idx, sm_scale: float, out, lse, ws,
                           block_table=None, block_size: int = 0, stream=None):
    """dsa_sparse_mla_attn over an 8-bit cache (q_rope None: codes of 512, no
    tail); out [T, H, 512] float32 or bfloat16, lse [T, H] float32 or None."""
    if not _DT:
        _bind()
    dev, T, H = _cuda(q_lat, "q_lat"), batch.q_pos.numel(), q_lat.shape[1]
    _shaped(q_lat, "q_lat", _t_bf16, (T, H, 512), dev)
    if q_rope is not None:
        _shaped(q_rope, "q_rope", _t_bf16, (T, H, 64), dev)
    _q8_cache(codes, scale, q_rope is not None, batch, dev)
    k = idx.shape[-1]
    _shaped(idx, "idx", _t_i32, (T, k), dev)
    dt = _dt(out, "out", _OUT_FLOAT)
    _shaped(out, "out", out.dtype, (T, H, 512), dev)
    if lse is not None:
        _shaped(lse, "lse", _t_f32, (T, H), dev)
    _call("dsa_sparse_mla_attn_q8", dev, stream, lib().dsa_sparse_mla_attn_q8, q_lat.data_ptr(),
          q_rope.data_ptr() if q_rope is not None else None, codes.data_ptr(), scale.data_ptr(),
          C.byref(_batch_desc(batch, dev)), _paging(block_table, block_size, batch, dev), idx.data_ptr(), k, H, sm_scale,
          out.data_ptr(), dt, lse.data_ptr() if lse is not None else None, *_workspace_arg(ws, dev))


def _norm_args(x, residual, sum, weight, dev):
    """Checked arguments of the norms up to the weight, x's DSA_DT_* and shape."""
    kind, shape = x.dtype, x.shape
    dt = _dt(x, "x")
    if len(shape) != 2:
        raise TypeError(f"x: expected rows [T, dim], got shape {tuple(shape)}")
    xs, rp, rs, sp, ss, wp, wt = _rows(x, "x", kind, shape, dev), None, 0, None, 0, None, dt
    if residual is not None:
        rp, rs = residual.data_ptr(), _rows(residual, "residual", kind, shape, dev)
    if sum is not None:
        sp, ss = sum.data_ptr(), _rows(sum, "sum", kind, shape, dev)
    if weight is not None:
        if weight.dtype is not kind:
            wt = DSA_DT_F32
        _shaped(weight, "weight", kind if wt == dt else _t_f32, shape[1:], dev)
        wp = weight.data_ptr()
    return (x.data_ptr(), xs, rp, rs, sp, ss, wp, wt), dt, shape


def dsa_rms_norm(x, residual, sum, weight, eps: float, out, stream=None):
    """out = h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual
    (rounded to x's dtype; stored in sum).  x, residual, sum, out: [T, dim] of one
    dtype (float32, float16, bfloat16), any row strides; residual, sum and weight may
    be None; weight [dim] of x's dtype or float32.  sum and out may be x or residual."""
    if not _DT:
        _bind()
    dev = _cuda(x, "x")
    args, dt, shape = _norm_args(x, residual, sum, weight, dev)
    stride = _rows(out, "out", x.dtype, shape, dev)
    _call("dsa_rms_norm", dev, stream, lib().dsa_rms_norm, *args, eps, out.data_ptr(), stride, dt, shape[0], shape[1])


def dsa_rms_norm_q8(x, residual, sum, weight, eps: float, codes, scale, stream=None):
    """dsa_rms_norm with e4m3 codes (uint8 [T, dim]) and one float32 scale per
    group as output; scale [T, dim / group] gives the group: 32, 64, 128 or dim."""
    if not _DT:
        _bind()
    dev = _cuda(x, "x")
    args, dt, shape = _norm_args(x, residual, sum, weight, dev)
    T, dim = shape
    _shaped(codes, "codes", _t_u8, shape, dev)
    groups = scale.shape[-1]
    _shaped(scale, "scale", _t_f32, (T, groups), dev)
    if groups < 1 or dim % groups:
        raise TypeError(f"scale: {groups} groups do not divide rows of {dim}")
    _call("dsa_rms_norm_q8", dev, stream, lib().dsa_rms_norm_q8, *args, eps, codes.data_ptr(), scale.data_ptr(),
          dim // groups, dt, T, dim)


def _mla_args(q_lat, q_rope, kv_cache, batch: Batch, out, lse, ws, block_table, block_size, dev):
    """Checked arguments of the calls over all visible rows: up to H, and from out on."""
    T, H = batch.q_pos.numel(), q_lat.shape[1]
    _shaped(q_lat, "q_lat", _t_bf16, (T, H, 512), dev)
    if q_rope is not None:
        _shaped(q_rope, "q_rope", _t_bf16, (T, H, 64), dev)
    rows = kv_cache.shape[0]
    _shaped(kv_cache, "kv_cache", _t_bf16, (rows, 512 if q_rope is None else 576), dev)
    if rows < batch.cache_rows:
        raise TypeError(f"kv_cache: {rows} rows, the batch names {batch.cache_rows}")
    dt = _dt(out, "out", _OUT_FLOAT)
    _shaped(out, "out", out.dtype, (T, H, 512), dev)
    if lse is not None:
        _shaped(lse, "lse", _t_f32, (T, H), dev)
    return ((q_lat.data_ptr(), q_rope.data_ptr() if q_rope is not None else None, kv_cache.data_ptr(),
             C.byref(_batch_desc(batch, dev)), _paging(block_table, block_size, batch, dev), H),
            (out.data_ptr(), dt, lse.data_ptr() if lse is not None else None, *_workspace_arg(ws, dev)))


def dsa_mla_attn(q_lat, q_rope, kv_cache, batch: Batch, sm_scale: float, out, lse, ws, block_table=None,
                 block_size: int = 0, stream=None):
    """Attention of q_lat [T, H, 512] (and tails q_rope [T, H, 64], or None) over
    all the cached rows each token sees; kv_cache [rows, 576] ([rows, 512] without
    tails), out [T, H, 512] float32 or bfloat16, lse [T, H] float32 or None."""
    if not _DT:
        _bind()
    dev = _cuda(q_lat, "q_lat")
    a, z = _mla_args(q_lat, q_rope, kv_cache, batch, out, lse, ws, block_table, block_size, dev)
    _call("dsa_mla_attn", dev, stream, lib().dsa_mla_attn, *a, sm_scale, *z)


def dsa_mla_attn_window(q_lat, q_rope, kv_cache, batch: Batch, window: int, n_sink: int, sink_pos0, sm_scale: float, out,
                        lse, ws, block_table=None, block_size: int = 0, stream=None):
    """dsa_mla_attn over the last `window` positions of each token and the first
    n_sink of its sequence (from sink_pos0[b], int32 [B], or 0 when None)."""
    if not _DT:
        _bind()
    dev = _cuda(q_lat, "q_lat")
    a, z = _mla_args(q_lat, q_rope, kv_cache, batch, out, lse, ws, block_table, block_size, dev)
    if sink_pos0 is not None:
        _shaped(sink_pos0, "sink_pos0", _t_i32, (batch.B,), dev)
    # beyond 32 bits: as many as there are, or refused
    window, n_sink = max(-1, min(window, 2 ** 31 - 1)), max(-1, min(n_sink, 2 ** 31 - 1))
    _call("dsa_mla_attn_window", dev, stream, lib().dsa_mla_attn_window, *a, window, n_sink,
          sink_pos0.data_ptr() if sink_pos0 is not None else None, sm_scale, *z)


def dsa_set_trace_events(events):
    """events: list of torch.cuda.Event (enable_timing=True) or None to disable."""
    global _TRACE_KEEP
    if not events:
        _TRACE_KEEP = None
        _check(lib().dsa_set_trace_events(None, 0), "dsa_set_trace_events")
        return
    for e in events:
        e.record()  # makes torch create the underlying event
    arr = (C.c_void_p * len(events))(*[e.cuda_event for e in events])
    _TRACE_KEEP = arr
    _check(lib().dsa_set_trace_events(C.cast(arr, C.c_void_p), len(events)), "dsa_set_trace_events")


_TRACE_KEEP = None


def dsa_set_timeline(buf):
    """buf: CUDA int64/uint64 tensor of 10 slots, or None to disable."""
    _check(lib().dsa_set_timeline(_ptr(buf)), "dsa_set_timeline")


def dsa_set_test_faults(wait_limit_ns: int = 0, skip_copies: bool = False):
    """Failure-path test hook: bound every device wait by wait_limit_ns (0:
    the default second) and, with skip_copies, make the score and attention
    producers issue no copies so that the waits run out (DSA_DEV_TIMEOUT)."""
    _check(lib().dsa_set_test_faults(int(wait_limit_ns), int(bool(skip_copies))), "dsa_set_test_faults")


def dsa_status_string(code: int) -> str:
    return lib().dsa_status_string(code).decode()


def dsa_version() -> int:
    return lib().dsa_version()
