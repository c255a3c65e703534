"""ctypes binding of libq3tts (include/q3tts.h, include/q3tts_branch.h,
include/q3tts_kv8.h): argument marshalling only.

Every step of the decode runs in the CUDA library; this module turns torch
tensors into device pointers and status codes into exceptions.  It refuses to
work without the built library (no CPU path exists).
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import struct
from typing import Dict, Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libq3tts.so")

OK = 0
ERR_ARG, ERR_CAPACITY, ERR_CUDA, ERR_TIMEOUT, ERR_UNSUPPORTED, ERR_STATE = -1, -2, -3, -4, -5, -6
ERR_SCRATCH = -7
STATIC_SCRATCH_BYTES = 786432
F32, BF16, FP8 = 0, 1, 2
MAX_STREAMS = 256
N_CODEBOOKS = 16

LAYER_KEYS = ("w_qkv", "w_o", "w_gateup", "w_down",
              "g_attn_norm", "g_ffn_norm", "g_q_norm", "g_k_norm")
LAYER_SCALES = ("s_qkv", "s_o", "s_gateup", "s_down")  # FP8 matrices' per-row scales


class Q3TTSError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


class Config(C.Structure):
    _fields_ = [(n, C.c_int) for n in (
        "talker_layers", "talker_hidden", "talker_ffn", "cp_layers", "cp_hidden", "cp_ffn",
        "n_q_heads", "n_kv_heads", "head_dim", "codec_vocab", "cp_vocab", "n_codebooks",
        "max_streams", "kv_cap_steps", "page_size", "kv_pages", "prefill_chunk",
        "weight_dtype", "kv_dtype", "qk_norm")] + [("rms_eps", C.c_float), ("rope_theta", C.c_float)]


class LayerWeights(C.Structure):
    _fields_ = [(k, C.c_void_p) for k in LAYER_KEYS + LAYER_SCALES]


class KVCache(C.Structure):
    _fields_ = [("pool", C.c_void_p)] + [(n, C.c_int) for n in (
        "layers", "n_pages", "n_kv_heads", "page_size", "head_dim", "kv_dtype")]


class KV8Cache(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("powers", C.c_void_p)] + [(n, C.c_int) for n in (
        "layers", "n_pages", "n_kv_heads", "page_size", "head_dim", "block")]


class KV8Rows(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("page_table", "lengths", "row_start", "status")] + [(n, C.c_int) for n in (
        "layer", "pages_per_seq", "n_seqs", "row_dtype", "n_rows", "max_rows")]


class Rows(C.Structure):
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("row_bytes", C.c_size_t),
                ("src_stride", C.c_size_t), ("dst_stride", C.c_size_t)]


class Weights(C.Structure):
    _fields_ = [("talker_layers", C.POINTER(LayerWeights)), ("talker_g_final", C.c_void_p),
                ("talker_w_head", C.c_void_p), ("talker_e_codec", C.c_void_p),
                ("cp_layers", C.POINTER(LayerWeights)), ("cp_g_final", C.c_void_p),
                ("cp_heads", C.c_void_p), ("cp_embeds", C.c_void_p), ("cp_w_proj", C.c_void_p),
                ("s_head", C.c_void_p), ("s_cp_heads", C.c_void_p), ("s_cp_proj", C.c_void_p)]


class Sampling(C.Structure):
    _fields_ = [("do_sample", C.c_int), ("top_k", C.c_int), ("top_p", C.c_float),
                ("temperature", C.c_float), ("repetition_penalty", C.c_float),
                ("sub_do_sample", C.c_int), ("sub_top_k", C.c_int), ("sub_top_p", C.c_float),
                ("sub_temperature", C.c_float), ("eos_token", C.c_int), ("special_from", C.c_int)]


EXPORTS = ("q3tts_workspace_size", "q3tts_create", "q3tts_prefill", "q3tts_step_frame",
           "q3tts_read_pending", "q3tts_reset", "q3tts_stream_length", "q3tts_sync_status",
           "q3tts_kernel_launches", "q3tts_destroy", "q3tts_strerror",
           "q3tts_step_frame_static", "q3tts_debug_fail_barrier", "q3tts_stream_finished",
           "q3tts_step_frames", "q3tts_frames_ready")
# include/q3tts_branch.h
BRANCH_EXPORTS = ("q3tts_fork", "q3tts_tree_step", "q3tts_tree_accept", "q3tts_beam_frame",
                  "q3tts_tree_attention", "q3tts_copy_pages", "q3tts_compact_rows",
                  "q3tts_beam_workspace_size", "q3tts_beam_select", "q3tts_reorder_rows",
                  "q3tts_debug_lose_tile")
# include/q3tts_kv8.h
KV8_EXPORTS = ("q3tts_kv8_write", "q3tts_kv8_read", "q3tts_kv8_attention")
MAX_CHUNK = 64
MAX_TREE_NODES = 64
MAX_BEAMS = 32

_lib = None


def load(path: str = LIB_PATH):
    """Loads libq3tts.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libq3tts.so is not built ({path}); run __graft_entry__.build()")
    L = C.CDLL(path)
    vp = C.c_void_p
    L.q3tts_workspace_size.restype = C.c_size_t
    L.q3tts_workspace_size.argtypes = [C.POINTER(Config)]
    L.q3tts_create.argtypes = [C.POINTER(Config), C.POINTER(Weights), vp, C.c_size_t, vp,
                               C.POINTER(vp)]
    L.q3tts_prefill.argtypes = [vp, C.c_int, vp, C.c_int]
    L.q3tts_step_frame.argtypes = [vp, C.POINTER(Sampling), C.POINTER(C.c_int32), C.c_int, vp, vp,
                                   vp, vp]
    L.q3tts_step_frame_static.argtypes = [vp, C.POINTER(Sampling), C.c_int, vp, vp, vp, vp]
    L.q3tts_read_pending.argtypes = [vp, C.c_int, vp, vp]
    L.q3tts_reset.argtypes = [vp, C.c_int]
    L.q3tts_stream_length.argtypes = [vp, C.c_int]
    L.q3tts_sync_status.argtypes = [vp]
    L.q3tts_destroy.argtypes = [vp]
    L.q3tts_kernel_launches.restype = C.c_uint64
    L.q3tts_kernel_launches.argtypes = [vp]
    L.q3tts_debug_fail_barrier.argtypes = [vp, C.c_int, C.c_int]
    L.q3tts_stream_finished.argtypes = [vp, C.c_int, C.POINTER(C.c_int)]
    L.q3tts_step_frames.argtypes = [vp, C.POINTER(Sampling), C.POINTER(C.c_int32), C.c_int, C.c_int, vp, vp,
                                    vp, vp]
    L.q3tts_frames_ready.argtypes = [vp]
    i32p = C.POINTER(C.c_int32)
    L.q3tts_fork.argtypes = [vp, C.c_int, i32p, C.c_int]
    L.q3tts_tree_step.argtypes = [vp, C.c_int, vp, i32p, C.c_int, vp, vp]
    L.q3tts_tree_accept.argtypes = [vp, C.c_int, i32p, C.c_int]
    L.q3tts_beam_frame.argtypes = [vp, C.POINTER(Sampling), i32p, C.c_int, C.c_int, vp, vp, vp, i32p]
    # structs by address: a ctypes instance (byref) or packed bytes
    L.q3tts_tree_attention.argtypes = [vp, C.c_int, vp, C.c_int, C.c_int, vp, vp, vp, C.c_int, C.c_int, C.c_int,
                                       vp, C.c_int, vp, C.c_int, vp, vp]
    L.q3tts_debug_lose_tile.argtypes = [C.c_int, C.c_int]
    L.q3tts_copy_pages.argtypes = [vp, vp, vp, C.c_int, vp]
    L.q3tts_compact_rows.argtypes = [vp, vp, C.c_int, C.c_int, vp, vp, C.c_int, vp, vp, vp]
    L.q3tts_beam_select.argtypes = [vp, C.c_size_t, vp, C.c_int, C.c_int, C.c_int, vp, vp, vp, C.c_int, C.c_int,
                                    C.c_float, C.c_int, vp, vp, vp, vp, C.c_size_t, vp]
    L.q3tts_beam_workspace_size.argtypes = [C.c_int] * 4
    L.q3tts_beam_workspace_size.restype = C.c_size_t
    L.q3tts_reorder_rows.argtypes = [vp, C.c_int, vp, vp, C.c_int, C.c_int, C.c_int, vp, vp]
    rows = [vp, C.c_int, vp, C.c_int]  # two row buffers with their pitches
    L.q3tts_kv8_write.argtypes = [vp, vp] + rows + [vp]
    L.q3tts_kv8_read.argtypes = [vp, vp, vp] + rows + [vp]
    L.q3tts_kv8_attention.argtypes = [vp, vp, vp] + rows + [C.c_int, vp]
    L.q3tts_strerror.restype = C.c_char_p
    L.q3tts_strerror.argtypes = [C.c_int]
    _lib = L
    return L


def strerror(code: int) -> str:
    try:
        return load().q3tts_strerror(code).decode()
    except RuntimeError:
        return f"error {code}"


def _check(rc: int, what: str):
    if rc != OK:
        raise Q3TTSError(rc, what)


def make_config(shape, max_streams: int, kv_cap: int, page_size: int = 16, kv_pages: int = 0,
                prefill_chunk: int = 0) -> Config:
    s = shape
    return Config(s.talker_layers, s.talker_hidden, s.talker_ffn, s.cp_layers, s.cp_hidden,
                  s.cp_ffn, s.n_q_heads, s.n_kv_heads, s.head_dim, s.codec_vocab, s.cp_vocab,
                  s.n_codebooks, max_streams, kv_cap, page_size, kv_pages, prefill_chunk,
                  s.weight_dtype, s.kv_dtype, s.qk_norm, float(s.rms_eps), float(s.rope_theta))


def sampling_struct(sp) -> Sampling:
    return Sampling(int(sp.do_sample), int(sp.top_k), float(sp.top_p), float(sp.temperature),
                    float(sp.repetition_penalty), int(sp.sub_do_sample), int(sp.sub_top_k),
                    float(sp.sub_top_p), float(sp.sub_temperature),
                    int(getattr(sp, "eos_token", -1)), int(getattr(sp, "special_from", 0)))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t, name: str, dtype, numel: int, what: str):
    """Raises Q3TTSError(ERR_ARG) unless t is a contiguous CUDA tensor of the
    given dtype with at least numel elements (checked before the C call, so a
    wrong buffer is an error instead of an out-of-bounds device write)."""
    import torch
    ok = (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and t.dtype == dtype
          and t.numel() >= numel)
    if not ok:
        raise Q3TTSError(ERR_ARG, f"{what}: {name} must be a contiguous CUDA {dtype} tensor "
                                  f"of at least {numel} elements")


# ---- branching-decode operators over caller-owned buffers (include/q3tts_branch.h).
# They run on the current torch stream of their tensors' device, whichever device
# is current.  A single call of the smallest sizes costs the GPU 3 to 10 us, so
# the checks here read few tensor attributes and structs travel as packed bytes.

_CACHE = struct.Struct("P6i")  # q3tts_kv_cache
_ROWS = "PPNNN"  # q3tts_rows


def _bad(what: str, name: str, want: str):
    raise Q3TTSError(ERR_ARG, f"{what}: {name} must be {want}")


def _cuda(t, name: str, dtype, dev: int, numel: int, what: str) -> int:
    """data_ptr of t; raises unless it is a contiguous tensor of dtype on CUDA
    device dev with numel elements."""
    if t.dtype != dtype or t.get_device() != dev or t.numel() != numel or not t.is_contiguous():
        _bad(what, name, f"a contiguous {dtype} tensor of {numel} elements on cuda:{dev}")
    return t.data_ptr()


@functools.lru_cache(maxsize=None)
def _cuda_state():
    """torch's functions for the current device and a device's current stream (an import
    statement in each call takes longer)."""
    from torch import _C
    return _C._cuda_getDevice, _C._cuda_getCurrentRawStream


def _call(dev: int, fn, what: str, *args):
    """fn(*args, the current stream of device dev) with that device current."""
    device, stream = _cuda_state()
    if dev < 0:
        _bad(what, "every tensor", "on a CUDA device")
    if dev == device():
        rc = fn(*args, stream(dev))
    else:
        import torch
        with torch.cuda.device(dev):
            rc = fn(*args, stream(dev))
    if rc != OK:
        raise Q3TTSError(rc, what)


def _cache(pool, what: str):
    """(device, packed q3tts_kv_cache, head dim)."""
    import torch
    dev, dt = pool.get_device(), pool.dtype
    kind = BF16 if dt == torch.bfloat16 else F32
    if dev < 0 or not pool.is_contiguous() or pool.dim() != 6 or (kind == F32 and dt != torch.float32):
        _bad(what, "pool", "a contiguous CUDA fp32 or bf16 tensor [layers, pages, 2, kv heads, page size, head dim]")
    layers, pages, two, heads, page, hd = pool.shape
    if two != 2:
        _bad(what, "pool", "[layers, pages, 2, kv heads, page size, head dim]")
    return dev, _CACHE.pack(pool.data_ptr(), layers, pages, heads, page, hd, kind), hd


def _pitch(t, rows: int, heads: int, hd: int, name: str, what: str) -> int:
    """Row pitch of a [rows, heads, head dim] view whose rows are contiguous."""
    if t.is_contiguous():
        return heads * hd
    n, h, d = t.stride()
    if (heads > 1 and h != hd) or d != 1 or (rows > 1 and not heads * hd <= n < 1 << 31):
        _bad(what, name, "[rows, heads, head dim] with contiguous rows")
    return n if rows > 1 else heads * hd


def tree_attention(pool, layer: int, page_table, lengths, node_start, masks, q, max_nodes: Optional[int] = None,
                   out=None, status=None):
    """q3tts_tree_attention.  pool: CUDA fp32/bf16 [layers, pages, 2, kv heads, page
    size, head dim]; page_table int32 [seqs, pages per seq]; lengths int32 [seqs];
    node_start int32 [seqs + 1]; masks int64 (or uint64) [rows], bit j of a row's
    word: the row's node sees node j of its sequence; q fp32 [rows, q heads, head
    dim] (rows contiguous, any row pitch); max_nodes: the most nodes of a sequence
    (default: as many as there are rows, up to MAX_TREE_NODES).  Returns out
    (fp32, as q; made if None, with zeroes in rows outside every sequence)."""
    import torch
    what = "q3tts_tree_attention"
    dev, kv, hd = _cache(pool, what)
    if q.dim() != 3 or q.dtype != torch.float32 or q.get_device() != dev or page_table.dim() != 2:
        _bad(what, "q and page_table", f"fp32 [rows, q heads, {hd}] and [seqs, pages per seq] on cuda:{dev}")
    rows, heads, width = q.shape
    seqs, pps = page_table.shape
    if width != hd:
        _bad(what, "q", f"[rows, q heads, {hd}]")
    i32 = torch.int32
    if out is None:
        out = torch.zeros(q.shape, dtype=torch.float32, device=q.device)
    elif out.shape != q.shape or out.dtype != torch.float32 or out.get_device() != dev:
        _bad(what, "out", f"an fp32 tensor of q's shape on cuda:{dev}")
    if max_nodes is None:
        max_nodes = max(1, min(rows, MAX_TREE_NODES))
    _call(dev, load().q3tts_tree_attention, what, kv, layer,
          _cuda(page_table, "page_table", i32, dev, seqs * pps, what), pps, seqs,
          _cuda(lengths, "lengths", i32, dev, seqs, what), _cuda(node_start, "node_start", i32, dev, seqs + 1, what),
          _cuda(masks, "masks", torch.uint64 if masks.dtype == torch.uint64 else torch.int64, dev, rows, what),
          rows, max_nodes, heads, q.data_ptr(), _pitch(q, rows, heads, hd, "q", what),
          out.data_ptr(), _pitch(out, rows, heads, hd, "out", what),
          None if status is None else _cuda(status, "status", i32, dev, 1, what))
    return out


def debug_lose_tile(tile: int, wait_us: int) -> None:
    """q3tts_debug_lose_tile: the calling thread's next tree_attention gives up."""
    rc = load().q3tts_debug_lose_tile(int(tile), int(wait_us))
    if rc != OK:
        raise Q3TTSError(rc, "q3tts_debug_lose_tile")


def _host_ids(v, name: str, what: str):
    """A CPU int32 tensor of ids (v: one, or a sequence of ints)."""
    import torch
    t = v if isinstance(v, torch.Tensor) else torch.tensor(list(v), dtype=torch.int32)
    if t.get_device() >= 0 or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        _bad(what, name, "page ids on the host (a sequence, or a contiguous CPU int32 tensor)")
    return t


def copy_pages(pool, src, dst):
    """q3tts_copy_pages: page src[i] to page dst[i] in every layer of pool (as for
    tree_attention).  src, dst: sequences of ints or CPU int32 tensors.  Returns pool."""
    what = "q3tts_copy_pages"
    dev, kv, _ = _cache(pool, what)
    src, dst = _host_ids(src, "src", what), _host_ids(dst, "dst", what)
    n = src.numel()
    if n != dst.numel():
        _bad(what, "dst", "as long as src")
    _call(dev, load().q3tts_copy_pages, what, kv, src.data_ptr(), dst.data_ptr(), n)
    return pool


def compact_rows(pool, page_table, lengths, path, path_len, status=None):
    """q3tts_compact_rows: positions lengths[s] + path[s, i] to lengths[s] + i, i <
    path_len[s], in place.  page_table int32 [seqs, pages per seq], lengths and
    path_len int32 [seqs], path int32 [seqs, most].  Returns pool."""
    import torch
    what = "q3tts_compact_rows"
    dev, kv, _ = _cache(pool, what)
    if page_table.dim() != 2 or path.dim() != 2:
        _bad(what, "page_table and path", "[seqs, ..]")
    seqs, pps = page_table.shape
    most = path.shape[1]
    i32 = torch.int32
    _call(dev, load().q3tts_compact_rows, what, kv, _cuda(page_table, "page_table", i32, dev, seqs * pps, what), pps,
          seqs, _cuda(lengths, "lengths", i32, dev, seqs, what), _cuda(path, "path", i32, dev, seqs * most, what), most,
          _cuda(path_len, "path_len", i32, dev, seqs, what),
          None if status is None else _cuda(status, "status", i32, dev, 1, what))
    return pool


def beam_workspace_size(groups: int, beams: int, vocab: int, k: int, device: Optional[int] = None) -> int:
    """Bytes of workspace beam_select uses for this shape on the CUDA device of that
    index (default: the current one)."""
    from torch import _C
    if device is None or device == _C._cuda_getDevice():
        return int(load().q3tts_beam_workspace_size(groups, beams, vocab, k))
    import torch
    with torch.cuda.device(device):
        return int(load().q3tts_beam_workspace_size(groups, beams, vocab, k))


_workspace_bytes = functools.lru_cache(maxsize=64)(beam_workspace_size)


def beam_select(logits, scores, k: Optional[int] = None, row_ids=None, finished=None, history=None,
                eos_token: int = -1, special_from: int = 0, repetition_penalty: float = 1.0, out=None,
                workspace=None):
    """q3tts_beam_select.  scores fp32 [groups, beams]; logits fp32 [groups, beams,
    vocab] with contiguous rows, or [rows, vocab] with row_ids int32 [groups,
    beams]; finished uint8 and history uint8 of logits' rows; k: candidates kept
    (default: beams).  Returns (tokens int32, parents int32, scores fp32), [groups,
    k] each; out: three tensors to write them to; workspace: a contiguous CUDA uint8
    tensor of beam_workspace_size bytes (made if None and any are needed)."""
    import torch
    what = "q3tts_beam_select"
    dev = logits.get_device()
    if scores.dim() != 2:
        _bad(what, "scores", "[groups, beams]")
    groups, beams = scores.shape
    n = groups * beams
    if dev < 0 or logits.dtype != torch.float32 or logits.dim() != (3 if row_ids is None else 2):
        _bad(what, "logits", "a CUDA fp32 tensor [groups, beams, vocab], or [rows, vocab] with row_ids")
    vocab = logits.shape[-1]
    rows = n if row_ids is None else logits.shape[0]
    ld = vocab
    if row_ids is None and (logits.shape[0] != groups or logits.shape[1] != beams):
        _bad(what, "logits", f"[{groups}, {beams}, vocab]")
    if not logits.is_contiguous():
        st = logits.stride()
        ld = st[-2] if logits.shape[-2] > 1 else (st[0] if logits.shape[0] > 1 else vocab)
        if st[-1] != 1 or (row_ids is None and groups > 1 and st[0] != beams * ld):
            _bad(what, "logits", "equally spaced rows of contiguous logits")
    i32 = torch.int32
    k = beams if k is None else int(k)
    if out is None:
        # (one block cut into views would cost the host more than three allocations)
        best = torch.empty_like(scores) if k == beams else scores.new_empty((groups, max(k, 0)))
        tokens = torch.empty_like(best, dtype=i32)
        parents = torch.empty_like(tokens)
        p_out = tokens.data_ptr(), parents.data_ptr(), best.data_ptr()
    else:
        tokens, parents, best = out
        p_out = (_cuda(tokens, "out[0]", i32, dev, groups * k, what), _cuda(parents, "out[1]", i32, dev, groups * k, what),
                 _cuda(best, "out[2]", torch.float32, dev, groups * k, what))
    n_ws, p_ws = _workspace_bytes(groups, beams, vocab, k, dev), None
    if workspace is None and n_ws:
        workspace = torch.empty(n_ws, dtype=torch.uint8, device=logits.device)
    if workspace is not None:
        n_ws = workspace.numel()
        p_ws = _cuda(workspace, "workspace", torch.uint8, dev, n_ws, what)
    _call(dev, load().q3tts_beam_select, what, logits.data_ptr(), ld,
          None if row_ids is None else _cuda(row_ids, "row_ids", i32, dev, n, what), groups, beams, vocab,
          _cuda(scores, "scores", torch.float32, dev, n, what),
          None if finished is None else _cuda(finished, "finished", torch.uint8, dev, rows, what),
          None if history is None else _cuda(history, "history", torch.uint8, dev, rows * vocab, what),
          eos_token, special_from, repetition_penalty, k, *p_out, p_ws, n_ws)
    return tokens, parents, best


def reorder_rows(src, dst, parents, status=None):
    """q3tts_reorder_rows: dst[i][g, j] = src[i][g, parents[g, j]] for lists of
    contiguous CUDA tensors [groups, beams, ..] of any type; dst[i] may be src[i],
    and shares no memory with the other tensors otherwise.  parents int32 [groups, beams out].  Returns dst."""
    import torch
    what = "q3tts_reorder_rows"
    if parents.dim() != 2 or len(src) != len(dst):
        _bad(what, "parents", "[groups, beams], with as many dst as src")
    groups, k = parents.shape
    dev = parents.get_device()
    p = _cuda(parents, "parents", torch.int32, dev, groups * k, what)
    sets = []
    beams = src[0].shape[1] if src and src[0].dim() > 1 else 0
    for a, b in zip(src, dst):
        sa = a.shape
        if len(sa) < 2 or sa[0] != groups or sa[1] != beams or b.shape != (groups, k, *sa[2:]):
            _bad(what, "src and dst", f"[{groups}, {beams}, ..] and [{groups}, {k}, ..]")
        if (a.dtype != b.dtype or a.get_device() != dev or b.get_device() != dev or not a.is_contiguous()
                or not b.is_contiguous()):
            _bad(what, "src and dst", f"contiguous tensors of one type on cuda:{dev}")
        n = a.numel() // (groups * beams or 1) * a.element_size()
        sets += a.data_ptr(), b.data_ptr(), n, n, n
    if sets:
        _call(dev, load().q3tts_reorder_rows, what, struct.pack(_ROWS * len(src), *sets), len(src), None, p, groups,
              beams, k, None if status is None else _cuda(status, "status", torch.int32, dev, 1, what))
    return dst


# ---- the paged cache in 8 bits (include/q3tts_kv8.h).  The smallest calls cost the GPU 3 us and the
# host several times that: types are looked up once, attributes read once, and what is wrong is
# told apart only when something is.

_CACHE8 = struct.Struct("2P6i")  # q3tts_kv8_cache
_ROWS8 = struct.Struct("4P6i")  # q3tts_kv8_rows


@functools.lru_cache(maxsize=None)
def _kv8_types():
    """(codes, powers as two types, row types with their codes, int32, masks' types)."""
    import torch
    return (torch.float8_e4m3fn, (torch.float8_e8m0fnu, torch.uint8), {torch.float32: F32, torch.bfloat16: BF16},
            torch.int32, (torch.int64, torch.uint64))


def _kv8(pool, scales, layer, page_table, lengths, start, what: str):
    """(device, kv heads, head dim, packed q3tts_kv8_cache, the first of a q3tts_kv8_rows up to its status, the next three)."""
    codes, powers, _, i32, _ = _kv8_types()
    dev, shape, blocks, table = pool.get_device(), pool.shape, scales.shape, page_table.shape
    if dev < 0 or pool.dtype != codes or len(shape) != 6 or shape[2] != 2 or not pool.is_contiguous():
        _bad(what, "pool", "a contiguous CUDA float8_e4m3fn tensor [layers, pages, 2, kv heads, page size, head dim]")
    layers, pages, _, heads, page, hd = shape
    per_page = blocks[-1] if len(blocks) == 5 else 0
    if (per_page < 1 or page % per_page or blocks != (layers, pages, 2, heads, per_page) or scales.dtype not in powers
            or scales.get_device() != dev or not scales.is_contiguous()):
        _bad(what, "scales", f"contiguous float8_e8m0fnu or uint8 [{layers}, {pages}, 2, {heads}, {page} / block] on cuda:{dev}")
    if len(table) != 2 or page_table.dtype != i32 or page_table.get_device() != dev or not page_table.is_contiguous():
        _bad(what, "page_table", f"contiguous int32 [seqs, pages per seq] on cuda:{dev}")
    n, pps = table
    return (dev, heads, hd, _CACHE8.pack(pool.data_ptr(), scales.data_ptr(), layers, pages, heads, page, hd, page // per_page),
            (page_table.data_ptr(), _cuda(lengths, "lengths", i32, dev, n, what), _cuda(start, "start", i32, dev, n + 1, what)),
            (layer, pps, n))


def _rows8(at, status, shape, dev: int, kind: int, n: int, most: int, what: str) -> bytes:
    """A packed q3tts_kv8_rows."""
    try:
        return _ROWS8.pack(*at, 0 if status is None else _cuda(status, "status", _kv8_types()[3], dev, 1, what), *shape, kind, n, most)
    except struct.error:
        _bad(what, "layer and max_rows", "32-bit whole numbers")


def _row_pair(a, b, names, heads, hd: int, dev: int, what: str):
    """(rows, heads, type code, [address and pitch of both]) of two tensors [rows,
    heads, head dim] of one type; heads None: as a has them."""
    kinds, dt, shape = _kv8_types()[2], a.dtype, a.shape
    if len(shape) != 3 or dt not in kinds or a.get_device() != dev or shape[2] != hd or shape[1] != (heads or shape[1]):
        _bad(what, names[0], f"an fp32 or bf16 tensor [rows, {heads or 'heads'}, {hd}] on cuda:{dev}")
    if b.shape != shape or b.dtype != dt or b.get_device() != dev:
        _bad(what, names[1], f"of {names[0]}'s shape and type on cuda:{dev}")
    n, h, _ = shape
    return n, h, kinds[dt], (a.data_ptr(), _pitch(a, n, h, hd, names[0], what), b.data_ptr(),
                             _pitch(b, n, h, hd, names[1], what))


def kv8_write(pool, scales, layer: int, page_table, lengths, start, k, v, max_rows: Optional[int] = None, status=None):
    """q3tts_kv8_write.  pool: CUDA float8_e4m3fn [layers, pages, 2, kv heads, page
    size, head dim]; scales: float8_e8m0fnu or uint8 [layers, pages, 2, kv heads,
    page size / block]; page_table int32 [seqs, pages per seq]; lengths int32
    [seqs]: positions held; start int32 [seqs + 1]: rows start[s] .. start[s + 1] - 1
    of k and v (fp32 or bf16 [rows, kv heads, head dim], rows contiguous, any row
    pitch) go to the positions after them; max_rows: the most rows of a sequence,
    which sizes the launch (default: as many as there are rows in all, right for any
    call and slow for many sequences).  Returns (pool, scales)."""
    what = "q3tts_kv8_write"
    dev, heads, hd, cache, at, shape = _kv8(pool, scales, layer, page_table, lengths, start, what)
    n, _, kind, pair = _row_pair(k, v, ("k", "v"), heads, hd, dev, what)
    rows = _rows8(at, status, shape, dev, kind, n, (n or 1) if max_rows is None else max_rows, what)
    _call(dev, (_lib or load()).q3tts_kv8_write, what, cache, rows, *pair)
    return pool, scales


def kv8_read(pool, scales, layer: int, page_table, lengths, start, path=None, max_rows: Optional[int] = None, out=None,
             status=None):
    """q3tts_kv8_read: keys and values of positions lengths[s] + i for rows start[s] +
    i, or lengths[s] + path[row] (int32 [rows]).  out: two tensors [rows, kv heads,
    head dim], fp32 or bf16 (rows contiguous, any row pitch); needed without a path, made
    as bf16 with zeroes in rows that are not read otherwise.  The other arguments as for
    kv8_write.  Returns out."""
    what = "q3tts_kv8_read"
    dev, heads, hd, cache, at, shape = _kv8(pool, scales, layer, page_table, lengths, start, what)
    if out is None:
        import torch
        if path is None:
            _bad(what, "out", "given, or a path")
        out = tuple(torch.zeros((path.numel(), heads, hd), dtype=torch.bfloat16, device=pool.device) for _ in range(2))
    n, _, kind, pair = _row_pair(out[0], out[1], ("out[0]", "out[1]"), heads, hd, dev, what)
    rows = _rows8(at, status, shape, dev, kind, n, (n or 1) if max_rows is None else max_rows, what)
    _call(dev, (_lib or load()).q3tts_kv8_read, what, cache, rows,
          None if path is None else _cuda(path, "path", _kv8_types()[3], dev, n, what), *pair)
    return out


def kv8_attention(pool, scales, layer: int, page_table, lengths, start, q, masks=None, max_rows: Optional[int] = None,
                  out=None, status=None):
    """q3tts_kv8_attention: q fp32 or bf16 [rows, q heads, head dim] (rows contiguous,
    any row pitch), rows start[s] .. start[s + 1] - 1 of sequence s at the positions
    after its lengths[s], whose keys and values the cache holds too.  masks: None (a
    row sees the sequence's rows up to itself) or int64 / uint64 [rows], bit j of a
    row's word: it sees row j of its sequence; max_rows: the most rows of a sequence,
    which sizes the launch and its tiles (default: as many as there are rows in all, with masks
    up to MAX_TREE_NODES).  The other arguments as for kv8_write.  Returns out (as q; made if None, with zeroes in rows
    outside every sequence)."""
    what = "q3tts_kv8_attention"
    dev, _, hd, cache, at, shape = _kv8(pool, scales, layer, page_table, lengths, start, what)
    if out is None:
        import torch
        out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    n, heads, kind, pair = _row_pair(q, out, ("q", "out"), None, hd, dev, what)
    if max_rows is None:
        max_rows = max(1, n if masks is None else min(n, MAX_TREE_NODES))
    rows = _rows8(at, status, shape, dev, kind, n, max_rows, what)
    m = None
    if masks is not None:
        wide = _kv8_types()[4]
        m = _cuda(masks, "masks", wide[1] if masks.dtype == wide[1] else wide[0], dev, n, what)
    _call(dev, (_lib or load()).q3tts_kv8_attention, what, cache, rows, m, *pair, heads)
    return out


class Engine:
    """One libq3tts handle over device weights (dict of CUDA tensors named as in
    ``synth.weight_specs``) and a workspace allocated here through torch."""

    def __init__(self, shape, weights: Dict[str, "object"], max_streams: int, kv_cap: int,
                 page_size: int = 16, kv_pages: int = 0, prefill_chunk: int = 0, stream=None):
        import torch
        L = load()
        self.shape = shape
        self.max_streams = max_streams
        self.cfg = make_config(shape, max_streams, kv_cap, page_size, kv_pages, prefill_chunk)
        self._w = weights
        for k, t in weights.items():
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"weight {k} must be a contiguous CUDA tensor")
        def layer(prefix):
            return LayerWeights(*[_ptr(weights.get(f"{prefix}.{k}")) for k in LAYER_KEYS + LAYER_SCALES])

        tl = (LayerWeights * shape.talker_layers)()
        for i in range(shape.talker_layers):
            tl[i] = layer(f"talker.{i}")
        cl = (LayerWeights * shape.cp_layers)()
        for i in range(shape.cp_layers):
            cl[i] = layer(f"cp.{i}")
        proj = weights.get("cp.w_proj")
        self._tl, self._cl = tl, cl
        self.wstruct = Weights(tl, weights["talker.g_final"].data_ptr(),
                               weights["talker.w_head"].data_ptr(),
                               weights["talker.e_codec"].data_ptr(), cl,
                               weights["cp.g_final"].data_ptr(), weights["cp.heads"].data_ptr(),
                               weights["cp.embeds"].data_ptr(), _ptr(proj), _ptr(weights.get("talker.s_head")),
                               _ptr(weights.get("cp.s_heads")), _ptr(weights.get("cp.s_proj")))
        n = L.q3tts_workspace_size(C.byref(self.cfg))
        if n == 0:
            raise Q3TTSError(ERR_ARG, "q3tts_workspace_size")
        self.workspace_bytes = int(n)
        self.workspace = torch.empty(int(n), dtype=torch.uint8, device="cuda")
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        h = C.c_void_p()
        _check(L.q3tts_create(C.byref(self.cfg), C.byref(self.wstruct),
                              self.workspace.data_ptr(), n, C.c_void_p(self.stream.cuda_stream),
                              C.byref(h)), "q3tts_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            # queued work still reads the workspace this object owns: wait for
            # it (a recorded error was the caller's to collect) before release
            load().q3tts_sync_status(self.h)
            load().q3tts_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, stream_id: int, embeds) -> None:
        import torch
        if embeds.dim() != 2 or embeds.shape[1] != self.shape.talker_hidden:
            raise Q3TTSError(ERR_ARG, "q3tts_prefill: embeds must be [len, talker_hidden]")
        _need(embeds, "embeds", torch.float32, embeds.shape[0] * self.shape.talker_hidden,
              "q3tts_prefill")
        _check(load().q3tts_prefill(self.h, stream_id, embeds.data_ptr(), embeds.shape[0]),
               "q3tts_prefill")

    def step_frame(self, stream_ids: Sequence[int], sampling, uniforms, codes, forced=None,
                   logits=None) -> None:
        """uniforms: CUDA fp32 [n, 16]; codes: CUDA int32 [n, 16] (written);
        forced: None or CUDA int32 [n, 16]; logits: None or CUDA fp32
        [n, V_t + 15 V_c].  `sampling` is one Sampling-like object or a list."""
        n = len(stream_ids)
        self._check_frame_buffers(n, uniforms, codes, forced, logits, "q3tts_step_frame")
        if not isinstance(sampling, (list, tuple)):
            sampling = [sampling] * n
        sp = (Sampling * n)(*[sampling_struct(x) for x in sampling])
        ids = (C.c_int32 * n)(*[int(i) for i in stream_ids])
        _check(load().q3tts_step_frame(self.h, sp, ids, n, uniforms.data_ptr(), codes.data_ptr(),
                                       _ptr(forced), _ptr(logits)), "q3tts_step_frame")

    def step_frame_static(self, stream_id: int, sampling, uniforms, codes, forced=None,
                          logits=None) -> None:
        """One frame of one stream through q3tts_step_frame_static (scratch in the
        library's static device array); tensors as for step_frame with n = 1."""
        self._check_frame_buffers(1, uniforms, codes, forced, logits, "q3tts_step_frame_static")
        sp = sampling_struct(sampling)
        _check(load().q3tts_step_frame_static(self.h, C.byref(sp), int(stream_id),
                                              uniforms.data_ptr(), codes.data_ptr(),
                                              _ptr(forced), _ptr(logits)),
               "q3tts_step_frame_static")

    def step_frames(self, stream_ids: Sequence[int], sampling, uniforms, codes, codes_host=None,
                    forced=None) -> None:
        """q3tts_step_frames: F = uniforms.shape[0] frames (<= MAX_CHUNK) enqueued back
        to back.  uniforms: CUDA fp32 [F, n, 16]; codes: CUDA int32 [F, n, 16]
        (written); codes_host: None or a pinned CPU int32 [F, n, 16] tensor (written
        asynchronously, frame by frame); forced: None or CUDA int32 [F, n, 16]."""
        import torch
        n = len(stream_ids)
        F = int(uniforms.shape[0])
        what = "q3tts_step_frames"
        _need(uniforms, "uniforms", torch.float32, F * n * N_CODEBOOKS, what)
        _need(codes, "codes", torch.int32, F * n * N_CODEBOOKS, what)
        if forced is not None:
            _need(forced, "forced", torch.int32, F * n * N_CODEBOOKS, what)
        hp = None
        if codes_host is not None:
            ok = (isinstance(codes_host, torch.Tensor) and not codes_host.is_cuda and codes_host.is_contiguous()
                  and codes_host.dtype == torch.int32 and codes_host.numel() >= F * n * N_CODEBOOKS)
            if not ok:
                raise Q3TTSError(ERR_ARG, f"{what}: codes_host must be a contiguous CPU int32 tensor")
            hp = codes_host.data_ptr()
        if not isinstance(sampling, (list, tuple)):
            sampling = [sampling] * n
        sp = (Sampling * n)(*[sampling_struct(x) for x in sampling])
        ids = (C.c_int32 * n)(*[int(i) for i in stream_ids])
        _check(load().q3tts_step_frames(self.h, sp, ids, n, F, uniforms.data_ptr(), codes.data_ptr(), hp,
                                        _ptr(forced)), what)

    def frames_ready(self) -> int:
        """Frames of the latest step_frames chunk whose codes have landed (non-blocking)."""
        r = load().q3tts_frames_ready(self.h)
        if r < 0:
            _check(r, "q3tts_frames_ready")
        return r

    def stream_codes(self, stream_ids: Sequence[int], sampling, uniforms, chunk: int):
        """Frame-incremental decode of the given streams, chunk frames at a time
        (the counterpart of a streaming session's next_audio_chunk): yields numpy
        int32 arrays [frames, n, 16] of codes in order.  uniforms: CUDA fp32
        [total_frames, n, 16].  Double-buffered: chunk k + 1 is enqueued before
        the host waits for chunk k, so the GPU never idles on the host."""
        import numpy as np
        import torch
        n = len(stream_ids)
        total = int(uniforms.shape[0])
        chunk = max(1, min(int(chunk), MAX_CHUNK))
        dev = [torch.zeros((chunk, n, N_CODEBOOKS), dtype=torch.int32, device="cuda") for _ in range(2)]
        host = [torch.zeros((chunk, n, N_CODEBOOKS), dtype=torch.int32).pin_memory() for _ in range(2)]
        done = [torch.cuda.Event(), torch.cuda.Event()]
        spans = [(f0, min(total, f0 + chunk)) for f0 in range(0, total, chunk)]

        def submit(k):
            f0, f1 = spans[k]
            b = k & 1
            self.step_frames(stream_ids, sampling, uniforms[f0:f1].contiguous(), dev[b][:f1 - f0],
                             codes_host=host[b][:f1 - f0])
            done[b].record(self.stream)

        if spans:
            submit(0)
        for k in range(len(spans)):
            if k + 1 < len(spans):
                submit(k + 1)
            done[k & 1].synchronize()
            f0, f1 = spans[k]
            yield np.array(host[k & 1][:f1 - f0].numpy(), copy=True)

    def _check_frame_buffers(self, n, uniforms, codes, forced, logits, what):
        import torch
        _need(uniforms, "uniforms", torch.float32, n * N_CODEBOOKS, what)
        _need(codes, "codes", torch.int32, n * N_CODEBOOKS, what)
        if forced is not None:
            _need(forced, "forced", torch.int32, n * N_CODEBOOKS, what)
        if logits is not None:
            s = self.shape
            _need(logits, "logits", torch.float32, n * (s.codec_vocab + 15 * s.cp_vocab), what)

    def read_pending(self, stream_id: int):
        import torch
        hdn = torch.empty(self.shape.talker_hidden, dtype=torch.float32, device="cuda")
        lg = torch.empty(self.shape.codec_vocab, dtype=torch.float32, device="cuda")
        _check(load().q3tts_read_pending(self.h, stream_id, hdn.data_ptr(), lg.data_ptr()),
               "q3tts_read_pending")
        return hdn, lg

    def reset(self, stream_id: int = -1) -> None:
        _check(load().q3tts_reset(self.h, stream_id), "q3tts_reset")

    def length(self, stream_id: int) -> int:
        rc = load().q3tts_stream_length(self.h, stream_id)
        if rc < 0:
            raise Q3TTSError(rc, "q3tts_stream_length")
        return rc

    def finished(self, stream_id: int) -> bool:
        """Whether the stream fed its end-of-stream code since its last prefill
        (waits for the engine's stream)."""
        f = C.c_int(0)
        _check(load().q3tts_stream_finished(self.h, stream_id, C.byref(f)), "q3tts_stream_finished")
        return bool(f.value)

    def fork(self, src: int, dst: Sequence[int]) -> None:
        """q3tts_fork: the streams dst become what stream src is now."""
        ids = (C.c_int32 * max(1, len(dst)))(*[int(i) for i in dst])
        _check(load().q3tts_fork(self.h, int(src), ids, len(dst)), "q3tts_fork")

    def tree_step(self, stream_id: int, codes, parents: Sequence[int], hidden=None, logits=None) -> None:
        """q3tts_tree_step: codes CUDA int32 [n, 16], parents n ints (-1: the context);
        hidden: None or CUDA fp32 [n, D_t], logits: None or CUDA fp32 [n, V_t] (written)."""
        import torch
        n, what = len(parents), "q3tts_tree_step"
        _need(codes, "codes", torch.int32, n * N_CODEBOOKS, what)
        if hidden is not None:
            _need(hidden, "hidden", torch.float32, n * self.shape.talker_hidden, what)
        if logits is not None:
            _need(logits, "logits", torch.float32, n * self.shape.codec_vocab, what)
        p = (C.c_int32 * max(1, n))(*[int(i) for i in parents])
        _check(load().q3tts_tree_step(self.h, int(stream_id), codes.data_ptr(), p, n, _ptr(hidden), _ptr(logits)),
               what)

    def tree_accept(self, stream_id: int, path: Sequence[int]) -> None:
        """q3tts_tree_accept: the path's frames become part of the stream."""
        p = (C.c_int32 * max(1, len(path)))(*[int(i) for i in path])
        _check(load().q3tts_tree_accept(self.h, int(stream_id), p, len(path)), "q3tts_tree_accept")

    def beam_frame(self, stream_ids: Sequence[Sequence[int]], sampling, scores, uniforms, codes):
        """q3tts_beam_frame: stream_ids [groups][beams]; scores CUDA fp32 [groups, beams]
        (read and written); uniforms CUDA fp32 and codes CUDA int32 [groups * beams,
        16].  Returns the parents, an int32 array [groups, beams]."""
        import numpy as np
        import torch
        what = "q3tts_beam_frame"
        groups, beams = len(stream_ids), len(stream_ids[0]) if stream_ids else 0
        if any(len(g) != beams for g in stream_ids):
            _bad(what, "stream_ids", "groups of equally many streams")
        n = groups * beams
        _need(scores, "scores", torch.float32, n, what)
        self._check_frame_buffers(n, uniforms, codes, None, None, what)
        ids = (C.c_int32 * max(1, n))(*[int(i) for g in stream_ids for i in g])
        par = (C.c_int32 * max(1, n))()
        sp = sampling_struct(sampling)
        _check(load().q3tts_beam_frame(self.h, C.byref(sp), ids, groups, beams, scores.data_ptr(), uniforms.data_ptr(),
                                       codes.data_ptr(), par), what)
        return np.frombuffer(par, dtype=np.int32)[:n].reshape(groups, beams).copy()

    def kernel_launches(self) -> int:
        return int(load().q3tts_kernel_launches(self.h))

    def debug_fail_barrier(self, barrier: int, wait_us: int) -> None:
        """Arms the next persistent frame to leave out CTA 0's arrival at grid
        barrier `barrier` with every wait bounded to wait_us (failure-path test)."""
        _check(load().q3tts_debug_fail_barrier(self.h, int(barrier), int(wait_us)),
               "q3tts_debug_fail_barrier")

    def sync(self) -> None:
        _check(load().q3tts_sync_status(self.h), "q3tts_sync_status")
