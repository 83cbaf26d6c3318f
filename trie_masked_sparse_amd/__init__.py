"""Python binding of libtms.so (include/tms.h): argument marshalling only.

Every function here forwards to the C entry point of the same name (without
the ``tms_`` prefix); all compute runs in the HIP kernels of the library.
Device buffers are torch tensors (only their data pointers are passed), the
stream defaults to torch's current stream.  There is no fallback: if the
library is not built, or no GPU is present, calls raise.

Fail loudly (page "Constraint made cheaper than no constraint", section
"Masked sampling inside the sampler": an empty mask or an unwalkable token is
an error, never a silent pick): the decode calls (decode_step_sparse,
decode_step_dense_masked, decode_k_pointers, advance_forced) synchronise the
stream after enqueueing their work and raise TmsError when any sequence holds a
device error (EMPTY_MASK, NOT_WALKABLE, NOT_DONE), unless called with
check=False, which leaves them asynchronous (for timed loops and for tests of
the error paths; State.status() then reports the per-sequence codes).  A state
is passed as a State or as its raw handle.

torch is imported before the library is loaded so that both use the same HIP
runtime (torch ships its own libamdhip64 with the same soname).
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtms.so")

OK, ERR_INVALID_ARG, ERR_CATALOG, ERR_FANOUT, ERR_K, ERR_EMPTY_MASK, ERR_NOT_WALKABLE, ERR_NOT_DONE, \
    ERR_BUSY, ERR_OOM, ERR_HIP = range(11)
F32, BF16 = 0, 1
PATH_AUTO, PATH_FAST, PATH_GLOBAL = 0, 1, 2
LOOP_RESIDENT, LOOP_GRAPH, LOOP_STREAM, LOOP_RESIDENT_SOLO, LOOP_RESIDENT_GROUPED = 0, 1, 2, 3, 4

# every symbol declared in include/tms.h
EXPORTS = (
    "tms_trie_build", "tms_trie_upload", "tms_charset_build", "tms_charset_upload", "tms_trie_info_get",
    "tms_trie_export_csr", "tms_trie_free",
    "tms_state_create", "tms_state_reset", "tms_state_sync_status", "tms_state_export", "tms_state_free",
    "tms_decode_step_sparse", "tms_decode_step_dense_masked", "tms_decode_k_pointers",
    "tms_advance_forced", "tms_legal_set", "tms_legal_mask", "tms_mask_to_rows", "tms_gather_gemv",
    "tms_debug_set_live",
    "tms_state_set_split", "tms_state_set_loop", "tms_state_set_norepeat", "tms_state_set_step_grouping",
    "tms_state_get_launch",
    "tms_decode_k_pointers_noalloc", "tms_read_reference",
    "tms_kv_work_bytes", "tms_kv_fork", "tms_kv_reserve", "tms_kv_write", "tms_kv_attention", "tms_kv_commit",
    "tms_kv_sync_status",
    "tms_status_str", "tms_last_error",
)
NOREPEAT_LIVE, NOREPEAT_BITMASK = 0, 1
KV_WORK_ZERO = 2048  # bytes of the work memory that are zero between calls
STEP_GROUP_AUTO, STEP_GROUP_OFF, STEP_GROUP_ROOT, STEP_GROUP_NODES = 0, 1, 2, 3
NOALLOC_SCRATCH_BYTES = 32 << 20


class TmsError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        super().__init__(f"{where}: status {code} ({status_str(code)}) {detail}".rstrip())


class TrieInfo(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_nodes", "n_edges", "n_entries", "cap", "max_depth", "sep", "stop",
                                         "vocab", "path")] + [("device_bytes", C.c_int64)]


class KvDescriptor(C.Structure):
    """tms_kv"""
    _fields_ = [(n, C.c_void_p) for n in ("kv", "table", "length", "held", "refs", "status", "work")] + \
        [("work_bytes", C.c_int64)] + \
        [(n, C.c_int32) for n in ("dtype", "layers", "pages", "kv_heads", "page_tokens", "head_dim", "seqs",
                                  "max_pages")]


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with python -m trie_masked_sparse_amd.build")
        L = C.CDLL(LIB_PATH)
        P, i32 = C.c_void_p, C.c_int32
        PP = C.POINTER(C.c_void_p)
        sig = {
            "tms_trie_build": [P, P, i32, i32, i32, i32, PP],
            "tms_trie_upload": [P, P, i32, i32, i32, i32, C.c_int, P, PP],
            "tms_charset_build": [P, P, i32, P, P, i32, i32, i32, PP],
            "tms_charset_upload": [P, P, i32, P, P, i32, i32, i32, C.c_int, P, PP],
            "tms_trie_info_get": [P, C.POINTER(TrieInfo)],
            "tms_trie_export_csr": [P, P, P, P, P, P],
            "tms_trie_free": [P],
            "tms_state_create": [P, i32, i32, P, C.c_int, i32, P, PP],
            "tms_state_reset": [P, P],
            "tms_state_sync_status": [P, P, P],
            "tms_state_export": [P, P, P, P, P, P, P, P, P, P],
            "tms_state_free": [P],
            "tms_decode_step_sparse": [P, P, P, P, P],
            "tms_decode_step_dense_masked": [P, P, P, P, P, P],
            "tms_decode_k_pointers": [P, P, i32, P, P, P, P],
            "tms_advance_forced": [P, P, P],
            "tms_legal_set": [P, P, P, P],
            "tms_legal_mask": [P, P, P],
            "tms_mask_to_rows": [P, i32, i32, i32, P, P, P],
            "tms_gather_gemv": [P, C.c_int, i32, i32, P, P, P, i32, i32, P, P],
            "tms_debug_set_live": [P, i32, i32, i32, P],
            "tms_state_set_split": [P, i32],
            "tms_state_set_loop": [P, i32],
            "tms_state_set_norepeat": [P, i32],
            "tms_state_set_step_grouping": [P, i32],
            "tms_read_reference": [P, C.c_int64, P, i32, i32, P],
            "tms_decode_k_pointers_noalloc": [P, P, C.c_int, i32, i32, i32, P, i32, P, P, P, P, P],
            "tms_state_get_launch": [P, P, P],
            "tms_kv_work_bytes": [P, P],
            "tms_kv_fork": [P, P, P],
            "tms_kv_reserve": [P, P, P],
            "tms_kv_write": [P, i32, P, i32, P, C.c_int64, i32, P, P, C.c_int64, P, C.c_int64, P, P, C.c_float, P, P,
                             i32, i32, P],
            "tms_kv_attention": [P, i32, P, C.c_int64, i32, P, i32, i32, P, C.c_float, P, P],
            "tms_kv_commit": [P, P, P, i32, P],
            "tms_kv_sync_status": [P, P, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = C.c_int
        L.tms_status_str.argtypes = [C.c_int]
        L.tms_status_str.restype = C.c_char_p
        L.tms_last_error.argtypes = []
        L.tms_last_error.restype = C.c_char_p
        _lib = L
    return _lib


def status_str(code: int) -> str:
    return lib().tms_status_str(int(code)).decode()


def _check(rc: int, where: str):
    if rc != OK:
        raise TmsError(rc, where, lib().tms_last_error().decode())


def _stream(stream):
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _dev(t, dtype=None, name="tensor"):
    """Data pointer of a contiguous GPU tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA/HIP torch tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return C.c_void_p(t.data_ptr())


def _host_i32(a):
    return np.ascontiguousarray(a, dtype=np.int32)


def _catalog_arrays(entries):
    if isinstance(entries, tuple) and len(entries) == 2:
        toks, offs = entries
    else:
        offs = np.zeros(len(entries) + 1, dtype=np.int64)
        offs[1:] = np.cumsum([len(e) for e in entries])
        toks = np.array([t for e in entries for t in e] or [0], dtype=np.int32)
    return _host_i32(toks), np.ascontiguousarray(offs, dtype=np.int64)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return BF16
    raise TypeError("embedding and hidden states are float32 or bfloat16 (raw 16-bit patterns allowed)")


# --------------------------------------------------------------------------- tries

def trie_build(entries, vocab: int, sep: int, stop: int):
    toks, offs = _catalog_arrays(entries)
    h = C.c_void_p()
    _check(lib().tms_trie_build(toks.ctypes.data, offs.ctypes.data, len(offs) - 1, vocab, sep, stop, C.byref(h)),
           "trie_build")
    return h


def trie_upload(entries, vocab: int, sep: int, stop: int, path: int = PATH_AUTO, stream=None):
    toks, offs = _catalog_arrays(entries)
    h = C.c_void_p()
    _check(lib().tms_trie_upload(toks.ctypes.data, offs.ctypes.data, len(offs) - 1, vocab, sep, stop, path,
                                 _stream(stream), C.byref(h)), "trie_upload")
    return h


def _bytes_arrays(items):
    off = np.zeros(len(items) + 1, dtype=np.int64)
    off[1:] = np.cumsum([len(x) for x in items])
    buf = np.frombuffer(b"".join(bytes(x) for x in items) or b"\0", np.uint8).copy()
    return buf, off


def charset_build(strings, vocab, sep: int, stop: int):
    """strings: catalog byte strings; vocab: byte string of every token id."""
    sb, so = _bytes_arrays(strings)
    tb, to = _bytes_arrays(vocab)
    h = C.c_void_p()
    _check(lib().tms_charset_build(sb.ctypes.data, so.ctypes.data, len(strings), tb.ctypes.data, to.ctypes.data,
                                   len(vocab), sep, stop, C.byref(h)), "charset_build")
    return h


def charset_upload(strings, vocab, sep: int, stop: int, path: int = PATH_AUTO, stream=None):
    sb, so = _bytes_arrays(strings)
    tb, to = _bytes_arrays(vocab)
    h = C.c_void_p()
    _check(lib().tms_charset_upload(sb.ctypes.data, so.ctypes.data, len(strings), tb.ctypes.data, to.ctypes.data,
                                    len(vocab), sep, stop, path, _stream(stream), C.byref(h)), "charset_upload")
    return h


def trie_info_get(trie) -> dict:
    info = TrieInfo()
    _check(lib().tms_trie_info_get(trie, C.byref(info)), "trie_info_get")
    return {n: getattr(info, n) for n, _ in TrieInfo._fields_}


def trie_export_csr(trie) -> dict:
    i = trie_info_get(trie)
    out = {"begin": np.zeros(i["n_nodes"] + 1, np.int32), "entry": np.zeros(i["n_nodes"], np.int32),
           "tok": np.zeros(i["n_edges"], np.int32), "child": np.zeros(i["n_edges"], np.int32),
           "live0": np.zeros(i["n_edges"], np.int32)}
    _check(lib().tms_trie_export_csr(trie, *(out[n].ctypes.data for n in ("begin", "entry", "tok", "child",
                                                                            "live0"))), "trie_export_csr")
    return out


def trie_free(trie):
    _check(lib().tms_trie_free(trie), "trie_free")


# --------------------------------------------------------------------------- states

def state_create(trie, B: int, k: int, emb: torch.Tensor, stream=None):
    if emb.dim() != 2:
        raise ValueError("emb must be [V][H]")
    h = C.c_void_p()
    _check(lib().tms_state_create(trie, B, k, _dev(emb, name="emb"), _dtype_code(emb), emb.shape[1],
                                  _stream(stream), C.byref(h)), "state_create")
    return h


def state_reset(st, stream=None):
    _check(lib().tms_state_reset(_handle(st), _stream(stream)), "state_reset")


def state_sync_status(st, B: int, stream=None, check: bool = True) -> np.ndarray:
    out = np.zeros(B, np.int32)
    rc = lib().tms_state_sync_status(_handle(st), out.ctypes.data, _stream(stream))
    if rc not in (OK, ERR_EMPTY_MASK, ERR_NOT_WALKABLE, ERR_NOT_DONE) or (check and rc != OK):
        _check(rc, "state_sync_status")
    return out


def state_export(st, B: int, k: int, n_edges: int, live: bool = False, stream=None) -> dict:
    out = {n: np.zeros(B, np.int32) for n in ("node", "depth", "done", "status", "finished", "n_emitted")}
    out["entries"] = np.zeros((B, k), np.int32)
    lv = np.zeros((B, n_edges), np.int32) if live else None
    _check(lib().tms_state_export(_handle(st), *(out[n].ctypes.data for n in ("node", "depth", "done", "status", "finished",
                                                                      "n_emitted", "entries")),
                                  lv.ctypes.data if live else None, _stream(stream)), "state_export")
    if live:
        out["live"] = lv
    return out


def state_free(st):
    _check(lib().tms_state_free(_handle(st)), "state_free")


def state_set_split(st, split: int):
    _check(lib().tms_state_set_split(_handle(st), split), "state_set_split")


def state_set_loop(st, mode: int):
    _check(lib().tms_state_set_loop(_handle(st), mode), "state_set_loop")


def state_set_norepeat(st, kind: int):
    _check(lib().tms_state_set_norepeat(_handle(st), kind), "state_set_norepeat")


def state_set_step_grouping(st, mode: int):
    _check(lib().tms_state_set_step_grouping(_handle(st), mode), "state_set_step_grouping")


def state_get_launch(st):
    s, g = C.c_int32(), C.c_int32()
    _check(lib().tms_state_get_launch(_handle(st), C.byref(s), C.byref(g)), "state_get_launch")
    return s.value, g.value


# --------------------------------------------------------------------------- decode

_HID = (torch.float32, torch.bfloat16, torch.int16, torch.uint16)


def _handle(st):
    return st.h if isinstance(st, State) else st


def _recording(stream) -> bool:
    """Whether the stream (default: the current one) is being recorded into a
    graph; False for a raw handle, which torch cannot ask about."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    if isinstance(stream, torch.cuda.Stream):
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()
    return False


def _refuse_check_while_recording(check: bool, stream, where: str):
    """check=True synchronises the stream, which a recording cannot do: refuse
    before anything is recorded, with what to do instead."""
    if check and _recording(stream):
        raise TmsError(ERR_INVALID_ARG, where, "check=True synchronises the stream, which is being recorded into a "
                       "graph: pass check=False and read State.status() after a replay")


def _raise_device_errors(st, stream, where: str):
    """Synchronise the stream and raise TmsError if any sequence of st holds a
    device error; the message names the first such sequence and, for a State,
    lists every sequence's status."""
    B = st.B if isinstance(st, State) else 0
    buf = np.zeros(max(B, 1), np.int32)
    rc = lib().tms_state_sync_status(_handle(st), buf.ctypes.data if B else None, _stream(stream))
    if rc != OK:
        detail = lib().tms_last_error().decode()
        if B:
            bad = {i: int(x) for i, x in enumerate(buf) if x != OK}
            detail += f"; {len(bad)} of {B} sequences in error: {dict(list(bad.items())[:16])}"
        raise TmsError(rc, where, detail)


def decode_step_sparse(st, hidden, tok, logit=None, stream=None, check: bool = True):
    _refuse_check_while_recording(check, stream, "decode_step_sparse")
    _check(lib().tms_decode_step_sparse(_handle(st), _dev(hidden, _HID, "hidden"), _dev(tok, torch.int32, "tok"),
                                        _dev(logit, torch.float32, "logit"), _stream(stream)),
           "decode_step_sparse")
    if check:
        _raise_device_errors(st, stream, "decode_step_sparse")


def decode_step_dense_masked(st, hidden, tok, logit=None, full_logits=None, stream=None, check: bool = True):
    _refuse_check_while_recording(check, stream, "decode_step_dense_masked")
    _check(lib().tms_decode_step_dense_masked(_handle(st), _dev(hidden, _HID, "hidden"),
                                              _dev(tok, torch.int32, "tok"), _dev(logit, torch.float32, "logit"),
                                              _dev(full_logits, torch.float32, "full_logits"), _stream(stream)),
           "decode_step_dense_masked")
    if check:
        _raise_device_errors(st, stream, "decode_step_dense_masked")


def decode_k_pointers(st, hidden_seq, tokens, len=None, entries=None, stream=None, check: bool = True):  # noqa: A002
    _refuse_check_while_recording(check, stream, "decode_k_pointers")
    T = hidden_seq.shape[0]
    _check(lib().tms_decode_k_pointers(_handle(st), _dev(hidden_seq, _HID, "hidden_seq"), T,
                                       _dev(tokens, torch.int32, "tokens"), _dev(len, torch.int32, "len"),
                                       _dev(entries, torch.int32, "entries"), _stream(stream)),
           "decode_k_pointers")
    if check:
        _raise_device_errors(st, stream, "decode_k_pointers")


def decode_k_pointers_noalloc(trie, emb, k: int, hidden_seq, tokens, status, len=None, entries=None,  # noqa: A002
                              stream=None, check: bool = True):
    """One whole answer per sequence with the decode state in the library's
    per-GPU scratch (no state handle, no allocation).  status: dev int32 [B].
    check: synchronise and raise TmsError on any per-sequence device error."""
    T, B, H = hidden_seq.shape
    if emb.dim() != 2 or emb.shape[1] != H:
        raise ValueError("emb must be [V][H] with the hidden size of hidden_seq")
    _refuse_check_while_recording(check, stream, "decode_k_pointers_noalloc")
    _check(lib().tms_decode_k_pointers_noalloc(trie.h if isinstance(trie, Trie) else trie, _dev(emb, name="emb"),
                                               _dtype_code(emb), H, B, k, _dev(hidden_seq, _HID, "hidden_seq"), T,
                                               _dev(tokens, torch.int32, "tokens"), _dev(len, torch.int32, "len"),
                                               _dev(entries, torch.int32, "entries"),
                                               _dev(status, torch.int32, "status"), _stream(stream)),
           "decode_k_pointers_noalloc")
    if check:
        torch.cuda.synchronize()
        bad = status.cpu().numpy()
        if (bad != OK).any():
            first = int(np.nonzero(bad != OK)[0][0])
            raise TmsError(int(bad[first]), "decode_k_pointers_noalloc",
                           f"sequence {first}; {int((bad != OK).sum())} of {B} sequences in error")


def advance_forced(st, tok, stream=None, check: bool = True):
    _refuse_check_while_recording(check, stream, "advance_forced")
    _check(lib().tms_advance_forced(_handle(st), _dev(tok, torch.int32, "tok"), _stream(stream)), "advance_forced")
    if check:
        _raise_device_errors(st, stream, "advance_forced")


def legal_set(st, legal_tok, n_legal, stream=None):
    _check(lib().tms_legal_set(_handle(st), _dev(legal_tok, torch.int32, "legal_tok"), _dev(n_legal, torch.int32, "n_legal"),
                               _stream(stream)), "legal_set")


def legal_mask(st, mask, stream=None):
    _check(lib().tms_legal_mask(_handle(st), _dev(mask, torch.int32, "mask"), _stream(stream)), "legal_mask")


def mask_to_rows(mask, V: int, rows, n_rows, stream=None):
    B, cap = rows.shape
    _check(lib().tms_mask_to_rows(_dev(mask, torch.int32, "mask"), B, V, cap, _dev(rows, torch.int32, "rows"),
                                  _dev(n_rows, torch.int32, "n_rows"), _stream(stream)), "mask_to_rows")


def gather_gemv(emb, hidden, rows, n_rows, out, stream=None):
    B, cap = rows.shape
    _check(lib().tms_gather_gemv(_dev(emb, _HID, "emb"), _dtype_code(emb), emb.shape[0], emb.shape[1],
                                 _dev(hidden, _HID, "hidden"), _dev(rows, torch.int32, "rows"),
                                 _dev(n_rows, torch.int32, "n_rows"), B, cap, _dev(out, torch.float32, "out"),
                                 _stream(stream)), "gather_gemv")


def read_reference(src, out, grid: int = 0, unroll: int = 0, nbytes: int | None = None, stream=None):
    """Streaming read of src (a contiguous GPU tensor; nbytes of it, default
    all) into the XOR words out (int32 [1024]): the bandwidth reference."""
    have = src.numel() * src.element_size()
    n = have if nbytes is None else int(nbytes)
    if n > have:
        raise ValueError(f"read_reference: {n} bytes asked of a {have}-byte tensor")
    if out.numel() < 1024:
        raise ValueError("read_reference: out must hold 1024 words")
    _check(lib().tms_read_reference(_dev(src, name="src"), n, _dev(out, torch.int32, "out"), grid, unroll,
                                    _stream(stream)), "read_reference")


def debug_set_live(st, s: int, edge: int, value: int, stream=None):
    _check(lib().tms_debug_set_live(_handle(st), s, edge, value, _stream(stream)), "debug_set_live")


# --------------------------------------------------------------------------- paged key/value cache

# The calls of a decode step are short: what they look up is bound here.
_Tensor, _int32 = torch.Tensor, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # not in a torch without GPUs


def _sized(t, dtype, numel: int, name: str):
    """Address of a contiguous GPU tensor of at least numel values."""
    if type(t) is _Tensor and t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    _dev(t, dtype, name)  # says what is wrong, or takes a subclass of Tensor
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} values, {numel} are needed")
    return t.data_ptr()


def _token_rows(t, dtype, dim: int, name: str):
    """(address, tokens, heads, row stride in elements) of a GPU tensor
    [T][heads][dim] whose tokens are contiguous (a slice of a wider projection
    may hold them)."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA/HIP torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"{name} must be [T][heads][{dim}]")
    T, heads, _ = shape
    if T == 0:  # no tokens: strides say nothing
        return None, 0, heads, heads * dim
    row, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), T, heads, row if T > 1 else heads * dim  # one token: no next row


class PagedCache:
    """Keys and values of a batch of sequences in shared pages: the caller's
    tensors, kept alive and changed in place by the kv_* calls, and the work
    memory those share (calls on several streams have to be ordered by the
    caller, as for one State).

    kv [layers][pages][2][kv_heads][page_tokens][head_dim] (float32 or
    bfloat16); int32 table [seqs][max_pages], length, held, status [seqs] and
    refs [pages].  PagedCache.empty() makes an empty one."""

    def __init__(self, kv, table, length, held, refs, status):
        if kv.dim() != 6 or kv.shape[2] != 2:
            raise ValueError("kv must be [layers][pages][2][kv_heads][page_tokens][head_dim]")
        if kv.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("kv must be float32 or bfloat16")
        if table.dim() != 2:
            raise ValueError("table must be [seqs][max_pages]")
        self.layers, self.pages, _, self.kv_heads, self.page_tokens, self.head_dim = kv.shape
        self.seqs, self.max_pages = table.shape
        self.dtype = kv.dtype
        for name, t, n in (("length", length, self.seqs), ("held", held, self.seqs), ("status", status, self.seqs),
                           ("refs", refs, self.pages)):
            if t.numel() != n:
                raise ValueError(f"{name} has {t.numel()} values, expected {n}")
        for t in (kv, table, length, held, refs, status):
            if t.device != kv.device:
                raise ValueError("the cache's tensors must be on one device")
        self.kv, self.table, self.length, self.held, self.refs, self.status_codes = kv, table, length, held, refs, status
        d = KvDescriptor(_dev(kv, name="kv"), _dev(table, torch.int32, "table"), _dev(length, torch.int32, "length"),
                         _dev(held, torch.int32, "held"), _dev(refs, torch.int32, "refs"),
                         _dev(status, torch.int32, "status"), None, 0, F32 if kv.dtype == torch.float32 else BF16,
                         self.layers, self.pages, self.kv_heads, self.page_tokens, self.head_dim, self.seqs,
                         self.max_pages)
        need = C.c_int64()
        _check(lib().tms_kv_work_bytes(C.byref(d), C.byref(need)), "PagedCache")
        self.work = torch.empty(need.value, dtype=torch.uint8, device=kv.device)
        self.work[:KV_WORK_ZERO].zero_()
        self._index = kv.device.index
        self._streams = set()  # that work on the cache
        d.work, d.work_bytes = self.work.data_ptr(), need.value
        self.d = d
        self.ref = C.byref(d)
        c = lib()
        self._c = c.tms_kv_fork, c.tms_kv_reserve, c.tms_kv_write, c.tms_kv_attention, c.tms_kv_commit

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, page_tokens: int, head_dim: int, seqs: int, max_pages: int,
              dtype=torch.bfloat16, device="cuda"):
        def ints(*shape, value=0):
            return torch.full(shape, value, dtype=torch.int32, device=device)
        return cls(torch.empty((layers, pages, 2, kv_heads, page_tokens, head_dim), dtype=dtype, device=device),
                   ints(seqs, max_pages, value=-1), ints(seqs), ints(seqs), ints(pages), ints(seqs))

    def status(self, stream=None, check: bool = False) -> np.ndarray:
        out = np.zeros(self.seqs, np.int32)
        rc = lib().tms_kv_sync_status(self.ref, out.ctypes.data, _stream(stream))
        if rc not in (OK, ERR_OOM, ERR_INVALID_ARG) or (check and rc != OK):
            _check(rc, "kv_sync_status")
        return out


def _kv_stream(cache: PagedCache, stream):
    """The stream of a call; the cache's tensors are told of it the first time, so
    that a cache that is dropped is not handed on while the stream works on it."""
    if stream is None:
        s = _raw_stream(cache._index)
    else:
        s = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if s not in cache._streams:
        on = torch.cuda.ExternalStream(s, device=cache.kv.device)
        for t in (cache.kv, cache.table, cache.length, cache.held, cache.refs, cache.status_codes, cache.work):
            t.record_stream(on)
        cache._streams.add(s)
    return s


def _raise_kv_errors(cache: PagedCache, stream, where: str):
    buf = np.zeros(cache.seqs, np.int32)
    rc = lib().tms_kv_sync_status(cache.ref, buf.ctypes.data, _stream(stream))
    if rc != OK:
        bad = {i: int(x) for i, x in enumerate(buf) if x != OK}
        raise TmsError(rc, where, f"{lib().tms_last_error().decode()}; {len(bad)} of {cache.seqs} sequences in error: "
                                  f"{dict(list(bad.items())[:16])}")


def kv_fork(cache: PagedCache, src, stream=None, check: bool = True):
    """Sequence s becomes what src[s] was (int32 [seqs]; itself: unchanged,
    -1: emptied).  check: synchronise and raise on device errors."""
    if check:
        _refuse_check_while_recording(check, stream, "kv_fork")
    rc = cache._c[0](cache.ref, _sized(src, _int32, cache.seqs, "src"), _kv_stream(cache, stream))
    if rc:
        _check(rc, "kv_fork")
    if check:
        _raise_kv_errors(cache, stream, "kv_fork")


def kv_reserve(cache: PagedCache, n_new, stream=None, check: bool = True):
    """Pages for n_new[s] more rows of every sequence (int32 [seqs])."""
    if check:
        _refuse_check_while_recording(check, stream, "kv_reserve")
    rc = cache._c[1](cache.ref, _sized(n_new, _int32, cache.seqs, "n_new"), _kv_stream(cache, stream))
    if rc:
        _check(rc, "kv_reserve")
    if check:
        _raise_kv_errors(cache, stream, "kv_reserve")


def kv_write(cache: PagedCache, layer: int, k, v, start, q=None, q_out=None, q_weight=None, k_weight=None,
             eps: float = 1e-6, pos=None, inv_freq=None, interleaved: bool = False, stream=None):
    """Norm, rotation and cache rows of the packed new tokens (tms_kv_write).
    k, v, q: [T][heads][head_dim], the tokens' rows any multiple of 16 bytes
    apart; start: int32 [seqs+1].  Asynchronous: PagedCache.status() reports."""
    dt, D, hkv = cache.dtype, cache.head_dim, cache.kv_heads
    kp, T, hk, ldk = _token_rows(k, dt, D, "k")
    vp, Tv, hv, ldv = _token_rows(v, dt, D, "v")
    if hk != hkv or hv != hkv or Tv != T:
        raise ValueError("k and v must be [T][kv_heads][head_dim]")
    qp, ldq, hq, qo = None, 0, 0, None
    if q is not None:
        qp, Tq, hq, ldq = _token_rows(q, dt, D, "q")
        if Tq != T:
            raise ValueError("q must have the tokens of k")
        if q_out is None:
            raise ValueError("q needs q_out")
        qo = _sized(q_out, dt, T * hq * D, "q_out")
    n_freq = 0 if inv_freq is None else inv_freq.numel()
    if n_freq and pos is None:
        raise ValueError("inv_freq needs pos")
    rc = cache._c[2](cache.ref, layer, _sized(start, _int32, cache.seqs + 1, "start"), T, qp, ldq, hq, qo, kp, ldk, vp, ldv,
                     None if q_weight is None else _sized(q_weight, dt, D, "q_weight"),
                     None if k_weight is None else _sized(k_weight, dt, D, "k_weight"), eps,
                     _sized(pos, _int32, T, "pos") if n_freq else None,
                     _sized(inv_freq, torch.float32, n_freq, "inv_freq") if n_freq else None, n_freq, int(interleaved),
                     _kv_stream(cache, stream))
    if rc:
        _check(rc, "kv_write")


_MAX_TREE = 1024  # drafts of a tree


def _longest(cache: PagedCache, start, stream, T: int) -> int:
    """The most tokens of a sequence, read back from start on the call's stream;
    T where that is being recorded into a graph."""
    s = torch.cuda.ExternalStream(_kv_stream(cache, stream), device=cache.kv.device)
    with torch.cuda.stream(s):
        if torch.cuda.is_current_stream_capturing():
            return T
        at = start.flatten()[:cache.seqs + 1].cpu()
    return int((at[1:] - at[:-1]).max().clamp(1, T))


def kv_attention(cache: PagedCache, layer: int, q, start, out, scale: float | None = None, parent=None,
                 max_new: int | None = None, stream=None):
    """Attention of the packed new tokens over the cache (tms_kv_attention):
    parent (int32 [T]) makes them a tree of drafts, without it they are causal.
    q, out: [T][q_heads][head_dim]; scale: head_dim ** -0.5 by default;
    max_new: the most tokens of a sequence.  Give it: the kernels are chosen by
    it, and without it (T) a batch of single tokens runs on those for whole
    prompts.  Asynchronous, but for trees of more than 1024 tokens in all
    without max_new, which read it from start."""
    dt, D = cache.dtype, cache.head_dim
    qp, T, hq, ldq = _token_rows(q, dt, D, "q")
    at = _sized(start, _int32, cache.seqs + 1, "start")
    if max_new is None:
        max_new = _longest(cache, start, stream, T) if parent is not None and T > _MAX_TREE else T
    rc = cache._c[3](cache.ref, layer, qp, ldq, hq, at, T, max_new, None if parent is None else _sized(parent, _int32, T, "parent"),
                     D ** -0.5 if scale is None else scale, _sized(out, dt, T * hq * D, "out"), _kv_stream(cache, stream))
    if rc:
        _check(rc, "kv_attention")


def kv_commit(cache: PagedCache, n_keep, keep=None, stream=None, check: bool = True):
    """Keep the accepted new rows: n_keep int32 [seqs], keep int32
    [seqs][stride] ascending indices (None: the first n_keep), and give the
    pages past them back."""
    if check:
        _refuse_check_while_recording(check, stream, "kv_commit")
    stride, at = 0, None
    if keep is not None:
        if keep.dim() != 2 or keep.shape[0] != cache.seqs:
            raise ValueError("keep must be [seqs][stride]")
        stride, at = keep.shape[1], _sized(keep, _int32, 1, "keep")
    rc = cache._c[4](cache.ref, _sized(n_keep, _int32, cache.seqs, "n_keep"), at, stride, _kv_stream(cache, stream))
    if rc:
        _check(rc, "kv_commit")
    if check:
        _raise_kv_errors(cache, stream, "kv_commit")


# --------------------------------------------------------------------------- handles

class Trie:
    """Owning wrapper of a tms_trie handle."""

    def __init__(self, entries, vocab: int, sep: int, stop: int, path: int = PATH_AUTO, upload: bool = True,
                 stream=None, _handle=None):
        if _handle is not None:
            self.h = _handle
        else:
            self.h = trie_upload(entries, vocab, sep, stop, path, stream) if upload else \
                trie_build(entries, vocab, sep, stop)
        self.info = trie_info_get(self.h)

    @classmethod
    def from_charset(cls, strings, vocab, sep: int, stop: int, path: int = PATH_AUTO, upload: bool = True,
                     stream=None):
        """A character-level catalog: byte strings and the byte string of
        every token id (answers pick one string, k = 1)."""
        h = charset_upload(strings, vocab, sep, stop, path, stream) if upload else \
            charset_build(strings, vocab, sep, stop)
        return cls(None, 0, 0, 0, _handle=h)

    def csr(self):
        return trie_export_csr(self.h)

    def close(self):
        if getattr(self, "h", None) is not None:
            trie_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class State:
    """Owning wrapper of a tms_state handle; keeps the embedding tensor alive."""

    def __init__(self, trie: Trie, B: int, k: int, emb: torch.Tensor, stream=None):
        self.trie, self.B, self.k, self.emb = trie, B, k, emb
        self.h = state_create(trie.h, B, k, emb, stream)

    def reset(self, stream=None):
        state_reset(self.h, stream)

    def status(self, stream=None, check: bool = False):
        return state_sync_status(self.h, self.B, stream, check)

    def export(self, live: bool = False, stream=None):
        return state_export(self.h, self.B, self.k, self.trie.info["n_edges"], live, stream)

    def close(self):
        if getattr(self, "h", None) is not None:
            state_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
