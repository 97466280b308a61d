"""Python binding of the gfx950 stable LSD radix sort library (``librs.so``).

The functions named ``rs_*`` mirror the C ABI in ``include/rs.h`` one for one:
they only turn tensors or integers into device pointers and sizes, call the
library and raise :class:`RsError` on a status other than ``RS_OK``.  Every
step of the computation runs in the library's HIP kernels.  The convenience
wrappers below them (``sort_keys_u32`` ...) allocate outputs and temporary
storage with torch on the tensors' device and launch on torch's current
stream; torch provides memory and streams only.

The wrappers on rows of scores (``route_topk``, ``route_topk_grad``,
``group_choices``, ``token_logprobs``, ``token_logprobs_grad``) take `stream`, a
torch stream of the tensors' device or its address (0: the default stream; None:
the current one).  Outputs are allocated on that stream, as a torch operation
under it would, and what a call is given may be dropped at once; to order the
stream behind what makes the inputs and before what uses the outputs is the
caller's.  `temp`, a contiguous tensor of at least the size query's bytes on the
tensors' device, is used by one call at a time.  None of them is part of torch's
autograd: outputs have no gradient function, whatever the inputs require, and
``route_topk_grad`` and ``token_logprobs_grad`` compute the gradients.

Loading fails with an error when ``librs.so`` has not been built; there is no
fallback implementation.  ``use_library(path)`` binds the functions to another
build of the same sources (the tests use it for the build with the ballot rank
forced on every path, ``librs_ballot.so``).
"""
import collections
import ctypes
import os

__all__ = [
    "RsError", "RS_OK", "RS_ERR_INVALID_VALUE", "RS_ERR_UNSUPPORTED_SIZE",
    "RS_ERR_TEMP_TOO_SMALL", "RS_ERR_OVERLAP", "RS_ERR_MISALIGNED", "RS_ERR_HIP",
    "RS_KEY_U32", "RS_KEY_I32", "RS_KEY_F32", "RS_KEY_U64", "RS_KEY_I64", "RS_KEY_F64",
    "rs_sort_keys_u32", "rs_sort_pairs_u32", "rs_sort_pairs_f32", "rs_sort_keys", "rs_sort_pairs",
    "rs_sort_two_keys_u32", "rs_digit_counts", "rs_compact_positive_f32",
    "rs_compact_positive_f32_noalloc", "rs_exclusive_scan_u32", "rs_inclusive_scan_u32",
    "rs_select", "rs_partition", "RS_OP_LT", "RS_OP_LE", "RS_OP_GT", "RS_OP_GE", "RS_OP_EQ",
    "RS_OP_NE", "RS_NO_TEMP", "RS_ELEM_F32", "RS_ELEM_F16", "RS_ELEM_BF16", "RS_SCORE_SOFTMAX",
    "RS_SCORE_SIGMOID", "rs_route_topk", "rs_route_topk_grad", "rs_group_choices",
    "rs_token_logprobs", "rs_token_logprobs_grad", "route_topk", "route_topk_grad",
    "group_choices", "token_logprobs", "token_logprobs_grad", "TokenLogprobs", "rs_bitonic_tile", "rs_status_string", "rs_timing_enable", "rs_timing_collect",
    "exclusive_scan_u32", "inclusive_scan_u32", "select", "partition",
    "sort_keys_u32", "sort_pairs_u32", "sort_pairs_f32", "sort_keys", "sort_pairs",
    "sort_two_keys_u32", "digit_counts", "compact_positive_f32", "bitonic_tile",
    "library_path", "use_library", "EXPORTED_SYMBOLS", "KERNEL_NAMES",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "librs.so")

RS_OK = 0
RS_ERR_INVALID_VALUE = 1
RS_ERR_UNSUPPORTED_SIZE = 2
RS_ERR_TEMP_TOO_SMALL = 3
RS_ERR_OVERLAP = 4
RS_ERR_MISALIGNED = 5
RS_ERR_HIP = 6

RS_KEY_U32 = 0
RS_KEY_I32 = 1
RS_KEY_F32 = 2
RS_KEY_U64 = 3
RS_KEY_I64 = 4
RS_KEY_F64 = 5

RS_KERNEL_UPSWEEP = 0
RS_KERNEL_ONESWEEP = 1
RS_KERNEL_SORT_INIT = 2
RS_KERNEL_COMPACT_INIT = 3
RS_KERNEL_COMPACT = 4
RS_KERNEL_BITONIC = 5
RS_KERNEL_COPY = 6
RS_KERNEL_TILE_SORT = 7
RS_KERNEL_BUCKET_SORT = 8
KERNEL_NAMES = {0: "upsweep", 1: "onesweep", 2: "sort_init", 3: "compact_init",
                4: "compact", 5: "bitonic", 6: "copy", 7: "tile_sort", 8: "bucket_sort",
                9: "scan_init", 10: "scan", 11: "select_init", 12: "select_count", 13: "select",
                14: "route", 15: "route_grad", 16: "group_count", 17: "group_scan",
                18: "group_place", 19: "logprobs", 20: "logprobs_join", 21: "logprobs_grad"}

RS_NO_TEMP = 16
RS_ELEM_F32, RS_ELEM_F16, RS_ELEM_BF16 = range(3)
RS_SCORE_SOFTMAX, RS_SCORE_SIGMOID = range(2)
_SCORES = {"softmax": RS_SCORE_SOFTMAX, "sigmoid": RS_SCORE_SIGMOID}

RS_OP_LT, RS_OP_LE, RS_OP_GT, RS_OP_GE, RS_OP_EQ, RS_OP_NE = range(6)
_OPS = {"<": RS_OP_LT, "<=": RS_OP_LE, ">": RS_OP_GT, ">=": RS_OP_GE, "==": RS_OP_EQ,
        "!=": RS_OP_NE}

EXPORTED_SYMBOLS = ["rs_sort_keys_u32", "rs_sort_pairs_u32", "rs_sort_pairs_f32",
                    "rs_sort_keys", "rs_sort_pairs", "rs_sort_two_keys_u32", "rs_digit_counts",
                    "rs_compact_positive_f32", "rs_compact_positive_f32_noalloc",
                    "rs_exclusive_scan_u32", "rs_inclusive_scan_u32", "rs_select", "rs_partition",
                    "rs_bitonic_tile", "rs_route_topk", "rs_route_topk_grad", "rs_group_choices",
                    "rs_token_logprobs", "rs_token_logprobs_grad", "rs_status_string",
                    "rs_timing_enable", "rs_timing_collect"]

_lib = None
_lib_path = _LIB_PATH


class RsError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: %s" % (what, rs_status_string(status)))


def library_path():
    return _lib_path


def use_library(path=None):
    """Bind every function to the library at `path` (None: the default
    librs.so); returns the previous path."""
    global _lib, _lib_path
    prev = _lib_path
    _lib_path = _LIB_PATH if path is None else os.path.abspath(path)
    _lib = None
    return prev


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_lib_path):
        raise RuntimeError("%s is not built; run "
                           "`python -m sorting_lsd_radix_amd.build` or "
                           "`python -c 'import __graft_entry__ as g; g.build()'`" % _lib_path)
    lib = ctypes.CDLL(_lib_path)
    vp, u64, i32, u32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint32
    szp = ctypes.POINTER(ctypes.c_size_t)
    lib.rs_sort_keys_u32.argtypes = [vp, vp, u64, i32, i32, vp, szp, vp]
    lib.rs_sort_pairs_u32.argtypes = [vp, vp, vp, vp, u64, i32, i32, vp, szp, vp]
    lib.rs_sort_pairs_f32.argtypes = [vp, vp, vp, vp, u64, i32, i32, vp, szp, vp]
    lib.rs_sort_keys.argtypes = [i32, i32, vp, vp, u64, i32, i32, vp, szp, vp]
    lib.rs_sort_pairs.argtypes = [i32, i32, vp, vp, vp, vp, u64, i32, i32, vp, szp, vp]
    lib.rs_sort_two_keys_u32.argtypes = [vp, vp, vp, vp, vp, vp, u64, vp, szp, vp]
    lib.rs_digit_counts.argtypes = [i32, i32, vp, u64, i32, i32, vp, vp]
    lib.rs_compact_positive_f32.argtypes = [vp, vp, vp, u64, vp, szp, vp]
    lib.rs_compact_positive_f32_noalloc.argtypes = [vp, vp, vp, u64, vp]
    lib.rs_compact_positive_f32_noalloc.restype = i32
    for f in (lib.rs_exclusive_scan_u32, lib.rs_inclusive_scan_u32):
        f.argtypes = [vp, vp, u64, vp, szp, vp]
        f.restype = i32
    for f in (lib.rs_select, lib.rs_partition):
        f.argtypes = [i32, i32, u32, vp, vp, vp, vp, vp, u64, vp, szp, vp]
        f.restype = i32
    lib.rs_bitonic_tile.argtypes = [vp, vp, u64, u32, i32, i32, vp]
    for f in (lib.rs_sort_keys_u32, lib.rs_sort_pairs_u32, lib.rs_sort_pairs_f32, lib.rs_sort_keys,
              lib.rs_sort_pairs, lib.rs_sort_two_keys_u32, lib.rs_digit_counts,
              lib.rs_compact_positive_f32, lib.rs_bitonic_tile):
        f.restype = i32
    f32 = ctypes.c_float
    lib.rs_route_topk.argtypes = [i32, vp, u64, vp, u64, u32, u32, i32, u32, u32, u32, i32, f32,
                                  vp, vp, vp]
    lib.rs_route_topk_grad.argtypes = [i32, vp, u64, vp, vp, vp, u64, u32, u32, i32, i32, f32, vp,
                                       u64, vp]
    lib.rs_group_choices.argtypes = [vp, u64, u32, u32, vp, vp, vp, vp, vp, szp, vp]
    lib.rs_token_logprobs.argtypes = [i32, vp, u64, vp, u64, u32, f32, u32, vp, vp, vp, vp, vp, vp,
                                      vp, vp, szp, vp]
    lib.rs_token_logprobs_grad.argtypes = [i32, vp, u64, vp, vp, vp, u64, u32, f32, vp, vp, vp, vp,
                                           u64, vp]
    for f in (lib.rs_route_topk, lib.rs_route_topk_grad, lib.rs_group_choices,
              lib.rs_token_logprobs, lib.rs_token_logprobs_grad):
        f.restype = i32
    lib.rs_status_string.argtypes = [i32]
    lib.rs_status_string.restype = ctypes.c_char_p
    lib.rs_timing_enable.argtypes = [i32]
    lib.rs_timing_enable.restype = i32
    lib.rs_timing_collect.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float),
                                      i32]
    lib.rs_timing_collect.restype = i32
    _lib = lib
    return lib


# --- argument marshalling ------------------------------------------------------------

def _ptr(x):
    """Device pointer of a tensor, or an integer address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(what, status):
    if status != RS_OK:
        raise RsError(status, what)


def rs_status_string(status):
    return _load().rs_status_string(int(status)).decode()


def _sort_call(fn, what, args, n, begin_bit, end_bit, d_temp, temp_bytes, stream):
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = fn(*[_ptr(a) for a in args], int(n), int(begin_bit), int(end_bit), _ptr(d_temp),
            ctypes.byref(size), _stream(stream) if d_temp is not None else None)
    _call(what, st)
    return size.value if d_temp is None else None


def rs_sort_keys_u32(keys_in, keys_out, n, begin_bit, end_bit, d_temp, temp_bytes, stream=None):
    """C: rs_sort_keys_u32.  With d_temp None, returns the temp size."""
    return _sort_call(_load().rs_sort_keys_u32, "rs_sort_keys_u32", (keys_in, keys_out), n,
                      begin_bit, end_bit, d_temp, temp_bytes, stream)


def rs_sort_pairs_u32(keys_in, keys_out, vals_in, vals_out, n, begin_bit, end_bit, d_temp,
                      temp_bytes, stream=None):
    """C: rs_sort_pairs_u32.  With d_temp None, returns the temp size."""
    return _sort_call(_load().rs_sort_pairs_u32, "rs_sort_pairs_u32",
                      (keys_in, keys_out, vals_in, vals_out), n, begin_bit, end_bit, d_temp,
                      temp_bytes, stream)


def rs_sort_pairs_f32(keys_in, keys_out, vals_in, vals_out, n, begin_bit, end_bit, d_temp,
                      temp_bytes, stream=None):
    """C: rs_sort_pairs_f32.  With d_temp None, returns the temp size."""
    return _sort_call(_load().rs_sort_pairs_f32, "rs_sort_pairs_f32",
                      (keys_in, keys_out, vals_in, vals_out), n, begin_bit, end_bit, d_temp,
                      temp_bytes, stream)


def rs_sort_keys(key_type, descending, keys_in, keys_out, n, begin_bit, end_bit, d_temp,
                 temp_bytes, stream=None):
    """C: rs_sort_keys.  With d_temp None, returns the temp size."""
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = _load().rs_sort_keys(int(key_type), int(bool(descending)), _ptr(keys_in), _ptr(keys_out),
                              int(n), int(begin_bit), int(end_bit), _ptr(d_temp),
                              ctypes.byref(size), _stream(stream) if d_temp is not None else None)
    _call("rs_sort_keys", st)
    return size.value if d_temp is None else None


def rs_sort_pairs(key_type, descending, keys_in, keys_out, vals_in, vals_out, n, begin_bit,
                  end_bit, d_temp, temp_bytes, stream=None):
    """C: rs_sort_pairs.  With d_temp None, returns the temp size."""
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = _load().rs_sort_pairs(int(key_type), int(bool(descending)), _ptr(keys_in), _ptr(keys_out),
                               _ptr(vals_in), _ptr(vals_out), int(n), int(begin_bit), int(end_bit),
                               _ptr(d_temp), ctypes.byref(size),
                               _stream(stream) if d_temp is not None else None)
    _call("rs_sort_pairs", st)
    return size.value if d_temp is None else None


def rs_sort_two_keys_u32(major_in, minor_in, major_out, minor_out, vals_in, vals_out, n, d_temp,
                         temp_bytes, stream=None):
    """C: rs_sort_two_keys_u32.  With d_temp None, returns the temp size."""
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = _load().rs_sort_two_keys_u32(_ptr(major_in), _ptr(minor_in), _ptr(major_out),
                                      _ptr(minor_out), _ptr(vals_in), _ptr(vals_out), int(n),
                                      _ptr(d_temp), ctypes.byref(size),
                                      _stream(stream) if d_temp is not None else None)
    _call("rs_sort_two_keys_u32", st)
    return size.value if d_temp is None else None


def rs_digit_counts(key_type, descending, keys, n, begin_bit, end_bit, d_counts, stream=None):
    """C: rs_digit_counts."""
    st = _load().rs_digit_counts(int(key_type), int(bool(descending)), _ptr(keys), int(n),
                                 int(begin_bit), int(end_bit), _ptr(d_counts), _stream(stream))
    _call("rs_digit_counts", st)


def rs_compact_positive_f32(x_in, x_out, d_count, n, d_temp, temp_bytes, stream=None):
    """C: rs_compact_positive_f32.  With d_temp None, returns the temp size."""
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = _load().rs_compact_positive_f32(_ptr(x_in), _ptr(x_out), _ptr(d_count), int(n),
                                         _ptr(d_temp), ctypes.byref(size),
                                         _stream(stream) if d_temp is not None else None)
    _call("rs_compact_positive_f32", st)
    return size.value if d_temp is None else None


def rs_compact_positive_f32_noalloc(x_in, x_out, d_count, n, stream=None):
    """C: rs_compact_positive_f32_noalloc (the library's static scratch, no temp)."""
    st = _load().rs_compact_positive_f32_noalloc(_ptr(x_in), _ptr(x_out), _ptr(d_count), int(n),
                                                 _stream(stream))
    _call("rs_compact_positive_f32_noalloc", st)


def _scan_call(fn, what, x_in, x_out, n, d_temp, temp_bytes, stream):
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = fn(_ptr(x_in), _ptr(x_out), int(n), _ptr(d_temp), ctypes.byref(size),
            _stream(stream) if d_temp is not None else None)
    _call(what, st)
    return size.value if d_temp is None else None


def rs_exclusive_scan_u32(x_in, x_out, n, d_temp, temp_bytes, stream=None):
    """C: rs_exclusive_scan_u32.  With d_temp None, returns the temp size."""
    return _scan_call(_load().rs_exclusive_scan_u32, "rs_exclusive_scan_u32", x_in, x_out, n,
                      d_temp, temp_bytes, stream)


def rs_inclusive_scan_u32(x_in, x_out, n, d_temp, temp_bytes, stream=None):
    """C: rs_inclusive_scan_u32.  With d_temp None, returns the temp size."""
    return _scan_call(_load().rs_inclusive_scan_u32, "rs_inclusive_scan_u32", x_in, x_out, n,
                      d_temp, temp_bytes, stream)


def _select_call(fn, what, key_type, op, threshold_bits, x_in, x_out, vals_in, vals_out, d_count,
                 n, d_temp, temp_bytes, stream):
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = fn(int(key_type), int(op), int(threshold_bits) & 0xFFFFFFFF, _ptr(x_in), _ptr(x_out),
            _ptr(vals_in), _ptr(vals_out), _ptr(d_count), int(n), _ptr(d_temp), ctypes.byref(size),
            _stream(stream) if d_temp is not None else None)
    _call(what, st)
    return size.value if d_temp is None else None


def rs_select(key_type, op, threshold_bits, x_in, x_out, vals_in, vals_out, d_count, n, d_temp,
              temp_bytes, stream=None):
    """C: rs_select.  With d_temp None, returns the temp size."""
    return _select_call(_load().rs_select, "rs_select", key_type, op, threshold_bits, x_in, x_out,
                        vals_in, vals_out, d_count, n, d_temp, temp_bytes, stream)


def rs_partition(key_type, op, threshold_bits, x_in, x_out, vals_in, vals_out, d_count, n, d_temp,
                 temp_bytes, stream=None):
    """C: rs_partition.  With d_temp None, returns the temp size."""
    return _select_call(_load().rs_partition, "rs_partition", key_type, op, threshold_bits, x_in,
                        x_out, vals_in, vals_out, d_count, n, d_temp, temp_bytes, stream)


def rs_bitonic_tile(keys_in, keys_out, n, tile, begin_bit, end_bit, stream=None):
    """C: rs_bitonic_tile."""
    st = _load().rs_bitonic_tile(_ptr(keys_in), _ptr(keys_out), int(n), int(tile),
                                 int(begin_bit), int(end_bit), _stream(stream))
    _call("rs_bitonic_tile", st)


def _check_counts(what, counts):
    """`counts`, or-ed, are numbers that the C interface takes in 32 bits: past them they would come
    out as others."""
    if counts >> 32:   # of a negative one, -1
        raise RsError(RS_ERR_UNSUPPORTED_SIZE, what)


def rs_route_topk(elem_type, scores, row_stride, bias, rows, experts, top_k, score_fn, groups,
                  top_groups, group_best, renormalize, scale, ids, weights, stream=None):
    """C: rs_route_topk."""
    _check_counts("rs_route_topk", experts | top_k | groups | top_groups | group_best)
    st = _load().rs_route_topk(int(elem_type), _ptr(scores), int(row_stride), _ptr(bias), int(rows),
                               int(experts), int(top_k), int(score_fn), int(groups),
                               int(top_groups), int(group_best), int(bool(renormalize)),
                               float(scale), _ptr(ids), _ptr(weights), _stream(stream))
    _call("rs_route_topk", st)


def rs_route_topk_grad(elem_type, scores, row_stride, ids, weights, dweights, rows, experts, top_k,
                       score_fn, renormalize, scale, dscores, dscores_stride, stream=None):
    """C: rs_route_topk_grad."""
    _check_counts("rs_route_topk_grad", experts | top_k)
    st = _load().rs_route_topk_grad(int(elem_type), _ptr(scores), int(row_stride), _ptr(ids),
                                    _ptr(weights), _ptr(dweights), int(rows), int(experts),
                                    int(top_k), int(score_fn), int(bool(renormalize)),
                                    float(scale), _ptr(dscores), int(dscores_stride),
                                    _stream(stream))
    _call("rs_route_topk_grad", st)


def rs_group_choices(ids, n, experts, align, order, place, starts, counts, d_temp, temp_bytes,
                     stream=None):
    """C: rs_group_choices.  With d_temp None, returns the temp size."""
    _check_counts("rs_group_choices", experts | align)
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = _load().rs_group_choices(_ptr(ids), int(n), int(experts), int(align), _ptr(order),
                                  _ptr(place), _ptr(starts), _ptr(counts), _ptr(d_temp),
                                  ctypes.byref(size),
                                  _stream(stream) if d_temp is not None else None)
    _call("rs_group_choices", st)
    return size.value if d_temp is None else None


def rs_token_logprobs(elem_type, logits, row_stride, targets, rows, vocab, scale, top_k, stats, lse,
                      entropy, logprob, rank, top_ids, top_logprobs, d_temp, temp_bytes,
                      stream=None):
    """C: rs_token_logprobs.  With d_temp None, returns the temp size."""
    _check_counts("rs_token_logprobs", vocab | top_k)
    size = ctypes.c_size_t(0 if temp_bytes is None else int(temp_bytes))
    st = _load().rs_token_logprobs(int(elem_type), _ptr(logits), int(row_stride), _ptr(targets),
                                   int(rows), int(vocab), float(scale), int(top_k), _ptr(stats),
                                   _ptr(lse), _ptr(entropy), _ptr(logprob), _ptr(rank),
                                   _ptr(top_ids), _ptr(top_logprobs), _ptr(d_temp),
                                   ctypes.byref(size),
                                   _stream(stream) if d_temp is not None else None)
    _call("rs_token_logprobs", st)
    return size.value if d_temp is None else None


def rs_token_logprobs_grad(elem_type, logits, row_stride, targets, stats, entropy, rows, vocab,
                           scale, dlogprob, dentropy, dlse, dlogits, dlogits_stride, stream=None):
    """C: rs_token_logprobs_grad."""
    _check_counts("rs_token_logprobs_grad", vocab)
    st = _load().rs_token_logprobs_grad(int(elem_type), _ptr(logits), int(row_stride),
                                        _ptr(targets), _ptr(stats), _ptr(entropy), int(rows),
                                        int(vocab), float(scale), _ptr(dlogprob), _ptr(dentropy),
                                        _ptr(dlse), _ptr(dlogits), int(dlogits_stride),
                                        _stream(stream))
    _call("rs_token_logprobs_grad", st)


def rs_timing_enable(enable):
    _call("rs_timing_enable", _load().rs_timing_enable(1 if enable else 0))


def rs_timing_collect():
    """[(kernel name, milliseconds), ...] of the launches recorded so far."""
    lib = _load()
    held = lib.rs_timing_collect(None, None, 0)
    if held < 0:
        raise RsError(RS_ERR_HIP, "rs_timing_collect")
    ids = (ctypes.c_int * max(held, 1))()
    ms = (ctypes.c_float * max(held, 1))()
    got = lib.rs_timing_collect(ids, ms, held)
    if got < 0:
        raise RsError(RS_ERR_HIP, "rs_timing_collect")
    return [(KERNEL_NAMES.get(ids[i], str(ids[i])), float(ms[i])) for i in range(min(got, held))]


# --- convenience wrappers (torch allocates; the library computes) -------------------

def _temp(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _check_tensor(t, dtype, name):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise TypeError("%s must be a contiguous CUDA tensor of %s" % (name, dtype))


def sort_keys_u32(keys, begin_bit=0, end_bit=32, out=None, temp=None, stream=None):
    """Stable sort of a uint32 tensor by bits [begin_bit, end_bit); returns the sorted keys."""
    import torch
    _check_tensor(keys, torch.uint32, "keys")
    n = keys.numel()
    out = torch.empty_like(keys) if out is None else out
    need = rs_sort_keys_u32(None, None, n, begin_bit, end_bit, None, 0)
    temp = _temp(need, keys.device) if temp is None else temp
    rs_sort_keys_u32(keys, out, n, begin_bit, end_bit, temp, temp.numel(), stream)
    return out


def sort_pairs_u32(keys, vals, begin_bit=0, end_bit=32, keys_out=None, vals_out=None, temp=None,
                   stream=None):
    """Stable sort of uint32 (key, value) tensors; returns (keys_out, vals_out)."""
    import torch
    _check_tensor(keys, torch.uint32, "keys")
    _check_tensor(vals, torch.uint32, "vals")
    n = keys.numel()
    keys_out = torch.empty_like(keys) if keys_out is None else keys_out
    vals_out = torch.empty_like(vals) if vals_out is None else vals_out
    need = rs_sort_pairs_u32(None, None, None, None, n, begin_bit, end_bit, None, 0)
    temp = _temp(need, keys.device) if temp is None else temp
    rs_sort_pairs_u32(keys, keys_out, vals, vals_out, n, begin_bit, end_bit, temp, temp.numel(),
                      stream)
    return keys_out, vals_out


def sort_pairs_f32(keys, vals, begin_bit=0, end_bit=32, keys_out=None, vals_out=None, temp=None,
                   stream=None):
    """Stable IEEE-total-order sort of float32 keys with uint32 values."""
    import torch
    _check_tensor(keys, torch.float32, "keys")
    _check_tensor(vals, torch.uint32, "vals")
    n = keys.numel()
    keys_out = torch.empty_like(keys) if keys_out is None else keys_out
    vals_out = torch.empty_like(vals) if vals_out is None else vals_out
    need = rs_sort_pairs_f32(None, None, None, None, n, begin_bit, end_bit, None, 0)
    temp = _temp(need, keys.device) if temp is None else temp
    rs_sort_pairs_f32(keys, keys_out, vals, vals_out, n, begin_bit, end_bit, temp, temp.numel(),
                      stream)
    return keys_out, vals_out


def _key_type(t):
    import torch
    table = {torch.uint32: RS_KEY_U32, torch.int32: RS_KEY_I32, torch.float32: RS_KEY_F32,
             torch.uint64: RS_KEY_U64, torch.int64: RS_KEY_I64, torch.float64: RS_KEY_F64}
    if not t.is_cuda or not t.is_contiguous() or t.dtype not in table:
        raise TypeError("keys must be a contiguous CUDA tensor of uint32, int32, float32, "
                        "uint64, int64 or float64")
    return table[t.dtype], t.element_size() * 8


def sort_keys(keys, descending=False, begin_bit=0, end_bit=None, out=None, temp=None, stream=None):
    """Stable sort of a typed key tensor (ascending or descending); returns the sorted keys."""
    kt, width = _key_type(keys)
    end_bit = width if end_bit is None else end_bit
    n = keys.numel()
    out = keys.new_empty(keys.shape) if out is None else out
    need = rs_sort_keys(kt, descending, None, None, n, begin_bit, end_bit, None, 0)
    temp = _temp(need, keys.device) if temp is None else temp
    rs_sort_keys(kt, descending, keys, out, n, begin_bit, end_bit, temp, temp.numel(), stream)
    return out


def sort_pairs(keys, vals, descending=False, begin_bit=0, end_bit=None, keys_out=None,
               vals_out=None, temp=None, stream=None):
    """Stable sort of typed keys with uint32 values; returns (keys_out, vals_out)."""
    import torch
    kt, width = _key_type(keys)
    _check_tensor(vals, torch.uint32, "vals")
    end_bit = width if end_bit is None else end_bit
    n = keys.numel()
    keys_out = keys.new_empty(keys.shape) if keys_out is None else keys_out
    vals_out = torch.empty_like(vals) if vals_out is None else vals_out
    need = rs_sort_pairs(kt, descending, None, None, None, None, n, begin_bit, end_bit, None, 0)
    temp = _temp(need, keys.device) if temp is None else temp
    rs_sort_pairs(kt, descending, keys, keys_out, vals, vals_out, n, begin_bit, end_bit, temp,
                  temp.numel(), stream)
    return keys_out, vals_out


def sort_two_keys_u32(major, minor, vals=None, temp=None, stream=None):
    """Stable sort by (major, minor) uint32 keys; returns (major, minor) or (major, minor, vals)."""
    import torch
    _check_tensor(major, torch.uint32, "major")
    _check_tensor(minor, torch.uint32, "minor")
    n = major.numel()
    mo, no = torch.empty_like(major), torch.empty_like(minor)
    vo = None
    if vals is not None:
        _check_tensor(vals, torch.uint32, "vals")
        vo = torch.empty_like(vals)
    need = rs_sort_two_keys_u32(None, None, None, None, None, None, n, None, 0)
    temp = _temp(need, major.device) if temp is None else temp
    rs_sort_two_keys_u32(major, minor, mo, no, vals, vo, n, temp, temp.numel(), stream)
    return (mo, no) if vals is None else (mo, no, vo)


def digit_counts(keys, descending=False, begin_bit=0, end_bit=None, stream=None):
    """Per-pass 8-bit digit counts of a typed key tensor: uint32 tensor [passes, 256]."""
    import torch
    kt, width = _key_type(keys)
    end_bit = width if end_bit is None else end_bit
    passes = (end_bit - begin_bit + 7) // 8
    counts = torch.zeros((max(passes, 1), 256), dtype=torch.uint32, device=keys.device)
    rs_digit_counts(kt, descending, keys, keys.numel(), begin_bit, end_bit, counts, stream)
    return counts[:passes]


def _scan_tensor(fn, x, out, temp, stream):
    import torch
    _check_tensor(x, torch.uint32, "x")
    out = torch.empty_like(x) if out is None else out
    need = fn(None, None, x.numel(), None, 0)
    temp = _temp(need, x.device) if temp is None else temp
    fn(x, out, x.numel(), temp, temp.numel(), stream)
    return out


def exclusive_scan_u32(x, out=None, temp=None, stream=None):
    """Exclusive prefix sums of a uint32 tensor, modulo 2^32."""
    return _scan_tensor(rs_exclusive_scan_u32, x, out, temp, stream)


def inclusive_scan_u32(x, out=None, temp=None, stream=None):
    """Inclusive prefix sums of a uint32 tensor, modulo 2^32."""
    return _scan_tensor(rs_inclusive_scan_u32, x, out, temp, stream)


def _threshold_bits(x, threshold):
    import numpy as np
    dt = {RS_KEY_U32: np.uint32, RS_KEY_I32: np.int32, RS_KEY_F32: np.float32}
    kt, _ = _key_type(x)
    if kt not in dt:
        raise TypeError("select and partition take uint32, int32 or float32 elements")
    return kt, int(np.array([threshold], dt[kt]).view(np.uint32)[0])


def _select_tensor(fn, x, op, threshold, vals, temp, stream):
    import torch
    kt, bits = _threshold_bits(x, threshold)
    out = torch.empty_like(x)
    vo = None
    if vals is not None:
        _check_tensor(vals, torch.uint32, "vals")
        vo = torch.empty_like(vals)
    count = torch.empty(1, dtype=torch.uint32, device=x.device)
    need = fn(kt, _OPS[op], bits, None, None, vals, vo, None, x.numel(), None, 0)
    temp = _temp(need, x.device) if temp is None else temp
    fn(kt, _OPS[op], bits, x, out, vals, vo, count, x.numel(), temp, temp.numel(), stream)
    return (out, count) if vals is None else (out, vo, count)


def select(x, op, threshold, vals=None, temp=None, stream=None):
    """Elements with `x op threshold` (op in <, <=, >, >=, ==, !=) in order at the front of
    the output; returns (out, count) or (out, vals_out, count); count is a 1-element tensor."""
    return _select_tensor(rs_select, x, op, threshold, vals, temp, stream)


def partition(x, op, threshold, vals=None, temp=None, stream=None):
    """Stable partition: kept elements in order, then the rest in order."""
    return _select_tensor(rs_partition, x, op, threshold, vals, temp, stream)


def compact_positive_f32(x, out=None, count=None, temp=None, stream=None):
    """(out, count): x > 0 kept in order at the front, +0.0 after; count is a 1-element tensor."""
    import torch
    _check_tensor(x, torch.float32, "x")
    n = x.numel()
    out = torch.empty_like(x) if out is None else out
    count = torch.empty(1, dtype=torch.uint32, device=x.device) if count is None else count
    need = rs_compact_positive_f32(None, None, None, n, None, 0)
    temp = _temp(need, x.device) if temp is None else temp
    rs_compact_positive_f32(x, out, count, n, temp, temp.numel(), stream)
    return out, count


def bitonic_tile(keys, tile, begin_bit=0, end_bit=32, out=None, stream=None):
    """Each run of `tile` (<= 1024) keys sorted on its own, stably."""
    import torch
    _check_tensor(keys, torch.uint32, "keys")
    out = torch.empty_like(keys) if out is None else out
    rs_bitonic_tile(keys, out, keys.numel(), tile, begin_bit, end_bit, stream)
    return out


# --- rows of scores -------------------------------------------------------------------
#
# Small calls of these are as long as the host takes to make them: the wrappers look torch's
# types up once, allocate with as few calls as they can and hand plain numbers to the library.

_torch = None
_ELEMS = {}
_INTS = ()


def _load_torch():
    global _torch, _INTS
    if _torch is None:
        import torch
        _ELEMS.update({torch.float32: RS_ELEM_F32, torch.float16: RS_ELEM_F16,
                       torch.bfloat16: RS_ELEM_BF16})
        _INTS = (torch.int32, torch.uint32)
        _torch = torch
    return _torch


def _rows(t, name, dtype=None):
    """(elem_type, rows, columns, row stride) of a matrix whose rows are dense."""
    shape = t.shape
    if not t.is_cuda or len(shape) != 2 or t.dtype not in _ELEMS or \
            (t.stride(1) != 1 and shape[1] > 1):
        raise TypeError("%s must be a 2-D CUDA tensor of float32, float16 or bfloat16 whose rows "
                        "are contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be of %s" % (name, dtype))
    return _ELEMS[t.dtype], shape[0], shape[1], t.stride(0)


def _check_like(t, name, shape, dtypes, index):
    """A contiguous CUDA tensor of `shape`, one of `dtypes`, on the device `index`; its address."""
    if t.dtype not in dtypes or t.shape != shape or not t.is_cuda or t.get_device() != index or \
            not t.is_contiguous():
        raise TypeError("%s must be a contiguous tensor of shape %s and %s on cuda:%d"
                        % (name, tuple(shape), " or ".join(str(d) for d in dtypes), index))
    return t.data_ptr()


def _check_out(out, name, rows, cols, dtype, index):
    """(address, row stride) of a matrix that a call writes."""
    _, orows, ocols, stride = _rows(out, "out", dtype)
    if (orows, ocols) != (rows, cols) or out.get_device() != index:
        raise TypeError("out must have the %s' shape and device" % name)
    return out.data_ptr(), stride


class _On:
    """A device as the current one and a stream (None: torch's current one) as torch's current
    one, so that what is allocated meanwhile belongs to that stream."""

    def __init__(self, index, stream):
        self._contexts = []
        if stream is not None and not isinstance(stream, int) and stream.device.index != index:
            raise TypeError("stream must be on cuda:%d, not %s" % (index, stream.device))
        if index != _torch.cuda.current_device():
            self._contexts.append(_torch.cuda.device(index))
        if stream is not None:
            if isinstance(stream, int):   # of address 0, the default stream's, torch would make a new one
                stream = _torch.cuda.ExternalStream(stream, device=index) if stream else \
                    _torch.cuda.default_stream(index)
            self._contexts.append(_torch.cuda.stream(stream))

    def __enter__(self):
        for c in self._contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._contexts):
            c.__exit__(*exc)


def _run_on(index, stream, call, given=()):
    """call(address of the stream) with the device and the stream as the current ones.  The memory
    of the tensors `given` to the call (Nones among them) is kept until a stream that is not the
    current one has run it: their owner may drop them at once."""
    if stream is None and index == _torch.cuda.current_device():
        return call(_torch._C._cuda_getCurrentRawStream(index))
    with _On(index, stream):
        result = call(_torch._C._cuda_getCurrentRawStream(index))
        if stream is not None:
            on = _torch.cuda.current_stream(index)
            for t in given:
                if t is not None:
                    t.record_stream(on)
        return result


# A size query that answers RS_NO_TEMP bytes or less says that the call does not touch its temp:
# it then gets this address, which no allocation has.
_NO_TEMP_ADDRESS = RS_NO_TEMP


def _temp_arg(temp, size, device):
    """(tensor to keep until the call, its address, its size) of a call's temp."""
    if temp is not None:
        if not temp.is_cuda or temp.device != device or not temp.is_contiguous():
            raise TypeError("temp must be a contiguous CUDA tensor on %s" % (device,))
        return temp, temp.data_ptr(), ctypes.c_size_t(temp.numel() * temp.element_size())
    if size.value <= RS_NO_TEMP:
        return None, _NO_TEMP_ADDRESS, size
    temp = _torch.empty(size.value, dtype=_torch.uint8, device=device)
    return temp, temp.data_ptr(), size


def route_topk(scores, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_best=1,
               renormalize=True, scale=1.0, stream=None):
    """The `top_k` experts of each row of router scores [rows, experts] (float32, float16 or
    bfloat16) and their weights: (ids int32 [rows, top_k], weights float32 [rows, top_k]).

    score: "softmax" (over all experts) or "sigmoid".  bias (float32 [experts]) is added to the
    probabilities for the choice only.  With groups > 1 the choice is among the experts of the
    top_groups groups whose group_best largest biased probabilities have the largest sum.
    Ties go to the lower expert.  The weights are scale * p, divided by the sum of the row's
    chosen p if renormalize.  No autograd: route_topk_grad gives the scores' gradient."""
    torch = _load_torch()
    et, rows, experts, stride = _rows(scores, "scores")
    _check_counts("rs_route_topk", experts | top_k | groups | top_groups | group_best)
    index = scores.get_device()
    at_bias = None if bias is None else _check_like(bias, "bias", (experts,), (torch.float32,), index)
    fn = _SCORES[score]
    lib = _load()

    def call(on):
        ids = torch.empty(rows, top_k, dtype=torch.int32, device=scores.device)
        weights = torch.empty(rows, top_k, dtype=torch.float32, device=scores.device)
        _call("rs_route_topk", lib.rs_route_topk(
            et, scores.data_ptr(), stride, at_bias, rows, experts, top_k, fn, groups, top_groups,
            group_best, 1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), on))
        return ids, weights

    return _run_on(index, stream, call, (scores, bias))


def route_topk_grad(scores, ids, weights, dweights, score="softmax", renormalize=True, scale=1.0,
                    out=None, stream=None):
    """Gradient for the scores of the weights that route_topk gave with these ids, score,
    renormalize and scale; dweights float32 [rows, top_k].  Returns dscores [rows, experts] of the
    scores' type (`out`, if given: a matrix whose rows are contiguous)."""
    torch = _load_torch()
    et, rows, experts, stride = _rows(scores, "scores")
    top_k = ids.shape[-1]
    _check_counts("rs_route_topk_grad", experts | top_k)
    index = scores.get_device()
    shape = (rows, top_k)
    f32 = (torch.float32,)
    args = (_check_like(ids, "ids", shape, _INTS, index),
            _check_like(weights, "weights", shape, f32, index),
            _check_like(dweights, "dweights", shape, f32, index))
    fn = _SCORES[score]
    lib = _load()

    def call(on):
        to = torch.empty(rows, experts, dtype=scores.dtype, device=scores.device) if out is None \
            else out
        at, ostride = _check_out(to, "scores", rows, experts, scores.dtype, index)
        _call("rs_route_topk_grad", lib.rs_route_topk_grad(
            et, scores.data_ptr(), stride, *args, rows, experts, top_k, fn,
            1 if renormalize else 0, scale, at, ostride, on))
        return to

    return _run_on(index, stream, call, (scores, ids, weights, dweights, out))


def group_choices(ids, experts, align=1, temp=None, stream=None):
    """The choices `ids` (int32 or uint32, any shape) ordered by expert, stably, each expert's
    segment padded to a multiple of `align`: (order, place, starts, counts), int32.  Contiguous ids
    that begin off a 16-byte boundary (some slices of a batch) are copied first.

    order [ids.numel() + experts * (align - 1)]: the flat index of the choice at each position,
    -1 in the padding and behind the last segment.  place (of the ids' shape): each choice's
    position, -1 where its id is not an expert (-1, or `experts` and above).  starts
    [experts + 1]: where each segment begins, and the length of all.  counts [experts]."""
    torch = _load_torch()
    shape = ids.shape
    index = ids.get_device() if ids.is_cuda else -1
    at = _check_like(ids, "ids", shape, _INTS, index)
    n = ids.numel()
    _check_counts("rs_group_choices", experts | align)
    lib = _load()
    size = ctypes.c_size_t(0)
    _call("rs_group_choices", lib.rs_group_choices(None, n, experts, align, None, None, None, None,
                                                   None, ctypes.byref(size), None))

    def call(on):
        dev, i32 = ids.device, torch.int32
        order = torch.empty(n + experts * (align - 1), dtype=i32, device=dev)
        place = torch.empty(shape, dtype=i32, device=dev)
        starts = torch.empty(experts + 1, dtype=i32, device=dev)
        counts = torch.empty(experts, dtype=i32, device=dev)
        _keep, work, have = _temp_arg(temp, size, dev)
        aligned = ids if at % 16 == 0 else ids.clone()   # the library reads from 16-byte boundaries on
        _call("rs_group_choices", lib.rs_group_choices(
            aligned.data_ptr(), n, experts, align, order.data_ptr(), place.data_ptr(), starts.data_ptr(),
            counts.data_ptr(), work, ctypes.byref(have), on))
        return order, place, starts, counts

    return _run_on(index, stream, call, (ids, temp))


TokenLogprobs = collections.namedtuple(
    "TokenLogprobs", "logprob entropy lse rank stats top_ids top_logprobs")


def token_logprobs(logits, targets=None, top_k=0, scale=1.0, temp=None, stream=None):
    """Log probabilities under softmax(scale * logits) of rows of logits [rows, vocab] (float32,
    float16 or bfloat16): a TokenLogprobs of

    logprob [rows] and rank [rows] (int32: logits before the target's, 0 for the first) of the
    targets (int32 or uint32 [rows]; -1 or `vocab` and above: none, logprob 0 and rank -1), both
    None without targets; entropy [rows] in nats; lse [rows], the log of the sum of exp; stats
    [rows, 2], the largest logit and the sum of exp relative to it, which token_logprobs_grad
    takes; top_ids (int32) and top_logprobs [rows, top_k], the largest logits in order, ties to
    the lower index, both None with top_k 0.  Floating outputs are float32; those of [rows] are
    views of one tensor.  No autograd: token_logprobs_grad gives the logits' gradient."""
    torch = _load_torch()
    et, rows, vocab, stride = _rows(logits, "logits")
    _check_counts("rs_token_logprobs", vocab | top_k)
    index = logits.get_device()
    at_targets = None if targets is None else _check_like(targets, "targets", (rows,), _INTS, index)
    lib = _load()
    size = ctypes.c_size_t(0)
    _call("rs_token_logprobs", lib.rs_token_logprobs(
        et, None, stride, None, rows, vocab, scale, top_k, None, None, None, None, None, None,
        None, None, ctypes.byref(size), None))
    wanted = targets is not None

    def call(on):
        dev, f32, i32 = logits.device, torch.float32, torch.int32
        stats = torch.empty(rows, 2, dtype=f32, device=dev)
        lse, entropy, *of_target = torch.empty(4 if wanted else 2, rows, dtype=f32,
                                               device=dev).unbind(0)
        logprob = rank = top_ids = top_logprobs = None
        if wanted:
            logprob, rank = of_target
            rank = rank.view(i32)
        if top_k:
            top_ids = torch.empty(rows, top_k, dtype=i32, device=dev)
            top_logprobs = torch.empty(rows, top_k, dtype=f32, device=dev)
        _keep, work, have = _temp_arg(temp, size, dev)
        _call("rs_token_logprobs", lib.rs_token_logprobs(
            et, logits.data_ptr(), stride, at_targets, rows, vocab, scale, top_k, stats.data_ptr(),
            lse.data_ptr(), entropy.data_ptr(), _ptr(logprob), _ptr(rank), _ptr(top_ids),
            _ptr(top_logprobs), work, ctypes.byref(have), on))
        return TokenLogprobs(logprob, entropy, lse, rank, stats, top_ids, top_logprobs)

    return _run_on(index, stream, call, (logits, targets, temp))


def token_logprobs_grad(logits, stats, targets=None, dlogprob=None, entropy=None, dentropy=None,
                        dlse=None, scale=1.0, out=None, stream=None):
    """Gradient for the logits of the sum over rows of dlogprob * logprob + dentropy * entropy +
    dlse * lse (each float32 [rows], or None), from the stats, and with dentropy the entropy, that
    token_logprobs gave.  Returns dlogits of the logits' type and shape (`out`, if given: a matrix
    whose rows are contiguous; it may be the logits themselves)."""
    torch = _load_torch()
    et, rows, vocab, stride = _rows(logits, "logits")
    _check_counts("rs_token_logprobs_grad", vocab)
    index = logits.get_device()
    f32 = (torch.float32,)
    at_stats = _check_like(stats, "stats", (rows, 2), f32, index)
    at_targets = None if targets is None else _check_like(targets, "targets", (rows,), _INTS, index)
    at_rows = [None if t is None else _check_like(t, name, (rows,), f32, index)
               for t, name in ((entropy, "entropy"), (dlogprob, "dlogprob"),
                               (dentropy, "dentropy"), (dlse, "dlse"))]
    lib = _load()

    def call(on):
        to = torch.empty(rows, vocab, dtype=logits.dtype, device=logits.device) if out is None \
            else out
        at, ostride = _check_out(to, "logits", rows, vocab, logits.dtype, index)
        _call("rs_token_logprobs_grad", lib.rs_token_logprobs_grad(
            et, logits.data_ptr(), stride, at_targets, at_stats, at_rows[0], rows, vocab, scale,
            *at_rows[1:], at, ostride, on))
        return to

    return _run_on(index, stream, call, (logits, stats, targets, entropy, dlogprob, dentropy, dlse, out))
