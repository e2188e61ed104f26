"""ctypes binding of libsketchssm.so (argument marshalling only).

The entry points keep the C names; those of the decode steps are
``sketchssm_read``, ``sketchssm_flush``, ``sketchssm_full_step`` and
``sketchssm_replay_step``.  Each of these takes the three argument structs (or pointers to them) and a HIP stream
handle, and returns the library's status code.  Loading fails loudly when the
library has not been built: there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsketchssm.so")

# constants of include/sketchssm.h
SKSSM_MAMBA2, SKSSM_GDN, SKSSM_KDA = 0, 1, 2
SKSSM_F32, SKSSM_BF16 = 0, 1
SKSSM_FLUSH_DUE, SKSSM_FLUSH_ALL, SKSSM_FLUSH_DUE_SCAN, SKSSM_FLUSH_CLOSE = 0, 1, 2, 3
SKSSM_COEF_FIXED, SKSSM_COEF_STATE = 0, 1
SKSSM_PULLBACK_SERIAL, SKSSM_PULLBACK_WY, SKSSM_PULLBACK_PROJ = 0, 1, 2
SKSSM_OK, SKSSM_EINVAL, SKSSM_EDIM, SKSSM_EDTYPE, SKSSM_EFLAG, SKSSM_ELAUNCH = 0, -1, -2, -3, -4, -5
SKSSM_ESCRATCH = -6
SKSSM_NOALLOC_SCRATCH_BYTES = 16777216
SKSSM_ERRBIT_COUNT, SKSSM_ERRBIT_GROUP, SKSSM_ERRBIT_SEQ, SKSSM_ERRBIT_SLOT, SKSSM_ERRBIT_LOGIT = 1, 2, 4, 8, 16
SKSSM_ACT_NONE, SKSSM_ACT_SILU, SKSSM_ACT_SIGMOID = 0, 1, 2

ENTRY_POINTS = ("sketchssm_read", "sketchssm_flush", "sketchssm_flush_seqs", "sketchssm_full_step",
                "sketchssm_replay_step", "sketchssm_workspace_bytes", "sketchssm_read_noalloc",
                "sketchssm_prefill", "sketchssm_prefill_workspace_bytes", "sketchssm_state_save",
                "sketchssm_state_load", "sketchssm_group_norm", "sketchssm_scan", "sketchssm_scan_workspace_bytes",
                "sketchssm_conv", "sketchssm_beam_select", "sketchssm_beam_workspace_bytes", "sketchssm_reorder",
                "sketchssm_version")


class sketchssm_layer(C.Structure):
    _fields_ = [("family", C.c_int32), ("batch", C.c_int32), ("heads", C.c_int32),
                ("qk_groups", C.c_int32), ("dk", C.c_int32), ("dv", C.c_int32),
                ("window", C.c_int32), ("act_dtype", C.c_int32), ("sketch_dtype", C.c_int32),
                ("rank_offsets_host", C.POINTER(C.c_int32)), ("coef_map", C.c_int32),
                ("coef_ridge", C.c_float), ("pullback", C.c_int32)]


class sketchssm_buffers(C.Structure):
    _fields_ = [("S", C.c_void_p), ("U", C.c_void_p), ("Pt", C.c_void_p), ("C", C.c_void_p),
                ("rank_offsets", C.c_void_p), ("ring_k", C.c_void_p), ("ring_v", C.c_void_p),
                ("ring_gate", C.c_void_p), ("ring_beta", C.c_void_p), ("count", C.c_void_p),
                ("A", C.c_void_p), ("err", C.c_void_p), ("work", C.c_void_p),
                ("Cstate", C.c_void_p), ("Scopy", C.c_void_p), ("ring_pc", C.c_void_p)]


class sketchssm_step(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("gate", C.c_void_p),
                ("beta", C.c_void_p), ("o", C.c_void_p)]


class sketchssm_prompts(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("gate", C.c_void_p),
                ("beta", C.c_void_p), ("o", C.c_void_p),
                ("q_stride", C.c_int64), ("k_stride", C.c_int64), ("v_stride", C.c_int64),
                ("gate_stride", C.c_int64), ("beta_stride", C.c_int64), ("o_stride", C.c_int64),
                ("tokens", C.c_int32), ("nseq", C.c_int32), ("seq_start", C.c_void_p),
                ("seqs", C.c_void_p), ("has_state", C.c_void_p), ("prime", C.c_int32),
                ("work", C.c_void_p), ("work_bytes", C.c_int64)]


class sketchssm_state_cache(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scale", C.c_void_p), ("slots", C.c_int32), ("bits", C.c_int32)]


class sketchssm_norm(C.Structure):
    _fields_ = [("x", C.c_void_p), ("gate", C.c_void_p), ("y", C.c_void_p), ("weight", C.c_void_p),
                ("bias", C.c_void_p), ("x_stride", C.c_int64), ("gate_stride", C.c_int64),
                ("y_stride", C.c_int64), ("rows", C.c_int64), ("first", C.c_void_p), ("end", C.c_void_p),
                ("groups", C.c_int32), ("width", C.c_int32),
                ("dtype", C.c_int32), ("group_weights", C.c_int32), ("centred", C.c_int32),
                ("activation", C.c_int32), ("gate_first", C.c_int32), ("eps", C.c_float)]


class sketchssm_scan_prompts(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("dt", C.c_void_p), ("o", C.c_void_p),
                ("q_stride", C.c_int64), ("k_stride", C.c_int64), ("v_stride", C.c_int64),
                ("dt_stride", C.c_int64), ("o_stride", C.c_int64),
                ("tokens", C.c_int32), ("nseq", C.c_int32), ("seq_start", C.c_void_p),
                ("seqs", C.c_void_p), ("has_state", C.c_void_p), ("prime", C.c_int32),
                ("work", C.c_void_p), ("work_bytes", C.c_int64)]


class sketchssm_conv_piece(C.Structure):
    _fields_ = [("y", C.c_void_p), ("y_stride", C.c_int64), ("channels", C.c_int32), ("unit", C.c_int32)]


class sketchssm_convolution(C.Structure):
    _fields_ = [("x", C.c_void_p), ("x_stride", C.c_int64), ("weight", C.c_void_p), ("bias", C.c_void_p),
                ("state", C.c_void_p), ("piece", sketchssm_conv_piece * 3), ("taps", C.c_int32),
                ("dtype", C.c_int32), ("activation", C.c_int32), ("eps", C.c_float), ("batch", C.c_int32),
                ("tokens", C.c_int32), ("nseq", C.c_int32), ("seq_start", C.c_void_p), ("seqs", C.c_void_p),
                ("has_state", C.c_void_p), ("err", C.c_void_p)]


class sketchssm_beams(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("stride", C.c_int64), ("scores", C.c_void_p), ("ended", C.c_void_p),
                ("new_scores", C.c_void_p), ("new_ended", C.c_void_p), ("parents", C.c_void_p),
                ("tokens", C.c_void_p), ("err", C.c_void_p), ("groups", C.c_int32), ("beams", C.c_int32),
                ("vocab", C.c_int32), ("dtype", C.c_int32), ("end_token", C.c_int32), ("work", C.c_void_p),
                ("work_bytes", C.c_int64)]


class sketchssm_rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("row_bytes", C.c_int64)]


_lib = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Load the HIP library; raises if it is missing (no CPU fallback)."""
    global _lib
    if _lib is None:
        # torch ships its own HIP runtime under the same soname as the
        # system's (libamdhip64.so.7); whichever is loaded first serves the
        # whole process.  Importing torch before the library keeps both on
        # torch's runtime, so that tensors allocated by torch are valid in
        # the library's launches whatever the caller imported first.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built: run __graft_entry__.build() "
                               "(or python ssm_decode_amd/build.py) first")
        lib = C.CDLL(path)
        L, Bf, St = C.POINTER(sketchssm_layer), C.POINTER(sketchssm_buffers), C.POINTER(sketchssm_step)
        for name in ("sketchssm_read", "sketchssm_read_noalloc", "sketchssm_full_step",
                     "sketchssm_replay_step"):
            fn = getattr(lib, name)
            fn.argtypes = [L, Bf, St, C.c_void_p]
            fn.restype = C.c_int
        lib.sketchssm_flush.argtypes = [L, Bf, St, C.c_int32, C.c_void_p]
        lib.sketchssm_flush.restype = C.c_int
        lib.sketchssm_flush_seqs.argtypes = [L, Bf, St, C.c_void_p, C.c_int32, C.c_void_p]
        lib.sketchssm_flush_seqs.restype = C.c_int
        lib.sketchssm_workspace_bytes.argtypes = [L]
        lib.sketchssm_workspace_bytes.restype = C.c_int64
        Ca, Pr = C.POINTER(sketchssm_state_cache), C.POINTER(sketchssm_prompts)
        lib.sketchssm_prefill.argtypes = [L, Bf, Pr, C.c_void_p]
        lib.sketchssm_prefill_workspace_bytes.argtypes = [L, C.c_int32, C.c_int32]
        lib.sketchssm_prefill_workspace_bytes.restype = C.c_int64
        lib.sketchssm_state_save.argtypes = [L, Bf, Ca, C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p]
        lib.sketchssm_state_load.argtypes = [L, Bf, Ca, C.c_void_p, C.c_void_p, C.c_int32, C.c_int32,
                                             C.c_void_p]
        lib.sketchssm_group_norm.argtypes = [C.POINTER(sketchssm_norm), C.c_void_p]
        Sc = C.POINTER(sketchssm_scan_prompts)
        lib.sketchssm_scan.argtypes = [L, Bf, Sc, C.c_void_p]
        lib.sketchssm_scan_workspace_bytes.argtypes = [L, C.c_int32, C.c_int32]
        lib.sketchssm_scan_workspace_bytes.restype = C.c_int64
        lib.sketchssm_conv.argtypes = [C.POINTER(sketchssm_convolution), C.c_void_p]
        lib.sketchssm_beam_select.argtypes = [C.POINTER(sketchssm_beams), C.c_void_p]
        lib.sketchssm_beam_workspace_bytes.argtypes = [C.c_int32] * 4
        lib.sketchssm_beam_workspace_bytes.restype = C.c_int64
        lib.sketchssm_reorder.argtypes = [L, Bf, C.POINTER(sketchssm_rows), C.c_int32, C.c_void_p, C.c_int32, C.c_void_p]
        for name in ("sketchssm_prefill", "sketchssm_state_save", "sketchssm_state_load",
                     "sketchssm_group_norm", "sketchssm_scan", "sketchssm_conv", "sketchssm_beam_select",
                     "sketchssm_reorder"):
            getattr(lib, name).restype = C.c_int
        lib.sketchssm_version.argtypes = []
        lib.sketchssm_version.restype = C.c_int
        _lib = lib
    return _lib


def _ref(x, ty):
    if x is None:
        return C.cast(None, C.POINTER(ty))
    if isinstance(x, ty):
        return C.byref(x)
    return x


def sketchssm_read(layer, bufs, step, stream=None) -> int:
    return load().sketchssm_read(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                 _ref(step, sketchssm_step), stream)


def sketchssm_read_noalloc(layer, bufs, step, stream=None) -> int:
    """sketchssm_read with the library's own scratch array as the workspace
    (bufs.work is ignored; nothing is allocated)."""
    return load().sketchssm_read_noalloc(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                         _ref(step, sketchssm_step), stream)


def sketchssm_flush(layer, bufs, step, flags, stream=None) -> int:
    return load().sketchssm_flush(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                  _ref(step, sketchssm_step), int(flags), stream)


def sketchssm_flush_seqs(layer, bufs, step, seqs, nseq, stream=None) -> int:
    """seqs: device address of nseq int32 sequence indices (or None with nseq = 0)."""
    return load().sketchssm_flush_seqs(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                       _ref(step, sketchssm_step), seqs, int(nseq), stream)


def sketchssm_full_step(layer, bufs, step, stream=None) -> int:
    return load().sketchssm_full_step(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                      _ref(step, sketchssm_step), stream)


def sketchssm_replay_step(layer, bufs, step, stream=None) -> int:
    return load().sketchssm_replay_step(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                        _ref(step, sketchssm_step), stream)


def sketchssm_workspace_bytes(layer) -> int:
    return load().sketchssm_workspace_bytes(_ref(layer, sketchssm_layer))


def sketchssm_prefill(layer, bufs, prompts, stream=None) -> int:
    return load().sketchssm_prefill(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                    _ref(prompts, sketchssm_prompts), stream)


def sketchssm_prefill_workspace_bytes(layer, tokens, nseq) -> int:
    return load().sketchssm_prefill_workspace_bytes(_ref(layer, sketchssm_layer), int(tokens), int(nseq))


def sketchssm_state_save(layer, bufs, cache, seqs, slots, n, stream=None) -> int:
    """seqs, slots: device addresses of n int32 indices (or None with n = 0)."""
    return load().sketchssm_state_save(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                       _ref(cache, sketchssm_state_cache), seqs, slots, int(n), stream)


def sketchssm_state_load(layer, bufs, cache, seqs, slots, n, prime, stream=None) -> int:
    return load().sketchssm_state_load(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                       _ref(cache, sketchssm_state_cache), seqs, slots, int(n), int(prime),
                                       stream)


def sketchssm_group_norm(norm, stream=None) -> int:
    return load().sketchssm_group_norm(_ref(norm, sketchssm_norm), stream)


def sketchssm_scan(layer, bufs, prompts, stream=None) -> int:
    return load().sketchssm_scan(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers),
                                 _ref(prompts, sketchssm_scan_prompts), stream)


def sketchssm_scan_workspace_bytes(layer, tokens, nseq) -> int:
    return load().sketchssm_scan_workspace_bytes(_ref(layer, sketchssm_layer), int(tokens), int(nseq))


def sketchssm_conv(conv, stream=None) -> int:
    return load().sketchssm_conv(_ref(conv, sketchssm_convolution), stream)


def sketchssm_beam_select(beams, stream=None) -> int:
    return load().sketchssm_beam_select(_ref(beams, sketchssm_beams), stream)


def sketchssm_beam_workspace_bytes(groups, beams, vocab, dtype) -> int:
    return load().sketchssm_beam_workspace_bytes(int(groups), int(beams), int(vocab), int(dtype))


def sketchssm_reorder(layer, bufs, extra, nextra, parents, beams, stream=None) -> int:
    """extra: an array of nextra sketchssm_rows (or None); parents: a device address."""
    return load().sketchssm_reorder(_ref(layer, sketchssm_layer), _ref(bufs, sketchssm_buffers), extra, int(nextra),
                                    parents, int(beams), stream)


def sketchssm_version() -> int:
    return load().sketchssm_version()
