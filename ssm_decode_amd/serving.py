"""What a serving loop runs around the decode steps, on torch tensors: prompts
through the gated delta rule (``Prompts``, ``DecodeLayer.prefill``), the
quantised state cache (``StateCache``, ``DecodeLayer.save_state`` and
``load_state``), the norm of the layers' outputs (``OutputNorm``,
``group_norm``), prompts through the selective state space scan
(``ScanPrompts``, ``DecodeLayer.scan``), the short convolution in front of the
layers (``ShortConv``, ``DecodeLayer.convolve``) and beams (``BeamSearch``,
``DecodeLayer.reorder``).  The tensors are checked here, where a wrong one would have
a kernel read what it must not; the work runs in the HIP library."""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

import numpy as np
import torch

from . import abi
from .layer import DTYPE, TORCH_DTYPE, DecodeLayer, _mark, _on_device, _ptr, _StreamUses

_DTYPES = {TORCH_DTYPE[k]: v for k, v in DTYPE.items()}
_PIECES = abi.sketchssm_conv_piece * 3
ACT = {"none": abi.SKSSM_ACT_NONE, "silu": abi.SKSSM_ACT_SILU, "sigmoid": abi.SKSSM_ACT_SIGMOID}


def _rows(name: str, x: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device) -> int:
    """Checks a tensor of token rows (each row contiguous, the rows at any
    stride) and gives the elements from one row to the next."""
    if x.shape != shape or x.dtype != dtype or x.device != device:
        raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)} on {device}, got {x.dtype} {tuple(x.shape)} on {x.device}")
    if x.is_contiguous():
        return math.prod(shape[1:])
    strides, row = x.stride(), 1
    for d in range(len(shape) - 1, 0, -1):
        if strides[d] != row and shape[d] != 1:
            raise ValueError(f"{name}: every row has to be contiguous, got strides {strides}")
        row *= shape[d]
    return strides[0] if shape[0] > 1 else row


def _shared(spans: list, n: int) -> Optional[tuple]:
    """The first two of several tensors of n token rows each that share memory (slices
    of the same rows may lie between each other), or None.  spans: in bytes, a tensor's
    first row's place, from a row to the next, and of a row."""
    if n == 0:
        return None
    ends = [p + (n - 1) * ps + pl for p, ps, pl in spans]
    for i in range(1, len(spans)):
        p, ps, pl = spans[i]
        for j in range(i):
            q, qs, ql = spans[j]
            if ends[i] <= q or ends[j] <= p or ps < pl or qs < ql:
                continue                         # (rows that overlap themselves are refused by the call)
            if ps == qs:
                if pl <= (q - p) % ps <= ps - ql:
                    continue
            else:                                # each row against the last of the others' that begins before its end
                start = q + qs * np.arange(n)
                at = np.minimum((start + ql - 1 - p) // ps, n - 1)
                if not ((at >= 0) & (p + at * ps + pl > start)).any():
                    continue
            return j, i
    return None


def _indices(name: str, x: torch.Tensor, n: Optional[int], device: torch.device) -> None:
    if x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name}: a contiguous 1-d int32 tensor on {device}")
    if n is not None and x.numel() != n:
        raise ValueError(f"{name}: {n} entries, got {x.numel()}")


def _shape(layer: DecodeLayer) -> tuple:
    return layer.family, layer.B, layer.H, layer.dk, layer.dv, layer.act, layer.S.device


def _prompt_lists(seq_start, seqs, has_state, dev) -> int:
    """Checks prompts' lists and gives the number of prompts."""
    _indices("seq_start", seq_start, None, dev)
    n = seq_start.numel() - 1
    if n < 0:
        raise ValueError("seq_start: the prompts' first tokens and the end of the last")
    for name, x in (("seqs", seqs), ("has_state", has_state)):
        if x is not None:
            _indices(name, x, n, dev)
    return n


class Prompts:
    """Token rows of several prompts, one behind the other, for
    ``DecodeLayer.prefill``: q, k [tokens, H, dk], v, o [tokens, H, dv] in the
    layer's activation dtype, gate (alpha) and beta [tokens, H] fp32 (rows at
    any stride of whole 16 bytes: slices of one projection will do);
    seq_start [n + 1] int32: prompt i holds tokens seq_start[i] up to
    seq_start[i + 1]; seqs [n]: its sequence (None: sequence i); has_state
    [n]: 0 starts it from a zero state (None: every prompt goes on from its
    sequence's state); prime: also write the sketches of the new states; norm
    (with norm_gate, like o): an ``OutputNorm`` of o, applied in place behind
    the prompts (to the rows from seq_start[0] up to seq_start[n], a refused
    prompt's among them: what o holds there then is undefined).  The index tensors are read on the device
    at the call, the tensors are held, and the workspace is allocated once:
    calls that may overlap take a ``Prompts`` each.  It may be dropped once its
    calls are made, on any stream that outlives it; a graph that captured one
    needs it for as long as it is replayed."""

    def __init__(self, layer: DecodeLayer, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: torch.Tensor,
                 beta: torch.Tensor, o: torch.Tensor, seq_start: torch.Tensor,
                 seqs: Optional[torch.Tensor] = None, has_state: Optional[torch.Tensor] = None,
                 prime: bool = True, norm: Optional["OutputNorm"] = None,
                 norm_gate: Optional[torch.Tensor] = None):
        dev, at = layer.S.device, TORCH_DTYPE[layer.act]
        N, H = q.shape[0], layer.H
        strides = [_rows("q", q, (N, H, layer.dk), at, dev), _rows("k", k, (N, H, layer.dk), at, dev),
                   _rows("v", v, (N, H, layer.dv), at, dev), _rows("gate", gate, (N, H), torch.float32, dev),
                   _rows("beta", beta, (N, H), torch.float32, dev), _rows("o", o, (N, H, layer.dv), at, dev)]
        n = _prompt_lists(seq_start, seqs, has_state, dev)
        if norm_gate is not None:
            # (what the norm would refuse is refused here: behind the prompts the states have moved on)
            st, es = _rows("norm_gate", norm_gate, (N, H, layer.dv), at, dev), norm_gate.element_size()
            if norm_gate.data_ptr() % 16 or st * es % 16 or not H * layer.dv <= st <= 1 << 25:
                raise ValueError("norm_gate: rows at whole 16 bytes, at most 2^25 elements apart")
        if norm is not None:
            norm.check((H, layer.dv), dev)
            if H > 65535:
                raise ValueError("norm: at most 65535 heads")
        elif norm_gate is not None:
            raise ValueError("norm_gate: without a norm")
        self.norm, self.norm_gate = norm, norm_gate
        self.shape = _shape(layer)
        need = abi.sketchssm_prefill_workspace_bytes(layer.layer_struct, N, n)
        if need < 0:
            raise ValueError(f"prompts that this layer does not take (code {need})")
        self.q, self.k, self.v, self.gate, self.beta, self.o = q, k, v, gate, beta, o
        self.seq_start, self.seqs, self.has_state, self.prime = seq_start, seqs, has_state, prime
        self.work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        self.uses = _StreamUses(q, k, v, gate, beta, o, seq_start, seqs, has_state, norm_gate, self.work,
                                *((norm.weight, norm.bias) if norm is not None else ()))
        self._struct = abi.sketchssm_prompts(
            _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(o), *strides, N, n, _ptr(seq_start),
            _ptr(seqs), _ptr(has_state), int(prime), _ptr(self.work), need)

    @property
    def struct(self) -> abi.sketchssm_prompts:
        return self._struct

    def check(self, layer: DecodeLayer) -> None:
        """Raises ValueError where these prompts are none of the layer's."""
        if self.shape != _shape(layer):
            raise ValueError(f"prompts of a layer {self.shape}, not {_shape(layer)}")


class ScanPrompts:
    """Token rows of several prompts, one behind the other, for
    ``DecodeLayer.scan`` (Mamba-2 layers): q, k [tokens, G, dk], v, o
    [tokens, H, dv] and dt [tokens, H] (as the decode steps take it: 0 or more)
    in the layer's activation dtype, q, k, v and o rows at any stride of whole
    16 bytes (o's share no memory with the others'); seq_start, seqs, has_state and prime as for ``Prompts``, and so are
    the workspace, held tensors and when it may be dropped."""

    def __init__(self, layer: DecodeLayer, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dt: torch.Tensor,
                 o: torch.Tensor, seq_start: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                 has_state: Optional[torch.Tensor] = None, prime: bool = True):
        dev, at = layer.S.device, TORCH_DTYPE[layer.act]
        N, H, G = q.shape[0], layer.H, layer.G
        strides = [_rows("q", q, (N, G, layer.dk), at, dev), _rows("k", k, (N, G, layer.dk), at, dev),
                   _rows("v", v, (N, H, layer.dv), at, dev), _rows("dt", dt, (N, H), at, dev),
                   _rows("o", o, (N, H, layer.dv), at, dev)]
        spans = [(x.data_ptr(), st * x.element_size(), w * x.element_size())
                 for x, st, w in zip((q, k, v, dt, o), strides, (G * layer.dk, G * layer.dk, H * layer.dv, H, H * layer.dv))]
        for name, span in zip(("q", "k", "v", "dt"), spans):
            if _shared([span, spans[4]], N):
                raise ValueError(f"o shares memory with {name}, which other workgroups still read")
        n = _prompt_lists(seq_start, seqs, has_state, dev)
        self.shape = _shape(layer) + (G,)
        need = abi.sketchssm_scan_workspace_bytes(layer.layer_struct, N, n)
        if need < 0:
            raise ValueError(f"prompts that this layer does not take (code {need})")
        self.q, self.k, self.v, self.dt, self.o = q, k, v, dt, o
        self.seq_start, self.seqs, self.has_state, self.prime = seq_start, seqs, has_state, prime
        self.work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        self.uses = _StreamUses(q, k, v, dt, o, seq_start, seqs, has_state, self.work)
        self._struct = abi.sketchssm_scan_prompts(
            _ptr(q), _ptr(k), _ptr(v), _ptr(dt), _ptr(o), *strides, N, n, _ptr(seq_start), _ptr(seqs),
            _ptr(has_state), int(prime), _ptr(self.work), need)

    @property
    def struct(self) -> abi.sketchssm_scan_prompts:
        return self._struct

    def check(self, layer: DecodeLayer) -> None:
        """Raises ValueError where these prompts are none of the layer's."""
        if self.shape != _shape(layer) + (layer.G,):
            raise ValueError(f"prompts of a layer {self.shape}, not {_shape(layer) + (layer.G,)}")


class ShortConv:
    """The short causal convolution in front of a layer, with the inputs that its
    sequences hold (``state`` [B, taps - 1, channels], oldest first, in the layer's
    activation dtype): weight [channels, taps] (the last tap is the token's own;
    2 to 8 taps) and bias [channels] in fp32, an activation behind it.  order: how
    the channels lie, a permutation of "q", "k" and "v"; unit: the heads of queries
    and keys are divided by sqrt(sum of squares + eps)."""

    def __init__(self, layer: DecodeLayer, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "silu",
                 order: str = "vkq", unit: bool = False, eps: float = 1e-6):
        dev, at = layer.S.device, TORCH_DTYPE[layer.act]
        self.sizes = {"q": layer.G * layer.dk, "k": layer.G * layer.dk, "v": layer.H * layer.dv}
        if sorted(order) != ["k", "q", "v"]:
            raise ValueError('order: a permutation of "q", "k" and "v"')
        if act not in ACT:
            raise ValueError(f"act: one of {tuple(ACT)}")
        if not (math.isfinite(C.c_float(eps).value) and eps >= 0):
            raise ValueError("eps: finite in fp32, 0 or more")
        channels = sum(self.sizes.values())
        if weight.dim() != 2 or weight.shape[0] != channels or not 2 <= weight.shape[1] <= 8:
            raise ValueError(f"weight: [{channels}, 2 to 8 taps], got {tuple(weight.shape)}")
        for name, x, shape in (("weight", weight, weight.shape), ("bias", bias, (channels,))):
            if x is not None and (x.dtype != torch.float32 or x.shape != shape or not x.is_contiguous() or x.device != dev or
                                  x.data_ptr() % 16):
                raise ValueError(f"{name}: a contiguous fp32 tensor {tuple(shape)} on {dev} at whole 16 bytes")
        self.weight, self.bias, self.act, self.order, self.unit, self.eps = weight, bias, act, order, bool(unit), float(eps)
        self.channels, self.taps, self.shape = channels, weight.shape[1], _shape(layer) + (layer.G,)
        self.state = torch.zeros((layer.B, self.taps - 1, channels), dtype=at, device=dev)
        self.err = torch.zeros(4, dtype=torch.int32, device=dev)
        self.rows = abi.sketchssm_rows(self.state.data_ptr(), self.state[:1].numel() * self.state.element_size())
        self.uses = _StreamUses(weight, bias, self.state, self.err)

    def check(self, layer: DecodeLayer) -> None:
        """Raises ValueError where this is no convolution of the layer's."""
        if self.shape != _shape(layer) + (layer.G,):
            raise ValueError(f"a convolution of a layer {self.shape}, not {_shape(layer) + (layer.G,)}")

    def call(self, layer, x, q, k, v, seq_start=None, seqs=None, has_state=None, stream=None) -> int:
        """``DecodeLayer.convolve``."""
        self.check(layer)
        dev, at = layer.S.device, TORCH_DTYPE[layer.act]
        N = x.shape[0]
        xs = _rows("x", x, (N, self.channels), at, dev)
        out = {"q": (q, (N, layer.G, layer.dk)), "k": (k, (N, layer.G, layer.dk)), "v": (v, (N, layer.H, layer.dv))}
        es = x.element_size()
        pieces, spans = [], [(x.data_ptr(), xs * es, self.channels * es)]
        for c in self.order:
            t, shape = out[c]
            place, st, size = t.data_ptr(), _rows(c, t, shape, at, dev), self.sizes[c]
            pieces.append((place, st, size, layer.dk if self.unit and c != "v" else 0))
            spans.append((place, st * es, size * es))
        both = _shared(spans, N)
        if both:
            raise ValueError(" and ".join(("x" + self.order)[i] for i in both) + " share memory")
        n = N
        if seq_start is not None:
            n = _prompt_lists(seq_start, seqs, has_state, dev)
        else:
            for name, t in (("seqs", seqs), ("has_state", has_state)):
                if t is not None:
                    _indices(name, t, n, dev)
        st = abi.sketchssm_convolution(
            x.data_ptr(), xs, self.weight.data_ptr(), None if self.bias is None else self.bias.data_ptr(),
            self.state.data_ptr(), _PIECES(*pieces), self.taps, DTYPE[layer.act], ACT[self.act],
            self.eps, layer.B, N, n, _ptr(seq_start), _ptr(seqs), _ptr(has_state), self.err.data_ptr())
        _mark(stream, dev, x, q, k, v, seq_start, seqs, has_state)
        return _on_device(dev.index, lambda s: abi.sketchssm_conv(st, self.uses.add(s)), stream)

    def error_word(self) -> int:
        return int(self.err[0].item())


class BeamSearch:
    """Selection of beams: ``groups`` requests of ``beams`` (1 to 16) consecutive
    sequences each.  ``select`` takes the sequences' logits [groups * beams,
    vocab] (bf16 or fp32, rows contiguous at any stride) and leaves, [groups,
    beams] each, ``parents`` (int32: the sequence that each goes on from, for
    ``DecodeLayer.reorder``), ``tokens`` (int32), ``scores`` (fp32: the sums of
    the tokens' log probabilities) and ``ended`` (int32: the end token has come).
    At first each request has its first beam alone (the others' scores are minus
    infinity)."""

    def __init__(self, groups: int, beams: int, vocab: int, end: int = -1, device="cuda"):
        if groups < 0 or not 1 <= beams <= 16 or not 1 <= vocab <= 1 << 24 or not -1 <= end < vocab:
            raise ValueError("groups: 0 or more, beams: 1 to 16, vocab: 1 to 2^24, end: -1 (none) to vocab - 1")
        need = max(abi.sketchssm_beam_workspace_bytes(groups, beams, vocab, d) for d in DTYPE.values())
        if need < 0:
            raise ValueError(f"beams of this many requests and tokens are not taken (code {need})")
        z = lambda dt: torch.zeros((groups, beams), dtype=dt, device=device)  # noqa: E731
        self.groups, self.beams, self.vocab, self.end = groups, beams, vocab, end
        self.scores, self.ended, self.parents, self.tokens = z(torch.float32), z(torch.int32), z(torch.int32), z(torch.int32)
        self.err = torch.zeros(4, dtype=torch.int32, device=device)
        self.work = torch.empty(need, dtype=torch.uint8, device=device)
        self.uses = _StreamUses(self.scores, self.ended, self.parents, self.tokens, self.err, self.work)
        self.reset()

    def reset(self) -> None:
        """A new search: every request's first beam alone."""
        self.scores.fill_(-math.inf)
        self.scores[:, 0] = 0.0
        self.ended.zero_()

    def select(self, logits: torch.Tensor, scores: Optional[torch.Tensor] = None, ended: Optional[torch.Tensor] = None,
               stream=None) -> int:
        """The next beams; scores and ended: others than the search's own as the
        beams' present ones.  Where a stream is given the tensors may be dropped once
        the call is made, as ``DecodeLayer.convolve``'s.  Returns the library's code."""
        dev, rows = self.scores.device, self.groups * self.beams
        if logits.dtype not in _DTYPES or dev.type != "cuda":
            raise ValueError("logits: a bf16 or fp32 device tensor [groups * beams, vocab]")
        stride = _rows("logits", logits, (rows, self.vocab), logits.dtype, dev)
        for name, t, own in (("scores", scores, self.scores), ("ended", ended, self.ended)):
            if t is not None and (t.shape != own.shape or t.dtype != own.dtype or t.device != dev or not t.is_contiguous()):
                raise ValueError(f"{name}: a contiguous {own.dtype} tensor {tuple(own.shape)} on {dev}")
        scores, ended = self.scores if scores is None else scores, self.ended if ended is None else ended
        st = abi.sketchssm_beams(
            logits.data_ptr(), stride, scores.data_ptr(), ended.data_ptr(), self.scores.data_ptr(), self.ended.data_ptr(),
            self.parents.data_ptr(), self.tokens.data_ptr(), self.err.data_ptr(), self.groups, self.beams, self.vocab,
            _DTYPES[logits.dtype], self.end, self.work.data_ptr(), self.work.numel())
        _mark(stream, dev, logits, scores, ended)
        return _on_device(dev.index, lambda s: abi.sketchssm_beam_select(st, self.uses.add(s)), stream)

    def error_word(self) -> int:
        return int(self.err[0].item())


class StateCache:
    """A pool of ``slots`` slots, each for one sequence's states of a layer in
    8 or 4 bits: codes [slots, H, dk, dv] int8 (4 bits: [.., dv / 2] uint8, the
    lower column in the low half) and scale [slots, H, dk, dv / 32].  It may be
    dropped as ``Prompts`` may."""

    def __init__(self, layer: DecodeLayer, slots: int, bits: int = 8):
        if bits not in (8, 4):
            raise ValueError("bits: 8 or 4")
        if slots < 0:
            raise ValueError("slots: 0 or more")
        H, dk, dv, dev = layer.H, layer.dk, layer.dv, layer.S.device
        self.slots, self.bits, self.shape = slots, bits, (H, dk, dv)
        self.codes = (torch.zeros((slots, H, dk, dv), dtype=torch.int8, device=dev) if bits == 8 else
                      torch.zeros((slots, H, dk, dv // 2), dtype=torch.uint8, device=dev))
        self.scale = torch.zeros((slots, H, dk, dv // 32), dtype=torch.float32, device=dev)
        self.uses = _StreamUses(self.codes, self.scale)
        self._struct = abi.sketchssm_state_cache(_ptr(self.codes), _ptr(self.scale), slots, bits)

    @property
    def struct(self) -> abi.sketchssm_state_cache:
        return self._struct

    def check(self, layer: DecodeLayer, seqs: torch.Tensor, slots: torch.Tensor) -> None:
        """Raises ValueError where these entries of this cache are none of the layer's."""
        if self.shape != (layer.H, layer.dk, layer.dv) or self.codes.device != layer.S.device:
            raise ValueError(f"a cache of states {self.shape} on {self.codes.device}, not of this layer's")
        _indices("seqs", seqs, None, layer.S.device)
        _indices("slots", slots, seqs.numel(), layer.S.device)


class OutputNorm:
    """How a layer's outputs are normalised: over each group of channels, by
    the root mean square or (centred) by mean and variance, times weight plus
    bias (fp32, [groups, width], or [width] for every group; None: 1 and 0),
    with an activation ("none", "silu" or "sigmoid") of the gate, multiplied
    on before the norm (gate_first) or after it; without a gate the
    activation is that of the result."""

    def __init__(self, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 eps: float = 1e-5, act: str = "silu", centred: bool = False, gate_first: bool = False):
        for name, x in (("weight", weight), ("bias", bias)):
            if x is not None and (x.dtype != torch.float32 or not x.is_contiguous() or x.dim() not in (1, 2)):
                raise ValueError(f"{name}: a contiguous fp32 tensor [groups, width] or [width]")
        if weight is not None and bias is not None and weight.shape != bias.shape:
            raise ValueError("weight and bias: of one shape")
        if not (math.isfinite(C.c_float(eps).value) and eps >= 0):
            raise ValueError("eps: finite in fp32, 0 or more")
        if act not in ACT:
            raise ValueError(f"act: one of {tuple(ACT)}")
        self.weight, self.bias, self.eps, self.act = weight, bias, float(eps), act
        self.centred, self.gate_first = bool(centred), bool(gate_first)

    def check(self, shape, device: torch.device) -> None:
        """Raises ValueError where weight or bias do not fit [groups, width] on the device."""
        for t in (self.weight, self.bias):
            if t is not None and (t.shape != shape[2 - t.dim():] or t.device != device):
                raise ValueError(f"weight and bias: {tuple(shape)} or {tuple(shape[1:])} on {device}, got {tuple(t.shape)} on {t.device}")
            if t is not None and t.data_ptr() % 16:
                raise ValueError("weight and bias: at whole 16 bytes")


def group_norm(x: torch.Tensor, norm: OutputNorm, y: torch.Tensor, gate: Optional[torch.Tensor] = None,
               stream=None, rows: Optional[torch.Tensor] = None) -> int:
    """y = the group norm of x [rows, groups, width] (bf16 or fp32, rows at any
    stride of whole 16 bytes), gated; y may be x.  rows: an int32 device
    tensor, say prompts' seq_start: only the rows from its first up to its last
    entry, which are read on the device.  Returns the library's code."""
    dt, shape, dev = x.dtype, x.shape, x.device
    if len(shape) != 3 or dt not in _DTYPES or dev.type != "cuda":
        raise ValueError("x: a bf16 or fp32 device tensor [rows, groups, width]")
    xs, ys = _rows("x", x, shape, dt, dev), _rows("y", y, shape, dt, dev)
    zs = _rows("gate", gate, shape, dt, dev) if gate is not None else 0
    norm.check(shape[1:], dev)
    w = norm.weight if norm.weight is not None else norm.bias
    first = end = None
    if rows is not None:
        _indices("rows", rows, None, dev)
        if rows.numel() == 0:
            raise ValueError("rows: the first row and the end")
        first = rows.data_ptr()
        end = first + 4 * (rows.numel() - 1)
    st = abi.sketchssm_norm(x.data_ptr(), gate.data_ptr() if gate is not None else None, y.data_ptr(),
                            norm.weight.data_ptr() if norm.weight is not None else None,
                            norm.bias.data_ptr() if norm.bias is not None else None, xs, zs, ys,
                            shape[0], first, end, shape[1], shape[2], _DTYPES[dt], int(w is not None and w.dim() == 2),
                            int(norm.centred), ACT[norm.act], int(norm.gate_first), norm.eps)
    return _on_device(dev.index, lambda s: abi.sketchssm_group_norm(st, s), stream)
