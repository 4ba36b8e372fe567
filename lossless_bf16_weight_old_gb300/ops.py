"""The operators on either side of the weight sync (binding over include/ops/bf16ops.h).

    AdamWBatch        one AdamW step over many tensors, moments in 32 or in 8 bits: what makes
                      the new weights that CompressBatch encodes
    AdapterSet, AdapterRows, adapter_forward, adapter_backward
                      low-rank adapters of many requests beside a shared projection
    TokenLogprobs     log probabilities of given tokens with entropy and top alternatives, and
                      the logits' gradient
    ExpertRouting     the experts of each token and their weights, per-expert counts and the
                      balance loss, and the gradient of the router's logits

Every computation runs in libbf16ops' CUDA kernels; this module checks and marshals arguments
and allocates device buffers with PyTorch.  The names are re-exported by the package.

Every call works in the order of the stream that it is given (the current one by default), and so
do the buffers that it makes for itself.  Tensors of the caller's must be ready in that order, and
stay allocated until the work is done.
"""
from __future__ import annotations

import ctypes
import math
from typing import Sequence

import torch

from . import _ops_lib

OK, ERR_INVALID_ARG = 0, 1
SKIPPED_NONFINITE = 16
BLOCK_ELEMS = 256
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_U64 = (1 << 64) - 1
_current_stream = torch._C._cuda_getCurrentRawStream

__all__ = ["AdamWBatch", "AdapterSet", "AdapterRows", "adapter_forward", "adapter_backward", "TokenLogprobs", "ExpertRouting", "SKIPPED_NONFINITE", "OpsError", "ops_status_name"]


class OpsError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = int(code)
        super().__init__(f"{what}: {ops_status_name(code)} ({code})")


def ops_status_name(code: int) -> str:
    """Description of a status of these operators."""
    return _ops_lib.load().bo_status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise OpsError(rc, what)


def _here(device: torch.device) -> None:
    """The library works on the current device, which has to be the tensors'."""
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _failed(rc: int, what: str, device: torch.device):
    _here(device)      # (of a handle from another device the library says no more than that it is one)
    raise OpsError(rc, what)


def _stream(stream, device: torch.device) -> int:
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
        return stream.cuda_stream
    return _current_stream(device.index)


class _Owner:
    """An object with device buffers of its own, which are made and filled in the order of the
    stream that its constructor was given (or the current one).  Its first use on another stream
    waits until they are filled, and the allocator learns of that stream."""

    def _made(self, buffers: list, device: torch.device) -> None:   # (on the constructor's stream)
        self._buffers, self.device, self._index = buffers, device, device.index
        self._home, self._others = _stream(None, device), set()
        self._filled = None
        if not torch.cuda.is_current_stream_capturing():
            self._filled = torch.cuda.Event()
            self._filled.record()

    def _on(self, stream) -> int:
        """The handle of the stream of a call."""
        # (the handle alone: a torch.cuda.Stream object would cost more than the launch)
        raw = _current_stream(self._index) if stream is None else _stream(stream, self.device)
        if raw != self._home and raw not in self._others:
            self._join(raw, stream)
        return raw

    def _join(self, raw: int, stream) -> None:
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        for t in self._buffers:
            t.record_stream(s)
        with torch.cuda.stream(s):
            # (a capture may not wait for what lies before it, and whoever began it has)
            if self._filled is None or torch.cuda.is_current_stream_capturing():
                return
            s.wait_event(self._filled)
        self._others.add(raw)


def _arena(t: torch.Tensor, name: str, dtype: torch.dtype, numel: int, device) -> torch.Tensor:
    if t.dtype != dtype or t.numel() != numel or not t.is_contiguous() or t.device != device:
        raise ValueError(f"state[{name!r}] must be a contiguous {dtype} tensor of {numel} "
                         f"elements on {device}")
    return t


class AdamWBatch(_Owner):
    """One AdamW step over fixed tensors: the tensor table, the state and the step count.

    weights       tensors to update: bfloat16, or float32 for 32-bit weights
    grads         their gradients, all bfloat16 or all float32
    news          (optional) where the new weights go instead, the old ones staying as they are:
                  CompressBatch(weights, news) then encodes the step
    master        keep an FP32 master copy of bfloat16 weights (default); without one the
                  bfloat16 weights are all there is, best rounded with stochastic=True
    state_bits    32, or 8 for moments coded per block of 256 elements
    weight_decay  one number, or one per tensor
    max_norm      clip by the global gradient norm and skip a step whose norm is not finite
                  (math.inf: only skip); None: neither
    stochastic    round bfloat16 weights without a master stochastically
    seed          of the random bits that this and 8-bit moments use
    step          steps taken so far
    state         (optional) dict of tensors to hold the state, as in `state` of another batch:
                  "m", "v", with 8 bits "m_scale" and "v_scale", with a master "master"; those
                  that are missing are made here (moments 0, master = weights)

    The arenas in `state` hold the tensors one after the other, each from a new block of 256 on;
    `view(name, i)` is tensor i's part.  Results on the device after `run`: the new weights, the
    state, `norm` (float32[1], with max_norm), `status` (int32[1]: OK or SKIPPED_NONFINITE) and
    `steps` (int64[1]).  Tensors must stay where they are for the life of the batch, and each be
    given once (tied weights: as one tensor, with the sum of their gradients)."""

    def __init__(self, weights: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], *,
                 news: Sequence[torch.Tensor] | None = None, master: bool | None = None,
                 state_bits: int = 32, lr: float = 1e-3, betas: tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: float | Sequence[float] = 0.0,
                 max_norm: float | None = None, stochastic: bool = False, seed: int = 0,
                 step: int = 0, state: dict | None = None, stream=None):
        k = len(weights)
        if k == 0:
            raise ValueError("no tensors")
        outs = list(news) if news is not None else list(weights)
        if len(grads) != k or len(outs) != k:
            raise ValueError("weights, grads and news differ in length")
        dev, wtype, gtype = weights[0].device, weights[0].dtype, grads[0].dtype
        if wtype not in _DTYPES or gtype not in _DTYPES:
            raise TypeError(f"weights and grads must be bfloat16 or float32, got {wtype} and {gtype}")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if master is None:
            master = wtype == torch.bfloat16
        if master and wtype != torch.bfloat16:
            raise ValueError("a master copy goes with bfloat16 weights")
        if stochastic and (master or wtype != torch.bfloat16):
            raise ValueError("stochastic rounding goes with bfloat16 weights without a master")
        decay = [float(weight_decay)] * k if isinstance(weight_decay, (int, float)) else \
            [float(d) for d in weight_decay]
        if len(decay) != k:
            raise ValueError("weight_decay must be one number or one per tensor")
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive")
        if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1) or not eps >= 0:
            raise ValueError("betas must lie in [0, 1) and eps must not be negative")
        if not 0 <= step < 1 << 62:
            raise ValueError("step must not be negative (or past 2**62)")
        for name, ts, dt in (("weights", weights, wtype), ("grads", grads, gtype), ("news", outs, wtype)):
            for i, t in enumerate(ts):
                if t.dtype != dt or not t.is_cuda or t.device != dev or not t.is_contiguous():
                    raise ValueError(f"{name}[{i}] must be a contiguous {dt} tensor on {dev}")
                if t.numel() != weights[i].numel():
                    raise ValueError(f"{name}[{i}] has {t.numel()} elements, its weights "
                                     f"{weights[i].numel()}")
        _here(dev)
        _stream(stream, dev)
        self.shapes = [w.shape for w in weights]
        self.ns = [w.numel() for w in weights]
        self.first_blocks, blocks = [], 0
        for n in self.ns:
            self.first_blocks.append(blocks)
            blocks += -(-n // BLOCK_ELEMS)
        self.blocks, self.state_bits = blocks, state_bits
        self.lr, self.betas, self.eps = float(lr), (float(betas[0]), float(betas[1])), float(eps)
        self.max_norm = max_norm

        given, elems = dict(state or {}), blocks * BLOCK_ELEMS
        want = {"m": torch.float32, "v": torch.float32} if state_bits == 32 else \
            {"m": torch.int8, "v": torch.uint8, "m_scale": torch.float32, "v_scale": torch.float32}
        if master:
            want["master"] = torch.float32
        if set(given) - set(want):
            raise ValueError(f"state has no place for {sorted(set(given) - set(want))}")
        self.state: dict[str, torch.Tensor] = {}
        with torch.cuda.stream(stream):
            for name, dt in want.items():
                numel = blocks if name.endswith("_scale") else elems
                self.state[name] = _arena(given[name], name, dt, numel, dev) if name in given else \
                    torch.zeros(numel, dtype=dt, device=dev)
            if master and "master" not in given:
                for i, w in enumerate(weights):
                    self.view("master", i).copy_(w)

        items = (_ops_lib.AdamWItem * k)()
        for i in range(k):
            items[i].d_weight = weights[i].data_ptr()
            items[i].d_out = outs[i].data_ptr()
            items[i].d_grad = grads[i].data_ptr()
            items[i].n = self.ns[i]
            items[i].first_block = self.first_blocks[i]
            items[i].weight_decay = decay[i]
        ptr = {n: t.data_ptr() if blocks else None for n, t in self.state.items()}
        st = _ops_lib.AdamWState(ptr["m"], ptr["v"], ptr.get("m_scale"), ptr.get("v_scale"),
                                 ptr.get("master"), blocks)
        lib = _ops_lib.load()
        self.handle = _ops_lib.AdamW()
        kind = 2 if wtype == torch.float32 else 0 if master else 1
        with torch.cuda.stream(stream):
            self.plan = torch.empty(int(lib.bo_adamw_plan_size(items, k)), dtype=torch.uint8, device=dev)
            _check(lib.bo_adamw_plan(items, k, ctypes.byref(st), kind, _DTYPES[gtype], state_bits,
                                     int(bool(stochastic)), int(step), self.plan.data_ptr(),
                                     self.plan.numel(), ctypes.byref(self.handle), _stream(None, dev)),
                   "bo_adamw_plan")
            self._made([self.plan] + [t for n, t in self.state.items() if n not in given], dev)
        self.steps = self.plan[:8].view(torch.int64)
        self.norm = self.plan[8:12].view(torch.float32)
        self.status = self.plan[16:20].view(torch.int32)
        self._args = _ops_lib.AdamWStepArgs(float(lr), None, self.betas[0], self.betas[1], self.eps,
                                            0.0 if max_norm is None else float(max_norm),
                                            int(seed) & _U64)
        self._refs = ctypes.byref(self.handle), ctypes.byref(self._args)
        self._step = lib.bo_adamw_step
        self._keep = (list(weights), list(grads), outs)

    def run(self, lr: float | torch.Tensor | None = None, stream=None) -> None:
        """Takes one step, with this learning rate (a number, or a float32[1] device tensor that
        the step reads when it runs) for this step alone, or the batch's own (`lr`)."""
        args, where = self._args, None
        if isinstance(lr, torch.Tensor):
            if lr.dtype != torch.float32 or lr.numel() != 1 or lr.device != self.device:
                raise ValueError(f"lr must be a number or a float32[1] tensor on {self.device}")
            if stream is not None:
                lr.record_stream(stream)
            self._lr, where, rate = lr, lr.data_ptr(), 0.0
        else:
            rate = self.lr if lr is None else float(lr)
        args.lr, args.d_lr = rate, where
        rc = self._step(*self._refs, self._on(stream))
        if rc != OK:
            _failed(rc, "bo_adamw_step", self.device)

    def grad_norm(self, stream=None) -> torch.Tensor:
        """The global norm of the gradients as they are now (`norm`), without a step."""
        _check(_ops_lib.load().bo_adamw_norm(self._refs[0], self._args.max_norm, self._on(stream)),
               "bo_adamw_norm")
        return self.norm

    def view(self, name: str, i: int) -> torch.Tensor:
        """Tensor i's part of a state arena, in its shape (scales: one per block)."""
        b = self.first_blocks[i]
        if name.endswith("_scale"):
            return self.state[name][b:b + -(-self.ns[i] // BLOCK_ELEMS)]
        return self.state[name][b * BLOCK_ELEMS:b * BLOCK_ELEMS + self.ns[i]].view(self.shapes[i])

    def moments(self, dtype: torch.dtype = torch.float32, stream=None):
        """Both moments as values of `dtype`, laid out as the arenas.  With 32-bit states these
        are the arenas themselves (dtype float32) or copies."""
        if dtype not in _DTYPES:
            raise TypeError("dtype must be bfloat16 or float32")
        raw = self._on(stream)
        with torch.cuda.stream(stream):
            if self.state_bits == 32:
                m, v = self.state["m"].to(dtype), self.state["v"].to(dtype)
            else:
                m = torch.empty(self.state["m"].numel(), dtype=dtype, device=self.device)
                v = torch.empty_like(m)
                _check(_ops_lib.load().bo_adamw_moments(self._refs[0], _DTYPES[dtype], m.data_ptr(),
                                                        v.data_ptr(), raw), "bo_adamw_moments")
        if stream is not None:   # (the caller may go on with them on the current one)
            m.record_stream(torch.cuda.current_stream(self.device))
            v.record_stream(torch.cuda.current_stream(self.device))
        return m, v


def _matrix(t: torch.Tensor, name: str, rows: int | None, width: int, device,
            dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Checks a matrix whose rows are contiguous (any row stride)."""
    if t.dim() != 2 or t.dtype != dtype or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a 2-dimensional {dtype} tensor on {device}")
    if t.shape[1] != width or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"({'any' if rows is None else rows}, {width})")
    if (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < width):
        raise ValueError(f"{name}'s rows must be contiguous and may not overlap")
    return t


def _ld(t: torch.Tensor) -> int:
    """Row stride in elements (of a single row: its width)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class AdapterSet(_Owner):
    """The adapters of one projection, read where they lie.

    downs, ups   factors: downs[i] is [rank_i, hidden], ups[i] is [out, rank_i], bfloat16, rows
                 contiguous; ranks from 1 to 128 may differ
    scales       one number per adapter (usually alpha / rank), or one for all
    d_downs, d_ups   (for a backward pass) their gradients, all bfloat16 or all float32; adapters may
                 share a factor, but each has gradients of its own

    The tensors must stay where they are for the life of the set; their values may change at any
    time (an optimizer step, a delta applied in place)."""

    def __init__(self, downs: Sequence[torch.Tensor], ups: Sequence[torch.Tensor],
                 scales: float | Sequence[float] = 1.0, *,
                 d_downs: Sequence[torch.Tensor] | None = None,
                 d_ups: Sequence[torch.Tensor] | None = None, stream=None):
        k = len(downs)
        if k == 0 or len(ups) != k:
            raise ValueError("downs and ups must hold the same number of adapters, at least one")
        scales = [float(scales)] * k if isinstance(scales, (int, float)) else [float(s) for s in scales]
        if len(scales) != k:
            raise ValueError("scales must be one number or one per adapter")
        if (d_downs is None) != (d_ups is None):
            raise ValueError("d_downs and d_ups come together")
        dev, hidden, out = downs[0].device, downs[0].shape[-1], ups[0].shape[0]
        gtype = torch.bfloat16
        if d_downs is not None:
            if len(d_downs) != k or len(d_ups) != k:
                raise ValueError("one gradient per factor")
            gtype = d_downs[0].dtype
            if gtype not in _DTYPES:
                raise TypeError(f"gradients must be bfloat16 or float32, got {gtype}")
        _here(dev)
        _stream(stream, dev)
        if not (1 <= hidden <= 1 << 24 and 1 <= out <= 1 << 24):
            raise ValueError("the factors' widths must lie in 1 .. 2**24")
        items = (_ops_lib.Adapter * k)()
        for i in range(k):
            r = downs[i].shape[0]
            if not 1 <= r <= 128:
                raise ValueError(f"adapter {i} has rank {r}; ranks are 1 to 128")
            _matrix(downs[i], f"downs[{i}]", r, hidden, dev)
            _matrix(ups[i], f"ups[{i}]", out, r, dev)
            it = items[i]
            it.d_down, it.ld_down = downs[i].data_ptr(), _ld(downs[i])
            it.d_up, it.ld_up = ups[i].data_ptr(), _ld(ups[i])
            it.rank, it.scale = r, scales[i]
            if d_downs is not None:
                _matrix(d_downs[i], f"d_downs[{i}]", r, hidden, dev, gtype)
                _matrix(d_ups[i], f"d_ups[{i}]", out, r, dev, gtype)
                it.d_grad_down, it.ld_grad_down = d_downs[i].data_ptr(), _ld(d_downs[i])
                it.d_grad_up, it.ld_grad_up = d_ups[i].data_ptr(), _ld(d_ups[i])
        lib = _ops_lib.load()
        self.handle = _ops_lib.AdapterSet()
        with torch.cuda.stream(stream):
            self.table = torch.empty(max(256, int(lib.bo_adapter_set_size(k))), dtype=torch.uint8, device=dev)
            _check(lib.bo_adapter_set_init(items, k, hidden, out, _DTYPES[gtype], self.table.data_ptr(),
                                           self.table.numel(), ctypes.byref(self.handle), _stream(None, dev)),
                   "bo_adapter_set_init")
            self._made([self.table], dev)
        self.k, self.hidden, self.out = k, hidden, out
        #: columns of `low`, the activations that the forward pass keeps for the backward
        self.rank = int(self.handle.rank)
        self._ref = ctypes.byref(self.handle)
        self._low_rows = int(lib.bo_adapter_low_rows(self._ref))
        self._forward, self._backward = lib.bo_adapter_forward, lib.bo_adapter_backward
        self._need = (-1, 0)     # rows, and the bytes that a backward pass of as many needs
        self._keep = (list(downs), list(ups), d_downs, d_ups)


class AdapterRows(_Owner):
    """The rows of a batch grouped by adapter, on the device: index[t] (int32) is the adapter of
    row t, -1 for none.  One grouping serves every projection of a model step; `update` regroups
    for new values of as many rows.  `status` (int32[1]) is ERR_INVALID_ARG when an index lies
    outside -1 .. k - 1 (such rows count as rows without an adapter), and ERR_CUDA from a call of
    adapter_forward or adapter_backward on that found a wait inside one of its kernels too long, until
    the next `update`: that call's outputs are not to be used."""

    def __init__(self, index: torch.Tensor, k: int, *, stream=None):
        if index.dtype != torch.int32 or index.dim() != 1 or not index.is_cuda:
            raise ValueError("index must be a 1-dimensional int32 CUDA tensor")
        self.rows, self.k = index.numel(), int(k)
        # (here, because the library's integers have 32 bits)
        if not 1 <= self.k <= 65535 or self.rows > 1 << 30:
            raise ValueError("k must lie in 1 .. 65535 and the rows be at most 2**30")
        need = int(_ops_lib.load().bo_adapter_rows_size(self.rows, self.k))
        _here(index.device)
        self.handle = _ops_lib.AdapterRows()
        self._ref = ctypes.byref(self.handle)
        _stream(stream, index.device)
        with torch.cuda.stream(stream):
            self.memory = torch.empty(need, dtype=torch.uint8, device=index.device)
            self.status = torch.zeros(1, dtype=torch.int32, device=index.device)
            self.device = index.device
            self._group(index, stream, _stream(None, index.device))
            self._made([self.memory, self.status], index.device)

    def update(self, index: torch.Tensor, stream=None) -> None:
        self._group(index, stream, self._on(stream))

    def _group(self, index: torch.Tensor, stream, raw: int) -> None:
        if index.dtype != torch.int32 or index.numel() != self.rows or index.device != self.device \
                or not index.is_contiguous():
            raise ValueError(f"index must be a contiguous int32 tensor of {self.rows} elements on "
                             f"{self.device}")
        _here(self.device)
        if stream is not None:
            index.record_stream(stream)   # (it may go before the grouping has read it)
        self.index = index
        _check(_ops_lib.load().bo_adapter_rows_init(
            index.data_ptr(), self.rows, self.k, self.memory.data_ptr(), self.memory.numel(),
            self._ref, self.status.data_ptr(), raw), "bo_adapter_rows_init")


def _pair(adapters: AdapterSet, rows: AdapterRows, stream) -> int:
    """Checks that the two go together; returns the handle of the call's stream."""
    if rows.k != adapters.k:
        raise ValueError(f"rows are grouped over {rows.k} adapters, the set has {adapters.k}")
    raw = adapters._on(stream)
    if raw != rows._home:
        rows._on(stream)
    return raw


def _unrecorded(a: torch.Tensor, b: torch.Tensor) -> None:
    if (a.requires_grad or b.requires_grad) and torch.is_grad_enabled():
        raise ValueError("autograd records this call's tensors, and would miss the adapters' part: "
                         "call under torch.no_grad() or with detached tensors, and adapter_backward "
                         "for the gradients")


def _scratch(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """Memory for one call, from the pool of the stream that the call runs on: what used it
    before, and what will after, is in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows_of(t: torch.Tensor, name: str, shape: tuple, device) -> int:
    """Checks an activation matrix; returns its row stride."""
    ld, one = t.stride() if t.dim() == 2 else (0, 0)
    if t.shape != shape or t.dtype is not torch.bfloat16 or t.device != device or one != 1 or \
            ld < shape[1]:
        _matrix(t, name, *shape, device)     # says what is wrong, or that strides do not matter
        return _ld(t)
    return ld


def _low(low: torch.Tensor, adapters: AdapterSet, rows: AdapterRows) -> int:
    if low.shape != (rows.rows, adapters.rank) or low.dtype is not torch.bfloat16 or \
            not low.is_contiguous() or low.device != adapters.device:
        raise ValueError(f"low must be a contiguous bfloat16 tensor of shape "
                         f"({rows.rows}, {adapters.rank}) on {adapters.device}")
    return low.data_ptr()


def adapter_forward(x: torch.Tensor, y: torch.Tensor, adapters: AdapterSet, rows: AdapterRows, *,
                    low: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] += scale * up @ (down @ x[t]) with the adapter of row t, in place; y is the shared
    projection's output.  x [rows, hidden] and y [rows, out] are bfloat16 with contiguous rows.
    low (optional, bfloat16 [rows, adapters.rank]) receives what adapter_backward needs.  Rows
    without an adapter are left alone.  Returns y.  `rows.status` tells of a kernel that gave up.
    Autograd does not see the call, which refuses an x or y that it records."""
    raw = _pair(adapters, rows, stream)
    _unrecorded(x, y)
    dev = adapters.device
    ldx = _rows_of(x, "x", (rows.rows, adapters.hidden), dev)
    ldy = _rows_of(y, "y", (rows.rows, adapters.out), dev)
    if low is None and rows.rows >= adapters._low_rows:   # (workspace, for many rows)
        low = _scratch((rows.rows, adapters.rank), torch.bfloat16, dev, stream)
    rc = adapters._forward(adapters._ref, rows._ref, x.data_ptr(), ldx, y.data_ptr(), ldy,
                           None if low is None else _low(low, adapters, rows), raw)
    if rc != OK:
        _failed(rc, "bo_adapter_forward", dev)
    return y


def adapter_backward(x: torch.Tensor, dy: torch.Tensor, low: torch.Tensor,
                     dx: torch.Tensor | None, adapters: AdapterSet, rows: AdapterRows, *,
                     accumulate: bool = False, workspace: torch.Tensor | None = None,
                     stream=None) -> None:
    """The backward pass of adapter_forward: dx[t] += the adapter's part (dx holds the shared
    projection's part; None: not wanted), in place, and the gradients given to the set are
    written, or with accumulate=True added to.  low is the forward pass's; `rows.status` tells of a
    kernel that gave up."""
    raw = _pair(adapters, rows, stream)
    _unrecorded(dy, dy if dx is None else dx)
    dev = adapters.device
    ldx = _rows_of(x, "x", (rows.rows, adapters.hidden), dev)
    lddy = _rows_of(dy, "dy", (rows.rows, adapters.out), dev)
    lddx = 0 if dx is None else _rows_of(dx, "dx", (rows.rows, adapters.hidden), dev)
    ws = workspace
    if ws is None:
        n, need = adapters._need
        if n != rows.rows:
            need = max(256, int(_ops_lib.load().bo_adapter_backward_workspace_size(adapters._ref,
                                                                                   rows.rows)))
            adapters._need = rows.rows, need
        ws = _scratch(need, torch.uint8, dev, stream)
    else:
        if ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        need = ws.numel() * ws.element_size()
    rc = adapters._backward(
        adapters._ref, rows._ref, x.data_ptr(), ldx, dy.data_ptr(), lddy,
        _low(low, adapters, rows), None if dx is None else dx.data_ptr(), lddx, accumulate,
        ws.data_ptr(), need, raw)
    if rc != OK:
        _failed(rc, "bo_adapter_backward", dev)


def _device_of(device) -> torch.device:
    """The current device, which has to be the one that was asked for."""
    dev = torch.device("cuda" if device is None else device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    _here(dev)
    return dev


_TOKENS, _FLOAT, _MASKS = (torch.int64, torch.int32), (torch.float32,), (torch.bool, torch.uint8)


class _Results(_Owner):
    """An object whose one buffer holds the results of its calls."""

    def _memory(self, nbytes: int, device: torch.device) -> torch.Tensor:
        self._at = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return self._at

    def _part(self, pointer: int | None, dtype: torch.dtype, *shape: int) -> torch.Tensor:
        """The part of the buffer that begins there."""
        numel = 1
        for n in shape:
            numel *= n
        if numel == 0 or not pointer:
            return torch.empty(shape, dtype=dtype, device=self.device)
        at = pointer - self._at.data_ptr()
        return self._at[at:at + numel * dtype.itemsize].view(dtype).view(shape)


def _rows_in(t: torch.Tensor, name: str, most: int, width: int, device: torch.device) -> tuple[int, int]:
    """Checks a matrix of at most `most` rows; returns how many it has, and its row stride."""
    if t.dim() == 2 and t.dtype in _DTYPES and t.get_device() == device.index:
        rows, cols = t.shape
        ld, one = t.stride()
        if cols == width and rows <= most and (one == 1 or width == 1) and (ld >= width or rows <= 1):
            return rows, ld if rows > 1 else width
        if cols != width or rows > most:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (up to {most}, {width})")
        raise ValueError(f"{name}'s rows must be contiguous and may not overlap")
    raise ValueError(f"{name} must be a 2-dimensional bfloat16 or float32 tensor on {device}")


def _column(t: torch.Tensor, name: str, rows: int, dtypes, device: torch.device) -> int:
    """Checks a vector of one number a row; returns its stride."""
    if t.dim() != 1 or t.numel() != rows or t.get_device() != device.index or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a 1-dimensional tensor of {rows} elements of type "
                         f"{' or '.join(str(d) for d in dtypes)} on {device}")
    return t.stride(0)


def _out_for(out: torch.Tensor | None, t: torch.Tensor, rows: int, width: int, ld: int, device: torch.device,
             stream) -> tuple[torch.Tensor, int]:
    """Where the gradient of the logits t goes, and its row stride: `out`, or memory of its own whose rows are
    as far apart as the logits', but for whole words of 32 bytes (in which the kernels read and write)."""
    if out is None:
        ld = width + (ld - width) % (32 // t.dtype.itemsize)
        out = _scratch((rows, ld), t.dtype, device, stream)
        if stream is not None:   # (the caller may go on with it on the current one)
            out.record_stream(torch.cuda.current_stream(device))
        return out[:, :width], ld
    _unrecorded_tensor(out, "out")
    if out.dtype is t.dtype:
        n, ld = _rows_in(out, "out", rows, width, device)
        if n == rows:
            return out, ld
    raise ValueError(f"out must have the logits' shape {tuple(t.shape)} and type {t.dtype}")


def _unrecorded_logits(t: torch.Tensor) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("autograd records these logits, and would miss the call's part: call under "
                         "torch.no_grad() or with detached logits, and backward() for the gradient")


def _unrecorded_tensor(t: torch.Tensor, name: str) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"autograd records {name}, and would miss the call's part: call under "
                         "torch.no_grad() or with a detached tensor")


class TokenLogprobs(_Results):
    """Log probabilities of given tokens, for up to `rows` rows of logits over `vocab` tokens.

    top       how many alternatives each row gets (at most 32)
    entropy   also the entropy of each row's distribution (and its gradient)
    device    the current CUDA device (default)

    Results on the device after `run`, of its rows (those behind them stay as they were):
    `logprobs` (float32[rows]), `entropy` (float32[rows], or None), `top_logprobs`
    (float32[rows, top]) and `top_tokens` (int32[rows, top]), the greatest first and of equal ones
    the lowest token first.  Each run overwrites them: calls at the same time, on several streams or
    in graphs that run side by side, want an object each.

    Rows whose token is negative are left out and not read: their results are 0, their top tokens -1
    and their gradients 0.  A token of `vocab` or more makes a row's log probability and gradient
    NaN, which a clipped AdamWBatch skips.  Logits of -inf are tokens of probability 0."""

    def __init__(self, rows: int, vocab: int, *, top: int = 0, entropy: bool = False, device=None,
                 stream=None):
        rows, vocab, top = int(rows), int(vocab), int(top)
        if not 0 <= rows <= 1 << 28 or not 1 <= vocab <= 1 << 24:
            raise ValueError("rows must lie in 0 .. 2**28 and vocab in 1 .. 2**24")
        if not 0 <= top <= min(32, vocab):
            raise ValueError("top must lie in 0 .. 32 and not exceed vocab")
        dev = _device_of(device)
        _stream(stream, dev)
        lib = _ops_lib.load()
        self.handle = _ops_lib.Logprobs()
        with torch.cuda.stream(stream):
            mem = self._memory(int(lib.bo_logprobs_size(rows, vocab, top, int(bool(entropy)))), dev)
            _check(lib.bo_logprobs_init(rows, vocab, top, int(bool(entropy)), mem.data_ptr(), mem.numel(),
                                        ctypes.byref(self.handle), _stream(None, dev)), "bo_logprobs_init")
            self._made([mem], dev)
        h = self.handle
        self.rows, self.vocab, self.top, self._ran = rows, vocab, top, 0
        self.logprobs = self._part(h.d_logprobs, torch.float32, rows)
        self.entropy = self._part(h.d_entropy, torch.float32, rows) if entropy else None
        self.top_logprobs = self._part(h.d_top_logprobs, torch.float32, rows, top)
        self.top_tokens = self._part(h.d_top_tokens, torch.int32, rows, top)
        self._ref = ctypes.byref(h)
        self._forward, self._backward = lib.bo_logprobs_forward, lib.bo_logprobs_backward

    def run(self, logits: torch.Tensor, tokens: torch.Tensor,
            temperature: float | torch.Tensor = 1.0, stream=None) -> None:
        """Log probabilities of tokens [n] (int32 or int64) under logits [n, vocab] (bfloat16 or
        float32, contiguous rows) divided by the temperature: one positive number, or float32[n].
        Autograd does not see the call, which refuses logits and temperatures that it records."""
        raw = self._on(stream)
        _unrecorded_logits(logits)
        dev = self.device
        n, ld = _rows_in(logits, "logits", self.rows, self.vocab, dev)
        step = _column(tokens, "tokens", n, _TOKENS, dev)
        heat, heats, heat_step = temperature, None, 0
        if type(heat) is not float:   # (which is quicker to ask than whether it is a tensor)
            if isinstance(temperature, torch.Tensor):
                _unrecorded_tensor(temperature, "the temperature")
                heat_step = _column(temperature, "temperature", n, _FLOAT, dev)
                heat, heats = 1.0, temperature.data_ptr() or None
            else:
                heat = float(temperature)
        if not 0.0 < heat < math.inf:
            raise ValueError("temperature must be a positive number")
        rc = self._forward(self._ref, logits.data_ptr(), _DTYPES[logits.dtype], ld, n, tokens.data_ptr(),
                           8 if tokens.dtype is torch.int64 else 4, step, heat, heats, heat_step, raw)
        if rc != OK:
            _failed(rc, "bo_logprobs_forward", dev)
        self._ran = n

    def backward(self, logits: torch.Tensor, d_logprobs: torch.Tensor | None,
                 d_entropy: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
        """The gradient of the last run's logits (the same ones, or their first rows) from those of
        its log probabilities and entropies (float32[n], either may be None).  Goes to `out`, which
        may be the logits themselves, or to memory of its own; returns it.  Tensors that autograd
        records are refused: it could not go on through the call."""
        raw = self._on(stream)
        _unrecorded_logits(logits)
        dev = self.device
        n, ld = _rows_in(logits, "logits", self._ran, self.vocab, dev)
        if d_logprobs is None and d_entropy is None:
            raise ValueError("d_logprobs or d_entropy must be given")
        if d_entropy is not None and self.entropy is None:
            raise ValueError("d_entropy needs an object with entropy=True")
        g = h = None
        g_step = h_step = 0
        if d_logprobs is not None:
            _unrecorded_tensor(d_logprobs, "d_logprobs")
            g_step, g = _column(d_logprobs, "d_logprobs", n, _FLOAT, dev), d_logprobs.data_ptr()
        if d_entropy is not None:
            _unrecorded_tensor(d_entropy, "d_entropy")
            h_step, h = _column(d_entropy, "d_entropy", n, _FLOAT, dev), d_entropy.data_ptr()
        out, ld_out = _out_for(out, logits, n, self.vocab, ld, dev, stream)
        rc = self._backward(self._ref, logits.data_ptr(), _DTYPES[logits.dtype], ld, n, g, g_step, h, h_step,
                            out.data_ptr(), ld_out, raw)
        if rc != OK:
            _failed(rc, "bo_logprobs_backward", dev)
        return out


class ExpertRouting(_Results):
    """Routing of up to `tokens` tokens to k of `experts` experts each.

    normalize   divide the chosen experts' weights by their sum (default)
    device      the current CUDA device (default)

    Results on the device after `run`: `experts` (int32[tokens, k], the likeliest first and of
    equal ones the lowest first) and `weights` (float32[tokens, k]), of the run's tokens (those
    behind them stay as they were); over the run's tokens `counts` (int32[experts]), `probs`
    (float32[experts], mean probabilities), `loss` (float32[1], the balance loss
    experts * sum(counts / counts.sum() * probs), 1 when all experts are alike) and `real`
    (int32[1], how many tokens counted).  Each run overwrites them: calls at the same time, on
    several streams or in graphs that run side by side, want an object each.

    Tokens that the mask leaves out have experts -1 and weights and gradients 0, and count
    nowhere.  A token's experts and normalized weights do not depend on how many others there are; the
    last bits of weights that are not normalized may."""

    def __init__(self, tokens: int, experts: int, k: int, *, normalize: bool = True, device=None,
                 stream=None):
        tokens, experts, k = int(tokens), int(experts), int(k)
        if not 0 <= tokens <= 1 << 28 or not 1 <= experts <= 1024:
            raise ValueError("tokens must lie in 0 .. 2**28 and experts in 1 .. 1024")
        if not 1 <= k <= min(32, experts):
            raise ValueError("k must lie in 1 .. 32 and not exceed experts")
        dev = _device_of(device)
        _stream(stream, dev)
        lib = _ops_lib.load()
        self.handle = _ops_lib.Routing()
        with torch.cuda.stream(stream):
            mem = self._memory(int(lib.bo_routing_size(tokens, experts, k)), dev)
            _check(lib.bo_routing_init(tokens, experts, k, int(bool(normalize)), mem.data_ptr(), mem.numel(),
                                       ctypes.byref(self.handle), _stream(None, dev)), "bo_routing_init")
            self._made([mem], dev)
        h = self.handle
        self.tokens, self.k, self.normalize, self._ran = tokens, k, bool(normalize), 0
        self.weights = self._part(h.d_weights, torch.float32, tokens, k)
        self.experts = self._part(h.d_experts, torch.int32, tokens, k)
        self.counts = self._part(h.d_counts, torch.int32, experts)
        self.probs = self._part(h.d_probs, torch.float32, experts)
        self.loss = self._part(h.d_loss, torch.float32, 1)
        self.real = self._part(h.d_real, torch.int32, 1)
        self._width, self._ref = experts, ctypes.byref(h)
        self._forward, self._backward = lib.bo_routing_forward, lib.bo_routing_backward

    def run(self, logits: torch.Tensor, mask: torch.Tensor | None = None, stream=None) -> None:
        """Routes by logits [n, experts] (bfloat16 or float32, contiguous rows).  mask (bool or
        uint8 [n]): tokens that are False or 0 are left out.  Autograd does not see the call, which
        refuses logits that it records."""
        raw = self._on(stream)
        _unrecorded_logits(logits)
        dev = self.device
        n, ld = _rows_in(logits, "logits", self.tokens, self._width, dev)
        at, step = None, 0
        if mask is not None:
            step, at = _column(mask, "mask", n, _MASKS, dev), mask.data_ptr() or None
        rc = self._forward(self._ref, logits.data_ptr(), _DTYPES[logits.dtype], ld, n, at, step, raw)
        if rc != OK:
            _failed(rc, "bo_routing_forward", dev)
        self._ran = n

    def backward(self, logits: torch.Tensor, d_weights: torch.Tensor | None,
                 d_loss: float | torch.Tensor = 0.0, out: torch.Tensor | None = None, *,
                 counts: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The gradient of the last run's logits (the same ones, or their first rows; `experts` and `real`
        as it left them) from those of its weights (float32[n, k], or None) and of its balance loss (a number or a float32[1]
        device tensor).  counts (int32[experts]): the experts' counts to take for the balance loss in
        place of the run's, as of several batches together.  Goes to `out`, which may be the logits
        themselves, or to memory of its own; returns it.  Tensors that autograd records are refused: it
        could not go on through the call."""
        raw = self._on(stream)
        _unrecorded_logits(logits)
        dev = self.device
        n, ld = _rows_in(logits, "logits", self._ran, self._width, dev)
        gw, steps = None, (0, 0)
        if d_weights is not None:
            if d_weights.shape != (n, self.k) or d_weights.dtype is not torch.float32 or \
                    d_weights.get_device() != dev.index:
                raise ValueError(f"d_weights must be a float32 tensor of shape ({n}, {self.k}) on {dev}")
            _unrecorded_tensor(d_weights, "d_weights")
            gw, steps = d_weights.data_ptr() or None, d_weights.stride()
        where, rate = None, d_loss
        if type(rate) is not float:
            if isinstance(d_loss, torch.Tensor):
                if d_loss.dtype != torch.float32 or d_loss.numel() != 1 or d_loss.device != dev:
                    raise ValueError(f"d_loss must be a number or a float32[1] tensor on {dev}")
                _unrecorded_tensor(d_loss, "d_loss")
                where, rate = d_loss.data_ptr(), 0.0
            else:
                rate = float(d_loss)
        if counts is not None and (counts.shape != (self._width,) or counts.dtype != torch.int32 or
                                   counts.device != dev or not counts.is_contiguous()):
            raise ValueError(f"counts must be a contiguous int32 tensor of {self._width} elements on {dev}")
        out, ld_out = _out_for(out, logits, n, self._width, ld, dev, stream)
        rc = self._backward(self._ref, logits.data_ptr(), _DTYPES[logits.dtype], ld, n, gw, *steps, rate, where,
                            None if counts is None else counts.data_ptr(), out.data_ptr(), ld_out, raw)
        if rc != OK:
            _failed(rc, "bo_routing_backward", dev)
        return out
