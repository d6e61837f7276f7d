"""Device-side drivers for stacks of HSTU layers (plumbing only).

Moves a seeded workload to the GPU and runs it through the C ABI: a forward
stack, a forward+backward training step, M-FALCON scoring (history pass
with K/V caching, then candidate microbatches against the cache), and
Stochastic Length sampling of a training batch.  Around the layers: an item
embedding that feeds a training step and takes its gradient, activation
checkpoints in 8 bits, and stacks with norms before and after each block.
Every layer step runs in libhstu.so.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional

import numpy as np
import torch

from . import hstu as H
from .workloads import Workload


def _t(a, dtype, device):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=dtype)


def _settled(device):
    """Ends a constructor: waits until what it queued has run, so that a first use on any stream
    comes after it (a fill of a gradient still queued on another stream would erase it)."""
    if device.type == "cuda" and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(device).synchronize()


def _zero(tensors, stream):
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None:
                t.zero_()


@dataclass
class DeviceWorkload:
    cfg: H.Config
    x: torch.Tensor
    offsets: torch.Tensor
    timestamps: torch.Tensor
    num_targets: Optional[torch.Tensor]
    layers: List[H.LayerWeights]
    dy: Optional[torch.Tensor]
    w: Workload

    @staticmethod
    def from_workload(w: Workload, device="cuda", with_targets=True,
                      io_dtype: int = H.HSTU_F32) -> "DeviceWorkload":
        """io_dtype: dtype of the residual stream (x, y, dy, dx)."""
        dtype_id = H.HSTU_BF16 if w.dtype == "bf16" else H.HSTU_F32
        dt = H.torch_dtype(dtype_id)
        io_dt = H.torch_dtype(io_dtype)
        cfg = H.make_config(w.d_model, w.num_heads, w.norm_N, dtype_id, w.num_pos_buckets,
                            w.num_time_buckets, max(int(w.lengths.max(initial=1)), 1), w.ln_eps,
                            io_dtype=io_dtype)
        layers = []
        for p in w.params:
            layers.append(H.LayerWeights(
                W1=_t(p.W1, dt, device), W2=_t(p.W2, dt, device),
                rab_pos=_t(p.rab_pos, torch.float32, device),
                rab_time=_t(p.rab_time, torch.float32, device),
                b1=_t(p.b1, dt, device), b2=_t(p.b2, dt, device),
                ln_gamma=_t(p.gamma, dt, device), ln_beta=_t(p.beta, dt, device)))
        nt = _t(w.num_targets, torch.int32, device) if (with_targets and w.num_targets is not None) \
            else None
        return DeviceWorkload(cfg, _t(w.x, io_dt, device), _t(w.seq_offsets, torch.int64, device),
                              _t(w.timestamps, torch.int64, device), nt, layers,
                              _t(w.dy, io_dt, device), w)

    @property
    def B(self):
        return self.offsets.numel() - 1

    @property
    def T(self):
        return self.x.shape[0]


def forward_stack(dw: DeviceWorkload, num_layers: Optional[int] = None, stream=None,
                  chain: bool = True):
    """Inference forward through the stack; returns the last layer's output.
    With an fp32 residual stream and bf16 operands, each layer's output
    epilogue also writes the bf16 copy the next layer reads (two alternating
    buffers) unless chain is False."""
    y = dw.x
    layers = dw.layers[:num_layers]
    n = len(layers)
    ch = chain and dw.cfg.io_dtype != dw.cfg.dtype and n > 1
    lo = []
    if ch:
        lt = H.torch_dtype(dw.cfg.dtype)
        lo = [H._empty((dw.T, dw.cfg.d_model), lt, dw.x.device, stream) for _ in range(2)]
    for i, w in enumerate(layers):
        y = H.fwd(dw.cfg, w, y, dw.offsets, dw.timestamps, dw.num_targets, stream=stream,
                  x_low=lo[i % 2] if ch and i > 0 else None,
                  y_low=lo[(i + 1) % 2] if ch and i + 1 < n else None)
    return y


class ItemEmbedding:
    """An item table [V][dim] (fp32 or bf16 on the device), the scale of its lookups (default
    sqrt(dim)) and its gradient: dense fp32 in `grad`, accumulated, or (rows=True, for tables
    too large for that) the last batch's non-zero rows in `row_ids`, `rows` and `count`."""

    def __init__(self, table: torch.Tensor, scale: Optional[float] = None, rows: bool = False):
        self.table = table
        self.scale = float(table.shape[1]) ** 0.5 if scale is None else float(scale)
        self.grad = None if rows else torch.zeros(table.shape, dtype=torch.float32, device=table.device)
        self.row_ids = self.rows = self.count = None
        self._room = self._room_of = None       # the rows form's buffers and the stream that they were made on
        self._captured = {}                     # those that captured calls write
        _settled(table.device)

    def lookup(self, ids, out, low=None, stream=None):
        """out[t] = scale * table[ids[t]], zero for padding ids and for columns past dim."""
        return H.embedding_fwd(self.table, ids, self.scale, out=out, low=low, stream=stream)

    def backward(self, dx, ids, stream=None):
        """Takes the gradient of lookup's out.  In the rows form the buffers of an earlier batch are
        written again (their entries past count hold nothing)."""
        if self.grad is not None:
            H.embedding_bwd(dx, ids, self.grad, self.scale, stream=stream)
            return
        V = self.table.shape[0]
        cap = min(ids.shape[0], V)
        self._make_room(cap, stream)
        row_ids, rows, self.count = self._room
        self.row_ids, self.rows = row_ids[:cap], rows[:cap]
        H.embedding_bwd_rows(dx, ids, V, self.row_ids, self.rows, self.count, self.scale, stream=stream)

    def _make_room(self, cap, stream):
        """Buffers for cap rows, on the stream that writes them.  Those that a batch needs more than are
        let go only once the streams that used them are through; those of a captured call stay."""
        dev = self.table.device
        on = None
        if dev.type == "cuda":
            on = torch.cuda.current_stream(dev) if stream is None else stream
        if self._room is None or self._room[0].shape[0] < cap:
            new = lambda *shape, t=torch.int64: H._empty(shape, t, dev, stream)
            self._room = (new(cap), new(cap, self.table.shape[1], t=torch.float32), new(1))
            self._room_of = on
        elif on != self._room_of:
            for t in self._room:
                t.record_stream(on)
        if on is not None and torch.cuda.is_current_stream_capturing():
            self._captured[id(self._room)] = self._room

    def zero_grad(self, stream=None):
        """Clears the dense gradient, on the stream that the next backward runs on."""
        _zero([self.grad], stream)


CHECKPOINTS = {"int8": H.CKPT_INT8, "e4m3": H.CKPT_E4M3}


class SavedBlocks:
    """The saved blocks of a stack's layers, or (checkpoints "int8" or "e4m3") two blocks that the
    layers take in turn and an 8-bit checkpoint of every layer but the last, whose backward is next."""

    def __init__(self, dw: DeviceWorkload, checkpoints: Optional[str]):
        if checkpoints is not None and checkpoints not in CHECKPOINTS:
            raise ValueError(f"checkpoints must be one of {sorted(CHECKPOINTS)} or None, got {checkpoints!r}")
        self.dw = dw
        self.fmt = None if checkpoints is None else CHECKPOINTS[checkpoints]
        L, dev = len(dw.layers), dw.x.device
        n = H.saved_layout(dw.cfg, dw.T)[H.SAVED_COUNT]
        blocks = [torch.empty(n, dtype=torch.uint8, device=dev)
                  for _ in range(L if self.fmt is None else min(L, 2))]
        self.blocks = [blocks[i % len(blocks)] for i in range(L)]
        self.ckpt = []
        if self.fmt is not None:
            m = H.checkpoint_bytes(dw.cfg, self.fmt, dw.T)
            self.ckpt = [torch.empty(m, dtype=torch.uint8, device=dev) for _ in range(L - 1)]

    def after_forward(self, i, stream=None):
        """Layer i's block has been filled."""
        if i < len(self.ckpt):
            H.checkpoint_save(self.dw.cfg, self.fmt, self.blocks[i], self.dw.T, self.ckpt[i], stream=stream)

    def before_backward(self, i, stream=None):
        """Layer i's block, as its backward reads it."""
        if i < len(self.ckpt):
            w = self.dw.layers[i]
            H.checkpoint_restore(self.dw.cfg, self.fmt, self.ckpt[i], self.dw.T, w.ln_gamma, w.ln_beta,
                                 self.blocks[i], stream=stream)
        return self.blocks[i]


class TrainStep:
    """Buffers for a forward+backward step over the whole stack, allocated once.

    checkpoints ("int8" or "e4m3"): hold the layers' saved activations in 8 bits between the
    forward and the backward; with an fp32 residual stream and bf16 operands neither the blocks
    nor the layers' inputs are then kept per layer (28d bytes a token and layer become 6.19d).
    embedding and ids: the stack's rows are looked up in an item table at the start of every run,
    and its gradient is taken at the end (dw.x is not used)."""

    def __init__(self, dw: DeviceWorkload, chain: bool = True, checkpoints: Optional[str] = None,
                 embedding: Optional[ItemEmbedding] = None, ids: Optional[torch.Tensor] = None):
        if (embedding is None) != (ids is None):
            raise ValueError("embedding and ids go together")
        self.dw = dw
        self.embedding, self.ids = embedding, ids
        T, L = dw.T, len(dw.layers)
        dev = dw.x.device
        self.store = SavedBlocks(dw, checkpoints)
        self.saved = self.store.blocks
        x = dw.x if embedding is None else torch.empty_like(dw.x)
        # the backward reads a layer's input only where the saved block has no operand copy of it
        keep = checkpoints is None or dw.cfg.io_dtype == dw.cfg.dtype
        bufs = [torch.empty_like(dw.x) for _ in range(L if keep else min(L, 2))]
        self.acts = [x] + [bufs[i % len(bufs)] for i in range(L)]
        self.gbuf = [torch.empty_like(dw.x), torch.empty_like(dw.x)]
        # fp32 residual stream with bf16 operands: each layer's output epilogue
        # also writes the bf16 copy the next layer reads (forward: straight
        # into that layer's saved block; backward: two alternating buffers)
        self.chain = chain and dw.cfg.io_dtype != dw.cfg.dtype
        self.xlow = []
        self.dlow = []
        if self.chain:
            self.xlow = [H.saved_views(dw.cfg, sv, T)["xlow"] for sv in self.saved]
            lt = H.torch_dtype(dw.cfg.dtype)
            self.dlow = [torch.empty(T, dw.cfg.d_model, dtype=lt, device=dev) for _ in range(2)]
        # every layer's fp32 gradients are views of one flat buffer (one
        # all-reduce in data-parallel training)
        names = ("W1", "W2", "b1", "b2", "ln_gamma", "ln_beta", "rab_pos", "rab_time")
        gnames = ("dW1", "dW2", "db1", "db2", "dgamma", "dbeta", "drab_pos", "drab_time")
        total = 0
        for w in dw.layers:
            for n in names:
                t = getattr(w, n)
                if t is not None:
                    total += (t.numel() + 63) // 64 * 64
        self.flat_grads = torch.zeros(max(total, 1), dtype=torch.float32, device=dev)
        self.grads = []
        # layer i's gradients occupy elements [sum(sizes[:i]), sum(sizes[:i+1]))
        # of the flat buffer: one bucket per layer for an overlapped all-reduce
        self.layer_grad_sizes = []
        o = 0
        for w in dw.layers:
            gb = H.LayerGradBufs()
            o0 = o
            for n, gn in zip(names, gnames):
                t = getattr(w, n)
                if t is not None:
                    setattr(gb, gn, self.flat_grads[o:o + t.numel()].view(t.shape))
                    o += (t.numel() + 63) // 64 * 64
            self.grads.append(gb)
            self.layer_grad_sizes.append(o - o0)
        _settled(dev)

    def zero_grads(self, stream=None):
        """Clears the layers' gradients, on the stream that the next run is given."""
        _zero([self.flat_grads], stream)

    def run(self, dy=None, stream=None, on_layer_grads=None):
        """Forward (keeping activations) then backward from dy; returns dX.
        on_layer_grads(i), when given, is called right after layer i's
        backward has been issued (layers in reverse order), e.g. to start the
        all-reduce of that layer's gradients, with the run's stream as the
        current one."""
        dw = self.dw
        L = len(dw.layers)
        ch = self.chain
        emb = self.embedding
        if emb is not None:
            emb.lookup(self.ids, self.acts[0], low=self.xlow[0] if ch and L else None, stream=stream)
        for i, w in enumerate(dw.layers):
            H.fwd(dw.cfg, w, self.acts[i], dw.offsets, dw.timestamps, dw.num_targets,
                  y=self.acts[i + 1], saved=self.saved[i], stream=stream,
                  x_low=self.xlow[i] if ch and (i > 0 or emb is not None) else None,
                  y_low=self.xlow[i + 1] if ch and i + 1 < L else None)
            self.store.after_forward(i, stream=stream)
        g = dw.dy if dy is None else dy
        for i in range(L - 1, -1, -1):
            out = self.gbuf[i % 2]
            H.bwd(dw.cfg, dw.layers[i], self.acts[i], g, self.store.before_backward(i, stream=stream),
                  dw.offsets, dw.timestamps,
                  dw.num_targets, dx=out, grads=self.grads[i], stream=stream,
                  dy_low=self.dlow[(i + 1) % 2] if ch and i < L - 1 else None,
                  dx_low=self.dlow[i % 2] if ch and i > 0 else None)
            if on_layer_grads is not None:
                with torch.cuda.stream(stream):
                    on_layer_grads(i)
            g = out
        if emb is not None:
            emb.backward(g, self.ids, stream=stream)
        return g

    @property
    def y(self):
        return self.acts[-1]


class NormedTrainStep:
    """Forward+backward of a stack whose blocks sit between norms: with f_i the layer without its
    residual sum (projection, attention, LayerNorm (.) U, projection) and joint i = joints[i],

        y_0 = x,  h_0 = Norm_pre(y_0);   b_i = f_i(h_i)
        y_(i+1) = y_i + s (.) (Norm_post(b_i) (.) act(gates[i])),  h_(i+1) = Norm_pre(y_(i+1))

    with Norm_pre of joint i before block i, and Norm_post, s and the gate's activation of joint
    i + 1 after it (so joints has one more entry than the stack has layers, the first joint's
    Norm_post and the last one's Norm_pre are not used).  gates: a [T][d] tensor (cfg->dtype) or
    None for each block; their gradients are left in dgates.  checkpoints: the saved blocks as in
    TrainStep; the joints' y and b (8d bytes a token and layer with an fp32 residual stream) are kept."""

    def __init__(self, dw: DeviceWorkload, joints: List[H.BlockNorm], gates=None,
                 checkpoints: Optional[str] = None):
        cfg, T, L, dev = dw.cfg, dw.T, len(dw.layers), dw.x.device
        if len(joints) != L + 1:
            raise ValueError(f"a stack of {L} layers has {L + 1} joints, got {len(joints)}")
        self.dw, self.joints = dw, joints
        self.gates = [None] * L if gates is None else list(gates)
        if len(self.gates) != L:
            raise ValueError(f"a stack of {L} layers has a gate or None for each, got {len(self.gates)}")
        dt = H.torch_dtype(cfg.dtype)
        d = cfg.d_model
        self.store = SavedBlocks(dw, checkpoints)
        self.views = [H.saved_views(cfg, b, T) for b in self.store.blocks]
        low = lambda: torch.empty(T, d, dtype=dt, device=dev)
        # a block's operand h lives in its saved block where that holds one
        self.h = [v["xlow"] if "xlow" in v else low() for v in self.views]
        self.y_ = [dw.x] + [torch.empty_like(dw.x) for _ in range(L)]
        self.b = [torch.empty_like(dw.x) for _ in range(L)]
        self.stats = [torch.empty(T, 4, dtype=torch.float32, device=dev) for _ in range(L + 1)]
        self.dgates = [None if g is None else torch.empty(T, d, dtype=dt, device=dev) for g in self.gates]
        self.grads = [H.LayerGradBufs.zeros_like(w, dev) for w in dw.layers]
        self.joint_grads = [H.BlockNormGrads.zeros_like(j) for j in joints]
        self.db, self.dz, self.do = low(), low(), low()
        self.dpre = torch.empty(T, 4 * d, dtype=dt, device=dev)
        self.dh, self.dy = torch.empty_like(dw.x), torch.empty_like(dw.x)
        _settled(dev)

    def zero_grads(self, stream=None):
        """Clears the gradients of the layers and joints, on the stream that the next run is given."""
        _zero([t for g in (*self.grads, *self.joint_grads) for t in vars(g).values()], stream)

    @property
    def y(self):
        return self.y_[-1]

    def run(self, dy=None, stream=None):
        """Forward, then backward from dy; returns dX (a buffer of this step)."""
        dw, cfg, st = self.dw, self.dw.cfg, {"stream": stream}
        L = len(dw.layers)
        g = dw.dy if dy is None else dy
        if g is None:
            raise ValueError("the workload has no dy: run needs one")
        H.block_norm_fwd(cfg, self.joints[0], self.y_[0], h=self.h[0] if L else None, stats=self.stats[0],
                         want_h=L > 0, **st)
        for i, w in enumerate(dw.layers):
            v = self.views[i]
            H.proj_in_fwd(cfg, w, self.h[i], v["pre"], v["g"], **st)
            H.attention_fwd(cfg, w.rab_pos, w.rab_time, v["g"], dw.offsets, dw.timestamps, dw.num_targets,
                            v["o"], **st)
            H.ln_gate_fwd(cfg, w.ln_gamma, w.ln_beta, v["o"], v["g"], v["z"], v["mean"], v["rstd"], **st)
            H.proj_out_fwd(cfg, w.W2, w.b2, v["z"], None, self.b[i], **st)
            self.store.after_forward(i, **st)
            last = i + 1 == L
            H.block_norm_fwd(cfg, self.joints[i + 1], self.y_[i], self.b[i], self.gates[i], y=self.y_[i + 1],
                             h=None if last else self.h[i + 1], stats=self.stats[i + 1], want_h=not last, **st)
        dh = None
        for i in range(L - 1, -1, -1):
            w, gr, v = dw.layers[i], self.grads[i], self.views[i]
            g = H.block_norm_bwd(cfg, self.joints[i + 1], self.y_[i + 1], self.b[i], self.gates[i],
                                 self.stats[i + 1], dy=g, dh=dh, dx=self.dy, db=self.db, dgate=self.dgates[i],
                                 grads=self.joint_grads[i + 1], **st)
            self.store.before_backward(i, **st)
            H.proj_out_bwd(cfg, w.W2, v["z"], self.db, self.dz, gr.dW2, gr.db2, **st)
            H.ln_gate_bwd(cfg, w.ln_gamma, w.ln_beta, self.dz, v["o"], v["g"], v["pre"], v["mean"], v["rstd"],
                          self.do, self.dpre, gr.dgamma, gr.dbeta, **st)
            H.attention_bwd(cfg, w.rab_pos, w.rab_time, v["g"], v["pre"], self.do, dw.offsets, dw.timestamps,
                            dw.num_targets, self.dpre, gr.drab_pos, gr.drab_time, **st)
            H.proj_in_bwd(cfg, w.W1, self.h[i], self.dpre, None, self.dh, gr.dW1, gr.db1, **st)
            dh = self.dh
        if L == 0:
            return g
        return H.block_norm_bwd(cfg, self.joints[0], self.y_[0], None, None, self.stats[0], dy=g, dh=dh,
                                dx=self.dy, grads=self.joint_grads[0], **st)


def _gather(src, rows: np.ndarray, out=None):
    """out[r] = src[rows[r]] through the library's row gather (the index and
    the row count are uploaded once per call; no PyTorch indexing)."""
    dev = src.device
    idx = torch.from_numpy(np.ascontiguousarray(rows, dtype=np.int64)).to(dev)
    count = torch.tensor([len(rows)], dtype=torch.int64, device=dev)
    if out is None:
        out = torch.empty((len(rows),) + tuple(src.shape[1:]), dtype=src.dtype, device=dev)
    return H.gather_rows(src, idx, count, out)


def mfalcon_score(dw: DeviceWorkload, history: int, candidates: int, microbatch: int, stream=None):
    """M-FALCON scoring of a workload whose users are `history` tokens followed
    by `candidates` tokens: one history pass caching each layer's V|K, then the
    candidates in microbatches against the cache.  Returns (y_hist, y_cand)
    with candidate rows in input order.  Row selection and reordering run in
    the library's gather kernel.
    Everything, the row selection included, runs on the stream (None: the current one)."""
    with torch.cuda.stream(stream):
        return _mfalcon_score(dw, history, candidates, microbatch)


def _mfalcon_score(dw: DeviceWorkload, history: int, candidates: int, microbatch: int):
    w = dw.w
    B = w.B
    dev = dw.x.device
    d = w.d_model
    n = history + candidates
    assert np.all(w.lengths == n)
    base = np.arange(B) * n
    hist_rows = (base[:, None] + np.arange(history)[None, :]).reshape(-1)
    x_hist = _gather(dw.x, hist_rows)
    ts_hist = _gather(dw.timestamps, hist_rows)
    hist_off = torch.arange(B + 1, dtype=torch.int64, device=dev) * history
    caches = []
    y = x_hist
    for lw in dw.layers:
        kv = torch.empty(y.shape[0], 2 * d, dtype=H.torch_dtype(dw.cfg.dtype), device=dev)
        y = H.fwd(dw.cfg, lw, y, hist_off, ts_hist, None, kv_out=kv)
        caches.append(kv)
    y_hist = y
    # microbatch k writes its B * mb_k rows (user-major) into its own slice of
    # ybuf; one gather then puts every candidate back in input order
    ybuf = torch.empty(B * candidates, d, dtype=dw.x.dtype, device=dev)
    src_rows = np.empty((B, candidates), dtype=np.int64)
    done = 0
    for k0 in range(0, candidates, microbatch):
        mb = min(microbatch, candidates - k0)
        rows = (base[:, None] + history + k0 + np.arange(mb)[None, :]).reshape(-1)
        xc = _gather(dw.x, rows)
        tc = _gather(dw.timestamps, rows)
        coff = torch.arange(B + 1, dtype=torch.int64, device=dev) * mb
        out = ybuf[done:done + B * mb]
        for li, lw in enumerate(dw.layers):
            last = li == len(dw.layers) - 1
            xc = H.fwd_cached(dw.cfg, lw, xc, coff, tc, caches[li], hist_off, ts_hist,
                              y=out if last else None)
        src_rows[:, k0:k0 + mb] = done + np.arange(B)[:, None] * mb + np.arange(mb)[None, :]
        done += B * mb
    y_cand = _gather(ybuf, src_rows.reshape(-1))
    return y_hist, y_cand


class StochasticLength:
    """Stochastic Length sampling of a jagged batch on the device, with
    buffers of the input's capacity allocated once.  `run` launches the
    sampler and the row gathers without synchronising; `batch` reads the
    sampled row count (one 8-byte device-to-host copy) and returns a
    DeviceWorkload of the sampled batch (weights and config shared)."""

    def __init__(self, dw: DeviceWorkload, alpha: float, max_len: Optional[int] = None):
        self.dw = dw
        self.sub_len = H.sl_subsequence_length(int(max_len or dw.cfg.max_seq_len), alpha)
        dev = dw.x.device
        self.new_offsets = torch.empty(dw.B + 1, dtype=torch.int64, device=dev)
        self.gather_index = torch.empty(max(dw.T, 1), dtype=torch.int64, device=dev)
        self.x = torch.empty_like(dw.x)
        self.timestamps = torch.empty_like(dw.timestamps)
        self._stream = None                     # of the last run

    def run(self, keep_draw: torch.Tensor, keys: torch.Tensor, stream=None):
        dw = self.dw
        self._stream = torch.cuda.current_stream(dw.x.device) if stream is None else stream
        H.stochastic_length(dw.offsets, dw.num_targets, self.sub_len, keep_draw, keys,
                            self.new_offsets, self.gather_index, stream=stream)
        count = self.new_offsets[dw.B:]
        H.gather_rows(dw.x, self.gather_index, count, self.x, stream=stream)
        H.gather_rows(dw.timestamps, self.gather_index, count, self.timestamps, stream=stream)

    def batch(self) -> DeviceWorkload:
        dw = self.dw
        with torch.cuda.stream(self._stream):   # comes after the run
            t = int(self.new_offsets[dw.B].item())
        return DeviceWorkload(dw.cfg, self.x[:t], self.new_offsets, self.timestamps[:t],
                              dw.num_targets, dw.layers, None, dw.w)
