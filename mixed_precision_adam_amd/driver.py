"""Host-side sequencing of one rank's ZeRO step over the C ABI.

Holds the device buffers of a simulated data-parallel rank (PyTorch
allocations) and calls the library entry points in the order of the step:
flatten -> square-norm -> (simulated all-reduce + decision) -> AdamW.  Three
ways of sequencing it: ``rank_step`` (decision on the host after a 16-byte
readback), ``DeviceDecision`` (decision on the GPU, nothing waits on the
host) and ``BucketPipeline`` (flatten + norm partials in constant-capacity
buckets as gradients arrive on a producer stream).  ``TensorList`` and
``ListDecision`` step many tensors where they lie.  ``TokenEmbedding``,
``LayerNorm`` and ``LossHead`` compute at a model's ends and norms, where the
gradients come from.  No arithmetic of the method happens here: every step is a library call.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import (ZERO_BF16, ZERO_FP16, ZERO_FP32, ZERO_LIST_HAS_PARAMS, ZERO_LIST_WHOLE_STATE, ZERO_STATE_8BIT,
               ZERO_STATE_ARRAYS, ZERO_STATE_NONE, ZERO_STATE_TILE, ZERO_STATE_TILED, _buf, read_step_state,
               zero_adamw_hparams, zero_adamw_step, zero_adamw_step_dev, zero_adamw_step_tiled,
               zero_adamw_step_tiled_dev, zero_bucket_segments, zero_embed_forward, zero_embed_grad,
               zero_embed_grad_workspace_bytes, zero_flatten_grads, zero_flatten_grads_partials,
               zero_flatten_grads_sqnorm, zero_flatten_partials_count, zero_flatten_plan, zero_grad_sqnorm,
               zero_grad_sqnorm_workspace_bytes, zero_layernorm_forward, zero_layernorm_grad,
               zero_layernorm_grad_workspace_bytes, zero_list_adamw8_step, zero_list_adamw8_step_dev,
               zero_list_adamw_step, zero_list_adamw_step_dev, zero_list_decision_dev, zero_list_grad_sqnorm,
               zero_list_grad_sqnorm_workspace_bytes, zero_list_plan, zero_list_repoint, zero_list_state8_pack,
               zero_list_state8_unpack, zero_list_tensor, zero_loss_head, zero_loss_head_grad,
               zero_loss_head_workspace_bytes, zero_loss_head_workspace_bytes_for, zero_shard_layout,
               zero_sqnorm_reduce, zero_state8_bytes, zero_state_tile, zero_state_tiled_numel, zero_state_untile,
               zero_step_decision, zero_step_decision_dev, zero_step_state_init)

_FORMAT = {torch.bfloat16: ZERO_BF16, torch.float16: ZERO_FP16, torch.float32: ZERO_FP32}
_ADDRESS = (int, type(None))  # what a call takes in place of a tensor
_TORCH16 = {ZERO_BF16: torch.bfloat16, ZERO_FP16: torch.float16}


# The current stream's handle without building a torch.cuda.Stream: 0.1 instead of 2.7 us, in calls of 5.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


@dataclass
class AdamWConfig:
    lr: float = 1e-4
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    max_norm: float = 1.0


@dataclass
class ScalerState:
    """Dynamic loss scale (1.0 and no growth for bf16 training)."""
    scale: float = 1.0
    good_steps: int = 0
    growth_interval: int = 2**31 - 1
    adam_step: int = 0  # Adam t of the last applied update


class RankShard:
    """One simulated rank: the flat 16-bit grad shard, the fp32 master/m/v state (three arrays, or one
    tiled array when ``tiled``), the 16-bit param shard (bf16, or fp16 with ``param_dtype=ZERO_FP16``) and
    the norm scratch."""

    def __init__(self, numels, world: int, rank: int, grad_dtype: int, device="cuda", sources=None,
                 tiled: bool = False, fused: bool = False, param_dtype: int = ZERO_BF16):
        self.layout, self.segments = zero_shard_layout(numels, world, rank)
        self.grad_dtype = grad_dtype
        self.device = torch.device(device)
        self.tiled = tiled
        self.fused = fused  # flatten and square-norm in one pass
        n = self.layout.shard_numel
        self.n = n
        self.grad = torch.empty(n, dtype=_TORCH16[grad_dtype], device=self.device)
        if tiled:
            self.state = torch.zeros(zero_state_tiled_numel(n), dtype=torch.float32, device=self.device)
        else:
            self.master = torch.zeros(n, dtype=torch.float32, device=self.device)
            self.m = torch.zeros(n, dtype=torch.float32, device=self.device)
            self.v = torch.zeros(n, dtype=torch.float32, device=self.device)
        self.param_dtype = param_dtype
        self.param = torch.zeros(n, dtype=_TORCH16[param_dtype], device=self.device)
        self.ws_bytes = zero_grad_sqnorm_workspace_bytes(n)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        # square-norm (double) and non-finite flag (int32) side by side: one 16-byte readback per step
        self.norm_dev = torch.zeros(2, dtype=torch.float64, device=self.device)
        self.sq_dev = self.norm_dev.data_ptr()
        self.flag_dev = self.norm_dev.data_ptr() + 8
        self.norm_host = torch.zeros(2, dtype=torch.float64).pin_memory()
        self._norm_np = self.norm_host.numpy()
        self.seg_table = None
        self.n_segs = 0
        if sources is not None:
            self.set_sources(sources)

    # -- state access (initialisation and checks) -------------------------------------------------

    def load_master(self, master: torch.Tensor) -> None:
        """Sets the fp32 master shard (device tensor of n floats); m and v start at zero."""
        if self.tiled:
            zeros = torch.zeros(self.n, dtype=torch.float32, device=self.device)
            zero_state_tile(master, zeros, zeros, self.state, self.n)
        else:
            self.master.copy_(master)
            self.m.zero_()
            self.v.zero_()

    def state_views(self, lo: int = 0, hi: int | None = None):
        """(master, m, v) device tensors for shard elements [lo, hi).  With the tiled layout lo and hi must
        be tile-aligned (hi may be n)."""
        hi = self.n if hi is None else hi
        if not self.tiled:
            return self.master[lo:hi], self.m[lo:hi], self.v[lo:hi]
        t = ZERO_STATE_TILE
        assert lo % t == 0 and (hi % t == 0 or hi == self.n)
        tiles = self.state.view(-1, 3, t)[lo // t: (hi + t - 1) // t]
        cnt = hi - lo
        return tuple(tiles[:, k, :].reshape(-1)[:cnt] for k in range(3))

    def read_state(self):
        """Whole (master, m, v) as separate device tensors (untiling when needed)."""
        if not self.tiled:
            return self.master, self.m, self.v
        out = [torch.empty(self.n, dtype=torch.float32, device=self.device) for _ in range(3)]
        zero_state_untile(self.state, *out, self.n)
        return tuple(out)

    # -- the step ------------------------------------------------------------------------------

    def set_sources(self, sources) -> None:
        """sources[t]: device tensor (or address) of tensor t's gradient; only tensors that land in the
        shard need one."""
        ptrs = [sources[t] if sources[t] is not None else 0 for t in range(len(sources))]
        table = zero_flatten_plan(self.segments, ptrs)
        self.n_segs = len(self.segments)
        host = torch.frombuffer(bytearray(table), dtype=torch.uint8) if table else torch.zeros(32, dtype=torch.uint8)
        self.seg_table = host.to(self.device)
        self._sources = sources  # keep the tensors alive

    def flatten(self, stream=None) -> None:
        if self.fused:
            zero_flatten_grads_sqnorm(self.seg_table, self.n_segs, self.grad_dtype, self.grad, self.n, self.ws,
                                      self.ws_bytes, self.sq_dev, self.flag_dev, stream)
        else:
            zero_flatten_grads(self.seg_table, self.n_segs, self.grad_dtype, self.grad, self.n, stream)

    def sqnorm(self, stream=None) -> None:
        """Square-norm and non-finite flag of the shard as it stands (a separate pass)."""
        zero_grad_sqnorm(self.grad, self.grad_dtype, self.n, self.ws, self.ws_bytes, self.sq_dev, self.flag_dev,
                         stream)

    def readback(self, stream=None) -> None:
        """Queue the 16-byte copy of the square-norm and flag to pinned host memory on `stream` (the stream
        the norm ran on, so the copy is ordered after it and a wait on that stream covers both)."""
        stream = stream or torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            self.norm_host.copy_(self.norm_dev, non_blocking=True)

    def norm_result(self):
        """Host copies of the last sqnorm; call after the stream has been synchronized."""
        return float(self._norm_np[0]), int(self._norm_np[1:2].view(np.int32)[0])

    def adamw_dev(self, step_state, stream=None) -> None:
        """The update with its scalars taken from a device-resident zero_step_state."""
        if self.tiled:
            zero_adamw_step_tiled_dev(self.grad, self.grad_dtype, self.state, self.param, self.n, step_state, stream,
                                      param_dtype=self.param_dtype)
        else:
            zero_adamw_step_dev(self.grad, self.grad_dtype, self.master, self.m, self.v, self.param, self.n,
                                step_state, stream, param_dtype=self.param_dtype)

    def adamw(self, cfg: AdamWConfig, grad_scale: float, step: int, stream=None) -> None:
        kw = dict(lr=cfg.lr, beta1=cfg.beta1, beta2=cfg.beta2, eps=cfg.eps, weight_decay=cfg.weight_decay,
                  grad_scale=grad_scale, step=step, stream=stream, param_dtype=self.param_dtype)
        if self.tiled:
            zero_adamw_step_tiled(self.grad, self.grad_dtype, self.state, self.param, self.n, **kw)
        else:
            zero_adamw_step(self.grad, self.grad_dtype, self.master, self.m, self.v, self.param, self.n, **kw)


class DeviceDecision:
    """Device-resident decision for a set of simulated ranks: their square-norms and flags land side by side
    in one device buffer, one GPU thread takes the decision, and the update kernels read it from device
    memory.  A step then needs no host round trip (and can be captured in a HIP graph)."""

    def __init__(self, shards, cfg: AdamWConfig, loss_scale: float = 1.0, growth_interval: int = 2**31 - 1):
        n = len(shards)
        dev = shards[0].device
        self.shards = shards
        self.cfg = cfg
        self.norms = torch.zeros(n + (n + 1) // 2, dtype=torch.float64, device=dev)  # n doubles, then n int32
        self.sq_base = self.norms.data_ptr()
        self.flag_base = self.sq_base + 8 * n
        for r, sh in enumerate(shards):
            sh.sq_dev = self.sq_base + 8 * r
            sh.flag_dev = self.flag_base + 4 * r
        self.state = torch.zeros(16, dtype=torch.float64, device=dev)  # 128 bytes >= sizeof(zero_step_state)
        zero_step_state_init(self.state, loss_scale, growth_interval)

    def step(self, flatten: bool = True, stream=None) -> None:
        """Enqueues one whole step; nothing waits on the host."""
        stream = stream or torch.cuda.current_stream()
        for sh in self.shards:
            if flatten:
                sh.flatten(stream)
            if not (flatten and sh.fused):
                sh.sqnorm(stream)
        c = self.cfg
        zero_step_decision_dev(self.sq_base, self.flag_base, len(self.shards), c.max_norm, self.state, lr=c.lr,
                               beta1=c.beta1, beta2=c.beta2, eps=c.eps, weight_decay=c.weight_decay, stream=stream)
        for sh in self.shards:
            sh.adamw_dev(self.state, stream)

    def read(self) -> dict:
        """The decided state (synchronizes)."""
        return read_step_state(self.state)


class BucketPipeline:
    """Constant-capacity buckets for one rank's shard: as backward produces gradients (last tensors first),
    each bucket of at most `bucket_numel` shard elements is flattened on the compute stream as soon as its
    source tensors are ready, overlapping with the production of the next bucket, and leaves its partial
    square-sums and flags in its own slice of one partials buffer.  One reduction folds them all (window
    order), the device decision follows, and the update runs over the whole shard (clipping needs the global
    norm first).  The bucket capacity is fixed: it does not grow with the model."""

    def __init__(self, shard: "RankShard", sources, bucket_numel: int, cfg: AdamWConfig, loss_scale: float = 1.0,
                 growth_interval: int = 2**31 - 1):
        assert bucket_numel > 0 and bucket_numel % 8 == 0, "whole 16-byte vectors per bucket"
        self.sh = shard
        self.cfg = cfg
        self.sources = sources
        n = shard.n
        self.windows = [(a, min(n, a + bucket_numel)) for a in range(0, n, bucket_numel)] or [(0, 0)]
        dev = shard.device
        counts = [zero_flatten_partials_count(b - a) for a, b in self.windows]
        self.part_first = np.cumsum([0] + counts).tolist()  # window k owns partials [first[k], first[k+1])
        total = max(self.part_first[-1], 1)
        self.part_sum = torch.zeros(total, dtype=torch.float64, device=dev)
        self.part_flag = torch.zeros(total, dtype=torch.int32, device=dev)
        self.norms = torch.zeros(2, dtype=torch.float64, device=dev)  # the rank's square-norm, then its flag
        self.tables, self.counts, self.tensors = [], [], []
        for a, b in self.windows:
            segs = zero_bucket_segments(shard.segments, a, b - a)
            ptrs = [sources[t] if sources[t] is not None else 0 for t in range(len(sources))]
            blob = zero_flatten_plan(segs, ptrs)
            table = torch.frombuffer(bytearray(blob), dtype=torch.uint8) if blob else torch.zeros(32, dtype=torch.uint8)
            self.tables.append(table.to(dev))
            self.counts.append(len(segs))
            self.tensors.append(sorted({sg.tensor for sg in segs}))
        self.state = torch.zeros(16, dtype=torch.float64, device=dev)
        zero_step_state_init(self.state, loss_scale, growth_interval)
        self.events = [torch.cuda.Event() for _ in self.windows]

    def step(self, produce=None, producer=None, stream=None) -> None:
        """One step.  `produce(tensor_indices, stream)` writes those source tensors' gradients (stands in for
        backward); it runs on `producer` in backward order, one bucket at a time, each followed by an event
        the compute stream waits for.  Without `produce` the sources are taken as ready."""
        stream = stream or torch.cuda.current_stream()
        if produce is not None:
            self.launch_production(produce, producer, stream)
        self.reduce_all(stream, wait=produce is not None)
        self.decide(stream)
        self.sh.adamw_dev(self.state, stream)

    def launch_production(self, produce, producer, stream) -> None:
        """Queues gradient production on `producer`, last bucket first, with one event per bucket."""
        producer.wait_stream(stream)  # the previous step has finished reading the sources
        done = set()
        for k in range(len(self.windows) - 1, -1, -1):
            need = [t for t in self.tensors[k] if t not in done]
            produce(need, producer)
            done.update(need)
            self.events[k].record(producer)

    def reduce_all(self, stream=None, wait: bool = False) -> None:
        """Flatten + norm partials of every bucket, last first; with `wait` each waits for its event."""
        for k in range(len(self.windows) - 1, -1, -1):
            if wait:
                stream.wait_event(self.events[k])
            self.reduce_bucket(k, stream)

    def reduce_bucket(self, k: int, stream=None) -> None:
        """Flatten of bucket k, leaving its partial square-sums and flags in its slice of the partials."""
        sh = self.sh
        a, b = self.windows[k]
        f = self.part_first[k]
        zero_flatten_grads_partials(self.tables[k], self.counts[k], sh.grad_dtype, sh.grad.data_ptr() +
                                    a * sh.grad.element_size(), b - a, self.part_sum.data_ptr() + 8 * f,
                                    self.part_flag.data_ptr() + 4 * f, stream)

    def decide(self, stream=None) -> None:
        """Folds every bucket's partials (window order), then the device decision."""
        c = self.cfg
        sq, fl = self.norms.data_ptr(), self.norms.data_ptr() + 8
        zero_sqnorm_reduce(self.part_sum, self.part_flag, self.part_first[-1], sq, fl, stream)
        zero_step_decision_dev(sq, fl, 1, c.max_norm, self.state, lr=c.lr, beta1=c.beta1, beta2=c.beta2, eps=c.eps,
                               weight_decay=c.weight_decay, stream=stream)

    def read(self) -> dict:
        return read_step_state(self.state)


class TensorList:
    """A planned list of tensors: gradients read and parameters written where they lie, with fp32 state (``state``
    tiled, or ``master``/``m``/``v``), 8-bit state (``state8``) or none (norm only). Every argument is a list with one
    contiguous GPU tensor per list entry; ``grads`` and ``params`` may hold views at any element offset, and a
    gradient may be None (no gradient in this step: that tensor is left as it is, though the step counts for its
    bias correction, which has one count for the whole list). Calls run on the current stream of the tensors'
    device unless a stream is given. The list keeps the tensors, its table and the norm's workspace alive: keep it
    until its calls are done, and give calls that may overlap in time lists of their own. It names the memory that
    the tensors had when it was made: parameters that get other memory (``p.data = ...``) need another list. A
    captured graph replays what the table names at the time: `set_grads` between replays is seen, and is itself not
    for capture."""

    def __init__(self, numels, grads=None, params=None, *, state=None, state8=None, master=None, m=None, v=None,
                 groups=None, n_groups: int = 1):
        given = [x for x in (grads, params, state, state8, master, m, v) if x is not None]
        for x in given + ([groups] if groups is not None else []):
            if len(x) != len(numels):
                raise ValueError(f"{len(x)} entries for {len(numels)} tensors")
        devices = {t.device for x in given for t in x if t is not None}
        if len(devices) > 1 or any(d.type != "cuda" for d in devices):
            raise ValueError(f"the tensors of a list belong on one GPU, got {sorted(map(str, devices))}")
        if (state is not None) + (state8 is not None) + any(x is not None for x in (master, m, v)) > 1:
            raise ValueError("one kind of state: tiled, 8-bit or master/m/v")
        for x, kinds in ((grads, _FORMAT), (params, _FORMAT), (state, {torch.float32}), (state8, {torch.uint8}),
                         (master, {torch.float32}), (m, {torch.float32}), (v, {torch.float32})):
            bad = [t.dtype for t in x or () if t is not None and t.dtype not in kinds]
            if bad:
                raise ValueError(f"dtype {bad[0]} where one of {sorted(map(str, kinds))} is needed")
        layout = (ZERO_STATE_TILED if state is not None else ZERO_STATE_8BIT if state8 is not None else
                  ZERO_STATE_ARRAYS if any(x is not None for x in (master, m, v)) else ZERO_STATE_NONE)
        self.device = devices.pop() if devices else torch.device("cuda", torch.cuda.current_device())
        state = next((x for x in (state, state8, master) if x is not None), None)
        self._kept = [tuple(x) for x in (params, state, m, v) if x is not None]  # the table names these tensors
        self._grads = list(grads) if grads is not None else [None] * len(numels)
        self._recs = (zero_list_tensor * len(numels))()
        state_bytes = (zero_state8_bytes if state8 is not None else lambda n: 4 * zero_state_tiled_numel(n)
                       if layout == ZERO_STATE_TILED else 4 * n)
        for k, rec in enumerate(self._recs):
            n = max(int(numels[k]), 0)
            rec.numel, rec.layout, rec.group = int(numels[k]), layout, groups[k] if groups is not None else 0
            if params is not None and params[k] is not None:
                rec.param, rec.pdt = _buf(params[k], n * params[k].element_size()), _FORMAT[params[k].dtype]
            rec.state = _buf(state[k], state_bytes(n)) if state is not None else None
            rec.m = _buf(m[k], 4 * n) if m is not None else None
            rec.v = _buf(v[k], 4 * n) if v is not None else None
        self._point(self._grads)
        self.list, self._host = zero_list_plan(self._recs, n_groups)
        self.table = torch.frombuffer(self._host, dtype=torch.uint8).to(self.device)
        self.list.table_dev = self.table.data_ptr()
        self.ws_bytes = zero_list_grad_sqnorm_workspace_bytes(self.list)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.state8 = state8 is not None

    def _point(self, grads) -> None:
        found = [(None, ZERO_BF16) if g is None else (_buf(g, max(rec.numel, 0) * g.element_size()), _FORMAT[g.dtype])
                 for g, rec in zip(grads, self._recs)]  # all of them checked before any is taken
        for rec, (address, dtype) in zip(self._recs, found):
            rec.grad, rec.gdt = address, dtype

    def set_grads(self, grads) -> None:
        """Other gradient tensors (or None) for the coming steps, on whatever stream: rewrites the table's descriptors
        and lets the old gradients go.  Steps in flight read both, on streams that the list does not know (a graph's
        replay, say), so the host waits for the device first."""
        if len(grads) != len(self._recs):
            raise ValueError(f"{len(grads)} gradients for {len(self._recs)} tensors")
        bad = [g for g in grads if g is not None and (g.device != self.device or g.dtype not in _FORMAT)]
        if bad:
            raise ValueError(f"gradients belong on {self.device} in bf16, fp16 or fp32, got {bad[0].dtype} on "
                             f"{bad[0].device}")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("set_grads cannot be captured: the table is written from the host")
        self._point(grads)
        try:
            zero_list_repoint(self._recs, self._host, self.list)
            torch.cuda.synchronize(self.device)
            n = self.list.grads_bytes
            if n:  # a copy from pageable memory: in place when it returns
                self.table[:n].copy_(torch.frombuffer(self._host, dtype=torch.uint8, count=n))
        except Exception:
            self._point(self._grads)  # the device's table still names them
            zero_list_repoint(self._recs, self._host, self.list)
            raise
        self._grads = list(grads)

    def _call(self, fn, *args, stream=None) -> None:
        if stream is None:
            stream = _current_raw_stream(self.device.index)
        elif not isinstance(stream, int) and getattr(stream, "device", self.device) != self.device:
            raise ValueError(f"a stream of {stream.device} for a list on {self.device}")
        if torch.cuda.current_device() == self.device.index:
            fn(*args, stream)
        else:  # kernels are launched from the device that holds the tensors
            with torch.cuda.device(self.device):
                fn(*args, stream)

    def _here(self, a, b) -> None:
        at = self.device.index
        if (isinstance(a, _ADDRESS) or a.get_device() == at) and (isinstance(b, _ADDRESS) or b.get_device() == at):
            return
        devices = " and ".join(str(t.device) for t in (a, b) if not isinstance(t, _ADDRESS))
        raise ValueError(f"buffers on {devices} for a list on {self.device}")

    def grad_sqnorm(self, sqnorm_out, nonfinite_out, stream=None) -> None:
        """fp64 sum of squares and inf/NaN flag over every gradient."""
        self._here(sqnorm_out, nonfinite_out)
        self._call(zero_list_grad_sqnorm, self.list, self.ws, self.ws_bytes, sqnorm_out, nonfinite_out, stream=stream)

    def adamw(self, hparams, stream=None, seed: int = 0) -> None:
        """The update with host scalars (zero_list_hparams); `seed` sets the rounding of 8-bit moments."""
        if self.state8:
            self._call(zero_list_adamw8_step, self.list, hparams, seed, stream=stream)
        else:
            self._call(zero_list_adamw_step, self.list, hparams, stream=stream)

    def adamw_dev(self, step_state, group_scalars, stream=None, seed: int = 0) -> None:
        """The update with the scalars of zero_list_decision_dev."""
        self._here(step_state, group_scalars)
        if self.state8:
            self._call(zero_list_adamw8_step_dev, self.list, step_state, group_scalars, seed, stream=stream)
        else:
            self._call(zero_list_adamw_step_dev, self.list, step_state, group_scalars, stream=stream)

    def _same_device(self, other: "TensorList") -> None:
        if other.device != self.device:
            raise ValueError(f"lists on {self.device} and {other.device}: a conversion runs on one GPU")

    def pack8(self, target: "TensorList", stream=None) -> None:
        """This list's fp32 state into the 8-bit state of `target` (a list of the same sizes on the same GPU, its
        state in memory of its own); of master, m and v, one that this list does not have becomes zeros there."""
        self._same_device(target)
        self._call(zero_list_state8_pack, self.list, target.list, stream=stream)

    def unpack8(self, target: "TensorList", stream=None) -> None:
        """This list's 8-bit state into the fp32 state of `target` (in memory of its own): those of master, m and v
        that it has."""
        self._same_device(target)
        self._call(zero_list_state8_unpack, self.list, target.list, stream=stream)


class ListDecision:
    """Device-resident steps over a TensorList: norm, decision (with the scalars of every group) and update are
    queued back to back with no host round trip, and can be captured in a HIP graph.  `cfgs`: one AdamWConfig for each
    group, read at every step (a captured step keeps those of its capture).  One norm over all of them is clipped, to
    their max_norm (the same in each) unless `max_norm` is given."""

    def __init__(self, tensors: TensorList, cfgs, max_norm: float | None = None, loss_scale: float = 1.0,
                 growth_interval: int = 2**31 - 1, seed: int = 0):
        dev = tensors.device
        self.tensors, self.seed = tensors, seed
        self.cfgs, self._norm_given = list(cfgs), max_norm is not None
        if len(self.cfgs) != tensors.list.n_groups:
            raise ValueError(f"{len(self.cfgs)} configurations for {tensors.list.n_groups} groups")
        whole = ZERO_LIST_HAS_PARAMS | ZERO_LIST_WHOLE_STATE
        if tensors.list.n_tensors and (tensors.list.state == 0 or tensors.list.flags & whole != whole):
            raise ValueError("a step needs a param, a master and both moments for every tensor")
        self.max_norm, self._seen, self._seen_norms = max_norm, [None] * len(self.cfgs), None
        self.hparams = (zero_adamw_hparams * len(self.cfgs))()
        self._follow()
        self.norms = torch.zeros(2, dtype=torch.float64, device=dev)  # square-norm, then its flag
        self._sq, self._flag = self.norms.data_ptr(), self.norms.data_ptr() + 8
        self.state = torch.zeros(16, dtype=torch.float64, device=dev)
        self.groups = torch.zeros(12 * len(self.hparams), dtype=torch.float32, device=dev)
        with torch.cuda.device(dev):
            zero_step_state_init(self.state, loss_scale, growth_interval)
            torch.cuda.current_stream().synchronize()  # the first step may come on any stream

    def _follow(self) -> None:
        """Takes over what changed in the configurations since it last looked."""
        if not self._norm_given:
            norms = [c.max_norm for c in self.cfgs]
            if norms != self._seen_norms:
                if len(set(norms)) != 1:
                    raise ValueError(f"the configurations differ in max_norm ({norms}): give one as an argument")
                self.max_norm, self._seen_norms = norms[0], norms
        for k, c in enumerate(self.cfgs):
            now = (c.lr, c.beta1, c.beta2, c.eps, c.weight_decay)
            if now != self._seen[k]:
                self.hparams[k] = zero_adamw_hparams(*now, 1.0, 1)
                self._seen[k] = now

    def step(self, stream=None) -> None:
        """Enqueues one whole step with the configurations as they are now; nothing waits on the host."""
        self._follow()
        self.tensors.grad_sqnorm(self._sq, self._flag, stream)
        self.tensors._call(zero_list_decision_dev, self._sq, self._flag, 1, self.max_norm, self.hparams, self.state,
                           self.groups, stream=stream)
        self.tensors.adamw_dev(self.state, self.groups, stream, self.seed)

    def read(self) -> dict:
        """The decided state of the last step queued, on whatever stream (synchronizes the device)."""
        torch.cuda.synchronize(self.tensors.device)
        return read_step_state(self.state)


class _Operator:
    """An operator over tensors of one GPU: its calls run on the current stream of that GPU unless a stream is given.
    It keeps its tensors and its workspace alive: keep it until its calls are done, and give calls that may overlap in
    time (two streams, two captured graphs) operators of their own.  Autograd does not see the calls: tensors that
    require gradients are taken like others, and results carry no history."""

    ws, ws_bytes = None, 0

    def _on(self, *tensors) -> None:
        at = self.device.index
        for t in tensors:
            if t is not None and t.get_device() != at:
                raise ValueError(f"a tensor on {t.device} for an operator on {self.device}")

    def _call(self, fn, *args, stream=None, **more) -> None:
        if stream is None:
            stream = _current_raw_stream(self.device.index)
        elif not isinstance(stream, int) and getattr(stream, "device", self.device) != self.device:
            raise ValueError(f"a stream of {stream.device} for an operator on {self.device}")
        if _current_device() == self.device.index:
            fn(*args, stream=stream, **more)
        else:  # kernels are launched from the device that holds the tensors
            with torch.cuda.device(self.device):
                fn(*args, stream=stream, **more)

    def _workspace(self, nbytes: int, workspace) -> None:
        """A workspace of its own, or a part of one that is shared with operators whose calls do not overlap."""
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._on(workspace)
        if workspace.dtype != torch.uint8 or workspace.numel() < nbytes:
            raise ValueError(f"a workspace of {nbytes} bytes (uint8) is needed")
        self.ws, self.ws_bytes = workspace, nbytes


class TokenEmbedding(_Operator):
    """Rows of `table` for tokens, times `scale`, and the table's gradient.  A rank that holds a slice of the vocabulary
    names its first row: tokens outside the slice get zeros, and give no gradient.  `max_tokens`: the most that one
    call of `grad` takes (0: no gradients, no workspace)."""

    def __init__(self, table, *, max_tokens: int = 0, scale: float = 1.0, first_row: int = 0, workspace=None):
        self.table, self.scale, self.first_row, self.max_tokens = table, float(scale), first_row, max_tokens
        self.device = table.device
        if max_tokens:
            need = zero_embed_grad_workspace_bytes(max_tokens, *table.shape)
            if need == 0:
                raise ValueError(f"{max_tokens} tokens over a table of {tuple(table.shape)}: out of range")
            self._workspace(need, workspace)

    def forward(self, ids, out, stream=None) -> None:
        """out[t] = scale * table[ids[t] - first_row]."""
        self._on(ids, out)
        self._call(zero_embed_forward, self.table, ids, out, scale=self.scale, first_row=self.first_row, stream=stream)

    def grad(self, ids, out_grad, table_grad, accumulate: bool = False, stream=None) -> None:
        """The table's gradient (any format and row stride), in place of what `table_grad` holds or added to it."""
        if not self.max_tokens:
            raise ValueError("made without gradients (max_tokens=0)")
        self._on(ids, out_grad, table_grad)
        if table_grad.shape != self.table.shape:
            raise ValueError(f"a gradient of {tuple(table_grad.shape)} for a table of {tuple(self.table.shape)}")
        if out_grad.shape[0] > self.max_tokens:
            raise ValueError(f"{out_grad.shape[0]} tokens, made for {self.max_tokens} (max_tokens)")
        self._call(zero_embed_grad, ids, out_grad, table_grad, self.ws, self.ws_bytes, scale=self.scale,
                   first_row=self.first_row, accumulate=accumulate, stream=stream)


class LayerNorm(_Operator):
    """Layer norm over the rows of a matrix (`mean=False`: without subtracting the mean), and its gradients.  Their
    workspace takes 4 KiB a column, 16 in rows of up to 1024: norms whose calls do not overlap in time may share one
    (`workspace=other.ws`), and with `gradients=False`, for the forward pass alone, there is none."""

    def __init__(self, weight, bias=None, *, eps: float = 1e-5, mean: bool = True, gradients: bool = True,
                 workspace=None):
        self.weight, self.bias, self.eps, self.mean = weight, bias, float(eps), bool(mean)
        self.gradients, self.device = bool(gradients), weight.device
        self._on(bias)
        need = zero_layernorm_grad_workspace_bytes(2**31 - 1, weight.numel())  # enough for any number of rows
        if need == 0:
            raise ValueError(f"rows of {weight.numel()} elements: out of range")
        if gradients:
            self._workspace(need, workspace)

    def forward(self, x, out, mean=None, rstd=None, stream=None) -> None:
        """The statistics of each row are left in `mean` and `rstd` (fp32) where these are given."""
        self._on(x, out, mean, rstd)
        self._call(zero_layernorm_forward, x, self.weight, self.bias, out, mean, rstd, eps=self.eps, center=self.mean,
                   stream=stream)

    def grad(self, x, out_grad, mean, rstd, x_grad=None, weight_grad=None, bias_grad=None, accumulate: bool = False,
             stream=None) -> None:
        """Those gradients that are given a place; `accumulate`: the weight's and the bias's are added to theirs."""
        if not self.gradients:
            raise ValueError("made without gradients")
        self._on(x, out_grad, mean, rstd, x_grad, weight_grad, bias_grad)
        self._call(zero_layernorm_grad, x, out_grad, self.weight, mean, rstd, x_grad, weight_grad, bias_grad, self.ws,
                   self.ws_bytes, center=self.mean, accumulate=accumulate, stream=stream)


class LossHead(_Operator):
    """Softmax cross entropy of the linear head `table` (words x columns, 16-bit) over hidden rows, without keeping the
    scores, and its gradients.  Labels outside the vocabulary do not count.  `max_tokens`: the most that one call
    takes; `gradients=False`: a smaller workspace, for losses alone."""

    def __init__(self, table, *, max_tokens: int, gradients: bool = True, workspace=None):
        self.table, self.max_tokens, self.gradients = table, max_tokens, bool(gradients)
        self.device = table.device
        if zero_loss_head_workspace_bytes(max_tokens, *table.shape, gradients) == 0:
            raise ValueError(f"{max_tokens} tokens over a table of {tuple(table.shape)}: out of range")
        need = zero_loss_head_workspace_bytes_for(max_tokens, table, gradients)
        if need == 0:
            raise ValueError(f"a table of 16-bit elements is required, got {table.dtype}, strides {table.stride()}")
        self._workspace(need, workspace)

    def _fits(self, x) -> None:
        if x.shape[0] > self.max_tokens:
            raise ValueError(f"{x.shape[0]} tokens, made for {self.max_tokens} (max_tokens)")

    def forward(self, x, labels, losses, loss, count, stream=None) -> None:
        """losses[t] (fp32; 0 where the label does not count), their mean in `loss` (fp32), and how many count (int64)
        in `count`."""
        self._on(x, labels, losses, loss, count)
        self._fits(x)
        self._call(zero_loss_head, x, self.table, labels, losses, loss, count, self.ws, self.ws_bytes, stream=stream)

    def grad(self, x, labels, losses, loss, count, x_grad, table_grad, accumulate: bool = False, step_state=None,
             scale: float = 1.0, stream=None) -> None:
        """The same, and the gradients of `loss` times `scale` and the loss scale in `step_state` (ListDecision.state,
        DeviceDecision.state; None: 1); `accumulate`: the table's is added to what `table_grad` holds."""
        if not self.gradients:
            raise ValueError("made without gradients")
        self._on(x, labels, losses, loss, count, x_grad, table_grad, step_state)
        self._fits(x)
        self._call(zero_loss_head_grad, x, self.table, labels, losses, loss, count, x_grad, table_grad, self.ws,
                   self.ws_bytes, scale=scale, accumulate=accumulate, step_state=step_state, stream=stream)


def wait_spin(stream) -> None:
    """Waits for the work queued on `stream` by polling an event: the decision that follows sits on the
    critical path between the norm and the update, and polling wakes within microseconds of completion."""
    done = torch.cuda.Event()
    done.record(stream)
    while not done.query():
        pass


def rank_norms(shards, cfg: AdamWConfig, scaler: ScalerState, flatten: bool = True, stream=None) -> dict:
    """First half of a step over the simulated ranks: flatten (and square-norm), the 16-byte readback, the
    simulated all-reduce and the decision.  Updates the loss-scale state; returns the decision."""
    stream = stream or torch.cuda.current_stream()
    for sh in shards:
        if flatten:
            sh.flatten(stream)
        if not (flatten and sh.fused):
            sh.sqnorm(stream)
        sh.readback(stream)
    wait_spin(stream)
    sq, fl = zip(*(sh.norm_result() for sh in shards))
    dec = zero_step_decision(sq, fl, cfg.max_norm, scaler.scale, scaler.good_steps, scaler.growth_interval)
    scaler.scale, scaler.good_steps = dec["loss_scale"], dec["good_steps"]
    dec["rank_sqnorms"] = list(sq)
    dec["rank_flags"] = list(fl)
    return dec


def rank_update(shards, cfg: AdamWConfig, scaler: ScalerState, dec: dict, stream=None) -> None:
    """Second half: the AdamW update of every simulated rank with the decision's factor (nothing on skip)."""
    if dec["skip"]:
        return
    stream = stream or torch.cuda.current_stream()
    scaler.adam_step += 1
    for sh in shards:
        sh.adamw(cfg, dec["grad_scale"], scaler.adam_step, stream)


def rank_step(shards, cfg: AdamWConfig, scaler: ScalerState, flatten: bool = True, stream=None) -> dict:
    """One training step over the simulated ranks; returns the decision (grad_scale, skip, norm, ...)."""
    dec = rank_norms(shards, cfg, scaler, flatten, stream)
    rank_update(shards, cfg, scaler, dec, stream)
    return dec
