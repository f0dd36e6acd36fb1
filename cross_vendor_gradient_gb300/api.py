"""Tensor-level interface over libgb.

torch supplies device memory and the current CUDA stream; every computation
runs in libgb's kernels (there is no CPU or PyTorch fallback).  Each method
marshals tensors to pointers, calls the C entry point of the same name on the
current stream and raises ``GbError`` on a non-OK status.
"""
from array import array
from operator import attrgetter

import torch

from . import binding as B

_get_dtype = attrgetter("dtype")

_DTYPES = {torch.float32: B.GB_F32, torch.bfloat16: B.GB_BF16, torch.float16: B.GB_F16,
           torch.float64: B.GB_F64, torch.int8: B.GB_I8, torch.uint8: B.GB_U8, torch.int32: B.GB_I32,
           torch.int64: B.GB_I64}
CODECS = {"none": B.GB_CODEC_NONE, "bf16": B.GB_CODEC_BF16, "e4m3": B.GB_CODEC_E4M3,
          "e5m2": B.GB_CODEC_E5M2}
OPS = {"sum": B.GB_SUM, "avg": B.GB_AVG, "max": B.GB_MAX, "min": B.GB_MIN}


class GbError(RuntimeError):
    def __init__(self, status, message=""):
        self.status = status
        super().__init__("%s%s" % (B.gb_status_string(status), (": " + message) if message else ""))


def _codec(c):
    return CODECS[c] if isinstance(c, str) else int(c)


def _op(o):
    return OPS[o] if isinstance(o, str) else int(o)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())  # current_stream() without its Stream object


def _capturing(stream):
    """Whether the stream (None: the current one) is being captured together with the current one."""
    if not torch._C._cuda_isCurrentStreamCapturing():  # torch.cuda.is_current_stream_capturing(), half its time
        return False
    if stream is None:
        return True
    with torch.cuda.stream(torch.cuda.ExternalStream(stream.cuda_stream)):  # of any kind that has this address
        return torch.cuda.is_current_stream_capturing()


def _dtype(tensors):
    dt = tensors[0].dtype
    if dt not in _DTYPES:
        raise GbError(B.GB_ERR_UNSUPPORTED_DTYPE, str(dt))
    for t in tensors:
        if t.dtype != dt or not t.is_contiguous() or t.device != tensors[0].device:
            raise GbError(B.GB_ERR_INVALID_ARG, "tensors must share dtype and device and be contiguous")
    return _DTYPES[dt]


def _row_pitch(tensors):
    """The byte distance between consecutive tensors when all of them lie in
    one storage (one host allocation) at equal, ascending spacing of at
    least one tensor's bytes; else None."""
    if len(tensors) < 2:
        return None
    base = tensors[0].untyped_storage().data_ptr()
    if any(t.untyped_storage().data_ptr() != base for t in tensors[1:]):
        return None
    nb = tensors[0].numel() * tensors[0].element_size()
    pitch = tensors[1].data_ptr() - tensors[0].data_ptr()
    if pitch < nb or any(t.data_ptr() != tensors[0].data_ptr() + r * pitch for r, t in enumerate(tensors)):
        return None
    return pitch


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cuda_dtype(tensors):
    """_dtype of CUDA tensors; without a Python loop, for there may be hundreds."""
    dtypes, devices = set(map(_get_dtype, tensors)), set(map(torch.Tensor.get_device, tensors))  # -1: on the host
    if len(dtypes) != 1 or len(devices) != 1 or -1 in devices or not all(map(torch.Tensor.is_contiguous, tensors)):
        raise GbError(B.GB_ERR_INVALID_ARG, "CUDA tensors of one dtype and device, contiguous")
    dtype, = dtypes
    if dtype not in _DTYPES:
        raise GbError(B.GB_ERR_UNSUPPORTED_DTYPE, str(dtype))
    return _DTYPES[dtype]


def _expect(t, dtype, n, name, device=None):
    """A contiguous CUDA tensor of n elements of dtype (on `device`, a get_device() number)."""
    at = t.get_device()
    if t.dtype != dtype or t.numel() != n or at < 0 or (device is not None and at != device) or not t.is_contiguous():
        raise GbError(B.GB_ERR_INVALID_ARG, "%s: a contiguous CUDA tensor of %d %s" % (name, n, dtype))


def payload_bytes(codec, block, n):
    return B.gb_payload_bytes(_codec(codec), block, n)


def island_payload_bytes(dtype, op, codec, block, n):
    """Bytes of one island's payload for any dtype and op (the exact path's
    fold, or the codec's payload)."""
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return B.gb_island_payload_bytes(dt, _op(op), _codec(codec), block, n)


def payload_scales_offset(codec, block, n):
    return B.gb_payload_scales_offset(_codec(codec), block, n)


def bucket_plan(numels, elem_bytes, cap_bytes=25 * 1024 * 1024, pad_elems=1):
    st, bo, off, bn = B.gb_bucket_plan(list(numels), elem_bytes, cap_bytes, pad_elems)
    if st != B.GB_OK:
        raise GbError(st, "bucket plan")
    return bo, off, bn


def rms_norm_payload_bytes(codec, block, rows, cols):
    """Bytes of rms_norm's 8-bit output."""
    return B.gb_rms_norm_payload_bytes(_codec(codec), block, rows, cols)


def kernel_launch_count():
    return B.gb_kernel_launch_count()


class Context:
    """W simulated ranks in contiguous islands on the current CUDA device."""

    def __init__(self, island_sizes):
        st, h = B.gb_create(list(island_sizes))
        if st != B.GB_OK:
            raise GbError(st, "gb_create(%s)" % (list(island_sizes),))
        self.handle = h
        self.island_sizes = tuple(int(v) for v in island_sizes)
        self.world_size = B.gb_world_size(h)

    def close(self):
        if self.handle:
            B.gb_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _check(self, st):
        if st != B.GB_OK:
            raise GbError(st, B.gb_last_error_message(self.handle))

    # ------------------------------------------------------------ topology
    def island_first_rank(self, i):
        return B.gb_island_first_rank(self.handle, i)

    def island_of_rank(self, r):
        return B.gb_island_of_rank(self.handle, r)

    def status(self):
        return B.gb_context_status(self.handle)

    def set_pipeline(self, chunk_bytes, use_graphs=True):
        """chunk_bytes > 0: pipelined bridge in chunks of about that many bytes
        of one island's payload (default 2 MiB); 0: one bridge hop per call."""
        self._check(B.gb_set_pipeline(self.handle, chunk_bytes, use_graphs))

    def set_sharded_bridge(self, on=True):
        """Sharded-bridge policy for all_reduce: k = smallest island size
        segments, each over its own bridge link (same bits)."""
        self._check(B.gb_set_sharded_bridge(self.handle, on))

    def reserve(self, n, dtype=torch.float32, codec="none", block=256):
        self._check(B.gb_reserve(self.handle, n, _DTYPES[dtype], _codec(codec), block))

    # ---------------------------------------------------------- collectives
    def all_reduce(self, tensors, op="sum", codec="none", block=256, stream=None):
        dt = _dtype(tensors)
        self._check(B.gb_all_reduce(self.handle, [t.data_ptr() for t in tensors], tensors[0].numel(), dt,
                                    _op(op), _codec(codec), block, _stream(stream)))

    def all_reduce_ef(self, tensors, residuals, op="sum", codec="none", block=256, stream=None):
        """all_reduce with error feedback; residuals: one float32 tensor of the
        buffers' size per island, zero before the first step, kept across steps."""
        dt = _dtype(tensors)
        for r in residuals:
            if r.dtype != torch.float32 or not r.is_contiguous() or r.numel() != tensors[0].numel():
                raise GbError(B.GB_ERR_INVALID_ARG, "residuals: contiguous float32 of the buffers' size")
        self._check(B.gb_all_reduce_ef(self.handle, [t.data_ptr() for t in tensors], [r.data_ptr() for r in residuals],
                                       tensors[0].numel(), dt, _op(op), _codec(codec), block, _stream(stream)))

    def reduce_scatter(self, inputs, outputs, op="sum", codec="none", block=256, stream=None):
        dt = _dtype(list(inputs) + list(outputs))
        self._check(B.gb_reduce_scatter(self.handle, [t.data_ptr() for t in inputs],
                                        [t.data_ptr() for t in outputs], inputs[0].numel(), dt, _op(op),
                                        _codec(codec), block, _stream(stream)))

    def all_gather(self, inputs, outputs, stream=None):
        dt = _dtype(list(inputs) + list(outputs))
        self._check(B.gb_all_gather(self.handle, [t.data_ptr() for t in inputs],
                                    [t.data_ptr() for t in outputs], inputs[0].numel(), dt,
                                    _stream(stream)))

    def broadcast(self, tensors, src, stream=None):
        dt = _dtype(tensors)
        self._check(B.gb_broadcast(self.handle, [t.data_ptr() for t in tensors], tensors[0].numel(), dt,
                                   src, _stream(stream)))

    def all_reduce_host(self, host_tensors, op="sum", codec="none", block=256, stream=None):
        """host_tensors: W host tensors (pinned for asynchronous copies), or
        one [W, n] host tensor whose rows are the ranks.  Rows of one
        storage at equal, ascending spacing go through
        gb_all_reduce_host_rows (2D staging copies); anything else through
        gb_all_reduce_host."""
        if isinstance(host_tensors, torch.Tensor):
            if host_tensors.dim() != 2:
                raise GbError(B.GB_ERR_INVALID_ARG, "a host tensor of ranks must be [W, n]")
            host_tensors = list(host_tensors.unbind(0))
        if any(t.device.type != "cpu" for t in host_tensors):
            raise GbError(B.GB_ERR_INVALID_ARG, "all_reduce_host takes host (CPU) tensors; use all_reduce for CUDA tensors")
        dt = _dtype(host_tensors)
        n = host_tensors[0].numel()
        pitch = _row_pitch(host_tensors)
        if pitch is not None:
            self._check(B.gb_all_reduce_host_rows(self.handle, host_tensors[0].data_ptr(), pitch, n, dt, _op(op),
                                                  _codec(codec), block, _stream(stream)))
            return
        self._check(B.gb_all_reduce_host(self.handle, [t.data_ptr() for t in host_tensors], n, dt, _op(op),
                                         _codec(codec), block, _stream(stream)))

    def all_reduce_buckets(self, buckets, op="sum", codec="none", block=256, stream=None):
        """buckets: list of per-bucket lists of W flat tensors."""
        flat = [t for b in buckets for t in b]
        dt = _dtype(flat)
        self._check(B.gb_all_reduce_buckets(self.handle, [t.data_ptr() for t in flat],
                                            [b[0].numel() for b in buckets], dt, _op(op), _codec(codec),
                                            block, _stream(stream)))

    def all_reduce_buckets_ef(self, buckets, residuals, op="sum", codec="none", block=256, stream=None):
        """buckets[b]: W flat tensors; residuals[b]: I float32 tensors of the
        bucket's length (zero at the start, kept across steps)."""
        flat = [t for b in buckets for t in b]
        res = [r for b in residuals for r in b]
        for r in res:
            if r.dtype != torch.float32 or not r.is_contiguous():
                raise GbError(B.GB_ERR_INVALID_ARG, "residuals must be contiguous float32 tensors")
        dt = _dtype(flat)
        self._check(B.gb_all_reduce_buckets_ef(self.handle, [t.data_ptr() for t in flat], [r.data_ptr() for r in res],
                                               [b[0].numel() for b in buckets], dt, _op(op), _codec(codec), block,
                                               _stream(stream)))

    def reduce_scatter_buckets(self, in_buckets, out_buckets, op="sum", codec="none", block=256, stream=None):
        """in_buckets[b]: W flat tensors of bucket b; out_buckets[b]: W
        tensors of numel / W elements."""
        ins = [t for b in in_buckets for t in b]
        outs = [t for b in out_buckets for t in b]
        dt = _dtype(ins)
        self._check(B.gb_reduce_scatter_buckets(self.handle, [t.data_ptr() for t in ins],
                                                [t.data_ptr() for t in outs], [b[0].numel() for b in in_buckets],
                                                dt, _op(op), _codec(codec), block, _stream(stream)))

    def all_gather_buckets(self, in_buckets, out_buckets, stream=None):
        """in_buckets[b]: W tensors of m_b elements; out_buckets[b]: W
        tensors of W * m_b elements."""
        ins = [t for b in in_buckets for t in b]
        outs = [t for b in out_buckets for t in b]
        dt = _dtype(ins)
        self._check(B.gb_all_gather_buckets(self.handle, [t.data_ptr() for t in ins], [t.data_ptr() for t in outs],
                                            [b[0].numel() for b in in_buckets], dt, _stream(stream)))

    # ------------------------------------------------------- phase blocks
    def island_reduce(self, island, tensors, island_sum, stream=None):
        dt = _dtype(tensors)
        self._check(B.gb_island_reduce(self.handle, island, [t.data_ptr() for t in tensors],
                                       tensors[0].numel(), dt, island_sum.data_ptr(), _stream(stream)))

    def bridge_compress(self, island_sum, codec, block, payload, stream=None):
        self._check(B.gb_bridge_compress(self.handle, island_sum.data_ptr(), island_sum.numel(),
                                         _codec(codec), block, payload.data_ptr(), _stream(stream)))

    def bridge_decompress_accumulate(self, payload, n, codec, block, accum, accumulate, stream=None):
        self._check(B.gb_bridge_decompress_accumulate(self.handle, payload.data_ptr(), n, _codec(codec),
                                                      block, accum.data_ptr(), accumulate,
                                                      _stream(stream)))

    def island_broadcast(self, island, total, op, tensors, stream=None):
        dt = _dtype(tensors)
        self._check(B.gb_island_broadcast(self.handle, island, total.data_ptr(), total.numel(), _op(op),
                                          [t.data_ptr() for t in tensors], dt, _stream(stream)))

    def island_reduce_compress(self, tensors, codec, block, payloads, stream=None):
        """Fused island reduce + encode of every island: payloads[i] (uint8
        device tensors of payload_bytes(codec, block, n) bytes) receive the
        encoded island sums."""
        dt = _dtype(tensors)
        self._check(B.gb_island_reduce_compress(self.handle, [t.data_ptr() for t in tensors],
                                                tensors[0].numel(), dt, _codec(codec), block,
                                                [p.data_ptr() for p in payloads], _stream(stream)))

    def island_reduce_compress_ef(self, tensors, residuals, codec, block, payloads, stream=None):
        """island_reduce_compress with error feedback: residuals are I
        float32 tensors of n elements (updated in place)."""
        dt = _dtype(tensors)
        self._check(B.gb_island_reduce_compress_ef(self.handle, [t.data_ptr() for t in tensors],
                                                   [r.data_ptr() for r in residuals], tensors[0].numel(), dt,
                                                   _codec(codec), block, [p.data_ptr() for p in payloads],
                                                   _stream(stream)))

    def decompress_island_broadcast(self, payloads, op, codec, block, tensors, stream=None):
        """Fused decode of every island's payload + accumulate + broadcast
        into all rank tensors.  payloads: I tensors (every leader holds the
        same ones) or I * I (row g: what leader g holds, island order)."""
        dt = _dtype(tensors)
        I = len(self.island_sizes)
        if len(payloads) == I and I > 1:  # one shared set: every leader's row
            payloads = [p for _ in range(I) for p in payloads]
        self._check(B.gb_decompress_island_broadcast(self.handle, [p.data_ptr() for p in payloads],
                                                     tensors[0].numel(), dt, _op(op), _codec(codec), block,
                                                     [t.data_ptr() for t in tensors], _stream(stream)))

    def island_reduce_compress_op(self, tensors, op, codec, block, payloads, stream=None):
        """The first fused half for every dtype and op: the codec path's
        encode, or the exact path's island fold (payloads of
        island_payload_bytes bytes)."""
        dt = _dtype(tensors)
        self._check(B.gb_island_reduce_compress_op(self.handle, [t.data_ptr() for t in tensors],
                                                   tensors[0].numel(), dt, _op(op), _codec(codec), block,
                                                   [p.data_ptr() for p in payloads], _stream(stream)))

    def decompress_scatter(self, payloads, n, op, codec, block, outputs, stream=None):
        """reduce_scatter's second half: outputs[r] (n / W elements) receives
        slice r of the decoded total.  payloads: I tensors (every leader holds
        the same ones) or I * I."""
        dt = _dtype(outputs)
        I = len(self.island_sizes)
        if len(payloads) == I and I > 1:
            payloads = [p for _ in range(I) for p in payloads]
        self._check(B.gb_decompress_scatter(self.handle, [p.data_ptr() for p in payloads], n, dt, _op(op),
                                            _codec(codec), block, [t.data_ptr() for t in outputs],
                                            _stream(stream)))

    # ------------------------------------------------ training-step operators
    def grad_norm(self, grads, out, max_norm=0.0, stream=None):
        """out (2 float32) = the 2-norm of all gradients together, and the
        factor that clips them to max_norm (1 when max_norm <= 0, NaN when
        the norm is not finite): adamw's grad_scale is out[1:]."""
        dt = _cuda_dtype(grads) if grads else B.GB_F32
        _expect(out, torch.float32, 2, "out", grads[0].get_device() if grads else None)
        self._check(B.gb_grad_norm(self.handle, array("Q", map(torch.Tensor.data_ptr, grads)),
                                   array("Q", map(torch.Tensor.numel, grads)), dt, max_norm, out.data_ptr(),
                                   _stream(stream)))

    def adamw_step(self, params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                   weight_decay=1e-2, copies=None, states="none", block=256, seed=0, grad_scale=None, stream=None):
        """One AdamW step over many tensors, in place.  params: float32;
        exp_avg, exp_avg_sq: float32 tensors (states="none") or uint8 E4M3
        payloads of payload_bytes("e4m3", block, n) bytes, zero at the start
        (states="e4m3"); copies: tensors of the gradients' type that receive
        the rounded parameters; grad_scale: a float32 device tensor of one
        element (the step is refused when it is not finite).  adamw() keeps
        the same arguments for many steps."""
        self.adamw(params, grads, exp_avg, exp_avg_sq, copies=copies, lr=lr, betas=betas, eps=eps,
                   weight_decay=weight_decay, states=states, block=block).step(step=step, seed=seed,
                                                                               grad_scale=grad_scale, stream=stream)

    def adamw(self, params, grads, exp_avg=None, exp_avg_sq=None, **options):
        """An AdamW optimizer over these tensors (see AdamW)."""
        return AdamW(self, params, grads, exp_avg, exp_avg_sq, **options)

    def rms_norm(self, x, weight, out, eps=1e-5, residual=None, sum_out=None, rstd=None, codec="none", block=256,
                 stream=None):
        """out = RMS norm of x + residual, times weight: rows are x's last
        dimension.  codec "none": out like x; "e4m3" / "e5m2": out a uint8
        tensor of rms_norm_payload_bytes(codec, block, rows, cols) bytes.
        sum_out receives x + residual, rstd (float32, rows) each row's
        1 / root mean square."""
        dt = _cuda_dtype([t for t in (x, weight, residual, sum_out) if t is not None])
        cols = weight.numel()
        if weight.dim() != 1 or x.dim() < 1 or x.shape[-1] != cols:
            raise GbError(B.GB_ERR_INVALID_ARG, "weight: one dimension, that of x's last")
        n = x.numel()
        rows = x.shape[:-1].numel()
        for t, name in ((residual, "residual"), (sum_out, "sum_out")):
            if t is not None and t.numel() != n:
                raise GbError(B.GB_ERR_INVALID_ARG, "%s: x's size" % name)
        cd, device = _codec(codec), x.get_device()
        if cd == B.GB_CODEC_NONE:
            _expect(out, x.dtype, n, "out", device)
        else:
            _expect(out, torch.uint8, B.gb_rms_norm_payload_bytes(cd, block, rows, cols), "out", device)
        if rstd is not None:
            _expect(rstd, torch.float32, rows, "rstd", device)
        self._check(B.gb_rms_norm(self.handle, x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, cols, dt, eps, cd,
                                  block, _ptr(sum_out), out.data_ptr(), _ptr(rstd), _stream(stream)))

    def rms_norm_backward(self, dy, h, weight, rstd, dx, dweight, dsum=None, stream=None):
        """The gradient of rms_norm: dx (of x, and of the residual) and
        dweight, from dy, the h (x, or sum_out) and rstd of the forward call,
        and dsum, the gradient that reaches h past the norm."""
        dt = _cuda_dtype([t for t in (dy, h, weight, dx, dweight, dsum) if t is not None])
        cols = weight.numel()
        if weight.dim() != 1 or h.dim() < 1 or h.shape[-1] != cols or dweight.numel() != cols:
            raise GbError(B.GB_ERR_INVALID_ARG, "weight and dweight: one dimension, that of h's last")
        n = h.numel()
        rows = h.shape[:-1].numel()
        for t, name in ((dy, "dy"), (dx, "dx"), (dsum, "dsum")):
            if t is not None and t.numel() != n:
                raise GbError(B.GB_ERR_INVALID_ARG, "%s: h's size" % name)
        _expect(rstd, torch.float32, rows, "rstd", h.get_device())
        self._check(B.gb_rms_norm_backward(self.handle, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                                           _ptr(dsum), rows, cols, dt, dx.data_ptr(), dweight.data_ptr(),
                                           _stream(stream)))

    # -------------------------------------------------------------- timing
    def set_phase_timing(self, capacity):
        """capacity > 0: keep the phase marks of the last `capacity` calls."""
        self._check(B.gb_set_phase_timing(self.handle, int(capacity)))

    def phase_times(self, age):
        st, ms = B.gb_phase_times(self.handle, age)
        self._check(st)
        return ms

    def last_phase_times(self):
        st, ms = B.gb_last_phase_times(self.handle)
        self._check(st)
        return ms

    def debug_inject(self, what):
        self._check(B.gb_debug_inject(self.handle, what))


class AdamW:
    """AdamW over many tensors: Context.adamw_step with its arguments kept.

    The tensors are checked, and their addresses taken, once: a step costs one
    call whatever their number.  Parameters, gradients and copies stay where
    they are (views into gradient buckets, for instance); the states are
    exp_avg / exp_avg_sq, made here (zero) unless given: the host then waits
    until they are, so that a step may run on any stream.
    """

    def __init__(self, ctx, params, grads, exp_avg=None, exp_avg_sq=None, copies=None, lr=1e-3, betas=(0.9, 0.999),
                 eps=1e-8, weight_decay=1e-2, states="none", block=256):
        self.ctx, self.params, self.grads, self.copies = ctx, list(params), list(grads), copies and list(copies)
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.states, self.block, self.steps = states, block, 0
        self._codec = _codec(states)
        self._dtype = _dtype(self.grads) if self.grads else B.GB_F32
        if self._codec not in (B.GB_CODEC_NONE, B.GB_CODEC_E4M3):
            raise GbError(B.GB_ERR_UNSUPPORTED_CODEC, "states are \"none\" (float32) or \"e4m3\"")
        numel = [p.numel() for p in self.params]
        size = [n if self._codec == B.GB_CODEC_NONE else B.gb_payload_bytes(self._codec, block, n) for n in numel]
        kind = torch.float32 if self._codec == B.GB_CODEC_NONE else torch.uint8
        device = self.params[0].get_device() if self.params else None
        self.exp_avg, self.exp_avg_sq = (
            [torch.zeros(n, dtype=kind, device=p.device) for n, p in zip(size, self.params)] if v is None else list(v)
            for v in (exp_avg, exp_avg_sq))
        for ts, dtype, counts, name in ((self.params, torch.float32, numel, "params"),
                                        (self.grads, self.grads[0].dtype if self.grads else None, numel, "grads"),
                                        (self.copies, self.grads[0].dtype if self.grads else None, numel, "copies"),
                                        (self.exp_avg, kind, size, "exp_avg"), (self.exp_avg_sq, kind, size, "exp_avg_sq")):
            if ts is None:
                continue
            if len(ts) != len(numel):
                raise GbError(B.GB_ERR_INVALID_ARG, "%s: %d tensors for %d parameters" % (name, len(ts), len(numel)))
            for t, n in zip(ts, counts):
                _expect(t, dtype, n, name, device)
        if (exp_avg is None or exp_avg_sq is None) and self.params and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(device).synchronize()
        self._arrays = [None if ts is None else B._ptrs([t.data_ptr() for t in ts])
                        for ts in (self.params, self.grads, self.exp_avg, self.exp_avg_sq, self.copies)]
        self._numel = B._sizes(numel)
        self._n = len(numel)

    def step(self, grad_scale=None, step=None, seed=0, stream=None):
        """One step, from the gradients as they are now.  step: its number
        (default: one more than the last; a step that the device refuses for
        a grad_scale that is not finite counts too); seed: of the 8-bit
        states' random numbers, another one on each rank that steps shards of
        its own.  The number, the seed and the learning rate
        are taken at the call: a graph repeats them in every replay, and with
        them the bias correction and the random numbers, so a captured step
        has to be given its number."""
        if step is None:
            if _capturing(stream):
                raise GbError(B.GB_ERR_INVALID_ARG, "a captured step needs its number, which every replay repeats")
            step = self.steps + 1
        if grad_scale is not None:
            _expect(grad_scale, torch.float32, 1, "grad_scale")
        cfg = B.Adamw(self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay, step, seed)
        self.ctx._check(B.lib().gb_adamw_step(self.ctx.handle, self._n, *self._arrays, self._numel, self._dtype,
                                              self._codec, self.block, cfg, _ptr(grad_scale), _stream(stream)))
        self.steps = step
