"""Python binding of the draft-head training operators in
``include/domino_train.h`` (ctypes): argument marshalling only, like
``rollout.py``.  ``DominoTrain`` takes torch CUDA tensors and the current torch
stream; ``distill_loss``, ``token_logprobs`` and ``embedding`` are the operators
as torch autograd functions.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes

from . import rollout as _r
from .rollout import DOMINO_DTYPE_BF16, DOMINO_DTYPE_FP32, DominoError, _check

DOMINO_TRAIN_MAX_V = 524288
DOMINO_TRAIN_MAX_K = 8192
DOMINO_TRAIN_MAX_TOKENS = 4194304
DOMINO_TRAIN_STATS = 8
DOMINO_TRAIN_MAX_ALTERNATIVES = 32
DOMINO_TRAIN_LOGPROB_STATS = 4

# every symbol the header declares
EXPORTED = (
    "domino_train_init", "domino_train_top_logits", "domino_train_distill_forward", "domino_train_distill_backward",
    "domino_train_distill_step", "domino_train_logprobs_forward", "domino_train_logprobs_backward",
    "domino_train_logprobs_step", "domino_train_embed", "domino_train_embed_grad", "domino_train_status",
    "domino_train_last_launch_count", "domino_train_destroy",
)


class domino_train_config(ctypes.Structure):
    _fields_ = [("V", ctypes.c_int), ("E", ctypes.c_int), ("max_tokens", ctypes.c_int), ("dtype", ctypes.c_int)]


_lib = None


def load_library() -> ctypes.CDLL:
    """The rollout's library with the training entry points declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _r.load_library()
    vp, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    lib.domino_train_init.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(domino_train_config), i]
    lib.domino_train_top_logits.argtypes = [vp, vp, i, ll, i, i, f, vp, vp, vp, vp]
    lib.domino_train_distill_forward.argtypes = [vp, vp, ll, i, vp, vp, vp, i, f, vp, vp, vp]
    lib.domino_train_distill_backward.argtypes = [vp, vp, ll, i, vp, vp, vp, i, f, vp, vp, vp, ll, vp]
    lib.domino_train_distill_step.argtypes = [vp, vp, ll, i, vp, vp, vp, i, f, vp, vp, vp, ll, vp]
    lib.domino_train_logprobs_forward.argtypes = [vp, vp, i, ll, i, vp, f, vp, vp, i, vp, vp, vp, vp]
    lib.domino_train_logprobs_backward.argtypes = [vp, vp, ll, i, vp, f, vp, vp, vp, vp, ll, vp]
    lib.domino_train_logprobs_step.argtypes = [vp, vp, ll, i, vp, f, vp, vp, vp, vp, vp, ll, vp]
    lib.domino_train_embed.argtypes = [vp, vp, vp, i, f, vp, ll, vp]
    lib.domino_train_embed_grad.argtypes = [vp, vp, ll, vp, i, f, vp, i, i, vp]
    lib.domino_train_status.argtypes = [vp, vp]
    lib.domino_train_last_launch_count.argtypes = [vp]
    lib.domino_train_destroy.argtypes = [vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib.domino_train_destroy.restype = None
    _lib = lib
    return lib


class DominoTrain:
    """Owns one training context (see the header for the formulas).

    V vocabulary, E embedding width (0: no embedding calls), max_tokens the
    most tokens of one ``embed_grad`` call, dtype "bf16" or "fp32".

    Tensors are on the context's device; rows may be strided (last dimension
    contiguous).  Every method takes ``out``, the tensors to write, and
    ``stream`` (a torch stream or raw handle; default: the current one).  With a
    stream other than the current one the caller orders the two, as for any
    kernel, and gives ``out``.  ``embed_grad`` calls of one context, whose
    workspace they share, run one after another on the device whatever their
    streams; only replays of captured graphs that hold one are the caller's to order.
    """

    def __init__(self, V, E=0, max_tokens=0, dtype="bf16", device=0):
        import torch
        if dtype not in ("bf16", "fp32"):
            raise ValueError(f"dtype: want 'bf16' or 'fp32', got {dtype!r}")
        self._lib = load_library()
        self.V, self.E, self.max_tokens, self.dtype = V, E, max_tokens, dtype
        self.device = torch.device("cuda", device)
        self.torch_dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self._index, self._bf16, self._f32, self._i32 = device, torch.bfloat16, torch.float32, torch.int32
        # the raw handle where torch gives it: a Stream object costs more than a launch
        self._current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                       lambda i: torch.cuda.current_stream(i).cuda_stream)
        cfg = domino_train_config(V, E, max_tokens, DOMINO_DTYPE_BF16 if dtype == "bf16" else DOMINO_DTYPE_FP32)
        self.ctx = ctypes.c_void_p()
        _check(self._lib.domino_train_init(ctypes.byref(self.ctx), ctypes.byref(cfg), device), "domino_train_init")

    # -- checks (on every call's path: plain integers and identities) -------------

    def _rows(self, t, cols, name, dtype=None, n=None):
        """Row stride of a [n, cols] tensor whose rows are contiguous."""
        shape = t.shape
        if (len(shape) == 2 and shape[1] == cols and t.dtype is (dtype or self.torch_dtype)
                and t.get_device() == self._index and (n is None or shape[0] == n)):
            ld, inner = t.stride()
            if inner == 1 or cols <= 1 or shape[0] == 0:  # no rows: strides mean nothing
                if ld >= cols:
                    return ld
                if shape[0] <= 1:
                    return cols
        raise ValueError(f"{name}: want CUDA [{'n' if n is None else n}, {cols}] {dtype or self.torch_dtype} with "
                         f"contiguous rows on {self.device}, got {tuple(shape)} {t.dtype} strides {t.stride()} on "
                         f"{t.device}")

    def _flat(self, t, shape, dtype, name):
        """The address of a contiguous tensor of exactly this shape and type."""
        if t.shape == shape and t.dtype is dtype and t.get_device() == self._index and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(f"{name}: want contiguous CUDA {tuple(shape)} {dtype} on {self.device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")

    def _stream(self, stream):
        if stream is None:
            return self._current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _new(self, shape, dtype):
        import torch
        return torch.empty(shape, dtype=dtype, device=self.device)

    def _record(self, ids, top, rest, n):
        if ids.dim() != 2:
            raise ValueError(f"ids: want [n, K], got {tuple(ids.shape)}")
        shape = (n, ids.shape[1])
        return (self._flat(ids, shape, self._i32, "ids"), self._flat(top, shape, self._f32, "top"),
                None if rest is None else self._flat(rest, (n,), self._f32, "rest"), shape[1])

    # -- operators ---------------------------------------------------------------

    def top_logits(self, logits, K, temperature=1.0, out=None, stream=None):
        """(ids [n, K] int32 ascending, top [n, K], rest [n]) of a teacher's
        logits [n, V] (bf16 or fp32)."""
        n, dtype = logits.shape[0], logits.dtype
        if dtype is not self._bf16 and dtype is not self._f32:
            raise ValueError(f"logits: want bfloat16 or float32, got {dtype}")
        ld = self._rows(logits, self.V, "logits", dtype)
        if out is None:
            out = self._new((n, max(K, 0)), self._i32), self._new((n, max(K, 0)), self._f32), self._new((n,), self._f32)
        ids, top, rest = out
        status = self._lib.domino_train_top_logits(
            self.ctx, logits.data_ptr(), DOMINO_DTYPE_BF16 if dtype is self._bf16 else DOMINO_DTYPE_FP32, ld, n, K,
            temperature, self._flat(ids, (n, K), self._i32, "ids"), self._flat(top, (n, K), self._f32, "top"),
            self._flat(rest, (n,), self._f32, "rest"), self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_top_logits")
        return ids, top, rest

    def distill_forward(self, logits, ids, top, rest=None, temperature=1.0, out=None, stream=None):
        """(loss [n], stats [n, 8]) of student logits [n, V]; ``stats`` is for distill_backward."""
        n = logits.shape[0]
        ld = self._rows(logits, self.V, "logits")
        pi, pt, pr, K = self._record(ids, top, rest, n)
        if out is None:
            out = self._new((n,), self._f32), self._new((n, DOMINO_TRAIN_STATS), self._f32)
        loss, stats = out
        status = self._lib.domino_train_distill_forward(
            self.ctx, logits.data_ptr(), ld, n, pi, pt, pr, K, temperature, self._flat(loss, (n,), self._f32, "loss"),
            self._flat(stats, (n, DOMINO_TRAIN_STATS), self._f32, "stats"), self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_distill_forward")
        return loss, stats

    def distill_backward(self, logits, ids, top, rest, stats, dloss, temperature=1.0, out=None, stream=None):
        """dlogits [n, V] from the gradient dloss [n] by each row's loss."""
        n = logits.shape[0]
        ld = self._rows(logits, self.V, "logits")
        pi, pt, pr, K = self._record(ids, top, rest, n)
        if out is None:
            out = self._new((n, self.V), self.torch_dtype)
        status = self._lib.domino_train_distill_backward(
            self.ctx, logits.data_ptr(), ld, n, pi, pt, pr, K, temperature,
            self._flat(stats, (n, DOMINO_TRAIN_STATS), self._f32, "stats"),
            self._flat(dloss, (n,), self._f32, "dloss"), out.data_ptr(), self._rows(out, self.V, "dlogits", n=n),
            self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_distill_backward")
        return out

    def distill_step(self, logits, ids, top, rest, weight, temperature=1.0, out=None, stream=None):
        """(loss [n], dlogits [n, V]) in one call; dlogits is the gradient of sum(weight * loss)."""
        n = logits.shape[0]
        ld = self._rows(logits, self.V, "logits")
        pi, pt, pr, K = self._record(ids, top, rest, n)
        if out is None:
            out = self._new((n,), self._f32), self._new((n, self.V), self.torch_dtype)
        loss, grad = out
        status = self._lib.domino_train_distill_step(
            self.ctx, logits.data_ptr(), ld, n, pi, pt, pr, K, temperature,
            self._flat(weight, (n,), self._f32, "weight"), self._flat(loss, (n,), self._f32, "loss"),
            grad.data_ptr(), self._rows(grad, self.V, "dlogits", n=n), self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_distill_step")
        return loss, grad

    def logprobs_forward(self, logits, tokens, temperature=1.0, alternatives=0, stats=None, out=None, stream=None):
        """(logprob [n], entropy [n]) of logits [n, V] (bf16 or fp32) and their tokens [n] int32
        (-1: the row takes no part); with ``alternatives`` = k > 0 also (ids [n, k] int32, logprobs
        [n, k]) of the k most likely ids, most likely first.  ``stats``: True or a [n, 4] tensor adds
        what logprobs_backward needs as the last value.  ``out``: the tensors before it."""
        n, dtype, k, f32 = logits.shape[0], logits.dtype, alternatives, self._f32
        if dtype is not self._bf16 and dtype is not f32:
            raise ValueError(f"logits: want bfloat16 or float32, got {dtype}")
        ld = self._rows(logits, self.V, "logits", dtype)
        if out is None:
            out = (self._new((n,), f32), self._new((n,), f32))
            if k > 0:
                out += (self._new((n, k), self._i32), self._new((n, k), f32))
        elif len(out) != (4 if k > 0 else 2):
            raise ValueError(f"out: want {4 if k > 0 else 2} tensors, got {len(out)}")
        ids = scores = pstats = None
        if k > 0:
            ids, scores = self._flat(out[2], (n, k), self._i32, "ids"), self._flat(out[3], (n, k), f32, "alternatives")
        if stats is not None and stats is not False:
            if stats is True:
                stats = self._new((n, DOMINO_TRAIN_LOGPROB_STATS), f32)
            pstats = self._flat(stats, (n, DOMINO_TRAIN_LOGPROB_STATS), f32, "stats")
        status = self._lib.domino_train_logprobs_forward(
            self.ctx, logits.data_ptr(), DOMINO_DTYPE_BF16 if dtype is self._bf16 else DOMINO_DTYPE_FP32, ld, n,
            self._flat(tokens, (n,), self._i32, "tokens"), temperature, self._flat(out[0], (n,), f32, "logprob"),
            self._flat(out[1], (n,), f32, "entropy"), k, ids, scores, pstats, self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_logprobs_forward")
        return tuple(out) if pstats is None else (*out, stats)

    def logprobs_backward(self, logits, tokens, stats, dlogprob, dentropy=None, temperature=1.0, out=None, stream=None):
        """dlogits [n, V] from the gradients dlogprob and dentropy [n] (None: zeros, not both) by each row's two values."""
        n = logits.shape[0]
        ld = self._rows(logits, self.V, "logits")
        if out is None:
            out = self._new((n, self.V), self.torch_dtype)
        status = self._lib.domino_train_logprobs_backward(
            self.ctx, logits.data_ptr(), ld, n, self._flat(tokens, (n,), self._i32, "tokens"), temperature,
            self._flat(stats, (n, DOMINO_TRAIN_LOGPROB_STATS), self._f32, "stats"),
            None if dlogprob is None else self._flat(dlogprob, (n,), self._f32, "dlogprob"),
            None if dentropy is None else self._flat(dentropy, (n,), self._f32, "dentropy"),
            out.data_ptr(), self._rows(out, self.V, "dlogits", n=n), self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_logprobs_backward")
        return out

    def logprobs_step(self, logits, tokens, weight, entropy_weight=None, temperature=1.0, out=None, stream=None):
        """(logprob [n], entropy [n], dlogits [n, V]) in one call; dlogits is the gradient of
        sum(weight * logprob + entropy_weight * entropy) (either may be None: zeros, not both)."""
        n = logits.shape[0]
        ld = self._rows(logits, self.V, "logits")
        if out is None:
            out = (self._new((n,), self._f32), self._new((n,), self._f32), self._new((n, self.V), self.torch_dtype))
        logprob, entropy, grad = out
        status = self._lib.domino_train_logprobs_step(
            self.ctx, logits.data_ptr(), ld, n, self._flat(tokens, (n,), self._i32, "tokens"), temperature,
            None if weight is None else self._flat(weight, (n,), self._f32, "weight"),
            None if entropy_weight is None else self._flat(entropy_weight, (n,), self._f32, "entropy_weight"),
            self._flat(logprob, (n,), self._f32, "logprob"), self._flat(entropy, (n,), self._f32, "entropy"),
            grad.data_ptr(), self._rows(grad, self.V, "dlogits", n=n), self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_logprobs_step")
        return logprob, entropy, grad

    def embed(self, table, tokens, scale=1.0, out=None, stream=None):
        """scale * table[tokens] for tokens [n] int32 (-1: zeros)."""
        n = tokens.shape[0]
        if out is None:
            out = self._new((n, self.E), self.torch_dtype)
        status = self._lib.domino_train_embed(
            self.ctx, self._flat(table, (self.V, self.E), self.torch_dtype, "table"),
            self._flat(tokens, (n,), self._i32, "tokens"), n, scale, out.data_ptr(),
            self._rows(out, self.E, "out", n=n), self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_embed")
        return out

    def embed_grad(self, dout, tokens, scale=1.0, out=None, grad_dtype=None, accumulate=False, stream=None):
        """dtable [V, E] (fp32 unless ``grad_dtype`` or ``out`` says bfloat16) from dout [n, E];
        ``accumulate`` adds to ``out``."""
        n = tokens.shape[0]
        ld = self._rows(dout, self.E, "dout", n=n)
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs out")
            out = self._new((self.V, self.E), grad_dtype or self._f32)
        dtype = out.dtype
        if (dtype is not self._bf16 and dtype is not self._f32) or (grad_dtype is not None and grad_dtype is not dtype):
            raise ValueError(f"dtable: want bfloat16 or float32 (grad_dtype {grad_dtype}), got {dtype}")
        status = self._lib.domino_train_embed_grad(
            self.ctx, dout.data_ptr(), ld, self._flat(tokens, (n,), self._i32, "tokens"), n, scale,
            self._flat(out, (self.V, self.E), dtype, "dtable"),
            DOMINO_DTYPE_BF16 if dtype is self._bf16 else DOMINO_DTYPE_FP32, 1 if accumulate else 0,
            self._stream(stream))
        if status:
            raise DominoError(status, "domino_train_embed_grad")
        return out

    # -- context -------------------------------------------------------------------

    def status(self, stream=None) -> int:
        """Synchronise the stream; return and clear the device's error word as a status code.
        After DOMINO_ERR_TIMEOUT all outputs of the distillation or scoring call that timed out are undefined."""
        return self._lib.domino_train_status(self.ctx, self._stream(stream))

    def last_launch_count(self) -> int:
        return self._lib.domino_train_last_launch_count(self.ctx)

    def close(self):
        if getattr(self, "ctx", None) is not None and self.ctx.value:
            self._lib.domino_train_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- autograd ------------------------------------------------------------------

def distill_loss(train: DominoTrain, logits, ids, top, rest=None, temperature=1.0):
    """Loss [n] of student logits [n, V], differentiable (once) by the logits."""
    return _functions()[0].apply(logits, train, ids, top, rest, temperature)


def token_logprobs(train: DominoTrain, logits, tokens, temperature=1.0, alternatives=0):
    """(logprob [n], entropy [n]) of logits [n, V] (the context's type) and their
    tokens, both differentiable (once) by the logits; with ``alternatives`` = k > 0
    also the k most likely ids [n, k] and their logprobs, which are not."""
    if logits.dtype is not train.torch_dtype:
        raise ValueError(f"logits: want {train.torch_dtype}, got {logits.dtype}")
    return _functions()[2].apply(logits, train, tokens, temperature, alternatives)


def embedding(train: DominoTrain, table, tokens, scale=1.0):
    """scale * table[tokens] [n, E], differentiable (once) by the table (whose
    gradient comes in the table's type).  Any number of tokens: more than
    ``max_tokens`` take several ``embed_grad`` calls."""
    return _functions()[1].apply(table, train, tokens, scale)


_autograd = None


def _functions():
    global _autograd
    if _autograd is None:
        import torch
        from torch.autograd.function import once_differentiable

        class Distill(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, train, ids, top, rest, temperature):
                loss, stats = train.distill_forward(logits, ids, top, rest, temperature)
                ctx.save_for_backward(logits, ids, top, rest, stats)
                ctx.train, ctx.temperature = train, temperature
                return loss

            @staticmethod
            @once_differentiable
            def backward(ctx, dloss):
                logits, ids, top, rest, stats = ctx.saved_tensors
                grad = ctx.train.distill_backward(logits, ids, top, rest, stats, dloss.contiguous(), ctx.temperature)
                return grad, None, None, None, None, None

        class Embedding(torch.autograd.Function):
            @staticmethod
            def forward(ctx, table, train, tokens, scale):
                ctx.save_for_backward(tokens)
                ctx.train, ctx.scale = train, scale
                return train.embed(table, tokens, scale)

            @staticmethod
            @once_differentiable
            def backward(ctx, dout):
                (tokens,) = ctx.saved_tensors
                if dout.stride(1) != 1 or dout.stride(0) < dout.shape[1]:
                    dout = dout.contiguous()
                train, n = ctx.train, tokens.shape[0]
                if n <= train.max_tokens:
                    return train.embed_grad(dout, tokens, ctx.scale, grad_dtype=train.torch_dtype), None, None, None
                if train.max_tokens < 1:
                    raise ValueError("embedding: the table's gradient needs a context with max_tokens > 0")
                # more tokens than one call takes: their parts add up in fp32 and are rounded once
                grad = None
                for i in range(0, n, train.max_tokens):
                    j = min(n, i + train.max_tokens)
                    grad = train.embed_grad(dout[i:j], tokens[i:j], ctx.scale, out=grad, accumulate=grad is not None)
                return grad.to(train.torch_dtype), None, None, None

        class Once(torch.autograd.Function):
            """A gradient that depends on `x` and has no derivative of its own."""
            @staticmethod
            def forward(ctx, grad, x):
                return grad.view_as(grad)

            @staticmethod
            def backward(ctx, _):
                raise RuntimeError("token_logprobs is differentiable once")

        class Logprobs(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, train, tokens, temperature, alternatives):
                *out, stats = train.logprobs_forward(logits, tokens, temperature, alternatives, stats=True)
                ctx.save_for_backward(logits, tokens, stats)
                ctx.train, ctx.temperature = train, temperature
                ctx.mark_non_differentiable(*out[2:])
                ctx.set_materialize_grads(False)
                return tuple(out)

            @staticmethod
            def backward(ctx, dlogprob, dentropy, *_):
                logits, tokens, stats = ctx.saved_tensors
                if dlogprob is None and dentropy is None:
                    return None, None, None, None, None
                d = [None if t is None else t.detach().contiguous() for t in (dlogprob, dentropy)]
                grad = ctx.train.logprobs_backward(logits.detach(), tokens, stats, *d, ctx.temperature)
                # under create_graph a second derivative raises, also where the incoming gradient has none
                return Once.apply(grad, logits) if torch.is_grad_enabled() else grad, None, None, None, None

        _autograd = (Distill, Embedding, Logprobs)
    return _autograd
