"""Python binding of the weights' update in ``include/domino_optim.h`` (ctypes, and
a C++ module that reads the tensors of a step): argument marshalling and the flat
buffers of the moments.  ``DominoAdamW`` takes
torch CUDA tensors and the current torch stream.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes

from . import rollout as _r
from .rollout import DOMINO_DTYPE_BF16, DOMINO_DTYPE_FP32, DominoError, _check

DOMINO_ADAMW_BLOCK = 128
DOMINO_ADAMW_MAX_TENSORS = 65536

# every symbol the header declares
EXPORTED = (
    "domino_adamw_init", "domino_adamw_step", "domino_adamw_grad_norm", "domino_adamw_last_launch_count",
    "domino_adamw_destroy",
)


class domino_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("n", ctypes.c_longlong), ("dtype", ctypes.c_int),
                ("master", ctypes.c_int)]


class domino_adamw_config(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int), ("tensors", ctypes.POINTER(domino_adamw_tensor)),
                ("state_bits", ctypes.c_int), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("count", ctypes.c_void_p), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("seed", ctypes.c_uint)]


_lib = None


def load_library() -> ctypes.CDLL:
    """The rollout's library with the update's entry points declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _r.load_library()
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.domino_adamw_init.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(domino_adamw_config), i]
    lib.domino_adamw_step.argtypes = [vp, vp, vp, ctypes.c_double, vp, vp, vp]
    lib.domino_adamw_grad_norm.argtypes = [vp, vp, vp, f, vp, vp, vp]
    lib.domino_adamw_last_launch_count.argtypes = [vp]
    lib.domino_adamw_destroy.argtypes = [vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib.domino_adamw_destroy.restype = None
    _lib = lib
    return lib


def _load_args():
    """The C++ module that reads a step's tensors (built beside the library)."""
    import torch  # its libraries first
    build = "python -m speculative_decoding_draft_lm_gb300.build"
    try:
        from . import _optim_args
    except ImportError as e:
        raise ImportError(f"the module that reads a step's tensors is not built for this Python and torch: {build}") from e
    built_for = getattr(_optim_args, "torch_version", None)
    if built_for != torch.__version__:
        raise ImportError(f"the module that reads a step's tensors was built for torch {built_for}, this is "
                          f"{torch.__version__}: {build}")
    return _optim_args


class _Buffers(dict):
    """A dict whose entries are settled; copied and pickled as an ordinary one."""

    def _refuse(self, *a, **kw):
        raise TypeError("the buffers of an optimizer are settled: copy into them, or make a new one with state=")

    __setitem__ = __delitem__ = __ior__ = update = setdefault = pop = popitem = clear = _refuse

    def __reduce__(self):
        return dict, (dict(self),)


class DominoAdamW:
    """AdamW over a list of tensors (see the header for the formulas).

    ``params``: contiguous bf16 or fp32 CUDA tensors on ``device``, updated in
    place; they may be leaves that require gradients.  ``state_bits``: 32 or 8.
    ``master``: an exact fp32 copy of the bf16 ones is kept and updated, and they
    get its values rounded; without it they are rounded stochastically, from
    ``seed`` (an integer below 2^32).

    ``state``: a dict of the flat buffers (a ``state_dict``), used as they are;
    None makes new ones.  Tensor i lies at ``offsets[i]`` of each; ``m`` and ``v``
    are float32, or float8_e4m3fn with float32 ``m_scale`` and ``v_scale`` for
    every 128 positions; ``master`` is float32; ``count`` int64 [1] holds the
    steps taken.

    The tensors and buffers are updated where they are: which ones is settled, and calls with one
    whose ``.data`` was replaced are refused.  A captured step reads the gradients at the
    capture's addresses on every replay.

    Every method takes ``stream`` (a torch stream or raw handle; default: the
    current one).  With a stream other than the current one the caller orders the
    two, as for any kernel, keeps the gradients until the call is done, and gives ``out``.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32, master=False,
                 seed=0, state=None, device=0):
        import torch
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits: want 8 or 32, got {state_bits!r}")
        if not isinstance(seed, int) or not 0 <= seed < 2 ** 32:
            raise ValueError(f"seed: want an integer in [0, 2^32), got {seed!r}")
        self._codes = {torch.bfloat16: DOMINO_DTYPE_BF16, torch.float32: DOMINO_DTYPE_FP32}
        self._params, self.lr, self.state_bits = list(params), lr, state_bits
        self.device, self._index = torch.device("cuda", device), device
        if not 1 <= len(self._params) <= DOMINO_ADAMW_MAX_TENSORS:
            raise ValueError(f"params: want 1 to {DOMINO_ADAMW_MAX_TENSORS} tensors, got {len(self._params)}")
        for i, p in enumerate(self._params):
            if p.dtype not in self._codes or p.get_device() != device or not p.is_contiguous():
                raise ValueError(f"params[{i}]: want contiguous CUDA bfloat16 or float32 on {self.device}, "
                                 f"got {tuple(p.shape)} {p.dtype} strides {p.stride()} on {p.device}")
        self.offsets, total = [], 0
        for p in self._params:
            self.offsets.append(total)
            total += -(-p.numel() // DOMINO_ADAMW_BLOCK) * DOMINO_ADAMW_BLOCK
        self.master = bool(master) and any(p.dtype is torch.bfloat16 for p in self._params)
        narrow, blocks = state_bits == 8, total // DOMINO_ADAMW_BLOCK
        moment = torch.float8_e4m3fn if narrow else torch.float32
        want = {"m": ((total,), moment), "v": ((total,), moment), "count": ((1,), torch.int64)}
        if narrow:
            want.update(m_scale=((blocks,), torch.float32), v_scale=((blocks,), torch.float32))
        if self.master:
            want["master"] = ((total,), torch.float32)
        if state is None:
            state = {n: torch.zeros(shape, dtype=dtype, device=self.device) for n, (shape, dtype) in want.items()}
            if self.master:
                for p, at in zip(self._params, self.offsets):
                    state["master"][at:at + p.numel()].copy_(p.detach().reshape(-1))
        if set(state) != set(want):
            raise ValueError(f"state: want {sorted(want)}, got {sorted(state)}")
        for n, (shape, dtype) in want.items():
            t = state[n]
            if tuple(t.shape) != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
                raise ValueError(f"state[{n!r}]: want contiguous CUDA {shape} {dtype} on {self.device}, "
                                 f"got {tuple(t.shape)} {t.dtype} on {t.device}")
        self._state = _Buffers((n, state[n]) for n in want)
        # the raw handle where torch gives it: a Stream object costs more than a launch
        self._current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                       lambda i: torch.cuda.current_stream(i).cuda_stream)
        self._f32 = torch.float32
        count = len(self._params)
        tensors = (domino_adamw_tensor * count)(*[
            domino_adamw_tensor(p.data_ptr(), p.numel(), self._codes[p.dtype],
                                int(self.master and p.dtype is torch.bfloat16)) for p in self._params])
        self._addresses, self._dtypes = (ctypes.c_uint64 * count)(), (ctypes.c_int * count)()
        self._held = (ctypes.c_uint64 * count)(*[p.data_ptr() for p in self._params])
        self._sizes = (ctypes.c_int64 * count)(*[p.numel() for p in self._params])
        self._types = (ctypes.c_int * count)(*[self._codes[p.dtype] for p in self._params])
        self._buffers = list(self._state.values())
        self._buffers_held = (ctypes.c_uint64 * (2 * len(self._buffers)))(
            *[x for t in self._buffers for x in (t.data_ptr(), t.numel() * t.element_size())])
        self._addresses_at, self._dtypes_at = ctypes.addressof(self._addresses), ctypes.addressof(self._dtypes)
        address = {n: self._state[n].data_ptr() if n in want else None
                   for n in ("m", "v", "m_scale", "v_scale", "master", "count")}
        cfg = domino_adamw_config(count, tensors, state_bits, address["m"], address["v"], address["m_scale"],
                                  address["v_scale"], address["master"], address["count"], betas[0], betas[1], eps,
                                  weight_decay, seed)
        self._lib = load_library()
        # reads a step's gradients, and counts its change of the parameters; the arrays and lists are this object's
        self._read, self._written = _load_args().plan(
            self._params, device, ctypes.addressof(self._held), self._addresses_at, self._dtypes_at,
            ctypes.addressof(self._sizes), ctypes.addressof(self._types), self._buffers,
            ctypes.addressof(self._buffers_held))
        self.ctx = ctypes.c_void_p()
        _check(self._lib.domino_adamw_init(ctypes.byref(self.ctx), ctypes.byref(cfg), device), "domino_adamw_init")

    @property
    def params(self):
        """The tensors, as a tuple: which ones they are is settled."""
        return tuple(self._params)

    @property
    def state(self):
        """The flat buffers by name, to read and to fill, not to replace."""
        return self._state

    # -- checks (on every call's path) ----------------------------------------------

    def _gradients(self, grads, stream):
        """Puts the gradients' addresses and types into this context's arrays.  Returns what has to live until the
        launch is enqueued."""
        if grads.__class__ is not list and not (grads is None or isinstance(grads, (list, tuple))):
            if stream is not None and hasattr(grads, "__next__"):
                raise ValueError("grads: want a list of tensors, which the caller keeps, where a stream is given")
            grads = list(grads)
        bad = self._read(grads)
        if bad < -1:
            i, n = -2 - bad, len(self._params)
            name = f"params[{i}]" if i < n else f"state[{list(self._state)[i - n]!r}]"
            raise ValueError(f"{name}: its elements are no longer what and where they were when this optimizer was made "
                             "(its .data was replaced): make a new one with state=state_dict()")
        if bad >= 0:
            g = self._params[bad].grad if grads is None else grads[bad]
            if not hasattr(g, "dtype"):
                raise ValueError(f"grads[{bad}]: want a tensor or None, got {type(g).__name__}")
            raise ValueError(f"grads[{bad}]: want contiguous CUDA {tuple(self._params[bad].shape)} bfloat16 or float32 on "
                             f"{self.device}, got {tuple(g.shape)} {g.dtype} strides {g.stride()} on {g.device}")
        return grads

    def _scalar(self, t, name):
        """The address of one fp32 number on the device, or None."""
        if t is None:
            return None
        if t.dtype is self._f32 and t.numel() == 1 and t.get_device() == self._index:
            return t.data_ptr()
        raise ValueError(f"{name}: want one float32 on {self.device}, got {tuple(t.shape)} {t.dtype} on {t.device}")

    def _stream(self, stream):
        if stream is None:
            return self._current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    # -- operators ---------------------------------------------------------------

    def grad_norm(self, max_norm=1.0, grads=None, out=None, stream=None):
        """(norm, scale): the norm of all gradients together and min(1, max_norm / norm), NaN where
        the norm is not finite; both stay on the device.  ``grads``: a tensor or None for every
        parameter (default: their ``.grad``)."""
        if out is None:
            import torch
            out = [torch.empty((), dtype=self._f32, device=self.device) for _ in range(2)]
        norm, scale = out
        grads = self._gradients(grads, stream)
        status = self._lib.domino_adamw_grad_norm(self.ctx, self._addresses_at, self._dtypes_at, max_norm,
                                                  self._scalar(norm, "norm"), self._scalar(scale, "scale"),
                                                  self._stream(stream))
        if status:
            raise DominoError(status, "domino_adamw_grad_norm")
        return norm, scale

    def step(self, grads=None, scale=None, lr=None, lr_factor=None, stream=None):
        """One step with the gradients times ``scale`` (one float32 on the device, such as
        ``grad_norm`` gives; a step whose scale is not finite is left out).  ``grads`` as for
        ``grad_norm``; a parameter without one is left as it is.  ``lr`` replaces the constructor's;
        ``lr_factor`` (one float32 on the device) multiplies it, for schedules of captured steps."""
        grads = self._gradients(grads, stream)
        status = self._lib.domino_adamw_step(self.ctx, self._addresses_at, self._dtypes_at,
                                             self.lr if lr is None else lr, self._scalar(lr_factor, "lr_factor"),
                                             self._scalar(scale, "scale"), self._stream(stream))
        if status:
            raise DominoError(status, "domino_adamw_step")
        self._written()

    # -- state ---------------------------------------------------------------------

    def steps(self) -> int:
        """The steps taken (synchronises with the device)."""
        return int(self.state["count"].item())

    def moments(self, i):
        """(m, v) of parameter i in float32, in its shape."""
        p, at = self._params[i], self.offsets[i]
        n, out = p.numel(), []
        for name in ("m", "v"):
            a = self._state[name][at:at + n].float()
            if self.state_bits == 8:
                j = at // DOMINO_ADAMW_BLOCK
                s = self._state[name + "_scale"][j:j + -(-n // DOMINO_ADAMW_BLOCK)]
                a = a * s.repeat_interleave(DOMINO_ADAMW_BLOCK)[:n]
            out.append(a.view(p.shape))
        return tuple(out)

    def state_dict(self):
        """The flat buffers themselves; ``state=`` of a new optimizer over tensors of the same sizes."""
        return dict(self._state)

    def zero_grad(self):
        for p in self._params:
            p.grad = None

    def last_launch_count(self) -> int:
        return self._lib.domino_adamw_last_launch_count(self.ctx)

    def close(self):
        if getattr(self, "ctx", None) is not None and self.ctx.value:
            self._lib.domino_adamw_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
