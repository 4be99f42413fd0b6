"""The update's Python binding without a GPU: a stand-in library, tensors on the CPU."""
import ctypes
import os
import pickle
import weakref
from copy import deepcopy

import pytest

torch = pytest.importorskip("torch")


class Library:
    """Takes calls and notes the gradients' addresses as they are at the time."""

    def __init__(self, count):
        self.count, self.calls, self.during = count, [], lambda: None

    def domino_adamw_init(self, ctx, cfg, device):
        return 0

    def _call(self, name, at):
        self.calls.append((name, list((ctypes.c_uint64 * self.count).from_address(at))))
        self.during()
        return 0

    def domino_adamw_step(self, ctx, addresses, dtypes, lr, lr_factor, scale, stream):
        return self._call("step", addresses)

    def domino_adamw_grad_norm(self, ctx, addresses, dtypes, most, norm, scale, stream):
        return self._call("norm", addresses)


@pytest.fixture
def make(monkeypatch):
    from speculative_decoding_draft_lm_gb300 import build, optim
    if not os.path.exists(build.ARGS):
        build.build()
    device = torch.device

    def make(params, **kw):
        params = list(params)
        lib = Library(len(params))
        with monkeypatch.context() as m:
            m.setattr(optim, "load_library", lambda: lib)
            m.setattr(torch, "device", lambda *a: device("cpu"))
            opt = optim.DominoAdamW(params, device=-1, **kw)
        opt._current_stream = lambda i: 0
        return opt, lib

    return make


def _both(opt, match, **kw):
    for call in (opt.step, opt.grad_norm):
        with pytest.raises(ValueError, match=match):
            call(**kw)


def test_calls_reach_the_library(make):
    p = [torch.zeros(4, 3), torch.zeros(5, dtype=torch.bfloat16), torch.zeros(0)]
    opt, lib = make(p)
    g = [torch.ones(4, 3), None, torch.ones(0)]
    opt.step(grads=g)
    opt.grad_norm(grads=g)
    assert lib.calls == [(n, [g[0].data_ptr(), 0, 0]) for n in ("step", "norm")]


def test_a_parameter_that_became_another_is_refused(make):
    """Fewer elements, another type or another order at the same address: the context holds what was there first."""
    def half(t):
        t.data = t.data[:2]

    def typed(t):
        t.data = t.data.view(torch.bfloat16)

    def turned(t):
        t.data = t.data.t()

    def larger(t):
        t.data = t.data.as_strided((8, 3), (0, 1))

    def moved(t):
        t.data = t.data.clone()

    for change in (half, typed, turned, larger, moved):
        p = [torch.zeros(7), torch.zeros(4, 3)]
        opt, lib = make(p)
        at = p[1].data_ptr()
        opt.step(grads=[torch.ones(7), torch.ones(4, 3)])
        change(p[1])
        assert change is moved or p[1].data_ptr() == at
        g = [torch.ones(7), torch.ones(p[1].shape).to(p[1].dtype)]
        _both(opt, "params.1.*no longer", grads=g)
        _both(opt, "params.1.*no longer", grads=[g[0], None])
        p[1].grad = g[1]
        _both(opt, "params.1.*no longer")
        assert len(lib.calls) == 1
    # the same elements in another shape are the same
    p = [torch.zeros(4, 3)]
    opt, lib = make(p)
    p[0].data = p[0].data.view(12)
    opt.step(grads=[torch.ones(12)])
    assert len(lib.calls) == 1


def test_what_the_context_holds_cannot_be_swapped(make):
    """The list of parameters and the dict of buffers are views to read: the context goes by what it was made with."""
    p = [torch.zeros(40), torch.zeros(50)]
    given = list(p)
    opt, lib = make(given)
    given.append(torch.zeros(3))
    given[0] = torch.zeros(2)
    assert len(opt.params) == 2 and all(a is b for a, b in zip(opt.params, p))
    for change in (lambda: opt.params.append(p[0]), lambda: opt.params.pop(), lambda: opt.params.clear()):
        with pytest.raises(AttributeError):
            change()
    with pytest.raises(TypeError):
        opt.params[0] = torch.zeros(40)
    with pytest.raises(AttributeError):
        opt.params = p[:1]
    for change in (lambda: opt.state.update(m=opt.state["v"]), lambda: opt.state.pop("m"), lambda: opt.state.clear()):
        with pytest.raises(TypeError, match="settled"):
            change()
    with pytest.raises(TypeError, match="settled"):
        opt.state["m"] = torch.zeros_like(opt.state["m"])
    with pytest.raises(TypeError):
        del opt.state["m"]
    with pytest.raises(AttributeError):
        opt.state = opt.state_dict()
    copy = opt.state_dict()
    copy["m"] = copy.pop("v")
    for other in (pickle.loads(pickle.dumps(opt.state)), deepcopy(opt.state)):  # ordinary dicts, of tensors of their own
        assert type(other) is dict and torch.equal(other["m"], opt.state["m"])
        other["m"] = other["m"] + 1
    assert set(opt.state) == {"m", "v", "count"} and opt.state["m"] is not copy["m"]
    opt.step(grads=[torch.ones(40), torch.ones(50)])
    assert len(lib.calls) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_a_buffer_that_became_another_is_refused(make, bits):
    names = ["m", "v", "master", "count"] + (["m_scale", "v_scale"] if bits == 8 else [])
    for name in names:
        opt, lib = make([torch.zeros(300, dtype=torch.bfloat16)], state_bits=bits, master=True)
        assert sorted(opt.state) == sorted(names)
        g = [torch.ones(300)]
        opt.step(grads=g)
        opt.state[name].data = opt.state[name].data.clone()
        _both(opt, f"state.'{name}'.*no longer", grads=g)
        opt, lib = make([torch.zeros(300, dtype=torch.bfloat16)], state_bits=bits, master=True)
        opt.state[name].data = opt.state[name].data[:0]
        _both(opt, f"state.'{name}'.*no longer", grads=g)
        assert lib.calls == []


def test_gradients_of_a_generator(make):
    """Tensors that nobody else holds live until the launch is enqueued; a bad one is named; an iterator's tensors on a
    stream of the caller's, whom nothing lets keep them, are refused."""
    p = [torch.zeros(40), torch.zeros(50)]
    opt, lib = make(p)
    for call in (opt.step, opt.grad_norm):
        held = []

        def gradients():
            for t in p:
                g = torch.ones_like(t)
                held.append((weakref.ref(g), g.data_ptr()))
                yield g

        alive = []
        lib.during = lambda: alive.extend(r() is not None for r, _ in held)
        call(grads=gradients())
        assert alive == [True, True] and lib.calls[-1][1] == [at for _, at in held]
        lib.during = lambda: None
        with pytest.raises(ValueError, match="grads.1.*float64"):
            call(grads=(g for g in [torch.ones(40), torch.ones(50).double()]))
        with pytest.raises(ValueError, match="grads.0.*want a tensor or None"):
            call(grads=(g for g in [3.0, None]))
        with pytest.raises(ValueError, match="2 tensors"):
            call(grads=(g for g in [None]))
        with pytest.raises(TypeError):
            call(grads=5)
        with pytest.raises(ValueError, match="list"):
            call(grads=gradients(), stream=7)
        call(grads=dict(enumerate(map(torch.ones_like, p))).values(), stream=7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float64])
@pytest.mark.parametrize("bits", [32, 8])
def test_another_default_type(make, dtype, bits):
    """What the binding makes itself is of its own types, whatever torch's default."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(dtype)
    try:
        opt, lib = make([torch.zeros(40, dtype=torch.float32), torch.zeros(50, dtype=torch.bfloat16)], state_bits=bits,
                        master=True)
        g = [torch.ones(40, dtype=torch.float32), None]
        norm, scale = opt.grad_norm(grads=g)
        opt.step(grads=g, scale=scale)
        m, v = opt.moments(1)
    finally:
        torch.set_default_dtype(before)
    assert all(t.dtype is torch.float32 for t in (norm, scale, m, v)) and len(lib.calls) == 2
