"""CPU checks of the weights' update: the C ABI, argument checks that answer without a
GPU, and the oracle."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import optim_oracle as O

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "domino_optim.h")).read()


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_lm_gb300 import build, optim, rollout
    if not (os.path.exists(rollout.LIB_PATH) and os.path.exists(build.ARGS)):
        build.build()
    return optim.load_library()


def test_library_exports_every_declared_symbol(lib):
    from speculative_decoding_draft_lm_gb300 import optim
    declared = sorted(set(re.findall(r"DOMINO_API\s+[\w\s\*]+?\b(domino_\w+)\s*\(", HEADER)))
    assert declared == sorted(optim.EXPORTED)
    for name in declared:
        assert hasattr(lib, name), name
    for name in ("DOMINO_ADAMW_BLOCK", "DOMINO_ADAMW_MAX_TENSORS"):
        assert int(re.search(rf"#define {name} +(\d+)", HEADER).group(1)) == getattr(optim, name)


def test_null_context(lib):
    from speculative_decoding_draft_lm_gb300 import rollout as R
    assert lib.domino_adamw_step(None, None, None, 1e-3, None, None, None) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_adamw_grad_norm(None, None, None, 1.0, None, None, None) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_adamw_last_launch_count(None) == 0
    lib.domino_adamw_destroy(None)


GOOD = dict(n_tensors=2, state_bits=8, m=0x10000, v=0x20000, m_scale=0x30000, v_scale=0x31000, master=None, count=0x32000,
            beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, seed=0)


def _init(lib, tensors=((0x40000, 1000, 1, 0), (0x50000, 7, 0, 0)), **kw):
    """Status of an init that never gets to use its addresses (or finds no device)."""
    from speculative_decoding_draft_lm_gb300 import optim
    a = (optim.domino_adamw_tensor * len(tensors))(*[optim.domino_adamw_tensor(*t) for t in tensors])
    f = dict(GOOD, tensors=a, n_tensors=len(tensors))
    f.update(kw)
    cfg, ctx = optim.domino_adamw_config(**f), ctypes.c_void_p()
    # device -1 exists nowhere: what passes the checks answers CUDA
    status = lib.domino_adamw_init(ctypes.byref(ctx), ctypes.byref(cfg), -1)
    assert not ctx.value
    return status


def test_config_validation_precedes_device_access(lib):
    from speculative_decoding_draft_lm_gb300 import rollout as R
    bad, unsupported, passed = R.DOMINO_ERR_INVALID_ARG, R.DOMINO_ERR_UNSUPPORTED, R.DOMINO_ERR_CUDA
    assert _init(lib) == passed
    assert _init(lib, state_bits=32) == passed
    assert _init(lib, state_bits=16) == unsupported
    assert _init(lib, tensors=((0x40000, 10, 2, 0),)) == unsupported
    assert _init(lib, tensors=((0x40000, 10, 1, 1),)) == bad           # a master without a buffer
    assert _init(lib, tensors=((0x40000, 10, 1, 1),), master=0x60000) == passed
    assert _init(lib, tensors=((0x40000, 10, 0, 1),), master=0x60000) == bad  # of fp32
    assert _init(lib, tensors=((0x40001, 10, 1, 0),)) == bad
    assert _init(lib, tensors=((0x40002, 10, 1, 0),)) == passed
    assert _init(lib, tensors=((0x40002, 10, 0, 0),)) == bad
    assert _init(lib, tensors=((None, 10, 0, 0),)) == bad
    assert _init(lib, tensors=((None, 0, 0, 0),)) == passed
    assert _init(lib, tensors=((0x40000, -1, 0, 0),)) == bad
    assert _init(lib, tensors=((0x40000, 1 << 39, 0, 0),)) == bad
    # the same tensor twice, one inside another, one over a buffer
    assert _init(lib, tensors=((0x40000, 10, 1, 0), (0x40000, 10, 1, 0))) == bad
    assert _init(lib, tensors=((0x40000, 1000, 1, 0), (0x40010, 4, 0, 0))) == bad
    assert _init(lib, tensors=((0x40000, 8, 1, 0), (0x40010, 4, 0, 0))) == passed
    assert _init(lib, tensors=((0x10040, 8, 1, 0),)) == bad
    for name in ("m", "v", "m_scale", "v_scale", "count"):
        assert _init(lib, **{name: None}) == bad
        assert _init(lib, **{name: GOOD[name] + 2}) == bad
    for kw in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-17),
               dict(eps=2.0), dict(weight_decay=-1e-3), dict(weight_decay=1.5), dict(n_tensors=0), dict(n_tensors=65537)):
        assert _init(lib, **kw) == bad, kw
    assert _init(lib, beta1=0.0, beta2=0.0, eps=1.0, weight_decay=1.0) == passed


def test_python_refusals():
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    p = torch.zeros(3)
    for kw, match in ((dict(state_bits=16), "state_bits"), (dict(seed=-1), "seed"), (dict(seed=2 ** 32), "seed"),
                      (dict(seed=0.5), "seed"), (dict(), "params")):
        with pytest.raises(ValueError, match=match):
            DominoAdamW([p], **kw)
    with pytest.raises(ValueError, match="1 to"):
        DominoAdamW([])


def test_gradients_are_read(lib):
    """The module that reads a step's tensors, on the CPU (device -1)."""
    from speculative_decoding_draft_lm_gb300 import optim
    args = optim._load_args()
    params = [torch.zeros(4, 3), torch.zeros(5, dtype=torch.bfloat16), torch.zeros(0)]
    at, codes = (ctypes.c_uint64 * 3)(), (ctypes.c_int * 3)()
    held = (ctypes.c_uint64 * 3)(*[p.data_ptr() for p in params])

    def read(grads, device=-1):
        return args.gradients(params, grads, device, ctypes.addressof(held), ctypes.addressof(at), ctypes.addressof(codes))

    g = [torch.ones(4, 3).bfloat16(), torch.ones(5), torch.ones(0)]
    assert read(g) == -1 and list(at)[:2] == [t.data_ptr() for t in g[:2]] and list(codes) == [1, 0, 0]
    assert read(tuple(g)) == -1
    assert read([None, g[1], None]) == -1 and list(at) == [0, g[1].data_ptr(), 0]
    assert read(None) == -1 and list(at) == [0, 0, 0]
    params[0].grad = torch.ones(4, 3)
    assert read(None) == -1 and at[0] == params[0].grad.data_ptr() and at[1] == 0
    assert read(g, device=0) == 0
    for place, wrong in ((0, torch.ones(3, 4)), (0, torch.ones(3, 4).t()), (0, torch.ones(12)), (1, torch.ones(5).half()),
                         (1, torch.ones(5).double()), (1, torch.ones(10)[::2]), (0, 3.0), (1, torch.ones(5).to_sparse())):
        bad = list(g)
        bad[place] = wrong
        assert read(bad) == place, wrong
    with pytest.raises(ValueError, match="3 tensors"):
        read(g[:2])
    with pytest.raises(TypeError):
        read(7)
    held[1] += 2  # a parameter that lies elsewhere by now
    assert read(g) == -3
    held[1] -= 2
    read([None, g[1], None])
    versions = [p._version for p in params]
    args.written(params, ctypes.addressof(at))
    assert [p._version for p in params] == [versions[0], versions[1] + 1, versions[2]]


def test_narrow_against_torch():
    """The oracle's codes are e4m3: torch reads the same values, a value on the grid stays, others go to a neighbour
    with the probability of their place."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    values = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(values[:127], O.VALUES[:127]) and np.array_equal(values[128:255], O.VALUES[128:255])
    g = np.random.default_rng(0)
    a = np.concatenate([O.VALUES[:127], [0.0]]).astype(np.float32)
    for random in (0, 2 ** 20 - 1):
        c, s = O.narrow(a, np.full(128, random), 0)
        assert s[0] == 1 and np.array_equal(O.VALUES[c], a)
    # 2^-9 * 0.3 of the largest's scale, and values in every binade
    a = np.tile(np.concatenate([[448.0], 448 * g.random(127) ** 8]), 4000).astype(np.float32)
    c, s = O.narrow(a, O.words(np.arange(a.size), 5, 9) >> np.uint64(12), 0)
    mean = O.VALUES[c].reshape(4000, 128).mean(0)
    x = a[:128].astype(np.float64)
    step = np.maximum(2.0 ** np.floor(np.log2(x)), 2.0 ** -6) / 8
    # the mean of 4000 draws of one step, each with a deviation of half a step at most: five deviations
    assert (np.abs(mean - x) <= 5 * 0.5 * step / np.sqrt(4000) + step * 2.0 ** -19).all()


def test_step_against_torch():
    g = torch.Generator().manual_seed(0)
    p = torch.randn(50, generator=g, dtype=torch.float64).requires_grad_()
    opt = torch.optim.AdamW([p], lr=1e-2, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        opt.step()
        q, m, v = O.step(q, m, v, p.grad.numpy(), t, lr=1e-2, decay=0.1)
        assert np.allclose(p.detach().numpy(), q, rtol=1e-12, atol=1e-14)


def test_words_are_uniform():
    """Mean and pairwise bits of the random words over positions and over steps."""
    for w in (O.words(np.arange(200000), 7, 1), np.asarray([int(O.words([5], t, 1)[0]) for t in range(20000)])):
        w = w.astype(np.uint64)
        n = w.size
        for b in range(32):
            ones = ((w >> np.uint64(b)) & np.uint64(1)).mean()
            assert abs(ones - 0.5) < 5 * 0.5 / np.sqrt(n), b
        x = w.astype(np.float64) / 2 ** 32
        assert abs(np.corrcoef(x[:-1], x[1:])[0, 1]) < 5 / np.sqrt(n)
