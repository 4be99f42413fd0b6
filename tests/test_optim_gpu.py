"""AdamW over many tensors and the gradients' norm against the oracle."""
import math

import numpy as np
import pytest

from oracle import optim_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BLOCK = 128
SIZES = [1, 127, 128, 129, 4096, 4097, 5, 12289, 70001]


def _optim(*a, **kw):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    return DominoAdamW(*a, **kw)


class Tensors:
    """Tensors of the given sizes cut out of one buffer, `shift` elements off its start and off each other, NaN around."""

    def __init__(self, sizes, dtype, shift, values):
        self.buf = torch.full((sum(sizes) + (len(sizes) + 1) * max(shift, 16),), float("nan"), dtype=dtype, device="cuda")
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.parts, at = [], shift
        for n, v in zip(sizes, values):
            self.parts.append(self.buf[at:at + n])
            self.parts[-1].copy_(torch.as_tensor(v))
            self.mask[at:at + n] = False
            at += n + shift if shift else -(-n // 16) * 16

    def check_around(self):
        assert torch.isnan(self.buf[self.mask]).all()


def _draw(g, sizes, scale, zeros=0.0):
    return [(g.normal(0, scale, n) * (g.random(n) >= zeros) * np.exp(g.normal(0, 1, n))).astype(np.float32) for n in sizes]


def update_tolerance(p, m, v, t, lr, eps, decay):
    """Of the new parameter before its rounding to its type: two products and a sum on |p|; the update's own factors
    (square root and quotient of 2 ulp each, a dozen roundings, the bias corrections' 4 each), and of m's
    two products and sum, which may cancel, through the parts it is made of."""
    root = np.sqrt(v / (1 - 0.999 ** t)) + eps
    return 3 * EPS32 * np.abs(p) * (1 + lr * decay) + lr / (1 - 0.9 ** t) * np.abs(m) / root * 40 * EPS32


def run_steps(sizes, dtype, grad, bits, master, shift, steps=3, gaps=True, grad_shift=None, seed=5, **kw):
    """Steps of the library with the oracle beside it, which starts every step from the library's own state."""
    g = np.random.default_rng(len(sizes) + bits + steps)
    lr, eps, decay = 1e-3, 1e-8, 0.1
    params = Tensors(sizes, TORCH[dtype], shift, _draw(g, sizes, 0.5))
    opt = _optim(params.parts, lr=lr, eps=eps, weight_decay=decay, state_bits=bits, master=master, seed=seed)
    names = [n for n in ("m", "v", "master") if n in opt.state]
    total = opt.state["m"].numel()
    gap = torch.ones(total, dtype=torch.bool, device="cuda")
    for at, n in zip(opt.offsets, sizes):
        gap[at:at + n] = False
    for n in names:  # what lies between two tensors is nobody's
        view = opt.state[n].view(torch.uint8) if bits == 8 and n != "master" else opt.state[n]
        view[gap] = 77
    scale = torch.full((), 0.75, device="cuda")
    for t in range(1, steps + 1):
        grads = Tensors(sizes, TORCH[grad], shift if grad_shift is None else grad_shift, _draw(g, sizes, 1e-2, zeros=0.3))
        before = [(wide(p), [wide(a) for a in opt.moments(i)],
                   wide(opt.state["master"][opt.offsets[i]:opt.offsets[i] + sizes[i]]) if "master" in opt.state else None)
                  for i, p in enumerate(params.parts)]
        opt.step(grads=grads.parts, scale=scale)
        torch.cuda.synchronize()
        assert opt.steps() == t
        params.check_around()
        grads.check_around()
        for i, n in enumerate(sizes):
            at, gr = opt.offsets[i], wide(grads.parts[i])
            p0, (m0, v0), w0 = before[i]
            p0 = p0 if w0 is None else w0
            p1, m1, v1 = O.step(p0, m0, v0, gr, t, lr=lr, eps=eps, decay=decay, scale=0.75)
            tol = update_tolerance(p0, 0.9 * np.abs(m0) + 0.1 * 0.75 * np.abs(gr), v1, t, lr, eps, decay)
            got = wide(params.parts[i])
            h = O.words(at + np.arange(n), t, seed)
            if w0 is not None:
                w1 = wide(opt.state["master"][at:at + n])
                assert (np.abs(w1 - p1) <= tol).all()
                assert torch.equal(params.parts[i], opt.state["master"][at:at + n].to(torch.bfloat16))
            elif dtype == "bf16":
                # one of the two neighbours, up where the place between them and the random bits carry
                carry = (torch.as_tensor(p1).float().view(torch.int32).long()
                         + torch.as_tensor((h >> np.uint64(4)).astype(np.int64) & 0xFFFF)).bitwise_and(~0xFFFF)
                want = carry.int().view(torch.float32).double().numpy()
                bad = got != want
                # where the place is within the tolerance of the random bits either neighbour may come
                place = np.abs(((torch.as_tensor(p1).float().view(torch.int32).long() & 0xFFFF).numpy()
                                + ((h >> np.uint64(4)).astype(np.int64) & 0xFFFF)) - 0x10000)
                unit = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(p1), 2.0 ** -126))) - 23)
                near = place * unit <= tol + unit
                assert not (bad & ~near).any(), (i, np.argwhere(bad & ~near)[:3])
                step = unit * 2.0 ** 16
                assert (np.abs(got - p1) <= step + tol).all()
            else:
                assert (np.abs(got - p1) <= tol).all(), (i, np.abs(got - p1).max())
            m32, v32 = O.moments32(m0, v0, gr, 0.75, 0.9, 0.999)
            if bits == 32:
                assert np.array_equal(opt.state["m"][at:at + n].cpu().numpy(), m32)
                assert np.array_equal(opt.state["v"][at:at + n].cpu().numpy(), v32)
            else:
                pad = np.zeros(-(-n // BLOCK) * BLOCK - n, np.float32)
                hp = O.words(at + np.arange(n + pad.size), t, seed)
                for name, a, random, least in (("m", m32, hp & np.uint64(0xFFFFF), 0), ("v", v32, hp >> np.uint64(12), 1)):
                    code, s = O.narrow(np.concatenate([a, pad]), random, least)
                    j = at // BLOCK
                    assert np.array_equal(opt.state[name + "_scale"][j:j + s.size].cpu().numpy(), s)
                    assert np.array_equal(opt.state[name].view(torch.uint8)[at:at + n].cpu().numpy(), code[:n])
            # and in 64 bits: within a rounding, or within one step of e4m3
            got_m, got_v = (wide(a) for a in opt.moments(i))
            if bits == 32:
                assert (np.abs(got_m - m1) <= 4 * EPS32 * (0.9 * np.abs(m0) + 0.1 * np.abs(gr))).all()
                assert (np.abs(got_v - v1) <= 6 * EPS32 * v1 + 1e-45).all()
            else:
                for got_a, a, name in ((got_m, m1, "m"), (got_v, v1, "v")):
                    s = wide(opt.state[name + "_scale"])[at // BLOCK:at // BLOCK + -(-n // BLOCK)].repeat(BLOCK)[:n]
                    y = np.abs(a) / s
                    step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(y, 2.0 ** -30))), 2.0 ** -6) / 8
                    assert (np.abs(got_a - a) <= s * step * 1.001).all()
                assert ((got_v > 0) == (v32 > 0)).all()
        for n in names:
            view = opt.state[n].view(torch.uint8) if bits == 8 and n != "master" else opt.state[n]
            assert (view[gap] == 77).all()
    return opt


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("fp32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_steps(bits, dtype, master, grad, shift):
    run_steps(SIZES, dtype, grad, bits, master, shift)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [4095], [4096 * 700 + 3], [3] * 17, [40] * 101, [130] * 1003])
def test_numbers_and_sizes_of_tensors(bits, sizes):
    """One tensor, many tiles, and every size of a launch's table; more tensors than a launch takes."""
    opt = run_steps(sizes, "bf16", "bf16", bits, False, 0, steps=1)
    assert opt.last_launch_count() == (2 if len(sizes) > 1000 else 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_aligned_otherwise_than_parameters(bits):
    run_steps(SIZES, "bf16", "fp32", bits, False, 0, steps=1, grad_shift=3)
    run_steps(SIZES, "fp32", "bf16", bits, False, 3, steps=1, grad_shift=0)


@pytest.mark.parametrize("bits", [32, 8])
def test_against_torch(bits):
    """Twenty steps beside torch.optim.AdamW: fp32 to its roundings; with 8 bits the moments are noisy, but not off."""
    torch.manual_seed(0)
    n = 200000
    p = torch.randn(n, device="cuda")
    q = p.double().requires_grad_()
    ref = torch.optim.AdamW([q], lr=1e-3, weight_decay=0.01)
    opt = _optim([p], lr=1e-3, state_bits=bits)
    start = p.clone()
    for _ in range(20):
        g = torch.randn(n, device="cuda") * 1e-3 + 1e-3
        q.grad = g.double()
        ref.step()
        opt.step(grads=[g])
    if bits == 32:
        # each step: 3 roundings of p and 40 of an update of at most 1e-3 * 2
        assert (p.double() - q.detach()).abs().max() < 20 * (3 * EPS32 * 5 + 2e-3 * 40 * EPS32)
    else:
        moved, want = (p - start).double().mean(), (q.detach() - start.double()).mean()
        assert abs(moved / want - 1) < 0.02
        m, v = opt.moments(0)
        state = ref.state[q]
        # rounding is unbiased: the means over 200,000 elements agree to their deviation, a step of 1/8 at most a
        # step, 20 steps, over sqrt(200000): 0.1 %
        assert abs(m.double().mean() / state["exp_avg"].mean() - 1) < 0.01
        assert abs(v.double().mean() / state["exp_avg_sq"].mean() - 1) < 0.01


def test_small_changes_add_up():
    """bf16 without master: a thousand updates of a fiftieth of a rounding step move the mean by as much."""
    n = 100000
    p = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    opt = _optim([p], lr=2.0 ** -8 / 50, weight_decay=0.0)
    g = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    for _ in range(1000):
        opt.step(grads=[g])
    moved = 1 - p.double().mean().item()
    # a sum of 1000 draws with deviations below 2^-8 * sqrt(1 / 50), over sqrt(100000) elements: six deviations
    assert abs(moved - 1000 * 2.0 ** -8 / 50) < 6 * 2.0 ** -8 * math.sqrt(1000 / 50) / math.sqrt(n) + 1e-4


@pytest.mark.parametrize("bits", [32, 8])
def test_missing_gradients_and_empty_tensors(bits):
    sizes = [300, 0, 5000, 17]
    p = [torch.randn(n, device="cuda") for n in sizes]
    opt = _optim(p, state_bits=bits)
    g = [torch.randn(n, device="cuda") for n in sizes]
    opt.step(grads=g)
    keep = [t.clone() for t in p], {n: t.clone() for n, t in opt.state.items()}
    opt.step(grads=[g[0], None, None, g[3]])
    assert opt.steps() == 2
    assert torch.equal(p[2], keep[0][2]) and not torch.equal(p[0], keep[0][0]) and not torch.equal(p[3], keep[0][3])
    at = opt.offsets[2]
    for name in ("m", "v"):
        a, b = (t[name][at:at + 5000].float() for t in (opt.state, keep[1]))
        assert torch.equal(a, b)
    opt.step(grads=[None] * 4)  # counts all the same
    assert opt.steps() == 3
    norm, scale = opt.grad_norm(1.0, grads=[None] * 4)
    assert norm.item() == 0 and scale.item() == 1


def test_parameters_gradients_are_the_default():
    p = [torch.randn(50, 3, device="cuda", requires_grad=True), torch.randn(7, device="cuda", requires_grad=True)]
    opt = _optim(p)
    (p[0].square().sum() + 0 * p[1].sum()).backward()
    version, old = p[0]._version, p[0].detach().clone()
    norm, _ = opt.grad_norm()
    opt.step()
    assert p[0]._version > version
    assert not torch.equal(old, p[0].detach()) and abs(norm.item() - (2 * old).norm().item()) < 1e-3
    opt.zero_grad()
    assert p[0].grad is None
    y = p[0].square().sum()
    p[0].grad = torch.ones_like(p[0])
    opt.step(grads=[p[0].grad, None])
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_no_number_leaves_the_step_out(bits, value):
    p = [torch.randn(5000, device="cuda", dtype=torch.float32).to(torch.bfloat16)]
    opt = _optim(p, state_bits=bits, master=True)
    opt.step(grads=[torch.randn_like(p[0])])
    keep = [t.clone() for t in (p[0], *opt.state.values())]
    opt.step(grads=[torch.full_like(p[0], value)], scale=torch.full((1,), value, device="cuda"))
    for a, b in zip(keep, (p[0], *opt.state.values())):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    norm, scale = opt.grad_norm(grads=[torch.full_like(p[0], value)])
    assert not math.isfinite(norm.item()) and math.isnan(scale.item())
    opt.step(grads=[torch.randn_like(p[0])], scale=scale)
    assert opt.steps() == 1
    opt.step(grads=[torch.randn_like(p[0])], scale=torch.zeros((), device="cuda"))  # 0 is a number
    assert opt.steps() == 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_that_are_not_numbers_spoil_their_elements_alone(dtype):
    p = [torch.randn(1000, device="cuda").to(TORCH[dtype]), torch.randn(1000, device="cuda").to(TORCH[dtype])]
    for bits in (32, 8):
        opt = _optim(p, state_bits=bits)
        g = [torch.randn_like(t) for t in p]
        g[0][300] = float("nan")
        g[0][901] = float("inf")
        opt.step(grads=g)
        assert torch.isfinite(p[1]).all()
        bad = ~torch.isfinite(p[0].float())
        assert bad[300] and bad[901] and bad.sum() == 2
        m, v = opt.moments(0)
        m1, v1 = opt.moments(1)
        assert torch.isfinite(m1).all() and torch.isfinite(v1).all() and not torch.isfinite(v[300])
        if bits == 8:  # their blocks, 256 to 383 and 896 to 999
            assert torch.isfinite(m[:256]).all() and torch.isfinite(m[384:896]).all()
        else:
            assert torch.isfinite(m).sum() == 998
        p = [torch.randn(1000, device="cuda").to(TORCH[dtype]), torch.randn(1000, device="cuda").to(TORCH[dtype])]


@pytest.mark.parametrize("bits", [32, 8])
def test_ends_of_the_range(bits):
    """Gradients of 1e-30 to 1e15, all of a block 0, and betas and decays at their ends."""
    n = 128 * 9
    g = (torch.randn(9, 128, device="cuda") * torch.tensor([1e-30, 1e-20, 1e-15, 1e-8, 1.0, 1e5, 1e10, 1e15, 0.0],
                                                          device="cuda")[:, None]).reshape(-1)
    for kw in (dict(), dict(betas=(0.0, 0.0)), dict(eps=1.0), dict(eps=1e-16), dict(weight_decay=1.0), dict(lr=0.0)):
        p = torch.ones(n, device="cuda")
        opt = _optim([p], state_bits=bits, **{"lr": 1e-2, "weight_decay": 0.0, **kw})
        for _ in range(3):
            opt.step(grads=[g])
            assert torch.isfinite(p).all()
        # Adam's first steps on equal gradients: at most lr each, and the decay
        assert ((p - 1).abs() <= 3 * 1.1e-2 + (0.04 if kw.get("weight_decay") else 0)).all(), kw
        if kw.get("lr") == 0.0:
            assert (p == 1).all()


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [[1], [5, 128, 4097, 0, 3], [4096 * 2000 + 1], [33] * 1500])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm(grad, sizes, shift):
    g = np.random.default_rng(8)
    p = [torch.zeros(n, device="cuda") for n in sizes]
    opt = _optim(p, state_bits=8)
    grads = Tensors(sizes, TORCH[grad], shift, _draw(g, sizes, 0.3))
    want = math.sqrt(sum(float((wide(t) ** 2).sum()) for t in grads.parts))
    for most in (1e-3, want * 0.999, want * 1.001 + 1e-3, 1e9):
        norm, scale = opt.grad_norm(most, grads=grads.parts)
        # a rounding of every square, of which the sums' are twice as exact, and the result's
        assert abs(norm.item() - want) <= 2 * EPS32 * want
        assert abs(scale.item() - min(1.0, most / (want + 1e-6))) <= 3 * EPS32 * scale.item()
    again = opt.grad_norm(most, grads=grads.parts)
    assert torch.equal(again[0], norm) and torch.equal(again[1], scale)
    grads.check_around()


def test_refusals():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    p = [torch.randn(10, 4, device="cuda"), torch.randn(9, device="cuda").to(torch.bfloat16)]
    opt = _optim(p)
    g = [torch.randn(10, 4, device="cuda"), torch.randn(9, device="cuda")]
    opt.step(grads=g)
    launches = opt.last_launch_count()
    assert launches == 2  # one for each kind of tensors
    for bad in ([g[0]], [g[0], g[1][:8]], [g[0].t().contiguous().t(), g[1]], [g[0].double(), g[1]], [g[0].cpu(), g[1]],
                [g[0].to(torch.float16), g[1]]):
        with pytest.raises(ValueError, match="grads"):
            opt.step(grads=bad)
        with pytest.raises(ValueError, match="grads"):
            opt.grad_norm(grads=bad)
    for bad in (torch.ones(2, device="cuda"), torch.ones((), device="cuda", dtype=torch.float64), torch.ones(())):
        with pytest.raises(ValueError, match="scale"):
            opt.step(grads=g, scale=bad)
        with pytest.raises(ValueError, match="lr_factor"):
            opt.step(grads=g, lr_factor=bad)
    for call in (lambda: opt.step(grads=[p[0], g[1]]), lambda: opt.step(grads=g, lr=-1.0), lambda: opt.step(grads=g, lr=float("nan")),
                 lambda: opt.grad_norm(0.0, grads=g), lambda: opt.grad_norm(float("nan"), grads=g)):
        with pytest.raises(DominoError):
            call()
    both = torch.empty((), device="cuda")
    with pytest.raises(DominoError):
        opt.grad_norm(1.0, grads=g, out=(both, both))
    assert opt.steps() == 1 and opt.last_launch_count() == launches
    with pytest.raises(DominoError):
        _optim([p[0], p[0]])
    with pytest.raises(DominoError):
        _optim([p[0], p[0].view(-1)[4:8]])
    with pytest.raises(ValueError, match="params"):
        _optim([p[0].t()])
    with pytest.raises(ValueError, match="state"):
        _optim(p, state={"m": opt.state["m"]})
    with pytest.raises(ValueError, match="state"):
        _optim(p, state=dict(opt.state, m=opt.state["m"][:-1]))
    with pytest.raises(DominoError):
        _optim(p, state=dict(opt.state, v=opt.state["m"]))


def test_a_parameter_that_moved_is_refused():
    p = [torch.nn.Parameter(torch.randn(100, device="cuda")), torch.randn(50, device="cuda")]
    opt = _optim(p)
    g = [torch.randn_like(t) for t in p]
    opt.step(grads=g)
    p[0].data = p[0].data.clone()
    for call in (opt.step, opt.grad_norm):
        with pytest.raises(ValueError, match="params.0.*no longer"):
            call(grads=g)
    assert opt.steps() == 1
    again = _optim(p, state=opt.state_dict())
    again.step(grads=g)
    assert again.steps() == 2


@pytest.mark.parametrize("bits", [32, 8])
def test_resume_from_a_state(bits):
    """A copy of the state and the parameters goes on as the original does, bit for bit."""
    torch.manual_seed(1)
    p = [torch.randn(3000, device="cuda").to(torch.bfloat16), torch.randn(77, device="cuda")]
    opt = _optim(p, state_bits=bits, seed=11)
    grads = [[torch.randn_like(t) for t in p] for _ in range(4)]
    for g in grads[:2]:
        opt.step(grads=g)
    q = [t.clone() for t in p]
    other = _optim(q, state_bits=bits, seed=11, state={n: t.clone() for n, t in opt.state_dict().items()})
    for g in grads[2:]:
        opt.step(grads=g)
        other.step(grads=g)
    assert other.steps() == 4
    for a, b in zip((*p, *opt.state.values()), (*q, *other.state.values())):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps(bits):
    """A captured clipped step, replayed, does what eager steps do: the count, the rate's factor and the norm are the
    device's."""
    torch.manual_seed(2)
    sizes = [5000, 300, 4097]
    start = [torch.randn(n, device="cuda").to(torch.bfloat16) for n in sizes]
    grads = [torch.randn(n, device="cuda").to(torch.bfloat16) for n in sizes]
    factor = torch.ones((), device="cuda")
    eager, captured = [t.clone() for t in start], [t.clone() for t in start]
    a, b = _optim(eager, state_bits=bits), _optim(captured, state_bits=bits)

    def step(opt):
        _, scale = opt.grad_norm(0.5, grads=grads)
        opt.step(grads=grads, scale=scale, lr_factor=factor)

    step(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    step(a)
    for k in range(4):
        factor.fill_(0.5 ** k)
        for t in grads:
            t.mul_(1.5)
        step(a)
        graph.replay()
    step(a)
    step(b)
    torch.cuda.synchronize()
    assert a.steps() == b.steps() == 6
    for x, y in zip((*eager, *a.state.values()), (*captured, *b.state.values())):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_calls_on_two_streams():
    """Calls of one context run one after another, whatever their streams."""
    torch.manual_seed(3)
    p = [torch.randn(3_000_000, device="cuda").to(torch.bfloat16)]
    q = [p[0].clone()]
    a, b = _optim(p, state_bits=8), _optim(q, state_bits=8)
    g = [[torch.randn_like(p[0])] for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    norms = []
    for turn in range(10):
        b.step(grads=g[turn % 2])
        out = torch.empty((), device="cuda"), torch.empty((), device="cuda")
        torch.cuda.synchronize()
        a.step(grads=g[turn % 2], stream=streams[turn % 2])
        a.grad_norm(1.0, grads=g[turn % 2], out=out, stream=streams[1 - turn % 2])
        norms.append(out[0])
    torch.cuda.synchronize()
    assert torch.equal(p[0], q[0]) and len({n.item() for n in norms}) == 2


def test_mixed_types_in_one_context():
    """fp32 and bf16 parameters, with and without the gradients' own type."""
    torch.manual_seed(4)
    p = [torch.randn(500, device="cuda"), torch.randn(700, device="cuda").to(torch.bfloat16)]
    q = [t.clone() for t in p]
    g = [torch.randn(500, device="cuda").to(torch.bfloat16), torch.randn(700, device="cuda")]
    opt = _optim(p, master=True)
    opt.step(grads=g)
    alone = [_optim([q[0]]), _optim([q[1]], master=True)]
    for o, t in zip(alone, g):
        o.step(grads=[t])
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
    norm, _ = opt.grad_norm(grads=g)
    want = math.sqrt(sum(float((wide(t) ** 2).sum()) for t in g))
    assert abs(norm.item() - want) <= 2 * EPS32 * want


def test_positions_beyond_32_bits():
    """8-bit moments of more than 2^32 positions: the last tensor's random words, codes and scales."""
    n = 2 ** 32
    g = torch.randn(1000, device="cuda").to(torch.bfloat16)
    big = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    p = torch.randn(1000, device="cuda").to(torch.bfloat16)
    opt = _optim([big, p], state_bits=8, seed=3)
    assert opt.offsets[1] == n
    opt.step(grads=[None, g])
    m32, v32 = O.moments32(np.zeros(1000), np.zeros(1000), wide(g), 1.0, 0.9, 0.999)
    pad = np.zeros(24, np.float32)
    h = O.words(np.uint64(n) + np.arange(1024, dtype=np.uint64), 1, 3)
    code, s = O.narrow(np.concatenate([m32, pad]), h & np.uint64(0xFFFFF), 0)
    assert np.array_equal(opt.state["m"].view(torch.uint8)[n:n + 1000].cpu().numpy(), code[:1000])
    assert np.array_equal(opt.state["m_scale"][-8:].cpu().numpy(), s)
    big_grad = torch.zeros_like(big)
    big_grad[-1] = 1.0
    opt.step(grads=[big_grad, None])
    assert (big[:-1] == 0).all() and big[-1] < 0 and (opt.state["m"].view(torch.uint8)[n - 128:n - 1] == 0).all()
