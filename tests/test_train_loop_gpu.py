"""The training operators as they are used together: embedding, scores, their
gradient, the gradients' norm and the weights' update, step by step beside torch in
64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_a_policy_step_beside_torch(bits):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    from speculative_decoding_draft_lm_gb300.train import DominoTrain, embedding, token_logprobs
    torch.manual_seed(0)
    V, E, N, T, lr = 501, 64, 40, 1.5, 1e-2
    p = [torch.randn(V, E, device="cuda") * 0.5, torch.randn(V, E, device="cuda") * 0.3]
    mine = [t.clone().requires_grad_() for t in p]
    ref = [t.double().requires_grad_() for t in p]
    train = DominoTrain(V, E=E, max_tokens=N, dtype="fp32")
    opt = DominoAdamW(mine, lr=lr, weight_decay=0.01, state_bits=bits)
    other = torch.optim.AdamW(ref, lr=lr, weight_decay=0.01)
    tokens = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    said = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    adv = torch.randn(N, device="cuda") / N
    for step in range(3):
        x = embedding(train, mine[0], tokens) @ mine[1].t()
        logprob, entropy = token_logprobs(train, x, said, T)
        opt.zero_grad()
        (-(adv * logprob).sum() - 0.01 * entropy.mean()).backward()
        norm, clip = opt.grad_norm(max_norm=0.05)
        opt.step(scale=clip)

        y = ref[0][tokens.long()] @ ref[1].t()
        log_q = torch.log_softmax(y / T, 1)
        H = -(log_q.exp() * log_q).sum(1)
        other.zero_grad()
        (-(adv * log_q.gather(1, said.long()[:, None])[:, 0]).sum() - 0.01 * H.mean()).backward()
        if step == 0:
            # fp32 products (tf32 is off), sums and exponentials against 64 bits
            for a, b in zip(mine, ref):
                assert ((a.grad.double() - b.grad).norm() / b.grad.norm()) < 1e-4
        total = torch.nn.utils.clip_grad_norm_(ref, 0.05)
        assert abs(norm.item() / total.item() - 1) < (1e-4 if step == 0 else 0.05)
        other.step()
    assert train.status() == 0 and opt.steps() == 3
    for a, b, start in zip(mine, ref, p):
        moved, want = (a.detach() - start).double(), b.detach() - start.double()
        # 32 bits: the two walk alike but where a gradient is nothing but rounding; 8 bits: the moments' steps of 1/8
        cos = torch.nn.functional.cosine_similarity(moved.flatten(), want.flatten(), dim=0)
        assert cos > (0.999 if bits == 32 else 0.9)


@pytest.mark.parametrize("N,V", [(3, 700), (400, 501), (200, 20011)])
@pytest.mark.parametrize("bits", [32, 8])
def test_calls_after_one_another_see_each_others_results(N, V, bits):
    """The logits are the parameter: scores and gradient, norm, step, over and over, each reading what the call before
    wrote, with and without a wait for the GPU between them."""
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    torch.manual_seed(0)
    start = torch.randn(N, V, device="cuda")
    tokens = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    weight, entropy_weight = torch.randn(N, device="cuda"), torch.rand(N, device="cuda")
    train = DominoTrain(V, dtype="fp32")
    ends = []
    for wait in (True, False):
        x = start.clone()
        opt = DominoAdamW([x], lr=1e-2, state_bits=bits, seed=1)
        grad, pair = torch.empty_like(x), torch.empty_like(x)
        out = [torch.empty(N, device="cuda") for _ in range(2)]
        clip = torch.empty((), device="cuda"), torch.empty((), device="cuda")
        stats = torch.empty(N, 4, device="cuda")
        more = [torch.empty(N, device="cuda"), torch.empty(N, device="cuda"),
                torch.empty(N, 5, device="cuda", dtype=torch.int32), torch.empty(N, 5, device="cuda")]
        for _ in range(40):
            for call in (lambda: train.logprobs_step(x, tokens, weight, entropy_weight, out=(*out, grad)),
                         lambda: opt.grad_norm(0.5, grads=[grad], out=clip), lambda: opt.step(grads=[grad], scale=clip[1]),
                         lambda: train.logprobs_forward(x, tokens, alternatives=5, stats=stats, out=more),
                         lambda: train.logprobs_backward(x, tokens, stats, weight, more[1], out=pair),
                         lambda: opt.step(grads=[pair])):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        ends.append([x, grad, pair, *out, *clip, *more, *opt.state.values()])
    for a, b in zip(*ends):
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
