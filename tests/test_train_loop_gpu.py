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
