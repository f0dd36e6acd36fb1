"""What the training-step operators read is what stands before them on their stream."""
import pytest
import torch

from cross_vendor_gradient_gb300 import Context

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with Context([1]) as c:
        yield c


@pytest.mark.parametrize("states", ["none", "e4m3"])
def test_a_step_takes_the_factor_of_the_norm_just_before_it(ctx, states):
    """Norm and step back to back, the gradients another size each time: the parameters of steps that the host waited
    between."""
    g = torch.Generator("cuda").manual_seed(3)
    base = torch.randn(3_000_000, device="cuda", generator=g)
    runs = []
    for wait in (False, True):
        p, grad, clip = torch.zeros(5000, device="cuda"), torch.empty(5000, device="cuda"), torch.zeros(2, device="cuda")
        opt = ctx.adamw([p], [grad], states=states, lr=0.1)
        sets = [base * 10.0 ** (i % 5 - 2) for i in range(40)]
        for s in sets:
            grad.copy_(s[:5000])
            ctx.grad_norm([s], clip, max_norm=1.0)
            if wait:
                torch.cuda.synchronize()
            opt.step(grad_scale=clip[1:], seed=1)
        torch.cuda.synchronize()
        runs.append((p, opt.exp_avg[0], opt.exp_avg_sq[0]))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("states", ["none", "e4m3"])
def test_states_made_by_the_optimizer_are_zero_before_a_step_on_another_stream(ctx, states):
    """The current stream is busy when the optimizer is made, the first step runs on another one."""
    p, grad = torch.zeros(3000, device="cuda"), torch.ones(3000, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    opt = ctx.adamw([p], [grad], states=states, lr=0.1, weight_decay=0.0, betas=(0.5, 0.5))
    opt.step(stream=side)
    torch.cuda.synchronize()
    if states == "none":
        assert bool((opt.exp_avg[0] == 0.5).all()) and bool((opt.exp_avg_sq[0] == 0.5).all())
    else:
        assert bool((opt.exp_avg[0][:3000] != 0).all()) and bool((opt.exp_avg_sq[0][:3000] != 0).all())
    assert bool(((p + 0.1).abs() < 1e-6).all())  # 0.1 m / (1 - 0.5) / (sqrt(v / (1 - 0.5)) + eps), m = v = 0.5
