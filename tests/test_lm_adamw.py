"""AdamW over parameters that were replaced after the optimiser was made."""

import pytest
import torch

import tensor_train_compressed_gather_amd as tt
from tensor_train_compressed_gather_amd import lm

F32, BF16 = torch.float32, torch.bfloat16
WRONG = [lambda p: p.to(BF16), lambda p: p[:7].clone(), lambda p: p.t().contiguous(), lambda p: p.repeat(1, 2)[:, ::2],
         lambda p: p.double()]


def on_the_host(copies=True):
    """What the constructor leaves, for host tensors: step() has to refuse
    before it reads any address."""
    lm._bind()
    opt = object.__new__(tt.AdamW)
    opt.params = [torch.zeros(8, 5), torch.zeros(3)]
    opt.copies = [p.to(BF16) for p in opt.params] if copies else None
    opt._shapes = [p.shape for p in opt.params]
    opt.device = torch.device("cuda", 0)
    return opt


@pytest.mark.parametrize("wrong", range(len(WRONG)))
@pytest.mark.parametrize("which", ["params", "copies"])
def test_replaced_tensors_are_checked(which, wrong):
    opt = on_the_host()
    ts = getattr(opt, which)
    ts[0] = WRONG[wrong](ts[0])
    if ts[0].dtype == BF16 and which == "copies" and wrong == 0:
        ts[0] = ts[0].float()
    with pytest.raises(tt.TTEmbError) as e:
        opt._whole(ts, which, F32 if which == "params" else BF16)
    assert e.value.status == tt.TT_EMB_ERR_ARG and f"{which}[0]" in str(e.value)


def test_lists_of_another_length_are_refused():
    opt = on_the_host()
    opt.params.append(torch.zeros(1))
    with pytest.raises(tt.TTEmbError) as e:
        opt._whole(opt.params, "params", F32)
    assert "3 params" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("wrong", range(len(WRONG)))
def test_a_step_refuses_replaced_parameters_and_changes_nothing(wrong):
    p, q = torch.ones(8, 5, device="cuda"), torch.ones(3, device="cuda")
    opt = tt.AdamW([p, q])
    grads = [torch.ones_like(p), torch.ones_like(q)]
    opt.step(grads)
    keep = [x.clone() for x in (p, q, opt.exp_avg, opt.exp_avg_sq)]
    good = p.data
    p.data = WRONG[wrong](p.data)
    with pytest.raises(tt.TTEmbError) as e:
        opt.step(grads)
    assert e.value.status == tt.TT_EMB_ERR_ARG and "params[0]" in str(e.value) and opt.steps == 1
    p.data = p.data.cpu()
    with pytest.raises(tt.TTEmbError):
        opt.step(grads)
    p.data = good
    assert all(torch.equal(x, k) for x, k in zip((p, q, opt.exp_avg, opt.exp_avg_sq), keep))
    p.data = good.clone()  # another place of the right kind is updated there
    opt.step(grads)
    assert torch.equal(good, keep[0]) and not torch.equal(p, keep[0]) and opt.steps == 2


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-8, 1e-15, 1e-20, 1e-30, 2e-38])
def test_second_moments_below_the_normal_numbers(eps):
    # v = g^2 / 1000 of gradients below 3e-18 is subnormal; its root is not
    g = torch.tensor([1e-10, 1e-16, 1e-17, 4e-18, 3e-18, 1e-18, 3e-19, 1e-19, 3e-20, -1e-18], device="cuda")
    p = torch.zeros_like(g)
    opt = tt.AdamW([p], lr=1.0, eps=eps, weight_decay=0.0)
    opt.step([g])
    m, v = opt.exp_avg[:10].double(), opt.exp_avg_sq[:10].double()
    assert (v > 0).all()
    ref = -(m / (1 - 0.9)) / ((v / (1 - 0.999)).sqrt() + eps)
    assert ((p.double() - ref).abs() <= 16 * 2.0 ** -24 * ref.abs()).all()
