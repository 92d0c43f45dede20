"""What train.AdamW does around its launches, with stand-ins for the list and the launch: no GPU."""
import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, train

BF = torch.bfloat16


class List:
    """Stands for api.AdamWList."""
    built = 0

    def __init__(self, params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, master):
        List.built += 1
        self.params, self.master, self.grads = list(params), list(master), list(grads)

    def set_grads(self, grads):
        self.grads = list(grads)


@pytest.fixture
def launches(monkeypatch):
    """The launches' (number of tensors, step, device's step): each takes lr from the values, behind autograd's back."""
    seen = []

    def launch(tensors, rule, step, norm=None, lr_step=None, stream=None):
        if rule.eps < 0:
            raise api.MoEError("moe_nvfp4_adamw", api.MOE_ERR_INVALID_ARG)
        seen.append((len(tensors.params), step, None if lr_step is None else float(lr_step[1])))
        for p, w in zip(tensors.params, tensors.master):
            at = p.data.float().reshape(-1) if w is None else w
            at -= rule.lr
            p.data.copy_(at.view(p.shape))
    List.built = 0
    monkeypatch.setattr(api, "AdamWList", List)
    monkeypatch.setattr(api, "moe_nvfp4_adamw", launch)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return seen


def parameters(n=3, dtype=torch.float32):
    return [torch.nn.Parameter(torch.full((4,), 2.0 + i, dtype=dtype)) for i in range(n)]


def give(params, *which):
    for i, p in enumerate(params):
        p.grad = torch.ones_like(p) if i in which else None


def test_a_graph_from_before_the_step_is_refused(launches):
    """Its saved parameters are other ones now: autograd raises, as for torch's optimizers."""
    params = parameters()
    opt = train.AdamW(params, lr=0.5)
    give(params, 0, 1)
    loss, other = (params[0] * params[1]).sum(), (params[2] * params[2]).sum()
    opt.step()
    assert bool((params[0] == 1.5).all())
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    other.backward()        # (of a parameter without a step)
    assert bool((params[2].grad == 8.0).all())


def tiny_steps(dtype=BF):
    """An optimizer whose masters hold what BF16 parameters cannot: three steps of 2^-12 from 2."""
    params = parameters(2, dtype)
    opt = train.AdamW(params, lr=2.0 ** -12)
    give(params, 0, 1)
    for _ in range(3):
        opt.step()
    assert bool((params[0] == 2.0).all()) and bool((opt.state[0]["master"] == 2.0 - 3 * 2.0 ** -12).all())
    return params, opt


@pytest.mark.parametrize("how", ["copy", "load", "data", "address", "address of the same"])
def test_parameters_that_change_between_steps(launches, how):
    """A checkpoint loaded after the optimizer was made, weights swapped in: the step is from them."""
    params, opt = tiny_steps()
    new = torch.tensor([7.0, 2.0, 8.0, 2.0], dtype=BF)
    if how == "copy":
        with torch.no_grad():
            params[0].copy_(new)
    elif how == "load":
        torch.nn.ParameterList(params).load_state_dict({"0": new, "1": params[1].detach().clone()})
    elif how == "data":             # nothing tells of this one
        params[0].data.copy_(new)
        opt.read_parameters()
    elif how == "address":
        params[0].data = new.clone()
    else:
        new = params[0].detach().clone()
        params[0].data = new.clone()
    opt.step()
    d = 2.0 ** -12
    want = torch.where(new == 2.0, 2.0 - 4 * d, new.float() - d)     # where nothing changed, the master's digits stay
    assert torch.equal(opt.state[0]["master"], want) and torch.equal(params[0], want.to(BF))
    assert bool((opt.state[1]["master"] == 3.0 - 4 * d).all())


def test_weights_swapped_in_and_out_keep_the_masters(launches):
    params, opt = tiny_steps()
    with torch.no_grad():
        mine = params[0].clone()
        params[0].fill_(5.0)
        params[0].copy_(mine)
    opt.step()
    assert bool((opt.state[0]["master"] == 2.0 - 4 * 2.0 ** -12).all())


@pytest.mark.parametrize("model_first", [False, True])
def test_a_checkpoint_of_both_keeps_the_masters(launches, model_first):
    params, opt = tiny_steps()
    mine = parameters(2, BF)
    again = train.AdamW(mine, lr=2.0 ** -12)
    for part in (model_first, not model_first):
        if part:
            with torch.no_grad():
                for p, q in zip(mine, params):
                    p.copy_(q)
        else:
            again.load_state_dict(opt.state_dict())
    give(mine, 0, 1)
    again.step()
    assert bool((again.state[0]["master"] == 2.0 - 4 * 2.0 ** -12).all())


def test_float_parameters_have_no_masters(launches):
    params = parameters(1)
    opt = train.AdamW(params, lr=0.5)
    with torch.no_grad():
        params[0].fill_(9.0)
    give(params, 0)
    opt.step()
    opt.read_parameters()
    assert bool((params[0] == 8.5).all())


def test_sets_of_parameters_that_change_from_step_to_step(launches):
    """Experts without tokens have no gradient: the lists kept are bounded, and sets that alternate are built once."""
    params = parameters(9)
    opt = train.AdamW(params, lr=2.0 ** -10)
    for k in range(1, 200):
        give(params, *[i for i in range(9) if k >> i & 1])
        opt.step()
    assert len(opt._lists) <= 16
    for i, (p, s) in enumerate(zip(params, opt.steps)):
        assert s == sum(k >> i & 1 for k in range(1, 200)) and bool((p == 2.0 + i - s * 2.0 ** -10).all())
    params = parameters(4)
    opt = train.AdamW(params)
    List.built = 0
    for k in range(20):
        give(params, *((0, 1) if k % 2 else (2, 3)))
        opt.step()
    assert List.built == 2
    # more numbers of steps at once than lists are kept for: a launch each, in every step
    params = parameters(40)
    opt = train.AdamW(params)
    for k in range(40):
        give(params, *range(k + 1))
        opt.step()
    launches.clear()
    List.built = 0
    for _ in range(3):
        opt.step()
    assert len(launches) == 120 and List.built <= 40 and len(opt._lists) <= 40


def test_capturable_parameters_are_the_same_in_every_step(launches):
    """They share the number of the step: another set would take the wrong one."""
    params = parameters(2)
    opt = train.AdamW(params, capturable=True)
    opt.step()                  # without any gradient
    give(params, 0)
    opt.step()
    for which in ((1,), (0, 1)):
        give(params, *which)
        with pytest.raises(ValueError, match="never"):
            opt.step()
    give(params, 0)
    opt.step()
    assert launches == [(1, 1, 1.0), (1, 2, 2.0)] and opt.state_dict()["steps"] == [2, 0]
    # and of a saved state's
    again = train.AdamW(parameters(2), capturable=True)
    again.load_state_dict(opt.state_dict())
    give(again.params, 1)
    with pytest.raises(ValueError, match="never"):
        again.step()
    give(again.params, 0)
    again.step()
    assert launches[-1] == (1, 3, 3.0)


def test_a_refused_step_does_not_count(launches):
    params = parameters(1)
    opt = train.AdamW(params, lr=0.5, capturable=True)
    give(params, 0)
    opt.step()
    opt.eps = -1.0
    with pytest.raises(api.MoEError):
        opt.step()
    assert opt.steps == [1] and opt.state_dict()["steps"] == [1]
    opt.eps = 1e-8
    opt.step()
    assert launches == [(1, 1, 1.0), (1, 2, 2.0)] and bool((params[0] == 1.0).all())


def test_a_learning_rate_that_a_capture_would_not_see(launches, monkeypatch):
    """It is on the device since the last step outside a capture."""
    params = parameters(1)
    opt = train.AdamW(params, lr=0.5, capturable=True)
    give(params, 0)
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    opt.step()
    opt.lr = 0.25
    with pytest.raises(ValueError, match="learning rate"):
        opt.step()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    opt.step()
    assert opt.lr_step.tolist() == [0.25, 4.0] and len(launches) == 4


def test_parameters_of_inference_mode(launches):
    """Autograd does not count their changes: they have masters all the same."""
    with torch.inference_mode():
        params = parameters(2, BF)
        opt = train.AdamW(params, lr=0.5)
        give(params, 0, 1)
        opt.step()
        assert bool((params[0] == 1.5).all())
        params[0].fill_(7.0)
        opt.read_parameters()
        opt.step()
        assert bool((params[0] == 6.5).all()) and bool((params[1] == 2.0).all())
