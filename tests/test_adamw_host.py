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
        if rule.lr < 0:
            raise api.MoEError("moe_nvfp4_adamw", api.MOE_ERR_INVALID_ARG)
        seen.append((len(tensors.params), step, None if lr_step is None else float(lr_step[1])))
        for p, w in zip(tensors.params, tensors.master):
            at = p.data.float().reshape(-1) if w is None else w
            at -= rule.lr
            p.data.copy_(at.view(p.shape))
    List.built = 0
    monkeypatch.setattr(api, "AdamWList", List)
    monkeypatch.setattr(api, "moe_nvfp4_adamw", launch)
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
