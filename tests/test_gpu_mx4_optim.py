"""GaLoreAdamW with MX4 projectors and compressed gradients on the GPU, where its calls can go
wrong: refused steps, gradients on streams of their own."""
import pytest
import torch

from memory_efficient_optimizers_amd import GaLoreAdamW, MeoError, _lib, mx4_quantize
from tests.test_gpu_mx4 import MX4, _backward, _model

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_a_step_that_turned_due_is_refused_and_can_be_taken_later():
    """The gap is lowered after gradients were compressed: the step would refresh from MX4 gradients.
    Nothing moves or counts; with the gap as it was, the step is that of an undisturbed run."""
    runs = []
    for disturbed in (False, True):
        m, groups = _model(11)
        opt = GaLoreAdamW(groups, lr=0.02, projector_dtype=MX4)
        for p in (m[0].weight, m[2].weight):
            p.register_post_accumulate_grad_hook(opt.compress_grad)
        for t in (1, 2):
            opt.zero_grad()
            _backward(m, t)
            if disturbed and t == 2:
                before = [p.detach().clone() for p in m.parameters()]
                opt.param_groups[0]["update_proj_gap"] = 1
                with pytest.raises(MeoError) as e:
                    opt.step()
                assert e.value.code == _lib.MEO_EDTYPE
                assert all(torch.equal(a, p.detach()) for a, p in zip(before, m.parameters()))
                assert all(opt.state[p]["step"] == 1 for p in m.parameters())
                opt.param_groups[0]["update_proj_gap"] = 3
            opt.step()
        assert all(opt.state[p]["step"] == 2 for p in m.parameters())
        runs.append([p.detach().clone() for p in m.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_compress_grad_on_another_stream_than_the_gradients():
    """The gradient's memory is not given out again while the other stream has yet to read it."""
    p = torch.nn.Parameter(torch.zeros(1024, 512, device=DEV))
    opt = GaLoreAdamW([dict(params=[p], rank=16)], lr=0.02, projector_dtype=MX4)
    p.grad = torch.randn(1024, 512, device=DEV)
    opt.step()
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 27, device=DEV)
    g = torch.randn(1024, 512, device=DEV)
    want = mx4_quantize(g)
    torch.cuda.synchronize()
    p.grad = g
    del g
    with torch.cuda.stream(side):
        for _ in range(40):  # some ms of work before the compression
            busy.add_(1)
        opt.compress_grad(p)
    junk = [torch.full((1024, 512), float(i), device=DEV) for i in range(8)]
    torch.cuda.synchronize()
    got = opt._compressed[p]
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales) and len(junk) == 8
