"""A tensor's step with an MX4 projector does not depend on the rest of the call's list, bit for
bit, whatever kernel forms the list chooses: the parts of a contraction in blocks of their own or
several in one, gradients staged as they lie or through registers, tiles of 64 or 128 rows, blocks of one
or several back-projection tiles."""
import pytest
import torch

from memory_efficient_optimizers_amd import _lib
from tests.test_gpu_mx4 import galore_case, run_step
from tests.test_gpu_mx4_forms import forms

pytestmark = pytest.mark.gpu
DEV = "cuda"

# shapes, rank, proj_type, grad, and what differs for the first tensor: (form field, in the list, alone)
CASES = [
    ([(1700, 1680), (32400, 8)], 16, "std", "bf16", [("item_parts", 4, 1), ("aligned", 0, 0)]),
    ([(1680, 1700), (8, 32400)], 16, "std", "bf16", [("item_parts", 4, 1), ("aligned", 0, 0)]),
    ([(1792, 1664), (32384, 128)], 40, "std", "bf16", [("item_parts", 4, 1), ("aligned", 1, 1)]),
    ([(1664, 1792), (128, 32384)], 40, "std", "bf16", [("item_parts", 4, 1), ("aligned", 1, 1)]),
    ([(1700, 1792), (32384, 72)], 200, "std", "bf16", [("item_parts", 4, 1), ("aligned", 0, 0)]),
    ([(1792, 1664), (300, 72)], 64, "std", "bf16", [("item_parts", 1, 1), ("aligned", 0, 1)]),
    ([(1792, 1664), (32400, 8)], 64, "std", "bf16", [("item_parts", 4, 1), ("aligned", 0, 1)]),
    ([(4096, 2048), (2048, 4096), (4096, 2048)], 256, "std", "bf16", [("item_parts", 4, 1), ("aligned", 1, 1)]),
    ([(70, 1801), (1801, 70), (2048, 64)], 33, "reverse_std", "bf16", [("item_parts", 1, 1)]),
    ([(512, 8192), (8192, 512), (512, 8192)], 64, "reverse_std", "bf16", [("item_parts", 2, 1), ("aligned", 1, 1)]),
    ([(500, 8187), (8187, 500), (512, 8192)], 40, "reverse_std", "bf16", [("item_parts", 2, 1), ("aligned", 0, 0)]),
    ([(3000, 2500), (1800, 2900), (2000, 2000)], 20, "std", "bf16", [("item_parts", 3, 1), ("aligned", 0, 0)]),
    ([(8200, 256), (256, 8300)], 200, "std", "mx4", [("rows", 128, 64)]),
    ([(2048, 1024), (2048, 6144)], 64, "std", "mx4", [("back_tiles", 4, 1)]),
    ([(2000, 1000), (2048, 6144)], 64, "std", "bf16", [("back_tiles", 4, 1)]),
    ([(256, 512), (512, 1024), (1024, 256), (640, 640)], 128, "std", "bf16", []),
    ([(256, 512), (512, 1024), (1024, 256), (640, 640)], 128, "std", "mx4", []),
]


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shapes,rank,proj_type,grad,differ", CASES)
def test_list_equals_singles_bitwise(shapes, rank, proj_type, grad, differ, pdt):
    inlist, alone = forms(shapes, rank, proj_type, grad, pdt), forms(shapes[:1], rank, proj_type, grad, pdt)
    for key, a, b in differ:
        assert (getattr(inlist[0], key), getattr(alone[0], key)) == (a, b), key
    h = _lib.galore_hparams(lr=0.05, rank=rank, proj_type=proj_type)
    p1, g1, s1, _ = galore_case(shapes, rank, 9, pdt, proj_type, grad)
    p2, g2, s2, _ = galore_case(shapes, rank, 9, pdt, proj_type, grad)
    x0 = [p.clone() for p in p1]
    ws = _lib.workspace(_lib.meo_galore_mx4_workspace_size(h, p1, g1), DEV)
    _lib.meo_galore_mx4_step(h, 3, p1, g1, s1, ws)
    for k in range(len(shapes)):
        wk = _lib.workspace(_lib.meo_galore_mx4_workspace_size(h, [p2[k]], [g2[k]]), DEV)
        _lib.meo_galore_mx4_step(h, 3, [p2[k]], [g2[k]], [s2[k]], wk)
    torch.cuda.synchronize()
    for k in range(len(shapes)):
        assert not torch.equal(p1[k], x0[k])
        assert torch.equal(p1[k], p2[k]), shapes[k]
        for key in ("exp_avg", "exp_avg_sq"):
            assert torch.equal(s1[k][key], s2[k][key]), (shapes[k], key)


@pytest.mark.parametrize("case", [0, 1, 2, 3, 6, 9, 10, 11])
def test_several_parts_in_a_block(case):
    """Against the oracle: all parts of the first tensor, or some, in one block."""
    shapes, rank, proj_type, grad, _ = CASES[case]
    f = forms(shapes, rank, proj_type, grad)[0]
    assert 1 < f.item_parts <= f.parts
    run_step(shapes, rank, grad=grad, hp=dict(proj_type=proj_type))
