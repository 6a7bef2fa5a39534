"""The kernel forms of the MX4 operators that only larger sizes choose, each asserted from the
library's own choice: the 128-row tiles of a product and of an MX4 gradient's projection,
back-projection blocks of three tiles and more, long contractions in one piece; sizes past
2^31 values; projectors and gradients that hold NaN blocks. Bars as in tests/test_gpu_mx4.py."""
import numpy as np
import pytest
import torch

from memory_efficient_optimizers_amd import MX4Tensor, _lib, mx4_dequantize, mx4_matmul, mx4_quantize
from oracle import galore as ga
from oracle import mx4 as ox
from tests.harness import to64
from tests.test_gpu_mx4 import check_product, check_quantized, galore_case, rand_mx4, run_step, spread

pytestmark = pytest.mark.gpu
DEV = "cuda"


def forms(shapes, rank, proj_type="std", grad="bf16", pdt=torch.float32):
    """The forms of a step over tensors of these shapes (their addresses aligned)."""
    h = _lib.galore_hparams(rank=rank, proj_type=proj_type)
    params, grads, states = [], [], []
    for s in shapes:
        p = torch.empty(s, dtype=pdt, device=DEV)
        right = ga.galore_side(tuple(s), proj_type) == "right"
        D, d = s if right else s[::-1]
        params.append(p)
        grads.append(MX4Tensor.empty(D, d, DEV) if grad == "mx4" else torch.empty(s, dtype=torch.bfloat16, device=DEV))
        states.append(_lib.galore_mx4_init_state(p, rank, proj_type))
    return _lib.meo_galore_mx4_forms(h, params, grads, states)


# ------------------------------------------------------------------------------ product

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(16500, 200, 777), (16449, 256, 32), (16500, 300, 520), (16400, 129, 2112)])
def test_matmul_in_128_row_tiles(m, n, k, dtype):
    assert _lib.meo_mx4_matmul_rows(m, n) == 128
    a, b = rand_mx4(m, k, 10), rand_mx4(n, k, 11)
    check_product(a, b, mx4_matmul(a, b, dtype))


def test_matmul_of_more_than_one_tile_of_columns():
    assert _lib.meo_mx4_matmul_rows(130, 600) == 64
    for dtype in (torch.float32, torch.bfloat16):
        a, b = rand_mx4(130, 1300, 12), rand_mx4(600, 1300, 13)
        check_product(a, b, mx4_matmul(a, b, dtype))


def test_matmul_rows_do_not_change_the_result():
    """The same rows in tiles of 128 and of 64."""
    a, b = rand_mx4(16500, 1000, 14), rand_mx4(200, 1000, 15)
    assert _lib.meo_mx4_matmul_rows(16500, 200) == 128 and _lib.meo_mx4_matmul_rows(1000, 200) == 64
    part = MX4Tensor(a.codes[15500:], a.scales[15500:], 1000)
    assert torch.equal(mx4_matmul(a, b)[15500:], mx4_matmul(part, b))


# ------------------------------------------------------------------------------ step

@pytest.mark.parametrize("shape,rank", [((16500, 256), 256), ((520, 16450), 200), ((16450, 777), 130), ((2080, 16400), 160)])
def test_projection_of_an_mx4_gradient_in_128_row_tiles(shape, rank):
    assert forms([shape], rank, grad="mx4")[0].rows == 128
    run_step([shape], rank, grad="mx4")


@pytest.mark.parametrize("shape,aligned", [((8320, 2048), 1), ((2048, 8320), 1), ((8321, 2050), 0), ((2050, 8321), 0),
                                           ((2100, 8320), 0)])
def test_projection_of_a_long_contraction_in_one_piece(shape, aligned):
    """16 steps of 128 and more."""
    f = forms([shape], 64)[0]
    assert (f.aligned, f.parts, f.rows) == (aligned, 1, 64)
    run_step([shape], 64)


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,rank,tiles", [((6080, 2048), 64, 3), ((2048, 6080), 40, 3), ((6430, 2040), 48, 4),
                                              ((2041, 6431), 256, 4), ((9000, 2048), 33, 5), ((2040, 9001), 16, 5)])
def test_back_projection_of_several_tiles_a_block(shape, rank, tiles, pdt):
    """Odd and even counts; whole matrices, and ones whose last band, chunk and row pieces are not."""
    assert forms([shape], rank, pdt=pdt)[0].back_tiles == tiles
    run_step([shape], rank, param_dtype=pdt, hp=dict(weight_decay=0.1))


# ------------------------------------------------------------------------------ past 2^31 values

def test_columns_past_2_31_elements():
    rows, cols = 33000, 65568  # of the values: blocks run down their columns
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    last = spread((3, rows), 7, torch.bfloat16).t()
    x[:, -3:] = last
    q = mx4_quantize(x, transposed=True)
    check_quantized(MX4Tensor(q.codes[-3:].clone(), q.scales[-3:].clone(), rows), to64(last.t().contiguous()))
    assert not q.codes[:-3].any() and not q.scales[:-3].any()
    x.fill_(1)
    mx4_dequantize(q, out=x, transposed=True)
    assert not x[:, :-3].any()
    assert np.array_equal(to64(x[:, -3:].t().contiguous()), ox.rounded(to64(last.t().contiguous())))


@pytest.mark.parametrize("m,n,k", [(33000, 65600, 64), (70000, 8, 65600)])
def test_matmul_past_2_31(m, n, k):
    """Outputs, then codes of one operand: the last rows as a product of their own."""
    a, b = MX4Tensor(torch.zeros(m, 16 * -(-k // 32), dtype=torch.uint8, device=DEV),
                     torch.zeros(m, -(-k // 32), dtype=torch.uint8, device=DEV), k), rand_mx4(n, k, 16)
    tail = rand_mx4(200, k, 17)
    a.codes[-200:], a.scales[-200:] = tail.codes, tail.scales
    c = torch.full((m, n), 3.0, dtype=torch.bfloat16, device=DEV)
    mx4_matmul(a, b, out=c)
    assert not c[:-200].any()
    cols = torch.arange(max(n - 300, 0), n, device=DEV)
    check_product(tail, MX4Tensor(b.codes[cols], b.scales[cols], k), c[-200:, cols].contiguous())


@pytest.mark.parametrize("grad", ["bf16", "mx4"])
@pytest.mark.parametrize("left", [False, True])
def test_step_past_2_31(grad, left):
    """A gradient of zeros but for the last rows of R's side: those move as in a matrix of their own,
    the others stay."""
    D, d, r, k = 65600, 33000, 8, 9
    shape = (d, D) if left else (D, d)
    small = (d, k) if left else (k, d)  # its longer side is projected, as d is here
    hp = dict(lr=0.05, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, scale=0.25)
    p2, g2, s2, oracle = galore_case([small], r, 19, torch.bfloat16, "reverse_std", grad)
    x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    (x[:, -k:] if left else x[-k:]).copy_(p2[0])
    st = dict(s2[0])
    for key in ("exp_avg", "exp_avg_sq"):
        st[key] = torch.zeros(D, r, device=DEV)
        st[key][-k:] = s2[0][key]
    if grad == "mx4":
        g = MX4Tensor(torch.zeros(D, g2[0].codes.shape[1], dtype=torch.uint8, device=DEV),
                      torch.zeros(D, g2[0].scales.shape[1], dtype=torch.uint8, device=DEV), d)
        g.codes[-k:], g.scales[-k:] = g2[0].codes, g2[0].scales
    else:
        g = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        (g[:, -k:] if left else g[-k:]).copy_(g2[0])
    h = _lib.galore_hparams(rank=r, **hp)
    ws = _lib.workspace(_lib.meo_galore_mx4_workspace_size(h, [x], [g]), DEV)
    _lib.meo_galore_mx4_step(h, 5, [x], [g], [st], ws)
    torch.cuda.synchronize()
    x0, g0, s0 = oracle[0]
    want_x, want_s = ga.galore_step_tensor(x0, g0, s0, dict(hp, rank=r, proj_type="reverse_std"), 5)
    got = to64((x[:, -k:] if left else x[-k:]).contiguous())
    assert np.all(np.abs(got - want_x) <= 2.0 ** -8 * np.abs(want_x) + 1e-4 * 0.05 * 0.25)
    for key in ("exp_avg", "exp_avg_sq"):
        w = want_s[key]
        assert np.all(np.abs(to64(st[key][-k:]) - w) <= 1e-4 * np.max(np.abs(w)))
        assert not st[key][:-k].any()
    assert not (x[:, :-k] if left else x[:-k]).any()


# ------------------------------------------------------------------------------ NaN blocks

NAN_SHAPES = [((192, 128), 32), ((128, 200), 40), ((300, 136), 64), ((70, 1801), 33), ((1700, 1664), 16)]


@pytest.mark.parametrize("grad", ["bf16", "mx4"])
@pytest.mark.parametrize("shape,rank", NAN_SHAPES)
def test_nan_block_of_the_projector(shape, rank, grad):
    """A NaN block in row c of U^T reaches column c of R and of the moments, no other, and
    through N every value of the parameter that a NaN column of N multiplies: all."""
    proj_type = "reverse_std" if shape == (70, 1801) else "std"
    h = _lib.galore_hparams(lr=0.05, rank=rank, proj_type=proj_type)
    p, g, s, _ = galore_case([shape], rank, 21, proj_type=proj_type, grad=grad)
    p2, g2, s2, _ = galore_case([shape], rank, 21, proj_type=proj_type, grad=grad)
    c = rank // 2
    s2[0]["projector"][c, -16:] = 0
    s2[0]["projector_scale"][c, -1] = 255
    ws = _lib.workspace(_lib.meo_galore_mx4_workspace_size(h, p, g), DEV)
    _lib.meo_galore_mx4_step(h, 5, p, g, s, ws)
    _lib.meo_galore_mx4_step(h, 5, p2, g2, s2, ws)
    keep = torch.arange(rank, device=DEV) != c
    for key in ("exp_avg", "exp_avg_sq"):
        assert bool(torch.isnan(s2[0][key][:, c]).all())
        assert torch.equal(s2[0][key][:, keep], s[0][key][:, keep])
    assert bool(torch.isnan(p2[0]).all())


@pytest.mark.parametrize("grad", ["bf16", "mx4"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape,rank", NAN_SHAPES)
def test_nonfinite_gradient_values_stay_in_their_rows_of_r(shape, rank, bad, grad):
    """Row i of R, so row i of the moments and row (left side: column) i of the parameter; every
    other one steps as without it."""
    proj_type = "reverse_std" if shape == (70, 1801) else "std"
    right = ga.galore_side(shape, proj_type) == "right"
    h = _lib.galore_hparams(lr=0.05, rank=rank, proj_type=proj_type)
    p, g, s, _ = galore_case([shape], rank, 23, proj_type=proj_type)
    p2, g2, s2, _ = galore_case([shape], rank, 23, proj_type=proj_type)
    D, d = shape if right else shape[::-1]
    i, j = D - 3, d - 5
    (g2[0] if right else g2[0].t())[i, j] = bad
    if grad == "mx4":
        g, g2 = ([mx4_quantize(x[0], transposed=not right)] for x in (g, g2))
        assert int((g2[0].scales == 255).sum()) == 1
    ws = _lib.workspace(_lib.meo_galore_mx4_workspace_size(h, p, g), DEV)
    _lib.meo_galore_mx4_step(h, 5, p, g, s, ws)
    _lib.meo_galore_mx4_step(h, 5, p2, g2, s2, ws)
    keep = torch.arange(D, device=DEV) != i
    for key in ("exp_avg", "exp_avg_sq"):
        assert not bool(torch.isfinite(s2[0][key][i]).any())
        assert torch.equal(s2[0][key][keep], s[0][key][keep])
    a, b = (p[0], p2[0]) if right else (p[0].t(), p2[0].t())
    assert bool(torch.isnan(b[i]).all()) and torch.equal(a[keep], b[keep])
