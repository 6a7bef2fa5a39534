"""MX4 on the host (no GPU): the oracle against hand-worked blocks, and the refusals of the
entry points and front ends, which all come before any device work."""
import math

import numpy as np
import pytest
import torch

from memory_efficient_optimizers_amd import GaLoreAdamW, MeoError, MX4Tensor, _lib, mx4_dequantize, mx4_matmul, mx4_quantize
from oracle import mx4 as ox

P = 0x7F0000001000  # a pointer value that validation inspects and never follows


# ------------------------------------------------------------------------------ oracle

def test_magnitudes():
    assert list(ox.MAGNITUDES) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


@pytest.mark.parametrize("amax,scale", [(4.0, 1.0), (7.99, 1.0), (8.0, 2.0), (3.99, 0.5), (6.0, 1.0), (1.0, 0.25)])
def test_scale_is_floor_log2_minus_two(amax, scale):
    _, s = ox.quantize(np.array([[amax] + [0.0] * 31]))
    assert 2.0 ** (int(s[0, 0]) - 127) == scale


def test_ties_go_to_the_even_code():
    x = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 5.01, 7.9, -7.9]
    want = [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.0, -1.0, -4.0, 6.0, 6.0, -6.0]
    got = ox.rounded(np.array([x + [0.0] * (32 - len(x))]))[0, :len(x)]
    assert list(got) == want
    assert math.copysign(1, got[8]) == -1  # -0.25 keeps its sign


def test_zero_and_nonfinite_blocks():
    x = np.zeros((1, 96))
    x[0, 40], x[0, 64] = np.inf, np.nan
    c, s = ox.quantize(x)
    assert list(s[0]) == [0, 255, 255] and not c.any()
    v = ox.values(c, s, 96)
    assert (v[0, :32] == 0).all() and np.isnan(v[0, 32:]).all()


def test_extremes_of_the_scale():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 32] = 2.0 ** -149, 3.4e38
    c, s = ox.quantize(x)
    assert list(s[0]) == [0, 252]
    assert list(ox.values(c, s, 64)[0, [0, 32]]) == [0.0, 6 * 2.0 ** 125]


def test_pack_round_trip():
    c = np.random.default_rng(0).integers(0, 16, (3, 64))
    assert ox.pack(c).shape == (3, 32)
    assert ox.pack(c)[0, 0] == c[0, 0] + 16 * c[0, 1]
    assert (ox.unpack(ox.pack(c)) == c).all()


# ------------------------------------------------------------------------------ C entry points

def _mat(**kw):
    a = dict(data=P, codes=P, scales=P, rows=4, cols=64, ld=64, dtype=_lib.MEO_F32)
    a.update(kw)
    return _lib.meo_mx4_matrix(a["data"], a["codes"], a["scales"], a["rows"], a["cols"], a["ld"], a["dtype"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "MEO_ESHAPE"), (dict(cols=-1), "MEO_ESHAPE"), (dict(rows=2 ** 31), "MEO_ESHAPE"),
    (dict(cols=2 ** 31, ld=2 ** 31), "MEO_ESHAPE"), (dict(ld=63), "MEO_ESHAPE"), (dict(ld=2 ** 31), "MEO_ESHAPE"),
    (dict(rows=2 ** 31 - 1, cols=2 ** 31 - 1, ld=2 ** 31 - 1), "MEO_ESHAPE"),  # more blocks than a launch holds
    (dict(rows=2 ** 31 - 1, cols=64), "MEO_ESHAPE"),  # one tile more than a launch holds
    (dict(dtype=_lib.MEO_I8), "MEO_EDTYPE"), (dict(dtype=_lib.MEO_MX4), "MEO_EDTYPE"),
    (dict(data=None), "MEO_ENULL"), (dict(codes=None), "MEO_ENULL"), (dict(scales=None), "MEO_ENULL"),
    (dict(data=P + 2), "MEO_EALIGN"), (dict(data=P + 1, dtype=_lib.MEO_BF16), "MEO_EALIGN"),
    (dict(codes=P + 8), "MEO_EALIGN"),
])
@pytest.mark.parametrize("call", ["meo_mx4_quantize", "meo_mx4_dequantize"])
def test_matrix_refusals(call, kw, code):
    lib = _lib.load()
    arr = (_lib.meo_mx4_matrix * 2)(_mat(rows=0, data=None, codes=None, scales=None), _mat(**kw))
    rc = getattr(lib, call)(2, arr, 0, None)
    assert _lib.ERROR_NAMES.get(rc) == code, (rc, _lib.meo_last_error())
    assert _lib.meo_last_error().startswith("matrix 1: ")


def test_transposed_leading_dimension():
    lib = _lib.load()
    arr = (_lib.meo_mx4_matrix * 1)(_mat(rows=100, cols=64, ld=64))  # data [64][100]
    assert lib.meo_mx4_quantize(1, arr, 1, None) == _lib.MEO_ESHAPE


def test_matrix_list_arguments():
    lib = _lib.load()
    assert lib.meo_mx4_quantize(0, None, 0, None) == _lib.MEO_OK
    assert lib.meo_mx4_quantize(-1, None, 0, None) == _lib.MEO_EINVAL
    assert lib.meo_mx4_dequantize(1, None, 0, None) == _lib.MEO_ENULL
    assert lib.meo_mx4_matmul(0, None, None) == _lib.MEO_OK
    assert lib.meo_mx4_matmul(-1, None, None) == _lib.MEO_EINVAL
    assert lib.meo_mx4_matmul(1, None, None) == _lib.MEO_ENULL


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), "MEO_ESHAPE"), (dict(n=-1), "MEO_ESHAPE"), (dict(k=-1), "MEO_ESHAPE"), (dict(k=2 ** 31), "MEO_ESHAPE"),
    (dict(k=2 ** 23 + 1), "MEO_ESHAPE"), (dict(m=2 ** 31 - 1, n=1, ldc=1), "MEO_ESHAPE"), (dict(ldc=7), "MEO_ESHAPE"), (dict(m=2 ** 31 - 1, n=2 ** 31 - 1, ldc=2 ** 31 - 1), "MEO_ESHAPE"),
    (dict(dtype=_lib.MEO_I8), "MEO_EDTYPE"), (dict(c=None), "MEO_ENULL"), (dict(a_codes=None), "MEO_ENULL"),
    (dict(b_scales=None), "MEO_ENULL"), (dict(c=P + 2), "MEO_EALIGN"), (dict(a_codes=P + 4), "MEO_EALIGN"),
    (dict(b_codes=P + 8), "MEO_EALIGN"),
])
def test_product_refusals(kw, code):
    a = dict(a_codes=P, a_scales=P, b_codes=P, b_scales=P, c=P, m=4, n=8, k=32, ldc=8, dtype=_lib.MEO_F32)
    a.update(kw)
    arr = (_lib.meo_mx4_product * 1)(_lib.meo_mx4_product(*a.values(), 0))
    rc = _lib.load().meo_mx4_matmul(1, arr, None)
    assert _lib.ERROR_NAMES.get(rc) == code, (rc, _lib.meo_last_error())


# ------------------------------------------------------------------------------ GaLore, MX4 projector

def _galore(shape=(64, 48), rank=8, **kw):
    p = torch.zeros(shape)
    st = _lib.galore_mx4_init_state(p, rank)
    st.update(kw)
    return p, torch.zeros(shape, dtype=torch.bfloat16), {k: v for k, v in st.items() if v is not None}


def _refused(code, hp, p, g, st, step=2):
    with pytest.raises(MeoError) as e:
        _lib.meo_galore_mx4_validate(hp, step, [p], [g], [st])
    assert _lib.ERROR_NAMES[e.value.code] == code, e.value.message


def test_galore_validate_accepts_and_refuses():
    hp = _lib.galore_hparams(rank=8)
    p, g, st = _galore()
    _lib.meo_galore_mx4_validate(hp, 2, [p], [g], [st])
    q = MX4Tensor(torch.zeros((64, 32), dtype=torch.uint8), torch.zeros((64, 2), dtype=torch.uint8), 48)
    _lib.meo_galore_mx4_validate(hp, 2, [p], [q], [st])
    _refused("MEO_EDTYPE", hp, p, g.float(), st)                       # a projected tensor's gradient is bf16 or MX4
    _refused("MEO_ENULL", hp, *_galore(projector=None))
    _refused("MEO_ENULL", hp, *_galore(projector_scale=None))
    _refused("MEO_EINVAL", hp, p, g, st, step=0)
    off = torch.zeros(8 * 32 + 8, dtype=torch.uint8)[8:].view(8, 32)
    assert off.data_ptr() % 16 == 8
    _refused("MEO_EALIGN", hp, *_galore(projector=off))
    big, gb, sb = _galore((600, 520), 512)
    _refused("MEO_EINVAL", _lib.galore_hparams(rank=512), big, gb, sb)  # rank past 256


def test_galore_validate_needs_the_gradient_scales():
    hp = _lib.galore_hparams(rank=8)
    p, g, st = _galore()
    tensors, arr = _lib._galore_mx4_args(hp, [p], [g], [st])
    tensors[0].grad_dtype = _lib.MEO_MX4
    tensors[0].grad = P
    rc = _lib.load().meo_galore_mx4_validate(hp, 2, 1, tensors, arr)
    assert rc == _lib.MEO_ENULL and "grad_scale" in _lib.meo_last_error()
    arr[0].grad_scale = P
    assert _lib.load().meo_galore_mx4_validate(hp, 2, 1, tensors, arr) == _lib.MEO_OK
    tensors[0].grad = P + 8
    assert _lib.load().meo_galore_mx4_validate(hp, 2, 1, tensors, arr) == _lib.MEO_EALIGN
    tensors[0].ndim = 3  # not projected: no MX4 gradient
    tensors[0].grad = P
    assert _lib.load().meo_galore_mx4_validate(hp, 2, 1, tensors, arr) == _lib.MEO_EDTYPE


@pytest.mark.parametrize("rows,cols", [(2 ** 24, 2 ** 23 + 1), (2 ** 29, 4), (4, 2 ** 29)])
def test_galore_validate_refuses_sizes_past_a_launch(rows, cols):
    hp = _lib.galore_hparams(rank=8)
    p, g, st = _galore()
    tensors, arr = _lib._galore_mx4_args(hp, [p], [g], [st])
    tensors[0].rows, tensors[0].cols = rows, cols
    assert _lib.load().meo_galore_mx4_validate(hp, 2, 1, tensors, arr) == _lib.MEO_ESHAPE


def test_bf16_projector_step_refuses_an_mx4_gradient():
    hp = _lib.galore_hparams(rank=8)
    p, g, _ = _galore()
    st = _lib.galore_init_state(p, 8)
    tensors = _lib._tensors([p], [g])
    tensors[0].grad_dtype = _lib.MEO_MX4
    assert _lib.load().meo_galore_validate(hp, 2, 1, tensors, _lib._galore_states([st])) == _lib.MEO_EDTYPE


def test_binding_refuses_states_of_other_shapes():
    hp = _lib.galore_hparams(rank=8)
    p, g, st = _galore()
    for key, bad, err in (("projector", torch.zeros((8, 16), dtype=torch.uint8), ValueError),
                          ("projector_scale", torch.zeros((8, 3), dtype=torch.uint8), ValueError),
                          ("exp_avg", torch.zeros((48, 8)), ValueError),
                          ("projector", torch.zeros((8, 32)), TypeError)):
        with pytest.raises(err):
            _lib.meo_galore_mx4_validate(hp, 2, [p], [g], [dict(st, **{key: bad})])
    q = MX4Tensor(torch.zeros((48, 32), dtype=torch.uint8), torch.zeros((48, 2), dtype=torch.uint8), 64)
    with pytest.raises(ValueError):  # the wrong orientation: 64 x 48 projects the columns' space
        _lib.meo_galore_mx4_validate(hp, 2, [p], [q], [st])


def test_state_is_an_eighth_of_two_bf16_copies():
    a = sum(v.numel() * v.element_size() for k, v in _lib.galore_init_state(torch.zeros(4096, 1024), 256).items()
            if k.startswith("proj"))
    b = sum(v.numel() for k, v in _lib.galore_mx4_init_state(torch.zeros(4096, 1024), 256).items()
            if k.startswith("proj"))
    assert a == 2 * 2 * 1024 * 256 and b == 17 * 1024 * 256 // 32


# ------------------------------------------------------------------------------ front ends

def test_mx4_tensor_refusals():
    c, s = torch.zeros((3, 32), dtype=torch.uint8), torch.zeros((3, 2), dtype=torch.uint8)
    assert MX4Tensor(c, s, 33).shape == (3, 33) and MX4Tensor(c, s, 64).shape == (3, 64)
    for cols in (32, 65, -1):
        with pytest.raises(ValueError):
            MX4Tensor(c, s, cols)
    with pytest.raises(TypeError):
        MX4Tensor(c.int(), s, 64)
    with pytest.raises(ValueError):
        MX4Tensor(torch.zeros((32, 3), dtype=torch.uint8).t(), s, 64)


def test_front_ends_need_a_gpu():
    q = MX4Tensor.empty(3, 40, "cpu")
    for f in (lambda: mx4_quantize(torch.zeros(3, 40)), lambda: mx4_dequantize(q), lambda: mx4_matmul(q, q)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        mx4_quantize(torch.zeros(5))


def test_binding_refusals():
    q = MX4Tensor.empty(3, 40, "cpu")
    with pytest.raises(TypeError):
        _lib.meo_mx4_quantize([torch.zeros(3, 40, dtype=torch.float16)], [q], stream=0)
    with pytest.raises(ValueError):
        _lib.meo_mx4_quantize([torch.zeros(40, 3)], [q], stream=0)
    with pytest.raises(ValueError):
        _lib.meo_mx4_quantize([torch.zeros(40, 3).t()], [q], stream=0)
    with pytest.raises(ValueError):
        _lib.meo_mx4_dequantize([torch.zeros(1, 40).expand(3, 40)], [q], stream=0)
    with pytest.raises(ValueError):
        _lib.meo_mx4_matmul([q], [MX4Tensor.empty(3, 41, "cpu")], [torch.zeros(3, 3)], stream=0)
    with pytest.raises(ValueError):
        _lib.meo_mx4_matmul([q], [q], [torch.zeros(3, 4)], stream=0)
    with pytest.raises(TypeError):
        _lib.meo_mx4_matmul([q], [q], [torch.zeros(3, 3, dtype=torch.float16)], stream=0)


def test_optimizer_refusals():
    p = torch.nn.Parameter(torch.zeros(8, 8))
    with pytest.raises(TypeError):
        GaLoreAdamW([p], projector_dtype=torch.float16)
    p.grad = torch.zeros(8, 8)
    with pytest.raises(RuntimeError):  # a bf16 projector takes whole gradients
        GaLoreAdamW([dict(params=[p], rank=4)]).compress_grad(p)
    opt = GaLoreAdamW([dict(params=[p], rank=4)], projector_dtype=torch.float4_e2m1fn_x2)
    with pytest.raises(ValueError):
        opt.compress_grad(torch.nn.Parameter(torch.zeros(2, 2)))
    opt.compress_grad(p)  # the first step refreshes the projector: the gradient stays
    assert p.grad is not None


# ------------------------------------------------------------------------------ kernel forms

def _forms(shapes, rank, grad="bf16", proj_type="std"):
    hp = _lib.galore_hparams(rank=rank, proj_type=proj_type)
    params, grads, states = [], [], []
    for s in shapes:
        p = torch.empty(s, device="meta")
        params.append(p)
        right = (s[0] >= s[1]) == (proj_type == "std") if len(s) == 2 else True
        n, m = s if right and len(s) == 2 else s[::-1] if len(s) == 2 else (0, 0)
        mx = grad == "mx4" and len(s) == 2
        grads.append(MX4Tensor.empty(n, m, "meta") if mx else torch.empty(s, dtype=torch.bfloat16, device="meta"))
        states.append(_lib.galore_mx4_init_state(p, rank, proj_type) if len(s) == 2 else
                      {k: torch.zeros(s, device="meta") for k in ("exp_avg", "exp_avg_sq")})
    tensors, arr = _lib._galore_mx4_args(hp, params, grads, states)
    for t, a in zip(tensors, arr):  # validation inspects pointers and follows none
        t.param = t.grad = a.exp_avg = a.exp_avg_sq = P
        if a.projector is not None or t.ndim == 2:
            a.projector = a.projector_scale = a.grad_scale = P
    out = (_lib.meo_galore_mx4_form * len(shapes))()
    _lib._check(_lib.load().meo_galore_mx4_forms(hp, len(shapes), tensors, arr, out))
    return out


def test_forms_of_a_step():
    f = _forms([(4096, 4096)], 64)[0]
    assert (f.rows, f.aligned, f.parts, f.item_parts) == (64, 1, 4, 1) and f.back_tiles >= 1
    f = _forms([(4096, 4097), (777,)], 64)
    assert (f[0].rows, f[0].aligned) == (64, 0) and not any(getattr(f[1], k) for k, _ in f[1]._fields_)
    assert _forms([(11008, 4096), (4096, 11008)], 256, grad="mx4")[0].rows == 128
    assert _forms([(11008, 4096)], 256, grad="mx4")[0].rows == 64
    with pytest.raises(MeoError):
        _forms([(600, 520)], 512)
    hp = _lib.galore_hparams(rank=8)
    p, g, st = _galore()
    tensors, arr = _lib._galore_mx4_args(hp, [p], [g], [st])
    assert _lib.load().meo_galore_mx4_forms(hp, 1, tensors, arr, None) == _lib.MEO_ENULL
    assert len(_lib.meo_galore_mx4_forms(hp, [p], [g], [st])) == 1


def test_rows_of_a_product():
    assert [_lib.meo_mx4_matmul_rows(*s) for s in ((0, 5), (5, 0), (1, 1), (40000, 128), (32000, 256), (16384, 256))] == \
        [0, 0, 64, 64, 128, 64]


def test_parts_of_a_contraction_follow_from_the_tensor_alone():
    """Whatever else is in the list; how many of them a block takes may not."""
    tensors = [(4096, 4096), (1700, 1680), (1951, 3810), (3750, 4266), (300, 72), (70, 9000)]
    for proj_type in ("std", "reverse_std"):
        alone = [_forms([s], 64, proj_type=proj_type)[0] for s in tensors]
        for rest in ([(64, 64)], [(32400, 8)], [(4096, 4096)] * 3, tensors):
            for i, s in enumerate(tensors):
                f = _forms([s] + rest, 64, proj_type=proj_type)[0]
                assert f.parts == alone[i].parts
    assert [f.parts for f in (_forms([s], 64)[0] for s in tensors)] == [4, 4, 4, 3, 1, 1]
    assert [f.item_parts for f in (_forms([s], 64)[0] for s in tensors)] == [1] * 6
    assert [_forms([s] * 4, 64)[0].item_parts for s in tensors] == [4, 4, 4, 3, 1, 1]


# ------------------------------------------------------------------------------ memory

def _memory(shapes, rank, proj_type="std"):
    """Bytes of projectors and workspace, bf16 and MX4."""
    hp = _lib.galore_hparams(rank=rank, proj_type=proj_type)
    ps = [torch.empty(s, device="meta") for s in shapes]
    tensors = _lib._tensors(ps, ps)
    for t in tensors:
        t.param = t.grad = P
    out = []
    for shapes_of, size, ws in ((_lib.galore_state_shapes, 2, _lib.load().meo_galore_workspace_size),
                                (_lib.galore_mx4_state_shapes, 1, _lib.load().meo_galore_mx4_workspace_size)):
        state = sum(size * math.prod(v) for s in shapes for k, v in shapes_of(s, rank, proj_type).items() if k.startswith("proj"))
        out.append((state, ws(hp, len(ps), tensors)))
    return out


LLAMA_LAYER = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]


@pytest.mark.parametrize("shapes,rank,proj_type", [
    (LLAMA_LAYER * 32 + [(32000, 4096)] * 2, 256, "std"), (LLAMA_LAYER, 256, "std"), (LLAMA_LAYER, 64, "std"),
    (LLAMA_LAYER, 100, "reverse_std"), ([(4096, 4096)], 256, "std"), ([(1024, 4096)], 128, "std"),
    ([(1024, 1024)] * 96, 32, "std"), ([(256, 512), (200, 96)], 64, "std"), ([(64, 160), (160, 48)], 16, "std")])
def test_mx4_projectors_take_less_memory(shapes, rank, proj_type):
    """With the workspace that the optimizer keeps: the refresh's scratch and the step's."""
    (state, ws), (state4, ws4) = _memory(shapes, rank, proj_type)
    assert state4 + ws4 < state + ws and state4 < state / 3
    if sum(s[0] * s[1] for s in shapes) > 10 ** 8:
        assert ws4 < ws and state4 < state / 7


@pytest.mark.parametrize("shape,rank", [((4096, 4096), 64), ((8192, 1700), 64), ((2048, 2048), 32), ((2048, 2048), 250)])
def test_memory_of_one_tensor_in_parts(shape, rank):
    """Stepped alone, a tensor's projection stores the sums of its parts: at most a fifth more then."""
    (state, ws), (state4, ws4) = _memory([shape], rank)
    assert state4 + ws4 < 1.2 * (state + ws)
