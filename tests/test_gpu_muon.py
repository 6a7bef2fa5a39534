"""Muon's operators on the GPU: orthogonalize and the Muon step against oracle/muon.py in float64.

Bars. The momentum is compared bit for bit (its float32 arithmetic is the oracle's). What the
orthogonalization rounds (fp16 operands) is derived in oracle/muon.py: after one step element
by element (bound_of_one_step); after several, whose roundings propagate, against
rounded_newton_schulz, which makes the same roundings in float64 otherwise: the library's
result is one more realization of them (float32 sums in another order put some values on the
other side of a border), so it may be as far from the exact one as that one is, twice over for
the chance in both. A bfloat16 result adds half a step, 2^-8 of the value; a float32 parameter
2^-24 of it and of the update. ``raw`` takes the results in float32: Muon's step on a parameter of
zeros without decay and with lr s = 1.
"""
import math

import numpy as np
import pytest
import torch

from memory_efficient_optimizers_amd import MeoError, Muon, _lib, orthogonalize
from oracle import galore as ga
from oracle import muon as om
from tests.harness import to64
from tests.test_muon_host import DOCUMENTED, _documented

pytestmark = pytest.mark.gpu
DEV = "cuda"


def matrix(shape, seed, kind="noise", dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    if kind == "low":  # rank 3 plus noise, rows of different size
        *b, m, n = shape
        x = torch.randn(*b, m, 3, generator=gen) @ torch.randn(*b, 3, n, generator=gen) + 1e-2 * x
        x = x * torch.exp(torch.randn(*b, m, 1, generator=gen))
    return x.to(dtype).to(DEV)


def each(x):
    return to64(x).reshape(-1, *x.shape[-2:])


def exact(x, **kw):
    return np.stack([om.newton_schulz(v, **kw) for v in each(x)]).reshape(tuple(x.shape))


def slack(x, **kw):
    """What the roundings may cost each matrix (Frobenius norm)."""
    return [2 * np.linalg.norm(om.rounded_newton_schulz(v, **kw) - om.newton_schulz(v, **kw)) for v in each(x)]


def muon_step(ps, gs, sts, step=1, **kw):
    hp = _lib.muon_hparams(**kw)
    ws = _lib.workspace(_lib.meo_muon_workspace_size(hp, ps, gs, sts), DEV)
    _lib.meo_muon_step(hp, step, ps, gs, sts, ws)


def raw(xs, **kw):
    """The orthogonalized xs in float32."""
    out = []
    for x in xs:
        r, c = x.shape[-2:]
        p = torch.zeros(x.shape, dtype=torch.float32, device=DEV)
        muon_step([p], [x], [dict(exp_avg=torch.zeros(x.shape, dtype=torch.float32, device=DEV))], lr=1.0 / (0.2 * math.sqrt(max(r, c))),
                  momentum=0.0, weight_decay=0.0, nesterov=False, adjust_lr="match_rms_adamw", **kw)
        out.append(-p)
    return out


def check(y, x, **kw):
    """y = orthogonalize(x) in bfloat16 or float32."""
    want, got = exact(x, **kw).reshape(-1, *x.shape[-2:]), each(y)
    step = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -22
    for k, lim in enumerate(slack(x, **kw)):
        err, norm = np.linalg.norm(got[k] - want[k]), np.linalg.norm(want[k])
        assert err <= lim + step * (norm + lim) + 1e-30, (k, err, lim, norm)


SHAPES = [(1, 1), (1, 7), (9, 1), (3, 2), (31, 33), (63, 65), (64, 64), (65, 64), (64, 129), (130, 70), (128, 200), (257, 129),
          (300, 520), (640, 250)]


# ------------------------------------------------------------------------------ orthogonalize

@pytest.mark.parametrize("shape", SHAPES)
def test_one_step_element_by_element(shape):
    x = matrix(shape, 1)
    y = raw([x], ns_steps=1)[0]
    want = exact(x, steps=1)
    lim = om.bound_of_one_step(to64(x)) + 2.0 ** -22 * np.abs(want)
    assert np.all(np.abs(to64(y) - want) <= lim), np.max(np.abs(to64(y) - want) / lim)


@pytest.mark.parametrize("kind", ["noise", "low"])
@pytest.mark.parametrize("shape", SHAPES + [(16, 4096), (4096, 16), (100, 2600), (1000, 1100)])
def test_steps(shape, kind):
    x = matrix(shape, 2, kind)
    check(raw([x])[0], x)
    check(orthogonalize(x), x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(3, 65, 40), (2, 2, 33, 130), (70, 5, 3), (1, 64, 64), (4, 40, 300)])
def test_batches(shape, dtype):
    x = matrix(shape, 3, dtype=dtype)
    y = orthogonalize(x)
    assert y.shape == x.shape and y.dtype == torch.bfloat16
    check(y, x)


def test_empty_and_single():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (3, 0, 4)):
        assert orthogonalize(torch.zeros(shape, device=DEV)).shape == shape
    ys = orthogonalize([torch.zeros(0, 5, device=DEV), matrix((4, 5), 1), torch.zeros(2, 0, device=DEV)])
    check(ys[1], matrix((4, 5), 1))
    assert _lib.meo_orthogonalize(_lib.orthogonalize_hparams(), [], []) is None


def test_layouts():
    """Row-major, strided rows, column-major, a batch of column-major ones, views that are copied."""
    base = matrix((5, 90, 200), 4)
    for x in (base[0, :, 3:150], base[:, :, 3:150], base[0].t(), base.mT, base[1, ::2], base[:, ::3, 1::2], base[0, :, 7:8],
              base[0, 3:4, 5:77], base[::2], base.permute(1, 0, 2)):
        y = orthogonalize(x)
        assert y.shape == x.shape
        check(y, x)
    x = base[0].t()
    assert orthogonalize(x).stride() == x.stride()


def test_out():
    x = matrix((90, 200), 5)
    whole = torch.full((92, 210), 7.0, dtype=torch.bfloat16, device=DEV)
    o = whole[1:91, 4:204]
    assert orthogonalize(x, out=o) is o
    check(o, x)
    rest = whole.clone()
    rest[1:91, 4:204] = 7.0
    assert (rest == 7.0).all()  # nothing beside the view
    c = torch.empty(200, 90, dtype=torch.bfloat16, device=DEV).t()
    assert torch.equal(orthogonalize(x, out=c), o) and c.stride() == (1, 90)
    b = x.bfloat16()
    want = orthogonalize(b)
    assert torch.equal(orthogonalize(b, out=b), want)  # in place
    t = x.bfloat16().t().contiguous().t()
    assert torch.equal(orthogonalize(t, out=t), want)


def test_values_at_the_ends_of_the_range():
    x = matrix((70, 130), 6)
    want = to64(raw([x])[0])
    for scale in (1e-30, 1e30):
        for v in raw([x * scale], eps=0.0):
            assert np.linalg.norm(to64(v) - want) <= 4e-3 * np.linalg.norm(want)  # (another realization)
    y = orthogonalize([torch.zeros(40, 30, device=DEV), x])
    assert (y[0] == 0).all()
    assert (orthogonalize(torch.zeros(40, 30, device=DEV), eps=0.0) == 0).all()
    z = x.clone()
    z[3] = 0.0
    z[:, 5] = 0.0
    o = orthogonalize(z)
    assert (o[3] == 0).all() and (o[:, 5] == 0).all()
    check(o, z)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_non_finite_matrices_are_nan_throughout_and_alone(value):
    x = matrix((3, 70, 40), 7)
    x[1, 69, 39] = value
    y = orthogonalize([x, matrix((30, 20), 8)])
    assert y[0][1].isnan().all() and y[0][0].isfinite().all() and y[0][2].isfinite().all() and y[1].isfinite().all()
    check(y[0][::2].contiguous(), x[::2].contiguous())


def test_norms_near_and_below_eps():
    x = matrix((20, 30), 9)
    x = x / x.norm()
    for f in (4.0, 1.0, 0.25, 2.0 ** -6):
        y = raw([x * f], eps=1.0)[0]
        check(y, x * f, eps=1.0)
    # far below: entries lose what is under 2^-24 of an orthonormal row's
    y, want = to64(raw([x * 1e-5], eps=1.0)[0]), exact(x * 1e-5, eps=1.0)
    assert np.max(np.abs(y - want)) <= 485 * 2.0 ** -24 / math.sqrt(30) * 2


@pytest.mark.parametrize("steps", [5, 10])
@pytest.mark.parametrize("kind", list(DOCUMENTED))
def test_documented_precision_on_the_gpu(kind, steps):
    """meo.h's table, and what the roundings of the very same matrices cost in the oracle. Not so where entries are
    equal, all or in blocks: the error is that of one or a few values, not a norm over many, and may vanish in the
    oracle by chance. One rounding of A that a float32 sum in another order turns round, 2^-11 of A, moves such a value
    by |b s^2 + 2 c s^4| 2^-11 <= 2.5 x 2^-11 = 1.2e-3 of it, in every step."""
    rng = np.random.default_rng(117)
    for m, n in ((70, 90), (128, 128), (200, 333), (500, 520), (700, 1400)):
        x = torch.from_numpy(_documented(kind, rng, m, n)).float().to(DEV)
        x = x.t().contiguous() if m == 200 else x
        if min(x.shape) <= 64:
            continue
        got, want = to64(raw([x], ns_steps=steps)[0]), exact(x, steps=steps)
        err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
        assert err <= DOCUMENTED[kind][steps // 10] * norm, (x.shape, err / norm)
        assert kind in ("ones", "blocks") or err <= slack(x, steps=steps)[0] + 8 * 2.0 ** -24 * norm, (x.shape, err / norm)


@pytest.mark.parametrize("shape", [(24, 40), (24, 1400), (100, 200), (3, 70, 40)])
def test_zero_matrices_at_any_eps(shape):
    """Zeros whatever eps is, also where 1 / eps is not finite; a matrix beside them is itself."""
    z, x = torch.zeros(shape, device=DEV), matrix(shape, 121)
    for eps in (0.0, 5e-324, 1e-310, 1e-305, 1e-300, 1e300):
        assert (orthogonalize(z, eps=eps) == 0).all()
        if eps < 1.0:
            assert torch.equal(orthogonalize([z, x], eps=eps)[1], orthogonalize(x))
        p = torch.ones(shape, device=DEV)
        muon_step([p], [z], [dict(exp_avg=z.clone())], lr=0.5, weight_decay=0.0, eps=eps)
        assert (p == 1).all()


def one_entry_rows(shape, kind):
    """Rows with one entry each, in order or not, of one size or not."""
    m, n = min(shape), max(shape)
    gen = torch.Generator().manual_seed(116)
    x = torch.zeros(m, n)
    at = torch.arange(m) if kind == "identity" else torch.randperm(n, generator=gen)[:m]
    x[torch.arange(m), at] = (torch.exp(1.5 * torch.randn(m, generator=gen)) if kind == "sizes"
                              else 1.0 - 2.0 * (torch.rand(m, generator=gen) < 0.5) if kind == "signs" else torch.ones(m))
    return (x if shape[0] == m else x.t().contiguous()).to(DEV)


@pytest.mark.parametrize("steps", [1, 5, 10])
@pytest.mark.parametrize("kind", ["identity", "signs", "sizes"])
@pytest.mark.parametrize("shape", [(100, 100), (300, 300), (343, 343), (481, 481), (364, 700), (700, 130), (1000, 1100), (65, 33000)])
def test_rows_of_one_entry(shape, kind, steps):
    """A's diagonal from both parts of X. Roundings to float32 do not average out either (X_0, the split's 2^-23, two
    sums, a row's factor, lr s and its product: 8 x 2^-24)."""
    x = one_entry_rows(shape, kind)
    got, want = to64(raw([x], ns_steps=steps)[0]), exact(x, steps=steps)
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= slack(x, steps=steps)[0] + 8 * 2.0 ** -24 * norm
    if steps == 5 and kind != "sizes":  # the bound of tests/test_muon_host.py
        assert err <= 3.1e-3 * norm


@pytest.mark.parametrize("shape", [(4096, 4096), (4096, 11008), (2048, 2048), (1024, 4096)])
def test_rows_of_one_entry_in_large_tiles(shape):
    """The same in every form (bound as above)."""
    x = one_entry_rows(shape, "signs")
    s = 1.0 / math.sqrt(shape[0])
    for a, b, c in [om.COEFFICIENTS] * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    for v in (x, x.t().contiguous()):
        assert (raw([v])[0].double() - s * v.double()).norm() <= 3.1e-3 * s * math.sqrt(shape[0])


@pytest.mark.parametrize("shape", [(1, 1), (2, 2), (40, 60), (20, 1500), (70, 130)])
def test_singular_values_up_to_8(shape):
    """The largest that coefficients may let grow, in a matrix of rank 1 (entries 8 and less). Beside the
    products' roundings one entry has most of the norm: X_0 to float32, two splits (2^-23), two sums, lr s, its product: 9 x 2^-24."""
    x = torch.ones(shape, device=DEV)
    x[0] = 2.0 ** -20  # (one row, or one entry, has most of it)
    x[:, 0] *= 2.0 ** 20
    for coefficients in ([(8.0, 0.0, 0.0), (0.9, -0.02, 0.0002)], [(8.0, 0.0, 0.0), (0.125, 0.0, 0.0)]):
        got, want = to64(raw([x], ns_steps=2, ns_coefficients=coefficients)[0]), exact(x, steps=2, coefficients=coefficients)
        lim = slack(x, steps=2, coefficients=coefficients)[0] + 9 * 2.0 ** -24 * np.linalg.norm(want)
        assert np.linalg.norm(got - want) <= lim, (np.linalg.norm(got - want), lim)


@pytest.mark.parametrize("steps,coefficients", [(1, om.COEFFICIENTS), (2, om.COEFFICIENTS), (8, om.COEFFICIENTS), (10, (2.0, -1.5, 0.5)),
                                                (4, [(8.2, -22.9, 16.46), (4.0, -2.9, 0.5), (3.9, -2.8, 0.5), (3.3, -2.4, 0.5)])])
def test_coefficients_and_steps(steps, coefficients):
    x = matrix((96, 160), 10)
    check(raw([x], ns_steps=steps, ns_coefficients=coefficients)[0], x, steps=steps, coefficients=coefficients)
    check(orthogonalize(x, steps=steps, coefficients=coefficients), x, steps=steps, coefficients=coefficients)


MIXED = [(64, 64), (16, 4096), (700, 130), (3, 65, 40), (1, 5), (1200, 1300), (130, 70), (2048, 2048), (40, 1000), (64, 129), (9, 1),
         (300, 520), (31, 33), (4, 4), (5, 5), (6, 6), (257, 129), (7, 7), (512, 512)]


def test_lists_match_single_calls_bit_for_bit():
    """More tensors than a launch holds, of every size: each as it comes out alone."""
    xs = [matrix(s, 20 + i, dtype=[torch.float32, torch.bfloat16][i % 2]) for i, s in enumerate(MIXED)]
    ys = orthogonalize(xs)
    for x, y in zip(xs, ys):
        assert torch.equal(y, orthogonalize(x))
    zs = orthogonalize(xs[::-1])
    assert all(torch.equal(a, b) for a, b in zip(ys, zs[::-1]))


def reference64(x, steps=5):
    """On the GPU in float64, for sizes that the host takes long for."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    x = x / x.norm()
    for _ in range(steps):
        g = x @ x.t().contiguous()
        x = 3.4445 * x + (-4.7750 * g + 2.0315 * (g @ g)) @ x
    return x.t() if tall else x


@pytest.mark.parametrize("shape", [(4096, 4096), (2048, 5461), (11008, 4096), (1951, 3810), (32000, 256)])
def test_large(shape):
    """(Rounding errors of large matrices are those of smaller ones: 4e-3, tests/test_muon_host.py.)"""
    x = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(11), device=DEV)
    want = reference64(x)
    err = (raw([x])[0].double() - want).norm() / want.norm()
    assert err <= 4e-3, err
    y = orthogonalize(x.t()).t().double()  # column-major: the same values turned round
    assert (y - want).norm() <= (4e-3 + 2.0 ** -8) * want.norm()


# Matrices whose ends lie inside a tile of every size, wide and tall; companions in a list that bring its tiles to
# every form, and the forms (of A, the polynomial, X).
ENDED = [(1250, 1700), (1600, 1300)]
COMPANIONS = [([(500, 500)], (64, 64, 64)), ([(1000, 1000)] * 4, (64, 64, 192)), ([(500, 500)] * 8, (64, 128, 128)),
              ([(500, 500)] * 2, (128, 128, 64)), ([(500, 500)] * 4, (128, 128, 128)), ([(750, 750)] * 8, (128, 128, 192)),
              ([(4096, 4096)], (128, 128, 256)), ([(2000, 2000)] * 3, (192, 192, 192)), ([(2500, 2500)] * 8, (256, 256, 128)),
              ([(2250, 2250)] * 4, (256, 256, 192)), ([(2500, 2500)] * 4, (256, 256, 256))]


@pytest.mark.parametrize("param,steps", [(torch.float32, 1), (torch.float32, 3), (torch.bfloat16, 2)])
def test_every_tile_form_gives_the_same_bits(param, steps):
    """As the matrices come out alone, which test_ends_of_tiles_element_by_element holds to the formula."""
    made = [matrix(s, 118 + i) for i, s in enumerate(ENDED)]

    def step(xs):
        ps = [torch.full(x.shape, 0.5, dtype=param, device=DEV) for x in xs]
        muon_step(ps, xs, [dict(exp_avg=torch.zeros(x.shape, device=DEV)) for x in xs], lr=0.1, momentum=0.0, nesterov=False,
                  ns_steps=steps)
        return ps

    want = [step([x])[0] for x in made]
    decayed = step([torch.zeros(70, 70, device=DEV)])[0][0, 0]
    for more, form in COMPANIONS:
        xs = made + [torch.zeros(s, device=DEV) for s in more]
        got = _lib.meo_orthogonalize_forms(_lib.orthogonalize_hparams(steps), xs, [x.bfloat16() for x in xs])
        assert all((f.pieces, f.gram, f.poly, f.apply) == (1, *form) for f in got), (more, form)
        ps = step(xs)
        assert all(torch.equal(a, b) for a, b in zip(ps, want)), (more, form)
        assert all((p == decayed).all() for p in ps[2:]), (more, form)


@pytest.mark.parametrize("shape", ENDED)
def test_ends_of_tiles_element_by_element(shape):
    x = matrix(shape, 118 + ENDED.index(shape))
    want = exact(x, steps=1)
    lim = om.bound_of_one_step(to64(x)) + 2.0 ** -22 * np.abs(want)
    assert np.all(np.abs(to64(raw([x], ns_steps=1)[0]) - want) <= lim)
    check(raw([x], ns_steps=3)[0], x, steps=3)


def test_several_parts_of_a_list():
    """Matrices past what is worked on together (2^26 values)."""
    xs = [torch.randn(s, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV).bfloat16()
          for i, s in enumerate([(4096, 8192), (3, 2048, 6000), (5000, 4000), (64, 64)])]
    ys = orthogonalize(xs)
    for k in (0, 2, 3):
        want = reference64(xs[k])
        assert (ys[k].double() - want).norm() <= (4e-3 + 2.0 ** -8) * want.norm()
    for b in range(3):
        assert torch.equal(ys[1][b], orthogonalize(xs[1][b]))


# ------------------------------------------------------------------------------ few rows

# One strip of 512 columns and up to 64 (32 of 64 rows) of them, either way round, and what lies beside.
FEW = [(1, 512), (513, 1), (15, 511), (16, 512), (513, 16), (17, 700), (32, 512), (32, 1025), (512, 33), (1025, 33), (64, 512), (64, 513),
       (63, 5000), (2000, 32), (5, 12000)]
ENDS = [(16, 32768), (32769, 16), (31, 32767), (64, 16384), (16385, 64)]


@pytest.mark.parametrize("shape", FEW)
def test_few_rows_one_step_element_by_element(shape):
    x = matrix(shape, 100)
    want = exact(x, steps=1)
    lim = om.bound_of_one_step(to64(x)) + 2.0 ** -22 * np.abs(want)
    assert np.all(np.abs(to64(raw([x], ns_steps=1)[0]) - want) <= lim)


@pytest.mark.parametrize("kind", ["noise", "low"])
@pytest.mark.parametrize("shape", FEW + ENDS)
def test_few_rows(shape, kind):
    x = matrix(shape, 101, kind)
    check(raw([x])[0], x)
    check(orthogonalize(x), x)


def single_newton_schulz(u):
    """In float32 throughout."""
    x, tall = om.start(u, 1e-7)
    x = x.astype(np.float32)
    a, b, c = (np.float32(v) for v in om.COEFFICIENTS)
    for _ in range(5):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.T if tall else x).astype(np.float64)


@pytest.mark.parametrize("kind", ["noise", "low"])
@pytest.mark.parametrize("shape", FEW + [(1, 1), (3, 2), (16, 16), (32, 32), (31, 33), (64, 64), (48, 200)])
def test_few_rows_keep_22_bits(shape, kind):
    """Two fp16 parts hold 22 bits, 2^-22 against float32's 2^-24: four times float32's errors, and once more for
    the float32 sums in another order; twice for the chance in both realizations. The result's own rounding 2^-22."""
    x = matrix(shape, 109, kind)
    u = to64(x)
    want, got = om.newton_schulz(u), to64(raw([x])[0])
    lim = 2 * 5 * np.linalg.norm(single_newton_schulz(u) - want) + 2.0 ** -22 * np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= lim, (np.linalg.norm(got - want), lim)


@pytest.mark.parametrize("shape", [(5, 1, 600), (3, 40, 600), (2, 700, 20), (4, 30, 30), (2, 3, 1100, 60)])
def test_batches_of_few_rows(shape):
    x = matrix(shape, 102, dtype=torch.bfloat16)
    y = orthogonalize(x)
    check(y, x)
    flat = x.reshape(-1, *shape[-2:])
    assert all(torch.equal(a, orthogonalize(b)) for a, b in zip(y.reshape(flat.shape), flat))


@pytest.mark.parametrize("shape", [(20, 1300), (1300, 20), (60, 90), (90, 60)])
def test_layouts_of_few_rows(shape):
    """Strided rows, column-major, results into a view whose surroundings stay."""
    r, c = shape
    base = matrix((r + 4, c + 9), 103)
    for x in (base[1:r + 1, 3:c + 3], base[1:r + 1, 3:c + 3].t()):
        whole = torch.full((x.shape[0] + 3, x.shape[1] + 5), 7.0, dtype=torch.bfloat16, device=DEV)
        o = whole[2:-1, 3:-2]
        assert orthogonalize(x, out=o) is o
        check(o, x)
        assert torch.equal(orthogonalize(x), o)
        whole[2:-1, 3:-2] = 7.0
        assert (whole == 7.0).all()
    b = base[1:r + 1, 3:c + 3].bfloat16()
    want = orthogonalize(b)
    assert torch.equal(orthogonalize(b, out=b), want)  # in place


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rows,cols", [(30, 20), (900, 40), (12, 2000), (70, 100), (300, 200)])
def test_non_finite_matrices_of_every_kind(rows, cols, value):
    x = matrix((3, rows, cols), 104)
    x[1, rows - 1, cols - 1] = value
    y = orthogonalize([x, matrix((30, 20), 8)])
    assert y[0][1].isnan().all() and y[0][0].isfinite().all() and y[0][2].isfinite().all() and y[1].isfinite().all()
    check(y[0][::2].contiguous(), x[::2].contiguous())
    p, g, st = init((rows, cols), 105, F, F, F)
    g[0, 0] = value
    muon_step([p], [g], [st], lr=0.1)
    assert p.isnan().all()


@pytest.mark.parametrize("shape", [(24, 40), (24, 1400), (100, 200)])
def test_values_at_the_ends_of_the_range_of_every_kind(shape):
    x = matrix(shape, 106)
    want = to64(raw([x])[0])
    for scale in (1e-30, 1e30):
        for v in raw([x * scale], eps=0.0):
            assert np.linalg.norm(to64(v) - want) <= 4e-3 * np.linalg.norm(want)  # (another realization)
    assert (orthogonalize(torch.zeros(shape, device=DEV)) == 0).all()
    assert (orthogonalize(torch.zeros(shape, device=DEV), eps=0.0) == 0).all()
    z = x.clone()
    z[3] = 0.0
    z[:, 5] = 0.0
    o = orthogonalize(z)
    assert (o[3] == 0).all() and (o[:, 5] == 0).all()
    check(o, z)


def test_long_lists_of_few_rows():
    """More of each kind than a launch takes: each as it comes out alone."""
    shapes = [(1 + i % 16, 20 + 3 * i) for i in range(50)] + [(600 + 40 * i, 17 + i % 16) for i in range(18)] + [(40, 64)] * 3
    xs = [matrix(s, 200 + i) for i, s in enumerate(shapes)]
    ys = orthogonalize(xs)
    assert all(torch.equal(y, orthogonalize(x)) for x, y in zip(xs, ys))


def test_more_matrices_than_a_launch_or_a_part_takes():
    """Past 2^22 matrices of one strip, past 2^26 values in strips: as they come out alone."""
    x = matrix((2 ** 22 + 9, 1, 1), 111)
    y, one = orthogonalize([x, matrix((2, 3), 112)])[0], orthogonalize(torch.ones(1, 1, device=DEV))
    want = one * x.sign().bfloat16()
    for k in (x.abs().flatten() < 1e-7).nonzero().flatten().tolist():  # (X_0 = x / eps there, not its sign)
        want[k] = orthogonalize(x[k])
    assert torch.equal(y, want)
    x = matrix((4200, 16, 1000), 113, dtype=torch.bfloat16)
    y = orthogonalize(x)
    for k in (0, 1, 2099, 4095, 4096, 4199):
        assert torch.equal(y[k], orthogonalize(x[k]))


def test_offsets_past_32_bits():
    """Matrices behind 2^31 values of their tensor."""
    for shape in ((2 ** 22 + 3, 20, 30), (33000, 60, 1100), (33000, 200, 400)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        last = matrix(shape[1:], 114, dtype=torch.bfloat16)
        x[-1] = last
        x[-3] = last
        y = orthogonalize(x)
        want = orthogonalize(last)
        assert torch.equal(y[-1], want) and torch.equal(y[-3], want) and not y[-2].any() and not y[0].any()
        del x, y


def test_steps_and_coefficients_of_few_rows():
    for shape in ((40, 100), (20, 1700)):
        x = matrix(shape, 107)
        for steps, coefficients in ((1, om.COEFFICIENTS), (2, om.COEFFICIENTS), (10, (2.0, -1.5, 0.5)),
                                    (4, [(8.2, -22.9, 16.46), (4.0, -2.9, 0.5), (3.9, -2.8, 0.5), (3.3, -2.4, 0.5)])):
            check(orthogonalize(x, steps=steps, coefficients=coefficients), x, steps=steps, coefficients=coefficients)


def scaled(shape, seed, kind):
    """Matrices whose entries have very different size: one strong entry over noise of 1e-6, sizes of the
    shorter side's rows over five decades, rank 1."""
    gen = torch.Generator().manual_seed(seed)
    m, n = min(shape), max(shape)
    x = torch.randn(m, n, generator=gen)
    if kind == "entry":
        x = 1e-6 * x
        x[m // 3, n // 2] = 1.0
    if kind == "decades":
        x = x * torch.logspace(0, -5, m).unsqueeze(1)
    if kind == "one":
        x = torch.randn(m, 1, generator=gen) @ torch.randn(1, n, generator=gen)
    return (x if shape[0] == m else x.t().contiguous()).to(DEV)


def few_slack(u, **kw):
    """Of matrices with few rows: operands in two parts and float32's own roundings, each in two realizations."""
    want = om.newton_schulz(u, **kw)
    return 2 * (np.linalg.norm(om.rounded_newton_schulz(u, parts=2, **kw) - want) + np.linalg.norm(om.single_newton_schulz(u, **kw) - want))


@pytest.mark.parametrize("kind,steps", [("entry", 5), ("entry", 10), ("decades", 5), ("decades", 10), ("one", 5)])
@pytest.mark.parametrize("shape", [(16, 16), (30, 20), (64, 64), (48, 200), (16, 900), (900, 16), (60, 2000), (2000, 32)])
def test_few_rows_of_very_different_size(shape, kind, steps):
    """The result's own rounding: 2^-22."""
    x = scaled(shape, 115, kind)
    u = to64(x)
    want, got = om.newton_schulz(u, steps), to64(raw([x], ns_steps=steps)[0])
    lim = few_slack(u, steps=steps) + 2.0 ** -22 * np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= lim, (np.linalg.norm(got - want), lim)


# ------------------------------------------------------------------------------ the Muon step

def init(shape, seed, param, grad, state, scale=1e-3):
    gen = torch.Generator().manual_seed(seed)
    p = (0.02 * torch.randn(shape, generator=gen)).to(param).to(DEV)
    g = (scale * torch.randn(shape, generator=gen)).to(grad).to(DEV)
    m = scale * 0.7 * torch.randn(shape, generator=gen)
    if state == torch.int8:
        c, s = om.quantize(m.numpy())
        return p, g, dict(exp_avg=torch.from_numpy(c).to(DEV), exp_avg_scale=torch.from_numpy(s).to(DEV))
    return p, g, dict(exp_avg=m.to(state).to(DEV))


def momentum_of(st):
    m = st["exp_avg"].cpu()
    return om.dequantize(m.numpy(), st["exp_avg_scale"].cpu().numpy()) if m.dtype == torch.int8 else m.float().numpy()


def check_step(p, st, p0, g, m0, kind, **kw):
    """kw: of oracle.muon.muon_step_tensor."""
    want, m, q = om.muon_step_tensor(p0, g, m0, kind=kind, **kw)
    if q is not None:
        assert np.array_equal(st["exp_avg"].cpu().numpy(), q[0])
        assert np.array_equal(st["exp_avg_scale"].cpu().numpy(), q[1], equal_nan=True)
    assert np.array_equal(momentum_of(st), m, equal_nan=True)
    rows, cols = p0.shape[-2:]
    u = om.direction(m, g, kw.get("momentum_", 0.95), kw.get("nesterov", True)).reshape(-1, rows, cols)
    c = kw.get("lr", 1e-3) * om.shape_scale(kw.get("adjust_lr", "original"), rows, cols)
    got, exp = to64(p).reshape(-1, rows, cols), want.reshape(-1, rows, cols)
    half = 2.0 ** -8 if p.dtype == torch.bfloat16 else 2.0 ** -23  # (fp32: the decayed value's rounding too)
    for k in range(len(u)):
        lim = c * 2 * np.linalg.norm(om.rounded_newton_schulz(u[k]) - om.newton_schulz(u[k]))
        err = np.linalg.norm(got[k] - exp[k])
        assert err <= lim + half * (np.linalg.norm(exp[k]) + c * math.sqrt(min(rows, cols)) * 2), (k, err, lim)


F, B, I = torch.float32, torch.bfloat16, torch.int8


@pytest.mark.parametrize("adjust_lr", ["original", "match_rms_adamw"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("param,grad,state", [(F, F, F), (F, B, F), (F, B, I), (B, B, B), (B, F, I), (F, F, B), (B, B, F)])
def test_step(param, grad, state, nesterov, adjust_lr):
    shapes = [(64, 48), (77, 130), (3, 64, 40), (200, 65), (1, 513), (300, 1)]
    made = [init(s, 30 + i, param, grad, state) for i, s in enumerate(shapes)]
    ps, gs, sts = ([v[k] for v in made] for k in range(3))
    before = [(to64(p), g.float().cpu().numpy(), momentum_of(st)) for p, g, st in made]
    kw = dict(lr=0.05, weight_decay=0.1, nesterov=nesterov, adjust_lr=adjust_lr)
    muon_step(ps, gs, sts, momentum=0.9, **kw)
    for p, st, (p0, g, m0) in zip(ps, sts, before):
        check_step(p, st, p0, g, m0, str(state).split(".")[1], momentum_=0.9, **kw)


@pytest.mark.parametrize("param,grad,state", [(F, F, F), (F, B, I), (B, B, B), (B, F, I), (F, F, B)])
def test_step_of_few_rows(param, grad, state):
    """One strip and several, either way round, odd sizes, a batch (8-bit: whole groups)."""
    shapes = [(16, 512), (40, 1003), (1030, 10), (3, 16, 1024), (2, 640, 32), (31, 30), (61, 513), (1, 1), (4097, 2)]
    made = [init(s, 300 + i, param, grad, state) for i, s in enumerate(shapes)]
    ps, gs, sts = ([v[k] for v in made] for k in range(3))
    before = [(to64(p), g.float().cpu().numpy(), momentum_of(st)) for p, g, st in made]
    kw = dict(lr=0.05, weight_decay=0.1, adjust_lr="match_rms_adamw")
    muon_step(ps, gs, sts, momentum=0.9, **kw)
    for p, st, (p0, g, m0) in zip(ps, sts, before):
        check_step(p, st, p0, g, m0, str(state).split(".")[1], momentum_=0.9, **kw)


@pytest.mark.parametrize("kind", ["noise", "entry", "decades"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, torch.int8])
def test_step_of_few_rows_keeps_22_bits(state, nesterov, kind):
    """On parameters of zeros without decay, so that what is stored is the update, rounded by 2^-22 of it at most
    (the product with lr s, the store)."""
    kw = dict(lr=0.5, weight_decay=0.0, nesterov=nesterov, adjust_lr="match_rms_adamw")
    for i, shape in enumerate(((16, 16), (40, 64), (64, 30), (16, 1024), (1100, 20), (60, 700))):
        p, g, st = init(shape, 320 + i, torch.float32, torch.float32, state)
        if kind != "noise":
            g = scaled(shape, 330 + i, kind)
            st = {k: torch.zeros_like(v) for k, v in st.items()}
        p.zero_()
        m0 = momentum_of(st)
        muon_step([p], [g], [st], momentum=0.9, **kw)
        m, _ = om.momentum(m0, g.cpu().numpy(), 0.9, str(state).split(".")[1])
        assert np.array_equal(momentum_of(st), m)
        u = om.direction(m, g.cpu().numpy(), 0.9, nesterov)
        want, c = om.newton_schulz(u), 0.5 * om.shape_scale("match_rms_adamw", *shape)
        lim = few_slack(u) + 2.0 ** -22 * np.linalg.norm(want)
        assert np.linalg.norm(to64(p) + c * want) <= c * lim, (shape, np.linalg.norm(to64(p) + c * want) / c, lim)


@pytest.mark.parametrize("shape", [(16, 77), (77, 16), (30, 1203), (1203, 30)])
def test_unaligned_tensors_of_few_rows(shape):
    for param, grad, state in ((F, B, F), (B, F, B), (F, F, I)):
        p, g, st = init(shape, 108, param, grad, state)
        t = {}
        for name, v in (("p", p), ("g", g), ("m", st["exp_avg"])):
            buf = torch.full((v.numel() + 2,), 3, dtype=v.dtype, device=DEV)
            buf[1:-1] = v.view(-1)
            t[name] = (buf, buf[1:-1].view(shape))
        p0, m0 = to64(p), momentum_of(st)
        new = dict(st, exp_avg=t["m"][1])
        muon_step([t["p"][1]], [t["g"][1]], [new], lr=0.1)
        check_step(t["p"][1], new, p0, g.float().cpu().numpy(), m0, str(state).split(".")[1], lr=0.1)
        assert all(b[0] == 3 and b[-1] == 3 for b, _ in t.values())


def test_8_bit_momentum_groups():
    """Groups that cross rows, a short last one, unaligned codes, a group of zeros and one with an infinity."""
    p, g, st = init((37, 131), 40, F, F, I)
    g.view(-1)[128:256] = 0.0
    st["exp_avg"].view(-1)[128:256] = 0
    whole = torch.zeros(37 * 131 + 3, dtype=torch.int8, device=DEV)
    whole[3:] = st["exp_avg"].view(-1)
    st["exp_avg"] = whole[3:].view(37, 131)
    p0, m0 = to64(p), momentum_of(st)
    muon_step([p], [g], [st], lr=0.1)
    check_step(p, st, p0, g.cpu().numpy(), m0, "int8", lr=0.1)
    assert (st["exp_avg_scale"][1] == 0).all()
    g[0, 0] = math.inf
    p0, m0 = to64(p), momentum_of(st)
    muon_step([p], [g], [st], lr=0.1)
    new, q = om.momentum(m0, g.cpu().numpy(), 0.95, "int8")
    assert np.array_equal(st["exp_avg"].cpu().numpy(), q[0]) and st["exp_avg_scale"][0].isnan() and st["exp_avg_scale"][2].isfinite()
    assert p.isnan().all()


def test_zero_gradient_and_lr():
    p, g, st = init((50, 70), 41, F, F, F)
    st["exp_avg"].zero_()
    g.zero_()
    p0 = p.clone()
    muon_step([p], [g], [st], lr=0.5, weight_decay=0.25)  # only the decay
    assert torch.equal(p, p0 * np.float32(1 - 0.5 * 0.25))
    p, g, st = init((50, 70), 42, B, B, B)
    p0 = p.clone()
    muon_step([p], [g], [st], lr=0.0)
    assert torch.equal(p, p0)


def test_unaligned_tensors():
    """Views one element off 16 bytes, as flat parameter buffers hold them."""
    for param, grad, state in ((F, B, F), (B, F, B)):
        p, g, st = init((60, 77), 43, param, grad, state)
        t = {}
        for name, v in (("p", p), ("g", g), ("m", st["exp_avg"])):
            buf = torch.full((v.numel() + 2,), 3.0, dtype=v.dtype, device=DEV)
            buf[1:-1] = v.view(-1)
            t[name] = (buf, buf[1:-1].view(60, 77))
        p0, m0 = to64(p), momentum_of(st)
        muon_step([t["p"][1]], [t["g"][1]], [dict(exp_avg=t["m"][1])], lr=0.1)
        check_step(t["p"][1], dict(exp_avg=t["m"][1]), p0, g.float().cpu().numpy(), m0, str(state).split(".")[1], lr=0.1)
        assert all(b[0] == 3.0 and b[-1] == 3.0 for b, _ in t.values())


def test_step_does_not_depend_on_its_list():
    made = [init(s, 50 + i, F, B, F) for i, s in enumerate(MIXED)]
    alone = [init(s, 50 + i, F, B, F) for i, s in enumerate(MIXED)]
    muon_step(*([v[k] for v in made] for k in range(3)), lr=0.1)
    for p, g, st in alone:
        muon_step([p], [g], [st], lr=0.1)
    for a, b in zip(made, alone):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2]["exp_avg"], b[2]["exp_avg"])


# ------------------------------------------------------------------------------ streams, graphs, refusals

def test_another_stream():
    x = matrix((300, 520), 60)
    want = orthogonalize(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x2 = x * 1.0
        got = orthogonalize(x2)
    s.synchronize()
    assert torch.equal(got, want)


def test_two_streams_at_once():
    xs = [matrix((700, 900), 61), matrix((800, 650), 62)]
    want = [orthogonalize(x) for x in xs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x in zip(ss, xs):
        with torch.cuda.stream(s):
            got.append([orthogonalize(x) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)


def test_captured_and_replayed():
    """A graph of a list's orthogonalization and a Muon step, replayed between eager work; the
    call needs no earlier one."""
    shapes = [(300, 520), (64, 64), (16, 4096), (3, 65, 40)]
    made, eager = ([init(s, 70 + i, F, B, F) for i, s in enumerate(shapes)] for _ in range(2))
    xs = [matrix(s, 80 + i) for i, s in enumerate(shapes)]
    outs = [torch.empty(s, dtype=B, device=DEV) for s in shapes]
    hp = _lib.muon_hparams(lr=0.1)
    args = [[v[k] for v in made] for k in range(3)]
    ws = _lib.workspace(_lib.meo_muon_workspace_size(hp, *args), DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orthogonalize(xs, out=outs)
        _lib.meo_muon_step(hp, 1, *args, ws)
    for i in range(4):
        for x in xs:
            x.mul_(-0.5).add_(0.01)
        for a, b in zip(made, eager):
            b[1].copy_(a[1].mul_(-1.25))
        graph.replay()
        muon_step(*([v[k] for v in eager] for k in range(3)), lr=0.1)
        want = orthogonalize(xs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for a, b in zip(made, eager):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2]["exp_avg"], b[2]["exp_avg"])


def test_few_rows_captured_and_replayed():
    shapes = [(40, 50), (20, 1500), (2, 1500, 60), (16, 16), (60, 400)]
    made, eager = ([init(s, 110 + i, F, B, I if i % 2 else F) for i, s in enumerate(shapes)] for _ in range(2))
    hp = _lib.muon_hparams(lr=0.1)
    args = [[v[k] for v in made] for k in range(3)]
    ws = _lib.workspace(_lib.meo_muon_workspace_size(hp, *args), DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.meo_muon_step(hp, 1, *args, ws)
    for i in range(4):
        for a, b in zip(made, eager):
            b[1].copy_(a[1].mul_(-1.25))
        graph.replay()
        muon_step(*([v[k] for v in eager] for k in range(3)), lr=0.1)
        torch.cuda.synchronize()
        for a, b in zip(made, eager):
            assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


def test_memory_refusals():
    hp = _lib.muon_hparams()
    p, g, st = init((64, 64), 90, F, F, F)
    need = _lib.meo_muon_workspace_size(hp, [p], [g], [st])
    p0, m0 = p.clone(), st["exp_avg"].clone()
    for ws, code in ((None, _lib.MEO_EWORKSPACE), (torch.empty(need - 1, dtype=torch.uint8, device=DEV), _lib.MEO_EWORKSPACE),
                     (torch.empty(need + 512, dtype=torch.uint8, device=DEV)[128:], _lib.MEO_EWORKSPACE)):
        with pytest.raises(MeoError) as e:
            _lib.meo_muon_step(hp, 1, [p], [g], [st], ws)
        assert e.value.code == code
    ws = _lib.workspace(need, DEV)
    for bad in ((p.cpu(), g, st), (p, g.cpu(), st), (p, g, dict(exp_avg=st["exp_avg"].cpu()))):
        with pytest.raises(MeoError) as e:
            _lib.meo_muon_step(hp, 1, [bad[0]], [bad[1]], [bad[2]], ws)
        assert e.value.code == _lib.MEO_EMEMORY
    h, x, o = _lib.orthogonalize_hparams(), matrix((64, 64), 91), torch.empty(64, 64, dtype=B, device=DEV)
    arr = (_lib.meo_ns_matrices * 1)(_lib.meo_ns_matrices(x.data_ptr(), o.data_ptr(), 2 ** 20, 64, 64, 64, 64, _lib.MEO_F32, 0))
    big = _lib.workspace(_lib.load().meo_orthogonalize_workspace_size(h, 1, arr), DEV)
    assert _lib.load().meo_orthogonalize(h, 1, arr, big.data_ptr(), big.numel(), None) == _lib.MEO_EMEMORY  # past its memory
    torch.cuda.synchronize()
    assert torch.equal(p, p0) and torch.equal(st["exp_avg"], m0)


def test_profile_names_the_passes():
    _lib.meo_profile_enable(True)
    try:
        orthogonalize([matrix((96, 128), 92), matrix((64, 64), 92), matrix((20, 10), 92)])
        got = _lib.meo_profile_collect()
    finally:
        _lib.meo_profile_enable(False)
    assert got["ns_gram"]["launches"] == got["ns_apply"]["launches"] == 5 and got["muon_scatter"]["launches"] == 1
    assert got["ns_whole"]["launches"] == 2  # (of 16 and of 64 rows)


# ------------------------------------------------------------------------------ Muon (front end)

def _model(seed, dtype=F):
    torch.manual_seed(seed)
    return torch.nn.Sequential(torch.nn.Linear(64, 160), torch.nn.GELU(), torch.nn.Linear(160, 96)).to(DEV).to(dtype)


@pytest.mark.parametrize("dtype,state", [(F, None), (F, I), (B, None)])
def test_muon_over_a_model(dtype, state):
    """Matrices against the oracle's Muon, biases and a group with muon=False against its AdamW."""
    m = _model(1, dtype)
    opt = Muon([dict(params=[m[0].weight, m[0].bias], lr=0.02), dict(params=[m[2].weight, m[2].bias], muon=False, lr=1e-2)],
               weight_decay=0.01, state_dtype=state)
    x = torch.randn(32, 64, generator=torch.Generator().manual_seed(2)).to(DEV).to(dtype)
    adam = {p: (np.zeros(p.numel()), np.zeros(p.numel())) for p in m.parameters()}
    for step in range(1, 4):
        opt.zero_grad()
        m(x).float().square().mean().backward()
        before = {p: (to64(p), p.grad.float().cpu().numpy()) for p in m.parameters()}
        w = m[0].weight
        m0 = momentum_of(opt.state[w]) if opt.state[w] else np.zeros(w.shape, np.float32)
        opt.step()
        torch.cuda.synchronize()
        kind = "int8" if state == I else str(dtype).split(".")[1]
        check_step(w, opt.state[w], before[w][0], before[w][1], m0, kind, lr=0.02, weight_decay=0.01)
        assert opt.state[w]["step"] == step
        for p in (m[0].bias, m[2].weight, m[2].bias):
            p0, g = before[p]
            lr = 0.02 if p is m[0].bias else 1e-2
            ea, es = adam[p]
            g = g.reshape(-1).astype(np.float64)
            ea, es = 0.9 * ea + 0.1 * g, 0.999 * es + 0.001 * g * g
            adam[p] = (ea, es)
            n = (ea / (1 - 0.9 ** step)) / (np.sqrt(es / (1 - 0.999 ** step)) + 1e-8)
            want = p0.reshape(-1) * (1 - lr * 0.01) - lr * n
            half = 2.0 ** -8 if dtype == B else 2.0 ** -22
            assert np.all(np.abs(to64(p).reshape(-1) - want) <= half * np.abs(want) + 1e-4 * lr)
            assert set(opt.state[p]) == {"step", "exp_avg", "exp_avg_sq"}


def test_muon_state_dict_and_together():
    """State dicts carry on where they were taken; orthogonalize is the step's direction."""
    ms = [_model(3), _model(3)]
    opts = [Muon(m.parameters(), lr=0.02, state_dtype=I) for m in ms]
    x = torch.randn(32, 64, generator=torch.Generator().manual_seed(4)).to(DEV)

    def step(k):
        opts[k].zero_grad()
        ms[k](x).square().mean().backward()
        opts[k].step()

    step(0)
    ms[1].load_state_dict(ms[0].state_dict())
    opts[1].load_state_dict(opts[0].state_dict())
    for _ in range(2):
        step(0), step(1)
    assert all(torch.equal(a, b) for a, b in zip(ms[0].parameters(), ms[1].parameters()))
    w = torch.nn.Parameter(matrix((96, 160), 5))
    w.grad = matrix((96, 160), 6)
    opt = Muon([w], lr=0.1, momentum=0.0, weight_decay=0.0)
    w0 = w.detach().clone()
    opt.step()
    o = orthogonalize(w.grad)
    assert ((w0 - w.detach()) / 0.1 - o.float()).abs().max() <= 2.0 ** -8 * o.abs().max() + 2.0 ** -22 * w0.abs().max() / 0.1


def test_muon_listed_twice_and_missing_gradients():
    a, b = (torch.nn.Parameter(matrix((40, 60), 7)) for _ in range(2))
    opt, twice = Muon([a], lr=0.1), Muon([dict(params=[b])], lr=0.1)
    twice.param_groups[0]["params"].append(b)
    c = torch.nn.Parameter(torch.zeros(3, 3, device=DEV))
    twice.param_groups[0]["params"].append(c)
    a.grad, b.grad = matrix((40, 60), 8), matrix((40, 60), 8)
    opt.step(), opt.step(), twice.step()
    assert torch.equal(a, b) and twice.state[b]["step"] == 2 and not twice.state[c]


def test_refused_step_changes_nothing():
    w = torch.nn.Parameter(matrix((40, 60), 9))
    b = torch.nn.Parameter(torch.zeros(7, device=DEV))
    opt = Muon([w, b], lr=0.1)
    w.grad, b.grad = torch.ones_like(w), torch.ones_like(b)
    opt.step()
    w0, b0 = w.detach().clone(), b.detach().clone()
    opt.param_groups[0]["betas"] = (1.5, 0.9)  # of the AdamW part
    with pytest.raises(MeoError):
        opt.step()
    torch.cuda.synchronize()
    assert torch.equal(w, w0) and torch.equal(b, b0) and opt.state[w]["step"] == 1 and opt.state[b]["step"] == 1
    opt.param_groups[0].update(betas=(0.9, 0.999), momentum=2.0)
    with pytest.raises(MeoError):
        opt.step()
    assert torch.equal(w, w0) and torch.equal(b, b0)


def test_galore_oracle_is_the_adamw_of_other_parameters():
    """(The AdamW formula of test_muon_over_a_model is the one oracle/galore.py has.)"""
    x, g = np.array([0.5, -1.0]), np.array([0.1, 0.2])
    st = {"exp_avg": np.zeros(2), "exp_avg_sq": np.zeros(2)}
    want, _ = ga.galore_step_tensor(x, g, st, dict(lr=0.1, weight_decay=0.01, rank=4), 1)
    n = g / (np.sqrt(g * g) + 1e-8)
    assert np.allclose(want, x * (1 - 0.1 * 0.01) - 0.1 * n, rtol=1e-9)
