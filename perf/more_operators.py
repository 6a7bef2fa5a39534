"""Muon's operators in their plain form, the cases they are measured on, and the
library's calls for the same work.

Two operators:

* orthogonalize  matrices X (their leading dims a batch) moved towards the nearest
                 matrices with orthonormal rows or columns by Newton-Schulz steps:
                 X0 = X / max(|X|, eps), then X <- a X + (b A + c A^2) X with A = X X^T
                 (the shorter side as rows); bfloat16 results;
* step           Muon: momentum m <- beta m + (1 - beta) g, direction m or, with Nesterov,
                 (1 - beta) g + beta m, orthogonalized, then
                 x <- x (1 - lr wd) - lr s O with s by the matrix' shape.

With ``own`` false, ``run`` computes them with elementary torch operations in float32.
"""
import math

import torch

own = False

_F32, _BF16, _I8 = "float32", "bfloat16", "int8"
_COEF = (3.4445, -4.7750, 2.0315)
_EPS = 1e-7
_LR, _WD, _BETA = 1e-4, 0.1, 0.95
_STEP = 5  # 1-based index of the timed step


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one small hidden matrix: launch latency
        dict(name="ortho_small", op="ortho", shapes="32x64", dtype=_F32, layout="rows", steps=5),
        # the two factors of four rank-16 adapters of a 4096-wide projection: few rows, a long axis
        dict(name="ortho_adapters", op="ortho", layout="rows", dtype=_BF16, steps=5,
             shapes="16x4096,4096x16,16x4096,4096x16,16x4096,4096x16,16x4096,4096x16"),
        # odd sizes, column-major, one step more
        dict(name="ortho_ragged", op="ortho", shapes="1003x777", dtype=_F32, layout="columns", steps=6),
        # an attention matrix of Llama-7B, and one of its MLP's (tall)
        dict(name="ortho_attention", op="ortho", shapes="4096x4096", dtype=_BF16, layout="rows", steps=5),
        dict(name="ortho_mlp", op="ortho", shapes="11008x4096", dtype=_F32, layout="rows", steps=5),
        # the smallest configuration's matrix
        dict(name="step_small", op="step", shapes="256x512", param=_F32, grad=_F32, state=_F32,
             nesterov=True, scale="original"),
        # a stack of experts (3-D parameters), 16-bit storage
        dict(name="step_experts", op="step", shapes="8x256x688,8x256x688,8x688x256", param=_BF16, grad=_BF16,
             state=_BF16, nesterov=True, scale="match_rms_adamw"),
        # odd sizes, 8-bit momentum whose groups cross rows
        dict(name="step_ragged", op="step", shapes="777x1001,130x2050,1x513", param=_F32, grad=_BF16, state=_I8,
             nesterov=False, scale="original"),
        # the matrices of a BERT-large layer
        dict(name="step_bert", op="step", shapes="1024x1024,1024x1024,1024x1024,1024x1024,4096x1024,1024x4096",
             param=_F32, grad=_F32, state=_F32, nesterov=True, scale="match_rms_adamw"),
        # the attention matrices of a Llama-7B layer, 8-bit momentum
        dict(name="step_attention", op="step", shapes="4096x4096,4096x4096,4096x4096,4096x4096", param=_F32,
             grad=_BF16, state=_I8, nesterov=True, scale="match_rms_adamw"),
        # all matrices of the layer, 16-bit storage: the largest
        dict(name="step_layer", op="step", param=_BF16, grad=_BF16, state=_BF16, nesterov=True,
             scale="match_rms_adamw",
             shapes="4096x4096,4096x4096,4096x4096,4096x4096,11008x4096,11008x4096,4096x11008"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    shapes = []
    for _ in range(rng.randint(1, 3)):
        a = _log(rng, 1, 4096)  # the shorter side
        b = _log(rng, a, max(a, min(16384, 24_000_000 // a)))
        if rng.random() < 0.5:  # whole tiles, as most models have
            a, b = min(4096, (a + 63) // 64 * 64), (b + 63) // 64 * 64
        shape = (a, b) if rng.random() < 0.5 else (b, a)
        batch = rng.choice([1, 1, 1, rng.randint(2, 6)])
        shapes.append("x".join(str(v) for v in (shape if batch == 1 or a * b > 4_000_000 else (batch, *shape))))
    shapes = ",".join(shapes)
    if rng.random() < 0.5:
        return dict(op="ortho", shapes=shapes, dtype=rng.choice([_F32, _BF16]),
                    layout=rng.choice(["rows", "rows", "columns"]), steps=rng.randint(1, 6))
    return dict(op="step", shapes=shapes, param=rng.choice([_F32, _BF16]), grad=rng.choice([_F32, _BF16]),
                state=rng.choice([_F32, _BF16, _I8]), nesterov=rng.random() < 0.5,
                scale=rng.choice(["original", "match_rms_adamw"]))


# ------------------------------------------------------------------------------- plain form

def _plain_ortho(x, steps):
    """X [..., m, n] float32 -> float32."""
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1) if tall else x
    a, b, c = _COEF
    norm = torch.sqrt((x.double() * x.double()).sum(dim=(-2, -1), keepdim=True))  # squares of 1e-30 as of 1e30
    x = (x / norm.clamp(min=_EPS)).float().contiguous()
    for _ in range(steps):
        g = x @ x.transpose(-2, -1).contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(-2, -1) if tall else x


def _scale(case, shape):
    r, c = shape[-2], shape[-1]
    return math.sqrt(max(1.0, r / c)) if case["scale"] == "original" else 0.2 * math.sqrt(max(r, c))


def _plain_quantize(m):
    """Groups of 128 consecutive values: int8 codes and one scale max|m| / 127 per group."""
    n = m.numel()
    v = torch.zeros((n + 127) // 128 * 128, dtype=torch.float32, device=m.device)
    v[:n] = m.reshape(-1)
    v = v.view(-1, 128)
    scale = v.abs().amax(dim=1) / 127
    q = torch.round(v / torch.where(scale > 0, scale, 1.0).unsqueeze(1)).clamp(-128, 127)
    return q.to(torch.int8).view(-1)[:n].view(m.shape), scale


def _plain_dequantize(codes, scale):
    s = scale.repeat_interleave(128)[: codes.numel()]
    return (codes.reshape(-1).float() * s).view(codes.shape)


def _plain_step(case, p, g, st):
    """In place: the momentum and the parameter."""
    m = _plain_dequantize(st["exp_avg"], st["exp_avg_scale"]) if case["state"] == _I8 else st["exp_avg"].float()
    g = g.float() * (1 - _BETA)
    m = m * _BETA + g
    if case["state"] == _I8:
        codes, scale = _plain_quantize(m)
        st["exp_avg"].copy_(codes)
        st["exp_avg_scale"].copy_(scale)
        m = _plain_dequantize(codes, scale)
    else:
        m = st["exp_avg"].copy_(m).float()
    o = _plain_ortho(g + m * _BETA if case["nesterov"] else m, 5)
    p.copy_(p.float() * (1 - _LR * _WD) - (_LR * _scale(case, p.shape)) * o)


# ------------------------------------------------------------------------------- states

def _dtype(name):
    return {_F32: torch.float32, _BF16: torch.bfloat16, _I8: torch.int8}[name]


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _gradient(shape, gen):
    """Entries around 1e-3: a few strong directions, rows of very different size, noise."""
    *batch, m, n = shape
    k = min(8, m, n)
    a = torch.randn(*batch, m, k, generator=gen, device="cuda")
    b = torch.randn(*batch, k, n, generator=gen, device="cuda")
    row = torch.exp(0.5 * torch.randn(*batch, m, 1, generator=gen, device="cuda"))
    return ((a @ b) * (1e-3 / math.sqrt(k)) + 1e-3 * torch.randn(shape, generator=gen, device="cuda")) * row


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "ortho":
        xs = []
        for shape in _shapes(case):
            x = _gradient(shape, gen).to(_dtype(case["dtype"]))
            if shape[-2] > 8:
                x[..., 3, :] = 0.0  # a unit that took no part
            if len(shape) > 2:
                x[1] = 0.0  # an expert that no token reached
            xs.append(x.transpose(-2, -1).contiguous().transpose(-2, -1) if case["layout"] == "columns" else x)
        return dict(case=case, xs=xs)
    params, grads, states = [], [], []
    for shape in _shapes(case):
        params.append((0.02 * torch.randn(shape, generator=gen, device="cuda")).to(_dtype(case["param"])))
        g = _gradient(shape, gen)
        m = 0.5 * _gradient(shape, gen) + 0.3 * g
        if len(shape) > 2:
            g[1] = 0.0  # an expert that no token reached in this step
        grads.append(g.to(_dtype(case["grad"])))
        if case["state"] == _I8:
            codes, scale = _plain_quantize(m)
            states.append(dict(exp_avg=codes, exp_avg_scale=scale))
        else:
            states.append(dict(exp_avg=m.to(_dtype(case["state"]))))
    # the workspace is the library's, made at its first step and kept, as a training loop does
    return dict(case=case, params=params, grads=grads, states=states, workspace=None)


# ------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["op"] == "ortho":
        if own:
            from memory_efficient_optimizers_amd import orthogonalize
            return orthogonalize(state["xs"], steps=case["steps"])
        return [_plain_ortho(x.float(), case["steps"]).to(torch.bfloat16) for x in state["xs"]]
    if own:
        from memory_efficient_optimizers_amd import _lib
        hp = _lib.muon_hparams(lr=_LR, weight_decay=_WD, momentum=_BETA, nesterov=case["nesterov"],
                               adjust_lr=case["scale"])
        if state["workspace"] is None:
            nbytes = _lib.meo_muon_workspace_size(hp, state["params"], state["grads"], state["states"])
            state["workspace"] = _lib.workspace(nbytes, "cuda")
        _lib.meo_muon_step(hp, _STEP, state["params"], state["grads"], state["states"], state["workspace"])
    else:
        for p, g, st in zip(state["params"], state["grads"], state["states"]):
            _plain_step(case, p, g, st)
    if case["state"] == _I8:  # the values that the codes stand for
        return [[p, st["exp_avg"].float().view(-1), st["exp_avg_scale"]]
                for p, st in zip(state["params"], state["states"])]
    return [[p, st["exp_avg"]] for p, st in zip(state["params"], state["states"])]


def work(case):
    size = {_F32: 4.0, _BF16: 2.0, _I8: 1.0 + 4.0 / 128}
    total, flops = 0.0, 0.0
    for shape in _shapes(case):
        batch = shape[0] if len(shape) > 2 else 1
        m, n = min(shape[-2:]), max(shape[-2:])
        # a symmetric product needs half of its entries; the linear term and the norm are of lower order
        flops += case.get("steps", 5) * batch * (3.0 * m * m * n + 1.0 * m * m * m)
        if case["op"] == "ortho":
            total += batch * m * n * (size[case["dtype"]] + 2.0)
        else:
            total += batch * m * n * (2 * size[case["param"]] + size[case["grad"]] + 2 * size[case["state"]])
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------------------- 64 bits

def _exact_ortho(x, steps):
    """In the polynomial's own terms: every iterate is P X0 with P a polynomial of S = X0 X0^T,
    whose Gram matrix is P S P; all of them commute."""
    x = x.double()
    if x.shape[-2] > x.shape[-1]:
        return _exact_ortho(x.transpose(-2, -1), steps).transpose(-2, -1)
    x = x / torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True).clamp_min(_EPS)
    x = x.contiguous()
    s = torch.matmul(x, x.transpose(-2, -1).contiguous())
    one = torch.eye(x.shape[-2], dtype=torch.float64, device=x.device).expand_as(s)
    p = one
    for _ in range(steps):
        q = _COEF[0] * one + torch.matmul(s, _COEF[1] * one + _COEF[2] * s)
        p, s = torch.matmul(q, p), torch.matmul(torch.matmul(q, s), q)
    return torch.matmul(p, x)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "ortho":
        return [_exact_ortho(x, case["steps"]) for x in state["xs"]]
    out = []
    for p, g, st in zip(state["params"], state["grads"], state["states"]):
        m, g = st["exp_avg"].double(), g.double()
        if case["state"] == _I8:
            group = torch.arange(m.numel(), device=m.device).div(128, rounding_mode="floor")
            m = m * st["exp_avg_scale"].double()[group].view(m.shape)
        m = _BETA * m + (1.0 - _BETA) * g
        stored = m
        if case["state"] == _I8:
            top = torch.zeros_like(st["exp_avg_scale"], dtype=torch.float64)
            top.scatter_reduce_(0, group, m.abs().reshape(-1), "amax")
            unit = top[group].view(m.shape) / 127.0
            codes = torch.where(unit > 0, (m / unit).round(), 0.0)
            stored, m = None, codes * unit  # a code next to a border may go either way
        elif case["state"] == _BF16:
            m = m.to(torch.bfloat16).double()  # the stored value is what the step uses
        u = (1.0 - _BETA) * g + _BETA * m if case["nesterov"] else m
        x = p.double() * (1.0 - _LR * _WD) - _LR * _scale(case, p.shape) * _exact_ortho(u, 5)
        if case["state"] == _I8:
            out.append([x, None, top / 127.0])
        else:
            out.append([x, stored])
    return out
