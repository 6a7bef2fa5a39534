"""The optimizer front ends on the host (no GPU): which steps are counted, with the library's
call replaced."""
import contextlib

import pytest
import torch

from memory_efficient_optimizers_amd import CAME, Adafactor, GaLoreAdamW, Lamb, MX4Tensor, _lib, optim

MX4 = torch.float4_e2m1fn_x2


@pytest.fixture
def host(monkeypatch):
    """Steps of CPU parameters reach `_call`, which records them and refuses what is in `refuse`."""
    calls, refuse = [], set()
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    for cls in (Adafactor, CAME, Lamb, GaLoreAdamW):
        def call(self, group, step, params, grads, states, ws):
            if any(p in refuse for p in params):
                raise RuntimeError("refused")
            calls.append((step, list(params), list(grads)))
        monkeypatch.setattr(cls, "_call", call)
        monkeypatch.setattr(cls, "_wsize", lambda self, params, grads: 0)
    return calls, refuse


def _params(n):
    ps = [torch.nn.Parameter(torch.zeros(8, 8)) for _ in range(n)]
    for p in ps:
        p.grad = torch.ones(8, 8)
    return ps


@pytest.mark.parametrize("make", [lambda g: Adafactor(g), lambda g: CAME(g, lr=1e-3), lambda g: Lamb(g), lambda g: GaLoreAdamW(g),
                                  lambda g: GaLoreAdamW(g, projector_dtype=MX4)])
def test_a_refused_call_counts_for_none_of_its_parameters(host, make):
    calls, refuse = host
    a, b, c = _params(3)
    opt = make([dict(params=[a]), dict(params=[b, c])])
    opt.step()
    refuse.add(c)
    for _ in range(2):
        with pytest.raises(RuntimeError):
            opt.step()
    assert [opt.state[p]["step"] for p in (a, b, c)] == [3, 1, 1]
    refuse.clear()
    opt.step()
    assert [opt.state[p]["step"] for p in (a, b, c)] == [4, 2, 2]
    assert [step for step, _, _ in calls] == [1, 1, 2, 3, 4, 2]


def test_a_state_that_could_not_be_made_is_made_again(host, monkeypatch):
    (p,) = _params(1)
    opt = Lamb([p])
    make = Lamb._state_for
    monkeypatch.setattr(Lamb, "_state_for", lambda *a: (_ for _ in ()).throw(MemoryError()))
    with pytest.raises(MemoryError):
        opt.step()
    monkeypatch.setattr(Lamb, "_state_for", make)
    opt.step()
    assert opt.state[p]["step"] == 1 and "exp_avg" in opt.state[p]


def test_a_parameter_listed_twice_takes_two_steps(host):
    calls, _ = host
    (p,) = _params(1)
    with pytest.warns(UserWarning):
        opt = Lamb([p, p])
    opt.step()
    assert opt.state[p]["step"] == 2 and [(s, len(ps)) for s, ps, _ in calls] == [(1, 1), (2, 1)]


def test_compressed_gradients_are_used_by_the_step_that_is_taken(host, monkeypatch):
    """One is dropped as soon as its group's call has been taken, and kept by one that was refused."""
    calls, refuse = host
    made = []

    def quantize(x, transposed=False):
        made.append(MX4Tensor.empty(*x.shape, "cpu"))
        return made[-1]

    monkeypatch.setattr(optim, "mx4_quantize", quantize)
    a, b = _params(2)
    opt = GaLoreAdamW([dict(params=[a], rank=4), dict(params=[b], rank=4)], projector_dtype=MX4)
    opt.step()
    for p in (a, b):
        p.grad = torch.ones(8, 8)
        opt.compress_grad(p)
    assert a.grad is None and b.grad is None
    refuse.add(b)
    with pytest.raises(RuntimeError):
        opt.step()
    refuse.clear()
    opt.step()  # a's gradient was used; b's waits for its step
    assert [opt.state[p]["step"] for p in (a, b)] == [2, 2]
    assert [(s, ps, gs) for s, ps, gs in calls[2:]] == [(2, [a], [made[0]]), (2, [b], [made[1]])]
    opt.step()
    assert len(calls) == 4


def test_only_the_optimizer_discards_compressed_gradients(host, monkeypatch):
    calls, _ = host
    monkeypatch.setattr(optim, "mx4_quantize", lambda x, transposed=False: MX4Tensor.empty(*x.shape, "cpu"))
    m = torch.nn.Linear(8, 8, bias=False)
    opt = GaLoreAdamW([dict(params=[m.weight], rank=4)], projector_dtype=MX4)
    m.weight.register_post_accumulate_grad_hook(opt.compress_grad)
    backward = lambda: m(torch.ones(2, 8)).sum().backward()  # noqa: E731
    backward()
    opt.step()  # refreshes: took the whole gradient
    m.zero_grad()
    backward()
    m.zero_grad()
    with pytest.raises(RuntimeError, match="already compressed"):
        backward()
    opt.zero_grad()
    opt.step()
    assert len(calls) == 1  # discarded: nothing to step
    backward()
    opt.step()
    assert opt.state[m.weight]["step"] == 2 and isinstance(calls[1][2][0], MX4Tensor)


def test_a_torch_without_the_4_bit_type_keeps_bf16_projectors(monkeypatch):
    monkeypatch.delattr(torch, "float4_e2m1fn_x2")
    p = torch.nn.Parameter(torch.zeros(8, 8))
    GaLoreAdamW([dict(params=[p], rank=4)])
    for dt in (None, torch.float16):
        with pytest.raises(TypeError):
            GaLoreAdamW([dict(params=[p], rank=4)], projector_dtype=dt)


def test_the_current_stream_without_torchs_private_call(monkeypatch):
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 88 + d, raising=False)
    assert _lib._stream(None) == 88
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert _lib._stream(None) == 77


def test_compress_grad_finds_a_group_without_searching_them_all(host, monkeypatch):
    """One pass over the parameters serves all of them; changed groups are found again."""
    class Counted(list):
        passes = 0

        def __iter__(self):
            Counted.passes += 1
            return super().__iter__()

    monkeypatch.setattr(optim, "mx4_quantize", lambda x, transposed=False: MX4Tensor.empty(*x.shape, "cpu"))
    ps = _params(50)
    opt = GaLoreAdamW([dict(params=ps[:25], rank=4), dict(params=ps[25:], rank=4)], projector_dtype=MX4)
    opt.step()
    for g in opt.param_groups:
        g["params"] = Counted(g["params"])
    for p in ps:
        p.grad = torch.ones(8, 8)
        opt.compress_grad(p)
    assert len(opt._compressed) == 50 and Counted.passes <= 2
    opt.zero_grad()
    (q,) = _params(1)
    with pytest.raises(ValueError):
        opt.compress_grad(q)
    opt.add_param_group(dict(params=[q], rank=4, update_proj_gap=1, scale=0.25, proj_type="std"))
    ps[3].grad = torch.ones(8, 8)
    del opt.param_groups[0]["params"][3]
    opt.param_groups[2]["params"].append(ps[3])
    opt.compress_grad(q)
    opt.compress_grad(ps[3])
    assert q.grad is not None and ps[3].grad is not None  # a gap of 1: every step is due


def test_a_group_added_later_gets_the_projections_defaults(host, monkeypatch):
    monkeypatch.setattr(optim, "mx4_quantize", lambda x, transposed=False: MX4Tensor.empty(*x.shape, "cpu"))
    a, b = _params(2)
    opt = GaLoreAdamW([dict(params=[a], rank=4)], projector_dtype=MX4)
    with pytest.raises(ValueError):
        opt.add_param_group(dict(params=[b], rank=4, proj_type="both"))
    opt.add_param_group(dict(params=[b], rank=4))
    fields = {k: v for k, v in opt.param_groups[0].items() if k != "params"}
    assert {k: v for k, v in opt.param_groups[1].items() if k != "params"} == fields
    assert (fields["update_proj_gap"], fields["scale"], fields["proj_type"]) == (200, 0.25, "std")
    opt.step()
    b.grad = torch.ones(8, 8)
    opt.compress_grad(b)
    assert b.grad is None
