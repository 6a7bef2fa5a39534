"""Launch tables of cached lists: those of a captured call outlive any number of other lists,
and calls of several threads over more lists than are cached use none that is freed."""
import threading

import pytest
import torch

import workloads
from memory_efficient_optimizers_amd import _lib, mx4_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Step:
    """One optimizer's step over a list of its own; equal seeds hold equal values."""

    def __init__(self, kind, seed, shapes=((96, 64), (64, 160), (40,))):
        shapes = list(shapes)
        if kind == "adafactor":
            gen = torch.Generator().manual_seed(seed)
            self.params = [torch.randn(s, generator=gen).to(DEV) for s in shapes]
            self.grads = [torch.randn(s, generator=gen).to(DEV) for s in shapes]
            self.states = [_lib.init_state("adafactor", p, beta1=True) for p in self.params]
            self.hp = _lib.adafactor_hparams(beta1=0.9)
            size, self.fn = _lib.meo_adafactor_workspace_size(self.params, self.grads), _lib.meo_adafactor_step
        else:
            self.params, self.grads, self.states = workloads.galore_inputs(shapes, 16, seed, device=DEV)
            self.hp = _lib.galore_hparams(lr=0.05, rank=16)
            size, self.fn = _lib.meo_galore_workspace_size(self.hp, self.params, self.grads), _lib.meo_galore_step
            if kind == "galore_mx4":
                for st in self.states:
                    if "projector_t" in st:
                        q = mx4_quantize(st.pop("projector_t"))
                        st["projector"], st["projector_scale"] = q.codes, q.scales
                size, self.fn = (_lib.meo_galore_mx4_workspace_size(self.hp, self.params, self.grads),
                                 _lib.meo_galore_mx4_step)
        self.ws = _lib.workspace(size, DEV)

    def step(self, t):
        self.fn(self.hp, t, self.params, self.grads, self.states, self.ws)

    def values(self):
        return self.params + [v for st in self.states for v in st.values() if torch.is_tensor(v)]


KINDS = ["adafactor", "galore", "galore_mx4"]


@pytest.mark.parametrize("kind", KINDS)
def test_a_captured_step_keeps_its_tables(kind):
    """Captured, then 70 other lists (64 are cached), then replayed between eager steps of a twin."""
    a, b = Step(kind, 1), Step(kind, 1)
    a.step(2)
    b.step(2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(2)
    others = [Step(kind, 100 + i, [(8 + i, 16 + i)]) for i in range(70)]
    for o in others:
        o.step(2)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        b.step(2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.values(), b.values()))
        others[0].step(2)


@pytest.mark.parametrize("kind", KINDS)
def test_threads_over_more_lists_than_are_cached(kind):
    """Four threads, 40 lists each, on streams of their own: as the same steps one after the other."""
    lists = [[Step(kind, 1000 + 50 * w + i, [(8 + i, 24 + w)]) for i in range(40)] for w in range(4)]
    streams = [torch.cuda.Stream() for _ in lists]
    torch.cuda.synchronize()
    errors = []

    def work(w):
        try:
            with torch.cuda.stream(streams[w]):
                for t in (2, 3):
                    for s in lists[w]:
                        s.step(t)
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(w,)) for w in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for w, mine in enumerate(lists):
        for i, s in enumerate(mine):
            twin = Step(kind, 1000 + 50 * w + i, [(8 + i, 24 + w)])
            for t in (2, 3):
                twin.step(t)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(s.values(), twin.values()))
