"""Dependent calls of the grouped and int8 operators back to back: on one stream
without a synchronisation between them, replayed from a graph, and on several
host threads' streams at once.  Every kernel is deterministic, so each result
equals, bit for bit, that of the same calls run one by one."""
import threading

import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc

pytestmark = pytest.mark.gpu


def normal(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype) * 0.1


class Chain:
    """Forward, its gradients added up twice, an update of the weights, the forward
    again over them (write after read), then the int8 product of the result; with
    odd widths on plain loads, few rows and many."""

    def __init__(self, rows, groups, width, hidden, seed):
        cuts = [rows * i * i // (groups * groups) for i in range(groups + 1)]  # ragged, the first one small
        self.offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        self.x, self.dy = normal((rows, width), seed), normal((rows, hidden), seed + 1)
        self.w0 = normal((groups, width, hidden), seed + 2)
        self.w, self.h, self.h2 = self.w0.clone(), torch.empty_like(self.dy), torch.empty_like(self.dy)
        self.dx, self.grad = torch.empty_like(self.x), torch.empty(self.w.shape, device="cuda")
        self.wq, self.ws = ttc.quantize_rows(normal((width, hidden), seed + 3))
        self.q, self.qs = torch.empty((rows, self.wq.stride(0)), dtype=torch.int8, device="cuda")[:, :hidden], \
            torch.empty(rows, device="cuda")
        self.out = torch.empty((rows, width), device="cuda")
        self.room = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

    def steps(self):
        yield lambda: self.w.copy_(self.w0)
        yield lambda: ttc.gemm_grouped(self.x, self.w, self.offsets, self.h, act="relu")
        yield lambda: ttc.gemm_grouped(self.dy, self.w.transpose(1, 2), self.offsets, self.dx)
        yield lambda: ttc.gemm_grouped_wgrad(self.x, self.dy, self.offsets, out=self.grad)
        yield lambda: ttc.gemm_grouped_wgrad(self.x, self.h, self.offsets, c=self.grad, out=self.grad, beta=1.0)
        yield lambda: ttc.gemm_grouped_wgrad(self.x, self.dy, self.offsets, c=self.w, out=self.w, alpha=-0.5, beta=1.0)
        yield lambda: ttc.gemm_grouped(self.x, self.w, self.offsets, self.h2, act="gelu_tanh")
        yield lambda: ttc.quantize_rows(self.h2, self.q, self.qs)
        yield lambda: ttc.gemm_i8_scaled(self.q, self.qs, self.wq, self.ws, self.out, workspace=self.room)

    def results(self):
        return [t.clone() for t in (self.h, self.dx, self.grad, self.w, self.h2, self.q, self.qs, self.out)]

    def one_by_one(self):
        for step in self.steps():
            step()
            torch.cuda.synchronize()
        return self.results()

    def at_once(self):
        for step in self.steps():
            step()


SHAPES = [(700, 3, 256, 520), (24, 4, 512, 256), (350, 5, 131, 257), (1300, 2, 1024, 2048)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("shape", SHAPES)
def test_back_to_back_and_from_a_graph(shape):
    c = Chain(*shape, seed=1)
    want = c.one_by_one()
    for _ in range(3):
        c.at_once()
    assert same(c.results(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.at_once()
        c.at_once()
    for t in (c.h, c.dx, c.grad, c.h2, c.out):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert same(c.results(), want)
    assert ttc.ttc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0


def test_threads_on_their_own_streams():
    chains = [Chain(*shape, seed=10 + i) for i, shape in enumerate(SHAPES)]
    wants = [c.one_by_one() for c in chains]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(6):
                    chains[i].at_once()
                got = chains[i].results()
            s.synchronize()
            if not same(got, wants[i]):
                wrong.append(i)
        except Exception as e:  # a refused call: told to the test
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(chains))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.parametrize("shape", SHAPES)
def test_device_memory_is_not_allocated(shape):
    c = Chain(*shape, seed=30)
    c.one_by_one()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(20):
        c.at_once()
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] < 1 << 20
