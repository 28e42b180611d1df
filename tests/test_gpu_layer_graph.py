"""The operators of include/qproj_layer.h inside captured graphs and on several
streams at once: they neither allocate nor synchronise, and each call reads
only its own arguments."""
import pytest
import torch

import gemv_nvfp4_int8_amd as qp
from examples import layer_step

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
H, I, IE, E, K = 640, 1376, 384, 20, 3


class Step:
    """A dense layer, then a mixture whose logits are given, on buffers of its own."""

    def __init__(self, rows, weights=None):
        self.dense = layer_step.Dense(rows, H, I, DEV)
        self.mix = layer_step.Mixture(min(rows, 16), H, IE, E, K, DEV)
        new = lambda: torch.empty((rows, H), dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.x, self.res, self.mid, self.out = new(), new(), new(), new()
        self.logits = torch.empty((min(rows, 16), E), device=DEV)

    def fill(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (self.x, self.res, self.logits):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        self.mid.fill_(float("nan"))
        self.out.fill_(float("nan"))

    def run(self):
        self.dense(self.x, self.res, self.mid)
        m, r = self.mix, self.logits.shape[0]
        qp.rmsnorm_residual_quant(self.mid[:r], self.res[:r], m.norm, 1e-6, qp.QP_ACT_BF16, m.y, None, self.res[:r])
        qp.moe_fp8_blockscale(m.y, self.logits, m.w13, m.s13, m.w2, m.s2, K, True, m.work, self.out[:r])

    def result(self):
        torch.cuda.synchronize()
        return [t.view(torch.int16).clone() for t in (self.mid, self.res, self.out[:self.logits.shape[0]])]


@pytest.mark.parametrize("rows", [1, 16, 200])
def test_replays_equal_the_eager_calls(rows):
    step = Step(rows)
    step.fill(0)
    step.run()                                        # loads the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for seed in range(1, 6):
        step.fill(seed)
        step.run()
        want = step.result()
        step.fill(seed)
        step.mix.work.fill_(0xFF)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(step.result(), want)), seed
        # the program's own work on the same buffers between two replays
        step.fill(100 + seed)
        step.run()
        (step.out.float().nan_to_num() @ step.out.float().nan_to_num().t()).sum().item()


def test_two_streams_at_once():
    steps = [Step(16) for _ in range(2)]
    want = []
    for n, s in enumerate(steps):
        s.fill(n)
        s.run()
        want.append(s.result())
        s.fill(n)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for s, st in zip(steps, streams):
        with torch.cuda.stream(st):
            s.run()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.result(), w))
