"""After a timeout was read, captured graphs run from zeroed counters too, in workspaces that a later call has outgrown as
well as in the one in use (GPU)."""

import pytest
import torch

from oracle.operators import quantise_q4
from tests._operators_common import paged

pytestmark = pytest.mark.gpu


class Decodes:
    """A 4-bit decode and a plain one whose contexts are cut into pieces, so that both count arrivals."""

    def __init__(self, pa, seed, lens, H=2, D=128, B=16):
        self.pa = pa
        gen = torch.Generator().manual_seed(seed)
        t, nb = paged(gen, lens, B)
        rn = lambda *s: torch.randn(*s, generator=gen).half()
        self.t, self.n = t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.q, self.kc, self.vc = (x.cuda() for x in (rn(len(lens), H, D), rn(nb, B, H, D), rn(nb, B, H, D)))
        self.k4, self.v4 = (torch.from_numpy(quantise_q4(rn(nb, H, B, D).float().numpy())).cuda() for _ in range(2))
        self.out = [torch.empty_like(self.q) for _ in range(2)]

    def run(self):
        self.pa.pa_decode_q4(self.q, self.k4, self.v4, self.t, self.n, 0.1, self.out[0])
        self.pa.pa_decode_ex(self.q, self.kc, self.vc, self.t, self.n, 0.1, self.out[1], params={"partition_tokens": 256})

    def captured(self, stream):
        """A graph of the calls, and their outputs."""
        with torch.cuda.stream(stream):
            self.run()
        torch.cuda.synchronize()
        want = [x.clone() for x in self.out]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self.run()
        return graph, want

    def replayed(self, graph, want):
        for x in self.out:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        return all(torch.equal(x, y) for x, y in zip(self.out, want))


def test_graphs_after_a_timeout(pa):
    stream = torch.cuda.Stream()
    small, big = Decodes(pa, 1, [3000, 17, 900]), Decodes(pa, 2, [3000] * 4 + [1] * 4300, H=4)
    g1, w1 = small.captured(stream)
    g2, w2 = big.captured(stream)          # a larger workspace: the first graph keeps the one it has
    for _ in range(2):
        assert pa.pa_get_device_status() == 0
        pa.pa_selftest_raise_counters()
        assert pa.pa_get_device_status() == pa.PA_DEV_TIMEOUT
        for _ in range(2):
            assert small.replayed(g1, w1)
            assert big.replayed(g2, w2)
    assert pa.pa_get_device_status() == 0
    with torch.cuda.stream(stream):
        small.run()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(small.out, w1))
