"""Several threads whose calls go to one stream (GPU): what a call's kernels pass to one another through the stream's
workspace stays that call's."""

import threading

import pytest
import torch

from tests._operators_common import paged

pytestmark = pytest.mark.gpu


class Selection:
    """pa_select_blocks and pa_decode_selected on fixed tensors, with what they give when alone."""

    def __init__(self, pa, seed, lens, H=4, g=2, D=64, B=8, K=9):
        self.pa, self.B = pa, B
        gen = torch.Generator().manual_seed(seed)
        t, nb = paged(gen, lens, B)
        rn = lambda *s: torch.randn(*s, generator=gen).half().cuda()
        self.t, self.n = t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.q, self.kc, self.vc = rn(len(lens), H * g, D), rn(nb, B, H, D), rn(nb, B, H, D)
        self.bounds = torch.zeros(nb, H, 2, D, dtype=torch.float16, device="cuda")
        pa.pa_block_bounds(self.kc, self.t, self.n, None, self.bounds)
        self.sel, self.out = torch.empty(len(lens), H, K, dtype=torch.int32, device="cuda"), torch.empty_like(self.q)
        self.run(None)
        torch.cuda.synchronize()
        self.want = self.sel.clone(), self.out.clone()
        self.wrong = torch.zeros((), dtype=torch.int64, device="cuda")

    def run(self, stream):
        self.pa.pa_select_blocks(self.q, self.bounds, self.t, self.n, self.B, self.sel, stream=stream)
        self.pa.pa_decode_selected(self.q, self.kc, self.vc, self.t, self.n, self.sel, 0.125, self.out, stream=stream)

    def loop(self, stream, times):
        with torch.cuda.stream(stream):
            for _ in range(times):
                self.run(stream)
                self.wrong += (self.sel != self.want[0]).any() | (self.out != self.want[1]).any()


def test_threads_on_one_stream(pa):
    work = [Selection(pa, i, [900 + 40 * i, 300, 777]) for i in range(6)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    errors = []

    def run(w):
        try:
            w.loop(stream, 400)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert [int(w.wrong) for w in work] == [0] * len(work)
    assert pa.pa_get_device_status() == 0
