"""The library's workspace of a stream: what a call may need more of, under capture and without, and how much memory
that takes (GPU)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

MB = 1 << 20


class Select:
    """pa_select_blocks of S short sequences under tables of `width` columns: 32 S width bytes of workspace."""

    def __init__(self, pa, S, width, H=8):
        self.pa = pa
        gen = torch.Generator().manual_seed(S)
        self.t = torch.zeros(S, width, dtype=torch.int32, device="cuda")
        self.t[:, :20] = torch.stack([torch.randperm(32, generator=gen)[:20] for _ in range(S)])
        self.n = torch.full((S,), 8 * 20, dtype=torch.int32, device="cuda")
        self.bounds = torch.randn(32, H, 2, 64, generator=gen).half().cuda().sort(dim=2).values.contiguous()
        self.q = torch.randn(S, H, 64, generator=gen).half().cuda()
        self.sel = torch.zeros(S, H, 5, dtype=torch.int32, device="cuda")

    def run(self):
        self.pa.pa_select_blocks(self.q, self.bounds, self.t, self.n, 8, self.sel)
        return self.sel


def capture(stream, run):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    return graph


def free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


def test_growth_takes_what_it_needs(pa):
    """Without graphs the outgrown buffer goes back, and the next is no larger than asked for."""
    wide = [Select(pa, S, 1 << 20) for S in (3, 4, 5)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        wide[0].run()
        before = free()
        for w in wide:
            w.run()
    grown = before - free()
    assert grown <= 2 * 32 * MB + 8 * MB, grown                # from 3 to 5 sequences


def test_growth_beside_a_graph_where_there_is_little_room(pa):
    """A graph keeps its buffer; twice as much does not fit any more, what is needed does."""
    wide = [Select(pa, S, 1 << 20) for S in (4, 5)]
    want = [w.run().clone() for w in wide]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        wide[0].run()
    torch.cuda.synchronize()
    graph = capture(stream, wide[0].run)
    graph.replay()
    rest = free() - 240 * MB                                   # 160 MB are needed, 256 MB are twice the graph's
    fill = torch.empty(rest, dtype=torch.uint8, device="cuda")
    try:
        with torch.cuda.stream(stream):
            wide[1].sel.zero_()
            wide[1].run()
        wide[0].sel.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [w.sel.clone() for w in wide]
    finally:
        del fill
        torch.cuda.empty_cache()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert pa.pa_get_device_status() == 0


class Decode:
    """pa_decode of sequences that may be cut into pieces: an arrival counter per (sequence, head)."""

    def __init__(self, pa, lens, H=4, D=64, B=8):
        self.pa = pa
        gen = torch.Generator().manual_seed(len(lens))
        width = -(-max(lens) // B)
        self.t = torch.randint(0, 64, (len(lens), width), generator=gen).int().cuda()
        self.n = torch.tensor(lens, dtype=torch.int32).cuda()
        self.kc, self.vc = (torch.randn(64, B, H, D, generator=gen).half().cuda() for _ in range(2))
        self.q = torch.randn(len(lens), H, D, generator=gen).half().cuda()
        self.out = torch.empty_like(self.q)

    def run(self):
        self.out.fill_(float("nan"))
        self.pa.pa_decode_ex(self.q, self.kc, self.vc, self.t, self.n, 0.125, self.out, params={"partition_tokens": 64})


def test_more_counters_under_capture(pa):
    """A captured call of more (sequence, head) pairs than any before it on the stream, where the buffer has room: the graph
    runs right beside direct calls whose partials lie where its counters are, before its first replay and after."""
    many, few, small = Decode(pa, [200] + [20] * 4999), Decode(pa, [3000, 1, 200, 3000]), Decode(pa, [200, 7])
    want = []
    for d in (many, few):
        d.run()
        want.append(d.out.clone())
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        # 32 MB of scores: room for the batch's partials; no counters asked for so far
        Select(pa, 1, 1 << 20).run()
        small.run()
    torch.cuda.synchronize()
    graph = capture(stream, many.run)
    for _ in range(3):
        with torch.cuda.stream(stream):
            few.run()
            torch.cuda.synchronize()
            assert torch.equal(few.out, want[1])
        many.out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(many.out, want[0])
    with torch.cuda.stream(stream):
        many.run()                                             # directly: a buffer of its own
        few.run()
    torch.cuda.synchronize()
    assert torch.equal(many.out, want[0]) and torch.equal(few.out, want[1])
    many.out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(many.out, want[0])
    assert pa.pa_get_device_status() == 0
