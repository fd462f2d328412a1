"""Window attention and the 8-bit cache as a serving loop uses them: with the block manager's forks and copy-on-write, chunks beside
single tokens, captured into graphs, on several streams and from several threads (GPU)."""

import threading

import numpy as np
import pytest
import torch

from oracle.windows import Cache8, attend_seen, seen
from tests._operators_common import TD, attention_tolerance, host64
from tests._windows_common import cache8, on_gpu, window_tables
from tests.test_gpu_canaries import assert_guards, guarded
from tests.test_gpu_windows import chunk_tolerance

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def tables_of(bm, seqs, width=64):
    t, n = bm.block_tables(seqs, width)
    return dev(t), dev(n)


@pytest.mark.parametrize("dtype,H,g,window,sinks", [("f16", 4, 2, 0, 0), ("bf16", 4, 4, 40, 5)])
def test_8_bit_loop_with_forks(pa, dtype, H, g, window, sinks):
    """Prompts, forks whose tails are copied with their steps, single tokens; the cache compared with the oracle's, byte for byte."""
    D, B, nb = 128, 16, 60
    gen = torch.Generator().manual_seed(1)
    rows = lambda n, h: (torch.randn(n, h, D, generator=gen) * torch.exp(torch.randn(n, 1, 1, generator=gen))).to(TD[dtype])
    bm = pa.BlockManager(nb, B)
    ref = [Cache8(np.zeros((nb, H, B, D), np.uint8), np.zeros((nb, H), np.float32)) for _ in range(2)]
    gpu = [on_gpu(c) for c in ref]

    def append(seqs, counts, k, v, start):
        t, n = tables_of(bm, seqs)
        pa.pa_cache_append_q8(k.cuda(), v.cuda(), t, n, gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], query_start=start)
        at = 0
        for s, c in zip(seqs, counts):
            for i, x in enumerate((k, v)):
                ref[i].append(bm.table(s), bm.seq_info(s)[0], x[at:at + c].float().numpy())
            at += c
        return t, n

    for seq, c in ((0, 100), (1, 17), (2, 32)):
        bm.add_seq(seq, c)
        append([seq], [c], rows(c, H), rows(c, H), dev(np.array([0, c], np.int32)))
    seqs = [0, 1, 2]
    for step in range(24):
        if step == 3:                                    # forks share frames; the next appends copy the tails
            bm.fork(0, 10)
            bm.fork(1, 11)
            seqs = [0, 10, 1, 11, 2]
        _, copies = bm.step(seqs)
        assert len(copies) == (2 if step == 3 else 0)
        if len(copies):
            pa.pa_copy_blocks(gpu[0][0], gpu[1][0], dev(copies))
            pa.pa_copy_blocks(gpu[0][1].view(nb, 1, 1, H), gpu[1][1].view(nb, 1, 1, H), dev(copies))
            for c in ref:
                for a, b in copies:
                    c.codes[b], c.steps[b] = c.codes[a], c.steps[a]
        n = len(seqs)
        k, v, q = rows(n, H), rows(n, H), rows(n, H * g).cuda()
        t, lens = append(seqs, [1] * n, k, v, None)
        out = torch.empty_like(q)
        pa.pa_decode_q8(q, gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], t, lens, D ** -0.5, out, window=window, sinks=sinks)
        assert pa.pa_get_device_status() == 0
        for (codes, steps), c in zip(gpu, ref):
            assert np.array_equal(codes.cpu().numpy(), c.codes) and np.array_equal(steps.cpu().numpy(), c.steps)
        for i, s in enumerate(seqs):
            L = int(lens[i])
            kk, vv = (c.values(bm.table(s), L) for c in ref)
            on = seen(L - 1, window, sinks)
            want = attend_seen(host64(q[i]), kk[on], vv[on], len(on) - 1, 0, 0, D ** -0.5)
            tol = attention_tolerance(want, TD[dtype], host64(q[i]), kk[on], vv[on], D ** -0.5, 2.0 ** -22)
            assert (np.abs(host64(out[i]) - want) <= tol).all()


def test_window_loop_gives_up_frames(pa):
    """Prompts in chunks, then single tokens; behind the window each step's table forgets the frames, and their rows are overwritten."""
    H, g, D, B, window, sinks, dtype = 2, 2, 128, 16, 50, 6, "f16"
    nb = 40
    gen = torch.Generator().manual_seed(2)
    kc, vc = (torch.zeros(nb, B, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    free = list(range(nb))
    table, dense = np.full((1, 32), -1, np.int32), [np.zeros((0, H, D)), np.zeros((0, H, D))]
    L = 0
    for c in (70, 33, 128, 1, 1, 1, 20, 1, 1) + (1,) * 30:
        k, v, q = (torch.randn(c, h, D, generator=gen).half() for h in (H, H, H * g))
        dense = [np.concatenate([d, host64(x)]) for d, x in zip(dense, (k, v))]
        for j in range(-(-L // B), -(-(L + c) // B)):
            table[0, j] = free.pop()
        slots = np.array([table[0, p // B] * B + p % B for p in range(L, L + c)], np.int32)
        pa.pa_cache_append(k.cuda(), v.cuda(), dev(slots), kc, vc)
        first, L = L, L + c
        out = torch.empty_like(q, device="cuda")
        lens = torch.tensor([L], dtype=torch.int32).cuda()
        if c > 1:
            pa.pa_prefill_window(q.cuda(), kc, vc, dev(table), lens, torch.tensor([0, c], dtype=torch.int32).cuda(), window, 0.09, out, sinks=sinks)
        else:
            pa.pa_decode_window(q.cuda(), kc, vc, dev(table), lens, window, 0.09, out, sinks=sinks)
        assert pa.pa_get_device_status() == 0
        for i in range(c):
            on = seen(first + i, window, sinks)
            kk, vv = dense[0][on], dense[1][on]
            want = attend_seen(host64(q[i]), kk, vv, len(on) - 1, 0, 0, 0.09)
            assert (np.abs(host64(out[i]) - want) <= chunk_tolerance(want, dtype, host64(q[i]), kk, vv, 0.09)).all(), (L, i)
        for j in range(-(-sinks // B), (L + 1 - window) // B if L >= window else 0):   # what no later query sees
            if table[0, j] >= 0:
                free.append(int(table[0, j]))
                kc[table[0, j]] = 1e4                                                  # (finite: pa_prefill_window's rule for slots it may read)
                vc[table[0, j]] = -1e4
                table[0, j] = -1
    assert len(free) >= nb - (window // B + 3)


def test_chunk_over_an_8_bit_prefix(pa):
    """A chunk's queries over a window of a prefix held in 8 bits: what they see read back into 16-bit frames, then pa_prefill_window."""
    H, g, D, B, L, n, window = 2, 4, 128, 16, 300, 40, 90
    gen = torch.Generator().manual_seed(3)
    bm = pa.BlockManager(30, B)
    slots = bm.add_seq(0, L)
    k, v = (torch.randn(L, H, D, generator=gen).half() for _ in range(2))
    ref = [Cache8(np.zeros((30, H, B, D), np.uint8), np.zeros((30, H), np.float32)) for _ in range(2)]
    gpu = [on_gpu(c) for c in ref]
    t, lens = tables_of(bm, [0], 30)
    pa.pa_cache_append_q8(k.cuda(), v.cuda(), t, lens, gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], query_start=dev(np.array([0, L], np.int32)))
    for c, x in zip(ref, (k, v)):
        c.append(bm.table(0), L, x.float().numpy())
    first = L - n + 1 - window
    some = dev(slots[first:])
    kr, vr = (torch.empty(len(some), H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q8(gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], some, kr, vr)
    k16, v16 = (torch.zeros(30, B, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_append(kr, vr, some, k16, v16)
    q = torch.randn(n, H * g, D, generator=gen).half().cuda()
    out = torch.empty_like(q)
    pa.pa_prefill_window(q, k16, v16, t, lens, dev(np.array([0, n], np.int32)), window, 0.09, out)
    kk, vv = (c.values(bm.table(0), L).astype(np.float32).astype(np.float16).astype(np.float64) for c in ref)
    for i in range(n):
        on = seen(L - n + i, window, 0)
        want = attend_seen(host64(q[i]), kk[on], vv[on], len(on) - 1, 0, 0, 0.09)
        assert (np.abs(host64(out[i]) - want) <= chunk_tolerance(want, "f16", host64(q[i]), kk[on], vv[on], 0.09)).all()
    assert pa.pa_get_device_status() == 0


@pytest.mark.parametrize("H,g", [(2, 2), (30, 1), (20, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunks_write_only_their_rows(pa, dtype, H, g):
    """Strided queries, outputs between canaries, for each kind of slots; the same bits as plain tensors give."""
    gen = torch.Generator().manual_seed(4)
    lens, fresh = [40, 300, 129, 513], [40, 130, 1, 257]
    tables, nb = window_tables(gen, lens, fresh, 16, 100, 5)
    kc, vc = (torch.randn(nb, 16, H, 128, generator=gen).to(TD[dtype]).cuda() for _ in range(2))
    T, start = sum(fresh), torch.tensor(np.cumsum([0] + fresh), dtype=torch.int32).cuda()
    wide = torch.full((T, H * g * 128 + 64), float("nan"), dtype=TD[dtype], device="cuda")
    wide[:, : H * g * 128] = torch.randn(T, H * g * 128, generator=gen).to(TD[dtype]).cuda()
    q = wide[:, : H * g * 128].unflatten(1, (H * g, 128))
    buf, out = guarded(T, H * g, 128, dtype)
    ref = torch.empty(T, H * g, 128, dtype=TD[dtype], device="cuda")
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    pa.pa_prefill_window(q, kc, vc, tables.cuda(), n, start, 100, 0.09, out, sinks=5)
    pa.pa_prefill_window(q.contiguous(), kc, vc, tables.cuda(), n, start, 100, 0.09, ref, sinks=5)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    assert_guards(buf, T, H * g, 128)
    assert torch.equal(out.contiguous().view(torch.int16), ref.view(torch.int16))


# ---- graphs, streams, threads --------------------------------------------------------------------------
class Step:
    """A step's calls on fixed tensors: append in 8 bits, decode over all tokens and over windows, a window over 16 bits, a chunk."""

    def __init__(self, pa, seed, lens=(700, 33, 16, 1, 250), H=2, g=4, D=128, B=16):
        self.pa = pa
        gen = torch.Generator().manual_seed(seed)
        S = len(lens)
        t, nb = window_tables(gen, lens, [1] * S, B, 0, 0)
        rn = lambda *s: torch.randn(*s, generator=gen).half().cuda()
        self.t, self.n = t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        (self.k8, self.ks), (self.v8, self.vs) = (on_gpu(cache8(gen, t, lens, nb, H, B, D, "f16")) for _ in range(2))
        self.kc, self.vc = rn(nb, B, H, D), rn(nb, B, H, D)
        self.k, self.v, self.q = rn(S, H, D), rn(S, H, D), rn(S, H * g, D)
        self.chunk = [min(n, 30) for n in lens]
        self.start = torch.tensor(np.cumsum([0] + self.chunk), dtype=torch.int32).cuda()
        self.qc = rn(sum(self.chunk), H * g, D)
        self.rows = torch.arange(nb * B, dtype=torch.int32).cuda()
        self.kr, self.vr = (torch.empty(nb * B, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
        self.out = [torch.empty_like(self.q) for _ in range(3)]
        self.outc = torch.empty_like(self.qc)

    def run(self, stream=None):
        pa, kw = self.pa, {"stream": stream}
        pa.pa_cache_append_q8(self.k, self.v, self.t, self.n, self.k8, self.v8, self.ks, self.vs, **kw)
        pa.pa_decode_q8(self.q, self.k8, self.v8, self.ks, self.vs, self.t, self.n, 0.1, self.out[0], **kw)
        pa.pa_decode_q8(self.q, self.k8, self.v8, self.ks, self.vs, self.t, self.n, 0.1, self.out[1], window=100, sinks=4, **kw)
        pa.pa_decode_window(self.q, self.kc, self.vc, self.t, self.n, 100, 0.1, self.out[2], sinks=4, **kw)
        pa.pa_prefill_window(self.qc, self.kc, self.vc, self.t, self.n, self.start, 100, 0.1, self.outc, sinks=4, **kw)
        pa.pa_cache_read_q8(self.k8, self.v8, self.ks, self.vs, self.rows, self.kr, self.vr, **kw)

    def results(self):
        return [x.clone() for x in (*self.out, self.outc, self.k8, self.v8, self.kr.nan_to_num(7), self.vr.nan_to_num(7))]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def eager(pa, seed, change=None, **more):
    s = Step(pa, seed, **more)
    if change:
        change(s)
    s.run()
    torch.cuda.synchronize()
    return s.results()


def test_captured_step_replays(pa):
    def change(s):
        gen = torch.Generator().manual_seed(77)
        for x in (s.k, s.v, s.q, s.qc):
            x.copy_(2 * torch.randn(x.shape, generator=gen).half())

    want = eager(pa, 5), eager(pa, 5, change)
    s = Step(pa, 5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        Step(pa, 5).run()                                # workspaces of this stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    graph.replay()
    torch.cuda.synchronize()
    assert same(s.results(), want[0])
    start = Step(pa, 5)                                  # the cache as it was before the first replay
    for a, b in ((s.k8, start.k8), (s.v8, start.v8), (s.ks, start.ks), (s.vs, start.vs)):
        a.copy_(b)
    change(s)
    graph.replay()
    torch.cuda.synchronize()
    assert same(s.results(), want[1])
    graph.replay()                                       # the same tokens once more: they fit already
    torch.cuda.synchronize()
    assert same(s.results(), want[1])
    assert pa.pa_get_device_status() == 0


def test_capture_without_a_workspace_is_refused_and_stays_valid(pa):
    s = Step(pa, 8)
    want = eager(pa, 8)
    x = torch.zeros(4, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        for call in (lambda: pa.pa_decode_q8(s.q, s.k8, s.v8, s.ks, s.vs, s.t, s.n, 0.1, s.out[0]),
                     lambda: pa.pa_decode_window(s.q, s.kc, s.vc, s.t, s.n, 9, 0.1, s.out[2]),
                     lambda: pa.pa_prefill_window(s.qc, s.kc, s.vc, s.t, s.n, s.start, 9, 0.1, s.outc)):
            with pytest.raises(pa.PAError) as e:
                call()
            assert e.value.code == pa.PA_ERR_SCRATCH_LIMIT
        x.add_(1)
        graph.capture_end()
    graph.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()
    s.run()
    torch.cuda.synchronize()
    assert same(s.results(), want)


def test_streams_at_once(pa):
    seeds = (11, 12, 13)
    want = [eager(pa, x) for x in seeds]
    steps = [Step(pa, x) for x in seeds]
    streams = [torch.cuda.Stream() for _ in seeds]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert same(s.results(), w)
    assert pa.pa_get_device_status() == 0


def test_threads_on_one_stream(pa):
    seeds = (21, 22, 23, 24)
    want = [eager(pa, x) for x in seeds]
    steps = [Step(pa, x) for x in seeds]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    bad = []

    def work(s):
        try:
            with torch.cuda.stream(stream):
                for _ in range(30):
                    s.run()
        except Exception as e:
            bad.append(e)

    ts = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    for s, w in zip(steps, want):
        assert same(s.results(), w)


def test_calls_after_shutdown(pa):
    want = eager(pa, 31)
    torch.cuda.synchronize()
    pa.pa_shutdown()
    assert same(eager(pa, 31), want)


def test_host_tensors_and_wrong_types_are_refused(pa):
    s = Step(pa, 41)
    n = pa.pa_launch_count()
    with pytest.raises(ValueError, match="CUDA tensors"):
        pa.pa_decode_q8(s.q.cpu(), s.k8, s.v8, s.ks, s.vs, s.t, s.n, 0.1, s.out[0])
    with pytest.raises(TypeError):
        pa.pa_decode_window(s.q, s.kc, s.vc, s.t.long(), s.n, 9, 0.1, s.out[2])
    with pytest.raises(TypeError):
        pa.pa_cache_append_q8(s.k, s.v, s.t, s.n, s.k8, s.v8, s.ks.double(), s.vs)
    with pytest.raises(TypeError):
        pa.pa_prefill_window(s.qc, s.kc, s.vc, s.t, s.n, None, 9, 0.1, s.outc)
    with pytest.raises(OverflowError):
        pa.pa_decode_window(s.q, s.kc, s.vc, s.t, s.n, 1 << 40, 0.1, s.out[2])
    for call in (lambda: pa.pa_decode_window(s.q, s.kc, s.vc, s.t, s.n, 0, 0.1, s.out[2]),
                 lambda: pa.pa_decode_q8(s.q, s.k8, s.v8, s.ks, s.vs, s.t, s.n, 0.1, s.out[0], sinks=4),
                 lambda: pa.pa_prefill_window(s.qc, s.kc, s.vc, s.t, s.n, s.start, 9, -0.1, s.outc),
                 lambda: pa.pa_cache_append_q8(s.k.bfloat16(), s.v, s.t, s.n, s.k8, s.v8, s.ks, s.vs),
                 lambda: pa.pa_cache_read_q8(s.k8, s.v8, s.ks, s.vs, s.rows, s.kr.float(), s.vr.float())):
        with pytest.raises(pa.PAError):
            call()
    assert pa.pa_launch_count() == n
