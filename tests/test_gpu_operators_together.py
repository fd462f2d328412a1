"""The rotating append, the 4-bit cache and the block-sparse decode as a serving loop uses them: with the block
manager's forks and copy-on-write, beside pa_prefill, captured into graphs, on several streams and from several
threads."""

import threading

import numpy as np
import pytest
import torch

from oracle.operators import attend, cos_sin_table, quantise_q4, rotate, values_q4
from tests._operators_common import TD, attention_tolerance, half_step, host64, paged, tiny

pytestmark = pytest.mark.gpu


class Loop:
    """Sequences of a block manager with rotated keys, and the same rows kept densely on the host."""

    def __init__(self, pa, H, g, D, B, nb, dtype, seed):
        self.pa, self.H, self.g, self.D, self.B, self.dtype = pa, H, g, D, B, dtype
        self.gen = torch.Generator().manual_seed(seed)
        self.bm = pa.BlockManager(nb, B)
        self.table = cos_sin_table(512, D)
        self.cs = torch.from_numpy(self.table).cuda()
        self.dense = {}                                  # sequence -> [rotated keys, values], float64 [n, H, D]

    def rows(self, n, heads):
        return torch.randn(n, heads, self.D, generator=self.gen).to(TD[self.dtype])

    def remember(self, seq, k, v, pos):
        self.dense.setdefault(seq, [[], []])
        self.dense[seq][0] += list(rotate(host64(k), self.table, pos, False))
        self.dense[seq][1] += list(host64(v))

    def tables(self, seqs, width=64):
        t, n = self.bm.block_tables(seqs, width)
        return torch.from_numpy(t.copy()).cuda(), torch.from_numpy(n.copy()).cuda()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("dtype,H,g", [("f16", 2, 4), ("bf16", 4, 1)])
def test_sparse_decode_loop_with_forks(pa, dtype, H, g):
    D, B, K = 128, 16, 5
    lp = Loop(pa, H, g, D, B, 200, dtype, 1)
    kc, vc = (torch.full((200, B, H, D), float("nan"), dtype=TD[dtype], device="cuda") for _ in range(2))
    bounds = torch.full((200, H, 2, D), float("nan"), dtype=TD[dtype], device="cuda")
    for seq, n in enumerate((200, 17, 33)):
        slots = lp.bm.add_seq(seq, n)
        k, v = lp.rows(n, H), lp.rows(n, H)
        pos = np.arange(n, dtype=np.int32)
        pa.pa_cache_append_rope(k.cuda(), v.cuda(), dev(slots), kc, vc, dev(pos), lp.cs)
        lp.remember(seq, k, v, pos)
    seqs = [0, 1, 2]
    t, n = lp.tables(seqs)
    pa.pa_block_bounds(kc, t, n, None, bounds)
    for step in range(20):
        if step == 3:                                    # forks share frames, the next appends copy the tails
            lp.bm.fork(0, 10)
            lp.bm.fork(2, 12)
            lp.dense[10], lp.dense[12] = [list(x) for x in lp.dense[0]], [list(x) for x in lp.dense[2]]
            seqs = [0, 10, 1, 2, 12]
        pos = np.array([lp.bm.seq_info(s)[0] for s in seqs], np.int32)
        slots, copies = lp.bm.step(seqs)
        assert len(copies) == (2 if step == 3 else 0)
        if len(copies):
            pa.pa_copy_blocks(kc, vc, dev(copies))
        k, v, q = lp.rows(len(seqs), H), lp.rows(len(seqs), H), lp.rows(len(seqs), H * g)
        qd = q.cuda()
        pa.pa_cache_append_rope(k.cuda(), v.cuda(), dev(slots), kc, vc, dev(pos), lp.cs, q=qd, q_out=qd)
        for i, s in enumerate(seqs):
            lp.remember(s, k[i:i + 1], v[i:i + 1], pos[i:i + 1])
        t, n = lp.tables(seqs)
        pa.pa_block_bounds(kc, t, n, n - 1, bounds)
        sel = torch.empty(len(seqs), H, K, dtype=torch.int32, device="cuda")
        pa.pa_select_blocks(qd, bounds, t, n, B, sel, keep_first=1, keep_last=1)
        out = torch.empty_like(qd)
        pa.pa_decode_selected(qd, kc, vc, t, n, sel, D ** -0.5, out)
        assert pa.pa_get_device_status() == 0
        th, oh, qh, selh = t.cpu().long(), host64(out), host64(qd), sel.cpu()
        for i, s in enumerate(seqs):
            L = int(n[i])
            f, o = th[i, torch.arange(L) // B], torch.arange(L) % B
            kk, vv = host64(kc.cpu()[f, o]), host64(vc.cpu()[f, o])
            dk, dv = np.array(lp.dense[s][0]), np.array(lp.dense[s][1])
            assert np.array_equal(vv, dv)
            # a rotated key: half a step of the type, and three roundings to fp32 of numbers below 2 max |k|
            assert (np.abs(kk - dk) <= half_step(TD[dtype]) * np.abs(dk) + 6 * 2.0 ** -24 * np.abs(dk).max() + tiny(TD[dtype])).all()
            blocks = -(-L // B)
            for h in range(H):
                lo = np.array([kk[b * B:(b + 1) * B, h].min(0) for b in range(blocks)])
                hi = np.array([kk[b * B:(b + 1) * B, h].max(0) for b in range(blocks)])
                fr = th[i, :blocks]
                assert np.array_equal(host64(bounds[fr, h, 0]), lo) and np.array_equal(host64(bounds[fr, h, 1]), hi)
                lst = [e for e in selh[i, h].tolist() if e >= 0]
                assert len(lst) == min(K, blocks) and lst[0] == 0 and lst[-1] == blocks - 1
                tok = np.concatenate([np.arange(e * B, min(L, (e + 1) * B)) for e in lst])
                ref = attend(qh[i, h * g:h * g + g], kk[tok, h:h + 1], vv[tok, h:h + 1], D ** -0.5)
                tol = attention_tolerance(ref, TD[dtype], qh[i, h * g:h * g + g], kk[tok, h], vv[tok, h], D ** -0.5,
                                          2.0 ** (-22 if dtype == "f16" else -16))
                assert (np.abs(oh[i, h * g:h * g + g] - ref) <= tol).all()


def test_4_bit_loop_with_forks(pa):
    H, g, D, B = 2, 4, 128, 16
    lp = Loop(pa, H, g, D, B, 100, "bf16", 2)
    kc, vc = (torch.full((100, H, B, 80), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    for seq, n in enumerate((100, 17)):
        slots = lp.bm.add_seq(seq, n)
        k, v = lp.rows(n, H), lp.rows(n, H)
        pos = np.arange(n, dtype=np.int32)
        pa.pa_cache_append_q4(k.cuda(), v.cuda(), dev(slots), kc, vc, dev(pos), lp.cs)
        # with bf16 queries a key enters its score as step * n + offset, not rounded to fp16
        lp.dense[seq] = [list(values_q4(quantise_q4(rotate(k.float().numpy(), lp.table, pos, False)), rounded=False)),
                         list(values_q4(quantise_q4(v.float().numpy())))]
    seqs = [0, 1]
    for step in range(6):
        if step == 2:
            lp.bm.fork(0, 10)
            lp.bm.fork(1, 11)
            lp.dense[10], lp.dense[11] = [list(x) for x in lp.dense[0]], [list(x) for x in lp.dense[1]]
            seqs = [0, 10, 1, 11]
        pos = np.array([lp.bm.seq_info(s)[0] for s in seqs], np.int32)
        slots, copies = lp.bm.step(seqs)
        if len(copies):
            pa.pa_copy_blocks(kc, vc, dev(copies))
        k, v, q = lp.rows(len(seqs), H), lp.rows(len(seqs), H), lp.rows(len(seqs), H * g)
        qd = q.cuda()
        pa.pa_cache_append_q4(k.cuda(), v.cuda(), dev(slots), kc, vc, dev(pos), lp.cs, q=qd, q_out=qd)
        kq = values_q4(quantise_q4(rotate(k.float().numpy(), lp.table, pos, False)), rounded=False)
        vq = values_q4(quantise_q4(v.float().numpy()))
        for i, s in enumerate(seqs):
            lp.dense[s][0].append(kq[i])
            lp.dense[s][1].append(vq[i])
        t, n = lp.tables(seqs)
        out = torch.empty_like(qd)
        pa.pa_decode_q4(qd, kc, vc, t, n, D ** -0.5, out)
        assert pa.pa_get_device_status() == 0
        for i, s in enumerate(seqs):
            kk, vv = np.array(lp.dense[s][0]), np.array(lp.dense[s][1])
            assert len(kk) == int(n[i])
            ref = attend(host64(qd[i]), kk, vv, D ** -0.5)
            tol = attention_tolerance(ref, torch.bfloat16, host64(qd[i]), kk, vv, D ** -0.5, 2.0 ** -11)
            assert (np.abs(host64(out[i]) - ref) <= tol).all()


def test_prefill_over_a_4_bit_prefix(pa):
    """A chunk's queries over a prefix held in 4 bits: the prefix read back into 16-bit frames, then pa_prefill."""
    H, D, B, L, n = 2, 128, 16, 100, 20
    gen = torch.Generator().manual_seed(3)
    bm = pa.BlockManager(20, B)
    slots = bm.add_seq(0, L)
    k, v = (torch.randn(L, H, D, generator=gen).half() for _ in range(2))
    kc, vc = (torch.zeros(20, H, B, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    pa.pa_cache_append_q4(k.cuda(), v.cuda(), dev(slots), kc, vc)
    kr, vr = (torch.empty(L, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_read_q4(kc, vc, dev(slots), kr, vr)
    k16, v16 = (torch.zeros(20, B, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_cache_append(kr, vr, dev(slots), k16, v16)
    t, lens = bm.block_tables([0], 8)
    q = torch.randn(n, H, D, generator=gen).half().cuda()
    out = torch.empty_like(q)
    pa.pa_prefill(q, k16, v16, dev(t), dev(lens), torch.tensor([0, n], dtype=torch.int32, device="cuda"), 0.09, out)
    kk, vv = values_q4(quantise_q4(k.float().numpy())), values_q4(quantise_q4(v.float().numpy()))
    for i in range(n):
        ref = attend(host64(q[i]), kk[: L - n + i + 1], vv[: L - n + i + 1], 0.09)
        assert np.abs(host64(out[i]) - ref).max() <= 2e-3 + np.abs(ref).max() * 2.0 ** -11   # pa_prefill's own tolerance


# ---- graphs, streams, threads --------------------------------------------------------------------------
class Step:
    """One decode step's calls on fixed tensors: rotated append, bounds, selection, sparse decode, and a 4-bit decode."""

    def __init__(self, pa, seed, lens=(700, 33, 16, 1, 250), H=2, g=4, D=128, B=16, K=6):
        self.pa, self.B, self.D = pa, B, D
        gen = torch.Generator().manual_seed(seed)
        S = len(lens)
        t, nb = paged(gen, lens, B)
        rn = lambda *s: torch.randn(*s, generator=gen).half().cuda()
        self.t, self.n = t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.kc, self.vc = rn(nb, B, H, D), rn(nb, B, H, D)
        self.k4, self.v4 = (torch.from_numpy(quantise_q4(rn(nb, H, B, D).float().cpu().numpy())).cuda() for _ in range(2))
        self.bounds = torch.zeros(nb, H, 2, D, dtype=torch.float16, device="cuda")
        pa.pa_block_bounds(self.kc, self.t, self.n, None, self.bounds)
        self.k, self.v, self.q = rn(S, H, D), rn(S, H, D), rn(S, H * g, D)
        last = torch.tensor([int(t[s, (lens[s] - 1) // B]) * B + (lens[s] - 1) % B for s in range(S)], dtype=torch.int32)
        self.slots, self.pos = last.cuda(), (self.n - 1).clone()
        self.cs = torch.from_numpy(cos_sin_table(max(lens) + 1, D)).cuda()   # a row for every position
        self.q_out, self.out, self.out4 = (torch.empty_like(self.q) for _ in range(3))
        self.sel = torch.empty(S, H, K, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        pa = self.pa
        pa.pa_cache_append_rope(self.k, self.v, self.slots, self.kc, self.vc, self.pos, self.cs, q=self.q, q_out=self.q_out, stream=stream)
        pa.pa_block_bounds(self.kc, self.t, self.n, self.pos, self.bounds, stream=stream)
        pa.pa_select_blocks(self.q_out, self.bounds, self.t, self.n, self.B, self.sel, stream=stream)
        pa.pa_decode_selected(self.q_out, self.kc, self.vc, self.t, self.n, self.sel, 0.1, self.out, stream=stream)
        pa.pa_cache_append_q4(self.k, self.v, self.slots, self.k4, self.v4, self.pos, self.cs, stream=stream)
        pa.pa_decode_q4(self.q_out, self.k4, self.v4, self.t, self.n, 0.1, self.out4, stream=stream)

    def results(self):
        return [x.clone() for x in (self.q_out, self.sel, self.out, self.out4, self.kc, self.k4, self.bounds)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def eager(pa, seed, change=None):
    s = Step(pa, seed)
    if change:
        change(s)
    s.run()
    torch.cuda.synchronize()
    return s.results()


def test_captured_step_replays(pa):
    def change(s):
        gen = torch.Generator().manual_seed(77)
        for x in (s.k, s.v, s.q):
            x.copy_(torch.randn(x.shape, generator=gen).half())

    want = eager(pa, 5), eager(pa, 5, change)
    s = Step(pa, 5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()                                          # workspaces of this stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    graph.replay()
    torch.cuda.synchronize()
    assert same(s.results(), want[0])
    change(s)
    graph.replay()
    torch.cuda.synchronize()
    assert same(s.results(), want[1])
    # a larger call on the same stream gets a larger workspace; the graph keeps its own
    big = Step(pa, 6, lens=(30000,) * 3 + (5,) * 300, H=8)
    with torch.cuda.stream(stream):
        big.run()
    torch.cuda.synchronize()
    first = big.results()
    for _ in range(3):
        for x in (s.out, s.out4, s.q_out):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same(s.results(), want[1])
    with torch.cuda.stream(stream):
        big.run()
    torch.cuda.synchronize()
    assert same(big.results(), first)
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
        with pytest.raises(pa.PAError) as e:
            pa.pa_decode_q4(s.q, s.k4, s.v4, s.t, s.n, 0.1, s.out4)
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
            s.run(stream=st)                             # the stream as an argument, not the current one
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert same(s.results(), w)
    assert pa.pa_get_device_status() == 0


def test_threads_at_once(pa):
    seeds = (21, 22, 23, 24)
    want = [eager(pa, x) for x in seeds]
    steps = [Step(pa, x) for x in seeds]
    torch.cuda.synchronize()
    bad = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
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
        pa.pa_decode_q4(s.q.cpu(), s.k4, s.v4, s.t, s.n, 0.1, s.out4)
    with pytest.raises(TypeError):
        pa.pa_decode_q4(s.q, s.k4, s.v4, s.t.long(), s.n, 0.1, s.out4)
    with pytest.raises(TypeError):
        pa.pa_decode_q4(None, s.k4, s.v4, s.t, s.n, 0.1, s.out4)
    with pytest.raises(pa.PAError):
        pa.pa_decode_q4(s.q.bfloat16(), s.k4, s.v4, s.t, s.n, 0.1, s.out4)
    with pytest.raises(OverflowError):
        pa.pa_select_blocks(s.q, s.bounds, s.t, s.n, 16, s.sel, keep_first=1 << 40)
    assert pa.pa_launch_count() == n
