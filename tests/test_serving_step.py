"""The operators of a serving step run together, as a scheduler would: the step's tables built
from request lengths on the GPU, the new rows appended, then the plain, the differential and the
windowed attention over the same pages -- captured once and replayed while requests arrive, grow,
finish and start again, against 64-bit definitions over each request's contiguous K/V."""
import numpy as np
import pytest

import workloads
from tests import _attn64 as ref64
from tests.test_batch_build import host_step

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_pages_gb300 as m
    return m


class Requests:
    """Each request's contiguous K and V (binary16 bits), and a pool laid out one after the other
    for the 64-bit reference."""

    def __init__(self, n, cap, Hkv, d):
        self.kv = np.zeros((2, n, cap, Hkv, d), np.uint16)

    def pools(self, P):
        _, n, cap, Hkv, d = self.kv.shape
        x = self.kv.reshape(2, n * (cap // P), P, Hkv, d).transpose(0, 1, 3, 2, 4)
        return np.ascontiguousarray(x), np.arange(n * (cap // P)).reshape(n, cap // P)


@pytest.mark.parametrize("P,d,Hq,Hkv", [(16, 64, 4, 2), (32, 128, 2, 2)])
def test_captured_serving_steps(pa, P, d, Hq, Hkv):
    rng = np.random.default_rng([P, d])
    n, max_pages, N, T, window = 7, 160 // P, 90, 96, 37
    cap, scale = max_pages * P, 1 / np.sqrt(d)
    dev = "cuda"
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    table, ln, nw, ref = i32(n, max_pages).fill_(-1), i32(n), i32(n), i32(N)
    err = i32(1)
    out = pa.new_batch(n, max_pages, T)._replace(seq_len=ln)
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16, device=dev)  # noqa: E731
    nan = float("nan")
    kp, vp = f16(N, Hkv, P, d).fill_(nan), f16(N, Hkv, P, d).fill_(nan)  # unwritten cells
    q, k, v = f16(T, Hq, d), f16(T, Hkv, d), f16(T, Hkv, d)
    y = [f16(T, Hq, d) for _ in range(3)]
    lam = torch.linspace(0.1, 0.9, Hq, device=dev)
    w = torch.linspace(0.5, 1.5, d, device=dev)
    sink = torch.linspace(-1, 2, Hq, device=dev)
    ws, wd, ww = (pa.new_workspace(T, Hq, Hkv, d), pa.new_diff_workspace(T, Hq, Hkv, d),
                  pa.new_workspace(T, Hq, Hkv, d))

    def step():
        pa.batch_build(table, ln, nw, ref, P, T, out=out, err=err)
        pa.kv_append(k, v, out.slot_mapping, kp, vp, err=err)
        args = (q, kp, vp, out.tok_page_table, out.tok_kv_len, scale)
        pa.forward(*args, out=y[0], workspace=ws)
        pa.diff_forward(*args, lam, w, 1e-5, 0.3, out=y[1], workspace=wd)
        pa.window_forward(*args, window, sink, out=y[2], workspace=ww)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # an empty step: every token is padding
    s.synchronize()
    assert all(x.eq(0).all() for x in y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()

    req = Requests(n, cap, Hkv, d)
    h_table, h_len, h_ref = (table.cpu().numpy(), np.zeros(n, np.int32), np.zeros(N, np.int32))
    both = {0: 0, 1: 0}
    for it in range(10):
        # a prompt's chunk for some requests, one token for the others; some have finished
        new = np.where(h_len == 0, rng.integers(0, 60, n), 1)
        new[(h_len > 100) & (rng.random(n) < 0.5)] = -1
        new = np.minimum(new, cap - h_len).astype(np.int32)
        hq = workloads.randn_f16(rng, (T, Hq, d))
        hk, hv = workloads.randn_f16(rng, (T, Hkv, d)), workloads.randn_f16(rng, (T, Hkv, d))
        want = host_step(h_table, h_len, new, h_ref, P, T)
        with torch.cuda.stream(s):
            nw.copy_(torch.from_numpy(new))
            for x, h in ((q, hq), (k, hk), (v, hv)):
                x.copy_(torch.from_numpy(h.view(np.float16)))
            err.zero_()
            graph.replay()
        s.synchronize()
        assert int(err.item()) == want[-1]
        assert [pa.read_error(x) for x in (ws, wd, ww)] == [0, 0, 0]
        tok_seq, tok_pos, kv = want[4], want[5], want[7]
        for got, exp in zip((table, ref) + tuple(out), want):
            assert np.array_equal(got.cpu().numpy(), exp)
        real = np.flatnonzero(tok_seq >= 0)
        req.kv[0, tok_seq[real], tok_pos[real]] = hk[real]
        req.kv[1, tok_seq[real], tok_pos[real]] = hv[real]
        (rk, rv), rows = req.pools(P)
        tpt = rows[np.maximum(tok_seq, 0)]
        big = np.full(T, 1 << 30)
        for i, (r, tol) in enumerate((
                ref64.window_attention(hq, rk, rv, tpt, kv, scale, int(big[0])),
                ref64.diff_attention(hq, rk, rv, tpt, kv, scale, lam.cpu().numpy(),
                                     w.cpu().numpy(), 1e-5, 0.3),
                ref64.window_attention(hq, rk, rv, tpt, kv, scale, window, sink.cpu().numpy()))):
            ref64.assert_within(y[i].cpu().numpy(), r, tol, f"step {it}, attention {i}")
        counts = np.bincount(tok_seq[real], minlength=n)
        both[0] += int((counts >= 16).any())
        both[1] += int((counts == 1).any())
        h_table, h_ref, h_len = want[0], want[1], want[3]
    assert both[0] and both[1]  # tiles and single tokens both ran


def test_two_streams_at_once(pa):
    """Runs of two ubatches on two streams, each with its own workspace, interleaved."""
    cases = [workloads.small_prefill(50 + i, P=16, d=64, Hq=4, Hkv=2,
                                     chunks=((0, 200 * i, 90 + 70 * i),), extra_decode=4) for i in (0, 1)]
    from tests._gpu import GpuCase, oracle_case
    made = []
    for c in cases:
        _, tpt, kv, _, kp, vp = oracle_case(c, tokens=[])
        made.append((GpuCase(pa, c), ref64.diff_attention(c.q, kp, vp, tpt, kv, 0.2,
                                                          np.linspace(0.2, 0.8, 4, dtype=np.float32))))
    lam = torch.from_numpy(np.linspace(0.2, 0.8, 4, dtype=np.float32)).cuda()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(g.q) for g, _ in made]
    wss = [pa.new_diff_workspace(c.T, 4, 2, 64) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, _), o, ws in zip(streams, made, outs, wss):
            pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, lam, out=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (_, (want, tol)), o, ws in zip(made, outs, wss):
        assert pa.read_error(ws) == 0
        ref64.assert_within(o.cpu().numpy(), want, tol)
