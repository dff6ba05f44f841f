"""Windowed attention with sinks over the pages (paged_attn_window_*), against its definition in
64 bits with a derived elementwise bound (tests/_attn64.py), on both kernels."""
import numpy as np
import pytest

import workloads
from tests import _attn64 as ref64
from tests._gpu import GpuCase, oracle_case

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_pages_gb300 as m
    return m


@pytest.fixture
def min_run(pa):
    old = pa.set_prefill_min_run(16)
    yield pa.set_prefill_min_run
    pa.set_prefill_min_run(old)


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def sinks(Hq, seed=0):
    return (2 * np.random.default_rng([seed, 5]).standard_normal(Hq)).astype(np.float32)


# ------------------------------------------------------------------ CPU

def test_the_plain_definition(pa):
    """A window past the longest row without sinks is the oracle's attention; a sink equal to the
    log of a row's sum halves it; window 1 is the last value."""
    import oracle
    case = workloads.tiny(4)
    _, tpt, kv, _, kp, vp = oracle_case(case, tokens=[])
    got, tol = ref64.window_attention(case.q, kp, vp, tpt, kv, 0.2, 1 << 30)
    np.testing.assert_allclose(got, oracle.paged_attention(case.q, kp, vp, tpt, kv, 0.2),
                               rtol=1e-10, atol=1e-12)
    less, _ = ref64.window_attention(case.q, kp, vp, tpt, kv, 0.2, 30)
    assert (np.abs(less - got) > tol).any()
    last, _ = ref64.window_attention(case.q, kp, vp, tpt, kv, 0.2, 1)
    for t in range(case.T):
        v = ref64.f64(vp[tpt[t][(kv[t] - 1) // case.P], :, (kv[t] - 1) % case.P])
        np.testing.assert_array_equal(last[t], np.repeat(v, case.Hq // case.Hkv, 0))
    t, h = 3, 1
    K = ref64.rows_of(kp, tpt[t], 0, kv[t], case.P, 0)
    lse = np.log(np.exp(0.2 * (K @ ref64.f64(case.q[t, h]))).sum())
    sunk, _ = ref64.window_attention(case.q[t:t + 1], kp, vp, tpt[t:t + 1], kv[t:t + 1], 0.2, 999,
                                     np.full(case.Hq, lse))
    np.testing.assert_allclose(sunk[0, h], got[t, h] / 2, rtol=1e-10)


def test_refusals(pa):
    L = pa.lib()
    A, big = 64, 1 << 40

    def run(q=A, k=A, v=A, t=A, mp=4, kv=A, T=8, Hq=4, Hkv=2, P=16, d=64, N=8, scale=0.1, sink=None,
            out=A, ws=A, size=big, window=None):
        own = [] if window is None else [window]
        fn = L.paged_attn_window_run if window is None else L.paged_attn_window_forward
        return fn(q, k, v, t, mp, kv, T, Hq, Hkv, P, d, N, scale, *own, sink, out, ws, size, None)
    for win in (None, 5):
        for bad in (dict(T=-1), dict(mp=0), dict(t=None), dict(Hq=0)):
            assert run(window=win, **bad) == pa.PA_EINVAL, bad
        for bad in (dict(d=80), dict(P=24), dict(Hq=5), dict(Hq=32)):
            assert run(window=win, **bad) == pa.PA_EUNSUPPORTED, bad
        assert run(window=win, ws=None) == pa.PA_EWORKSPACE
        assert run(window=win, T=0) == pa.PA_OK
    for w in (0, -1):
        assert run(window=w) == pa.PA_EINVAL
        assert L.paged_attn_plan_window(A, 4, A, 8, 4, 2, 16, 64, w, A, big, None) == pa.PA_EINVAL


# ------------------------------------------------------------------ GPU

def check(pa, g, case, r, window, sink=None, what="", tpt=None):
    scale = 1 / np.sqrt(case.d)
    ws = pa.new_workspace(case.T, case.Hq, case.Hkv, case.d)
    got = pa.window_forward(g.q, g.kp, g.vp, g.tpt if tpt is None else tpt, g.kv, scale, window,
                            sink=cuda(sink), workspace=ws)
    err = pa.read_error(ws)
    assert err == 0, hex(err)
    want, tol = ref64.window_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], scale, window,
                                       sink)
    ref64.assert_within(got.cpu().numpy(), want, tol, what)
    return got, ws


def whole(pa, case):
    _, tpt, kv, _, kp, vp = oracle_case(case, tokens=[])
    return GpuCase(pa, case), dict(kp=kp, vp=vp, tpt=tpt, kv=kv)


@pytest.mark.gpu
@pytest.mark.parametrize("route", [16, 1, 10 ** 6])
@pytest.mark.parametrize("window", [1, 5, 16, 40, 1 << 30])
def test_tiny(pa, min_run, route, window):
    min_run(route)
    case = workloads.tiny(1)
    g, r = whole(pa, case)
    check(pa, g, case, r, window, what="no sink")
    if window == 1 << 30:  # a window that no int32 holds is "all" too
        check(pa, g, case, r, (1 << 33) + 5, what="wide")
        with pytest.raises(pa.PagedAttnError) as e:
            check(pa, g, case, r, 5 - (1 << 33), what="negative")
        assert e.value.status == pa.PA_EINVAL
    check(pa, g, case, r, window, sinks(case.Hq), what="sink")


@pytest.mark.gpu
@pytest.mark.parametrize("route", [16, 1, 10 ** 6])
@pytest.mark.parametrize("P,d,Hq,Hkv,window", [
    (16, 64, 2, 2, 1), (16, 64, 8, 1, 77), (32, 128, 4, 2, 128), (64, 64, 4, 2, 129),
    (128, 128, 8, 2, 255), (16, 128, 4, 4, 300), (128, 64, 8, 1, 3), (32, 128, 8, 1, 640),
])
def test_ragged_chunks_and_single_tokens(pa, min_run, route, P, d, Hq, Hkv, window):
    min_run(route)
    case = workloads.small_prefill(P + d + Hq, P=P, d=d, Hq=Hq, Hkv=Hkv,
                                   chunks=((0, 130, 141), (1, 0, 33), (2, 500, 1)), extra_decode=5)
    g, r = whole(pa, case)
    check(pa, g, case, r, window, sinks(Hq) if window % 2 else None, what=f"route {route}")


@pytest.mark.gpu
def test_a_window_past_every_row_is_plain_attention(pa):
    """Nothing of the window is left: paged_attn_forward's rows, within the two roundings that
    each kernel may take (the two plans cut the work at different places)."""
    case = workloads.small_prefill(31, P=32, d=128, Hq=8, Hkv=2, extra_decode=4)
    g, r = whole(pa, case)
    got, _ = check(pa, g, case, r, case.max_pages * case.P)
    want, tol = ref64.window_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"],
                                       1 / np.sqrt(128), 1 << 30)
    plain = g.forward(pa).double().cpu().numpy()
    assert (np.abs(got.double().cpu().numpy() - plain) <= 2 * tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("route", [16, 1, 10 ** 6])
@pytest.mark.parametrize("P", [16, 128])
def test_pages_before_the_window_are_gone(pa, min_run, route, P):
    """Table entries before every token's window may be anything, cells before it may hold NaN
    or infinities, and the result is the same."""
    min_run(route)
    case = workloads.build_case("gone", 12, [900, 2000, 333],
                                [(0, p) for p in range(780, 900)] + [(1, 1999), (2, 332)], P=P,
                                Hq=4, Hkv=2, d=64)
    g, r = whole(pa, case)
    window = 201
    tpt = g.tpt.clone()
    first = {0: 780 + 1 - window, 1: 2000 - window, 2: 333 - window}
    for t in range(case.T):
        s = int(case.tok_seq[t])
        tpt[t, :first[s] // P] = [-1, 10 ** 9, -(2 ** 31)][s]
        for p in range(first[s]):
            pg, bad = int(r["tpt"][t][p // P]), [float("nan"), float("inf"), -65504.0][p % 3]
            if t == list(case.tok_seq).index(s):
                g.kp[pg, :, p % P] = bad
                g.vp[pg, :, p % P] = bad
    check(pa, g, case, r, window, sinks(4), tpt=tpt)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (4, 2)])
def test_rows_split_over_many_parts(pa, Hq, Hkv):
    lens = [9020, 12000, 3, 700]
    tokens = [(0, p) for p in range(9000, 9020)] + [(s, lens[s] - 1) for s in (1, 2, 3)]
    case = workloads.build_case("split", 5, lens, tokens, P=64, Hq=Hq, Hkv=Hkv, d=128)
    g, r = whole(pa, case)
    for window in (500, 8001):
        sink = sinks(Hq)
        a, ws = check(pa, g, case, r, window, sink)
        for _ in range(3):
            b = pa.window_run(g.q, g.kp, g.vp, g.tpt, g.kv, 1 / np.sqrt(128), sink=cuda(sink),
                              workspace=ws)
            assert torch.equal(a, b)
        assert pa.read_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("route", [16, 1, 10 ** 6])
def test_extreme_sinks_and_empty_rows(pa, min_run, route):
    """-inf: no sink; +inf or far above every score: a zero row; the lowest value: no sink; empty
    rows stay zero under any sink, and rows behind the last token are not touched."""
    min_run(route)
    case = workloads.build_case("ext", 13, [60, 300], [(0, p) for p in range(40, 60)] + [(-1, 0)] * 18
                                + [(1, 299), (-1, 0)], P=16, Hq=8, Hkv=2, d=64)
    g, r = whole(pa, case)
    low = np.finfo(np.float32).min
    sink = np.array([-np.inf, np.inf, 1e4, low, 0, 3e38, -1e4, 88.5], np.float32)
    buf = torch.full((case.T + 2, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    ws = pa.new_workspace(case.T, 8, 2, 64)
    got = pa.window_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.125, 33, sink=cuda(sink),
                            out=buf[:case.T], workspace=ws)
    assert pa.read_error(ws) == 0
    want, tol = ref64.window_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.125, 33, sink)
    ref64.assert_within(got.cpu().numpy(), want, tol)
    assert buf[case.T:].eq(7).all() and buf[20:38].eq(0).all() and buf[39].eq(0).all()
    assert got[:, 1].eq(0).all() and got[:, 2].eq(0).all()


@pytest.mark.gpu
def test_foreign_plans_and_bad_pages_are_flagged(pa):
    case = workloads.small_prefill(9, P=16, d=64, Hq=4, Hkv=2, chunks=((0, 60, 40),), extra_decode=2)
    g, r = whole(pa, case)
    ws = pa.new_workspace(case.T, 4, 2, 64)
    out = torch.full_like(g.q, 3.0)
    args = (g.q, g.kp, g.vp, g.tpt, g.kv, 0.2)
    pa.plan(g.tpt, g.kv, 4, 2, 16, 64, ws)
    pa.window_run(*args, out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    pa.plan_window(g.tpt, g.kv, 4, 2, 16, 64, 21, ws)
    pa.prefill(*args, out, ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    wider = torch.nn.functional.pad(g.tpt, (0, 3), value=-1)     # a plan of other sizes
    pa.plan_window(wider, g.kv, 4, 2, 16, 64, 21, ws)
    pa.window_run(*args, out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    tpt = g.tpt.clone()
    tpt[:40, 5] = case.num_pages                     # positions 80..95: inside the windows
    pa.window_forward(*args[:3], tpt, *args[4:], 21, out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PAGE_RANGE
    pa.window_forward(*args, 21, out=out, workspace=ws)
    assert pa.read_error(ws) == 0
    want, tol = ref64.window_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.2, 21)
    ref64.assert_within(out.cpu().numpy(), want, tol)


@pytest.mark.gpu
def test_binding_refusals(pa):
    case = workloads.tiny(2)
    g = GpuCase(pa, case)
    ok = [g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, 9]
    for i, bad in ((0, g.q.float()), (1, g.kp.cpu()), (2, g.vp[:, :1]), (3, g.tpt.long()),
                   (4, g.kv[:-1])):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            pa.window_forward(*args)
    with pytest.raises(ValueError):
        pa.window_forward(*ok, sink=torch.zeros(case.Hq + 1, device="cuda"))
    with pytest.raises(ValueError):
        pa.window_run(*ok[:6])
    for bad in (0, -3):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.window_forward(*ok[:6], bad)
        assert e.value.status == pa.PA_EINVAL
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.window_forward(*ok[:5], scale, 9)
        assert e.value.status == pa.PA_EINVAL
    odd = torch.empty(g.q.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(g.q)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.window_forward(odd, *ok[1:])
    assert e.value.status == pa.PA_EALIGN
