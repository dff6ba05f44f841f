"""Differential attention over the pages (paged_attn_diff_*), against its definition in 64 bits
with a derived elementwise bound (tests/_attn64.py), on both kernels and every split."""
import numpy as np
import pytest

import oracle
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
    """set_prefill_min_run for one test."""
    old = pa.set_prefill_min_run(16)
    yield pa.set_prefill_min_run
    pa.set_prefill_min_run(old)


def params(seed, Hq, d, norm=True):
    rng = np.random.default_rng([seed, 77])
    lam = rng.uniform(0.05, 1.1, Hq).astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32) if norm else None
    return lam, w, 1e-5, 0.2 if norm else 1.0


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ CPU

def test_the_plain_definition(pa):
    """The 64-bit form equals two of the oracle's attentions over halved rows, and its norm and
    weights the closed form; a swapped or dropped map breaks it."""
    case = workloads.tiny(3)
    _, tpt, kv, _, kp, vp = oracle_case(case, tokens=[])
    lam, w, eps, c = params(3, case.Hq, case.d)
    scale, e = 0.21, case.d // 2
    got, tol = ref64.diff_attention(case.q, kp, vp, tpt, kv, scale, lam)
    halves = []
    for i in (0, e):  # zero the other half of q: its keys then add nothing to a score
        q = case.q.copy()
        q[..., (e if i == 0 else 0):(case.d if i == 0 else e)] = 0
        halves.append(oracle.paged_attention(q, kp, vp, tpt, kv, scale))
    want = halves[0] - lam[None, :, None].astype(np.float64) * halves[1]
    np.testing.assert_allclose(got, want, rtol=1e-10, atol=1e-12)
    assert (np.abs(halves[1] - lam[None, :, None] * halves[0] - want) > tol).any()
    assert (np.abs(halves[0] - want) > tol).any()
    normed, _ = ref64.diff_attention(case.q, kp, vp, tpt, kv, scale, lam, w, eps, c)
    rms = np.sqrt((want ** 2).mean(-1, keepdims=True) + eps)
    np.testing.assert_allclose(normed, c * want / rms * w.astype(np.float64), rtol=1e-9)


def test_refusals(pa):
    L = pa.lib()
    A = 64  # any aligned address: nothing is launched by a refused call
    big = 1 << 40

    def run(fn="paged_attn_diff_run", q=A, k=A, v=A, t=A, mp=4, kv=A, T=8, Hq=4, Hkv=2, P=16, d=64,
            N=8, scale=0.1, lam=A, w=None, eps=1e-5, c=1.0, out=A, ws=A, size=big):
        return getattr(L, fn)(q, k, v, t, mp, kv, T, Hq, Hkv, P, d, N, scale, lam, w, eps, c, out,
                              ws, size, None)
    for fn in ("paged_attn_diff_run", "paged_attn_diff_forward"):
        for bad in (dict(T=-1), dict(mp=0), dict(t=None), dict(Hq=0)):
            assert run(fn, **bad) == pa.PA_EINVAL, bad
        for bad in (dict(d=80), dict(P=24), dict(Hq=5), dict(Hq=32)):
            assert run(fn, **bad) == pa.PA_EUNSUPPORTED, bad
        assert run(fn, ws=None) == pa.PA_EWORKSPACE
        assert run(fn, T=0) == pa.PA_OK


def test_workspace(pa):
    assert pa.diff_workspace_size(8, 4, 2, 64) >= pa.workspace_size(8, 4, 2, 64)
    assert pa.diff_workspace_size(8, 64, 8, 128) > 0      # a group of eight heads
    assert pa.diff_workspace_size(8, 4, 2, 80) == 0
    assert pa.diff_workspace_size(8, 6, 4, 64) == 0


# ------------------------------------------------------------------ GPU

def check(pa, g, case, seed, norm=True, what="", kp=None, vp=None, tpt=None, kv=None, out=None):
    lam, w, eps, c = params(seed, case.Hq, case.d, norm)
    scale = 1 / np.sqrt(case.d / 2)
    ws = pa.new_diff_workspace(case.T, case.Hq, case.Hkv, case.d)
    got = pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, scale, cuda(lam), cuda(w), eps, c, out=out,
                          workspace=ws)
    err = pa.read_error(ws)
    assert err == 0, hex(err)
    want, tol = ref64.diff_attention(case.q, kp, vp, tpt, kv, scale, lam, w, eps, c)
    ref64.assert_within(got.cpu().numpy(), want, tol, what)
    return got, ws


def whole(pa, case):
    _, tpt, kv, _, kp, vp = oracle_case(case, tokens=[])
    return GpuCase(pa, case), dict(kp=kp, vp=vp, tpt=tpt, kv=kv)


@pytest.mark.gpu
@pytest.mark.parametrize("route", [16, 1, 10 ** 6])
def test_tiny(pa, min_run, route):
    min_run(route)
    case = workloads.tiny(1)
    g, r = whole(pa, case)
    check(pa, g, case, 1, what=f"route {route}", **r)


@pytest.mark.gpu
@pytest.mark.parametrize("route", [16, 1, 10 ** 6])
@pytest.mark.parametrize("P,d,Hq,Hkv", [(16, 64, 2, 2), (128, 128, 4, 2), (32, 128, 8, 2),
                                        (64, 64, 8, 1), (16, 128, 8, 1), (128, 64, 4, 4)])
def test_ragged_chunks_and_single_tokens(pa, min_run, route, P, d, Hq, Hkv):
    min_run(route)
    case = workloads.small_prefill(P + d + Hq, P=P, d=d, Hq=Hq, Hkv=Hkv,
                                   chunks=((0, 130, 141), (1, 0, 33), (2, 500, 1)), extra_decode=5)
    g, r = whole(pa, case)
    check(pa, g, case, P + Hq, norm=Hq != 4, what=f"P {P} d {d} {Hq}/{Hkv} route {route}", **r)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (4, 2)])
def test_rows_split_over_many_parts(pa, Hq, Hkv):
    """Few rows over long contexts: every row of keys is cut over CTAs, on both kernels (a chunk
    of 20 tokens at position 9000, single tokens over 12000 and 3 keys)."""
    lens = [9020, 12000, 3, 700]
    tokens = [(0, p) for p in range(9000, 9020)] + [(s, lens[s] - 1) for s in (1, 2, 3)]
    case = workloads.build_case("split", 5, lens, tokens, P=64, Hq=Hq, Hkv=Hkv, d=128)
    g, r = whole(pa, case)
    a, ws = check(pa, g, case, 5, what="split", **r)
    lam, w, eps, c = params(5, Hq, 128)
    for _ in range(3):  # the arrival counters of the plan serve every later run, same bits
        b = pa.diff_run(g.q, g.kp, g.vp, g.tpt, g.kv, 1 / np.sqrt(64), cuda(lam), cuda(w), eps, c,
                        workspace=ws)
        assert torch.equal(a, b)
    assert pa.read_error(ws) == 0


@pytest.mark.gpu
def test_empty_rows_and_padding(pa, min_run):
    """Rows without keys are zero (with and without a norm) on both kernels; rows behind the
    ubatch's last token are left as they were."""
    case = workloads.build_case("pad", 6, [40, 300], [(0, p) for p in range(20, 40)] + [(-1, 0)] * 19
                                + [(1, 299), (-1, 0)], P=16, Hq=4, Hkv=2, d=64)
    g, r = whole(pa, case)
    for route in (16, 1, 10 ** 6):
        min_run(route)
        for norm in (True, False):
            buf = torch.full((case.T + 3, case.Hq, case.d), 7.0, dtype=torch.float16, device="cuda")
            check(pa, g, case, 6, norm, out=buf[:case.T], what=f"{route} {norm}", **r)
            assert buf[case.T:].eq(7).all() and buf[20:39].eq(0).all() and buf[40].eq(0).all()


@pytest.mark.gpu
def test_one_key_and_equal_maps(pa):
    """One key: both maps are 1, y = (1 - lam) v.  Equal maps with lam = 1: y is 0, and the norm's
    epsilon keeps it 0."""
    case = workloads.build_case("one", 7, [1, 1, 400], [(0, 0), (1, 0), (2, 399)], P=16, Hq=2, Hkv=1,
                                d=64)
    g, r = whole(pa, case)
    half = case.d // 2
    g.q[..., half:] = g.q[..., :half]
    g.kp[..., half:] = g.kp[..., :half]
    one = torch.ones(2, device="cuda")
    for w in (None, torch.ones(64, device="cuda")):
        y = pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, one, w)
        assert y.eq(0).all()
    y = pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, one * 0.25)
    v = ref64.f64(r["vp"][r["tpt"][0][0], 0, 0])
    np.testing.assert_allclose(y[0].double().cpu().numpy(), np.tile(0.75 * v, (2, 1)), rtol=2 ** -10)


@pytest.mark.gpu
def test_pages_past_two_gigabytes_of_elements(pa):
    """A pool whose last pages lie past 2^31 elements and 2^32 bytes."""
    case = workloads.build_case("far", 8, [700, 520], [(0, p) for p in range(660, 700)] + [(1, 519)],
                                P=128, Hq=8, Hkv=8, d=128)
    _, tpt, kv, _, kp, vp = oracle_case(case, tokens=[])
    N = 2 ** 31 // (8 * 128 * 128) + 40
    far = torch.empty((2, N, 8, 128, 128), dtype=torch.float16, device="cuda")
    used = np.unique(tpt[tpt >= 0])
    to = N - 1 - np.arange(case.num_pages)
    for x, p in ((far[0], kp), (far[1], vp)):
        x[torch.from_numpy(to[used]).cuda()] = torch.from_numpy(p[used].view(np.float16)).cuda()
    lam, w, eps, c = params(8, 8, 128)
    t2 = np.where(tpt >= 0, to[np.maximum(tpt, 0)], -1).astype(np.int32)
    got = pa.diff_forward(cuda(case.q.view(np.float16)), far[0], far[1], cuda(t2), cuda(kv), 0.125,
                          cuda(lam), cuda(w), eps, c)
    want, tol = ref64.diff_attention(case.q, kp, vp, tpt, kv, 0.125, lam, w, eps, c)
    ref64.assert_within(got.cpu().numpy(), want, tol)


@pytest.mark.gpu
def test_bad_pages_and_foreign_plans_are_flagged(pa):
    case = workloads.small_prefill(9, P=16, d=64, Hq=4, Hkv=2, chunks=((0, 60, 40),), extra_decode=2)
    g, r = whole(pa, case)
    lam, w, eps, c = params(9, 4, 64)
    args = (g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, cuda(lam), cuda(w), eps, c)
    ws = pa.new_diff_workspace(case.T, 4, 2, 64)
    out = torch.full_like(g.q, 3.0)
    pa.plan(g.tpt, g.kv, 4, 2, 16, 64, ws)                       # another operator's plan
    pa.diff_run(*args, out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    pa.plan_window(g.tpt, g.kv, 4, 2, 16, 64, 7, ws)
    pa.diff_run(*args, out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    pa.plan_diff(g.tpt, g.kv, 4, 2, 16, 64, ws)                  # and the other way round
    pa.prefill(g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, out, ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    pa.plan_diff(g.tpt[:-1], g.kv[:-1], 4, 2, 16, 64, ws)        # one of other sizes
    pa.diff_run(*args, out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PLAN and out.eq(3).all()
    tpt = g.tpt.clone()
    tpt[:, 1] = case.num_pages + 5
    pa.diff_forward(*args[:3], tpt, *args[4:], out=out, workspace=ws)
    assert pa.read_error(ws) == pa.PA_ERR_PAGE_RANGE
    pa.diff_forward(*args, out=out, workspace=ws)                # and the context goes on
    assert pa.read_error(ws) == 0
    want, tol = ref64.diff_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.2, lam, w, eps, c)
    ref64.assert_within(out.cpu().numpy(), want, tol)


@pytest.mark.gpu
def test_binding_refusals(pa):
    case = workloads.tiny(2)
    g = GpuCase(pa, case)
    lam = torch.ones(case.Hq, device="cuda")
    ok = [g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, lam]
    for i, bad in ((0, g.q.float()), (0, g.q.transpose(0, 1)), (1, g.kp.cpu()), (2, g.vp[:, :1]),
                   (3, g.tpt.long()), (4, g.kv[:-1]), (6, lam.half()), (6, lam[:-1])):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            pa.diff_forward(*args)
    with pytest.raises(ValueError):
        pa.diff_forward(*ok, norm_weight=torch.ones(case.d + 1, device="cuda"))
    with pytest.raises(ValueError):
        pa.diff_run(*ok)
    with pytest.raises(ValueError):
        pa.diff_forward(*ok[:6], None)
    inf, nan = float("inf"), float("nan")
    for scale in (0.0, -1.0, inf, nan):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.diff_forward(*ok[:5], scale, lam)
        assert e.value.status == pa.PA_EINVAL
    for eps in (-1.0, nan):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.diff_forward(*ok, norm_weight=torch.ones(case.d, device="cuda"), eps=eps)
        assert e.value.status == pa.PA_EINVAL
    ws = pa.new_diff_workspace(case.T, case.Hq, case.Hkv, case.d)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.diff_forward(*ok, workspace=ws[:-256])
    assert e.value.status == pa.PA_EWORKSPACE
    odd = torch.empty(g.q.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(g.q)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.diff_forward(odd, *ok[1:])
    assert e.value.status == pa.PA_EALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_error_of_the_tiles(pa, d):
    """The error's norm is what two roundings leave.  A rounding to binary16 is off by a uniform
    share of half a step, so by 2^-11 / sqrt(3) of 1 / the mantissa; over mantissas spread evenly
    in their logarithm the mean square of that is 2^-22 / 3 * 0.75 / (2 ln 2).  P's rounding adds
    it times (p v)^2 for each key of each map, but for the first 32 of a block of 128, whose
    low part the products take; the output's adds it times y^2.  5% for the sample."""
    case = workloads.small_prefill(35, P=16, d=d, Hq=4, Hkv=2, chunks=((0, 400, 181),),
                                   extra_decode=0)
    g, r = whole(pa, case)
    lam, e, scale = params(35, 4, d)[0], d // 2, 1 / np.sqrt(d // 2)
    got = pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, scale, cuda(lam)).cpu().numpy()
    q, step2 = ref64.f64(case.q), 2.0 ** -22 / 3 * 0.75 / (2 * np.log(2))
    off = of_p = of_y = 0.0
    for t in range(case.T):
        for kv_head in range(2):
            K, V = (ref64.rows_of(p, r["tpt"][t], 0, r["kv"][t], 16, kv_head)
                    for p in (r["kp"], r["vp"]))
            h = slice(2 * kv_head, 2 * kv_head + 2)
            a1, a2 = (ref64.weighted(q[t, h, i:i + e], K[:, i:i + e], np.eye(len(K)), scale)[0]
                      for i in (0, e))
            a2 = a2 * lam[h, None]
            y = (a1 - a2) @ V
            rounded = np.arange(len(K)) % 128 >= 32
            of_p += step2 * (((a1 ** 2 + a2 ** 2) * rounded) @ (V ** 2)).sum()
            of_y += step2 * (y ** 2).sum()
            off += ((got[t, h].astype(np.float64) - y) ** 2).sum()
    assert off <= 1.05 ** 2 * (of_p + of_y), (off, of_p, of_y)
    assert of_p < 1.2 * of_y  # P's rounding weighs about what the output's does


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["diff", "window"])
def test_waits_that_give_up_end_the_launch(pa, kind):
    """With a limit of 1 us the split-KV launch's waits give up: the call ends with
    PA_ERR_TIMEOUT (small cases, beside a prefill of 120 tokens and without one, may end in
    time: a CTA has a block or two), and the next call at the usual limit is right."""
    def run(case, g, ws):
        if kind == "diff":
            lam, w, eps, c = params(33, case.Hq, 128)
            return pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.125, cuda(lam), cuda(w), eps,
                                   c, workspace=ws)
        return pa.window_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.125, 2222, workspace=ws)

    def short_of_time(case, g, ws):
        old = pa.set_decode_wait_limit(1000)
        try:
            run(case, g, ws)
            return pa.read_error(ws)
        finally:
            pa.set_decode_wait_limit(old)

    for chunks in (((0, 500, 120),), ()):
        case = workloads.small_prefill(33, P=16, d=128, Hq=4, Hkv=2, chunks=chunks, extra_decode=6)
        g, r = whole(pa, case)
        lam, w, eps, c = params(33, 4, 128)
        ws = pa.new_diff_workspace(case.T, 4, 2, 128)
        assert short_of_time(case, g, ws) in (0, pa.PA_ERR_TIMEOUT)
        y = run(case, g, ws)
        assert pa.read_error(ws) == 0
        want, tol = (ref64.diff_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.125, lam, w,
                                          eps, c) if kind == "diff" else
                     ref64.window_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.125,
                                            2222))
        ref64.assert_within(y.cpu().numpy(), want, tol, kind)
    case = workloads.decode(0)
    g = GpuCase(pa, case)
    ws = pa.new_diff_workspace(case.T, case.Hq, case.Hkv, 128)
    y = run(case, g, ws)
    assert pa.read_error(ws) == 0
    assert short_of_time(case, g, ws) == pa.PA_ERR_TIMEOUT
    assert torch.equal(run(case, g, ws), y) and pa.read_error(ws) == 0


@pytest.mark.gpu
def test_buffers_made_by_a_call_on_another_stream(pa):
    """No output and no workspace given, on another stream than the current one, while the
    current one allocates: the call's buffers are not handed out again under it."""
    case = workloads.small_prefill(34, P=16, d=64, Hq=4, Hkv=2, chunks=((0, 400, 90),))
    g, r = whole(pa, case)
    lam, w, eps, c = params(34, 4, 64)
    dl, dw, s = cuda(lam), cuda(w), torch.cuda.Stream()
    want, tol = ref64.diff_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.2, lam, w, eps, c)
    torch.cuda.synchronize()
    ys = []
    for _ in range(10):
        ys.append(pa.diff_forward(g.q, g.kp, g.vp, g.tpt, g.kv, 0.2, dl, dw, eps, c, stream=s))
        junk = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
        del junk
    torch.cuda.synchronize()
    for y in ys:
        ref64.assert_within(y.cpu().numpy(), want, tol)


@pytest.mark.gpu
def test_two_graphs_share_a_workspace_on_another_stream(pa):
    """Two captured steps of different ubatches in one workspace, replayed in turn."""
    s = torch.cuda.Stream()
    cases = [workloads.small_prefill(20 + i, P=16, d=128, Hq=4, Hkv=2,
                                     chunks=((0, 30 * i, 60 + 50 * i),), extra_decode=3) for i in (0, 1)]
    made = [whole(pa, c) for c in cases]
    ws = pa.new_diff_workspace(max(c.T for c in cases), 4, 2, 128)
    lam, w, eps, c = params(20, 4, 128)
    dl, dw = cuda(lam), cuda(w)
    outs, graphs = [torch.zeros_like(g.q) for g, _ in made], []
    torch.cuda.synchronize()
    for (g, _), o in zip(made, outs):
        args = (g.q, g.kp, g.vp, g.tpt, g.kv, 0.125, dl, dw, eps, c)
        with torch.cuda.stream(s):
            pa.diff_forward(*args, out=o, workspace=ws)
        s.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            pa.diff_forward(*args, out=o, workspace=ws)
    with torch.cuda.stream(s):
        for o in outs:
            o.zero_()
        for _ in range(3):
            for gr in graphs:
                gr.replay()
    s.synchronize()
    assert pa.read_error(ws) == 0
    for (g, r), case, o in zip(made, cases, outs):
        want, tol = ref64.diff_attention(case.q, r["kp"], r["vp"], r["tpt"], r["kv"], 0.125, lam, w,
                                         eps, c)
        ref64.assert_within(o.cpu().numpy(), want, tol)
