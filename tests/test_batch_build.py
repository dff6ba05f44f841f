"""paged_batch_build: a step's tables from request lengths, against a plain host model that
takes and returns its pages through the host pool (pa_pool_*).  Everything is a whole number,
so every comparison is exact."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_pages_gb300 as m
    return m


# ------------------------------------------------------------------ the host model

def host_step(table, length, new, ref, P, T):
    """The step by its definition, request by request, on copies.  Returns (table, ref, q_start,
    seq_len, tok_seq, tok_pos, tok_page_table, tok_kv_len, slot_mapping, err bits)."""
    table, ref, length = table.copy(), ref.copy(), length.astype(np.int64)
    n, max_pages = table.shape
    err = 0
    for i in range(n):
        if new[i] >= 0:
            continue
        for c in range(max_pages):
            pg = table[i, c]
            if pg < 0:
                continue
            table[i, c] = -1
            if pg >= len(ref):
                err |= 0x1
            elif ref[pg] <= 0:
                err |= 0x40
            else:
                ref[pg] -= 1
    free = list(np.flatnonzero(ref == 0))
    q_start, seq, pos, stop = [0], [], [], False
    out_len = length.copy()
    for i in range(n):
        k = int(new[i])
        if k < 0:
            out_len[i] = 0
        if k > 0:
            if length[i] < 0 or length[i] + k > max_pages * P:
                err |= 0x10
            else:
                a, b = -(-length[i] // P), -(-(length[i] + k) // P)
                stop = stop or b - a > len(free) or len(seq) + k > T
                if not stop:
                    for c in range(a, b):
                        table[i, c] = free.pop(0)
                        ref[table[i, c]] = 1
                    seq += [i] * k
                    pos += range(length[i], length[i] + k)
                    out_len[i] += k
                else:
                    err |= 0x20
        q_start.append(len(seq))
    tpt = np.full((T, max_pages), -1, np.int32)
    slot = np.full(T, -1, np.int64)
    kv = np.zeros(T, np.int32)
    for t, (s, p) in enumerate(zip(seq, pos)):
        tpt[t] = table[s]
        kv[t] = p + 1
        pg = table[s, p // P]
        slot[t] = -1 if pg < 0 else int(pg) * P + p % P
    fill = T - len(seq)
    i32 = lambda x: np.array(x, np.int32)  # noqa: E731
    return (table, ref, i32(q_start), i32(out_len), i32(seq + [-1] * fill), i32(pos + [0] * fill),
            tpt, kv, slot, err)


def make(rng, n, P, max_pages, num_pages, p_new=0.6, p_end=0.15, share=0.1, chunk=40):
    """Random requests over a pool: (table, len, new, ref)."""
    cap = max_pages * P
    length = rng.integers(0, cap + 1, n)
    table = np.full((n, max_pages), -1, np.int32)
    ref = np.zeros(num_pages, np.int32)
    perm = rng.permutation(num_pages)
    at = 0
    for i in range(n):
        k = -(-int(length[i]) // P)
        if at + k > num_pages * 3 // 4:
            length[i] = 0
            continue
        table[i, :k] = perm[at:at + k]
        ref[perm[at:at + k]] = 1
        at += k
    live = np.flatnonzero(ref)
    ref[live[rng.random(len(live)) < share]] += 1
    new = np.where(rng.random(n) < p_new, rng.integers(0, chunk + 1, n), rng.integers(0, 2, n))
    new = np.minimum(new, cap - length)
    new[rng.random(n) < p_end] = -1
    return table, length.astype(np.int32), new.astype(np.int32), ref


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def check(pa, table, length, new, ref, P, T, alias=False):
    want = host_step(table, length, new, ref, P, T)
    t, ln, nw, rf = dev(table, length, new, ref)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.new_batch(len(new), table.shape[1], T)
    for x in out:
        x.fill_(-77)
    if alias:
        out = out._replace(seq_len=ln)
    pa.batch_build(t, ln, nw, rf, P, T, out=out, err=err)
    torch.cuda.synchronize()
    for name, g, w in zip(("seq_page_table", "page_ref") + pa.Batch._fields, (t, rf) + tuple(out),
                          want):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(err.item()) == want[-1]
    return want


# ------------------------------------------------------------------ CPU

def test_host_model_agrees_with_the_host_pool(pa):
    """The model hands out and takes back the pages that pa_pool_alloc / _release would."""
    rng = np.random.default_rng(3)
    P, max_pages, n = 4, 6, 9
    pool = pa.PagePool(40)
    table = np.full((n, max_pages), -1, np.int32)
    ref, length = np.zeros(40, np.int32), np.zeros(n, np.int32)
    for step in range(30):
        new = np.minimum(rng.integers(0, 4, n), max_pages * P - length).astype(np.int32)
        new[rng.random(n) < 0.1] = -1
        T = int(np.maximum(new, 0).sum())
        for i in np.flatnonzero(new < 0):
            pool.release([int(x) for x in table[i] if x >= 0])
        want = {i: pool.alloc(-(-int(length[i] + new[i]) // P) - -(-int(length[i]) // P))
                for i in range(n) if new[i] > 0
                and pool.num_free >= -(-int(length[i] + new[i]) // P) - -(-int(length[i]) // P)}
        got = host_step(table, length, new, ref, P, T)
        assert got[-1] == 0
        for i, pages in want.items():
            a = -(-int(length[i]) // P)
            assert list(got[0][i, a:a + len(pages)]) == pages
        table, ref, length = got[0], got[1], got[3]
        assert [pool.refcount(p) for p in range(40)] == list(ref)


def test_refusals(pa):
    L = pa.lib()
    P = 16  # any 16-byte aligned address: nothing is launched by a refused call
    ok = dict(pt=P, n=4, mp=8, ln=P, nw=P, ref=P, N=32, P=16, T=4)

    def call(out=(P,) * 7, **kw):
        c = dict(ok, **kw)
        return L.paged_batch_build(c["pt"], c["n"], c["mp"], c["ln"], c["nw"], c["ref"], c["N"],
                                   c["P"], c["T"], *out, None, None)
    for bad in (dict(n=-1), dict(mp=0), dict(N=-1), dict(P=0), dict(T=-1), dict(pt=None),
                dict(ln=None), dict(nw=None), dict(ref=None)):
        assert call(**bad) == pa.PA_EINVAL, bad
    for i in range(7):
        out = [P] * 7
        out[i] = None
        assert call(out=out) == pa.PA_EINVAL, i
    assert call(n=8193) == pa.PA_EUNSUPPORTED
    assert call(mp=1 << 20, P=1 << 12) == pa.PA_EUNSUPPORTED
    assert call(N=2 ** 30) == pa.PA_EUNSUPPORTED
    assert call(pt=24) == pa.PA_EALIGN and call(ref=8) == pa.PA_EALIGN
    assert call(out=[P, P, P, P, 40, P, P]) == pa.PA_EALIGN


def test_binding_refuses_wrong_tensors(pa):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # not on a CUDA device
        pa.batch_build(i32(2, 4), i32(2), i32(2), i32(8), 16, 4)


# ------------------------------------------------------------------ GPU

@pytest.mark.gpu
@pytest.mark.parametrize("n,P,max_pages,num_pages,spare", [
    (1, 128, 1, 1, 0), (1, 16, 3, 7, 2), (5, 16, 8, 61, 0), (33, 1, 40, 900, 7),
    (64, 128, 129, 8192, 3), (300, 16, 33, 9001, 100), (1025, 32, 20, 20000, 0),
    (2500, 7, 12, 40003, 11),
])
@pytest.mark.parametrize("seed", [0, 1])
def test_steps_match_the_host_model(pa, n, P, max_pages, num_pages, spare, seed):
    rng = np.random.default_rng([n, seed])
    table, length, new, ref = make(rng, n, P, max_pages, num_pages)
    T = int(np.maximum(new, 0).sum()) + spare
    check(pa, table, length, new, ref, P, T, alias=bool(seed))


@pytest.mark.gpu
def test_a_large_pool_and_the_last_pages(pa):
    """Free pages only at the far end of a pool of more pages than the cluster has threads x 4,
    and a size that is no multiple of four."""
    N, P = 1_000_003, 16
    ref = np.ones(N, np.int32)
    free = np.r_[5, np.arange(N - 70, N)]
    ref[free] = 0
    table = np.full((3, 64), -1, np.int32)
    length = np.zeros(3, np.int32)
    new = np.array([P * 30, 1, P * 40], np.int32)
    got = check(pa, table, length, new, ref, P, int(new.sum()))
    assert got[-1] == 0 and got[0][2, 39] == N - 1
    new = np.array([P * 30, 1, P * 41], np.int32)
    assert check(pa, table, length, new, ref, P, int(new.sum()))[-1] == pa.PA_ERR_NO_SPACE


@pytest.mark.gpu
def test_admission_stops_at_the_first_that_does_not_fit(pa):
    P, N = 16, 10
    table = np.full((4, 8), -1, np.int32)
    length = np.zeros(4, np.int32)
    ref = np.zeros(N, np.int32)
    new = np.array([40, 100, 1, 1], np.int32)       # 3, 7, 1 and 1 pages for 10 free ones
    got = check(pa, table, length, new, ref, P, 200)
    assert list(got[2]) == [0, 40, 140, 140, 140] and got[-1] == pa.PA_ERR_NO_SPACE
    got = check(pa, table, length, new, ref, P, 139)  # pages fit, tokens do not
    assert list(got[2]) == [0, 40, 40, 40, 40]
    got = check(pa, table, length, np.zeros(4, np.int32), ref, P, 0)  # an idle step
    assert got[-1] == 0
    full = np.ones(N, np.int32)
    length = np.array([5, 0, 16, 3], np.int32)
    table[0, 0], table[2, 0], table[3, 0] = 1, 2, 3
    got = check(pa, table, length, np.array([11, 0, 0, 2], np.int32), full, P, 20)
    assert got[-1] == 0 and got[2][-1] == 13         # no page needed: a full pool is no bar


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_flagged_not_followed(pa):
    P, N = 16, 12
    table = np.full((6, 4), -1, np.int32)
    table[0, :2] = 3, 99999                          # an id outside the pool
    table[1, :2] = 4, 5                              # page 5 is free already
    table[2, 0] = 6
    ref = np.zeros(N, np.int32)
    ref[[3, 4, 6]] = 1
    length = np.array([20, 20, 60, -4, 2 ** 31 - 1, 0], np.int32)
    new = np.array([-1, -1, 5, 3, 2 ** 31 - 1, 64], np.int32)  # rows 2..4: outside their rows
    got = check(pa, table, length, new, ref, P, 64)
    assert got[-1] == pa.PA_ERR_PAGE_RANGE | pa.PA_ERR_REFCOUNT | pa.PA_ERR_SEQ_RANGE
    assert list(got[0][5]) == [0, 1, 2, 3] and got[1][3] == 1 and got[1][4] == 0


@pytest.mark.gpu
def test_the_same_page_in_two_finished_rows(pa):
    P, N = 16, 9
    table = np.full((3, 4), -1, np.int32)
    table[0, :2], table[1, :2], table[2, :2] = (2, 7), (2, 7), (7, 8)
    ref = np.zeros(N, np.int32)
    ref[[2, 7, 8]] = 2, 3, 1
    got = check(pa, table, np.array([30, 20, 32], np.int32), np.array([-1, -1, 16], np.int32), ref,
                P, 16)
    assert got[-1] == 0 and got[0][2, 2] == 0 and got[1][7] == 1


@pytest.mark.gpu
def test_no_requests_no_pages(pa):
    out = pa.batch_build(torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                         *dev(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32)),
                         16, 5)
    assert out.q_start.tolist() == [0] and out.tok_seq.tolist() == [-1] * 5
    assert out.tok_page_table.eq(-1).all() and out.tok_kv_len.eq(0).all()
    assert out.slot_mapping.eq(-1).all() and out.tok_pos.eq(0).all()


@pytest.mark.gpu
def test_a_captured_step_replayed_over_a_growing_batch(pa):
    """The step captured once (lengths updated in place) and replayed on another stream with
    new request lengths each time, against the host model over 25 steps."""
    rng = np.random.default_rng(9)
    n, P, max_pages, N, T = 37, 16, 12, 300, 90
    table = np.full((n, max_pages), -1, np.int32)
    length, ref = np.zeros(n, np.int32), np.zeros(N, np.int32)
    t, ln, rf = dev(table, length, ref)
    nw = torch.zeros(n, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.new_batch(n, max_pages, T)._replace(seq_len=ln)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pa.batch_build(t, ln, nw, rf, P, T, out=out, err=err)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pa.batch_build(t, ln, nw, rf, P, T, out=out, err=err)
    for step in range(25):
        new = np.minimum(rng.integers(0, 6, n), max_pages * P - length).astype(np.int32)
        new[rng.random(n) < 0.08] = -1
        want = host_step(table, length, new, ref, P, T)
        with torch.cuda.stream(s):
            nw.copy_(torch.from_numpy(new))
            err.zero_()
            graph.replay()
        s.synchronize()
        for name, g, w in zip(("seq_page_table", "page_ref") + pa.Batch._fields,
                              (t, rf) + tuple(out), want):
            assert np.array_equal(g.cpu().numpy(), w), (step, name)
        assert int(err.item()) == want[-1]
        table, ref, length = want[0], want[1], want[3]
