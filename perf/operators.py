"""Workloads of the serving operators around the paged KV cache, with their plain forms.

Three operators of one serving step:
  batch   block tables, token lists and slot maps of a step built on the GPU from request
          lengths, with the pages taken from (and given back to) a reference-counted pool
  diff    differential attention over the paged cache: the difference of two softmax maps
          with a learned weight per head and a norm per head, for single tokens and chunks
  window  attention of single tokens and chunks over the last W cached positions, with a
          learned sink logit per head

A case's request lengths come from the case itself (``lens``); the values, the page
assignment and the pool come from the seed of ``prepare``.
"""
import math
import random

import numpy as np
import torch

own = False

I32, I64, F32, F64 = torch.int32, torch.int64, torch.float32, torch.float64


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 8 running requests, page size 128: the smallest call, all latency
        _batch("batch decode 8", P=128, decode=8, lo=1024, hi=4096, max_pages=32, lens=1),
        # a mixed step: 60 running requests, 4 prompts in chunks of up to 512, 8 that finished
        _batch("batch mixed 72", P=128, decode=60, lo=1024, hi=16000, chunks=4, chunk=512,
               plo=0, phi=15000, finished=8, spare=37, max_pages=128, lens=2),
        # many running requests over a pool of small pages
        _batch("batch decode 512 p16", P=16, decode=512, lo=256, hi=32000, finished=40,
               max_pages=2048, lens=3),
        # a large prompt step over small pages: the expanded table is the bulk of the bytes
        _batch("batch chunks 256 p16", P=16, decode=192, lo=256, hi=32000, chunks=64, chunk=256,
               plo=0, phi=30000, finished=16, spare=101, max_pages=2048, lens=4),
        # 8 sequences decoding, lengths 1024 to 4096: the decode workload's shape
        _attn("diff decode 8", "diff", decode=8, lo=1024, hi=4096, norm=True, lens=11),
        # 64 sequences decoding, lengths over two orders of magnitude
        _attn("diff long tail 64", "diff", decode=64, lo=256, hi=32768, norm=True, lens=12),
        # one prefill ubatch of four 512-token chunks at prefixes up to 16K
        _attn("diff chunks 2048", "diff", chunks=4, chunk=512, plo=0, phi=15800, norm=True,
              lens=13),
        # ragged chunks, decode and padding tokens together over small pages, narrow heads
        _attn("diff ragged d64 p16", "diff", P=16, d=64, Hq=8, Hkv=4, decode=13, lo=1, hi=900,
              chunks=3, chunk=229, plo=0, phi=1100, pad=5, norm=False, ragged=True, lens=14),
        # 64 sequences decoding within a window of the last 1024 positions
        _attn("window decode 64", "window", decode=64, lo=256, hi=32768, window=1024, sink=True,
              lens=21),
        # a prefill ubatch of four 512-token chunks, window 4096, at prefixes up to 16K
        _attn("window chunks 2048", "window", chunks=4, chunk=512, plo=0, phi=15800, window=4096,
              sink=False, lens=22),
        # a long prompt step through a short window, narrow heads in groups of eight
        _attn("window chunks d64 w128", "window", P=16, d=64, Hq=64, Hkv=8, chunks=8, chunk=512,
              plo=0, phi=12000, window=128, sink=True, lens=23),
        # an odd window over ragged chunks, decode and padding tokens, one query head a KV head
        _attn("window ragged p32", "window", P=32, Hq=4, Hkv=4, decode=21, lo=1, hi=3000,
              chunks=3, chunk=301, plo=0, phi=2500, pad=3, window=333, sink=True, ragged=True,
              lens=24),
    ]


def _batch(name, P, decode=0, lo=1, hi=1, chunks=0, chunk=1, plo=0, phi=0, finished=0, spare=0,
           max_pages=32, lens=0):
    c = dict(kind="batch", P=P, decode=decode, lo=lo, hi=hi, chunks=chunks, chunk=chunk, plo=plo,
             phi=phi, finished=finished, spare=spare, max_pages=max_pages, ragged=True, lens=lens)
    return dict(c, name=name) if name else c


def _attn(name, kind, P=128, d=128, Hq=32, Hkv=8, decode=0, lo=1, hi=1, chunks=0, chunk=1, plo=0,
          phi=0, pad=0, norm=False, window=0, sink=False, ragged=False, lens=0):
    c = dict(kind=kind, P=P, d=d, Hq=Hq, Hkv=Hkv, decode=decode, lo=lo, hi=hi, chunks=chunks,
             chunk=chunk, plo=plo, phi=phi, pad=pad, ragged=ragged, lens=lens)
    c.update(dict(norm=norm) if kind == "diff" else dict(window=window, sink=sink))
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["batch", "diff", "diff", "window", "window"])
    P = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1 << 30)
    if kind == "batch":
        hi = _log(rng, 300, 32000)
        return _batch("", P=P, decode=_log(rng, 1, 512), lo=rng.randint(1, 256), hi=hi,
                      chunks=rng.choice([0, _log(rng, 1, 32)]), chunk=_log(rng, 2, 300),
                      plo=0, phi=hi - 300, finished=rng.randint(0, 40),
                      spare=rng.choice([0, rng.randint(1, 200)]),
                      max_pages=-(-(hi + 300) // P) + rng.randint(0, 9), lens=lens)
    d, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    if G * Hkv > 32:
        Hkv = 4
    c = dict(P=P, d=d, Hq=G * Hkv, Hkv=Hkv, pad=rng.choice([0, 0, rng.randint(1, 9)]), ragged=True,
             lens=lens)
    what = rng.choice(["decode", "chunks", "both"])
    if what != "chunks":
        c.update(decode=_log(rng, 1, 64), lo=rng.randint(1, 300), hi=_log(rng, 400, 20000))
    if what != "decode":
        c.update(chunks=rng.randint(1, 4), chunk=_log(rng, 17, 512), plo=0,
                 phi=_log(rng, 1, 12000))
    if kind == "diff":
        return _attn("", "diff", norm=rng.random() < 0.7, **c)
    return _attn("", "window", window=_log(rng, 1, 9000), sink=rng.random() < 0.6, **c)


def _requests(case):
    """Per request (cached positions, new positions), in order: decoding requests, chunks of
    prompts, then for a batch the finished ones (new = -1)."""
    rng = random.Random(case["lens"])
    got = [(_log(rng, max(1, case["lo"]), case["hi"]) - 1, 1) for _ in range(case["decode"])]
    for _ in range(case["chunks"]):
        n = rng.randint(max(1, case["chunk"] // 2), case["chunk"]) if case["ragged"] else case["chunk"]
        got.append((rng.randint(case["plo"], case["phi"]), n))
    got += [(_log(rng, max(1, case["lo"]), case["hi"]), -1) for _ in range(case.get("finished", 0))]
    return got


def _pages(n, P):
    return -(-n // P)


def _lens(case):
    req = _requests(case)
    return [c for c, _ in req], [n for _, n in req]


def _live_pages(case):
    """(request, position in its row) of every page that holds cached positions."""
    cached, _ = _lens(case)
    n = np.array([_pages(c, case["P"]) for c in cached], np.int64)
    row = np.repeat(np.arange(len(n)), n)
    return row, np.arange(n.sum()) - np.repeat(np.cumsum(n) - n, n)


def work(case):
    req = _requests(case)
    if case["kind"] == "batch":
        n, T = len(req), sum(max(0, k) for _, k in req) + case["spare"]
        live = sum(_pages(c, case["P"]) for c, _ in req)
        new = sum(_pages(c + k, case["P"]) - _pages(c, case["P"]) for c, k in req if k > 0)
        gone = sum(_pages(c, case["P"]) for c, k in req if k < 0)
        # the lengths, the live part of the table and the pool's counts up to the pages taken,
        # each once; the expanded rows and lists of every token, the new and the cleared entries
        return {"bytes": 4.0 * (4 * n + live + 2 * new + 4 * gone + T * case["max_pages"] + 5 * T),
                "flops": 0.0}
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    W = case.get("window", 0) or 1 << 40
    keys = sum(sum(min(W, c + i + 1) for i in range(k)) for c, k in req)
    rows = sum(c + k - max(0, c + 1 - W) for c, k in req)  # cached rows that some token reads
    T = sum(k for _, k in req) + case["pad"]
    # q and the output; each K and V row once per KV head; the products of the scores and one
    # weighted sum of V (the two maps of the difference share it)
    return {"bytes": 2.0 * (2 * T * Hq * d + 2 * rows * Hkv * d), "flops": 4.0 * d * Hq * keys}


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    if case["kind"] == "batch":
        return _prepare_batch(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    P, d, Hq, Hkv = case["P"], case["d"], case["Hq"], case["Hkv"]
    cached, new = _lens(case)
    total = np.array(cached) + np.array(new)
    npg = -(-total // P)
    max_pages, used = int(npg.max()), int(npg.sum())
    N = _pages(4 * used, 3)
    perm = np.random.default_rng(seed).permutation(N).astype(np.int32)
    table = np.full((len(new), max_pages), -1, np.int32)
    row = np.repeat(np.arange(len(new)), npg)
    table[row, np.arange(used) - np.repeat(np.cumsum(npg) - npg, npg)] = perm[:used]
    T0 = int(np.sum(new))
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.arange(T0) - np.repeat(np.cumsum(new) - np.array(new), new) + np.array(cached)[seq]
    T = T0 + case["pad"]
    tpt = np.full((T, max_pages), -1, np.int32)
    tpt[:T0] = table[seq]
    kv = np.zeros(T, np.int32)
    kv[:T0] = pos + 1
    s = dict(case=case, q=torch.randn(T, Hq, d, generator=g, device="cuda").half(),
             kp=torch.randn(N, Hkv, P, d, generator=g, device="cuda", dtype=torch.float16),
             vp=torch.randn(N, Hkv, P, d, generator=g, device="cuda", dtype=torch.float16),
             table=torch.from_numpy(table).cuda(), tpt=torch.from_numpy(tpt).cuda(),
             kv=torch.from_numpy(kv).cuda(), T=T)
    s["out"] = torch.empty(T, Hq, d, dtype=torch.float16, device="cuda")
    D = case["decode"]
    # the tokens of each group of requests (single tokens, chunks), padded with -1
    s["groups"] = [(0, D, torch.arange(D, device="cuda")[:, None])] if D else []
    if case["chunks"]:
        n = np.array(new[D:])
        i = np.arange(n.max())[None]
        tok = np.where(i < n[:, None], D + (np.cumsum(n) - n)[:, None] + i, -1)
        s["groups"].append((D, D + len(n), torch.from_numpy(tok).cuda()))
    if case["kind"] == "diff":
        s["scale"] = 1.0 / math.sqrt(d // 2)
        s["lam"] = torch.rand(Hq, generator=g, device="cuda") * 0.8 + 0.1
        s["w"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
        s["eps"], s["out_scale"] = 1e-5, 0.2 if case["norm"] else 1.0
    else:
        s["scale"] = 1.0 / math.sqrt(d)
        s["sink"] = torch.randn(Hq, generator=g, device="cuda") * 2 if case["sink"] else None
    if own:
        # the plan of the step, made once and used by every layer of a model
        import paged_kv_cache_pages_gb300 as pa
        if case["kind"] == "diff":
            s["ws"] = pa.new_diff_workspace(T, Hq, Hkv, d)
            pa.plan_diff(s["tpt"], s["kv"], Hq, Hkv, P, d, s["ws"])
        else:
            s["ws"] = pa.new_workspace(T, Hq, Hkv, d)
            pa.plan_window(s["tpt"], s["kv"], Hq, Hkv, P, d, case["window"], s["ws"])
    return s


def _prepare_batch(case, seed):
    P = case["P"]
    cached, new = _lens(case)
    row, col = _live_pages(case)
    need = sum(_pages(c + k, P) - _pages(c, P) for c, k in zip(cached, new) if k > 0)
    N = _pages(4 * (len(row) + need), 3) + 1
    rng = np.random.default_rng(seed)
    perm = rng.permutation(N).astype(np.int32)
    table = np.full((len(new), case["max_pages"]), -1, np.int32)
    table[row, col] = perm[: len(row)]
    ref = np.zeros(N, np.int32)
    ref[perm[: len(row)]] = 1
    # a prefix shared by two rows: the second row's pages stay in use when the first one ends
    ref[perm[: len(row)][rng.random(len(row)) < 0.05]] = 2
    T = sum(max(0, k) for k in new) + case["spare"]
    s = dict(case=case, table0=torch.from_numpy(table).cuda(), ref0=torch.from_numpy(ref).cuda(),
             len=torch.tensor(cached, dtype=I32, device="cuda"),
             new=torch.tensor(new, dtype=I32, device="cuda"), T=T)
    # the step works on the pool and the table in place: every pass starts from the same ones
    s["table"], s["ref"] = s["table0"].clone(), s["ref0"].clone()
    if own:
        import paged_kv_cache_pages_gb300 as pa
        s["out"] = pa.new_batch(len(new), case["max_pages"], T)
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    if s["case"]["kind"] == "batch":
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
        if own:
            import paged_kv_cache_pages_gb300 as pa
            return (s["table"], s["ref"]) + tuple(
                pa.batch_build(s["table"], s["len"], s["new"], s["ref"], s["case"]["P"], s["T"],
                               out=s["out"]))
        return plain_batch(s["table"], s["len"], s["new"], s["ref"], s["case"]["P"], s["T"])
    if s["case"]["kind"] == "diff":
        if own:
            import paged_kv_cache_pages_gb300 as pa
            return pa.diff_run(s["q"], s["kp"], s["vp"], s["tpt"], s["kv"], s["scale"], s["lam"],
                               norm_weight=s["w"], eps=s["eps"], out_scale=s["out_scale"],
                               out=s["out"], workspace=s["ws"])
        return plain_attention(s, plain_diff)
    if own:
        import paged_kv_cache_pages_gb300 as pa
        return pa.window_run(s["q"], s["kp"], s["vp"], s["tpt"], s["kv"], s["scale"],
                             sink=s["sink"], out=s["out"], workspace=s["ws"])
    return plain_attention(s, plain_window)


# ----------------------------------------------------------------------------- plain forms

def plain_batch(table, length, new, ref, P, T):
    """Finished requests (new < 0) give their pages back; then, in order, every request up to
    the first whose pages or tokens do not fit takes free pages, lowest ids first, for its new
    positions; then the tokens' lists."""
    n, max_pages = table.shape
    dev = table.device
    end = new < 0
    given = end[:, None] & (table >= 0)
    ref.scatter_add_(0, table.clamp(min=0).flatten().long(), -given.flatten().to(I32))
    table.masked_fill_(end[:, None], -1)
    length = torch.where(end, 0, length)
    new = new.clamp(min=0)
    first = (length + P - 1) // P
    need = (length + new + P - 1) // P - first
    free = ref == 0
    pages_end, toks_end = need.cumsum(0), new.cumsum(0)
    admitted = (pages_end <= free.sum()) & (toks_end <= T)
    new, need = torch.where(admitted, new, 0), torch.where(admitted, need, 0)
    q_start = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(I32)
    rank = free.cumsum(0) - 1
    ids = torch.arange(ref.numel(), device=dev)
    free_list = torch.zeros(ref.numel() + 1, dtype=I64, device=dev)
    free_list.scatter_(0, torch.where(free, rank, ref.numel()), ids)
    at = torch.arange(max_pages, device=dev)[None] - first[:, None]
    take = (at >= 0) & (at < need[:, None])
    src = ((need.cumsum(0) - need)[:, None] + at).clamp(0, ref.numel())
    table.copy_(torch.where(take, free_list[src].to(I32), table))
    ref.masked_fill_(free & (rank < need.sum()), 1)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    real = t < q_start[-1]
    safe = seq.clamp(max=n - 1)
    pos = length[safe] + t - q_start[safe]
    tok_seq = torch.where(real, seq, -1).to(I32)
    tok_pos = torch.where(real, pos, 0).to(I32)
    tok_table = torch.where(real[:, None], table[safe], -1)
    page = tok_table.gather(1, (tok_pos // P).long()[:, None])[:, 0].long()
    slot = torch.where(real, page * P + tok_pos % P, -1)
    kv = torch.where(real, tok_pos + 1, 0).to(I32)
    return table, ref, q_start, (length + new).to(I32), tok_seq, tok_pos, tok_table, kv, slot


def _rows(pages, table, dtype):
    """The cached rows of each request: [R][Hkv][positions][d]."""
    x = pages[table.clamp(min=0).long()].to(dtype)  # [R][pages][Hkv][P][d]
    R, n, Hkv, P, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * P, d)


def _group(s, form, group):
    lo, hi, tok = group
    Hkv, d = s["case"]["Hkv"], s["case"]["d"]
    q = s["q"][tok.clamp(min=0)].to(F32)  # [R][n][Hq][d]
    R, n, Hq, _ = q.shape
    q = q.permute(0, 2, 1, 3).reshape(R, Hkv, Hq // Hkv, n, d)
    kv = torch.where(tok >= 0, s["kv"][tok.clamp(min=0)], 0)
    k, v = (_rows(s[x], s["table"][lo:hi], F32)[:, :, None] for x in ("kp", "vp"))
    y = form(s, q, k, v, kv[:, None, None, :, None])
    y = y.reshape(R, Hq, n, d).permute(0, 2, 1, 3)
    return tok.flatten(), y.reshape(R * n, Hq, d)


def plain_attention(s, form):
    done = [_group(s, form, g) for g in s["groups"]]
    out = torch.zeros(s["T"] + 1, s["case"]["Hq"], s["case"]["d"], dtype=F32, device="cuda")
    tok, y = (torch.cat(x) for x in zip(*done))
    out[torch.where(tok >= 0, tok, s["T"])] = y
    return out[: s["T"]].half()


def _softmax(x, keep):
    x = x.masked_fill_(~keep, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top.isfinite(), top, 0)).exp_()
    return x, x.sum(-1, keepdim=True), top


def plain_diff(s, q, k, v, kv):
    h = q.shape[-1] // 2
    keep = torch.arange(k.shape[-2], device=q.device) < kv
    p1, l1, _ = _softmax(q[..., :h] @ k[..., :h].mT * s["scale"], keep)
    p2, l2, _ = _softmax(q[..., h:] @ k[..., h:].mT * s["scale"], keep)
    lam = s["lam"].reshape(1, q.shape[1], q.shape[2], 1, 1)
    p1.div_(l1.clamp(min=1e-30)).sub_(p2.mul_(lam / l2.clamp(min=1e-30)))
    y = p1 @ v
    if s["w"] is not None:
        y = y * (y.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * s["w"]
    return y * s["out_scale"]


def plain_window(s, q, k, v, kv):
    j = torch.arange(k.shape[-2], device=q.device)
    p, l, top = _softmax(q @ k.mT * s["scale"], (j < kv) & (j >= kv - s["case"]["window"]))
    if s["sink"] is not None:
        sink = s["sink"].reshape(1, q.shape[1], q.shape[2], 1, 1)
        l = l + torch.where(top.isfinite(), (sink - top).exp(), 1)
    return p @ v / l.clamp(min=1e-30)


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    if case["kind"] == "batch":
        return _exact_batch(_prepare_batch(case, seed))
    s = prepare(case, seed)
    kv, P, G = s["kv"].tolist(), case["P"], case["Hq"] // case["Hkv"]
    out = torch.zeros(s["T"], case["Hq"], case["d"], dtype=F64, device="cuda")
    cached, new = _lens(case)
    t0 = 0
    for r, n in enumerate(new):
        L = kv[t0 + n - 1]
        lo = max(0, kv[t0] - case["window"]) if case["kind"] == "window" else 0
        pos = torch.arange(lo, L, device="cuda")
        page = s["table"][r][pos // P].long()
        last = torch.arange(t0, t0 + n, device="cuda")
        for h in range(case["Hq"]):
            K = s["kp"][page, h // G, pos % P].double()
            V = s["vp"][page, h // G, pos % P].double()
            q = s["q"][t0:t0 + n, h].double()
            seen = pos[None] < s["kv"][last][:, None]
            if case["kind"] == "window":
                seen &= pos[None] >= s["kv"][last][:, None] - case["window"]
                extra = s["sink"][h].double() if case["sink"] else None
                x = torch.where(seen, q @ K.T * s["scale"], -math.inf)
                z = x.logsumexp(-1, keepdim=True)
                z = z if extra is None else torch.logaddexp(z, extra)
                out[t0:t0 + n, h] = (x - z).exp() @ V
            else:
                e = case["d"] // 2
                a = [torch.where(seen, q[:, i:i + e] @ K[:, i:i + e].T * s["scale"], -math.inf)
                     for i in (0, e)]
                a = [(x - x.logsumexp(-1, keepdim=True)).exp() @ V for x in a]
                y = a[0] - s["lam"][h].double() * a[1]
                if s["w"] is not None:
                    y = y / (y.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * s["w"].double()
                out[t0:t0 + n, h] = y * s["out_scale"]
        t0 += n
    return out


def _exact_batch(s):
    P, T = s["case"]["P"], s["T"]
    table, ref = s["table0"].cpu().numpy(), s["ref0"].cpu().numpy()
    length, new = s["len"].cpu().numpy().copy(), s["new"].cpu().numpy()
    for i in np.nonzero(new < 0)[0]:
        ref[table[i][table[i] >= 0]] -= 1  # the pages of one row are distinct
        table[i] = -1
        length[i] = 0
    free = list(np.nonzero(ref == 0)[0])
    q_start, seq, pos, used, closed = [0], [], [], 0, False
    for i, n in enumerate(np.maximum(new, 0)):
        first, last = _pages(length[i], P), _pages(length[i] + n, P)
        closed = closed or used + last - first > len(free) or len(seq) + n > T
        if not closed:
            table[i, first:last] = free[used:used + last - first]
            ref[table[i, first:last]] = 1
            used += last - first
            seq += [i] * int(n)
            pos += list(range(length[i], length[i] + n))
            length[i] += n
        q_start.append(len(seq))
    pad = T - len(seq)
    a = lambda x, fill, t: np.array(x + [fill] * pad, t)  # noqa: E731
    seq, pos = a(seq, -1, np.int32), a(pos, 0, np.int32)
    rows = np.where(seq[:, None] >= 0, table[seq], -1)
    slot = np.where(seq >= 0, rows[np.arange(T), pos // P].astype(np.int64) * P + pos % P, -1)
    return (table, ref, np.array(q_start, np.int32), length, seq, pos, rows,
            np.where(seq >= 0, pos + 1, 0).astype(np.int32), slot)
