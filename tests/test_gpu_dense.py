"""Attention of each sequence's newest tokens over its whole cache
(ts_dense_attn) against the definition in 64 bits.

Bounds.  With w the softmax weights and A = sum_j w_j |V_j| of an output, the
weights are rounded to bf16 (2^-8 of each) and so is the result (2^-8 of it).
A logit is a sum of d products in fp32 (at most d steps of 2^-23 of
sum |q||k| scale, and its scaling 2^-22), which moves each weight and the
normaliser by that much; sums over n tokens add at most n 2^-23 (accumulators
that truncate count 2^-23 a step), the exponentials 2^-21."""
import math

import numpy as np
import pytest
import torch

import gpu_helpers as H
import workloads as W

pytestmark = pytest.mark.gpu


def definition(q, k, v, n, scale=None):
    """q [f, h_q, d], k and v [n, h_kv, d] of one sequence: out, lse and the
    two bounds, float64."""
    f, h_q, d = q.shape
    h_kv = k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros((f, h_q, d), dtype=torch.float64, device=q.device)
    lse = torch.full((f, h_q), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or f == 0:
        return out, lse, tol, tol_lse
    seen = torch.arange(n, device=q.device).unsqueeze(0) <= torch.arange(n - f, n, device=q.device).unsqueeze(1)
    some = seen.any(1)
    for h in range(h_q):
        kk, vv, qq = k[:, h // (h_q // h_kv)].double(), v[:, h // (h_q // h_kv)].double(), q[:, h].double()
        s = (qq @ kk.t() * scale).masked_fill(~seen, -math.inf)
        size = (qq.abs() @ kk.abs().t() * abs(scale)).masked_fill(~seen, 0.0).amax(1)
        m = torch.where(some, s.amax(1), torch.zeros_like(size))
        w = torch.exp(s - m.unsqueeze(1)) * seen
        z = w.sum(1)
        w = w / torch.where(z > 0, z, torch.ones_like(z)).unsqueeze(1)
        out[:, h] = w @ vv
        lse[:, h] = torch.where(some, m + torch.log(z), torch.full_like(m, -math.inf))
        ds = size * (d * 2.0 ** -23 + 2.0 ** -22)
        fp32 = 2 * ds + n * 2.0 ** -23 + 2.0 ** -20
        a = w @ vv.abs()
        tol[:, h] = a * (2.0 ** -8 + fp32.unsqueeze(1)) * (1 + 2.0 ** -8) + out[:, h].abs() * 2.0 ** -8 + 1e-30
        tol_lse[:, h] = ds + n * 2.0 ** -23 + 2.0 ** -20 + lse[:, h].abs().nan_to_num(posinf=0.0) * 2.0 ** -22
    return out, lse, tol, tol_lse


def check(case_rows, q_off, q, out, lse, scale=None):
    """case_rows: [(k, v)] of each sequence's tokens; out, lse from the GPU."""
    for b, (k, v) in enumerate(case_rows):
        lo, hi = int(q_off[b]), int(q_off[b + 1])
        want, want_lse, tol, tol_lse = definition(q[lo:hi], k, v, k.shape[0], scale)
        err = (out[lo:hi].double() - want).abs()
        bad = ~(err <= tol)
        assert not bad.any(), "sequence %d: %d values off, worst %.3g of the bound" % (
            b, int(bad.sum()), float((err / tol).max()))
        dead = want_lse == -math.inf
        assert torch.equal(lse[lo:hi].double() == -math.inf, dead)
        err = (lse[lo:hi].double() - want_lse).abs()[~dead]
        assert (err <= tol_lse[~dead]).all(), "sequence %d: lse off by %.3g" % (b, float(err.max()))


def paged(k, v, off, page, seed, junk=float("nan")):
    """The packed rows in a pool of pages in random order, NaN in every row
    that no token owns; the block table's unused entries are -1."""
    lengths = np.diff(off)
    counts = [-(-int(n) // page) for n in lengths]
    used, stride = sum(counts), max(1, max(counts))
    pool = used + used // 2 + 1
    rng = np.random.default_rng(seed)
    phys = rng.permutation(pool)[:used]
    kp = torch.full((pool * page,) + tuple(k.shape[1:]), junk, dtype=torch.bfloat16, device=k.device)
    vp = kp.clone()
    table = np.full((len(lengths), stride), -1, np.int32)
    at = 0
    for b, n in enumerate(lengths):
        i = np.arange(int(n))
        table[b, :counts[b]] = phys[at:at + counts[b]]
        rows = torch.from_numpy(table[b][i // page].astype(np.int64) * page + i % page).to(k.device)
        kp[rows] = k[int(off[b]):int(off[b + 1])]
        vp[rows] = v[int(off[b]):int(off[b + 1])]
        at += counts[b]
    return kp, vp, torch.from_numpy(table).to(k.device)


def inputs(lengths, fresh, h_q, h_kv, d, seed, peaked=False):
    off, q_off = W.seq_offsets(lengths), W.seq_offsets(fresh)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn((int(off[-1]), h_kv, d), device="cuda", generator=g).to(torch.bfloat16)
    v = torch.randn((int(off[-1]), h_kv, d), device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn((int(q_off[-1]), h_q, d), device="cuda", generator=g)
    if peaked:      # logits far apart, growing along the sequence: the running maximum moves all the time
        q, k = q * 4, (k * torch.linspace(0.1, 4, max(1, k.shape[0]), device="cuda").view(-1, 1, 1)).to(torch.bfloat16)
    return off, q_off, q.to(torch.bfloat16), k, v


def attend(k, v, off, q, q_off, h_q, scale=0.0, table=None, page=0, capacity=0):
    m = H.ts()
    kv = m.KVCache(k, v, off, h_q, scale, capacity=capacity, page_table=table, page_size=page)
    buf = m.DenseBuffers(kv, q_off)
    buf.out.fill_(float("nan"))
    buf.lse.fill_(float("nan"))
    m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)
    torch.cuda.synchronize()
    assert m.ts_get_device_status(buf.ws) == (m.TS_OK, 0)
    return buf


def sequences(k, v, off):
    return [(k[int(off[b]):int(off[b + 1])], v[int(off[b]):int(off[b + 1])]) for b in range(len(off) - 1)]


HEADS = [(4, 2, 64), (28, 4, 128), (32, 8, 128), (8, 1, 128), (32, 2, 128), (16, 1, 64), (3, 1, 64), (8, 8, 64), (12, 4, 128)]
PROMPTS = [[1], [2], [17], [63, 64, 65], [127, 128, 129, 1], [255, 0, 256, 257], [300, 5, 777], [1500]]


@pytest.mark.parametrize("lengths", PROMPTS, ids=str)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_whole_prompts(heads, lengths):
    h_q, h_kv, d = heads
    off, q_off, q, k, v = inputs(lengths, lengths, h_q, h_kv, d, 11)
    buf = attend(k, v, off, q, q_off, h_q)
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse)


CHUNKS = {
    # cached, fresh
    "decode": ([0, 1, 15, 16, 17, 127, 128, 1000, 4095], [1] * 9),
    "decode_gaps": ([100, 200, 300, 400], [1, 0, 1, 0]),
    "few": ([5, 100, 1000, 2049], [2, 3, 5, 9]),
    "chunks": ([130, 0, 999], [70, 300, 129]),
    "mixed": ([2000, 50, 0, 700, 129, 1], [1, 200, 33, 1, 1, 600]),
    "long": ([9000], [150]),
    "long_few": ([20011], [3]),
}


@pytest.mark.parametrize("page", [0, 8, 16, 64, 128, 512])
@pytest.mark.parametrize("name", sorted(CHUNKS))
@pytest.mark.parametrize("heads", [(4, 2, 64), (28, 4, 128), (32, 8, 128), (16, 1, 128), (8, 8, 64)], ids=str)
def test_chunks_over_a_cache(heads, name, page):
    h_q, h_kv, d = heads
    cached, fresh = CHUNKS[name]
    off, q_off, q, k, v = inputs([c + f for c, f in zip(cached, fresh)], fresh, h_q, h_kv, d, 23)
    if page:
        kp, vp, table = paged(k, v, off, page, 3)
        buf = attend(kp, vp, off, q, q_off, h_q, table=table, page=page)
    else:
        buf = attend(k, v, off, q, q_off, h_q)
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse)


@pytest.mark.parametrize("fresh", [[1], [400], [1024]], ids=str)
@pytest.mark.parametrize("scale", [0.0, 0.5, -0.07])
def test_a_maximum_that_moves_and_other_scales(scale, fresh):
    off, q_off, q, k, v = inputs([1024], fresh, 28, 4, 128, 5, peaked=scale != 0.5)
    buf = attend(k, v, off, q, q_off, 28, scale=scale)
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse, scale=float(np.float32(scale)) or None)


def test_views_of_one_projection():
    """q, k and v as views of [tokens, (h_q + 2 h_kv) d], and a K / V layout
    with gaps between heads."""
    h_q, h_kv, d, n = 28, 4, 128, 500
    x = torch.randn((n, h_q + 2 * h_kv, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    buf = attend(k, v, [0, n], q, [0, n], h_q)
    check([(k, v)], [0, n], q, buf.out, buf.lse)
    wide = torch.full((n, 2 * h_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    gk, gv = wide[:, ::2], wide.clone()[:, ::2]
    gk.copy_(k)
    gv.copy_(v)
    again = attend(gk, gv, [0, n], q, [0, n], h_q)
    assert torch.equal(again.out, buf.out) and torch.equal(again.lse, buf.lse)


def test_more_queries_than_tokens():
    """Rows before the first token see nothing: zeros and -inf."""
    off, q_off, q, k, v = inputs([10, 0, 300], [25, 7, 310], 8, 2, 128, 9)
    buf = attend(k, v, off, q, q_off, 8)
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse)
    for lo, hi in ((0, 15), (25, 32), (32, 42)):
        assert (buf.out[lo:hi] == 0).all() and (buf.lse[lo:hi] == -math.inf).all()


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("fresh", [1, 90, 333])
@pytest.mark.parametrize("h_q", [14, 32])
def test_no_token_reaches_rows_that_do_not_see_it(h_q, fresh, page):
    """NaN and infinities in K and V of one token: rows before it are as if it
    were not there, rows from it on are NaN or infinite in its channels."""
    n, h_kv, d = 333, 2, 128
    off, q_off, q, k, v = inputs([n, 50], [fresh, 50], h_q, h_kv, d, 31)
    clean = attend(k, v, off, q, q_off, h_q)
    at = n - fresh // 2 - 1
    for what in ("v_nan", "v_inf", "k_nan"):
        k2, v2 = k.clone(), v.clone()
        if what == "k_nan":
            k2[at] = float("nan")
        else:
            v2[at, :, 5] = float("nan") if what == "v_nan" else float("inf")
            v2[at, :, 127] = float("-inf") if what == "v_inf" else float("nan")
        if page:
            kp, vp, table = paged(k2, v2, off, page, 1)
            buf = attend(kp, vp, off, q, q_off, h_q, table=table, page=page)
        else:
            buf = attend(k2, v2, off, q, q_off, h_q)
        first = at - (n - fresh)          # the first query row that sees the token
        assert torch.equal(buf.out[:first], clean.out[:first])
        assert torch.equal(buf.out[fresh:], clean.out[fresh:])
        hit = buf.out[first:fresh]
        if what == "k_nan":
            assert hit.isnan().all() and buf.lse[first:fresh].isnan().all()
        else:
            if what == "v_nan":
                assert hit[:, :, 5].isnan().all() and hit[:, :, 127].isnan().all()
            else:
                assert (hit[:, :, 5] == math.inf).all() and (hit[:, :, 127] == -math.inf).all()
            rest = [c for c in range(d) if c not in (5, 127)]
            assert torch.equal(hit[:, :, rest], clean.out[first:fresh][:, :, rest])
            assert torch.equal(buf.lse[:fresh], clean.lse[:fresh])


def test_rows_behind_the_last_stay():
    off, q_off, q, k, v = inputs([200, 40], [30, 40], 8, 2, 64, 2)
    m = H.ts()
    kv = m.KVCache(k, v, off, 8)
    buf = m.DenseBuffers(kv, q_off)
    q = torch.cat([q, torch.full((5, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full((75, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((75, 8), 7.0, device="cuda")
    m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, out, lse, buf.ws)
    torch.cuda.synchronize()
    assert (out[70:] == 7).all() and (lse[70:] == 7).all()
    check(sequences(k, v, off), q_off, q, out[:70], lse[:70])
    out2 = torch.full_like(out, 7.0)
    m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, out2, None, buf.ws)      # without lse
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


def test_a_growing_cache_under_a_graph():
    """Capacity mode: the current length is read on the device; one captured
    graph of [append, attend] serves every length, bit for bit as a fresh call
    on a cache of that length up to the split of the work."""
    m = H.ts()
    n0, cap, h_q, h_kv, d, steps = 250, 400, 28, 4, 128, 20
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v, kn, vn = (torch.randn((r, h_kv, d), device="cuda", generator=g).to(torch.bfloat16) for r in (cap, cap, 1, 1))
    q = torch.randn((1, h_q, d), device="cuda", generator=g).to(torch.bfloat16)
    kv = m.KVCache(k, v, [0, n0], h_q, capacity=cap)
    buf, ws = m.DenseBuffers(kv, [0, 1]), torch.zeros(m.ts_workspace_bytes(kv, 16, 4, 16), dtype=torch.uint8, device="cuda")

    def step():
        m.ts_append_kv(kv, kn[0], vn[0], ws)
        m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()                             # warm-up: the length is n0 + 1 now
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            step()
    for i in range(steps):
        kn.normal_(generator=g)
        vn.normal_(generator=g)
        q.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        n = n0 + 2 + i
        assert int(kv.seq_offsets_dev[1]) == n
        check([(k[:n], v[:n])], [0, 1], q, buf.out, buf.lse)
    assert m.ts_get_device_status(buf.ws) == (m.TS_OK, 0)


def test_two_streams_two_workspaces():
    cases = [inputs([700, 900], [700, 1], 28, 4, 128, 1), inputs([40, 5000], [40, 64], 8, 1, 64, 2)]
    m = H.ts()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    kvs = [m.KVCache(k, v, off, q.shape[1]) for off, _, q, k, v in cases]
    bufs = [m.DenseBuffers(kv, c[1]) for kv, c in zip(kvs, cases)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, kv, buf, c in zip(streams, kvs, bufs, cases):
            m.ts_dense_attn(kv, c[2], buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws, stream=st)
    torch.cuda.synchronize()
    for buf, (off, q_off, q, k, v) in zip(bufs, cases):
        check(sequences(k, v, off), q_off, q, buf.out, buf.lse)


def test_the_same_bits_every_time():
    off, q_off, q, k, v = inputs([5000, 300, 40], [1, 300, 17], 28, 4, 128, 8)
    a = attend(k, v, off, q, q_off, 28)
    for _ in range(5):
        b = attend(k, v, off, q, q_off, 28)
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_one_token_matches_the_sparse_attention_over_every_token():
    """f = 1 sees what ts_sparse_attn sees when every token is selected."""
    m = H.ts()
    n = 900
    off, q_off, q, k, v = inputs([n], [1], 28, 4, 128, 6)
    buf = attend(k, v, off, q, q_off, 28)
    kv = m.KVCache(k, v, off, 28)
    step = m.StepBuffers(kv, n, 0, 0)
    step.ids.copy_(torch.arange(n, dtype=torch.int32).view(1, -1))
    step.count.fill_(n)
    m.ts_sparse_attn(kv, q, step.ids, step.count, step.out, step.ws)
    torch.cuda.synchronize()
    _, _, tol, _ = definition(q, k, v, n)
    assert ((buf.out.double() - step.out.double()).abs() <= 2 * tol).all()


def test_prompt_in_chunks_then_a_decode_step():
    """The operators as a server uses them: requests' prompts enter a paged
    cache chunk by chunk (room, rows, attention), each chunk's output is the
    whole prompt's, and the selection step then runs on the same cache as on a
    packed one."""
    m = H.ts()
    h_q, h_kv, d, page, B = 28, 4, 128, 16, 3
    total = np.array([700, 130, 401])
    off, q_off, q, k, v = inputs(total, total, h_q, h_kv, d, 77)
    whole = attend(k, v, off, q, q_off, h_q)
    pages = 2 * int(sum(-(-total // page)))
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()
    pool_k = torch.full((pages * page, h_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool_v = pool_k.clone()
    table = torch.full((B, int(-(-total.max() // page))), -1, dtype=torch.int32, device="cuda")
    done, used = np.zeros(B, np.int64), 0
    for chunk in ([300, 130, 1], [300, 0, 200], [100, 0, 200]):
        fresh = np.array(chunk)
        kv = m.KVCache(pool_k, pool_v, W.seq_offsets(done + fresh), h_q, page_table=table, page_size=page)
        buf = m.DenseBuffers(kv, W.seq_offsets(fresh))
        slots = torch.zeros(int(fresh.sum()), dtype=torch.int64, device="cuda")
        n_used = torch.zeros(1, dtype=torch.int64, device="cuda")
        m.ts_extend_pages(torch.from_numpy(done).cuda(), torch.from_numpy(fresh).cuda(), page, free[used:].contiguous(), pages,
                          table, kv.seq_offsets_dev, buf.q_offsets_dev, slots, n_used)
        rows = torch.cat([torch.arange(int(off[b] + done[b]), int(off[b] + done[b] + fresh[b])) for b in range(B)]).cuda()
        m.chunk_step(kv, q[rows], k[rows], v[rows], slots, buf)
        torch.cuda.synchronize()
        used += int(n_used)
        done = done + fresh
        assert kv.seq_offsets_dev.cpu().tolist() == W.seq_offsets(done).tolist()
        for b in range(B):
            lo, hi = buf.q_offsets_host[b], buf.q_offsets_host[b + 1]
            seq = (k[int(off[b]):int(off[b] + done[b])], v[int(off[b]):int(off[b] + done[b])])
            check([seq], [0, hi - lo], q[rows][lo:hi], buf.out[lo:hi], buf.lse[lo:hi])
            _, _, tol, _ = definition(q[rows][lo:hi], *seq, int(done[b]))
            assert ((buf.out[lo:hi].double() - whole.out[rows][lo:hi].double()).abs() <= 2 * tol).all()
    qd = torch.randn((B, h_q, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    got, want = m.StepBuffers(kv, 64, 4, 32), m.StepBuffers(m.KVCache(k, v, off, h_q), 64, 4, 32)
    m.decode_step(kv, qd, got)
    m.decode_step(m.KVCache(k, v, off, h_q), qd, want)
    torch.cuda.synchronize()
    assert torch.equal(got.ids, want.ids) and torch.equal(got.count, want.count)
    assert (got.out - want.out).abs().max() <= H.OUT_ATOL


@pytest.mark.parametrize("fresh", [1, 100])
def test_a_short_sequence_in_a_cache_with_room_for_a_long_one(fresh):
    """The launch is sized for the capacity, the work for the current length."""
    m = H.ts()
    cap, h_q, h_kv, d = 200000, 28, 4, 128
    g = torch.Generator(device="cuda").manual_seed(12)
    k, v = (torch.randn((cap, h_kv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((fresh, h_q, d), device="cuda", generator=g).to(torch.bfloat16)
    kv = m.KVCache(k, v, [0, 50000], h_q, capacity=cap)
    buf = m.DenseBuffers(kv, [0, fresh])
    for n in (fresh, 129, 1000, 1027, 5003, 20011, 130000):
        kv.seq_offsets_dev[1] = n
        buf.out.fill_(float("nan"))
        m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)
        torch.cuda.synchronize()
        check([(k[:n], v[:n])], [0, fresh], q, buf.out, buf.lse)
    assert m.ts_get_device_status(buf.ws) == (m.TS_OK, 0)


def test_many_sequences():
    """1024 sequences, some empty, some without queries, some of one token."""
    rng = np.random.default_rng(5)
    n = rng.integers(0, 60, 1024)
    f = np.minimum(rng.choice([0, 1, 1, 1, 2, 7, 40], 1024), n)
    n[700], f[700] = 3000, 1
    n[333], f[333] = 900, 500
    off, q_off, q, k, v = inputs(n, f, 8, 2, 64, 3)
    buf = attend(k, v, off, q, q_off, 8)
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse)
    kp, vp, table = paged(k, v, off, 8, 2)
    again = attend(kp, vp, off, q, q_off, 8, table=table, page=8)
    check(sequences(k, v, off), q_off, q, again.out, again.lse)


def test_one_workspace_for_several_shapes_and_graphs():
    """Calls of different shapes take turns on one workspace, captured ones too."""
    m = H.ts()
    cases = [inputs([9000, 40], [1, 1], 28, 4, 128, 1), inputs([700], [700], 32, 8, 128, 2), inputs([3000] * 3, [1, 70, 1], 8, 1, 64, 3),
             inputs([20000], [1], 32, 2, 128, 4)]
    kvs = [m.KVCache(k, v, off, q.shape[1]) for off, _, q, k, v in cases]
    bufs = [m.DenseBuffers(kv, c[1]) for kv, c in zip(kvs, cases)]
    ws = torch.empty(max(b.ws.numel() for b in bufs), dtype=torch.uint8, device="cuda")
    m.ts_workspace_init(ws)

    def call(i):
        b = bufs[i]
        m.ts_dense_attn(kvs[i], cases[i][2], b.q_offsets_dev, b.q_offsets_host, b.out, b.lse, ws)

    def checked(i):
        torch.cuda.synchronize()
        off, q_off, q, k, v = cases[i]
        check(sequences(k, v, off), q_off, q, bufs[i].out, bufs[i].lse)
        bufs[i].out.zero_()

    for i in (0, 1, 2, 3, 2, 0, 3, 1, 0):
        call(i)
        checked(i)
    s, graphs = torch.cuda.Stream(), []
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for i in range(len(cases)):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                call(i)
        for i in (3, 0, 2, 1, 0, 3):
            graphs[i].replay()
            s.synchronize()
            checked(i)
    assert m.ts_get_device_status(ws) == (m.TS_OK, 0)


@pytest.mark.parametrize("fresh", [1, 40])
def test_pages_past_two_to_the_31_elements(fresh):
    m = H.ts()
    rows, h_q, h_kv, d, page, n = 2 ** 21 + 1024, 32, 8, 128, 16, 500
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.full((rows, h_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    pages = torch.randperm(rows // page, generator=torch.Generator().manual_seed(1))[:32]
    pages[:16] = rows // page - 1 - torch.arange(16)          # the last ones among them
    table = pages.to(torch.int32).view(1, -1).contiguous().cuda()
    i = torch.arange(n)
    at = (pages[i // page] * page + i % page).cuda()
    kk, vv = (torch.randn((n, h_kv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    k[at], v[at] = kk, vv
    q = torch.randn((fresh, h_q, d), device="cuda", generator=g).to(torch.bfloat16)
    buf = attend(k, v, [0, n], q, [0, fresh], h_q, table=table, page=page)
    check([(kk, vv)], [0, fresh], q, buf.out, buf.lse)


def test_ragged_batches_at_random():
    rng = np.random.default_rng(99)
    for trial in range(25):
        h_q, h_kv, d = HEADS[trial % len(HEADS)]
        B = int(rng.integers(1, 9))
        n = rng.integers(0, int(rng.choice([50, 700, 6000])), B)
        f = np.array([int(rng.choice([0, 1, min(2, x), rng.integers(0, x + 1), x])) if x else int(rng.integers(0, 3)) for x in n])
        off, q_off, q, k, v = inputs(n, f, h_q, h_kv, d, trial, peaked=trial % 3 == 0)
        page = int(rng.choice([0, 8, 16, 32, 256]))
        if page:
            kp, vp, table = paged(k, v, off, page, trial)
            buf = attend(kp, vp, off, q, q_off, h_q, table=table, page=page)
        else:
            buf = attend(k, v, off, q, q_off, h_q)
        check(sequences(k, v, off), q_off, q, buf.out, buf.lse)


@pytest.mark.parametrize("fresh", [1, 2, 100, 400])
@pytest.mark.parametrize("first", [3, 40, 128, 200])
def test_scores_of_minus_infinity(first, fresh):
    """Keys whose scores are -inf weigh nothing, the first tokens' too: as if
    the sequence began behind them (for rows that see others)."""
    n, h_q, h_kv, d = 600, 14, 2, 128
    off, q_off, q, k, v = inputs([n], [fresh], h_q, h_kv, d, 41)
    q[:, :, 3] = q[:, :, 3].abs() + 1
    k[:first, :, 3] = float("-inf")
    buf = attend(k, v, off, q, q_off, h_q)
    check([(k[first:], v[first:])], q_off, q, buf.out, buf.lse)
    low = k.clone()
    low[:first, :, 3] = torch.finfo(torch.bfloat16).min      # so far below the others that they weigh 0
    again = attend(low, v, off, q, q_off, h_q)
    check([(k[first:], v[first:])], q_off, q, again.out, again.lse)
