"""ts_dense_attn where a row's scores, values or cache are out of the ordinary:
against the definition in 64 bits of test_gpu_dense.py, with its bounds."""
import numpy as np
import pytest
import torch

import gpu_helpers as H
import workloads as W
from test_gpu_dense import attend, check, definition, inputs, paged, sequences

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fresh", [2, 60, 400])
@pytest.mark.parametrize("first", [40, 128])
def test_a_tile_done_again_beside_rows_without_a_reference(first, fresh):
    """Every other head's scores of the first tokens are -inf, so that it has no
    reference yet at the second tile, where the other heads' scores rise 45
    above theirs: their sums so far are rescaled twice at one tile."""
    n, h_q, h_kv, d = 600, 14, 2, 128
    off, q_off, q, k, v = inputs([n], [fresh], h_q, h_kv, d, 43)
    k[:first, :, 3] = -3e38
    k[first:, :, 3] = 0
    q[:, ::2, 3], q[:, 1::2, 3] = 0, 1e5
    k[:128, :, 5], k[128:, :, 5] = 0, 64
    q[:, :, 5] = 8
    buf = attend(k, v, off, q, q_off, h_q)
    for heads, behind in ((slice(0, None, 2), 0), (slice(1, None, 2), first)):
        want, want_lse, tol, tol_lse = (x[:, heads] for x in definition(q, k[behind:], v[behind:], n - behind))
        assert ((buf.out[:, heads].double() - want).abs() <= tol).all()
        assert ((buf.lse[:, heads].double() - want_lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("fresh", [1, 40])
@pytest.mark.parametrize("n,low", [(120, (16, 32)), (700, (128, 384)), (5000, (0, 2000)), (5000, (3000, 4200))], ids=str)
@pytest.mark.parametrize("h_q", [14, 32])
def test_what_a_row_sees_far_below_its_maximum_stays_visible(h_q, n, low, fresh):
    """A NaN in K, or a NaN or infinity in V, of a token whose neighbours' scores
    lie 135 below the others': their weights are 0 in fp32, but the row does
    see the token, wherever the work was cut."""
    h_kv, d = 2, 128
    off, q_off, q, k, v = inputs([n], [fresh], h_q, h_kv, d, 47)
    q[:, :, 5] = 8
    k[:, :, 5] = 0
    k[low[0]:low[1], :, 5] = -192
    clean = attend(k, v, off, q, q_off, h_q)
    assert clean.out.isfinite().all()
    at = (low[0] + low[1]) // 2
    for what in ("k_nan", "v_nan", "v_inf"):
        k2, v2 = k.clone(), v.clone()
        if what == "k_nan":
            k2[at] = float("nan")
        else:
            v2[at, :, 7] = float("nan") if what == "v_nan" else float("inf")
        buf = attend(k2, v2, off, q, q_off, h_q)
        if what == "k_nan":
            assert buf.out.isnan().all() and buf.lse.isnan().all()
        else:
            assert not buf.out[:, :, 7].isfinite().any(), what
            rest = [c for c in range(d) if c != 7]
            assert torch.equal(buf.out[:, :, rest], clean.out[:, :, rest]) and torch.equal(buf.lse, clean.lse)


@pytest.mark.parametrize("fresh", [1, 30])
@pytest.mark.parametrize("page", [16, 256])
def test_lengths_on_the_device_that_pass_the_block_table(page, fresh):
    """What stands in memory behind a sequence's row of the table is not taken
    for its pages: here they would be pages of NaN."""
    m = H.ts()
    h_q, h_kv, d, n, stride = 8, 2, 128, 4 * page, 4
    off, q_off, q, k, v = inputs([n], [fresh], h_q, h_kv, d, 51)
    kp, vp, table = paged(k, v, off, page, 1)
    owned = set(table.flatten().tolist())
    stray = next(p for p in range(kp.shape[0] // page) if p not in owned)
    around = torch.full((64 * stride,), stray, dtype=torch.int32, device="cuda")
    around[:stride] = table.flatten()
    kv = m.KVCache(kp, vp, off, h_q, page_table=around[:stride].view(1, stride), page_size=page)
    buf = m.DenseBuffers(kv, q_off)
    kv.seq_offsets_dev[1] = n + 20 * page
    m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)
    torch.cuda.synchronize()
    assert m.ts_get_device_status(buf.ws) == (m.TS_OK, 0)
    assert buf.out.isfinite().all() and buf.lse.isfinite().all()
    kv.seq_offsets_dev[1] = n
    m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)
    torch.cuda.synchronize()
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse)


@pytest.mark.parametrize("longest", [True, False])
@pytest.mark.parametrize("fresh", [[1, 1, 1], [1, 0, 5], [2, 40, 1]], ids=str)
def test_a_captured_step_of_a_growing_paged_batch(fresh, longest):
    """One graph of [room, rows, attention] on a paged batch: the lengths grow on
    the device from replay to replay.  Captured with the longest lengths to
    come in the host's offsets, or with the first ones."""
    m = H.ts()
    h_q, h_kv, d, page, steps = 28, 4, 128, 16, 30
    start = np.array([700, 5, 130])
    fresh = np.array(fresh)
    end = start + (steps + 1) * fresh
    stride = int(-(-end.max() // page))
    pool = int((-(-end // page)).sum()) + 7
    g = torch.Generator(device="cuda").manual_seed(61)
    new = [torch.randn((steps + 1, int(fresh.sum()), h, d), device="cuda", generator=g).to(torch.bfloat16) for h in (h_q, h_kv, h_kv)]
    first = [[torch.randn((int(n), h_kv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)] for n in start]
    pool_k = torch.full((pool * page, h_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool_v = pool_k.clone()
    dev = {"dtype": torch.int64, "device": "cuda"}
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    table = torch.full((3, stride), -1, dtype=torch.int32, device="cuda")
    host = W.seq_offsets(end if longest else start)
    kv = m.KVCache(pool_k, pool_v, host, h_q, page_table=table, page_size=page)
    buf = m.DenseBuffers(kv, W.seq_offsets(fresh))
    cached, count, used = torch.zeros(3, **dev), torch.from_numpy(start).cuda(), torch.zeros(1, **dev)
    slots = torch.zeros(int(start.sum()), **dev)
    qo = torch.zeros(4, **dev)
    m.ts_extend_pages(cached, count, page, order, pool, table, kv.seq_offsets_dev, qo, slots, used)
    m.ts_write_kv(kv, torch.cat([x[0] for x in first]), torch.cat([x[1] for x in first]), slots)
    torch.cuda.synchronize()
    taken = int(used)
    cached.copy_(count)
    count.copy_(torch.from_numpy(fresh))
    free, slots = order.clone(), torch.zeros(int(fresh.sum()), **dev)
    q, kn, vn = (x[0].clone() for x in new)

    def step():
        m.ts_extend_pages(cached, count, page, free, pool, table, kv.seq_offsets_dev, buf.q_offsets_dev, slots, used)
        m.chunk_step(kv, q, kn, vn, slots, buf)
        cached.add_(count)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    for i in range(steps + 1):
        free[:pool - taken] = order[taken:]
        for to, x in zip((q, kn, vn), new):
            to.copy_(x[i])
        torch.cuda.synchronize()
        if i == 0:
            with torch.cuda.stream(s):
                step()                     # warm-up
                s.synchronize()
                with torch.cuda.graph(graph, stream=s):
                    step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        taken += int(used)
        lengths = start + (i + 1) * fresh
        assert cached.tolist() == lengths.tolist() and kv.seq_offsets_dev.tolist() == W.seq_offsets(lengths).tolist()
        if i % 7 and i != steps:
            continue
        at = W.seq_offsets(fresh)
        rows = [tuple(torch.cat([first[b][c]] + [x[j, int(at[b]):int(at[b + 1])] for j in range(i + 1)]) for c, x in ((0, new[1]), (1, new[2])))
                for b in range(3)]
        check(rows, at, q, buf.out, buf.lse)
    assert m.ts_get_device_status(buf.ws) == (m.TS_OK, 0)


def test_a_workspace_with_fewer_bytes_than_elements_is_refused():
    """An expanded or strided tensor counts elements that it does not hold."""
    m = H.ts()
    off, q_off, q, k, v = inputs([40], [40], 8, 2, 64, 5)
    kv = m.KVCache(k, v, off, 8)
    buf = m.DenseBuffers(kv, q_off)
    n = buf.ws.numel()
    for ws in (buf.ws[:1].expand(n), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, ws)
    with pytest.raises(m.TsError, match="too small"):
        m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws[:n - 256])
    m.ts_dense_attn(kv, q, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)
    torch.cuda.synchronize()
    check(sequences(k, v, off), q_off, q, buf.out, buf.lse)


def cancelling(lengths, h_q, h_kv, d, seed):
    """One query token a sequence whose weights nearly cancel in V, so that the
    output's own rounding hides nothing: 16 tokens with weights of one size and
    a heavier one whose V takes their sum away (channel c: for head c % G of its
    kv head), the others 40 and more below them.  K has one channel, so the
    scores are one exact product each.  On the CPU, from the seed alone."""
    g = torch.Generator().manual_seed(seed)
    G, scale = h_q // h_kv, d ** -0.5
    B, off = len(lengths), W.seq_offsets(lengths)
    q = torch.zeros((B, h_q, d), dtype=torch.bfloat16)
    q[:, :, 0] = 1 + torch.rand((B, h_q), generator=g)
    k = torch.zeros((int(off[-1]), h_kv, d), dtype=torch.bfloat16)
    v = torch.randn(k.shape, generator=g).to(torch.bfloat16)
    k[:, :, 0] = -1000
    want = torch.zeros((B, h_q, d), dtype=torch.float64)
    size, plain_bf16 = torch.zeros_like(want), torch.zeros_like(want)      # sum w |V|; with weights of 8 bits
    for b in range(B):
        at = int(off[b]) + torch.randperm(int(lengths[b]), generator=g)[:17]
        for h in range(h_kv):
            k[at, h, 0] = torch.cat([torch.rand(16, generator=g) * 12 - 8, torch.tensor([8.0])]).to(torch.bfloat16)
            s = q[b, h * G:(h + 1) * G, 0].double().unsqueeze(1) * k[at, h, 0].double() * scale
            e = torch.exp(s - s.amax(1, keepdim=True))
            w = e / e.sum(1, keepdim=True)
            for c in range(d):
                v[at[16], h, c] = -(w[c % G, :16] @ v[at[:16], h, c].double()) / w[c % G, 16]
            rows, vv = slice(h * G, (h + 1) * G), v[at, h].double()
            want[b, rows], size[b, rows] = w @ vv, w @ vv.abs()
            plain_bf16[b, rows] = e.to(torch.bfloat16).double() @ vv / e.sum(1, keepdim=True)
    return off, q, k, v, want, size, plain_bf16


@pytest.mark.parametrize("lengths", [[60], [1000], [300, 17, 128, 129] * 10], ids=["whole", "shared", "many"])
@pytest.mark.parametrize("heads", [(28, 4, 128), (8, 1, 128), (32, 2, 128), (12, 1, 128), (4, 2, 64), (16, 1, 64)], ids=str)
def test_the_weights_of_one_token_are_a_bf16_and_its_remainder(heads, lengths):
    """Up to 8 heads a group a weight's bf16 is off by 2^-8 of it and the
    remainder's by 2^-8 of that: 2^-16.  Above, the first is cut off (2^-7):
    2^-15.  The rest as in test_gpu_dense.py, the scores being one exact product
    and its scaling (at most 2 in size): n 2^-23 for the sums, 2^-20 for the
    exponentials and the normaliser, 2 x 2 x 2^-22 for the scaling.  Weights
    40 below add less than 2^-40.  Weights without their remainder (the oracle's)
    are far outside."""
    h_q, h_kv, d = heads
    off, q, k, v, want, size, plain_bf16 = cancelling(lengths, h_q, h_kv, d, 71)
    n = torch.tensor(lengths, dtype=torch.float64).view(-1, 1, 1)
    weight = 2.0 ** -16 if h_q // h_kv <= 8 else 2.0 ** -15
    tol = size * (weight + n * 2.0 ** -23 + 2.0 ** -19) + want.abs() * 2.0 ** -8
    assert ((plain_bf16 - want).abs() > tol).double().mean() > 0.25
    buf = attend(k.cuda(), v.cuda(), off, q.cuda(), list(range(len(lengths) + 1)), h_q)
    err = (buf.out.double().cpu() - want).abs()
    assert (err <= tol).all(), "worst %.3g of the bound" % float((err / tol).max())


@pytest.mark.parametrize("fresh", [1, 2, 200])
@pytest.mark.parametrize("n", [100, 200, 3100])
@pytest.mark.parametrize("h_q", [14, 32])
def test_rows_of_infinite_scores(h_q, n, fresh):
    """Scores that are all -inf leave nothing: zeros and -inf.  One of +inf, like
    one of NaN, makes the row NaN."""
    h_kv, d = 2, 128
    fresh = min(fresh, n)
    off, q_off, q, k, v = inputs([n, 40], [fresh, 40], h_q, h_kv, d, 83)
    clean = attend(k, v, off, q, q_off, h_q)
    q[:fresh, :, 3] = 1
    k2 = k.clone()
    k2[:n, :, 3] = float("-inf")
    buf = attend(k2, v, off, q, q_off, h_q)
    assert (buf.out[:fresh] == 0).all() and (buf.lse[:fresh] == float("-inf")).all()
    assert torch.equal(buf.out[fresh:], clean.out[fresh:]) and torch.equal(buf.lse[fresh:], clean.lse[fresh:])
    at = n - fresh // 2 - 1
    k2 = k.clone()
    k2[at, :, 3] = float("inf")
    buf = attend(k2, v, off, q, q_off, h_q)
    first = at - (n - fresh)              # the first query row that sees the token
    assert buf.out[:first].isfinite().all() and buf.lse[:first].isfinite().all()
    assert buf.out[first:fresh].isnan().all() and buf.lse[first:fresh].isnan().all()
    assert torch.equal(buf.out[fresh:], clean.out[fresh:]) and torch.equal(buf.lse[fresh:], clean.lse[fresh:])
