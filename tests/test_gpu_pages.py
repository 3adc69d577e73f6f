"""Room for new tokens in a paged cache (ts_extend_pages) and their rows in it
(ts_write_kv) against plain loops; whole numbers and copies, so equality."""
import numpy as np
import pytest
import torch

import gpu_helpers as H

pytestmark = pytest.mark.gpu


def plain(cached, fresh, page, free, pool_pages, table, n_slots):
    """The definition, token by token."""
    table = table.copy()
    stride = table.shape[1]
    slots, used, q_off, s_off = np.full(n_slots, -1, np.int64), 0, [0], [0]
    for b, (c, f) in enumerate(zip(cached, fresh)):
        have = min(-(-c // page), stride)
        new = min(-(-(c + f) // page), stride) - have
        for i in range(new):
            first = (have + i) * page - c           # the token that opens the page, among the sequence's new ones
            if q_off[-1] + first < n_slots:
                at = used + i
                ok = at < len(free) and 0 <= free[at] < pool_pages
                table[b, have + i] = free[at] if ok else -1
        for j in range(f):
            t, r = c + j, q_off[-1] + j
            if r < n_slots and t // page < stride:
                p = table[b, t // page]
                slots[r] = p * page + t % page if 0 <= p < pool_pages else -1
        used += new
        q_off.append(q_off[-1] + f)
        s_off.append(s_off[-1] + c + f)
    return table, np.array(s_off), np.array(q_off), slots, used


def extend(cached, fresh, page, free, pool_pages, table, n_slots):
    dev = {"dtype": torch.int64, "device": "cuda"}
    t = torch.from_numpy(table).cuda()
    B = len(cached)
    so, qo = torch.full((B + 1,), -7, **dev), torch.full((B + 1,), -7, **dev)
    slots, used = torch.full((n_slots,), -7, **dev), torch.full((1,), -7, **dev)
    args = (torch.tensor(cached, **dev), torch.tensor(fresh, **dev), page,
            torch.tensor(free, dtype=torch.int32, device="cuda"), pool_pages, t, so, qo, slots, used)
    H.ts().ts_extend_pages(*args)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, so, qo, slots)] + [int(used)], args


def case(B, page, hi_cached, hi_fresh, seed, pad=0, zeros=0.2):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, hi_cached + 1, B)
    fresh = rng.integers(0, hi_fresh + 1, B)
    cached[rng.random(B) < zeros] = 0
    fresh[rng.random(B) < zeros] = 0
    have = -(-cached // page)
    need = int((-(-(cached + fresh) // page) - have).sum())
    pool = int(have.sum()) + need + 5
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((B, max(1, int((-(-(cached + fresh) // page)).max()))), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    return cached.tolist(), fresh.tolist(), page, perm[at:].tolist(), pool, table, int(fresh.sum()) + pad


@pytest.mark.parametrize("B,page,hi_cached,hi_fresh,pad", [
    (1, 16, 0, 1, 0), (1, 8, 7, 9, 3), (3, 16, 100, 1, 0), (5, 64, 1000, 700, 11), (31, 8, 50, 3, 1), (33, 16, 300, 40, 0),
    (256, 16, 4000, 1, 0), (257, 32, 200, 100, 5), (1023, 128, 500, 30, 0), (1024, 8, 30, 20, 2), (2, 4096, 9000, 9000, 0),
    (4, 16, 100, 40000, 0)])
def test_extend_pages(B, page, hi_cached, hi_fresh, pad):
    for seed in range(3):
        c = case(B, page, hi_cached, hi_fresh, seed, pad)
        got, args = extend(*c)
        for g, w in zip(got, plain(*c)):
            assert np.array_equal(g, w)
        H.ts().ts_extend_pages(*args)              # the same again: nothing is kept
        torch.cuda.synchronize()
        assert np.array_equal(args[5].cpu().numpy(), got[0]) and np.array_equal(args[8].cpu().numpy(), got[3])


def test_extend_pages_when_the_free_list_runs_out():
    cached, fresh, page, free, pool, table, n = case(9, 16, 100, 200, 4)
    for keep in (0, 1, 5):
        c = (cached, fresh, page, free[:keep], pool, table, n)
        got, _ = extend(*c)
        for g, w in zip(got, plain(*c)):
            assert np.array_equal(g, w)
        assert got[4] > keep
    bad = list(free)
    bad[2], bad[3] = pool, -5                      # no pages of the pool
    c = (cached, fresh, page, bad, pool, table, n)
    got, _ = extend(*c)
    for g, w in zip(got, plain(*c)):
        assert np.array_equal(g, w)


def test_extend_pages_beyond_its_bounds():
    """A table too narrow, a slot map too short, a table with entries outside
    the pool, lengths below zero: bounded, and -1 or left out."""
    cached, fresh, page, free, pool, table, n = case(6, 8, 60, 90, 7)
    narrow = np.ascontiguousarray(table[:, :5])
    for c in ((cached, fresh, page, free, pool, narrow, n), (cached, fresh, page, free, pool, table, n // 2),
              (cached, fresh, page, free, pool, table, 0),
              (cached, fresh, page, free, pool, np.where(table % 3 == 0, 10 ** 6, table).astype(np.int32), n)):
        got, _ = extend(*c)
        for g, w in zip(got, plain(*c)):
            assert np.array_equal(g, w)
    got, _ = extend([-5, 3], [4, -2], 8, [1, 0], 2, np.full((2, 2), -1, np.int32), 6)
    want = plain([0, 3], [4, 0], 8, [1, 0], 2, np.full((2, 2), -1, np.int32), 6)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_extend_pages_captured_and_replayed_with_other_lengths():
    B, page, pool = 5, 16, 64
    dev = {"dtype": torch.int64, "device": "cuda"}
    cached, fresh = torch.zeros(B, **dev), torch.ones(B, **dev)
    free = torch.randperm(pool, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    so, qo, slots, used = torch.zeros(B + 1, **dev), torch.zeros(B + 1, **dev), torch.zeros(40, **dev), torch.zeros(1, **dev)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        H.ts().ts_extend_pages(cached, fresh, page, free, pool, table, so, qo, slots, used)
    torch.cuda.synchronize()
    rng = np.random.default_rng(0)
    for _ in range(4):
        c, f = rng.integers(0, 90, B), rng.integers(0, 9, B)
        t0 = np.arange(B * 8, dtype=np.int32).reshape(B, 8)
        cached.copy_(torch.from_numpy(c))
        fresh.copy_(torch.from_numpy(f))
        table.copy_(torch.from_numpy(t0))
        graph.replay()
        torch.cuda.synchronize()
        want = plain(c.tolist(), f.tolist(), page, free.tolist(), pool, t0, 40)
        for g, w in zip((table, so, qo, slots, used), want):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w).reshape(g.shape))


@pytest.mark.parametrize("layout", ["packed", "paged", "gaps", "capacity"])
@pytest.mark.parametrize("h_kv,d", [(1, 64), (4, 128), (8, 128), (2, 64), (8, 64)])
@pytest.mark.parametrize("n_new", [0, 1, 3, 500, 2049])
def test_write_kv(n_new, h_kv, d, layout):
    m = H.ts()
    rows = 4096
    g = torch.Generator(device="cuda").manual_seed(n_new + d)

    def bits(*shape):      # every bit pattern, NaN's among them: a copy
        return torch.randint(-32768, 32768, shape, device="cuda", generator=g, dtype=torch.int16).view(torch.bfloat16)

    wide = bits(rows, 2 * h_kv, d)
    k, v = (wide[:, ::2], wide.clone()[:, ::2]) if layout == "gaps" else (bits(rows, h_kv, d), bits(rows, h_kv, d))
    if layout == "paged":
        kv = m.KVCache(k, v, [0, 100], h_kv, page_table=torch.zeros((1, 7), dtype=torch.int32, device="cuda"), page_size=16)
    elif layout == "capacity":
        kv = m.KVCache(k, v, [0, 100], h_kv, capacity=rows)
    else:
        kv = m.KVCache(k, v, [0, 50, rows], h_kv)
    x = bits(n_new + 3, 5 * h_kv, d)
    k_new, v_new = x[:n_new, h_kv:2 * h_kv], x[:n_new, 3 * h_kv:4 * h_kv]
    slots = torch.randperm(rows, device="cuda", generator=g)[:n_new].contiguous()
    slots[1::7] = -1
    slots[2::11] = rows                    # outside the cache
    slots[5::13] = 2 ** 40
    want_k, want_v = k.contiguous().view(torch.int16), v.contiguous().view(torch.int16)
    keep = (slots >= 0) & (slots < rows)
    want_k[slots[keep]] = k_new.contiguous().view(torch.int16)[keep]
    want_v[slots[keep]] = v_new.contiguous().view(torch.int16)[keep]
    gaps = wide[:, 1::2].clone().view(torch.int16)
    m.ts_write_kv(kv, k_new, v_new, slots)
    torch.cuda.synchronize()
    assert torch.equal(k.contiguous().view(torch.int16), want_k)
    assert torch.equal(v.contiguous().view(torch.int16), want_v)
    assert torch.equal(wide[:, 1::2].contiguous().view(torch.int16), gaps)


def test_write_kv_to_one_slot_twice():
    """Each 16-byte piece is one of the two rows'."""
    m = H.ts()
    k = torch.zeros((16, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv = m.KVCache(k, k.clone(), [0, 16], 2)
    new = torch.stack([torch.full((2, 64), 1.0), torch.full((2, 64), 2.0)]).to(torch.bfloat16).cuda()
    m.ts_write_kv(kv, new, new, torch.tensor([3, 3], device="cuda"))
    torch.cuda.synchronize()
    piece = kv.k[3].view(-1, 8)
    assert ((piece == 1).all(1) | (piece == 2).all(1)).all()
    assert (kv.k[:3] == 0).all() and (kv.k[4:] == 0).all()


def test_rows_past_two_to_the_31_elements():
    """A pool whose last rows lie past 2^31 elements of K."""
    m = H.ts()
    rows, h_kv, d = 2 ** 21 + 48, 8, 128
    k = torch.zeros((rows, h_kv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    kv = m.KVCache(k, v, [0, 16], h_kv, page_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"), page_size=16)
    new = torch.ones((2, h_kv, d), dtype=torch.bfloat16, device="cuda")
    m.ts_write_kv(kv, new, 2 * new, torch.tensor([rows - 1, rows], device="cuda"))
    torch.cuda.synchronize()
    assert (k[-1] == 1).all() and (v[-1] == 2).all() and (k[-2] == 0).all()
    assert float(k.sum(dtype=torch.float64)) == h_kv * d


def test_the_binding_refuses_what_the_kernels_could_not_read():
    """Wrong types, sizes, strides and devices, told by name, before any launch."""
    m = H.ts()
    c = case(3, 16, 100, 50, 1)
    _, good = extend(*c)
    t = torch.zeros
    for at, bad in ((0, good[0].int()), (1, good[1][:2]), (3, good[3].long()), (5, good[5].t()), (5, good[5][:2]), (6, good[6][:3]),
                    (7, good[7].cpu()), (8, t(40, dtype=torch.int64, device="cuda")[::2]), (8, good[8].float()),
                    (9, t(2, dtype=torch.int64, device="cuda")), (9, [0])):
        args = list(good)
        args[at] = bad
        with pytest.raises((TypeError, ValueError, AttributeError)):
            m.ts_extend_pages(*args)
    k = t((32, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv, new = m.KVCache(k, k.clone(), [0, 32], 2), t((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = t(4, dtype=torch.int64, device="cuda")
    for args in ((new, new, slots.int()), (new, new, slots[:3]), (new, new[:3], slots), (new.float(), new, slots),
                 (new, new.cpu(), slots), (new[:, :1], new[:, :1], slots), (new, torch.cat([new, new], 1)[:, :2], slots),
                 (new.transpose(1, 2), new, slots), (new, new, slots.cpu())):
        with pytest.raises((TypeError, ValueError)):
            m.ts_write_kv(kv, *args)
    buf = m.DenseBuffers(kv, [0, 4])
    ok = (kv, new, buf.q_offsets_dev, buf.q_offsets_host, buf.out, buf.lse, buf.ws)
    for at, bad in ((1, new[:3]), (1, new.float()), (2, buf.q_offsets_dev.int()), (2, buf.q_offsets_dev[:1]), (3, [0, 1, 2]),
                    (4, buf.out.float()), (4, buf.out[:3]), (4, torch.cat([buf.out, buf.out], 1)[:, :2]), (5, buf.lse[:3]),
                    (5, buf.lse.double()), (6, buf.ws.cpu())):
        args = list(ok)
        args[at] = bad
        with pytest.raises((TypeError, ValueError)):
            m.ts_dense_attn(*args)
    with pytest.raises(m.TsError) as e:
        m.ts_dense_attn(*ok[:6], buf.ws[:16])
    assert e.value.status == m.TS_ERR_WORKSPACE
    with pytest.raises(m.TsError, match="non-decreasing"):
        m.ts_dense_attn(*ok[:3], [0, -1], *ok[4:])
