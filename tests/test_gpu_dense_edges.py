"""ts_dense_attn where a row's scores, values or cache are out of the ordinary:
against the definition in 64 bits of test_gpu_dense.py, with its bounds."""
import pytest
import torch

import gpu_helpers as H
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
