"""What the binding of the new-token calls keeps and refuses, without a GPU: the
library's own calls are replaced where they would need one."""
import numpy as np
import pytest
import torch


@pytest.fixture
def ts(monkeypatch):
    import query_aware_kv_ts_b200 as m
    monkeypatch.setattr(m, "ts_dense_attn_workspace_bytes", lambda kv, off: 1024)
    monkeypatch.setattr(m, "ts_workspace_init", lambda ws, stream=None: None)
    return m


def cache(ts, n=40, batch=2):
    rows = torch.zeros((n, 2, 64), dtype=torch.bfloat16)
    return ts.KVCache(rows, rows.clone(), np.linspace(0, n, batch + 1).astype(np.int64), 8)


@pytest.mark.parametrize("kind", ["array", "tensor", "list"])
def test_buffers_keep_the_offsets_they_were_made_for(ts, kind):
    """A serving loop may update its own offsets in place: the buffers' host and
    device copies stay equal to each other."""
    own = {"array": np.array, "tensor": torch.tensor, "list": list}[kind]([0, 3, 7])
    buf = ts.DenseBuffers(cache(ts), own)
    for b in (1, 2):
        own[b] = b
    assert buf.q_offsets_host.tolist() == [0, 3, 7] == buf.q_offsets_dev.tolist()
    assert buf.rows == 7 and buf.out.shape[0] == 7


def test_a_cache_refuses_parts_on_another_device_and_short_tables(ts):
    """K decides where the calls run: V and the block table have to be there, and
    the table needs a row for every sequence."""
    k = torch.zeros((32, 2, 64), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    kept = ts.KVCache(k, k.clone(), [0, 16, 32], 8, page_table=table, page_size=16)
    assert kept.struct.page_table_stride == 2
    with pytest.raises(ValueError, match="device"):
        ts.KVCache(k, k.to("meta"), [0, 32], 8)
    with pytest.raises(ValueError, match="device"):
        ts.KVCache(k, k.clone(), [0, 16, 32], 8, page_table=table.to("meta"), page_size=16)
    with pytest.raises(ValueError, match="sequences"):
        ts.KVCache(k, k.clone(), [0, 8, 16, 32], 8, page_table=table, page_size=16)


def test_a_cache_refuses_offsets_that_pass_its_rows(ts):
    k = torch.zeros((32, 2, 64), dtype=torch.bfloat16)
    for off, capacity in (([0, 32], 0), ([0, 10], 32), ([0, 0], 0)):
        ts.KVCache(k, k.clone(), off, 8, capacity=capacity)
    for off, capacity in (([0, 33], 0), ([0, 10], 33)):
        with pytest.raises(ValueError, match="rows"):
            ts.KVCache(k, k.clone(), off, 8, capacity=capacity)
    table = torch.zeros((1, 4), dtype=torch.int32)
    ts.KVCache(k, k.clone(), [0, 60], 8, page_table=table, page_size=16)       # pages may be shared
