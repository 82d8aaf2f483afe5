"""PagedKV as an object (no GPU needed): the calls read the tensors that it was made of."""
import pytest
import torch

import q8_block_quantized_act_gb300 as q8


@pytest.fixture
def kv(monkeypatch):
    q8._load_torch()
    monkeypatch.setattr(q8, "_current", lambda: -1)
    k = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    i32 = dict(dtype=torch.int32)
    return q8.PagedKV(k, k.clone(), torch.zeros((2, 3), **i32), torch.zeros(3, **i32), torch.ones(2, **i32))


def test_contents_change_in_place(kv):
    kv.lens += 1
    kv.lens[0] = 7
    kv.starts[1:] = 1
    kv.table.fill_(3)
    kv.lens = kv.lens
    assert kv.lens.tolist() == [7, 2] and kv.c.lens == kv.lens.data_ptr() and kv.c.table == kv.table.data_ptr()


@pytest.mark.parametrize("name", ["k", "v", "table", "starts", "lens"])
def test_another_tensor_is_refused(kv, name):
    """It would be read by no call, and the one that is read could be freed."""
    old = getattr(kv, name)
    with pytest.raises(AttributeError, match="in place"):
        setattr(kv, name, old + 1)
    assert getattr(kv, name) is old


@pytest.mark.parametrize("name", ["c", "at", "device", "heads", "dim"])
def test_what_was_checked_stays(kv, name):
    with pytest.raises(AttributeError):
        setattr(kv, name, None)
