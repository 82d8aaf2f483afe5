"""Outputs of the paged cache's calls that overlap what other parts of the call still read: refused by the C ABI before any
CUDA call.  Layouts that share rows without sharing values pass that check; a later one refuses these calls here, so that
nothing is launched whatever machine this runs on."""
import pytest
import torch

import q8_block_quantized_act_gb300 as q8
from q8_block_quantized_act_gb300 import build as q8build

A = 1 << 24                      # a fake address, never dereferenced by these calls
F32, F16, BF16 = q8.Q8ACT_F32, q8.Q8ACT_F16, q8.Q8ACT_BF16
SIZE = {F32: 4, F16: 2, BF16: 2}
DIMS, ALIGN, WS, TYPE = q8.Q8ACT_ERR_DIMS, q8.Q8ACT_ERR_ALIGN, q8.Q8ACT_ERR_WORKSPACE, q8.Q8ACT_ERR_TYPE
D = 64


@pytest.fixture(scope="module", autouse=True)
def built():
    q8build.build()


def batch(t, heads=2):
    return q8.q8act_paged_kv(1 << 40, 1 << 41, heads * 16 * D, 4, 1 << 42, 3, 1 << 42, 1 << 42, 2, 3, 16, heads, D, t)


def attention(m, ldq, out, ldo, hq=4, t=F16, ot=F16):
    """The workspace is missing: what passes the check of overlaps is refused for that."""
    return q8.q8act_attention(batch(t), A, ldq, out, ldo, ot, hq, 0.125, 0, 1, m, None, 0, 0)


def append(m, ldq, qo, ldqo, k=1 << 30, ldk=256, v=1 << 31, ldv=256, hq=4, t=F16):
    """The frequencies stand askew: likewise."""
    return q8.q8act_append_kv(batch(F16), A, ldq, k, ldk, v, ldv, t, qo, ldqo, hq, (1 << 42) + 4, 64, 0, m, 0)


def touch(a, lda, na, b, ldb, nb, m):
    """Whether rows of na and nb bytes, lda and ldb apart, share a byte: looked at one by one."""
    mine = {x // 16 for i in range(m) for x in range(a + i * lda, a + i * lda + na, 16)}
    return any(x // 16 in mine for i in range(m) for x in range(b + i * ldb, b + i * ldb + nb, 16))


def test_attention_against_rows_one_by_one():
    """Rows equally far apart: exactly those that share a value are refused."""
    row, ld = 4 * D * 2, 4 * D * 2 + 3 * 128
    found = set()
    for ot in (F16, F32):
        width = 4 * D * SIZE[ot]
        for m in (1, 2, 3):
            for ld in (row + 128, 2 * row, row + width, 3 * row):
                if ld < width:
                    continue
                for off in range(-m * ld - width, m * ld + width, 64):
                    rc = attention(m, ld // 2, A + off, ld // SIZE[ot], ot=ot)
                    want = touch(A, ld, row, A + off, ld, width, m)
                    assert rc == (DIMS if want else WS), (ot, m, ld, off)
                    found.add((want, off > 0))
    assert len(found) == 4


@pytest.mark.parametrize("m,ldq,off,ldo,rc", [
    (1, 256, 256 * 2 - 16, 256, DIMS), (1, 256, 256 * 2, 256, WS),               # one row: what lies in it
    (1, 1 << 40, 256 * 2, 1 << 40, WS),
    (3, 256, 3 * 256 * 2, 512, WS), (3, 256, 2 * 256 * 2, 512, DIMS), (3, 512, -256 * 2, 256, DIMS),
    (3, 1024, 256 * 2, 512, DIMS),               # between each other, rows unequally far apart
    (1 << 20, 1 << 39, 256 * 2, 1 << 39, WS), (1 << 20, 1 << 39, 16, 1 << 39, DIMS), (1 << 20, 1 << 39, -16, 1 << 39, DIMS),
])
def test_attention(m, ldq, off, ldo, rc):
    assert attention(m, ldq, A + off, ldo) == rc


def test_append_queries():
    row = 4 * D
    assert append(3, row, A, row) == ALIGN                                       # the queries themselves
    for off in (-16, 16, 2 * row, -2 * row):
        assert append(3, row, A + off, row) == DIMS
    assert append(3, row, A + 2 * 3 * row, row) == ALIGN
    assert append(3, 3 * row, A + 2 * row, 3 * row) == ALIGN                     # beside them in wider rows
    assert append(3, 3 * row, A + 2 * row - 16, 3 * row) == DIMS
    # rows of another type end elsewhere: f32 queries, f16 rotated ones
    assert append(3, 2 * row, A + 4 * row, 4 * row, t=F32) == ALIGN
    assert append(3, 2 * row, A + 2 * row, 4 * row, t=F32) == DIMS


def test_append_keys_and_values():
    """Rotated queries over keys or values that another part of the call has still to read."""
    row, kv = 4 * D, 2 * D
    wide = row + 2 * kv                                                          # a fused projection's row
    at = dict(k=A + 2 * row, ldk=wide, v=A + 2 * (row + kv), ldv=wide)
    assert append(5, wide, A, wide, **at) == ALIGN
    for off in (row, row + kv, row - 8, row + 2 * kv - 8):
        assert append(5, wide, A + 2 * off, wide, **at) == DIMS
    assert append(1, wide, A + 2 * wide, wide, **at) == ALIGN


def test_helper_says_so(monkeypatch):
    """The same through the helpers, on tensors of this machine's memory."""
    q8._load_torch()
    monkeypatch.setattr(q8, "_current", lambda: -1)
    monkeypatch.setattr(q8, "_stream", lambda dev: 0)
    cache = torch.zeros((4, 2, 16, D), dtype=torch.float16)
    i32 = dict(dtype=torch.int32)
    kv = q8.PagedKV(cache, cache.clone(), torch.zeros((2, 3), **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    rows = torch.zeros((4, 4, D), dtype=torch.float16)
    ws = torch.zeros(1 << 26, dtype=torch.uint8)
    with pytest.raises(q8.Q8ActError) as e:
        q8.attention(kv, rows[:3], ws=ws, out=rows[1:])
    assert e.value.rc == DIMS
    with pytest.raises(q8.Q8ActError) as e:
        q8.append_kv(kv, rows[:3], cache[0, :, :3].transpose(0, 1).contiguous(), cache[0, :, :3].transpose(0, 1).contiguous(),
                     out=rows[1:])
    assert e.value.rc == DIMS


def test_helper_refuses_two_types(monkeypatch):
    """A dtype that `out` does not have (the same one passes: a later check refuses the window)."""
    q8._load_torch()
    monkeypatch.setattr(q8, "_current", lambda: -1)
    monkeypatch.setattr(q8, "_stream", lambda dev: 0)
    monkeypatch.setattr(q8, "lib", lambda: pytest.fail("reached the library"))
    cache = torch.zeros((4, 2, 16, D), dtype=torch.float16)
    i32 = dict(dtype=torch.int32)
    kv = q8.PagedKV(cache, cache.clone(), torch.zeros((2, 3), **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    q, ws = torch.zeros((3, 4, D), dtype=torch.float16), torch.zeros(64, dtype=torch.uint8)
    for out in (torch.zeros((3, 4, D)), torch.zeros((3, 4, D), dtype=torch.bfloat16)):
        with pytest.raises(q8.Q8ActError) as e:
            q8.attention(kv, q, ws=ws, out=out, dtype=torch.float16)
        assert e.value.rc == TYPE
    with pytest.raises(q8.Q8ActError) as e:
        q8.attention(kv, q, ws=ws, out=torch.zeros((3, 4, D)), dtype=torch.float32, window=-1)
    assert e.value.rc == DIMS
