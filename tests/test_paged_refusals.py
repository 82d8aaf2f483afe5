"""Refusals of the paged cache's calls: by the C ABI before any CUDA call, and by the torch helpers before
they pass an address (no GPU needed, nothing is launched)."""
import ctypes

import pytest
import torch

import q8_block_quantized_act_gb300 as q8
from q8_block_quantized_act_gb300 import build as q8build

A, B = 1 << 20, 1 << 21          # fake, 16-byte aligned addresses: never dereferenced by these calls
MIS = A + 4
F32, F16, BF16 = q8.Q8ACT_F32, q8.Q8ACT_F16, q8.Q8ACT_BF16
NULL, DIMS, ALIGN, WS, TYPE = (q8.Q8ACT_ERR_NULL, q8.Q8ACT_ERR_DIMS, q8.Q8ACT_ERR_ALIGN, q8.Q8ACT_ERR_WORKSPACE,
                               q8.Q8ACT_ERR_TYPE)


@pytest.fixture(scope="module", autouse=True)
def built():
    q8build.build()


def batch(k=A, v=A, stride=2 * 16 * 64, pages=4, table=A, table_ld=3, starts=A, lens=A, seqs=2, width=3, page=16, heads=2,
          dim=64, type=F16):
    return q8.q8act_paged_kv(k, v, stride, pages, table, table_ld, starts, lens, seqs, width, page, heads, dim, type)


def append(kv=None, q=A, ldq=256, k=A, ldk=128, v=A, ldv=128, t=F32, qo=B, ldqo=256, hq=4, turns=A, rot=64, il=0, m=3, **b):
    kv = batch(**b) if kv is None else kv
    return q8.q8act_append_kv(kv or None, q, ldq, k, ldk, v, ldv, t, qo, ldqo, hq, turns, rot, il, m, 0)


def attend(kv=None, q=A, ldq=256, out=B, ldo=256, ot=F16, hq=4, scale=0.125, window=0, max_new=1, m=3, ws=A, nb=None, **b):
    kv = batch(**b) if kv is None else kv
    nb = 1 << 40 if nb is None else nb
    return q8.q8act_attention(kv or None, q, ldq, out, ldo, ot, hq, scale, window, max_new, m, ws, nb, 0)


BATCH = [
    (NULL, dict(kv=False)), (NULL, dict(k=None)), (NULL, dict(table=None)), (NULL, dict(starts=None)), (NULL, dict(lens=None)),
    (TYPE, dict(type=F32)), (TYPE, dict(type=7)), (TYPE, dict(type=-1)),
    (DIMS, dict(dim=32)), (DIMS, dict(dim=96)), (DIMS, dict(dim=256)), (DIMS, dict(page=8)), (DIMS, dict(page=48)),
    (DIMS, dict(page=2048)), (DIMS, dict(page=0)), (DIMS, dict(page=-16)), (DIMS, dict(heads=0)), (DIMS, dict(heads=-1)),
    (DIMS, dict(heads=4096)), (DIMS, dict(pages=0)), (DIMS, dict(pages=2 ** 31)), (DIMS, dict(stride=2 * 16 * 64 - 8)),
    (DIMS, dict(stride=1 << 40)), (DIMS, dict(seqs=0)), (DIMS, dict(seqs=(1 << 16) + 1)), (DIMS, dict(width=0)),
    (DIMS, dict(width=1 << 27, table_ld=1 << 27)), (DIMS, dict(table_ld=2)), (DIMS, dict(m=0)), (DIMS, dict(m=-1)),
    (DIMS, dict(m=1 << 40)), (DIMS, dict(m=1 << 28)),
    (ALIGN, dict(k=MIS)), (ALIGN, dict(stride=2 * 16 * 64 + 4)), (ALIGN, dict(table=A + 2)), (ALIGN, dict(starts=A + 1)),
    (ALIGN, dict(lens=A + 3)),
]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("rc,args", BATCH, ids=str)
def test_batch(call, rc, args):
    assert call(**args) == rc


@pytest.mark.parametrize("rc,args", [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(q=None)), (NULL, dict(qo=None)), (NULL, dict(hq=0)),
    (NULL, dict(turns=None)), (NULL, dict(rot=0)), (TYPE, dict(t=9)),
    (DIMS, dict(rot=8)), (DIMS, dict(rot=72)), (DIMS, dict(rot=80)), (DIMS, dict(rot=-16)), (DIMS, dict(il=2)),
    (DIMS, dict(hq=5000)), (DIMS, dict(hq=-1)), (DIMS, dict(ldq=255)), (DIMS, dict(ldk=127)), (DIMS, dict(ldv=64)),
    (DIMS, dict(ldqo=128)), (ALIGN, dict(ldq=258)), (ALIGN, dict(ldk=129)), (ALIGN, dict(ldv=130)), (ALIGN, dict(ldqo=260)),
    (TYPE, dict(qo=A)), (TYPE, dict(qo=A, t=BF16)), (DIMS, dict(qo=A, t=F16, ldq=512)),
    (ALIGN, dict(q=MIS)), (ALIGN, dict(v=MIS)), (ALIGN, dict(qo=MIS)), (ALIGN, dict(turns=A + 4)),
], ids=str)
def test_append(rc, args):
    if "k" in args or "v" in args:                   # the projection's, not the cache's
        kv = batch()
        kw = dict(q=A, ldq=256, k=A, ldk=128, v=A, ldv=128)
        kw.update(args)
        assert q8.q8act_append_kv(kv, kw["q"], 256, kw["k"], 128, kw["v"], 128, F32, A, 256, 4, A, 64, 0, 3, 0) == rc
    else:
        assert append(**args) == rc


@pytest.mark.parametrize("rc,args", [
    (NULL, dict(q=None)), (NULL, dict(out=None)), (DIMS, dict(out=A)), (TYPE, dict(ot=3)), (DIMS, dict(hq=3)), (DIMS, dict(hq=0)),
    (DIMS, dict(hq=1)), (DIMS, dict(hq=8192)), (DIMS, dict(scale=0.0)), (DIMS, dict(scale=-1.0)), (DIMS, dict(scale=float("nan"))),
    (DIMS, dict(scale=float("inf"))), (DIMS, dict(scale=2.0 ** 101)), (DIMS, dict(window=-1)), (DIMS, dict(window=2 ** 31 - 1)), (DIMS, dict(max_new=-1)),
    (DIMS, dict(ldq=255)), (DIMS, dict(ldo=128)), (ALIGN, dict(ldq=260)), (ALIGN, dict(ldo=257)), (ALIGN, dict(q=MIS)),
    (ALIGN, dict(out=MIS)), (WS, dict(ws=None)), (WS, dict(nb=100)), (ALIGN, dict(ws=MIS)),
], ids=str)
def test_attention(rc, args):
    assert attend(**args) == rc


def test_workspace():
    n = q8.q8act_attention_workspace_bytes(32, 8, 128)
    assert 0 < n < 1 << 30 and attend(hq=4, nb=q8.q8act_attention_workspace_bytes(4, 2, 64) - 1) == WS
    for bad in ((0, 8, 128), (8, 0, 128), (4, 8, 128), (12, 8, 128), (32, 8, 96), (32, 8, 0), (-8, 8, 128), (8192, 1, 64)):
        assert q8.q8act_attention_workspace_bytes(*bad) == 0


def test_struct_has_the_c_layout():
    assert ctypes.sizeof(q8.q8act_paged_kv) == 88 and q8.q8act_paged_kv.seqs.offset == 64


@pytest.fixture
def here(monkeypatch):
    """Lets CPU tensors pass as tensors of the current device; nothing may reach the library."""
    q8._load_torch()
    monkeypatch.setattr(q8, "_current", lambda: -1)
    monkeypatch.setattr(q8, "_stream", lambda dev: 0)
    monkeypatch.setattr(q8, "lib", lambda: pytest.fail("reached the library"))


def tensors(pages=4, heads=2, page=16, dim=64, seqs=2, t=torch.float16):
    k = torch.zeros((pages, heads, page, dim), dtype=t)
    i32 = torch.int32
    return [k, k.clone(), torch.zeros((seqs, 3), dtype=i32), torch.zeros(seqs + 1, dtype=i32), torch.zeros(seqs, dtype=i32)]


def raises(rc, f, *args, **kw):
    with pytest.raises(q8.Q8ActError) as e:
        f(*args, **kw)
    assert e.value.rc == rc, str(e.value)


def test_helper_cache(here):
    q8.PagedKV(*tensors())
    for rc, i, x in [
        (TYPE, 0, torch.zeros((4, 2, 16, 64))), (TYPE, 1, torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)),
        (DIMS, 0, torch.zeros((4, 2, 16), dtype=torch.float16)), (DIMS, 1, torch.zeros((5, 2, 16, 64), dtype=torch.float16)),
        (DIMS, 0, torch.zeros((4, 16, 2, 64), dtype=torch.float16).transpose(1, 2)),
        (DIMS, 0, torch.zeros((4, 2, 16, 128), dtype=torch.float16)[..., ::2]),
        (DIMS, 1, torch.zeros((4, 2, 2, 16, 64), dtype=torch.float16)[:, 0]),
        (DIMS, 2, torch.zeros(3, dtype=torch.int32)), (DIMS, 2, torch.zeros((2, 6), dtype=torch.int32)[:, ::2]),
        (DIMS, 2, torch.zeros((2, 0), dtype=torch.int32)), (TYPE, 2, torch.zeros((2, 3), dtype=torch.int64)),
        (DIMS, 3, torch.zeros(2, dtype=torch.int32)), (TYPE, 3, torch.zeros(3, dtype=torch.int64)),
        (DIMS, 4, torch.zeros(4, dtype=torch.int32)[::2]), (TYPE, 4, torch.zeros(2)),
    ]:
        a = tensors()
        a[i] = x
        raises(rc, q8.PagedKV, *a)
    both = torch.zeros((4, 2, 2, 16, 64), dtype=torch.float16)
    assert q8.PagedKV(both[:, 0], both[:, 1], *tensors()[2:]).c.page_stride == 2 * 2 * 16 * 64


def test_helper_append(here):
    kv = q8.PagedKV(*tensors())
    q, k = torch.zeros((3, 4, 64)), torch.zeros((3, 2, 64))
    turns = torch.zeros(32, dtype=torch.int64)
    f = q8.append_kv
    raises(DIMS, f, kv, q, torch.zeros((3, 3, 64)), k, turns)
    raises(DIMS, f, kv, q, torch.zeros((3, 64, 2)).transpose(1, 2), k, turns)
    raises(DIMS, f, kv, q, k, torch.zeros((2, 2, 64)), turns)
    raises(TYPE, f, kv, q, k, k.half(), turns)
    raises(TYPE, f, kv, q.half(), k, k, turns)
    raises(TYPE, f, kv, q.double(), k.double(), k.double(), turns)
    raises(DIMS, f, kv, q[:2], k, k, turns)
    raises(DIMS, f, kv, q[0], k, k, turns)
    raises(DIMS, f, kv, q[..., ::2], k, k, turns)
    raises(TYPE, f, kv, q, k, k, turns, out=torch.zeros((3, 4, 64)))
    raises(DIMS, f, kv, q, k, k, turns, out=torch.zeros((3, 5, 64), dtype=torch.float16))
    raises(TYPE, f, kv, q, k, k, turns.double())
    raises(NULL, f, kv, None, k, k, turns, out=torch.zeros((3, 4, 64), dtype=torch.float16))
    raises(DIMS, q8.rope_turns, [float("inf")])


def test_helper_attention(here):
    kv = q8.PagedKV(*tensors())
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    ws = torch.zeros(1 << 26, dtype=torch.uint8)
    f = q8.attention
    raises(TYPE, f, kv, q.float(), ws=ws)
    raises(DIMS, f, kv, q[0], ws=ws)
    raises(DIMS, f, kv, q[..., :32], ws=ws)
    raises(DIMS, f, kv, q.transpose(0, 1), ws=ws)
    raises(DIMS, f, kv, q[:0], ws=ws)
    raises(WS, f, kv, q, ws=ws.view(torch.int32))
    raises(WS, f, kv, q, ws=ws[::2])
    raises(DIMS, f, kv, q, ws=ws, out=torch.zeros((3, 4, 32), dtype=torch.float16))
    raises(TYPE, f, kv, q, ws=ws, dtype=torch.float64)
    raises(DIMS, f, kv, q, ws=ws, window=-1)
    raises(DIMS, f, kv, q, ws=ws, max_new=2 ** 31)


def test_helpers_of_another_device(here, monkeypatch):
    kv, q = q8.PagedKV(*tensors()), torch.zeros((3, 4, 64), dtype=torch.float16)
    monkeypatch.setattr(q8, "_current", lambda: 1)
    raises(q8.Q8ACT_ERR_DEVICE, q8.attention, kv, q)
    raises(q8.Q8ACT_ERR_DEVICE, q8.append_kv, kv, q, q[:, :2], q[:, :2])
    raises(q8.Q8ACT_ERR_DEVICE, q8.PagedKV, *tensors())
