"""attention of thousands of short sequences, call after call: a CTA takes dozens of row tiles one after another, while the
joining kernel's CTAs begin beside it."""
import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,most,hk,group,d", [(10000, 16, 1, 2, 64), (3000, 70, 2, 4, 128), (20000, 33, 1, 1, 64), (40000, 16, 1, 3, 64)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("max_new", [1, 1000], ids=["rows", "chunks"])
def test_every_row_each_time(n, most, hk, group, d, t, max_new):
    ensure_built()
    t, page, hq = ref.TYPES[t], 16, hk * group
    g = torch.Generator("cuda").manual_seed(n)
    width = -(-most // page)
    lens = torch.randint(1, most + 1, (n,), device="cuda", dtype=torch.int32, generator=g)
    k, v = (torch.randn((n * width, hk, page, d), device="cuda", generator=g).to(t) for _ in range(2))
    table = torch.randperm(n * width, device="cuda", generator=g).to(torch.int32).view(n, width)
    kv = q8.PagedKV(k, v, table, torch.arange(n + 1, device="cuda", dtype=torch.int32), lens)
    q = torch.randn((n, hq, d), device="cuda", generator=g).to(t)
    want, tol = torch.empty((n, hq, d), dtype=torch.float64, device="cuda"), torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
    U = 2.0 ** -23
    for a in range(0, n, 2500):
        e = min(n, a + 2500)
        kk, vv = (c[table[a:e].long()].transpose(1, 2).reshape(e - a, hk, width * page, d).double() for c in (k, v))
        x = q[a:e].view(e - a, hk, group, d).double()
        hidden = (torch.arange(width * page, device="cuda")[None] >= lens[a:e, None])[:, None, None]
        w = (x @ kk.transpose(-1, -2) * d ** -0.5).masked_fill(hidden, float("-inf")).softmax(-1)
        ds = (d + 4) * U * (x.abs() @ kk.abs().transpose(-1, -2)).amax(-1, keepdim=True) * d ** -0.5
        want[a:e] = (w @ vv).view(e - a, hq, d)
        # the weights' rounding (f16 also by 2^-32 of the largest), the scores', sums
        tol[a:e] = (w @ vv.abs() * (ref.half(t) + 2 * ds + (2 * most + 16) * U) + most * 2.0 ** -32 * 8).view(e - a, hq, d)
    ws, out = q8.attention_workspace(kv, hq), torch.empty((n, hq, d), device="cuda")
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(40):
        out.fill_(7.0)
        q8.attention(kv, q, max_new=max_new, ws=ws, out=out)
        bad += (~((out - want).abs() <= tol)).any(-1).sum()
    device_ok()
    assert int(bad) == 0, f"{int(bad)} of {40 * n * hq} rows"
