"""append_kv of two sequences to the same place: each 16 bytes of it are what one of the two alone would have left."""
import pytest
import torch

import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_same_place_twice(n, interleaved):
    ensure_built()
    hk, d, page = 2, 128, 64
    pages = -(-n // page)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.randn((2 * n, 2 * hk, d), generator=torch.Generator("cuda").manual_seed(n), device="cuda")
    turns = q8.rope_turns([10000.0 ** (-2 * i / d) for i in range(d // 2)], "cuda")

    def appended(rows, seqs):
        k, v = (torch.full((pages, hk, page, d), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        kv = q8.PagedKV(k, v, torch.arange(pages, **i32).expand(seqs, -1).contiguous(), n * torch.arange(seqs + 1, **i32),
                        torch.full((seqs,), n, **i32))
        q8.append_kv(kv, None, rows[:, :hk], rows[:, hk:], turns=turns, interleaved=interleaved)
        device_ok()
        return [c.view(torch.int16).view(-1, 8) for c in (k, v)]

    both, first, second = appended(x, 2), appended(x[:n], 1), appended(x[n:], 1)
    for got, a, b in zip(both, first, second):
        assert bool(((got == a).all(1) | (got == b).all(1)).all())
