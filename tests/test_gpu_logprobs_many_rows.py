"""More rows of logits than the grid has CTAs: each CTA goes over several rows, whose results must not
depend on the row before.  Compared with the same calls on parts of the rows, and a sample with 64 bits."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built
from test_gpu_logprobs import check

pytestmark = pytest.mark.gpu
GRID = 1 << 24


def test_logprobs_of_more_rows_than_ctas():
    ensure_built()
    m, v, top = GRID + 40000, 13, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((m, v), generator=g, device="cuda").half()
    x[torch.rand((m, v), generator=g, device="cuda") < 0.3] = float("-inf")
    x[::7] = float("-inf")                                     # whole rows, among both of a CTA's
    x[GRID + 3::1000, 5] = float("nan")
    tokens = torch.randint(-1, v, (m,), generator=g, device="cuda", dtype=torch.int32)
    got = q8.logprobs(x, tokens, top=top)
    half = m // 2 // 8 * 8                                     # the second part starts 16-byte aligned, as the whole
    parts = [q8.logprobs(x[a:b], tokens[a:b].clone(), top=top) for a, b in ((0, half), (half, m))]
    device_ok()
    for i, t in enumerate(got):
        assert torch.equal(t.view(torch.int32), torch.cat([p[i] for p in parts]).view(torch.int32)), i
    at = torch.from_numpy(np.r_[0:50, GRID - 50:GRID + 50, m - 100:m])
    check(tuple(t[at.cuda()] for t in got), x[at.cuda()].cpu(), tokens[at.cuda()].cpu(), top)
