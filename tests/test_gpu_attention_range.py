"""The range of attention's scores and weights: weights far below the largest one, scores beyond f32's range."""
import math

import pytest
import torch

import paged_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built

pytestmark = pytest.mark.gpu

D, HQ, NEW, PAGE = 64, 4, 5, 16
# Of a batch of NEW tokens and HQ query heads to one of keys: the kernel for few rows, the one for chunks.
KERNELS = pytest.mark.parametrize("max_new", [1, NEW], ids=["rows", "chunks"])


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def one_sequence(k, v, seed=0):
    """k, v [positions, D] as a cache of one head, its pages shuffled; the last NEW positions are new tokens."""
    n = k.shape[0]
    pages = -(-n // PAGE)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    caches = []
    for x in (k, v):
        c = torch.zeros((pages * PAGE, D), dtype=x.dtype)
        c[:n] = x
        at = torch.empty((pages, 1, PAGE, D), dtype=x.dtype)
        at[order] = c.view(pages, 1, PAGE, D)
        caches.append(at.cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    return q8.PagedKV(*caches, order.to(torch.int32).view(1, -1).cuda(), torch.tensor([0, NEW], **i32), torch.tensor([n], **i32))


@KERNELS
@pytest.mark.parametrize("n", [700, 6000, 131071])
@pytest.mark.parametrize("t,bits", [("f16", 26), ("f16", 29), ("bf16", 29)])
def test_many_small_weights(t, bits, n, max_new):
    """Every 16th position has values of 0 and all but a little of the weight; the others weigh 2^-bits of it each and make the
    output.  Weights are held to half a step of the type, in f16 also to 2^-32 of the largest."""
    t = ref.TYPES[t]
    g = torch.Generator().manual_seed(n)
    k, v = torch.zeros((n, D), dtype=t), (1 + 0.25 * torch.randn((n, D), generator=g)).to(t)
    k[::16, 0] = bits
    v[::16] = 0
    q = torch.zeros((NEW, HQ, D), dtype=t)
    q[:, :, 0] = 1
    scale = math.log(2.0)
    got = q8.attention(one_sequence(k, v), q.cuda(), scale=scale, max_new=max_new, dtype=torch.float32)
    device_ok()
    U = 2.0 ** -23
    seen = torch.arange(n - NEW, n)[:, None] + 1.0                               # positions of each token
    large = torch.ceil(seen / 16)
    sums, size = (x.double().cumsum(0)[n - NEW:] for x in (v, v.abs()))
    w = 2.0 ** -bits
    total = large + (seen - large) * w
    want, a = w * sums / total, w * size / total
    rel = ref.half(t) + 2 * (D + 4) * U * scale * bits + (2 * seen + 16) * U
    floor = 2.0 ** -32 if t is torch.float16 else ref.tiny(t)
    tol = a * rel + floor * size / total + ref.half(torch.float32) * want.abs()
    assert bool((tol < 0.25 * want).all())
    ref.close(got, want[:, None].expand(-1, HQ, -1), tol[:, None].expand(-1, HQ, -1))


@KERNELS
@pytest.mark.parametrize("n", [40, 700, 6000])
@pytest.mark.parametrize("t,big,scale", [("bf16", 2.0 ** 50, 2.0 ** 30), ("f16", 2.0 ** 15, 2.0 ** 99)])
def test_scores_beyond_f32(t, big, scale, n, max_new):
    """A finite product whose scaled score is beyond f32: NaN where it is positive, nothing where it is negative."""
    t = ref.TYPES[t]
    k, v = torch.zeros((n, D), dtype=t), torch.randn((n, D), generator=torch.Generator().manual_seed(n)).to(t)
    k[n // 2, 0] = big
    q = torch.zeros((NEW, HQ, D), dtype=t)
    q[:, 1, 0], q[:, 2, 0] = big, -big
    got = q8.attention(one_sequence(k, v), q.cuda(), scale=scale, max_new=max_new, dtype=torch.float32).cpu()
    device_ok()
    assert bool(torch.isnan(got[:, 1]).all())
    for h, left_out in ((0, False), (2, True), (3, False)):
        x = v.double()
        if left_out:
            x[n // 2] = 0
        seen = torch.arange(n - NEW, n)[:, None] + 1.0
        mean = lambda y: y.cumsum(0)[n - NEW:] / (seen - int(left_out))           # noqa: E731
        ref.close(got[:, h], mean(x), mean(x.abs()) * (2 * seen + 16) * 2.0 ** -23, f"head {h}")
