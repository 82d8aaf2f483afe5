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


@KERNELS
@pytest.mark.parametrize("n", [40, 700, 6000])
@pytest.mark.parametrize("t,size", [("f16", 2.0 ** 8), ("f16", 1800.0), ("f16", 2.0 ** 13 + 8), ("f16", 65504.0),
                                    ("bf16", 1e4), ("bf16", 1e8), ("bf16", 1e17)])
def test_large_equal_scores(t, size, n, max_new):
    """Finite scores whose products with the scale lie between numbers of f32 that are far apart: equal ones weigh the same,
    those that are far below nothing."""
    t = ref.TYPES[t]
    g = torch.Generator().manual_seed(n)
    v = torch.randn((n, D), generator=g).to(t)
    high = torch.rand(n, generator=g) < 0.4
    high[n // 3] = True
    k = torch.where(high[:, None], size, -size).expand(n, D).to(t).contiguous()
    q = torch.full((NEW, HQ, D), size).to(t)
    q[:, 1] = -q[:, 1]                                                           # the others win
    q[:, 2] *= 0.5
    q[:, 3] = 0
    for scale in (0.125, 0.1, 0.3):
        got = q8.attention(one_sequence(k, v), q.cuda(), scale=scale, max_new=max_new, dtype=torch.float32).cpu()
        device_ok()
        for h, mine in ((0, high), (1, ~high), (2, high), (3, torch.ones_like(high))):
            x = torch.where(mine[:, None], v.double(), 0.0)
            count = mine.double().cumsum(0)[n - NEW:, None]
            mean = lambda y: y.cumsum(0)[n - NEW:] / count                        # noqa: B023, E731
            # equal weights below 1, each rounded to the type once (in f16 at 2^-32 of the largest, at the least)
            tol = mean(x.abs()) * (ref.half(t) + (2 * n + 16) * 2.0 ** -23)
            ref.close(got[:, h], mean(x), tol, f"head {h}, scale {scale}")


@KERNELS
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("steps", [1, 4])
@pytest.mark.parametrize("e", [20, 24, 25, 26, 27, 28, 30])
def test_large_rising_scores(e, steps, t, max_new):
    """Scores of 2^e (to the base of 2) that rise by so many steps of f32 every 128 positions: the last ones have the weight.
    A scaled score is known to half a step, so one below them may weigh 2^step times as much."""
    t, n = ref.TYPES[t], 900
    step = 2.0 ** (e - 23)
    k = torch.zeros((n, D))
    k[:, 0], k[:, 1] = 2.0 ** (e - 15), (torch.arange(n) // 128).float() * steps
    v = torch.randn((n, D), generator=torch.Generator().manual_seed(e)).to(t)
    q = torch.zeros((NEW, HQ, D))
    q[:, :, 0], q[:, :, 1] = 2.0 ** 15, step
    q[:, 1, 1] = 0                                                               # all the same
    got = q8.attention(one_sequence(k.to(t), v), q.to(t).cuda(), scale=math.log(2.0), max_new=max_new, dtype=torch.float32).cpu()
    device_ok()
    for i in range(NEW):
        seen = n - NEW + 1 + i
        x = v[:seen].double()
        for h in range(HQ):
            s = k[:seen, 1].double() * (0.0 if h == 1 else step)
            w = 2.0 ** (s - s.max())
            below = torch.where(s < s.max(), w, torch.zeros_like(w)).sum() * (2.0 ** step if step > 2.0 ** -3 else 4 * step)
            w = w / w.sum()
            a = (w[:, None] * x.abs()).sum(0)
            tol = a * (ref.half(t) + (2 * seen + 16) * 2.0 ** -23) + below / w.sum() * (x.abs().amax(0) + a)
            ref.close(got[i, h], (w[:, None] * x).sum(0), tol, f"token {i}, head {h}")


@KERNELS
@pytest.mark.parametrize("n", [40, 6000, 131071])
@pytest.mark.parametrize("t,size", [("bf16", torch.finfo(torch.bfloat16).max), ("bf16", 2.0 ** 120), ("bf16", 2.0 ** -100),
                                    ("f16", 65504.0), ("f16", 2.0 ** -24)])
def test_values_of_any_size(t, size, n, max_new):
    """An average is as large as its values, however many of the largest there are, and however small they are."""
    t = ref.TYPES[t]
    g = torch.Generator().manual_seed(n)
    k, v = torch.randn((n, D), generator=g).to(t), torch.full((n, D), size)
    v[:, 1::2] *= torch.where(torch.rand((n, D // 2), generator=g) < 0.25, -1.0, 1.0)
    v = v.to(t)
    q = torch.randn((NEW, HQ, D), generator=g).to(t)
    q[:, 0] = 0                                                                  # equal weights
    got = q8.attention(one_sequence(k, v), q.cuda(), max_new=max_new, dtype=torch.float32).cpu()
    device_ok()
    U, unit = 2.0 ** -23, v.double() / size
    for i in range(NEW):
        seen = n - NEW + 1 + i
        s = (q[i].double() @ k[:seen].double().T) * D ** -0.5
        w = torch.softmax(s, -1)
        want = w @ unit[:seen]
        ds = (D + 4) * U * (q[i].double().abs() @ k[:seen].double().abs().T).amax(-1, keepdim=True) * D ** -0.5
        tol = ref.half(t) + 2 * ds + (2 * seen + 16) * U                         # (every |unit| is 1)
        # where products with weights are below f32's normal numbers: each to 2^-149, of weights relative to 2^-28
        tol = tol + seen * 2.0 ** -149 / (2.0 ** -28 * size)
        if t is torch.float16:
            tol = tol + seen * 2.0 ** -32
        ref.close(got[i].double() / size, want, tol.expand_as(want), f"token {i}")
