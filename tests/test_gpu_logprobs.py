"""Log probabilities, entropy and alternatives vs their 64-bit form.

Tolerances.  S is a sum of at most v non-negative terms in which no term passes through more than
depth = v / 512 + 32 additions; an exponential is good to 4 * 2^-24 + |z| 2^-24 relative and
z e^z <= 1/e, so S is within rel = (depth + 8) * 2^-24 of its value, log S within rel absolute, and
x - max within 2^-24 |x - max| (it enters twice).  T's terms are of one sign, so T / S is within
2 rel + 2^-22 of its own size, which is at most H + log v.  Ids are exact."""
import numpy as np
import pytest
import torch

import ops_ref as ref
import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built, host

pytestmark = pytest.mark.gpu


def make(m, v, kind, seed=0, masked=0.0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, v), generator=g) * spread
    x[torch.arange(m), torch.randint(0, v, (m,), generator=g)] += 8
    if masked:
        x[torch.rand((m, v), generator=g) < masked] = float("-inf")
    tokens = torch.randint(0, v, (m,), generator=g, dtype=torch.int32)
    return x.to(ref.TYPES[kind]), tokens


def check(got, x, tokens, top):
    lp, ent, ids, tlp = (None if t is None else host(t) for t in got)
    v = x.shape[1]
    rlp, rent, rids, rtlp = ref.logprobs(ref.f64(x), None if tokens is None else tokens.numpy(), top)
    rel = (v / 512 + 40) * ref.U

    def near(a, b, tol, what):
        fine = np.isfinite(b)
        assert np.array_equal(fine, np.isfinite(a)) and np.array_equal(a[~fine], b[~fine], equal_nan=True), what
        assert np.all(np.abs(a - b)[fine] <= np.broadcast_to(tol, b.shape)[fine]), what

    if tokens is not None:
        near(lp.astype(np.float64), rlp, rel + 2.0 ** -22 * (1 + np.abs(rlp)), "logprob")
    near(ent.astype(np.float64), rent, (2 * rel + 2.0 ** -22) * (2 + np.abs(rent) + np.log(v)), "entropy")
    if top:
        assert np.array_equal(ids, rids)
        near(tlp.astype(np.float64), rtlp, rel + 2.0 ** -22 * (1 + np.abs(rtlp)), "top")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,v,top", [(1, 1, 1), (1, 64448, 20), (2, 31, 32), (3, 257, 5), (7, 4097, 8), (1, 128896, 1),
                                     (40, 5000, 32), (200, 1003, 20), (5, 50257, 32), (1, 300001, 8), (330, 2049, 3),
                                     (9, 64448, 0)])
def test_logprobs_match_64_bits(m, v, top, kind):
    ensure_built()
    x, tokens = make(m, v, kind, seed=v)
    got = q8.logprobs(x.cuda(), tokens.cuda(), top=top)
    device_ok()
    check(got, x, tokens, top)


def test_logprobs_long_rows_one_cta_each():
    """Rows long enough that a kept maximum stands for several steps, too many rows to share."""
    ensure_built()
    m, v = 320, 70001
    x, tokens = make(m, v, "f32", seed=8)
    x[7] = 0.5                                                # a row of equal logits: more keys than the list
    x[11, 5::2048] = 30.0                                     # one thread's places
    got = q8.logprobs(x.cuda(), tokens.cuda(), top=16)
    device_ok()
    check(got, x, tokens, 16)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("m,v", [(1, 64448), (33, 9001), (160, 1500)])
def test_logprobs_masks(m, v, kind):
    """Masked logits, rows with fewer unmasked tokens than alternatives, rows masked as a whole."""
    ensure_built()
    x, tokens = make(m, v, kind, seed=5, masked=0.5)
    if m > 1:
        x[1] = float("-inf")
        x[2] = float("-inf")
        x[2, [v - 1, 3]] = 1.5
        x[3] = float("-inf")
        x[3, tokens[3]] = -7.0
        x[4] = torch.finfo(x.dtype).min                       # the lowest value is no mask
        x[5] = torch.finfo(x.dtype).min
        x[5, 17] = 0.0
        tokens[6], tokens[7], tokens[8] = -1, v, 2 ** 31 - 1
        tokens[9] = -2 ** 31
    got = q8.logprobs(x.cuda(), tokens.cuda(), top=20)
    device_ok()
    check(got, x, tokens, 20)
    whole = torch.full_like(x[:1], float("-inf"))
    got = q8.logprobs(whole.cuda(), tokens[:1].cuda(), top=4)
    device_ok()
    check(got, whole, tokens[:1], 4)


@pytest.mark.parametrize("m", [1, 2, 170])
@pytest.mark.parametrize("pattern", ["equal", "rising", "falling", "few", "signed zeros"])
def test_logprobs_ties_and_orders(m, pattern):
    """Equal logits come by the lower index, whatever order the row has them in."""
    ensure_built()
    v = 20011
    i = torch.arange(v, dtype=torch.float32)
    row = {"equal": torch.full((v,), -3.25), "rising": i / 1000, "falling": -i / 1000, "few": (i * 7919 % 5),
           "signed zeros": torch.where(i % 3 == 0, torch.tensor(-0.0), torch.tensor(0.0))}[pattern]
    x = torch.stack([torch.roll(row, 13 * r) for r in range(m)])
    tokens = torch.zeros(m, dtype=torch.int32)
    for t in (torch.float32, torch.bfloat16):
        got = q8.logprobs(x.to(t).cuda(), tokens.cuda(), top=32)
        device_ok()
        check(got, x.to(t), tokens, 32)


def test_logprobs_nonfinite_rows():
    ensure_built()
    x, tokens = make(40, 3000, "f32", seed=2)
    x[1, 2999], x[2, 0], x[3, 1500] = float("nan"), float("inf"), float("-inf")
    x[4] = float("nan")
    x[5] = float("-inf")
    x[5, 7] = float("nan")
    got = q8.logprobs(x.cuda(), tokens.cuda(), top=3)
    device_ok()
    check(got, x, tokens, 3)
    for r in (1, 2):                                          # the same rows one at a time
        got = q8.logprobs(x[r:r + 1].cuda(), tokens[r:r + 1].cuda(), top=3)
        device_ok()
        check(got, x[r:r + 1], tokens[r:r + 1], 3)


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_logprobs_any_row_start(kind):
    """Rows of a wider buffer, starting at every alignment, and nothing read beyond them."""
    ensure_built()
    m, v = 6, 777
    x, tokens = make(m, v, kind, seed=3)
    for lead in range(9):
        wide = torch.full((m, v + 17), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, lead:lead + v] = x.cuda()
        got = q8.logprobs(wide[:, lead:lead + v], tokens.cuda(), top=6)
        device_ok()
        check(got, x, tokens, 6)


def test_logprobs_optional_outputs_and_bounds():
    ensure_built()
    m, v, top = 5, 2000, 4
    x, tokens = make(m, v, "f32")
    lp, ent, ids, tlp = q8.logprobs(x.cuda(), top=0)
    device_ok()
    assert lp is None and ids.shape == (m, 0)
    check((None, ent, ids, tlp), x, None, 0)
    dev = torch.device("cuda")
    bufs = [torch.full((m + 2,), 9.0, device=dev), torch.full((m + 2,), 9.0, device=dev),
            torch.full((m + 2, top), 9, dtype=torch.int32, device=dev), torch.full((m + 2, top), 9.0, device=dev)]
    got = q8.logprobs(x.cuda(), tokens.cuda(), top=top, out=tuple(b[1:m + 1] for b in bufs))
    device_ok()
    check(got, x, tokens, top)
    for b in bufs:
        assert bool((b[0] == 9).all()) and bool((b[m + 1] == 9).all())


def test_logprobs_extreme_logits():
    """Far-apart, huge and tiny logits: nothing overflows, small probabilities keep their log."""
    ensure_built()
    x = torch.zeros((4, 5000))
    x[0] = -3e38
    x[0, 10] = 3e38
    x[1] = torch.linspace(-1e4, 1e4, 5000)
    x[2] = torch.linspace(-80, 0, 5000)
    x[3] = 1e-30
    tokens = torch.tensor([3, 0, 0, 4999], dtype=torch.int32)
    lp, ent, ids, tlp = q8.logprobs(x.cuda(), tokens.cuda(), top=5)
    device_ok()
    assert float(lp[0]) == -float("inf") or float(lp[0]) < -3e38     # beyond f32's range
    assert float(ent[0]) == 0.0 and float(tlp[0, 0]) == 0.0
    check(tuple(t[1:] for t in (lp, ent, ids, tlp)), x[1:], tokens[1:], 5)
