"""The torch helpers of the norm, MXFP4 and log-probability calls refuse a tensor that is not on the
current CUDA device, whichever argument it is, before anything is launched.  Stand-ins report the
devices and the C ABI is a recorder, so this needs no GPU and launches nothing."""
import pytest
import torch

import q8_block_quantized_act_gb300 as q8

M, K, N, V, TOP = 4, 512, 96, 50, 3
F32, I8, U8, U16, I32 = torch.float32, torch.int8, torch.uint8, torch.uint16, torch.int32


class Stand:
    """A contiguous tensor on cuda:index, as far as the helpers look at one."""

    def __init__(self, index, dtype, *shape):
        self.index, self.dtype, self.shape = index, dtype, torch.Size(shape)
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def stride(self, i):
        return self.shape[1] if i == 0 else 1

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()


def scales(rows):
    return (rows + 127) // 128 * (K // 128) * 512


CALLS = {
    "rmsnorm_q8_1": (dict(x=(F32, M, K), weight=(F32, K), residual=(F32, M, K), residual_out=(F32, M, K), y=(F32, M, K),
                          q=(I8, M, K), d=(F32, M, K // 32)),
                     lambda t: q8.rmsnorm_q8_1(t["x"], t["weight"], residual=t["residual"],
                                               residual_out=t["residual_out"], y=t["y"], out=(t["q"], t["d"]))),
    "rmsnorm_q8_1_mmq": (dict(x=(F32, M, K), q=(U16, M, K), d=(F32, K // 32, M)),
                         lambda t: q8.rmsnorm_q8_1_mmq(t["x"], out=(t["q"], t["d"]))),
    "rmsnorm": (dict(x=(F32, M, K), out=(F32, M, K)), lambda t: q8.rmsnorm(t["x"], out=t["out"])),
    "quantize_mxfp4": (dict(x=(F32, M, K), codes=(U8, M, K // 2), scales=(U8, scales(M))),
                       lambda t: q8.quantize_mxfp4(t["x"], out=(t["codes"], t["scales"]))),
    "dequant_mxfp4": (dict(codes=(U8, M, K // 2), scales=(U8, scales(M)), out=(F32, M, K)),
                      lambda t: q8.dequant_mxfp4(t["codes"], t["scales"], out=t["out"])),
    "gemm_mxfp4": (dict(w=(U8, N, K // 2), wscales=(U8, scales(N)), x=(F32, M, K), ws=(U8, 1 << 20), out=(F32, M, N)),
                   lambda t: q8.gemm_mxfp4(t["w"], t["wscales"], t["x"], ws=t["ws"], out=t["out"])),
    "gemm_mxfp4_preq": (dict(w=(U8, N, K // 2), wscales=(U8, scales(N)), xq=(U8, M, K // 2), xscales=(U8, scales(M)),
                             out=(F32, M, N)),
                        lambda t: q8.gemm_mxfp4_preq(t["w"], t["wscales"], t["xq"], t["xscales"], out=t["out"])),
    "logprobs": (dict(logits=(F32, M, V), tokens=(I32, M), lp=(F32, M), ent=(F32, M), ids=(I32, M, TOP), tlp=(F32, M, TOP)),
                 lambda t: q8.logprobs(t["logits"], t["tokens"], top=TOP, out=(t["lp"], t["ent"], t["ids"], t["tlp"]))),
}


@pytest.fixture
def launches(monkeypatch):
    """Calls that reach the C ABI; the current device is 0."""
    seen = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: seen.append(name) or 0

    q8._load_torch()
    monkeypatch.setattr(q8, "_current", lambda: 0, raising=False)
    monkeypatch.setattr(q8, "_stream", lambda device: 0, raising=False)
    monkeypatch.setattr(q8, "lib", Recorder)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_is_on_the_current_device(launches, name):
    spec, call = CALLS[name]
    make = lambda elsewhere: {a: Stand(int(a in elsewhere), *s) for a, s in spec.items()}   # noqa: E731
    call(make(()))
    assert len(launches) == 1                              # what is in order goes through
    for elsewhere in [(a,) for a in spec] + [tuple(spec)]:
        with pytest.raises(q8.Q8ActError) as e:
            call(make(elsewhere))
        assert e.value.rc == q8.Q8ACT_ERR_DEVICE, elsewhere
    assert len(launches) == 1


def test_tiling_of_scales_is_on_the_current_device(launches):
    with pytest.raises(q8.Q8ActError) as e:
        q8.tile_mxfp4_scales(Stand(1, U8, M, K // 32))
    assert e.value.rc == q8.Q8ACT_ERR_DEVICE and not launches
