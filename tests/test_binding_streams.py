"""A call given ``stream=`` takes every buffer that it makes itself (outputs,
workspaces and their zero fill, gathered scales) on that stream: made on the
current one, nothing would order the fill, or what still runs on a recycled
block, before the kernels. Returned tensors are recorded as used on the
caller's stream. Runs without a GPU: the library, the allocator and the streams
are stand-ins that note what happens where."""
import contextlib

import pytest
import torch

from nvfp4_w4a4_quantized_elem_b200 import nvfp4 as nv

CUDA = torch.device("cuda", 0)


class Fake(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    device = property(lambda self: CUDA)
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        Fake.recorded.append((self.data_ptr(), stream))


class Stream:
    def __init__(self, name, handle):
        self.name, self.cuda_stream = name, handle


@pytest.fixture
def world(monkeypatch):
    """(events, run): (what, stream name) of every allocation, fill, copy and
    launch in order, and the side stream."""
    events, here = [], [Stream("current", 0)]
    Fake.recorded = []

    @contextlib.contextmanager
    def on(stream):
        here.append(stream)
        yield
        here.pop()

    def made(name, real):
        def call(*args, **kw):
            kw.pop("device", None)
            events.append((name, here[-1].name))
            return real(*args, **kw).as_subclass(Fake)
        return call

    for name in ("empty", "zeros", "cat"):
        monkeypatch.setattr(torch, name, made(name, getattr(torch, name)))
    real_copy = torch.Tensor.copy_
    monkeypatch.setattr(Fake, "copy_", lambda self, *a: (events.append(("copy", here[-1].name)),
                                                         real_copy(self, *a))[1], raising=False)

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 4096
                stream = args[-1]
                events.append((name, {0: "current", 7: "side"}[stream]))
                return 0
            return call

    monkeypatch.setattr(nv, "_lib", Lib())
    monkeypatch.setattr(nv, "lib", lambda: nv._lib)
    monkeypatch.setattr(nv, "_stream", lambda s: here[-1].cuda_stream if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return events, Stream("side", 7)


def fake(*shape, dtype=torch.bfloat16):
    return torch.ones(shape, dtype=dtype).as_subclass(Fake)


def nvfp4_tensor(rows, k):
    return nv.NVFP4Tensor(fake(rows, k // 2, dtype=torch.uint8), fake(4096, dtype=torch.uint8),
                          fake(1, dtype=torch.float32), rows, k)


def attention(n):
    return (fake(n, 1, 64), fake(n, 1, 64), fake(n, 2, 32), fake(n, 2, dtype=torch.float32),
            fake(n, 2, dtype=torch.float32))


CALLS = {
    "quantize": lambda s: nv.quantize(fake(4, 64), stream=s),
    "gemm": lambda s: nv.gemm(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), stream=s),
    "gemm epilogue": lambda s: nv.gemm(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), bias=fake(64), stream=s),
    "linear": lambda s: nv.linear(fake(4, 64), nvfp4_tensor(64, 64), stream=s),
    "linear epilogue": lambda s: nv.linear(fake(4, 64), nvfp4_tensor(64, 64), activation="silu", stream=s),
    "swiglu": lambda s: nv.gemm_swiglu_quant(nvfp4_tensor(4, 64), nvfp4_tensor(256, 64),
                                             fake(1, dtype=torch.float32), stream=s),
    "swiglu dynamic": lambda s: nv.gemm_swiglu_quant_dynamic(nvfp4_tensor(4, 64), nvfp4_tensor(256, 64), stream=s),
    "fuse_group": lambda s: nv.fuse_group([nvfp4_tensor(4, 64), nvfp4_tensor(4, 64)], stream=s),
    "silu_mul": lambda s: nv.silu_mul(fake(4, 64), stream=s),
    "calibrate": lambda s: nv.Calibrator.observe(calibrator(), fake(4, 64), stream=s),
    "linear_attention": lambda s: nv.linear_attention(*attention(5), stream=s),
    "linear_attention_step": lambda s: nv.linear_attention_step(*attention(2), state=fake(2, 2, 64, 32, dtype=torch.float32), stream=s),
    "selftest_gemm_stall": lambda s: nv.selftest_gemm_stall(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), stream=s),
}


def calibrator():
    c = nv.Calibrator.__new__(nv.Calibrator)
    c.running_amax = c.global_scale = fake(1, dtype=torch.float32)
    c._ws = c._ws_stream = None
    return c


def tensors(x):
    if isinstance(x, nv.NVFP4Tensor):
        return [x.codes, x.sf, x.global_scale]
    return [] if x is None else [x]


@pytest.mark.parametrize("name", CALLS)
def test_buffers_are_made_where_the_kernels_run(world, name):
    events, side = world
    given = CALLS[name](side)
    assert any(what.startswith("nvfp4_") for what, _ in events)
    assert {where for _, where in events} == {"side"}, events
    if name != "calibrate":   # what a caller keeps over calls is the caller's own
        recorded = {p for p, s in Fake.recorded if s.name == "current"}
        assert {t.data_ptr() for t in tensors(given)} <= recorded


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_taken(world, name):
    events, _ = world
    CALLS[name](None)
    assert {where for _, where in events} == {"current"}, events
    assert not Fake.recorded
