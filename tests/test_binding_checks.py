"""What the binding hands to the library as bare pointers is checked first: a
workspace, a global scale or a part of an NVFP4 tensor that lies elsewhere, or
is not laid out as the call says, is refused on the host. Without a GPU, on
stand-ins (test_binding_streams)."""
import pytest
import torch

from nvfp4_w4a4_quantized_elem_b200 import nvfp4 as nv
from test_binding_streams import attention, fake, nvfp4_tensor, world  # noqa: F401


def calls(**kw):
    """The calls that take these arguments, by name."""
    f32 = lambda: fake(1, dtype=torch.float32)  # noqa: E731
    every = {
        "quantize": lambda: nv.quantize(fake(4, 64), **kw),
        "gemm": lambda: nv.gemm(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), **kw),
        "gemm epilogue": lambda: nv.gemm(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), bias=fake(64), **kw),
        "linear": lambda: nv.linear(fake(4, 64), nvfp4_tensor(64, 64), **kw),
        "linear epilogue": lambda: nv.linear(fake(4, 64), nvfp4_tensor(64, 64), bias=fake(64), **kw),
        "swiglu dynamic": lambda: nv.gemm_swiglu_quant_dynamic(nvfp4_tensor(4, 64), nvfp4_tensor(256, 64), **kw),
        "linear_attention": lambda: nv.linear_attention(*attention(5), **kw),
        "swiglu": lambda: nv.gemm_swiglu_quant(nvfp4_tensor(4, 64), nvfp4_tensor(256, 64),
                                               kw.get("global_scale", f32())),
        "noalloc": lambda: nv.quantize_noalloc(fake(4, 64), nvfp4_tensor(4, 64), **kw),
    }
    takes = {"workspace": ("quantize", "gemm", "gemm epilogue", "linear", "linear epilogue",
                           "swiglu dynamic", "linear_attention"),
             "global_scale": ("quantize", "linear", "linear epilogue", "swiglu", "noalloc")}
    return {name: every[name] for name in takes[next(iter(kw))]}


def launched(events):
    return [what for what, _ in events if what.startswith("nvfp4_")]


WORKSPACES = {"on the host": lambda: torch.ones(8192, dtype=torch.uint8),
              "with gaps": lambda: fake(16384, dtype=torch.uint8)[::2]}


@pytest.mark.parametrize("what", WORKSPACES)
@pytest.mark.parametrize("name", calls(workspace=None))
def test_a_bad_workspace_is_refused(world, name, what):
    with pytest.raises(ValueError):
        calls(workspace=WORKSPACES[what]())[name]()
    assert not launched(world[0])


@pytest.mark.parametrize("name", calls(workspace=None))
def test_a_good_workspace_passes(world, name):
    calls(workspace=fake(8192, dtype=torch.uint8))[name]()
    calls(workspace=fake(4096, dtype=torch.bfloat16))[name]()   # any type: bytes count
    assert len(launched(world[0])) == 2


GLOBALS = {"on the host": lambda: torch.ones(1), "bf16": lambda: fake(1),
           "fp64": lambda: fake(1, dtype=torch.float64), "empty": lambda: fake(0, dtype=torch.float32)}


@pytest.mark.parametrize("what", GLOBALS)
@pytest.mark.parametrize("name", calls(global_scale=None))
def test_a_bad_global_scale_is_refused(world, name, what):
    with pytest.raises(ValueError):
        calls(global_scale=GLOBALS[what]())[name]()
    assert not launched(world[0])


@pytest.mark.parametrize("name", calls(global_scale=None))
def test_a_good_global_scale_passes(world, name):
    for g in (fake(1, dtype=torch.float32), fake(1, dtype=torch.float32).reshape(())):
        calls(global_scale=g)[name]()
    assert len(launched(world[0])) == 2


OUTPUTS = {"too few rows": lambda: fake(3, 64), "too wide": lambda: fake(4, 72), "flat": lambda: fake(256),
           "fp16": lambda: fake(4, 64, dtype=torch.float16), "columns": lambda: fake(64, 4).t(),
           "on the host": lambda: torch.ones(4, 64, dtype=torch.bfloat16)}


@pytest.mark.parametrize("what", OUTPUTS)
@pytest.mark.parametrize("bias", [True, False])
def test_a_bad_output_is_refused(world, what, bias):
    kw = dict(bias=fake(64)) if bias else {}
    for call in (lambda y: nv.linear(fake(4, 64), nvfp4_tensor(64, 64), out=y, **kw),
                 lambda y: nv.gemm(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), out=y, **kw)):
        with pytest.raises(ValueError):
            call(OUTPUTS[what]())
        call(fake(4, 64))
    assert len(launched(world[0])) == 2


def spoilt(**parts):
    t = nvfp4_tensor(64, 64)
    return nv.NVFP4Tensor(**{**vars(t), **parts})


OPERANDS = {
    "codes too few": lambda: dict(codes=fake(63, 32, dtype=torch.uint8)),
    "codes with gaps": lambda: dict(codes=fake(64, 64, dtype=torch.uint8)[:, ::2]),
    "codes not 8 bits": lambda: dict(codes=fake(64, 32)),
    "codes on the host": lambda: dict(codes=torch.ones(64, 32, dtype=torch.uint8)),
    "scales too few": lambda: dict(sf=fake(511, dtype=torch.uint8)),
    "scales with gaps": lambda: dict(sf=fake(8192, dtype=torch.uint8)[::2]),
    "scales on the host": lambda: dict(sf=torch.ones(4096, dtype=torch.uint8)),
    "more rows than it has": lambda: dict(rows=65),
    "global on the host": lambda: dict(global_scale=torch.ones(1)),
    "global not FP32": lambda: dict(global_scale=fake(1)),
    "no global": lambda: dict(global_scale=fake(0, dtype=torch.float32)),
}


@pytest.mark.parametrize("what", OPERANDS)
def test_a_bad_operand_is_refused(world, what):
    h = fake(1, dtype=torch.float32)
    for call in (lambda t: nv.gemm(nvfp4_tensor(4, 64), t), lambda t: nv.gemm(t, nvfp4_tensor(64, 64)),
                 lambda t: nv.linear(fake(4, 64), t), lambda t: nv.linear(fake(4, 64), t, activation="silu"),
                 lambda t: nv.quantize(fake(64, 64), out=t),
                 lambda t: nv.gemm_swiglu_quant(t, nvfp4_tensor(256, 64), h),
                 lambda t: nv.gemm_swiglu_quant_dynamic(t, nvfp4_tensor(256, 64))):
        with pytest.raises(ValueError):
            call(spoilt(**OPERANDS[what]()))
    assert not launched(world[0])


@pytest.mark.parametrize("rows,k", [(32, 64), (128, 64), (64, 32)])
def test_an_nvfp4_output_of_another_size_is_refused(world, rows, k):
    h, out = fake(1, dtype=torch.float32), nvfp4_tensor(rows, k)
    for call in (lambda: nv.quantize(fake(64, 64), out=out), lambda: nv.quantize_noalloc(fake(64, 64), out),
                 lambda: nv.gemm_swiglu_quant(nvfp4_tensor(64, 64), nvfp4_tensor(128, 64), h, out=out),
                 lambda: nv.gemm_swiglu_quant_dynamic(nvfp4_tensor(64, 64), nvfp4_tensor(128, 64), out=out)):
        with pytest.raises(ValueError):
            call()
    assert not launched(world[0])


@pytest.mark.parametrize("call", [lambda: nv.linear(fake(4, 64), nvfp4_tensor(64, 64), out_dtype=torch.float16),
                                  lambda: nv.gemm(nvfp4_tensor(4, 64), nvfp4_tensor(64, 64), out_dtype=torch.float64)])
def test_a_bad_output_type_is_refused(world, call):
    with pytest.raises(ValueError):
        call()
    assert not launched(world[0])


def test_a_group_of_modules_is_checked(world):
    a, b = nvfp4_tensor(4, 64), nvfp4_tensor(8, 64)
    nv.fuse_group_scales([a, b])
    nv.fuse_group_scales([a, b], sf_out=fake(4096, dtype=torch.uint8), global_out=fake(1, dtype=torch.float32))
    assert len(launched(world[0])) == 2
    for modules, kw in (([a, nvfp4_tensor(8, 128)], {}),
                        ([a, spoilt(sf=torch.ones(4096, dtype=torch.uint8))], {}),
                        ([a, b], dict(sf_out=fake(4095, dtype=torch.uint8))),
                        ([a, b], dict(sf_out=torch.ones(4096, dtype=torch.uint8))),
                        ([a, b], dict(sf_out=fake(8192, dtype=torch.uint8)[::2])),
                        ([a, b], dict(global_out=torch.ones(1))), ([a, b], dict(global_out=fake(1)))):
        with pytest.raises(ValueError):
            nv.fuse_group_scales(modules, **kw)
    assert len(launched(world[0])) == 2


def test_silu_mul_is_checked(world):
    nv.silu_mul(fake(4, 64), out=fake(4, 32))
    assert len(launched(world[0])) == 1
    for y, out in ((fake(4, 63), None), (fake(64, 4).t(), None), (fake(256), None), (fake(4, 64), fake(3, 32)),
                   (fake(4, 64), fake(4, 64)), (fake(4, 64), fake(4, 32, dtype=torch.float32)),
                   (fake(4, 64), fake(32, 4).t()), (fake(4, 64), torch.ones(4, 32, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            nv.silu_mul(y, out=out)
    assert len(launched(world[0])) == 1
