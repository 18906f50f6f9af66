"""Refusals of the 8-bit and ragged products (include/nvfp4_moe_products.h): every
check runs on the host before anything is enqueued, so none of these needs a GPU and
none of the made-up addresses is ever dereferenced."""
import ctypes as C

import pytest
import torch

import nvfp4_mixture_experts_03_b200 as nv
from nvfp4_mixture_experts_03_b200 import products

INVALID, DIMS, MISALIGNED, NO_DEVICE = -1, -2, -3, -9
BF16, F16, F32, INT8 = 0, 1, 2, 3
BASE = 1 << 40
CALLS = {"fwd": nv.nvfp4_moe_grouped_gemm, "dx": nv.nvfp4_moe_grouped_gemm_dx, "dw": nv.nvfp4_moe_grouped_gemm_dw}


@pytest.fixture(scope="module", autouse=True)
def built():
    from nvfp4_mixture_experts_03_b200 import build
    build.build()
    return nv.lib()


def _gemm(**over):
    d = dict(groups=4, rows=100, n=96, k=64, type=BF16, out_type=BF16, accumulate=0, offsets=BASE,
             x=BASE + (1 << 20), x_stride=64, x_scale=BASE + (2 << 20), dy=BASE + (3 << 20), dy_stride=96,
             w=BASE + (4 << 20), w_stride=64, w_scale=BASE + (5 << 20), out=BASE + (6 << 20), out_stride=96)
    d.update(over)
    return nv.GemmIO(**d)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the made-up addresses pass every check; needs a machine without a GPU")
@pytest.mark.parametrize("which", sorted(CALLS))
def test_good_arguments_reach_the_device_check(which):
    assert CALLS[which](_gemm(), 0) == NO_DEVICE


GEMM_REFUSALS = [
    (dict(groups=0), INVALID, "all"), (dict(groups=-1), INVALID, "all"), (dict(groups=1025), DIMS, "all"),
    (dict(rows=(1 << 30) + 1), DIMS, "all"), (dict(n=(1 << 30) + 1), DIMS, "all"), (dict(k=(1 << 30) + 1), DIMS, "all"),
    (dict(n=1 << 29), DIMS, "dw"),                              # 4 * n rows of dw
    (dict(rows=-1), INVALID, "all"), (dict(n=0), INVALID, "all"), (dict(k=0), INVALID, "all"),
    (dict(type=F32), INVALID, "all"), (dict(type=7), INVALID, "all"), (dict(type=-1), INVALID, "all"),
    (dict(type=INT8), INVALID, "dx dw"),
    (dict(out_type=INT8), INVALID, "all"), (dict(out_type=9), INVALID, "all"),
    (dict(accumulate=1), INVALID, "all"),                       # a 16-bit output
    (dict(accumulate=1, out_type=F16), INVALID, "all"),
    (dict(offsets=None), INVALID, "all"),                       # four groups
    (dict(offsets=BASE + 2), MISALIGNED, "all"),
    (dict(x=None), INVALID, "fwd dw"), (dict(x=BASE + 8), MISALIGNED, "fwd dw"),
    (dict(x_stride=63), INVALID, "fwd dw"), (dict(x_stride=66), MISALIGNED, "fwd dw"),
    (dict(x_stride=1 << 40), DIMS, "fwd dw"), (dict(x_stride=-64), INVALID, "fwd dw"), (dict(x_stride=0), INVALID, "fwd dw"),
    (dict(dy=None), INVALID, "dx dw"), (dict(dy=BASE + 4), MISALIGNED, "dx dw"),
    (dict(dy_stride=95), INVALID, "dx dw"), (dict(dy_stride=100), MISALIGNED, "dx dw"),
    (dict(w=None), INVALID, "fwd dx"), (dict(w=BASE + 2), MISALIGNED, "fwd dx"),
    (dict(w_stride=56), INVALID, "fwd dx"), (dict(w_stride=65), MISALIGNED, "fwd dx"),
    (dict(w_stride=1 << 36), DIMS, "fwd dx"),                   # n rows of it pass a tensor map's stride
    (dict(out=None), INVALID, "all"), (dict(out=BASE + 1), MISALIGNED, "all"),
    (dict(out=BASE + 2, out_type=F32), MISALIGNED, "all"),
    (dict(out_stride=60), INVALID, "all"), (dict(out_stride=95), INVALID, "fwd"),
    (dict(out=BASE + (1 << 20)), INVALID, "fwd dw"),            # out is x
    (dict(out=BASE + (3 << 20)), INVALID, "dx dw"),             # out is dy
    (dict(out=BASE + (4 << 20)), INVALID, "fwd dx"),            # out is w
    (dict(type=INT8, k=131072, x_stride=131072, w_stride=131072), DIMS, "fwd"),
    (dict(type=INT8, x_scale=None), INVALID, "fwd"), (dict(type=INT8, w_scale=None), INVALID, "fwd"),
    (dict(type=INT8, x_scale=BASE + 2), MISALIGNED, "fwd"), (dict(type=INT8, w_scale=BASE + 3), MISALIGNED, "fwd"),
    (dict(type=INT8, k=60, x_stride=72), MISALIGNED, "fwd"),
]


@pytest.mark.parametrize("over,code,which", GEMM_REFUSALS)
def test_products_refuse(over, code, which):
    for name in sorted(CALLS) if which == "all" else which.split():
        assert CALLS[name](_gemm(**over), 0) == code, name


def test_null_io_is_refused():
    L = nv.lib()
    for name in ("nvfp4_moe_quantize_int8", "nvfp4_moe_grouped_gemm", "nvfp4_moe_grouped_gemm_dx", "nvfp4_moe_grouped_gemm_dw"):
        assert getattr(L, name)(None, None) == INVALID


def test_no_rows_is_a_no_op_of_the_products_and_the_quantiser():
    for name in ("fwd", "dx"):
        assert CALLS[name](_gemm(rows=0, x=None, dy=None, out=None), 0) == 0
    assert nv.nvfp4_moe_quantize_int8(nv.QuantizeIO(0, 16, BF16, 0, None, 16, None, 16, None), 0) == 0


def _quant(**over):
    d = dict(rows=4, cols=64, in_type=BF16, swiglu=0, in_=BASE, in_stride=64, q=BASE + 4096, q_stride=64, scale=BASE + 8192)
    d.update(over)
    return nv.QuantizeIO(**d)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(in_type=INT8), INVALID), (dict(in_type=5), INVALID),
    (dict(swiglu=2), INVALID), (dict(swiglu=1), INVALID),       # a stride of one row of values, not of gate | up
    (dict(cols=(1 << 30) + 1, in_stride=1 << 31, q_stride=1 << 31), DIMS),
    (dict(in_=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(in_stride=63), INVALID), (dict(q_stride=63), INVALID), (dict(q=BASE), INVALID),
    (dict(in_=BASE + 1), MISALIGNED), (dict(in_=BASE + 2, in_type=F32), MISALIGNED), (dict(scale=BASE + 2), MISALIGNED),
])
def test_quantiser_refuses(over, code):
    assert nv.nvfp4_moe_quantize_int8(_quant(**over), 0) == code


def test_structures_match_the_header(tmp_path):
    """sizeof and every field's offset, as a C compiler lays the header's structures out."""
    import os
    import subprocess
    from conftest import ROOT
    rename = {"in_": "in"}
    lines = []
    for c_name, cls in (("nvfp4_moe_quantize_io", nv.QuantizeIO), ("nvfp4_moe_gemm_io", nv.GemmIO)):
        lines.append(f'printf("%zu\\n", sizeof({c_name}));')
        lines += [f'printf("%zu\\n", offsetof({c_name}, {rename.get(f, f)}));' for f, _ in cls._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "nvfp4_moe_products.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = str(tmp_path / "t")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe])
    got = [int(v) for v in subprocess.check_output([exe]).split()]
    want = []
    for cls in (nv.QuantizeIO, nv.GemmIO):
        want += [C.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want
    # the same layouts as the tensor calls pack them
    import struct
    assert [struct.calcsize("@4iPqPqP"), struct.calcsize("@7iPPqPPqPqPPq")] == [C.sizeof(nv.QuantizeIO), C.sizeof(nv.GemmIO)]
    v = list(range(1, 19))
    assert products._pack_gemm(*v) == bytes(nv.GemmIO(*v))
    assert products._pack_quantize(*v[:9]) == bytes(nv.QuantizeIO(*v[:9]))
    assert (products.TYPE_BF16, products.TYPE_F16, products.TYPE_F32, products.TYPE_INT8) == (BF16, F16, F32, INT8)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: nv.quantize_int8(_t(4, 64)),                                            # not on a GPU
    lambda: nv.quantize_int8(_t(4, 64, dtype=torch.int8)),
    lambda: nv.quantize_int8(_t(4, 7), swiglu=True),
    lambda: nv.quantize_int8(_t(4, 64).t()),
    lambda: nv.quantize_int8(_t(64)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(2, 8, 64)),                               # two groups, no offsets
    lambda: nv.grouped_gemm(_t(4, 64), _t(8, 64)),                                  # not on a GPU
    lambda: nv.grouped_gemm(_t(4, 64), _t(8, 64, dtype=torch.float16)),
    lambda: nv.grouped_gemm(_t(4, 64, dtype=torch.float32), _t(8, 64, dtype=torch.float32)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(2, 8, 64), torch.zeros(3, dtype=torch.int64)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(2, 8, 64), torch.zeros(4, dtype=torch.int32)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(8, 72)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(8, 64), accumulate=True),
    lambda: nv.grouped_gemm(_t(4, 64), _t(8, 64), out=_t(4, 9)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(8, 64), x_scale=torch.zeros(4), w_scale=torch.zeros(8)),
    lambda: nv.grouped_gemm(_t(4, 64), _t(64, 8).t()),
    lambda: nv.grouped_gemm(_t(4, 64), _t(4, 8, 64)[::2], torch.zeros(3, dtype=torch.int32)),
    lambda: nv.gemm_int8(_t(4, 64), _t(8, 64), torch.zeros(4), torch.zeros(8)),
    lambda: nv.gemm_int8(_t(4, 64, dtype=torch.int8), _t(8, 64, dtype=torch.int8), torch.zeros(5), torch.zeros(8)),
    lambda: nv.gemm_int8(_t(4, 64, dtype=torch.int8), _t(8, 64, dtype=torch.int8), torch.zeros(4), torch.zeros(8, dtype=torch.float64)),
    lambda: nv.grouped_gemm_dx(_t(4, 64, dtype=torch.int8), _t(64, 8, dtype=torch.int8)),
    lambda: nv.grouped_gemm_dx(_t(4, 64), _t(65, 8)),
    lambda: nv.grouped_gemm_dw(_t(4, 64), _t(5, 8)),
    lambda: nv.grouped_gemm_dw(_t(4, 64), _t(4, 8), torch.zeros(1, dtype=torch.int32)),
])
def test_python_calls_refuse(call):
    with pytest.raises((ValueError, nv.NVFP4MoEError)):
        call()


def test_what_is_misaligned_is_said():
    with pytest.raises(nv.NVFP4MoEError, match="16 bytes.*MISALIGNED") as e:
        products._failed(MISALIGNED, "nvfp4_moe_grouped_gemm")
    assert e.value.code == MISALIGNED
    with pytest.raises(nv.NVFP4MoEError) as e:
        products._failed(DIMS, "nvfp4_moe_grouped_gemm")
    assert "16 bytes" not in str(e.value)


def test_the_library_is_built_without_the_binding(monkeypatch, tmp_path, capsys):
    """No compiler, no headers, no torch: the library is built all the same, and first."""
    from nvfp4_mixture_experts_03_b200 import build
    monkeypatch.setattr(build, "marshal_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setenv("CXX", "/bin/false")
    seen = []
    monkeypatch.setattr(build, "build_library", lambda *a: seen.append(a) or build.LIB)
    assert build.build() == build.LIB and len(seen) == 1
    assert "binding" in capsys.readouterr().err


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    from nvfp4_mixture_experts_03_b200 import build
    import sysconfig
    assert products._load_marshal() is not None
    assert build.marshal_path().endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert products._load_marshal() is None


def test_the_binding_follows_every_header(monkeypatch):
    """Newer than its source and one header, older than the other that it includes: built again."""
    import os
    from nvfp4_mixture_experts_03_b200 import build
    path = build.build_marshal()
    called = []
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd: called.append(cmd) or open(cmd[cmd.index("-o") + 1], "wb").close())
    monkeypatch.setattr(build.os, "replace", lambda a, b: os.unlink(a))
    assert build.build_marshal() == path and not called
    real = os.path.getmtime
    monkeypatch.setattr(build.os.path, "getmtime", lambda p: real(p) + (1e6 if p.endswith("nvfp4_moe.h") else 0))
    assert build.build_marshal() == path and len(called) == 1
