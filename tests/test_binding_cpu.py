"""The Python binding without a GPU."""
import subprocess
import sys

import pytest


def test_the_package_imports_where_torch_has_no_cuda():
    """A torch built without CUDA lacks torch._C's CUDA functions; calls raise there, the import does not."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "import fp8_int8_quantized_gb300 as kvq\n"
            "c = kvq.KVCache(4, 2, 16, 64, 'e4m3', 'cpu')\n"
            "t, i = torch.zeros(4, 2, 64, dtype=torch.float16), torch.zeros(4, dtype=torch.int64)\n"
            "try:\n"
            "    kvq.append_rotary(t, t, t, c, i, i, torch.zeros(8, 64))\n"
            "except TypeError:\n"
            "    print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr


def rotary_status(out, out_stride, q=(1 << 20, 512), k=(2 << 20, 256), v=(3 << 20, 256), T=8):
    """kvq_append_rotary with 4 q-heads and 2 kv-heads of 128 channels; nothing is launched where it refuses."""
    import ctypes

    import fp8_int8_quantized_gb300 as kvq
    kvq.build()
    c = kvq.KvqCacheDesc(16, 16, None, None, 8, 16, 2, 128, kvq.E4M3, 0)
    return kvq.lib().kvq_append_rotary(*q, *k, *v, 0, 4, ctypes.byref(c), 16, T, 16, 1, None, 16, 100, 128, 0, None, kvq.E4M3,
                                       out, out_stride, None)


@pytest.mark.parametrize("kw", [
    dict(out=2 << 20, out_stride=512),                        # over k
    dict(out=3 << 20, out_stride=512),                        # over v
    dict(out=(2 << 20) + 2 * (7 * 256 + 248), out_stride=512),   # over the last elements of k's last row
    dict(out=(3 << 20) - 2 * (7 * 512 + 8), out_stride=512),     # its last row's last elements over v's first
    dict(out=(2 << 20) - 2 * (511 - 7), out_stride=512, T=1),
    dict(out=1 << 20, out_stride=520), dict(out=1 << 20, out_stride=504 + 16 + 512),   # over q, other rows
    # one fused buffer [q | k | v], rows of 1024: over k, over v, into the next token's q
    dict(q=(1 << 20, 1024), k=((1 << 20) + 1024, 1024), v=((1 << 20) + 1536, 1024), out=(1 << 20) + 1024, out_stride=1024),
    dict(q=(1 << 20, 1024), k=((1 << 20) + 1024, 1024), v=((1 << 20) + 1536, 1024), out=(1 << 20) + 1040, out_stride=1024),
    dict(q=(1 << 20, 1024), k=((1 << 20) + 1024, 1024), v=((1 << 20) + 1536, 1024), out=(1 << 20) + 16, out_stride=1024),
    dict(q=(1 << 20, 1024), k=((1 << 20) + 1024, 1024), v=((1 << 20) + 1536, 1024), out=(1 << 20) - 1024, out_stride=1024)])
def test_rotated_queries_are_refused_over_the_rows_that_are_read(kw):
    assert rotary_status(**kw) == 1


@pytest.mark.parametrize("sizes", [(2, 18, 2, 128, 4, 1000, 1), (4097, 8, 2, 128, 4, 1000, 1), (2, 8, 2, 96, 4, 1000, 1), (2, 8, 2, -128, 4, 1000, 1),
                                   (2, 8, 2, 128, 4, (1 << 30) + 1, 1), (2, 8, 2, 128, 4, 1000, 9), (2, (1 << 31) - 1, 1, 128, 64, 1000, 1)])
def test_no_workspace_for_what_is_not_taken(sizes):
    import fp8_int8_quantized_gb300 as kvq
    kvq.build()
    assert kvq.lib().kvq_verify_workspace_size(*sizes) == 0
    assert kvq.lib().kvq_verify_workspace_size(2, 16, 2, 128, 4, 1 << 30, 1) > 0


def test_a_stream_of_another_device_is_refused():
    """The call would run on the current stream of the cache's device instead."""
    from types import SimpleNamespace

    import torch

    import fp8_int8_quantized_gb300 as kvq
    with pytest.raises(ValueError, match="cuda:1"):
        kvq._on(0, SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7), lambda s: s)


def test_the_build_checks_registers():
    from fp8_int8_quantized_gb300 import build_lib as b
    report = ("ptxas info    : Compiling entry function '{}' for 'sm_103a'\n"
              "ptxas info    : Function properties for {}\n    0 bytes stack frame\n"
              "ptxas info    : Used {} registers, used 16 barriers, 448 bytes smem\n")
    tc, other = "_ZN3kvq6verify2tc16verify_tc_kernelILi3ELi64ELi1EEE", "_ZN3kvq6verify13verify_kernelILi3E"
    b.check_registers(report.format(tc, tc, 96) + report.format(other, other, 255))
    with pytest.raises(RuntimeError, match="88 registers"):
        b.check_registers(report.format(other, other, 255) + report.format(tc, tc, 96) + report.format(tc, tc, 88))


def test_a_kernel_with_other_registers_is_not_built(tmp_path, monkeypatch):
    """Through the build itself, on a source of its own whose kernel bears the checked name."""
    from fp8_int8_quantized_gb300 import build_lib as b
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "k.cu").write_text("__global__ void verify_tc_kernel(float* x) { x[threadIdx.x] += 1.f; }\n")
    for name, value in (("CSRC", tmp_path / "csrc"), ("BUILD", tmp_path / "b"), ("LIB", tmp_path / "l.so")):
        monkeypatch.setattr(b, name, str(value))
    with pytest.raises(RuntimeError, match="registers per thread"):
        b.build()
    assert not (tmp_path / "l.so").exists() and not (tmp_path / "b" / "k.o").exists()
