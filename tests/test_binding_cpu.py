"""The Python binding without a GPU."""
import subprocess
import sys


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
