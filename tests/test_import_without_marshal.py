"""The package without its marshalling module (not built, or built against
another torch): the calls that go to libbgg.so through ctypes alone keep
working, the decoder-layer calls say what is missing.  Each case in a process
of its own; no GPU calls."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

ABSENT = "import sys; sys.modules['bit_gemv_gemm_amd._marshal'] = None"
# the module of another torch imports, but what it knows of tensors is not
# this torch's: nothing of it may be called
OTHER = """
import sys, types
class Other(types.ModuleType):
    torch_version = '0.0.1'
    def bind(self, *a):
        raise AssertionError('bound')
    product = paged_attention = rotary_append = bind
sys.modules['bit_gemv_gemm_amd._marshal'] = Other('bit_gemv_gemm_amd._marshal')
"""
BODY = """
import numpy as np, torch
import bit_gemv_gemm_amd as bgg
d = bgg.bgg_describe('PQ2_0', 64, 128)
packed = bgg.bgg_pack_weights(d, np.ones((64, 128), np.int8), np.ones((64, 1), np.float16))
bgg.bgg_validate_packed(d, packed)
assert bgg.bgg_gemv_workspace_size(d, 1) > 0 and bgg.bgg_gemv_kernel_name(d, 1)
c = bgg.bgg_cache_describe('f16', 2, 16, 1, 64)
assert bgg.bgg_attention_workspace_size(c, 1, 1) > 0 and len(bgg.bgg_rotary_frequencies(64, 1e4)[0]) == 32
t = torch.zeros(1)
for call in (lambda: bgg.bgg_ternary_gemv_epilogue(d, t, t, t, 1, 0, t), lambda: bgg.bgg_gemv_run_epilogue(d, t, t, 1, t),
             lambda: bgg.bgg_ternary_gemm_epilogue(d, t, t, t, 1, 0, t),
             lambda: bgg.bgg_rotary_append(c, t, t, t, t, t, q=t, q_out=t),
             lambda: bgg.bgg_paged_attention(c, t, t, t, t, t, t, t, scale=1.0)):
    try:
        call()
    except ImportError as e:
        assert '_marshal' in str(e) and 'build' in str(e), e
    else:
        raise AssertionError('no error')
print('done')
"""


@pytest.mark.parametrize("missing", [ABSENT, OTHER], ids=["absent", "of another torch"])
def test_import_and_the_older_calls(missing):
    r = subprocess.run([sys.executable, "-c", missing + BODY], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-1500:]


def test_the_built_module_names_its_torch():
    torch = pytest.importorskip("torch")
    import bit_gemv_gemm_amd as bgg
    assert bgg._marshal.torch_version == torch.__version__.split("+")[0]
