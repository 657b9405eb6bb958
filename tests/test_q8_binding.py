"""The extension that marshals the 8-bit calls is the 8-bit calls' matter only
(no GPU needed)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "hybrid_sparse_gemm_b200")

PROGRAM = """
import torch
import hybrid_sparse_gemm_b200 as hsg
assert hsg.version() > 0
tables, size = hsg.patch_plan(256, 256, [0, 1, 1, 0])
assert size > 0 and tables[0].size == 8
x, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
for call in (lambda: hsg.patch_quantize_q8(x, q, s), lambda: hsg.patch_silu_mul_q8(x, x, q, s),
             lambda: hsg.patch_dequantize_q8(q, s, x)):
    try:
        call()
    except ImportError as e:
        assert "_binding" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("an 8-bit call ran without its extension")
"""


def test_package_without_the_extension(tmp_path):
    shutil.copytree(PACKAGE, tmp_path / "hybrid_sparse_gemm_b200", ignore=shutil.ignore_patterns("*.so", "csrc", "__pycache__"))
    env = dict(os.environ, PATCH_HYBRID_LIB=os.path.join(PACKAGE, "libpatch_hybrid.so"))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_extension_is_of_this_interpreter():
    """One built for another Python is neither loaded nor taken for this one's."""
    import hybrid_sparse_gemm_b200 as hsg
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert hsg._binding.__file__.endswith("_binding" + suffix) and suffix != ".so"
    build = pytest.importorskip("hybrid_sparse_gemm_b200.build")
    assert os.path.samefile(build.BINDING, hsg._binding.__file__)
