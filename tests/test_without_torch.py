"""The C library builds, and the package imports, where torch cannot be imported (CPU only)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, *args):
    head = "import sys; sys.modules['torch'] = None\n"  # import torch: ImportError
    r = subprocess.run([sys.executable, "-c", head + code, *args], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stderr


BUILD = """
import os
from bit_ptq_reconstruction_amd import build
build.OBJ_DIR, build.LIB, build.BINDING = (os.path.join(sys.argv[1], n) for n in ("obj", "libqv.so", "_decode.so"))
build.SOURCES = ["qv_decode_abi.cpp"]  # any one of them
"""


def test_library_builds(tmp_path):
    note = run(BUILD + "build.build_library()\nassert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)",
               str(tmp_path))
    assert "_decode.so is not built" in note


def test_library_is_there_when_the_binding_fails(tmp_path):
    run(BUILD + """
sys.modules['torch'] = type(sys)('torch')
def fail(): raise RuntimeError("no headers")
build._compile_binding = fail
try:
    build.build_library()
except RuntimeError as e:
    assert "no headers" in str(e)
else:
    assert False
assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
""", str(tmp_path))


def test_package_imports():
    """Every public name, the single-token calls among them; those need torch when they are called."""
    run("""
from bit_ptq_reconstruction_amd import *
import bit_ptq_reconstruction_amd as qv
assert qv_paged_attention is qv.qv_paged_attention and QV_KV_INT8 == 1 and callable(qv_w4a4_gemm)
""")
