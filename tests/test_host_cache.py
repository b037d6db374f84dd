"""The library's host-side caches against a driver that counts (no GPU)."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_nothing_is_asked_of_the_driver_twice(tmp_path):
    """Forty layers' buffers and every kernel of the library in turn, twice:
    the second time around no descriptor is encoded and no limit raised, so
    that calls on many layers or of many forms do not slow one another down;
    and whatever is asked for comes back right."""
    exe = str(tmp_path / "client")
    csrc = os.path.join(ROOT, "long_context_sparse_gated_b200", "csrc")
    subprocess.run(["g++", "-x", "c++", "-std=c++17", "-O1", f"-I{CUDA}/include", f"-I{ROOT}/include", f"-I{csrc}",
                    os.path.join(ROOT, "tests", "host_cache_client.cpp"), "-o", exe, "-lpthread"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    assert out.stdout.split() == ["160", "0", "96", "0", "0"]
