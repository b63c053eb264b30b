"""The refusal tests under an allocator that overwrites what is freed: a structure whose address the library got is alive."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_refusal_tests_read_no_freed_memory():
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_cache_cpu.py", "-q", "-k", "refusals"], cwd=ROOT,
                       env=dict(os.environ, PYTHONMALLOC="debug"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
