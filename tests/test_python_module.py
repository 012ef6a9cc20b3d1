"""The package without its compiled calls (_pagedattn_calls): the others work, and the
calls that need the module say so."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
from paged_kv_attention_06_gb300 import build
build.PYTHON_LIB = sys.argv[1]
import paged_kv_attention_06_gb300 as pa
c = pa.KVCache(8, 4)
c.add(1)
c.plan([1], [5], 4, 5)
assert c.context_len(1) == 5 and pa.version()
try:
    pa.pa_decode_window(None, None, None, None, None, 16, window=4)
except ImportError as e:
    print("refused:", e)
"""


def run(path):
    r = subprocess.run([sys.executable, "-c", SCRIPT, path], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_without_the_module():
    from paged_kv_attention_06_gb300 import build
    build.build()
    assert "not built" in run(os.path.join(ROOT, "no_such_module.so"))


def test_with_a_module_that_does_not_load(tmp_path):
    from paged_kv_attention_06_gb300 import build
    build.build()
    bad = tmp_path / "_pagedattn_calls.so"
    bad.write_bytes(b"another torch's")
    assert "refused:" in run(str(bad))
