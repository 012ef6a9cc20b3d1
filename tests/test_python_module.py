"""The package without its compiled calls (_pagedattn_calls): the others work, and the
calls that need the module say so."""
import os
import subprocess
import sys

import pytest

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


@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    """build.build() into tmp_path, with compilers that only make their output file.
    .fails: a text; the commands that contain it fail. .ran: the commands."""
    from paged_kv_attention_06_gb300 import build

    class Fake:
        fails = "\0"
        ran = []

    def run(cmd, **kw):
        fake.ran.append(cmd)
        failed = any(fake.fails in str(x) for x in cmd)
        if not failed:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("made")
        return subprocess.CompletedProcess(cmd, int(failed), "", "")

    fake = Fake()
    fake.build, fake.ran = build, []
    for name in ("LIB", "BENCH_LIB", "PYTHON_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "_nvcc", lambda: sys.executable)
    monkeypatch.setattr(build.subprocess, "run", run)
    return fake


@pytest.mark.parametrize("what", ["pa_python.cpp", "-ltorch_python"])
def test_the_library_is_built_where_the_module_cannot_be(fake_build, what):
    fake_build.fails = what
    with pytest.raises(RuntimeError):
        fake_build.build.build()
    assert os.path.exists(fake_build.build.LIB) and os.path.exists(fake_build.build.BENCH_LIB)
    assert not os.path.exists(fake_build.build.PYTHON_LIB)
    fake_build.fails = "\0"
    fake_build.build.build()
    assert os.path.exists(fake_build.build.PYTHON_LIB) and fake_build.build.up_to_date()


def test_another_torch_means_another_build(fake_build, monkeypatch):
    import torch
    fake_build.build.build()
    assert fake_build.build.up_to_date()
    n = len(fake_build.ran)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not fake_build.build.up_to_date()
    fake_build.build.build()
    assert len(fake_build.ran) > n and fake_build.build.up_to_date()
