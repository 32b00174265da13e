"""Loading the library: first calls from several threads, and what a failed load leaves behind (fresh processes, no GPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def fresh(code: str) -> str:
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


def test_first_calls_from_several_threads():
    """Every one of them finds the library whole, also one that comes while another is still loading the extension: the
    refusal of its argument, and nothing else."""
    out = fresh("""
import threading, time
import sparse_attention_02_gb300 as dsa
load, loading, seen = dsa._load_fastcall, threading.Event(), []
def slow(path):
    loading.set()
    time.sleep(0.5)
    return load(path)
dsa._load_fastcall = slow
def first():
    try:
        dsa.dsa_rmsnorm(None, None, 1e-6)
    except Exception as e:
        seen.append(type(e).__name__ + ": " + str(e))
threads = [threading.Thread(target=first) for _ in range(8)]
threads[0].start()
loading.wait()
[t.start() for t in threads[1:]]
[t.join() for t in threads]
assert len(seen) == 8
print("|".join(sorted(set(seen))))
""")
    assert out == "TypeError: x must be a torch.Tensor"


def test_a_failed_load_is_told_every_time():
    """A library that cannot be loaded is named by each call, and one that can be later is loaded then."""
    out = fresh("""
import sparse_attention_02_gb300 as dsa
whole, dsa.LIB_PATH = dsa.LIB_PATH, dsa.LIB_PATH + ".none"
for _ in range(2):
    try:
        dsa.dsa_rmsnorm(None, None, 1e-6)
    except RuntimeError as e:
        assert "is missing" in str(e)
        print("missing")
dsa.LIB_PATH = whole
try:
    dsa.dsa_rmsnorm(None, None, 1e-6)
except TypeError as e:
    print(e)
""")
    assert out.split("\n") == ["missing", "missing", "x must be a torch.Tensor"]


def test_a_failed_extension_is_told_every_time():
    """What goes wrong while the extension loads is not left for later calls to trip over."""
    out = fresh("""
import sparse_attention_02_gb300 as dsa
load, seen = dsa._load_fastcall, []
def broken(path):
    raise OSError("cannot load it")
dsa._load_fastcall = broken
for _ in range(2):
    try:
        dsa.dsa_rmsnorm(None, None, 1e-6)
    except Exception as e:
        print(type(e).__name__, e)
dsa._load_fastcall = load
try:
    dsa.dsa_rmsnorm(None, None, 1e-6)
except TypeError as e:
    print(e)
""")
    assert out.split("\n") == ["OSError cannot load it"] * 2 + ["x must be a torch.Tensor"]


def test_without_the_extension_calls_take_the_python_form():
    """libdsa.so alone serves every entry point; that the extension is missing is said once."""
    out = fresh("""
import sys, warnings
sys.modules["sparse_attention_02_gb300._fastcall"] = None  # its import fails
import sparse_attention_02_gb300 as dsa
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for call in (lambda: dsa.dsa_rmsnorm(None, None, 1e-6), lambda: dsa.dsa_index_rope_backward(None, None, None, None),
                 lambda: dsa.dsa_quantize_fp8(None, None, None)):
        try:
            call()
        except (TypeError, ValueError, AttributeError) as e:
            print(type(e).__name__)
    print(dsa.dsa_mla_decode_workspace_size(2, 16) > 0, dsa.dsa_rmsnorm_backward_workspace_size(4, 64) > 0)
print([str(w.message).split(" (")[0] for w in seen])
""")
    lines = out.split("\n")
    assert lines[:2] == ["TypeError", "TypeError"] and lines[3:] == ["True True", "['the native call path is not used']"]


def test_without_headers_the_extension_is_left_out(monkeypatch, tmp_path):
    from sparse_attention_02_gb300 import build

    monkeypatch.setattr(build, "FAST", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(RuntimeWarning, match="Python.h is missing"):
        build._build_fastcall()
    assert not os.listdir(tmp_path)


def test_an_extension_for_another_pytorch_is_not_loaded():
    """It is known by what stands beside it, without importing it."""
    out = fresh("""
import sys, warnings
import sparse_attention_02_gb300 as dsa
from sparse_attention_02_gb300 import build
assert build.fastcall_built_for() == build.fastcall_abi()
build.fastcall_abi = lambda: "another"
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    dsa.load_library()
print(dsa._fast, "sparse_attention_02_gb300._fastcall" in sys.modules, len(seen))
""")
    assert out == "None False 1"


def test_the_extension_is_built_anew_for_another_interpreter_pytorch_or_compiler(monkeypatch, tmp_path):
    """Whatever its files' times say: a PyTorch that was put back is older than the extension built for the other."""
    from sparse_attention_02_gb300 import build

    built = []

    def run(cmd, **kw):
        built.append(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "FAST", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build, "FAST_KEY", str(tmp_path / "_fastcall.key"))
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setenv("CXX", "one")
    for _ in range(2):
        build._build_fastcall()
    assert built == ["one"]
    monkeypatch.setenv("CXX", "two")
    build._build_fastcall()
    assert built == ["one", "two"]
    was = build.fastcall_abi()
    monkeypatch.setattr(build, "fastcall_abi", lambda: "another")
    for _ in range(2):
        build._build_fastcall()
    assert built == ["one", "two", "two"] and build.fastcall_built_for() == "another" != was
    os.remove(tmp_path / "_fastcall.key")  # a build that was cut short
    build._build_fastcall()
    assert len(built) == 4 and sorted(os.listdir(tmp_path)) == ["_fastcall.key", "_fastcall.so"]


def test_a_pytorch_that_does_not_say_its_version_leaves_the_python_form():
    out = fresh("""
import warnings
import sparse_attention_02_gb300 as dsa
from sparse_attention_02_gb300 import build
build._torch_root = lambda: "/nowhere"
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    dsa.load_library()
print(dsa._fast, len(seen))
""")
    assert out == "None 1"
