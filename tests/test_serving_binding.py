"""Host-side checks of the compiled binding of the serving calls: frequencies, and what the
package does without it.  No GPU: every call is refused, or is an empty call, before anything
is enqueued."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def C():
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def calls(C, f):
    dm = C.dims(1, 2, 1, 64)
    yield lambda: C.kvs_rope(dm, 0, None, 64, f, False, None, None, None, None, stream=0)
    yield lambda: C.kvs_append_paged(dm, 0, 0, None, None, 64, f, False, None, None, None, None, 16,
                                     None, None, 0, None, None, None, 1, None, None, None, 0, stream=0)


def test_frequencies_off_the_host_are_refused(C):
    """Reading them one by one would wait for the device each time and cannot be captured."""
    for dtype in (torch.float64, torch.float32):
        for call in calls(C, torch.zeros(32, dtype=dtype, device="meta")):
            with pytest.raises(ValueError, match="inv_freq must be in host memory"):
                call()


def test_frequencies_of_other_types(C):
    """CPU tensors of any real type and layout; the library refuses a value that is not finite,
    so that it shows which ones were read."""
    for dtype in (torch.float64, torch.float32, torch.float16, torch.bfloat16):
        good = torch.linspace(1, 0.01, 32).to(dtype)
        bad = good.clone()
        bad[31] = float("inf")
        behind = torch.cat([good, bad[31:]])               # what is not needed is not read
        twice = torch.stack([good, bad], 1)[:, 0]          # nor what lies between
        for f in (good, behind, twice, good.clone().requires_grad_()):
            for call in calls(C, f):
                call()
        for f in (bad, torch.stack([good, bad], 1)[:, 1], bad.clone().requires_grad_()):
            for call in calls(C, f):
                with pytest.raises(C.KvsError, match=r"inv_freq\[31\] is not finite"):
                    call()
        for call in calls(C, good[:31]):
            with pytest.raises(ValueError, match="31 frequencies, 32 needed"):
                call()
    for call in calls(C, torch.ones(32, dtype=torch.int64)):
        call()
    for call in calls(C, torch.ones(32, dtype=torch.complex64)):
        with pytest.raises(TypeError):
            call()


# ----------------------------------------------------------------------------- loading

PACKAGE = "kv_cache_eviction_lse_gb300"
USE = """
import ctypes, sys
sys.path.insert(0, {root!r})
from kv_cache_eviction_lse_gb300 import capi as C
assert "kvs" in C.kvs_version() and C.kvs_compact_workspace_size(C.dims(1, 2, 1, 64), 100) > 0
assert C.kvs_attn_decode_workspace_size(C.dims(1, 2, 1, 64), 3) > 0
def call():
    C.kvs_rope(C.dims(1, 2, 1, 64), 0, None, 0, None, False, None, None, None, None, stream=0)
for _ in range(2):
    try:
        call()
    except ImportError as e:
        assert all(x in str(e) for x in ("kvs binding", {why!r}, "kv_cache_eviction_lse_gb300.build")), e
    else:
        raise AssertionError("no binding, no error")
"""


def copy_of_package(C, tmp_path, binding):
    """The package's Python files and its built library, and of the binding what is named."""
    src = os.path.dirname(C.__file__)
    to = tmp_path / PACKAGE
    (to / "_lib").mkdir(parents=True)
    for f in os.listdir(src):
        if f.endswith(".py"):
            shutil.copy(os.path.join(src, f), to)
    for f in ("libkvs.so", *binding):
        shutil.copy(os.path.join(src, "_lib", f), to / "_lib")
    return to


@pytest.mark.parametrize("binding", [[], ["kvs_binding.so"], ["kvs_binding.txt"]], ids=str)
def test_without_the_binding_the_other_calls_work(C, tmp_path, binding):
    copy_of_package(C, tmp_path, binding)
    r = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path), why="not built")],
                       capture_output=True, text=True, cwd=tmp_path)
    assert r.returncode == 0, r.stderr


def test_a_binding_of_another_python_or_torch_is_not_loaded(C, tmp_path):
    to = copy_of_package(C, tmp_path, ["kvs_binding.txt"])
    (to / "_lib" / "kvs_binding.so").write_bytes(b"not to be opened")
    mark = to / "_lib" / "kvs_binding.txt"
    here = mark.read_text()
    assert torch.__version__ in here and f"cpython-{sys.version_info[0]}{sys.version_info[1]}" in here
    for other in (here.replace("cpython-3", "cpython-2"), here + ".post1"):
        mark.write_text(other)
        r = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path), why=other)],
                           capture_output=True, text=True, cwd=tmp_path)
        assert r.returncode == 0, r.stderr


def test_the_library_is_built_where_the_binding_cannot_be(C, tmp_path, monkeypatch):
    """No g++, or no headers: the library is there, a warning says what is not, and the binding
    of another build is not left to be loaded."""
    from kv_cache_eviction_lse_gb300 import build
    out = copy_of_package(C, tmp_path, ["kvs_binding.txt", "kvs_binding.so"]) / "_lib"
    for name, f in (("OUT", ""), ("LIB", "libkvs.so"), ("BINDING", "kvs_binding.so"),
                    ("BUILT_FOR", "kvs_binding.txt")):
        monkeypatch.setattr(build, name, str(out / f))
    monkeypatch.setattr(build, "sources", lambda: [])
    done = []

    def run(what, cmd, verbose=False):
        if what == "binding.cpp":
            raise FileNotFoundError("g++")
        done.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "_run", run)
    with pytest.warns(UserWarning, match="binding of the serving calls was not built: g"):
        assert build.build(force=True) == str(out / "libkvs.so")
    assert done == ["link"] and os.path.getsize(out / "libkvs.so") == 0
    assert not os.path.exists(out / "kvs_binding.txt")
    monkeypatch.undo()
    assert build.build() == C.LIB_PATH and C.load_binding().rope
