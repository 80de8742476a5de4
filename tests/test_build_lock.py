"""Several ranks that find the library stale build it once: one compiles, the others wait for it and take what it made
(no GPU; the compilers are stand-ins)."""
import os
import sysconfig
import threading
import time
import types

import pytest

from lossless_bf16_exponent_zc_gb300 import _build


class Compilers:
    """Stands in for subprocess.run: writes the output file slowly, in two halves, and counts who is at it."""

    def __init__(self):
        self.lock, self.writing, self.overlaps, self.runs = threading.Lock(), {}, [], []

    def run(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        for name in cmd:  # what is linked is whole
            if name.endswith(".o") and name != out and os.path.exists(name):
                with open(name) as f:
                    if f.read() != "whole":
                        self.overlaps.append(("read", name))
        with self.lock:
            self.runs.append(out)
            if self.writing.get(out):
                self.overlaps.append(("write", out))
            self.writing[out] = self.writing.get(out, 0) + 1
        with open(out, "w") as f:
            f.write("wh")
            f.flush()
            time.sleep(0.05)
            f.write("ole")
        with self.lock:
            self.writing[out] -= 1
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    c = Compilers()
    monkeypatch.setattr(_build.subprocess, "run", c.run)
    for name, path in (("BUILD", "build"), ("SAN_BUILD", "build/san"), ("LIBDIR", "lib")):
        monkeypatch.setattr(_build, name, str(tmp_path / path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib" / "libzc.so"))
    return c


def together(f, n=4):
    results, errors = [], []

    def work():
        try:
            results.append(f())
        except Exception as e:  # raised again by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    return results


@pytest.mark.parametrize("what", ["build_all", "build_extension", "build"])
def test_one_builds_and_the_others_wait(compilers, what):
    together(getattr(_build, what))
    assert not compilers.overlaps
    objects = [os.path.basename(o) for o in compilers.runs if o.endswith(".o")]
    assert len(objects) == len(set(objects)) == len(_build.SOURCES) + (what != "build")
    assert os.path.exists(_build.LIB) and (what == "build" or os.path.exists(_build.torch_extension_path()))
    before = len(compilers.runs)
    together(getattr(_build, what))  # up to date
    assert len(compilers.runs) == before


def test_a_failed_build_lets_the_next_one_try(compilers, monkeypatch):
    failed = types.SimpleNamespace(returncode=1, stdout="", stderr="no")
    with monkeypatch.context() as m:
        m.setattr(_build.subprocess, "run", lambda *a, **kw: failed)
        with pytest.raises(RuntimeError):
            _build.build_extension()
    assert os.path.exists(_build.build_extension())


def test_the_extension_is_named_for_its_interpreter_and_machine():
    """An extension module loads into one Python on one kind of machine only."""
    assert _build.torch_extension_path().endswith(sysconfig.get_config_var("EXT_SUFFIX"))
