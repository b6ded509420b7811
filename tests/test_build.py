"""What the build needs, and when it builds again (nothing is compiled here
beyond what is out of date anyway)."""
import os
import subprocess
import sys

import pytest

from chunk_gated_delta_02_b200 import build as cbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def nowhere(tmp_path, monkeypatch):
    """The library up to date, the binding not built yet."""
    cbuild.build()
    monkeypatch.setattr(cbuild, "BINDING", str(tmp_path / "_mixer.so"))
    monkeypatch.setattr(cbuild, "BINDING_MADE", str(tmp_path / "_mixer.txt"), raising=False)
    return tmp_path


def test_library_without_a_cxx_compiler(nowhere, monkeypatch, capsys):
    monkeypatch.setattr(cbuild, "CXX", str(nowhere / "no-such-compiler"))
    assert cbuild.build() == cbuild.LIB and os.path.exists(cbuild.LIB)
    assert "no-such-compiler" in capsys.readouterr().err
    assert not os.path.exists(cbuild.BINDING)


def test_library_without_torch(nowhere):
    """-S: an interpreter without its installed packages."""
    code = ("import sys; sys.path.insert(0, %r)\n"
            "from chunk_gated_delta_02_b200 import build\n"
            "build.BINDING = %r\n"
            "assert build.build() == build.LIB" % (ROOT, cbuild.BINDING))
    r = subprocess.run([sys.executable, "-S", "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "torch" in r.stderr and not os.path.exists(cbuild.BINDING)


def test_a_failing_compiler_is_an_error(nowhere, monkeypatch):
    monkeypatch.setattr(cbuild, "_binding_command", lambda out: ["false"])
    with pytest.raises(subprocess.CalledProcessError):
        cbuild.build()


def test_binding_is_rebuilt_for_another_torch(nowhere, monkeypatch):
    made = []

    def command(out):
        made.append(out)
        return ["touch", out]

    monkeypatch.setattr(cbuild, "_binding_command", command)
    cbuild.build()
    cbuild.build()
    assert len(made) == 1
    monkeypatch.setattr(cbuild.importlib.metadata, "version", lambda name: "0.0.1")
    cbuild.build()
    cbuild.build()
    assert len(made) == 2
