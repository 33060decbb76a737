"""The binding's host extension belongs to the operators of a decode step alone;
the other entry points work without it (no GPU is needed)."""
import pytest
import torch

import gemm_w4a16_gemv_gb300 as w4
from gemm_w4a16_gemv_gb300 import build


@pytest.fixture
def unloaded(monkeypatch):
    build.build()
    monkeypatch.setattr(w4, "_lib", None)
    monkeypatch.setattr(w4, "_fast", None)
    return monkeypatch


@pytest.mark.parametrize("content", [None, b"not a shared object"])
def test_other_entry_points_without_the_extension(unloaded, tmp_path, content):
    path = tmp_path / "_marshal.so"
    if content is not None:
        path.write_bytes(content)
    unloaded.setattr(w4, "_MARSHAL_PATH", str(path))
    assert w4.lib().w4a16_version() == w4.w4a16_version()
    assert w4.kv4_attention_scratch_bytes(16, 8, 256) > 0
    with pytest.raises(RuntimeError, match="_marshal.so.*build"):
        w4.w4a16_sample(torch.zeros(2, 9), torch.zeros(2))
    assert w4.lib() is not None


def test_a_library_that_is_not_built(unloaded, tmp_path):
    unloaded.setattr(w4, "_LIB_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="not built"):
        w4.w4a16_version()
    with pytest.raises(RuntimeError, match="not built"):
        w4.w4a16_sample(torch.zeros(2, 9), torch.zeros(2))


def test_the_library_is_built_where_the_extension_cannot_be(monkeypatch, tmp_path):
    # an extension that fails to compile is reported, after the library is in place
    made = []

    def fails():
        raise RuntimeError("no compiler for the host")

    monkeypatch.setattr(build, "build_marshal", fails)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libw4a16.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):      # (the compiler is not run again for this)
        out = cmd[cmd.index("-o") + 1]
        made.append(out)
        open(out, "wb").close()
        return Done

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no compiler"):
        build.build()
    assert (tmp_path / "libw4a16.so").exists()
    n = len(made)
    with pytest.raises(RuntimeError, match="no compiler"):
        build.build()
    assert len(made) == n    # the library was there: only the extension is tried again
