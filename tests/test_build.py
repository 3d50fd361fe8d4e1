"""The build: libqg.so does not depend on the module of the decoder-layer calls, which is built for one torch."""
import os
import shutil

import pytest


@pytest.fixture()
def small(tmp_path, monkeypatch):
    """The build with one small translation unit in a folder of its own."""
    from gguf_block_quantized_quant_gb300 import build as b
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("no nvcc")
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int qg_version() { return 1; }\n')
    out = tmp_path / "out"
    monkeypatch.setattr(b, "OUT_DIR", str(out))
    monkeypatch.setattr(b, "LIB", str(out / "libqg.so"))
    monkeypatch.setattr(b, "TORCH_MODULE", str(out / "qg_torch.so"))
    monkeypatch.setattr(b, "TORCH_STAMP", str(out / "qg_torch.so.for"), raising=False)
    monkeypatch.setattr(b, "_units", lambda: [(str(src), str(out / "one.o"), [])])
    monkeypatch.setattr(b, "_torch_commands", lambda tmp: (["true"], ["cp", str(src), tmp]))
    return b


def test_library_is_built_where_the_module_cannot_be(small, monkeypatch):
    for step in (0, 1):
        commands = [["true"], ["true"]]
        commands[step] = ["sh", "-c", "echo no such header >&2; exit 1"]
        monkeypatch.setattr(small, "_torch_commands", lambda tmp: commands)
        with pytest.warns(UserWarning, match="no such header"):
            assert small.build(force=True) == small.LIB
        assert os.path.exists(small.LIB) and not os.path.exists(small.TORCH_MODULE)
        assert small.module_is_for() is None and not small.up_to_date()


def test_module_is_built_again_for_another_torch(small, monkeypatch):
    small.build()
    assert small.up_to_date()
    before = os.path.getmtime(small.LIB)
    monkeypatch.setattr(small, "_torch_id", lambda: "torch of another day")
    assert not small.up_to_date()
    small.build()
    assert small.up_to_date() and small.module_is_for() == "torch of another day"
    assert os.path.getmtime(small.LIB) == before  # the library knows nothing of torch
    os.remove(small.TORCH_MODULE)
    assert small.module_is_for() is None


def test_calls_say_that_their_module_is_missing(monkeypatch):
    import gguf_block_quantized_quant_gb300 as qg
    from gguf_block_quantized_quant_gb300 import build as b
    b.build()
    monkeypatch.setattr(qg, "_module", None)
    for built_for, word in ((None, "missing"), ("torch 0", "torch 0")):
        monkeypatch.setattr(b, "module_is_for", lambda: built_for)
        with pytest.raises(RuntimeError, match=word):
            qg.qg_norm_residual(None, None, None)


def test_a_library_that_does_not_compile_is_an_error(small, tmp_path):
    (tmp_path / "one.cu").write_text("no such thing\n")
    with pytest.raises(RuntimeError, match="nvcc"):
        small.build()
