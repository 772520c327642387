"""The order of the build: the library, which takes hipcc alone, does not wait for
the Python binding of the decoder operators.  The compilers are stand-ins here."""

import os

import pytest

from q4_weight_only_amd import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into tmp_path whose commands write their output files; `fail` is
    the part of a command line that makes one fail."""
    for name in ("BUILD_DIR", "LIB", "BINDING"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    monkeypatch.setattr(B, "BUILD_INFO", str(tmp_path / "build_info.json"))
    monkeypatch.setattr(B, "_hipcc", lambda: "/opt/rocm/bin/hipcc")
    state = {"fail": None, "ran": []}

    def run(cmd):
        state["ran"].append(cmd)
        if state["fail"] and any(state["fail"] in part for part in cmd):
            raise RuntimeError(f"command failed (1): {' '.join(cmd)}")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return ""

    monkeypatch.setattr(B, "_run", run)
    return state


def test_both_are_built(tree):
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.BINDING)


@pytest.mark.parametrize("fail", ["decoder_binding.cpp", "decoder_binding.o"])
def test_library_is_there_where_the_binding_cannot_be_compiled_or_linked(tree, fail):
    with open(B.BINDING, "w") as f:
        f.write("an older build's")
    tree["fail"] = fail
    with pytest.raises(RuntimeError, match="is built .* binding is not"):
        B.build()
    assert os.path.exists(B.LIB)
    assert not os.path.exists(B.BINDING)


def test_library_is_there_without_torch(tree, monkeypatch):
    def no_torch(out):
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(B, "_binding_command", no_torch)
    with pytest.raises(RuntimeError, match="is built"):
        B.build()
    assert os.path.exists(B.LIB)


def test_library_alone(tree, monkeypatch):
    monkeypatch.setattr(B, "_binding_command", lambda out: pytest.fail("not asked for"))
    assert B.build(binding=False) == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_a_source_that_does_not_compile_leaves_the_library_alone(tree):
    with open(B.LIB, "w") as f:
        f.write("an older build's")
    tree["fail"] = "q4_logits.hip"
    with pytest.raises(RuntimeError, match="command failed"):
        B.build()
    assert open(B.LIB).read() == "an older build's"
