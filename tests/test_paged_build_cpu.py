"""When the torch side of the paged operators counts as built, and what a build
leaves behind without it."""

import os

import pytest

from speculative_prefill_token_gb300 import _build, paged


def test_a_torch_side_of_another_torch_is_built_again_and_not_loaded(tmp_path, monkeypatch):
    _build.build()
    assert _build.up_to_date() and _build.torch_side_fits()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(_build, "TORCH_STAMP", str(stamp))
    monkeypatch.setattr(paged, "_side", None)
    for text in (None, "", _build.torch_stamp() + " ", "torch 2.0.0 cxx11_abi 0 cpython-38"):
        if text is not None:
            stamp.write_text(text)
        assert not _build.up_to_date() and not _build.torch_side_fits()
        with pytest.raises(RuntimeError, match="not built for this torch"):
            paged.torch_side()
    stamp.write_text(_build.torch_stamp())
    assert _build.up_to_date() and _build.torch_side_fits()
    paged.torch_side()


def _fake(tmp_path, monkeypatch, fails=()):
    """A build into tmp_path whose commands only leave their outputs."""
    ran = []

    def run(cmd, verbose, what):
        ran.append(os.path.basename(cmd[0]))
        if ran[-1] in fails:
            raise RuntimeError(f"{cmd[0]} failed")
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(_build, "_run", run)
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    for name in ("LIB", "TORCH_LIB", "TORCH_STAMP"):
        monkeypatch.setattr(_build, name, str(tmp_path / name))
    return ran


def test_without_torch_the_library_is_built_alone(tmp_path, monkeypatch):
    ran = _fake(tmp_path, monkeypatch)
    monkeypatch.setattr(_build, "torch_stamp", lambda: None)
    assert not _build.up_to_date()
    assert os.path.exists(_build.build()) and not os.path.exists(_build.TORCH_LIB)
    assert _build.up_to_date() and "g++" not in ran


def test_the_library_is_in_place_when_the_torch_side_fails(tmp_path, monkeypatch):
    _fake(tmp_path, monkeypatch, fails=("g++",))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.TORCH_LIB) and not _build.up_to_date()


def test_only_what_is_old_is_built(tmp_path, monkeypatch):
    ran = _fake(tmp_path, monkeypatch)
    _build.build()
    assert _build.up_to_date() and ran.count("nvcc") == len(_build.SOURCES) + 1 and ran.count("g++") == 2
    ran.clear()
    _build.build()
    assert not ran
    open(_build.TORCH_STAMP, "w").close()
    _build.build()
    assert ran == ["g++", "g++"] and _build.up_to_date()
