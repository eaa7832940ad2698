"""The module of the fast calls is an addition: without it, or without what it
is built with, everything else works (CPU)."""

import os

import pytest
import torch

import exact_attention_47_gb300 as attn
from exact_attention_47_gb300 import _binding, build_lib
from test_rope_kv4_checks import BF, F32, I32, dev, lib, no_library_calls  # noqa: F401


@pytest.fixture
def without_module(monkeypatch, tmp_path, lib):  # noqa: F811
    monkeypatch.setattr(_binding, "fast_path", lambda: str(tmp_path / "absent.so"))
    _binding._fast.cache_clear()
    yield
    _binding._fast.cache_clear()


def test_calls_go_the_python_way_without_the_module(without_module, monkeypatch):
    made = []
    monkeypatch.setattr(_binding, "_call", lambda func, device, *args: made.append(func))
    monkeypatch.setattr(_binding, "_stream_handle", lambda *a: 0)
    T, S, Hq, Hkv, d = 6, 2, 4, 2, 64
    rec = attn.kv4_record_bytes(d, 32)
    q, k, f, pos = dev((2, Hq, 8, d), BF), dev((2, Hkv, 8, d), BF), dev((32,), F32), dev((8,), I32)
    rows = dev((T, Hq, d), BF), dev((T, Hkv, d), BF), dev((T, Hkv, d), BF)
    kv, table, ids, at = dev((9, Hkv, rec), torch.uint8), dev((S, 4), I32), dev((T,), I32), dev((T,), I32)
    with pytest.warns(RuntimeWarning, match="absent.so is not built"):
        attn.rope_fwd(q, k, pos, f, q_out=q, k_out=k)
    attn.rope_bwd(q, k, pos, f, dq=q, dk=k)
    attn.rope_append_paged(*rows, dev((9, Hkv, 16, d), BF), dev((9, Hkv, 16, d), BF), table, ids, at, f, q_out=rows[0])
    attn.rope_append_paged_kv4(*rows, kv, table, ids, at, 32, f, q_out=rows[0])
    attn.kv4_read_paged(kv, table, ids, at, d, 32, rows[1], rows[2])
    need = attn.attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d)
    attn.attn_decode_paged_kv4(dev((S, Hq, d), BF), kv, table, dev((S,), I32), 32, o=dev((S, Hq, d), BF),
                               lse=dev((S, Hq), F32), workspace=dev((need,), torch.uint8))
    assert made == ["rope_fwd", "rope_bwd", "rope_append_paged", "rope_append_paged_kv4", "kv4_read_paged",
                    "attn_decode_paged_kv4"]
    with pytest.raises(ValueError, match="positions of an axis"):
        attn.rope_fwd(q, k, dev((9,), I32), f, q_out=q, k_out=k)


@pytest.mark.parametrize("command,told", [(["/nonexistent/g++"], "nonexistent"), (["false"], "command failed")])
def test_the_library_builds_without_the_module(monkeypatch, tmp_path, capfd, lib, command, told):  # noqa: F811
    """No compiler for it, or one that fails: the library is there, the reason
    is told, and a module from older sources is gone."""
    old = tmp_path / "fast.so"
    old.write_text("older")
    os.utime(old, (0, 0))
    monkeypatch.setattr(build_lib, "fast_path", lambda: str(old))
    monkeypatch.setattr(build_lib, "_fast_command", lambda out: command)
    assert os.path.exists(build_lib.build())
    err = capfd.readouterr().err
    assert "fast calls was not built" in err and told in err and not old.exists()


def test_the_library_builds_without_torch(monkeypatch, capfd, lib):  # noqa: F811
    def absent():
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(build_lib, "_torch", absent)
    assert os.path.exists(build_lib.build())
    assert "No module named 'torch'" in capfd.readouterr().err


def test_the_module_of_another_interpreter_is_not_loaded(monkeypatch, lib):  # noqa: F811
    """Each Python has a file of its own, so another's is as good as none."""
    mine = build_lib.fast_path()
    monkeypatch.setattr(build_lib.sysconfig, "get_config_var", lambda name: ".cpython-399-other.so")
    assert build_lib.fast_path() != mine and not os.path.exists(build_lib.fast_path())
    _binding._fast.cache_clear()
    try:
        with pytest.warns(RuntimeWarning, match="cpython-399-other.so is not built"):
            assert _binding._fast() is _binding._NoFastCalls
    finally:
        _binding._fast.cache_clear()
