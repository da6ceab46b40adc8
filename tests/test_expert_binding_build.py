"""The expert-layer calls' binding: the library builds, and the calls run,
where it cannot be built."""
import os
import stat
import warnings

import pytest
import torch

from allreduce_sum_residual_gb300 import _build

needs_cuda_torch = pytest.mark.skipif(torch.version.cuda is None, reason="no binding without it")


@needs_cuda_torch
@pytest.mark.parametrize("compiler", ["missing", "failing"])
def test_the_library_builds_without_the_binding(arlib, tmp_path, monkeypatch, compiler):
    cxx = tmp_path / "cxx"
    if compiler == "failing":
        cxx.write_text("#!/bin/sh\necho no Python.h >&2\nexit 1\n")
        cxx.chmod(cxx.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(_build, "CXX", str(cxx))
    monkeypatch.setattr(_build, "BINDING_DIR", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="not built"):
        assert _build.build() == _build.LIB
    assert [f for f in os.listdir(tmp_path) if f != "cxx"] == []
    with pytest.raises((RuntimeError, OSError)):
        _build.build_binding()


@needs_cuda_torch
def test_a_binding_that_is_there_is_kept(arlib, recwarn):
    warnings.simplefilter("always")
    path = _build.build_binding()
    before = os.stat(path).st_mtime_ns
    assert _build.build() == _build.LIB and os.stat(path).st_mtime_ns == before
    assert not [w for w in recwarn if issubclass(w.category, RuntimeWarning)]


@pytest.fixture
def without_binding(arlib, tmp_path, monkeypatch):
    from allreduce_sum_residual_gb300 import experts
    monkeypatch.setattr(_build, "BINDING_DIR", str(tmp_path))
    monkeypatch.setattr(experts, "_native", None)
    monkeypatch.setattr(experts, "_bound_to", None)
    return experts


def test_calls_without_a_binding_go_the_long_way(without_binding):
    x = torch.zeros((4, 64))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        with pytest.raises(ValueError, match="CUDA device"):
            without_binding.ar_route_experts(x, 2)
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # said once
        with pytest.raises(ValueError, match="CUDA device"):
            without_binding.ar_combine(x, x)


@pytest.mark.gpu
def test_results_without_a_binding_are_the_same(arlib, tmp_path, monkeypatch):
    from allreduce_sum_residual_gb300 import experts
    from test_gpu_experts_binding import as_tuple, operands
    calls = operands()
    want = {name: as_tuple(call()) for name, call in calls.items()}
    monkeypatch.setattr(_build, "BINDING_DIR", str(tmp_path))
    monkeypatch.setattr(experts, "_native", None)
    monkeypatch.setattr(experts, "_bound_to", None)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        got = {name: as_tuple(call()) for name, call in calls.items()}
    assert experts._native is experts._LongWay
    for name in calls:
        for a, b in zip(want[name], got[name]):
            assert torch.equal(a, b), name


@needs_cuda_torch
def test_another_python_or_torch_has_a_binding_of_its_own(arlib, monkeypatch):
    """However old its files are: what is compiled against this torch's
    internals is never loaded with another's."""
    import sysconfig
    path = _build.build_binding()
    git = torch.version.git_version or ""
    assert path == _build.binding_path(torch.__version__, git) and os.path.exists(path)
    others = {_build.binding_path("0.0.0+other", git), _build.binding_path(torch.__version__, "0" * 40)}
    monkeypatch.setattr(sysconfig, "get_config_var", lambda _: ".cpython-000-other.so")
    others.add(_build.binding_path(torch.__version__, git))
    assert len(others) == 3 and path not in others
    assert all(os.path.dirname(p) == _build.BINDING_DIR and p.endswith(".so") for p in others)


@needs_cuda_torch
def test_the_binding_of_another_torch_is_not_loaded(arlib, tmp_path, monkeypatch):
    import shutil
    from allreduce_sum_residual_gb300 import experts
    mine = _build.build_binding()
    monkeypatch.setattr(_build, "BINDING_DIR", str(tmp_path))
    monkeypatch.setattr(experts, "_native", None)
    monkeypatch.setattr(experts, "_bound_to", None)
    shutil.copy(mine, _build.binding_path("0.0.0+other", torch.version.git_version or ""))
    shutil.copy(mine, tmp_path / "_binding.so")  # a name without either
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert experts._fast() is experts._LongWay
    shutil.copy(mine, tmp_path)
    monkeypatch.setattr(experts, "_native", None)
    monkeypatch.setattr(experts, "_bound_to", None)
    assert experts._fast() is not experts._LongWay
