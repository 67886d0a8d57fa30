"""What the build leaves: a C library that programs link as before, and the binding beside it."""
import os
import shutil
import subprocess

import pytest
import torch

from dynamic_sparse_attention_est_b200 import build_lib, minf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_program_linked_by_the_librarys_path_finds_it(minf_lib, tmp_path):
    """No install step and no search path: the path given to the linker is the one the program loads."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text('#include <stdio.h>\n#include "minf.h"\nint main(void) { return puts(minf_version()) < 0; }\n')
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), str(src), minf_lib, "-o", str(exe)])
    env = {k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"}
    out = subprocess.run([str(exe)], env=env, cwd=tmp_path, capture_output=True, text=True)
    assert out.returncode == 0 and "sm_100a" in out.stdout, out.stderr


def test_headers_come_from_the_toolkit_of_nvcc(tmp_path, monkeypatch):
    for part in ("bin", "include"):
        (tmp_path / part).mkdir()
    (tmp_path / "include" / "cuda_runtime_api.h").write_text("")
    (tmp_path / "bin" / "nvcc").write_text("")
    (tmp_path / "bin" / "nvcc").chmod(0o755)
    monkeypatch.setenv("NVCC", str(tmp_path / "bin" / "nvcc"))
    assert build_lib.cuda_include() == str(tmp_path / "include")
    # a link to the compiler, in a place of its own
    link = tmp_path / "elsewhere"
    link.mkdir()
    (link / "nvcc").symlink_to(tmp_path / "bin" / "nvcc")
    monkeypatch.setenv("NVCC", str(link / "nvcc"))
    assert build_lib.cuda_include() == str(tmp_path / "include")


def test_the_library_is_built_where_the_binding_cannot_be(minf_lib, tmp_path, monkeypatch):
    monkeypatch.setattr(build_lib, "binding_path", lambda: str(tmp_path / "_paged.so"))
    monkeypatch.setattr(build_lib, "cxx", lambda: "false")
    with pytest.warns(UserWarning, match="binding"):
        assert build_lib.build() == minf_lib
    monkeypatch.setattr(build_lib, "cxx", lambda: str(tmp_path / "no-such-compiler"))
    with pytest.warns(UserWarning, match="binding"):
        assert build_lib.build() == minf_lib


def test_a_binding_of_another_torch_is_not_loaded(minf_lib, monkeypatch):
    mine = build_lib.binding_path()
    assert os.path.exists(mine)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build_lib.binding_path() != mine and build_lib._binding_stale()
    monkeypatch.setattr(minf, "_paged_module", None)
    with pytest.raises(ImportError, match="build_lib"):
        minf._paged()
