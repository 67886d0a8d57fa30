"""What the build leaves: a C library that programs link as before, and the binding beside it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_program_linked_by_the_librarys_path_finds_it(minf_lib, tmp_path):
    """No install step and no search path: the path given to the linker is the one the program loads."""
    cc = shutil.which(os.environ.get("CC", "gcc"))
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text('#include <stdio.h>\n#include "minf.h"\nint main(void) { return puts(minf_version()) < 0; }\n')
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), str(src), minf_lib, "-o", str(exe)])
    env = {k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"}
    out = subprocess.run([str(exe)], env=env, cwd=tmp_path, capture_output=True, text=True)
    assert out.returncode == 0 and "sm_100a" in out.stdout, out.stderr
