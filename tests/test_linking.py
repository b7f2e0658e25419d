"""How programs find liblogmel.so (no GPU)."""
import pathlib
import subprocess
import sys

import pytest

ROOT = pathlib.Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def lib():
    from log_mel_spectrogram_gb300 import build
    return build.build()


def test_a_program_linked_by_path_runs(lib, tmp_path):
    """gcc prog.c /path/liblogmel.so, without an rpath or LD_LIBRARY_PATH."""
    (tmp_path / "p.c").write_text('#include "logmel.h"\nint main(void) { return lm_version() != 100; }\n')
    exe = tmp_path / "p"
    r = subprocess.run(["gcc", "-std=c99", f"-I{ROOT / 'include'}", str(tmp_path / "p.c"), "-o", str(exe), str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, env={})
    assert r.returncode == 0, r.stderr


def test_the_binding_and_the_package_share_one_library(lib):
    """The library is loaded once, whoever loads it first: its tables of devices and its error words are one."""
    code = ("import sys; sys.path.insert(0, %r)\n"
            "from log_mel_spectrogram_gb300 import _native, decode\n"
            "_native.lib(); decode._binding()\n"
            "print({l.split()[4] for l in open('/proc/self/maps') if 'liblogmel' in l})\n" % str(ROOT))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert len(eval(r.stdout)) == 1, r.stdout
