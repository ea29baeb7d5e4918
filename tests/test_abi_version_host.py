"""The options' layout belongs to the library's minor version: header, library and binding agree on both, and the binding
takes no library of another one."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

L = pytest.importorskip("gated_deltanet_recurrence_03_gb300._lib")


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_03_gb300 import build
    build.build()
    return L.load()


def compile_c(tmp_path, text, *args):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, out = tmp_path / "a.c", tmp_path / "a.out"
    src.write_text(text)
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(out), *args])
    return str(out)


def test_header_library_and_binding_are_of_one_version_and_layout(lib, tmp_path):
    names = [n for n, _ in L.GdnOpts._fields_]
    prints = "".join(f'printf("%zu\\n", offsetof(gdn_opts_t, {n}));' for n in names)
    exe = compile_c(tmp_path, '#include <stdio.h>\n#include "gdn.h"\n'
                    f'int main(void) {{ printf("%d\\n%zu\\n", GDN_VERSION, sizeof(gdn_opts_t)); {prints} return 0; }}')
    version, size, *offsets = map(int, subprocess.check_output([exe]).split())
    assert version == lib.gdn_version() == L.VERSION
    assert size == ctypes.sizeof(L.GdnOpts) and offsets == [getattr(L.GdnOpts, n).offset for n in names]


def test_the_version_that_grew_the_options_is_another_one(lib):
    """The options of 0.3 end before conv_bias: a caller of that version must be able to tell."""
    assert L.GdnOpts.conv_bias.offset == 128 and lib.gdn_version() // 100 > 3


@pytest.mark.parametrize("version,taken", [(300, False), (L.VERSION + 100, False), (L.VERSION + 10000, False), (L.VERSION + 1, True)])
def test_the_binding_takes_its_own_minor_version_alone(version, taken, tmp_path):
    path = compile_c(tmp_path, f"int gdn_version(void) {{ return {version}; }}", "-shared", "-fPIC")
    # a library of the right version goes on to its entry points, of which this one has none
    with pytest.raises(AttributeError if taken else ImportError, match="gdn_opts_init" if taken else "version"):
        L.load(path)
