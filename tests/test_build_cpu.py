"""What a build leaves behind: the libraries in the package, and everything that
only the build reads (objects, notes on the torch that a binding was built
against) in the build directory."""
from __future__ import annotations

from dense_tiled_gemm_03_gb300 import build as b


def test_a_bindings_stamps_lie_in_the_build_directory():
    stamps = {b._binding_stamp(), b._ff_stamp()}
    assert len(stamps) == 2
    for stamp in stamps:
        assert stamp.parent == b.BUILD_DIR and stamp.suffix == ".txt"


def test_a_stamp_names_the_torch_it_was_built_against():
    b.build()
    where = b.torch_dir()
    for stamp in (b._binding_stamp(), b._ff_stamp()):
        assert stamp.read_text() == f"{where} {b.torch_version(where)}"
    assert not b.binding_is_stale(where) and not b.ff_binding_is_stale(where)
