"""What the copy of rows that the TMA cannot address reads (csrc/ff_pad.h, the
arithmetic of the kernel itself, compiled for the CPU): for every piece of the
copy, loads that lie within the source's own 16-byte pieces, and from them the
row's elements and no others."""
from __future__ import annotations

import ctypes
import subprocess

import pytest

from dense_tiled_gemm_03_gb300 import build as native_build

DRIVER = """
#include "ff_pad.h"
extern "C" long long pitch(long long cols) { return gemm_tn_dev::ff::pad_pitch(cols); }
extern "C" void piece(unsigned long long row, long long cols, long long col, long long* out) {
  const gemm_tn_dev::ff::PadPiece p = gemm_tn_dev::ff::pad_piece(row, cols, col);
  out[0] = p.valid > 0 ? p.valid : 0;
  out[1] = p.shift;
  out[2] = p.first ? static_cast<long long>(p.at) : 0;
  out[3] = p.second ? static_cast<long long>(p.at) + 16 : 0;
}
"""


@pytest.fixture(scope="module")
def pad(tmp_path_factory):
    where = tmp_path_factory.mktemp("pad")
    (where / "driver.cpp").write_text(DRIVER)
    so = where / "driver.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", str(native_build.CSRC),
                    str(where / "driver.cpp"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.pitch.restype = ctypes.c_longlong
    lib.pitch.argtypes = [ctypes.c_longlong]
    lib.piece.argtypes = [ctypes.c_ulonglong, ctypes.c_longlong, ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)]
    return lib


def pieces(pad, row, cols):
    """(column, valid, shift, lo, hi) of every piece of a row's copy."""
    out = (ctypes.c_longlong * 4)()
    for col in range(0, pad.pitch(cols), 8):
        pad.piece(row, cols, col, out)
        yield col, *out


COLUMNS = [*range(1, 200), 1000, 1015, 4095, 4097, (1 << 30) - 1]


def test_rows_of_the_copy_hold_the_row_and_can_be_addressed(pad):
    for cols in COLUMNS:
        assert pad.pitch(cols) >= cols and pad.pitch(cols) % 8 == 0


@pytest.mark.parametrize("start", range(0, 16, 2))
def test_no_load_leaves_the_row(pad, start):
    """A row may be the last of its storage, which may end with its mapping: a load reads only aligned 16-byte pieces
    that hold an element of the row."""
    row = 0x7F0000000000 + start
    for cols in COLUMNS[:-1]:
        first, end = row, row + 2 * cols
        for col, valid, shift, lo, hi in pieces(pad, row, cols):
            for at in (lo, hi):
                assert at == 0 or (at % 16 == 0 and at < end and at + 16 > first), (cols, col, at - row)


@pytest.mark.parametrize("start", range(0, 16, 2))
def test_the_loads_hold_the_pieces_elements(pad, start):
    row = 0x7F0000000000 + start
    for cols in COLUMNS[:-1]:
        for col, valid, shift, lo, hi in pieces(pad, row, cols):
            assert valid == max(0, min(8, cols - col))
            if valid == 0:
                continue
            assert lo + shift == row + 2 * col and 0 <= shift < 16
            assert hi in (0, lo + 16)
            assert lo + (32 if hi else 16) >= row + 2 * (col + valid)


def test_the_copy_of_narrow_rows_stays_small(pad):
    """At most twice what rows of whole 16-byte pieces take, whatever the width."""
    for cols in COLUMNS:
        assert pad.pitch(cols) <= 2 * ((cols + 7) // 8 * 8), cols
