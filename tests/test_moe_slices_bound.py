"""Host check of the workspace of the bias gradient's sums: a slice of 16 or 64
rows of a group has a row of `wide` floats there.  For group ends that do not
decrease, the rows behind the last group counted as one, the slices never exceed
the space that the library asks for; ends that decrease pass it many times over,
and the kernels, which count the slices on the device, stop at the number that
the space was made for."""
import numpy as np
import pytest

from mxfp8_quantization_moe_amd import _capi, build

WIDE = 64  # a multiple of 64 floats: no rounding in the sizes


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return _capi.load()


def room(lib, rows, E, wide=WIDE):
    """Slices that the workspace of the sums holds."""
    need = [lib.mxq_moe_linear_backward_workspace_bytes(rows, 8, E, wide, 0, 0, bias, 1) for bias in (0, 1)]
    assert (need[1] - need[0]) % (4 * wide) == 0
    return (need[1] - need[0]) // (4 * wide)


def slices(offs, rows, slice):
    """Of every group and of the rows behind the last one, as a kernel counts them."""
    ends = np.clip(np.asarray(offs, dtype=np.int64), 0, rows)
    starts = np.concatenate([[0], ends])
    return int(((np.maximum(np.concatenate([ends, [rows]]) - starts, 0) + slice - 1) // slice).sum())


def slice_of(rows, E, n):
    """16 rows where 64 would leave less than four workgroups per CU."""
    tiles = -(-rows // 64) if E == 1 else rows // 64 + E // 2 if 2 * rows >= E * 64 else min(E, rows)
    return 16 if tiles * -(-n // 512) < 4 * 256 else 64


@pytest.mark.parametrize("E", [1, 2, 7, 64, 300, 4096])
def test_ends_that_do_not_decrease_fit(lib, E):
    rng = np.random.default_rng(E)
    for rows in (1, 2, 15, 16, 17, 63, 64, 65, 1000, 4097, 70000):
        s = slice_of(rows, E, WIDE)
        most = room(lib, rows, E)
        cases = [np.full(E, rows), np.zeros(E), np.minimum(np.arange(1, E + 1), rows), np.minimum(np.arange(1, E + 1) * (s + 1), rows)]
        cases += [np.sort(rng.integers(0, rows + 1, E)) for _ in range(200)]
        cases += [np.sort(rng.integers(-5, rows + 9, E)) for _ in range(50)]
        assert max(slices(c, rows, s) for c in cases) <= most, rows


def test_the_largest_slices(lib):
    """Slices of 64 rows, and the bound is reached: every group one row past a slice."""
    rows, E, wide = 8192, 64, 4096
    assert slice_of(rows, E, wide) == 64
    most = room(lib, rows, E, wide)
    assert most == rows // 64 + E
    short = np.cumsum(np.full(E, 65))
    assert slices(short, rows, 64) == 2 * E + -(-(rows - 65 * E) // 64) <= most
    assert room(lib, 40, 64) == 40 == slices(np.arange(1, 65), 40, 16)


def test_ends_that_decrease_do_not(lib):
    rows, E = 1000, 64
    offs = [rows, 0] * (E // 2)
    assert slice_of(rows, E, WIDE) == 16
    # 32 groups of all rows, and all of them behind the last end, 63 slices each
    assert slices(offs, rows, 16) == 33 * 63 > 16 * room(lib, rows, E)
