"""The orthogonalisation's accuracy on every tile size, half tiles, split sums
and several bands of tiles, on matrices where the parts beside f16 show: a few
large directions over a small floor, whose error is five times larger without
X's low part, and gradients of tokens."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq
from test_gpu_muon import update

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# The rounding of the output to bf16 is 1.67e-3 of the 2-norm (half an ulp of
# 2^-8 to 2^-7 relative, uniform).  The operands' formats add at most 6.6e-4
# on these inputs (host simulation with f16 + e4m3 parts and fp32 diagonals,
# 64 x 2048 to 1536 x 2000), independent of it: sqrt(1.67^2 + 0.66^2) =
# 1.80e-3, and a tenth for the spread.  Without X's low part the
# first kind comes to 8.7e-3 to 9.9e-3; without the diagonals the second comes
# to 1.9e-3 to 2.7e-3.
BOUND = 2e-3


def reference(g):
    a, b, c = mxq.MUON_COEFFICIENTS
    out = []
    for m in g.to(DEV):
        x = m.double()
        x = (x.t() if x.shape[0] > x.shape[1] else x).contiguous()
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        for _ in range(5):
            s = x @ x.t().contiguous()
            x = a * x + (b * s + c * (s @ s)) @ x
        out.append(x.t() if m.shape[0] > m.shape[1] else x)
    return torch.stack(out)


def check(g, bound=BOUND):
    got, want = mxq.muon_orthogonalize(g.to(DEV)).double(), reference(g)
    e = torch.linalg.vector_norm(got - want, dim=(1, 2)) / torch.linalg.vector_norm(want, dim=(1, 2))
    assert (e <= bound).all(), e.max()  # NaN fails too


# 64 x 64 tiles; 128 x 64; 256 x 256 with the symmetric products as halves, and with a last round of halves
TILES = [(2, 130, 260), (1, 400, 400), (44, 250, 380), (48, 380, 250), (20, 760, 1000), (24, 1000, 765)]
# sums in parts: of 64 x 64 tiles, of 128 x 64 and of 256 x 256
SPLITS = [(1, 64, 2048), (3, 175, 7481), (2, 5000, 130), (1, 1000, 8100), (9, 1024, 4100)]
# 256 x 256 tiles in more than one band of eight row tiles
BANDS = [(1, 2300, 2600), (1, 5200, 2310)]


@pytest.mark.parametrize("shape", TILES + SPLITS + BANDS)
def test_few_directions_over_a_floor(shape):
    check(update(*shape, torch.bfloat16, 21, "lowrank"))


@pytest.mark.parametrize("shape", TILES + SPLITS[:3])
def test_gradients_of_tokens(shape):
    check(update(*shape, torch.bfloat16, 22, "tokens"))


@pytest.mark.parametrize("shape", BANDS)
def test_close_singular_values_in_several_bands(shape):
    check(update(*shape, torch.bfloat16, 23, "gauss"))


# Equal rows: the diagonals no longer hold the large entries.  The formats
# simulated on the host give up to 7.2e-3 (rows that come 32 times) with the
# output's rounding; a quarter more for the spread.
EQUAL_ROWS = 9e-3


@pytest.mark.parametrize("copies", [2, 32])
@pytest.mark.parametrize("shape", [(64, 2048), (250, 380), (2300, 2600)])
def test_rows_that_repeat(shape, copies):
    r, k = shape
    g = update(1, -(-r // copies), k, torch.bfloat16, 5, "tokens")
    check(g.repeat(1, copies, 1)[:, :r], EQUAL_ROWS)
