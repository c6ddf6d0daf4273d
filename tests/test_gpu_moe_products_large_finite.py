"""The products past 2^31 elements once more, with a comparison that no NaN
passes: memory that is read or left unwritten by mistake shows as one."""
import pytest

import test_gpu_moe_products_large as large

pytestmark = pytest.mark.gpu


def near(got, want, size, terms, what):
    bad = ~((got.double() - want).abs() <= large.HALF * want.abs() + terms * large.SUM * size + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(large, "near", near)


@pytest.mark.parametrize("width", [4096, 4095])
def test_long_batches(width):
    large.test_long_batches(width)


def test_wide_results():
    large.test_wide_results()


@pytest.mark.parametrize("per,width", [(4, 4096), (70, 4096), (4, 4095)])
def test_many_large_experts(per, width):
    large.test_many_large_experts(per, width)
