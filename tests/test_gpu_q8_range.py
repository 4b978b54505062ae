"""The 8-bit cache's attention where blocks of slots, scores and rows lie far apart, against 64 bits."""

import numpy as np
import pytest

import q8_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import looped_transformer_kv_gb300 as rq  # noqa: F401
    from test_gpu_q8 import MARK, Case, fill_cache


@pytest.mark.parametrize("B,n,longest", [(60, 40, 600), (60, 100, 2500), (60, 300, 900), (12, 300, 6000)])
def test_row_tiles_without_rows(B, n, longest):
    """Many units of which one row tile has no rows: a CTA walks several, some in turn with full ones, and
    neither runs ahead of the other tile's products nor falls behind them."""
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, longest, B)
    ctx[7] = longest
    c = Case(B, 4, 4, 64, "int8", ctx.tolist(), n, rng.integers(0, n + 1, B).tolist(), fill=False)
    fill_cache(c)
    c.append()
    for _ in range(3):
        c.out.fill_(MARK)
        c.attend()
    c.check()
