"""Pages of the 8-bit caches whose keys are all infinite in a channel."""
import numpy as np
import pytest

from block_util import D, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("new", [0, 2, 40])
def test_every_key_of_a_page_infinite(new):
    """int8: such a page counts as NaN, whatever the signs of queries and codes."""
    rng = np.random.default_rng(28)
    c = make_cache(rng, [0], "int8", H_q=4, H_kv=1)
    k, v = randn(rng, 1, 200, D), randn(rng, 1, 200, D)
    k[0, 64:128, 7] = float("inf")
    c.prefill(0, k, v)
    for sign in (1.0, -1.0):
        q = randn(rng, max(new, 1), 4, D)
        q[..., 7] = sign
        x = randn(rng, max(new, 1), 2, D)
        out = c.chunk_attn(c.plan([new]), q, x[:, :1], x[:, 1:]) if new else c.decode_attn(q)
        assert bool(out.isnan().all())
    assert c.read_status() == 0
