"""Paged decode of so few tokens and heads that warps have no items: 16-token and packed tiles
fewer than the warps of a CTA."""
import numpy as np
import pytest

from block_util import D, randn, softmax_rows
from chunk_util import cached_rows, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("H_kv", [1, 2, 3])
@pytest.mark.parametrize("S, lens", [(2, [258]), (16, [300]), (32, [300]), (8, [264]), (2, [1300]), (2, [300, 0, 62, 129]), (0, [5]), (0, [128])], ids=str)
def test_decode(S, lens, H_kv):
    rng = np.random.default_rng(12)
    c = make_cache(rng, lens, S=S, H_q=4 * H_kv, H_kv=H_kv)
    q = randn(rng, len(lens), 4 * H_kv, D)
    out = c.decode_attn(q).cpu().double().numpy()
    for b, n in enumerate(lens):
        if not n:
            continue
        K, V = cached_rows(c, b)
        for h in range(H_kv):
            ref, _, _ = softmax_rows(q[b, 4 * h: 4 * h + 4].cpu().double().numpy(), K[h], V[h])
            assert np.all(np.abs(out[b, 4 * h: 4 * h + 4] - ref) <= 2e-3 + 2e-3 * np.abs(ref)), (b, h)
    assert c.read_status() == 0
