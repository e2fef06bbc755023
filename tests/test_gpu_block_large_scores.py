"""Scores near the largest ones over the 8-bit caches with one scale per page and head."""
import numpy as np
import pytest
import torch

from block_util import D, DEV, U16, cached_rows, make_cache, randn

pytestmark = pytest.mark.gpu
MODES = ["e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def tied_scores():
    """j1, j2: products 2^28 + 32 j whose exponents, the fp32 product with log2(e) / sqrt(128), are
    a multiple of 8 beyond 2^25, and 8 more."""
    scale = np.float32(np.float32(1.4426950408889634) * np.float32(0.08838834764831845))
    y = [int(np.float32((1 << 28) + 32 * j) * scale) for j in range(64)]
    return next((i, j) for i in range(64) for j in range(64) if y[i] % 8 == 0 and y[i] > 1 << 25 and y[j] == y[i] + 8)


@pytest.mark.parametrize("new", [0, 1], ids=["decode", "few rows"])
def test_largest_scores(new):
    """Scores of 2^25 and more, one token 8 above an earlier one's: no weight leaves fp16."""
    j1, j2 = tied_scores()
    rng = np.random.default_rng(26)
    k, v = torch.zeros(1, 100, D, dtype=torch.float16, device=DEV), randn(rng, 1, 100, D)
    for t, j in ((3, j1), (70, j2)):  # 16-token tiles 0 and 4: one warp's
        k[0, t, 0] = 16384.0
        k[0, t, 1] = j
    c = make_cache(rng, [0], "e4m3", H_q=1, H_kv=1, S=100, R=128)
    c.prefill(0, k, v)
    q = torch.zeros(1, 1, D, dtype=torch.float16, device=DEV)
    q[0, 0, 0], q[0, 0, 1] = 16384.0, 32.0
    if new:
        z = torch.zeros(1, 1, D, dtype=torch.float16, device=DEV)
        out = c.chunk_attn(c.plan([1]), q, z, z)
    else:
        out = c.decode_attn(q)
    # an exponent is off by half a step of 4 each in the products: the later token has 2^4 times the
    # weight of the earlier one at least
    got, a, b = (x.cpu().double().numpy().reshape(D) for x in (out, v[0, 3], v[0, 70]))
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - b) <= np.abs(a - b) / 17 + 4 * U16 * (np.abs(a) + np.abs(b)))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [0, 2, 40])
def test_large_scores_of_like_keys(new, mode):
    """Queries and keys near fp16's largest and keys that are nearly alike: every output lies
    between the values (weights are not negative and sum to 1)."""
    rng = np.random.default_rng(27)
    c = make_cache(rng, [0, 0], mode, H_q=4, H_kv=1, S=20)
    for b, n in enumerate((700, 90)):
        k = randn(rng, 1, 1, D, scale=9000.0).clamp(-60000, 60000).repeat(1, n, 1)
        k[:, :, 5] += randn(rng, 1, n, scale=20.0)
        c.prefill(b, k, randn(rng, 1, n, D))
    for scale in (3.0, 100.0, 9000.0):
        if new:
            q, x = randn(rng, 2 * new, 4, D, scale=scale).clamp(-60000, 60000), randn(rng, 2 * new, 2, D)
            out = c.chunk_attn(c.plan([new, new]), q, x[:, :1], x[:, 1:])
        else:
            out = c.decode_attn(randn(rng, 2, 4, D, scale=scale).clamp(-60000, 60000))
        out = out.cpu().double().numpy()
        for b in range(2):
            _, V = cached_rows(c, b)
            V = V[0] if not new else np.concatenate([V[0], x[new * b: new * b + new, 1].cpu().double().numpy()])
            got = out[b][None] if not new else out[new * b: new * b + new]
            room = 4 * U16 * np.abs(V).max()
            assert np.all(np.isfinite(got)) and np.all((got >= V.min(0) - room) & (got <= V.max(0) + room))
    assert c.read_status() == 0
