"""Few new tokens over long 8-bit caches beside slots of many: two attention kernels in a call."""
import numpy as np
import pytest
import torch

from block_bounds import rows_of, worst
from block_util import D, DEV, cached_rows, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("mode", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [[3, 300, 0, 8, 40, 1], [0, 7, 1, 16, 20, 3], [4, 0, 2, 16, 64, 200]], ids=str)
def test_few_beside_wide(new, mode):
    """8 heads of two slots of 66 000 tokens are 8192 tiles of 128 and more: slots of up to 16 and of
    up to 32 rows a key head run in a launch of their own, in parts that are joined, and so do
    the other slots, whole and in ranges that are cut; the workspace serves both.  With half as
    many (the second case) one launch serves all.  Infinite and NaN values reach the rows that
    see them."""
    rng = np.random.default_rng(sum(new))
    lens = [66000, 500, 100, 66100, 2000, 0]
    c = make_cache(rng, lens, mode, H_q=16, H_kv=8, G=128, max_T=66304, S=2, spare=16)
    tiles = 8 * sum(c.lengths(b)["T"] // 128 for b in range(6) if 0 < 2 * new[b] <= 32)
    assert tiles >= 8192 if new[0] else tiles < 5120
    n = sum(new)
    x = randn(rng, n, 32, D)
    q, k, v = x[:, :16], x[:, 16:24], x[:, 24:]
    v[0, 0, 5] = float("inf")
    v[n - 1, 1, 7] = float("nan")
    c.view("v_res")[3, 2, 1, 9] = -float("inf")
    ch = c.plan(new)
    out = torch.full((n + 2, 16, D), 7.0, dtype=torch.float16, device=DEV)
    c.chunk_attn(ch, q, k, v, out=out)
    again = c.chunk_attn(ch, q, k, v)
    assert torch.equal(out[:n].view(torch.int16), again.view(torch.int16)) and bool((out[n:] == 7.0).all())
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.chunk_attn(ch, q, k, v, out=again)
    for _ in range(2):
        again.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:n].view(torch.int16), again.view(torch.int16))
    got, qd, k, v = (x.cpu().double().numpy() for x in (again, q, k, v))
    at = 0
    for b, m in enumerate(new):
        if not m:
            continue
        K, V = cached_rows(c, b)
        L = K.shape[1]
        hid = np.arange(L + m)[None, :] > L + np.arange(m)[:, None]
        for h in range(8):
            Kh = np.concatenate([K[h], k[at:at + m, h]])
            Vh = np.concatenate([V[h], v[at:at + m, h]])
            odd = np.nonzero(~np.isfinite(Vh))
            Vf = np.where(np.isfinite(Vh), Vh, 0.0)
            for j in (2 * h, 2 * h + 1):
                p, ref, mag = rows_of(qd[at:at + m, j], Kh, Vf, hid)
                bound = worst(p, Vf, ref, mag)
                for t, d in zip(*odd):
                    ref[~hid[:, t], d] += Vh[t, d]
                y, fin = got[at:at + m, j], np.isfinite(ref)
                assert np.array_equal(np.isnan(y), np.isnan(ref)) and np.array_equal(y[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
                err = np.where(fin, np.abs(np.where(fin, y, 0.0) - np.where(fin, ref, 0.0)), 0.0)
                assert np.all(err <= bound), "slot %d head %d: %g of its bound" % (b, j, (err / bound).max())
        at += m
    assert c.read_status() == 0
