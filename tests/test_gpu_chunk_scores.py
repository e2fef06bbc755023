"""The chunk attention's softmax over the whole range of scores: references that move along
the keys, and scores as large as fp16 queries and keys can make them, against float64."""
import math

import numpy as np
import pytest
import torch

from chunk_util import DEV, U16, cached_rows, randn

pytestmark = pytest.mark.gpu
D = 128

# Forms of a unit: (slots' cached tokens, new tokens, query heads, key heads)
FORMS = {
    "wide": ([2500], [100], 8, 2),                   # 400 rows: a whole row tile and a partial one
    "wide_second_half": ([700], [40], 4, 1),         # 160 rows
    "narrow": ([2900], [25], 8, 2),                  # 100 rows, cut into parts
    "two_copies": ([3100], [12], 8, 2),              # 48 rows, cut
    "four_copies": ([3000], [4], 8, 2),              # 16 rows, cut
    "many_units": ([1500] * 20, [4] * 20, 8, 8),     # more units than ranges: some whole, some cut
    "first_chunk": ([0], [300], 4, 1),               # fp16 rows alone
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def filled(rng, form, level, rest):
    """A cache and a chunk of a form.  Channel 0 of the keys holds level(position), constant
    over each page of 128 tokens (a group of equal values is held exactly); the other channels
    are normal values times `rest`.  Returns the cache, the counts, k and v of the chunk."""
    import bit_kv_cache_gb300 as kvq
    lens, new, H_q, H = FORMS[form]
    c = kvq.KVQPagedCache(len(lens), H_q, H, D, 128, 2, n_pages=sum(n // 128 for n in lens) + 8, max_T=4096, device=DEV)
    ks, vs = [], []
    for b, (L, n) in enumerate(zip(lens, new)):
        k, v = randn(rng, H, L + n, D, scale=rest), randn(rng, H, L + n, D)
        pos = np.arange(L + n)
        pos[: L // 128 * 128] = pos[: L // 128 * 128] // 128 * 128
        k[..., 0] = torch.from_numpy(level(pos).astype(np.float16)).to(DEV)
        if L:
            c.prefill(b, k[:, :L].contiguous(), v[:, :L].contiguous())
        ks.append(k[:, L:].transpose(0, 1))
        vs.append(v[:, L:].transpose(0, 1))
    return c, new, torch.cat(ks).contiguous(), torch.cat(vs).contiguous()


def check(c, new, q, k, v, out):
    """Against softmax in float64.  Channel 0 of every key is exact, and so are its products.
    The error of a score: the rounding of the other channels' packed keys to fp16 (U16 of each
    product), and fp32 sums of 128 products formed 16 at a time (8 roundings or truncations of
    2^-23 each: 2^-20 of the sum of magnitudes).  Of a weight, relative: that, and 2^-14 for
    the exponent, its reference and its hardware approximation (a multiple of 2^-15 in log2
    units below 2^10, 2^-22 for the approximation), in the weight and in the sum; U16 for the
    weight's and U16 for the packed value's rounding; the output's own U16.  Weights 2^-20
    below the reference are off by 2^-25 of 2^6 at most: 3e-8 a key."""
    g = c.cfg.H_q // c.cfg.H_kv
    q, k, v, out = (x.detach().cpu().double().numpy() for x in (q, k, v, out))
    at = 0
    for b, n in enumerate(new):
        K, V = cached_rows(c, b)
        L, T = K.shape[1], c.lengths(b)["T"]
        K = np.concatenate([K, k[at:at + n].transpose(1, 0, 2)], 1)
        V = np.concatenate([V, v[at:at + n].transpose(1, 0, 2)], 1)
        hid = np.arange(L + n)[None, :] > L + np.arange(n)[:, None]
        for h in range(c.cfg.H_q):
            Kh, Vh, qh = K[h // g], V[h // g], q[at:at + n, h]
            s = np.where(hid, -np.inf, (qh @ Kh.T) / math.sqrt(D))
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            ref, size = p @ Vh, p @ np.abs(Vh)
            rest = np.abs(qh[:, 1:]) @ np.abs(Kh[:, 1:]).T / math.sqrt(D)
            one = np.abs(qh[:, :1]) @ np.abs(Kh[:, :1]).T / math.sqrt(D)
            # exact sums, where channel 0 is all there is, have no rounding
            ds = U16 * rest[:, :T].max(1, initial=0.0) + np.where(hid | (rest == 0), 0.0, (rest + one) * 2.0 ** -20).max(1)
            bound = size * (2 * (ds[:, None] + 2.0 ** -14) + 3 * U16) + U16 * np.abs(ref) + 3e-8 * (L + n) * np.abs(Vh).max()
            err = np.abs(out[at:at + n, h] - ref)
            assert np.isfinite(out[at:at + n, h]).all(), "slot %d head %d" % (b, h)
            i = np.unravel_index(np.argmax(err - bound), err.shape)
            assert np.all(err <= bound), "slot %d head %d row %d channel %d: %g, bound %g" % (b, h, i[0], i[1], err[i], bound[i])
        at += n


LEVELS = {
    "rising": lambda t: 11.0 * (t // 128),                       # about 4 nats a page
    "rising_in_tiles": lambda t: 6.0 * (t // 64),
    "falling": lambda t: 300.0 - 11.0 * (t // 128),
    "jumps": lambda t: 37.0 * ((t // 128) * 7 % 5) + 2.0 * (t // 128),
}


@pytest.mark.parametrize("levels", list(LEVELS))
@pytest.mark.parametrize("form", list(FORMS))
def test_reference_moves(form, levels):
    """Scores that rise along the sequence move a row's reference again and again, and each
    move rescales what it has summed."""
    rng = np.random.default_rng(len(form) + len(levels))
    c, new, k, v = filled(rng, form, LEVELS[levels], 1.0)
    q = randn(rng, sum(new), c.cfg.H_q, D, scale=0.25)
    q[..., 0] = 4.0
    out = c.chunk_attn(c.plan(new), q, k, v)
    check(c, new, q, k, v, out)
    assert c.read_status() == 0


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("form", list(FORMS))
def test_largest_scores(form, sign):
    """|q . k| up to 4.3e9, among them products whose scaled value lies up to 31 from the
    nearest fp32 number: differences of scores are exact, equal ones share their weight."""
    rng = np.random.default_rng(len(form))
    top = np.array([100.0, 64896.0, 9000.0, 65248.0, -64960.0, 65248.0, 64544.0, 1.0])

    def level(t):
        return sign * np.where(t % 128 < 64, top[t // 128 % 8], top[(t // 128 + t // 3) % 8])

    c, new, k, v = filled(rng, form, level, 0.0)
    q = torch.zeros(sum(new), c.cfg.H_q, D, dtype=torch.float16, device=DEV)
    scale = torch.tensor([65504.0, 65472.0, -65504.0, 3000.0, 1.0, 0.0, 2.0 ** -12, 59008.0], dtype=torch.float16, device=DEV)
    q[..., 0] = scale[torch.arange(q.shape[0] * q.shape[1], device=DEV).view(q.shape[:2]) % 8]
    out = c.chunk_attn(c.plan(new), q, k, v)
    check(c, new, q, k, v, out)
    assert c.read_status() == 0


@pytest.mark.parametrize("cached", [1300, 2000, 3100])
@pytest.mark.parametrize("new", [3, 12, 25, 90])
def test_infinite_value_under_a_small_weight(new, cached):
    """A weight is positive however small: an infinite value of a key far below the others makes
    the output infinite, whole or joined from parts."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(new)
    H, S = 2, 256
    c = kvq.KVQPagedCache(1, 8, H, D, 128, 2, n_pages=40, max_T=4096, S=S, device=DEV)
    k, v = randn(rng, H, cached, D, scale=0.25), randn(rng, H, cached, D)
    k[:, :, 0], k[:, :S, 0] = 500.0, 0.0                 # 177 below the others
    v[0, 7, 3], v[0, 200, 4], v[1, 255, 5] = float("inf"), float("-inf"), float("inf")
    c.prefill(0, k, v)
    q = randn(rng, new, 8, D, scale=0.25)
    q[..., 0] = 4.0
    kn, vn = randn(rng, new, H, D, scale=0.25), randn(rng, new, H, D)
    kn[..., 0] = 500.0
    out = c.chunk_attn(c.plan([new]), q, kn, vn).float()
    want = torch.zeros(new, 8, D, device=DEV)
    want[:, :4, 3], want[:, :4, 4], want[:, 4:, 5] = float("inf"), float("-inf"), float("inf")
    bad = ~torch.isfinite(want)
    assert torch.equal(out[bad], want[bad])
    assert torch.isfinite(out[~bad]).all()
