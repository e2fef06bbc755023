"""Plain 64-bit forms of the 8-bit caches with one scale per page and head, and such caches to
run them on.  Nothing here uses the package's kernels but the calls under test."""
import math

import numpy as np
import torch

DEV = "cuda:0"
D = 128
U16 = 2.0 ** -11  # half a step of fp16, relative
TOP = {"e4m3": 448.0, "int8": 127.0}


def randn(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float16)).to(DEV)


def e4m3_values():
    """The 256 values of e4m3 by byte, from its definition."""
    v = np.zeros(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = np.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = -x if b >> 7 else x
    return v


E4M3 = e4m3_values()


def pack_ref(x, mode):
    """float16 blocks [..., G, D] -> (values of the codes, fp32 scales): products in fp32, codes
    from them by a search of the nearest value, ties to the even code."""
    x = x.astype(np.float32)
    amax = np.abs(x).max((-2, -1))
    with np.errstate(all="ignore"):
        scale = np.where(amax == 0, np.float32(1), amax / np.float32(TOP[mode])).astype(np.float32)
        inv = np.where(amax == 0, np.float32(0), np.float32(TOP[mode]) / amax).astype(np.float32)
        y = (x * inv[..., None, None]).astype(np.float32)
    if mode == "int8":
        return np.clip(np.rint(np.nan_to_num(y)), -127, 127), scale
    v = E4M3[:127].astype(np.float32)  # ascending, the even codes at even indices
    a = np.minimum(np.abs(y), np.float32(448))
    i = np.clip(np.searchsorted(v, a), 1, 126)
    lo, hi = v[i - 1], v[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return np.copysign(np.where(up, hi, lo), y).astype(np.float64), scale


def logical(c, pages):
    """Code values of physical pages in logical order: keys and values [n][H][G][D]."""
    G, H = c.cfg.G, c.cfg.H_kv
    out = []
    for name in ("k_codes", "v_codes"):
        x = c.view(name).view(torch.int8)[pages].cpu().numpy()
        x = x.astype(np.float64) if c.view(name).dtype == torch.int8 else E4M3[x.view(np.uint8)]
        if name == "k_codes":
            t = np.arange(G)[:, None]
            d = np.arange(D)[None, :]
            x = np.take_along_axis(x, np.broadcast_to(d ^ (64 * (t % 2)), x.shape), -1)
        else:
            x = x.swapaxes(-1, -2).reshape(len(x), H, G, D)
        out.append(x)
    return out


def make_cache(rng, lens, mode, H_q=8, H_kv=2, G=64, R=None, S=0, max_T=4096, spare=64, scale=1.0):
    """A cache whose slots hold lens[b] prefilled tokens (0: empty), with shuffled pages; what
    holds no token is filled with NaN."""
    import bit_kv_cache_gb300 as kvq
    B = len(lens)
    n_pages = sum(max(0, n - S) // G for n in lens) + spare
    c = kvq.KVQPagedCache(B, H_q, H_kv, D, G, 8, n_pages=n_pages, max_T=max_T, S=S, R=R or G, device=DEV, mode=mode)
    c.free = [int(x) for x in rng.permutation(n_pages)]
    for b in c.buf.values():
        b.fill_(0xFF)
    for b, n in enumerate(lens):
        if n:
            k = randn(rng, H_kv, n, D, scale=scale)
            k[..., :3] *= 4.0
            c.prefill(b, k, randn(rng, H_kv, n, D, scale=scale))
    return c


def cached_rows(c, b):
    """Keys and values of slot b in float64 as the cache holds them: [H_kv][L][D] each."""
    l, G = c.lengths(b), c.cfg.G
    pages = c.table[b, : l["T"] // G].long()
    both = []
    for side, code in zip("kv", logical(c, pages)):
        scale = c.view(side + "_meta")[pages].cpu().numpy().astype(np.float64)
        with np.errstate(invalid="ignore"):
            x = (code * scale[:, :, None, None]).transpose(1, 0, 2, 3).reshape(c.cfg.H_kv, l["T"], D)
        half = lambda n, k: c.view(side + n)[b][:, :k].cpu().numpy().astype(np.float64)  # noqa: E731
        both.append(np.concatenate([half("_sink", l["n_sink"]), x, half("_res", l["n_res"])], 1))
    return both


def softmax_rows(q, K, V, hid=None):
    """Rows q [n][D] over K, V [L][D] in float64: (outputs, their size for bound_of, largest
    |q| . |k| / sqrt D)."""
    s = q @ K.T / math.sqrt(D)
    mag = np.abs(q) @ np.abs(K).T / math.sqrt(D)
    if hid is not None:
        s, mag = np.where(hid, -np.inf, s), np.where(hid, 0.0, mag)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ V, p @ np.abs(V) + TINY * len(V) * np.abs(V).max(), mag.max(1, keepdims=True)


# Weights below fp16's normal numbers are off by half its smallest step, 2^-25, where the largest
# weight of the row is 2^6 at least.  A weight counts the value scale s in: w = 2^x p s, with
# sum w / s >= 2^6 / s_top for the token of the largest weight, so an output is off by
#   2^-25 sum |code_t| / (2^6 / s_top) <= 2^-31 L (M s_top) <= 2^-31 L max |v|
# (fp16 tokens: s = 1 and |v| in place of the code, the same).  In units of U16:
TINY = 2.0 ** -31 / U16


def bound_of(ref, size, mag):
    """What rounding may do to an element: operands are exact; a weight is rounded to fp16 once
    (U16 of its product; TINY is in the size), the output once; scores are fp32 sums of 128
    products (2^-24 of the magnitudes each, an error of the exponent, twice in numerator and
    denominator), the exponential and the fp32 sums over tiles add 2^-19."""
    ds = mag * 128 * 2.0 ** -24 + 2.0 ** -20
    return size * (2 * ds + 1.1 * U16 + 2.0 ** -19) + U16 * np.abs(ref) + 2.0 ** -24
