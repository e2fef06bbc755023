"""Plain 64-bit forms of the chunk operators, and paged caches to run them on."""
import math

import numpy as np
import torch

from parity_util import _np, keys_logical, values_logical

DEV = "cuda:0"
D = 128
U16 = 2.0 ** -11  # half a step of fp16, relative


def randn(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float16)).to(DEV)


def make_cache(rng, lens, H_q=8, H_kv=2, bits=2, v_bits=0, G=128, R=None, S=0, max_T=4096, spare=64):
    """A paged cache whose slots hold lens[b] prefilled tokens (0: empty), with shuffled
    pages; everything that holds no token is filled with NaN (or all-ones codes)."""
    import bit_kv_cache_gb300 as kvq
    B = len(lens)
    n_pages = sum(max(0, n - S) // G for n in lens) + spare
    c = kvq.KVQPagedCache(B, H_q, H_kv, D, G, bits, n_pages=n_pages, max_T=max_T, S=S, R=R or G, device=DEV, v_bits=v_bits)
    c.free = [int(x) for x in rng.permutation(n_pages)]
    for name, b in c.buf.items():
        b.fill_(0xFF)  # fp16 0xFFFF is a NaN
    for b, n in enumerate(lens):
        if n:
            k = randn(rng, H_kv, n, D)
            k[..., :3] *= 4.0
            c.prefill(b, k, randn(rng, H_kv, n, D))
    return c


def cached_rows(c, b):
    """Dequantized keys and values of slot b in float64: [H_kv][L][D] each."""
    cfg, l = c.cfg, c.lengths(b)
    H, G, T = cfg.H_kv, cfg.G, l["T"]
    kb, vb = cfg.bits, cfg.v_bits or cfg.bits
    pages = c.table[b, : T // G].cpu().numpy()
    ks, vs = [_np(c.view("k_sink")[b][:, : l["n_sink"]]).astype(np.float64)], [_np(c.view("v_sink")[b][:, : l["n_sink"]]).astype(np.float64)]
    if T:
        kw = keys_logical(_np(c.view("k_codes"))[pages], G, 32 // kb).transpose(1, 0, 2, 3).astype(np.int64) & 0xFFFFFFFF
        sh = (kb * np.arange(32 // kb))[:, None]
        km = _np(c.view("k_meta"))[pages].transpose(1, 0, 2, 3).astype(np.float64)  # [H][J][D][2]
        code = ((kw[..., None, :] >> sh) & ((1 << kb) - 1)).reshape(H, T // G, G, D)
        ks.append((code * km[:, :, None, :, 0] + km[:, :, None, :, 1]).reshape(H, T, D))
        vw = values_logical(_np(c.view("v_codes"))[pages].swapaxes(0, 1)).astype(np.int64) & 0xFFFFFFFF  # [H][T][D/fpi]
        sh = vb * np.arange(32 // vb)
        code = ((vw[..., None] >> sh) & ((1 << vb) - 1)).reshape(H, T, D)
        vm = _np(c.view("v_meta"))[pages].transpose(1, 0, 2, 3, 4).reshape(H, T, 1, 2).astype(np.float64)
        vs.append(code * vm[..., 0] + vm[..., 1])
    ks.append(_np(c.view("k_res")[b][:, : l["n_res"]]).astype(np.float64))
    vs.append(_np(c.view("v_res")[b][:, : l["n_res"]]).astype(np.float64))
    return np.concatenate(ks, 1), np.concatenate(vs, 1)


def attn_check(c, n_new, q, k, v, out, what=""):
    """Every row of the chunk against softmax in float64.  The bound of an element counts the
    roundings on its way: dequantized keys (U16 of each product), softmax weights, values and
    the output (U16 each), and fp32 sums and exponentials."""
    cfg = c.cfg
    g = cfg.H_q // cfg.H_kv
    q, k, v, out = (x.detach().cpu().double().numpy() for x in (q, k, v, out))
    at = 0
    for b, n in enumerate(n_new):
        if not n:
            continue
        K, V = cached_rows(c, b)
        L = K.shape[1]
        K = np.concatenate([K, k[at:at + n].transpose(1, 0, 2)], 1)
        V = np.concatenate([V, v[at:at + n].transpose(1, 0, 2)], 1)
        hid = np.arange(L + n)[None, :] > L + np.arange(n)[:, None]
        for h in range(cfg.H_q):
            Kh, Vh, qh = K[h // g], V[h // g], q[at:at + n, h]
            s = np.where(hid, -np.inf, qh @ np.where(np.isfinite(Kh), Kh, 0.0).T / math.sqrt(D))
            mag = np.abs(qh) @ np.abs(np.where(np.isfinite(Kh), Kh, 0.0)).T / math.sqrt(D)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            Vf = np.where(np.isfinite(Vh), Vh, 0.0)
            ref, size = p @ Vf, p @ np.abs(Vf)
            for t, d in zip(*np.nonzero(~np.isfinite(Vh))):
                ref[~hid[:, t], d] += Vh[t, d]
            ds = np.where(hid, 0.0, mag).max(1, keepdims=True) * (U16 + 2.0 ** -15) + 1e-6
            bound = size * (2.2 * ds + 3 * U16) + U16 * np.abs(np.where(np.isfinite(ref), ref, 0.0)) + 1e-6
            got = out[at:at + n, h]
            fin = np.isfinite(ref)
            assert np.array_equal(np.isnan(got), np.isnan(ref)), "%s slot %d head %d: NaN" % (what, b, h)
            assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), "%s slot %d head %d: inf" % (what, b, h)
            err = np.abs(np.where(fin, got - np.where(fin, ref, 0.0), 0.0))
            i = np.unravel_index(np.argmax(err - bound), err.shape)
            assert np.all(err <= bound), "%s slot %d head %d row %d channel %d: %g, bound %g" % (what, b, h, i[0], i[1], err[i], bound[i])
        at += n
