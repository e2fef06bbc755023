"""The 8-bit caches with one scale per page and head on the GPU: pages, decode attention."""
import numpy as np
import pytest
import torch

from block_util import D, DEV, bound_of, cached_rows, logical, make_cache, pack_ref, randn, softmax_rows

pytestmark = pytest.mark.gpu
MODES = ["e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def check_pages(c, b, K, V):
    """Slot b holds exactly the tokens K, V [H][L][D] (float16 arrays)."""
    l, G, S, H = c.lengths(b), c.cfg.G, c.cfg.S, c.cfg.H_kv
    ns, T, nr = l["n_sink"], l["T"], l["n_res"]
    assert ns + T + nr == K.shape[1]
    pages = c.table[b, : T // G].long()
    for side, x, code in zip("kv", (K, V), logical(c, pages)):
        bits = lambda y: np.ascontiguousarray(y).view(np.uint16)  # noqa: E731
        if ns:
            assert np.array_equal(bits(c.view(side + "_sink")[b][:, :ns].cpu().numpy()), bits(x[:, :ns]))
        assert np.array_equal(bits(c.view(side + "_res")[b][:, :nr].cpu().numpy()), bits(x[:, ns + T:]))
        want, scale = pack_ref(x[:, ns: ns + T].reshape(H, T // G, G, D).transpose(1, 0, 2, 3), c.mode_name)
        assert np.array_equal(c.view(side + "_meta")[pages].cpu().numpy(), scale, equal_nan=True)
        fin = np.isfinite(scale)
        assert np.array_equal(code[fin], want[fin]), "codes of side %s" % side


def named(c, mode):
    c.mode_name = mode
    return c


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("kw", [dict(G=64), dict(G=64, R=128, S=5), dict(G=128), dict(G=128, R=256, S=70), dict(G=256), dict(G=256, R=512)],
                         ids=str)
def test_prefill_append_flush(mode, kw):
    """Pages of a prompt and of full residuals, bit for bit."""
    rng = np.random.default_rng(kw["G"])
    R = kw.get("R", kw["G"])
    c = named(make_cache(rng, [0, 0, 0], mode, spare=40, **kw), mode)
    toks = []
    for b, n in enumerate((3 * R + 17 if R < 512 else R + 17, 1, 2 * kw["G"] + kw.get("S", 0))):
        k, v = randn(rng, 2, n, D), randn(rng, 2, n, D)
        k[..., :2] *= 6
        c.prefill(b, k, v)
        toks.append([k.cpu().numpy(), v.cpu().numpy()])
    c.flush()
    for b in range(3):
        check_pages(c, b, *toks[b])
    for _ in range(R + 3):
        kn, vn = randn(rng, 3, 2, D), randn(rng, 3, 2, D)
        c.append(kn, vn)
        for b in range(3):
            toks[b] = [np.concatenate([x, y[b].cpu().numpy()[:, None]], 1) for x, y in zip(toks[b], (kn, vn))]
        c.flush()
    for b in range(3):
        check_pages(c, b, *toks[b])
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_blocks_at_the_edge(mode):
    """Zeros, one value, fp16's smallest and largest, values on and beside ties, signed zero."""
    rng = np.random.default_rng(8)
    G = 64
    c = named(make_cache(rng, [0], mode, H_kv=1, H_q=1, G=G), mode)
    x = np.zeros((7, G, D), np.float16)
    x[1, 5, 7] = -3.0
    x[2] = rng.standard_normal((G, D)) * 2.0 ** -24
    x[3] = np.where(rng.random((G, D)) < 0.5, 65504, -65504)
    x[4] = -0.0
    top = 448 if mode == "e4m3" else 127
    half = (np.arange(G * D).reshape(G, D) % (2 * top + 1) - top) * 0.5  # codes, and the values half-way between them
    x[5] = half * (1 if mode == "e4m3" else 2) / 2
    x[5, 0, 0] = top if mode == "int8" else 224
    x[6] = np.nextafter(x[5], np.float16(1000))
    k = torch.from_numpy(x.reshape(1, 7 * G, D)).to(DEV)
    c.prefill(0, k, k.flip(1).contiguous())
    check_pages(c, 0, k.cpu().numpy(), k.flip(1).cpu().numpy())


@pytest.mark.parametrize("mode", MODES)
def test_blocks_with_infinity_or_nan(mode):
    """Such a block has no finite scale, and its neighbours know nothing of it."""
    rng = np.random.default_rng(9)
    c = named(make_cache(rng, [0, 0], mode, G=64), mode)
    for b, bad in enumerate((float("inf"), float("nan"))):
        k, v = randn(rng, 2, 200, D), randn(rng, 2, 200, D)
        k[0, 70, 3] = bad
        v[1, 5, 100] = -bad
        c.prefill(b, k, v)
        check_pages(c, b, k.cpu().numpy(), v.cpu().numpy())
        pages = c.table[b, :3].long()
        ks, vs = c.view("k_meta")[pages].cpu(), c.view("v_meta")[pages].cpu()
        assert [not bool(x.isfinite()) for x in ks[:, 0]] == [False, True, False] and bool(ks[:, 1].isfinite().all())
        assert [not bool(x.isfinite()) for x in vs[:, 1]] == [True, False, False] and bool(vs[:, 0].isfinite().all())
    q = randn(rng, 2, 8, D)
    out = c.decode_attn(q).cpu()
    assert bool(out.isnan().all())  # every head: keys of head 0, values of head 1
    assert c.read_status() == 0


DECODE = {
    "one_token": dict(lens=[1]),
    "short": dict(lens=[300, 5, 64]),
    "only_packed": dict(lens=[64, 128, 640]),
    "ragged_inactive": dict(lens=[700, 0, 129, 63, 1030, 0]),
    "sink": dict(lens=[3, 70, 69, 900], S=69),
    "g128_r256": dict(lens=[383, 128, 3000], G=128, R=256),
    "g256_r512": dict(lens=[900, 260, 511], G=256, R=512),
    "mha": dict(lens=[300, 40], H_q=3, H_kv=3),
    "g8": dict(lens=[300, 1040], H_q=16, H_kv=2),
    "g5": dict(lens=[300, 1], H_q=5, H_kv=1),
    "one_head_long": dict(lens=[30011], H_q=4, H_kv=1, max_T=32768),
    "many_slots": dict(lens=[(37 * i) % 400 for i in range(512)], H_q=2, H_kv=1, max_T=512),
}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("name", list(DECODE))
def test_decode(name, mode):
    kw = dict(DECODE[name])
    lens = kw.pop("lens")
    rng = np.random.default_rng(len(name))
    c = make_cache(rng, lens, mode, **kw)
    H_q, g = c.cfg.H_q, c.cfg.H_q // c.cfg.H_kv
    q = randn(rng, len(lens), H_q, D)
    out = torch.full((len(lens), H_q, D), 7.0, dtype=torch.float16, device=DEV)
    before = {m: x.clone() for m, x in c.buf.items()}
    c.decode_attn(q, out=out)
    assert all(torch.equal(x, c.buf[m]) for m, x in before.items()), "the cache was changed"
    on = [b for b, n in enumerate(lens) if n]
    x = q.clone()
    assert torch.equal(out[on], c.decode_attn(q)[on]) and torch.equal(out[on], c.decode_attn(x, out=x)[on])
    got, qd = out.cpu().double().numpy(), q.cpu().double().numpy()
    for b, n in enumerate(lens):
        if not n:
            assert np.all(got[b] == 7.0), "row of an empty slot was written"
            continue
        if len(lens) > 100 and b % 37:
            continue
        K, V = cached_rows(c, b)
        for h in range(c.cfg.H_kv):
            ref, size, mag = softmax_rows(qd[b, h * g: h * g + g], K[h], V[h])
            err = np.abs(got[b, h * g: h * g + g] - ref)
            bound = bound_of(ref, size, mag)
            assert np.all(err <= bound), "slot %d head %d: %g of its bound" % (b, h, (err / bound).max())
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_decode_of_uneven_blocks(mode):
    """Scales of blocks that differ by orders of magnitude: the weight of a block of small values
    is not lost, whether attention lies on it or not."""
    rng = np.random.default_rng(11)
    c = make_cache(rng, [0, 0], mode, G=64, H_q=4, H_kv=1)
    for b, sizes in enumerate(([1e-3, 200.0, 1.0, 3e-5], [300.0, 2e-4, 2e-4, 1.0])):
        k, v = randn(rng, 1, 256 + 9, D), randn(rng, 1, 256 + 9, D)
        for j, x in enumerate(sizes):
            v[:, 64 * j: 64 * j + 64] *= x
            k[:, 64 * j: 64 * j + 64] *= (0.1, 3.0, 1.0, 0.5)[j]
        c.prefill(b, k, v)
    for size in (0.1, 1.0, 12.0):
        q = randn(rng, 2, 4, D, scale=size)
        if size == 12.0:  # towards a token of a block of small values
            K, _ = cached_rows(c, 0)
            q[0] = torch.from_numpy(np.sign(K[0, 200])).half().to(DEV) * 8
        out = c.decode_attn(q).cpu().double().numpy()
        for b in range(2):
            K, V = cached_rows(c, b)
            ref, s, mag = softmax_rows(q[b].cpu().double().numpy(), K[0], V[0])
            err, bound = np.abs(out[b] - ref), bound_of(ref, s, mag)
            assert np.all(err <= bound), (b, size, (err / bound).max())


@pytest.mark.parametrize("mode", MODES)
def test_decode_large_scores(mode):
    """Queries near fp16's limit: one token takes all the weight."""
    rng = np.random.default_rng(12)
    c = make_cache(rng, [500], mode, G=128, H_q=4, H_kv=2)
    q = randn(rng, 1, 4, D, scale=8000.0)
    out = c.decode_attn(q).cpu().double().numpy()
    K, V = cached_rows(c, 0)
    for h in range(2):
        ref, s, mag = softmax_rows(q[0, 2 * h: 2 * h + 2].cpu().double().numpy(), K[h], V[h])
        assert np.all(np.abs(out[0, 2 * h: 2 * h + 2] - ref) <= U_LARGE(ref))


def U_LARGE(ref):
    return 3 * 2.0 ** -11 * np.abs(ref) + 1e-6


def test_decode_bad_page_is_reported():
    rng = np.random.default_rng(13)
    c = make_cache(rng, [300], "e4m3", G=64)
    c.table[0, 1] = c.n_pages
    c.decode_attn(randn(rng, 1, 8, D))
    assert c.read_status() == 2 and c.read_status() == 0
