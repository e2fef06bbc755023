"""Chunks of new tokens over the 8-bit caches with one scale per page and head: attention,
extend, and their run together."""
import numpy as np
import pytest
import torch

from block_util import D, DEV, bound_of, cached_rows, make_cache, randn, softmax_rows

pytestmark = pytest.mark.gpu
MODES = ["e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def chunk_inputs(rng, c, n, rows=None):
    """q, k, v of n tokens as views of one fused projection, `rows` rows in all; the rows
    behind n hold NaN."""
    H_q, H = c.cfg.H_q, c.cfg.H_kv
    x = randn(rng, rows or n, H_q + 2 * H, D)
    x[:, H_q: H_q + H, :3] *= 4.0
    x[n:] = float("nan")
    return x[:, :H_q], x[:, H_q: H_q + H], x[:, H_q + H:]


def attn_check(c, new, q, k, v, out):
    """Every row against softmax in float64; infinite and NaN values reach the rows that see them."""
    g = c.cfg.H_q // c.cfg.H_kv
    q, k, v, out = (x.detach().cpu().double().numpy() for x in (q, k, v, out))
    at = 0
    for b, n in enumerate(new):
        if not n:
            continue
        K, V = cached_rows(c, b)
        L = K.shape[1]
        K = np.concatenate([K, k[at:at + n].transpose(1, 0, 2)], 1)
        V = np.concatenate([V, v[at:at + n].transpose(1, 0, 2)], 1)
        hid = np.arange(L + n)[None, :] > L + np.arange(n)[:, None]
        for h in range(c.cfg.H_q):
            Vh = V[h // g]
            Vf = np.where(np.isfinite(Vh), Vh, 0.0)
            ref, size, mag = softmax_rows(q[at:at + n, h], K[h // g], Vf, hid)
            bound = bound_of(ref, size, mag)
            for t, d in zip(*np.nonzero(~np.isfinite(Vh))):
                ref[~hid[:, t], d] += Vh[t, d]
            got, fin = out[at:at + n, h], np.isfinite(ref)
            assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
            err = np.where(fin, np.abs(np.where(fin, got, 0.0) - np.where(fin, ref, 0.0)), 0.0)
            assert np.all(err <= bound), "slot %d head %d: %g of its bound" % (b, h, (err / bound).max())
        at += n


ATTN = {
    "one_token_empty": dict(lens=[0], new=[1]),
    "one_token": dict(lens=[300], new=[1]),
    "first_chunk": dict(lens=[0, 0], new=[200, 33]),
    "page_inside_tile": dict(lens=[64, 192, 320, 63], new=[1, 2, 40, 3]),
    "ragged": dict(lens=[700, 0, 129, 5, 1030], new=[5, 70, 0, 1, 130]),
    "sink_r128": dict(lens=[700, 3, 140], new=[9, 20, 64], S=8, R=128),
    "page128": dict(lens=[900, 260], new=[40, 300], G=128),
    "page256_r512": dict(lens=[900, 600], new=[40, 300], G=256, R=512),
    "wide_inside_tile": dict(lens=[448, 64], new=[300, 257], H_q=4, H_kv=2),
    "mha": dict(lens=[300, 40], new=[257, 3], H_q=2, H_kv=2),
    "g8": dict(lens=[300, 64], new=[90, 7], H_q=16, H_kv=2),
    "g5_long": dict(lens=[2500], new=[201], H_q=5, H_kv=1),
    "sink_wide": dict(lens=[150, 400], new=[6, 2], S=200),
}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("name", list(ATTN))
def test_chunk_attention(name, mode):
    kw = dict(ATTN[name])
    lens, new = kw.pop("lens"), kw.pop("new")
    rng = np.random.default_rng(len(name))
    c = make_cache(rng, lens, mode, **kw)
    n = sum(new)
    q, k, v = chunk_inputs(rng, c, n, n + 3)
    out = torch.full((n + 3, c.cfg.H_q, D), 7.0, dtype=torch.float16, device=DEV)
    ch = c.plan(new)
    before = {m: x.clone() for m, x in c.buf.items()}
    c.chunk_attn(ch, q, k, v, out=out)
    assert torch.all(out[n:] == 7.0), "rows behind the chunk were written"
    assert all(torch.equal(x, c.buf[m]) for m, x in before.items()), "the cache was changed"
    attn_check(c, new, q[:n], k[:n], v[:n], out[:n])
    assert torch.equal(out[:n], c.chunk_attn(ch, q[:n], k[:n], v[:n]))
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("H_q, new", [(4, [1, 0, 1]), (4, [2, 1, 2]), (4, [4, 0, 3]), (4, [8, 8, 5]), (3, [10, 1, 4]), (8, [4, 1, 3]), (8, [5, 4, 40]),
                                      (5, [6, 100, 1]), (1, [32, 33, 7])], ids=str)
def test_few_rows(H_q, new, mode):
    """Slots of up to 32 rows a key head, alone and beside slots of more, whole and cut into
    parts; infinite and NaN values of new, cached and sink tokens."""
    rng = np.random.default_rng(sum(new))
    c = make_cache(rng, [3000, 200, 0], mode, H_q=H_q, H_kv=1, S=3)
    q, k, v = chunk_inputs(rng, c, sum(new))
    attn_check(c, new, q, k, v, c.chunk_attn(c.plan(new), q, k, v))
    v[new[0] - 1, 0, 5] = float("inf")
    v[sum(new) - 1, 0, 7] = -float("inf")
    v[0, 0, 9] = float("nan")
    c.view("v_sink")[0, 0, 1, 3] = float("inf")
    c.view("v_res")[1, 0, 2, 4] = -float("inf")
    ch = c.plan(new)
    out = c.chunk_attn(ch, q, k, v)
    attn_check(c, new, q, k, v, out)
    assert torch.equal(out.view(torch.int16), c.chunk_attn(ch, q, k, v).view(torch.int16))
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_decode_infinite_values(mode):
    """Infinite and NaN values in the sink and the residual, of a slot in several parts too."""
    rng = np.random.default_rng(14)
    c = make_cache(rng, [5000, 90], mode, S=2, H_kv=1, H_q=4, max_T=8192)
    c.view("v_sink")[0, 0, 1, 3] = float("inf")
    c.view("v_res")[1, 0, 2, 4] = float("nan")
    c.view("v_res")[0, 0, 3, 6] = -float("inf")
    q = randn(rng, 2, 4, D)
    out = c.decode_attn(q).cpu().double().numpy()
    for b in range(2):
        K, V = cached_rows(c, b)
        Vf = np.where(np.isfinite(V[0]), V[0], 0.0)
        ref, size, mag = softmax_rows(q[b].cpu().double().numpy(), K[0], Vf)
        bound = bound_of(ref, size, mag)
        ref = ref + np.where(np.isfinite(V[0]), 0.0, V[0]).sum(0)
        fin = np.isfinite(ref)
        assert np.array_equal(np.isnan(out[b]), np.isnan(ref)) and np.array_equal(out[b][~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
        assert (~fin).sum() == (8 if b == 0 else 4) and np.all(np.abs(out[b] - ref)[fin] <= bound[fin])


@pytest.mark.parametrize("mode", MODES)
def test_chunk_attention_long_split(mode):
    """One short chunk over a long cache: its key tiles are spread over many ranges."""
    rng = np.random.default_rng(3)
    c = make_cache(rng, [20000 + 77], mode, max_T=20480)
    for new in ([1], [6], [40], [90]):
        q, k, v = chunk_inputs(rng, c, new[0])
        ch = c.plan(new)
        out = c.chunk_attn(ch, q, k, v)
        attn_check(c, new, q, k, v, out)
        assert torch.equal(out, c.chunk_attn(ch, q, k, v))
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_blocks_of_other_sizes_and_large_scores(mode):
    """Scales that differ by orders of magnitude from page to page, and queries near fp16's
    limit: references far from the scores of the next tile."""
    rng = np.random.default_rng(5)
    c = make_cache(rng, [0, 0], mode, H_q=4, H_kv=1)
    for b in range(2):
        k, v = randn(rng, 1, 64 * 9 + 5, D), randn(rng, 1, 64 * 9 + 5, D)
        for j in range(9):
            k[:, 64 * j: 64 * j + 64] *= (0.1, 3.0, 1.0, 0.5, 2.0, 0.01, 1.0, 5.0, 0.3)[j]
            v[:, 64 * j: 64 * j + 64] *= (1e-3, 200.0, 1.0, 3e-5, 50.0, 1.0, 1e-4, 0.1, 300.0)[8 - j if b else j]
        c.prefill(b, k, v)
    for scale in (1.0, 30.0):
        new = [80, 7]
        q, k, v = chunk_inputs(rng, c, 87)
        q = (q * scale).contiguous()
        attn_check(c, new, q, k, v, c.chunk_attn(c.plan(new), q, k, v))
    q = randn(rng, 87, 4, D, scale=8000.0)
    out = c.chunk_attn(c.plan(new), q, k, v).cpu().double().numpy()
    at = 0
    for b, n in enumerate(new):  # one token takes all the weight
        K, V = cached_rows(c, b)
        K = np.concatenate([K, k[at:at + n].cpu().double().numpy().transpose(1, 0, 2)], 1)
        V = np.concatenate([V, v[at:at + n].cpu().double().numpy().transpose(1, 0, 2)], 1)
        hid = np.arange(K.shape[1])[None, :] > K.shape[1] - n + np.arange(n)[:, None]
        for h in range(4):
            qd = q[at:at + n, h].cpu().double().numpy()
            s = np.where(hid, -np.inf, qd @ K[0].T / np.sqrt(D))
            two = np.sort(s, 1)[:, -2:]
            sure = two[:, 1] - two[:, 0] > 64  # and no tie within the fp32 sums' error
            ref = V[0][s.argmax(1)]
            err = np.abs(out[at:at + n, h] - ref)[sure]
            assert sure.sum() > n // 2 and np.all(err <= (2.0 ** -10 * np.abs(ref) + 1e-6)[sure])
        at += n
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_values_not_finite(mode):
    """New tokens' infinite and NaN values reach the rows that see them, and no others; a page
    that holds one makes its slot's rows NaN for that head alone."""
    rng = np.random.default_rng(4)
    new = [140, 3]
    c = make_cache(rng, [260, 0], mode)
    q, k, v = chunk_inputs(rng, c, 143)
    v[100, 0, 5] = float("inf")
    v[120, 1, 7] = float("nan")
    v[139, 0, 9] = -float("inf")
    ch = c.plan(new)
    attn_check(c, new, q, k, v, c.chunk_attn(ch, q, k, v))
    kk, vv = randn(rng, 2, 200, D), randn(rng, 2, 200, D)
    vv[1, 70, 3] = float("inf")
    c.release(1)
    c.prefill(1, kk, vv)
    out = c.chunk_attn(c.plan(new), q, k, torch.zeros_like(v))
    assert bool(out[:140].isfinite().all()) and bool(out[140:, :4].isfinite().all()) and bool(out[140:, 4:].isnan().all())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("kw", [dict(G=64), dict(G=64, R=192, S=5), dict(G=128, R=128), dict(G=128, R=256, S=70), dict(G=256)], ids=str)
def test_extend_is_append_and_flush(mode, kw):
    """Any cut of the tokens into chunks leaves the state of append and flush, bit for bit."""
    rng = np.random.default_rng(6)
    lens, counts = [0, 300, 0, 64], [[5, 1, 0, 70], [400, 130, 0, 1], [0, 64, 3, 700], [127, 0, 66, 2]]
    a, b = make_cache(rng, lens, mode, **kw), None
    rng = np.random.default_rng(6)
    b = make_cache(rng, lens, mode, **kw)
    for i, new in enumerate(counts):
        n = sum(new)
        x = randn(rng, n, 4, D)
        k, v = x[:, :2], x[:, 2:]
        a.extend(a.plan(new), k, v)
        at = np.concatenate([[0], np.cumsum(new)])
        for s in range(4):  # one slot after the other
            for t in range(new[s]):
                kn, vn = torch.zeros(4, 2, D, dtype=torch.float16, device=DEV), torch.zeros(4, 2, D, dtype=torch.float16, device=DEV)
                kn[s], vn[s] = k[at[s] + t], v[at[s] + t]
                on = [b.lens_host[4 * j + 3] for j in range(4)]
                if not on[s]:
                    b.prefill(s, kn[s][:, None].contiguous(), vn[s][:, None].contiguous())
                    b.flush()
                    continue
                hold = [b.lens_host[4 * j: 4 * j + 4] for j in range(4)]
                for j in range(4):  # only slot s takes a token
                    if j != s:
                        b.lens_host[4 * j + 3] = 0
                b.lens.copy_(torch.tensor([b.lens_host[4 * j: 4 * j + 4] for j in range(4)], dtype=torch.int32))
                b.append(kn, vn)
                b.flush()
                for j in range(4):
                    if j != s:
                        b.lens_host[4 * j: 4 * j + 4] = hold[j]
                b.lens.copy_(torch.tensor([b.lens_host[4 * j: 4 * j + 4] for j in range(4)], dtype=torch.int32))
        for s in range(4):
            assert a.lengths(s) == b.lengths(s), (i, s)
            assert a.lens[s].tolist() == b.lens[s].tolist()
            if a.lengths(s)["active"]:
                for x, y in zip(cached_rows(a, s), cached_rows(b, s)):
                    assert np.array_equal(x, y), (i, s)
    assert a.read_status() == 0 and b.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_chunk_step(mode):
    """Plan, norm and rotation, attention and extend in one call, over several steps."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(7)
    c = make_cache(rng, [0, 100], mode, S=3)
    w = randn(rng, D)
    for new in ([70, 1], [1, 1], [0, 200], [64, 5]):
        n = sum(new)
        x = randn(rng, n, 12, D)
        q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
        before = [c.lengths(b) for b in range(2)]
        pos = torch.tensor([sum(list(before[b].values())[:3]) + i for b in range(2) for i in range(new[b])], dtype=torch.int32, device=DEV)
        qr, kr = kvq.qk_norm_rope(q, k, w, w, pos)
        held = [cached_rows(c, b) for b in range(2)]
        out, ch = c.chunk_step(new, q, k, v, w, w)
        assert ch.n_tokens == n
        at = 0
        for b, m in enumerate(new):
            if not m:
                continue
            K = np.concatenate([held[b][0], kr[at:at + m].cpu().double().numpy().transpose(1, 0, 2)], 1)
            V = np.concatenate([held[b][1], v[at:at + m].cpu().double().numpy().transpose(1, 0, 2)], 1)
            hid = np.arange(K.shape[1])[None, :] > K.shape[1] - m + np.arange(m)[:, None]
            for h in range(8):
                ref, size, mag = softmax_rows(qr[at:at + m, h].cpu().double().numpy(), K[h // 4], V[h // 4], hid)
                err, bound = np.abs(out[at:at + m, h].cpu().double().numpy() - ref), bound_of(ref, size, mag)
                assert np.all(err <= bound), (err / bound).max()
            at += m
    assert c.read_status() == 0


def test_captured_calls_and_streams():
    """Decode and chunk attention captured and replayed, on a stream of their own, give what the
    calls give."""
    rng = np.random.default_rng(8)
    c = make_cache(rng, [3000, 200, 70], "e4m3")
    new = [3, 60, 1]
    q, k, v = chunk_inputs(rng, c, 64)
    qd = randn(rng, 3, 8, D)
    ch = c.plan(new)
    want, wantd = c.chunk_attn(ch, q, k, v), c.decode_attn(qd)
    out, outd = torch.zeros_like(want), torch.zeros_like(wantd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.chunk_attn(ch, q, k, v, out=out)
        c.decode_attn(qd, out=outd)
    for _ in range(3):
        out.zero_(), outd.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(outd, wantd)
    with torch.cuda.stream(s):
        assert torch.equal(c.decode_attn(qd), wantd)
    assert c.read_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_replay_after_growth(mode):
    """A captured decode attends over the lengths of its replay, also behind a page boundary and
    with a slot that has become empty."""
    rng = np.random.default_rng(15)
    c = make_cache(rng, [3000, 60, 200, 1], mode, H_kv=1, H_q=4, S=2)
    q, out = randn(rng, 4, 4, D), torch.zeros(4, 4, D, dtype=torch.float16, device=DEV)
    c.decode_attn(q, out=out)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.decode_attn(q, out=out)
    for n in (1, 70, 130):
        new = [n, n, 0, n]
        x = randn(rng, 3 * n, 2, D)
        c.extend(c.plan(new), x[:, :1], x[:, 1:])
        if n == 70:
            c.release(2)
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for b in (0, 1, 2, 3):
            if not c.lengths(b)["active"]:
                assert torch.all(out[b] == 7.0)
                continue
            K, V = cached_rows(c, b)
            ref, size, mag = softmax_rows(q[b].cpu().double().numpy(), K[0], V[0])
            assert np.all(np.abs(out[b].cpu().double().numpy() - ref) <= bound_of(ref, size, mag)), (n, b)
    assert c.read_status() == 0


def test_pages_beyond_4_gb():
    """Pages whose codes lie more than 2^32 bytes behind the pool's start, in every call."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(16)
    n_pages = 36000  # 131072 bytes a side each
    c = kvq.KVQPagedCache(2, 16, 8, D, 128, 8, n_pages=n_pages, max_T=4096, device=DEV, mode="e4m3")
    c.free = list(range(n_pages - 40, n_pages))
    k, v = randn(rng, 8, 700, D), randn(rng, 8, 700, D)
    c.prefill(0, k, v)
    x = randn(rng, 380, 32, D)
    ch = c.plan([300, 80])
    out = c.chunk_attn(ch, x[:, :16], x[:, 16:24], x[:, 24:])
    attn_check(c, [300, 80], x[:, :16], x[:, 16:24], x[:, 24:], out)
    c.extend(ch, x[:, 16:24], x[:, 24:])
    for _ in range(30):
        y = randn(rng, 2, 32, D)
        q = c.append_rope(y[:, :16], y[:, 16:24], y[:, 24:])
    assert int(c.table[0, : c.lengths(0)["T"] // 128].min()) >= n_pages - 40
    ch = c.plan([2, 1])
    few = c.chunk_attn(ch, x[:3, :16], x[:3, 16:24], x[:3, 24:])
    attn_check(c, [2, 1], x[:3, :16], x[:3, 16:24], x[:3, 24:], few)
    out = c.decode_attn(q)
    for b in range(2):
        K, V = cached_rows(c, b)
        for h in range(8):
            ref, size, mag = softmax_rows(q[b, 2 * h: 2 * h + 2].cpu().double().numpy(), K[h], V[h])
            assert np.all(np.abs(out[b, 2 * h: 2 * h + 2].cpu().double().numpy() - ref) <= bound_of(ref, size, mag))
    assert c.read_status() == 0


def test_calls_on_a_stream_of_their_own():
    """Every call on a side stream, ordered by events alone."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(17)
    a, b = (make_cache(np.random.default_rng(18), [300, 64], "int8") for _ in range(2))
    x = randn(rng, 70, 12, D)
    y = randn(rng, 2, 12, D)
    s = torch.cuda.Stream()
    res = []
    for c, st in ((a, torch.cuda.current_stream()), (b, s)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            out, _ = c.chunk_step([65, 5], x[:, :8], x[:, 8:10], x[:, 10:])
            q = c.append_rope(y[:, :8], y[:, 8:10], y[:, 10:])
            res.append((out, q, c.decode_attn(q)))
            c.flush()
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(*res)) and torch.equal(a.lens, b.lens)
    for name in a.buf:
        assert torch.equal(a.buf[name], b.buf[name]), name
