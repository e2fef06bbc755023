"""The chunk operators of the paged cache on the GPU: plan, chunk attention, extend and
their run together, against plain 64-bit forms and against append and flush."""
import numpy as np
import pytest
import torch

from chunk_util import DEV, attn_check, cached_rows, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def chunk_inputs(rng, c, n, rows=None):
    """q, k, v of n tokens as views of one fused projection, `rows` rows in all; the rows
    behind n hold NaN."""
    H_q, H = c.cfg.H_q, c.cfg.H_kv
    x = randn(rng, rows or n, H_q + 2 * H, 128)
    x[:, H_q: H_q + H, :3] *= 4.0
    x[n:] = float("nan")
    return x[:, :H_q], x[:, H_q: H_q + H], x[:, H_q + H:]


ATTN = {
    "one_token_empty": dict(lens=[0], new=[1]),
    "one_token": dict(lens=[300], new=[1]),
    "first_chunk": dict(lens=[0, 0], new=[200, 33]),
    "one_key": dict(lens=[1, 128, 129, 127], new=[1, 2, 1, 3]),
    "ragged": dict(lens=[700, 0, 129, 5, 1030], new=[5, 70, 0, 1, 130]),
    "k4v2_sink": dict(lens=[700, 3, 140], new=[9, 20, 64], bits=4, v_bits=2, S=8),
    "k8v8_page256": dict(lens=[900, 260], new=[40, 300], bits=8, G=256, R=512),
    "k2v4_r256": dict(lens=[383, 128], new=[129, 7], v_bits=4, R=256),
    "k4v8": dict(lens=[513], new=[65], bits=4, v_bits=8),
    "k8v2": dict(lens=[400, 513], new=[31, 3], bits=8, v_bits=2),
    "mha": dict(lens=[300, 40], new=[257, 3], H_q=2, H_kv=2),
    "g3": dict(lens=[300, 0], new=[90, 47], H_q=6, H_kv=2),
    "g2_long": dict(lens=[2500], new=[300], H_q=4, H_kv=2, bits=4),
    "sink_wide": dict(lens=[150, 400], new=[6, 2], S=200),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_chunk_attention(name):
    kw = dict(ATTN[name])
    lens, new = kw.pop("lens"), kw.pop("new")
    rng = np.random.default_rng(len(name))
    c = make_cache(rng, lens, **kw)
    n = sum(new)
    q, k, v = chunk_inputs(rng, c, n, n + 3)
    out = torch.full((n + 3, c.cfg.H_q, 128), 7.0, dtype=torch.float16, device=DEV)
    ch = c.plan(new)
    before = {m: x.clone() for m, x in c.buf.items()}
    c.chunk_attn(ch, q, k, v, out=out)
    assert torch.all(out[n:] == 7.0), "rows behind the chunk were written"
    assert all(torch.equal(x, c.buf[m]) for m, x in before.items()), "the cache was changed"
    attn_check(c, new, q[:n], k[:n], v[:n], out[:n], name)
    assert c.read_status() == 0


def test_chunk_attention_long_split():
    """One short chunk over a long cache: its key tiles are spread over many ranges."""
    rng = np.random.default_rng(3)
    c = make_cache(rng, [20000 + 77], H_q=8, H_kv=2, max_T=20480)
    for new in ([1], [6], [40]):
        q, k, v = chunk_inputs(rng, c, new[0])
        out = c.chunk_attn(c.plan(new), q, k, v)
        attn_check(c, new, q, k, v, out)
        again = c.chunk_attn(c.plan(new), q, k, v)
        assert torch.equal(out, again)


def test_chunk_attention_values_not_finite():
    """Infinite and NaN values reach the rows that see them, and no others."""
    rng = np.random.default_rng(4)
    new = [140, 3]
    c = make_cache(rng, [260, 0])
    q, k, v = (x.clone() for x in chunk_inputs(rng, c, sum(new)))
    v[100, 0, 5] = float("inf")
    v[120, 1, 6] = float("nan")
    v[130, 0, 5] = float("-inf")
    v[142, 0, 0] = float("inf")
    out = c.chunk_attn(c.plan(new), q, k, v)
    attn_check(c, new, q, k, v, out)


def test_chunk_attention_masked_keys_not_finite():
    """Keys that a row may not see do not reach it, whatever they hold."""
    rng = np.random.default_rng(5)
    c = make_cache(rng, [130])
    q, k, v = (x.clone() for x in chunk_inputs(rng, c, 20))
    ch = c.plan([20])
    want = c.chunk_attn(ch, q, k, v)
    k[15:] = float("nan")
    k[16:] = float("inf")
    got = c.chunk_attn(ch, q, k, v)
    assert torch.equal(want[:15], got[:15])
    assert torch.isnan(got[15:]).all()


def test_chunk_attention_large_scores():
    """Scores of several thousand: the running maximum keeps every weight finite."""
    rng = np.random.default_rng(6)
    c = make_cache(rng, [520])
    q, k, v = (x.clone() for x in chunk_inputs(rng, c, 30))
    q = (q.float() * 200).half()
    out = c.chunk_attn(c.plan([30]), q, k, v)
    assert torch.isfinite(out).all()
    big = cached_rows(c, 0)[1]
    assert out.abs().max() <= max(np.abs(big).max(), v.abs().max().item()) * (1 + 2.0 ** -8)


def test_chunk_attention_bad_page_is_reported():
    rng = np.random.default_rng(7)
    c = make_cache(rng, [300])
    q, k, v = chunk_inputs(rng, c, 2)
    ch = c.plan([2])
    c.table[0, 1] = 10 ** 6
    c.chunk_attn(ch, q, k, v)
    assert c.read_status() == 2


def test_chunk_attention_matches_decode():
    """One new token per slot: the result of append and decode_attn."""
    rng = np.random.default_rng(8)
    lens = [1000, 129, 5, 2048]
    c = make_cache(rng, lens, H_q=16, H_kv=4)
    q, k, v = chunk_inputs(rng, c, 4)
    out = c.chunk_attn(c.plan([1] * 4), q, k, v)
    c.append(k.contiguous(), v.contiguous())
    ref = c.decode_attn(q.contiguous())
    assert torch.all((out - ref).float().abs() <= 2e-3 + 2e-3 * ref.float().abs())


def test_chunk_attention_captured():
    """Two captured calls with a chunk each, replayed on new inputs."""
    rng = np.random.default_rng(9)
    c = make_cache(rng, [700, 40])
    new = [9, 20]
    q, k, v = (x.clone() for x in chunk_inputs(rng, c, 29))
    chunks = [c.plan(new), c.plan(new)]
    outs = [torch.zeros(29, c.cfg.H_q, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    c.chunk_attn(chunks[0], q, k, v, out=outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for ch, o in zip(chunks, outs):
            c.chunk_attn(ch, q, k, v, out=o)
    for _ in range(2):
        for x in (q, k, v):
            x.copy_(randn(rng, *x.shape))
        for o in outs:
            o.zero_()
        graph.replay()
        for o in outs:
            attn_check(c, new, q, k, v, o)


@pytest.mark.parametrize("B,S,R,G", [(1, 0, 128, 128), (5, 8, 256, 128), (512, 3, 256, 256), (33, 0, 128, 128)])
def test_plan(B, S, R, G):
    rng = np.random.default_rng(B)
    import bit_kv_cache_gb300 as kvq
    max_T = 8 * R
    c = kvq.KVQPagedCache(B, 1, 1, 128, G, 2, n_pages=4 * B * max_T // G, max_T=max_T, S=S, R=R, device=DEV)
    lens = np.zeros((B, 4), np.int32)
    for b in range(B):
        if rng.random() < 0.7:
            L = int(rng.integers(1, 3 * R))
            ns = min(S, L)
            lens[b] = ns, (L - ns) // G * G, (L - ns) % G, 1
    c.lens.copy_(torch.from_numpy(lens))
    for i, x in enumerate(lens.ravel()):
        c.lens_host[i] = int(x)
    new = rng.integers(0, 2 * R, B).astype(np.int32)
    new[rng.random(B) < 0.3] = 0
    if B == 1:
        new[0] = 1
    N = int(new.sum())
    ch = c.new_chunk(N + 5)
    ch.slot.fill_(-7)
    ch.pos.fill_(-7)
    c.table.fill_(-1)
    pages = torch.from_numpy(rng.permutation(c.n_pages).astype(np.int32)).to(DEV)
    c.plan(torch.from_numpy(new), ch, pages=pages)
    assert ch.n_tokens == N
    cu = np.concatenate([[0], np.cumsum(new)])
    assert np.array_equal(ch.cu.cpu().numpy(), cu)
    slot = np.repeat(np.arange(B), new)
    assert np.array_equal(ch.slot.cpu().numpy(), np.r_[slot, [-7] * 5])
    pos = np.concatenate([lens[b, :3].sum() + np.arange(new[b]) for b in range(B)] + [[-7] * 5])
    assert np.array_equal(ch.pos.cpu().numpy(), pos)
    table, at, ids = np.full((B, max_T // G), -1), 0, pages.cpu().numpy()
    for b in range(B):
        to_sink = min(int(new[b]), S - lens[b, 0])
        n = (lens[b, 2] + new[b] - to_sink) // R * R // G if new[b] else 0
        table[b, lens[b, 1] // G: lens[b, 1] // G + n] = ids[at: at + n]
        at += n
    assert np.array_equal(c.table.cpu().numpy(), table)
    assert np.array_equal(ch.desc.cpu().numpy().ravel(), np.frombuffer(ch.host, np.int32))


EXTEND = {
    "step": dict(lens=[125, 127, 0, 120, 3], new=[8, 1, 5, 0, 1]),
    "chunk": dict(lens=[1000, 0, 64], new=[700, 513, 64]),
    "k4v8_sink": dict(lens=[0, 3, 500], new=[400, 130, 260], bits=4, v_bits=8, S=8),
    "k8v4_r256": dict(lens=[383, 128, 1], new=[130, 700, 3], bits=8, v_bits=4, R=256),
    "k2v2_page256": dict(lens=[255, 700], new=[1, 600], G=256, R=512),
    "k4v2_page256": dict(lens=[30, 255], new=[300, 1], bits=4, v_bits=2, G=256, R=256),
    "k8v8_page256": dict(lens=[200], new=[900], bits=8, G=256),
}


def poke(rng, x):
    """Values that a quantizer finds hard: constant rows and channels, huge, tiny and tied ones."""
    x = x.clone()
    n = x.shape[0]
    x[n // 3, 0] = 0.25
    x[:, 0, 7] = -1.5
    x[:, 0, 8] = (torch.arange(n, device=x.device) % 4).half() * 0.5
    x[n // 2, 0, :40] = torch.from_numpy(rng.integers(0, 0x0800, 40, dtype=np.uint16).view(np.float16)).to(x.device)
    x[-1, 0, 3] = 60000.0
    return x


@pytest.mark.parametrize("name", list(EXTEND))
def test_extend_is_append_and_flush(name):
    """The cache that a chunk leaves is, bit for bit, the one that its tokens leave one by
    one; rows that hold no token keep what they held."""
    kw = dict(EXTEND[name])
    lens, new = kw.pop("lens"), kw.pop("new")
    B = len(lens)
    a = make_cache(np.random.default_rng(1), lens, **kw)
    one = make_cache(np.random.default_rng(1), lens, **kw)
    rng = np.random.default_rng(2)
    q, k, v = chunk_inputs(rng, a, sum(new))
    k, v = poke(rng, k), poke(rng, v)
    x = torch.stack([k, v], 2)  # strided views: heads of a token adjacent
    x = torch.cat([k, v], 1)
    ch = a.plan(new)
    a.extend(ch, x[:, : a.cfg.H_kv], x[:, a.cfg.H_kv:])
    cu = np.concatenate([[0], np.cumsum(new)])
    for b in range(B):  # slot after slot: the others are parked as empty meanwhile
        if new[b] and not one.lens_host[4 * b + 3]:
            one.lens_host[4 * b + 3] = 1
            one.lens[b, 3] = 1
        for i in range(new[b]):
            keep = [one.lens_host[4 * s + 3] for s in range(B)]
            for s in range(B):
                if s != b:
                    one.lens_host[4 * s + 3] = 0
            on = one.lens[:, 3].clone()
            one.lens[:, 3] = 0
            one.lens[b, 3] = 1
            kn = torch.zeros(B, a.cfg.H_kv, 128, dtype=torch.float16, device=DEV)
            vn = kn.clone()
            kn[b], vn[b] = k[cu[b] + i], v[cu[b] + i]
            one.append(kn, vn)
            one.flush()
            one.lens[:, 3] = on
            for s in range(B):
                one.lens_host[4 * s + 3] = keep[s]
    assert list(a.lens_host) == list(one.lens_host)
    assert torch.equal(a.lens.cpu(), torch.tensor(list(a.lens_host), dtype=torch.int32).view(B, 4))
    for b in range(B):
        l = a.lengths(b)
        J = l["T"] // a.cfg.G
        pa, po = a.table[b, :J].long(), one.table[b, :J].long()
        assert a.pages[b][:J] == pa.tolist()
        for m in ("k_codes", "k_meta", "v_codes", "v_meta"):
            assert torch.equal(a.view(m)[pa].view(torch.int16), one.view(m)[po].view(torch.int16)), "slot %d %s" % (b, m)
        for m, n in (("k_res", l["n_res"]), ("v_res", l["n_res"]), ("k_sink", l["n_sink"]), ("v_sink", l["n_sink"])):
            if a.buf[m].numel() > 16:
                assert torch.equal(a.view(m)[b][:, :n].view(torch.int16), one.view(m)[b][:, :n].view(torch.int16)), "slot %d %s" % (b, m)
        # rows behind the new residual: as make_cache left them (NaN), unless an old token was there
        old = lens[b] - min(lens[b], a.cfg.S)
        old -= old // a.cfg.G * a.cfg.G
        assert (a.view("k_res")[b][:, max(l["n_res"], old):].view(torch.int16) == -1).all()
    used = torch.cat([a.table[b, : a.lengths(b)["T"] // a.cfg.G] for b in range(B)]).long()
    idle = torch.ones(a.n_pages, dtype=torch.bool, device=DEV)
    idle[used] = False
    assert (a.view("k_codes")[idle] == -1).all() and (a.view("v_codes")[idle] == -1).all()
    assert a.read_status() == 0


def test_extend_bad_page_is_reported():
    rng = np.random.default_rng(3)
    c = make_cache(rng, [100])
    q, k, v = chunk_inputs(rng, c, 40)
    ch = c.plan([40])
    c.table[0, 0] = -5
    c.extend(ch, k, v)
    assert c.read_status() == 2


@pytest.mark.parametrize("R", [128, 256])
@pytest.mark.parametrize("bits", [2, 8])
def test_extend_bad_page_stores_nothing(R, bits):
    rng = np.random.default_rng(R)
    c = make_cache(rng, [100, 0], R=R, bits=bits)
    n = 2 * R - 100
    q, k, v = chunk_inputs(rng, c, n)
    ch = c.plan([n, 0])
    good = int(c.table[0, 1])
    c.table[0, 0] = c.n_pages
    before = {name: c.buf[name].clone() for name in ("k_codes", "k_meta", "v_codes", "v_meta")}
    c.extend(ch, k, v)
    assert c.read_status() == 2
    for name, old in before.items():
        same = (c.buf[name].view(c.n_pages, -1) == old.view(c.n_pages, -1)).all(1)
        assert not same[good] and same.sum() == c.n_pages - (2 * R // 128 - 1), name


def test_captured_chunk_is_not_planned_again():
    """A replay reads the plan's arrays."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(31)
    c = make_cache(rng, [300, 40])
    q, k, v = chunk_inputs(rng, c, 12)
    ch, other = c.plan([10, 2]), c.plan([10, 2])
    out = c.chunk_attn(other, q, k, v)
    got = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.chunk_attn(ch, q, k, v, out=got)
    with pytest.raises(kvq.KvqError) as e:
        c.plan([1, 2], ch)
    assert e.value.code == -2
    c.plan([1, 2], other)
    graph.replay()
    assert torch.equal(got, out)


def test_refused_plan_takes_no_pages():
    """The pages of a plan that the library refuses go back, so that a later flush maps them."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(32)
    c = make_cache(rng, [127, 0])
    free = list(c.free)
    with pytest.raises(kvq.KvqError):
        c.plan([130, 0], c.new_chunk(8))
    assert c.free == free and c.pages == [[], []]
    with pytest.raises(kvq.KvqError):
        c.plan([1 << 20, 0], c.new_chunk(8), pages=torch.zeros(4, dtype=torch.int32, device=DEV))
    for _ in range(2):
        c.append(randn(rng, 2, 2, 128), randn(rng, 2, 2, 128))
        c.flush()
    assert c.lengths(0)["T"] == 128 and int(c.table[0, 0]) == free[-1] and c.read_status() == 0


def test_extend_after_released_pages():
    """A plan's pages that went back to the pool are another slot's."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(33)
    c = make_cache(rng, [0, 0])
    q, k, v = chunk_inputs(rng, c, 130)
    for give_back in (lambda: c.release(0), c.clear):
        ch = c.plan([130, 0])
        give_back()
        with pytest.raises(kvq.KvqError) as e:
            c.extend(ch, k, v)
        assert e.value.code == -1
    c.extend(c.plan([130, 0], ch), k, v)
    assert c.lengths(0)["T"] == 128 and c.read_status() == 0


def test_plan_goes_stale():
    """A plan holds for the lengths it was made for, and extends a cache once."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(4)
    c = make_cache(rng, [100, 0])
    q, k, v = chunk_inputs(rng, c, 4)
    ch = c.plan([3, 1])
    c.extend(ch, k, v)
    state = list(c.lens_host)
    for call in (lambda: c.extend(ch, k, v), lambda: c.chunk_attn(ch, q, k, v)):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.code == -1
    assert list(c.lens_host) == state
    ch = c.plan([0, 0], ch)
    assert ch.n_tokens == 0
    c.chunk_attn(ch, q, k, v)
    c.extend(ch, k, v)
    assert list(c.lens_host) == state


def test_plan_of_another_cache():
    """A plan's slot maps serve a cache of the same lengths; its pages are not that cache's."""
    import bit_kv_cache_gb300 as kvq
    a, b = (make_cache(np.random.default_rng(s), [100, 0]) for s in (1, 2))
    q, k, v = chunk_inputs(np.random.default_rng(3), a, 50)
    ch = a.plan([40, 10])
    for c in (a, b):
        attn_check(c, [40, 10], q, k, v, c.chunk_attn(ch, q, k, v))
    with pytest.raises(kvq.KvqError):
        b.extend(ch, k, v)
    assert b.lengths(0)["n_res"] == 100
    a.extend(ch, k, v)
    b.extend(b.plan([40, 10], ch), k, v)
    assert b.read_status() == 0 and list(a.lens_host) == list(b.lens_host)


def test_many_slots():
    """200 slots of many lengths: units far smaller than a range, empty slots between them."""
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 500, 200)]
    new = [int(x) for x in rng.integers(0, 4, 200)]
    lens[7], new[9], new[199], new[100] = 0, 0, 0, 90
    c = make_cache(rng, lens, H_q=4, H_kv=1, max_T=1024, spare=16)
    n = sum(new)
    q, k, v = chunk_inputs(rng, c, n)
    ch = c.plan(new)
    attn_check(c, new, q, k, v, c.chunk_attn(ch, q, k, v))
    c.extend(ch, k, v)
    assert [sum(c.lens_host[4 * b: 4 * b + 3]) for b in range(200)] == [x + y for x, y in zip(lens, new)]
    assert c.read_status() == 0


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 32, 33, 63, 64, 65])
def test_row_counts(rows):
    """Every form of a unit (copies of its rows, one tile, two), cut into ranges and whole."""
    rng = np.random.default_rng(rows)
    c = make_cache(rng, [3000, 120], H_q=4, H_kv=1)
    new = [rows, rows]
    q, k, v = chunk_inputs(rng, c, 2 * rows)
    attn_check(c, new, q, k, v, c.chunk_attn(c.plan(new), q, k, v))


RANGES = {
    "whole": dict(lens=[300], new=[4]),
    "parts_of_two": dict(lens=[2000], new=[4]),
    "parts_and_whole": dict(lens=[3000, 0, 250], new=[2, 0, 5]),
    "short_slots": dict(lens=[300, 900, 100, 500], new=[1, 1, 1, 1]),
    "wide": dict(lens=[0], new=[200]),
    "wide_and_narrow": dict(lens=[2100, 40, 700], new=[301, 3, 20]),
    "long_units": dict(lens=[9000, 40], new=[3, 1]),
    "a_unit_per_range": dict(lens=[200] * 19, new=[1] * 19),
    "more_units": dict(lens=[200] * 20, new=[1] * 20),
}


@pytest.mark.parametrize("name", RANGES)
def test_ranges(name):
    """Units whole, in parts of their own, and cut evenly: the attention, and that a second call
    gives the same bits."""
    rng = np.random.default_rng(len(name))
    case = RANGES[name]
    c = make_cache(rng, case["lens"], H_q=16, H_kv=8, max_T=16384)
    q, k, v = chunk_inputs(rng, c, sum(case["new"]))
    ch = c.plan(case["new"])
    out = c.chunk_attn(ch, q, k, v)
    attn_check(c, case["new"], q, k, v, out, name)
    assert torch.equal(out, c.chunk_attn(ch, q, k, v))
    assert c.read_status() == 0


def test_out_may_not_overlap():
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(14)
    c = make_cache(rng, [100])
    q, k, v = (x.contiguous() for x in chunk_inputs(rng, c, 4))
    ch = c.plan([4])
    big = torch.cat([q, q])
    for x, out in ((q, q), (big[:4], big[3:7])):
        with pytest.raises(kvq.KvqError) as e:
            c.chunk_attn(ch, x, k, v, out=out)
        assert e.value.code == -1


def test_two_streams():
    """Two caches on two streams at once, with a chunk each."""
    rng = np.random.default_rng(15)
    cs = [make_cache(np.random.default_rng(i), [2000, 40], max_T=4096) for i in range(2)]
    io = [chunk_inputs(rng, cs[0], 60) for _ in range(2)]
    chunks = [c.plan([50, 10]) for c in cs]
    outs = [torch.zeros(60, 8, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                cs[i].chunk_attn(chunks[i], *io[i], out=outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        attn_check(cs[i], [50, 10], *io[i], outs[i])


def test_plan_and_extend_refuse_capture():
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(5)
    c = make_cache(rng, [100])
    q, k, v = chunk_inputs(rng, c, 4)
    ch = c.plan([4])
    state = list(c.lens_host)
    codes = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (lambda: c.plan([4], ch), lambda: c.extend(ch, k, v)):
            try:
                call()
                codes.append(0)
            except kvq.KvqError as e:
                codes.append(e.code)
    assert codes == [-2, -2]
    assert list(c.lens_host) == state
    c.extend(ch, k, v)  # and the plan still holds


def test_pool_exhausted_and_capacity():
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(6)
    c = make_cache(rng, [100, 0], max_T=512, spare=1)
    free = list(c.free)
    with pytest.raises(kvq.KvqError) as e:
        c.plan([300, 0])
    assert e.value.code == -3 and c.free == free
    with pytest.raises(kvq.KvqError) as e:
        c.plan([0, 1000])  # past max_T
    assert e.value.code == -3 and c.free == free
    with pytest.raises(kvq.KvqError) as e:
        c.plan([0, 9], c.new_chunk(8))
    assert e.value.code == -3


def test_run_together():
    """A prompt in chunks beside decoding slots, then decode steps with append and flush:
    each chunk's attention, the final cache against one prefill, and its decode attention."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(10)
    lens = [0, 500, 127]
    c = make_cache(rng, lens, H_q=8, H_kv=2, bits=4, S=4)
    w_q, w_k = randn(rng, 128), randn(rng, 128)
    prompt_k, prompt_v = [], []
    chunk = c.new_chunk(400)
    for new in ([130, 1, 1], [301, 5, 0], [1, 1, 3], [64, 0, 130]):
        n = sum(new)
        q, k, v = chunk_inputs(rng, c, n, n + 2)
        kept = {b: cached_rows(c, b) for b in range(3)}
        base = [sum(c.lens_host[4 * b + i] for i in range(3)) for b in range(3)]
        # the rotated rows, for the check (the operator has its own tests)
        pos = torch.tensor([base[b] + i for b in range(3) for i in range(new[b])], dtype=torch.int32, device=DEV)
        qr, kr = kvq.qk_norm_rope(q[:n], k[:n], w_q, w_k, pos, rope_base=500000.0, halves=True)
        twin = c.plan(new)
        attn = c.chunk_attn(twin, qr, kr, v)
        attn_check(c, new, qr, kr, v[:n], attn)
        out, chunk = c.chunk_step(new, q, k, v, w_q, w_k, rope_base=500000.0, halves=True, chunk=chunk)
        assert torch.equal(out[:n], attn)
        assert torch.equal(chunk.pos[:n], pos)
        prompt_k.append(kr[: new[0]])
        prompt_v.append(v[: new[0]])
        for b in range(3):  # what was cached before is still the front of the cache
            L = kept[b][0].shape[1]
            same = min(L, 4)
            assert np.array_equal(cached_rows(c, b)[0][:, :same], kept[b][0][:, :same])
    # slot 0 holds what a prefill of the same rows holds
    k = torch.cat(prompt_k).transpose(0, 1).contiguous()
    v = torch.cat(prompt_v).transpose(0, 1).contiguous()
    ref = kvq.KVQPagedCache(1, 8, 2, 128, 128, 4, n_pages=16, max_T=4096, S=4, device=DEV)
    ref.prefill(0, k, v)
    assert ref.lengths(0) == c.lengths(0)
    for x, y in zip(cached_rows(ref, 0), cached_rows(c, 0)):
        assert np.array_equal(x, y)
    for _ in range(3):
        q, k, v = (x.contiguous() for x in chunk_inputs(rng, c, 3))
        want = c.chunk_attn(c.plan([1, 1, 1]), q, k, v)
        c.append(k, v)
        got = c.decode_attn(q)
        assert torch.all((got - want).float().abs() <= 2e-3 + 2e-3 * want.float().abs())
        c.flush()
    assert c.read_status() == 0


def test_clear_and_refill():
    rng = np.random.default_rng(11)
    c = make_cache(rng, [0, 0])
    q, k, v = chunk_inputs(rng, c, 300)
    c.extend(c.plan([200, 100]), k, v)
    first = [cached_rows(c, b) for b in range(2)]
    pages = [list(p) for p in c.pages]
    c.clear(unmap=False)
    assert not any(c.lens_host) and not c.lens.any()
    c.extend(c.plan([200, 100]), k, v)
    assert [list(p) for p in c.pages] == pages
    for b in range(2):
        assert np.array_equal(first[b][0], cached_rows(c, b)[0]) and np.array_equal(first[b][1], cached_rows(c, b)[1])
    free = len(c.free)
    c.clear()
    assert len(c.free) == free + sum(map(len, pages)) and sorted(c.free) == list(range(c.n_pages))
    c.prefill(1, k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous())
    assert c.lengths(1)["T"] == 256


def test_callers_pages():
    """Pages that the caller hands out: the cache's own list stays out of it."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(12)
    c = make_cache(rng, [0], spare=8)
    q, k, v = chunk_inputs(rng, c, 300)
    pages = torch.tensor([6, 2], dtype=torch.int32, device=DEV)
    with pytest.raises(kvq.KvqError):
        c.plan([300], pages=pages[:1])
    c.extend(c.plan([300], pages=pages), k, v)
    assert c.table[0, :2].tolist() == [6, 2]
    with pytest.raises(kvq.KvqError):
        c.plan([300])
    assert c.lengths(0)["T"] == 256 and c.read_status() == 0


@pytest.mark.parametrize("n", [1, 100, 128, 300])
@pytest.mark.parametrize("R,bits", [(128, 2), (128, 4), (128, 8), (256, 2)])
def test_extend_over_a_full_residual(R, bits, n):
    """A residual that append has filled and nothing has flushed: extend packs it and refills
    it in the same call."""
    caches = [make_cache(np.random.default_rng(1), [R - 2, 40], R=R, bits=bits, S=0) for _ in range(2)]
    rng = np.random.default_rng(n)
    tokens = [(randn(rng, 2, 2, 128), randn(rng, 2, 2, 128)) for _ in range(R // 128 * 128 - (R - 2) % 128)]
    q, k, v = chunk_inputs(rng, caches[0], n + 3)
    for c in caches:
        while c.lens_host[2] < R:
            c.append(*tokens[c.lens_host[2] % len(tokens)])
    a, b = caches
    assert a.lengths(0)["n_res"] == R
    b.flush()
    for c in caches:
        c.extend(c.plan([n, 3]), k, v)
        assert c.read_status() == 0
    assert list(a.lens_host) == list(b.lens_host)
    for s in range(2):
        for x, y in zip(cached_rows(a, s), cached_rows(b, s)):
            assert np.array_equal(x, y)


def test_callers_pages_until_cleared():
    """Calls that need no page work beside the caller's pages; an emptied cache has its own list
    again, and a chunk planned before is stale."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(34)
    c = make_cache(rng, [0, 0], spare=8)
    q, k, v = chunk_inputs(rng, c, 300)
    ch = c.plan([300, 0], pages=torch.tensor([6, 2], dtype=torch.int32, device=DEV))
    c.extend(ch, k, v)
    rows = [randn(rng, 2, 200, 128) for _ in range(2)]
    c.prefill(1, *(x[:, :5].contiguous() for x in rows))
    c.append(randn(rng, 2, 2, 128), randn(rng, 2, 2, 128))
    assert c.flush() == [] and c.lengths(1)["n_res"] == 6
    c.release(1)
    with pytest.raises(kvq.KvqError):
        c.prefill(1, *rows)
    c.clear(unmap=False)
    with pytest.raises(kvq.KvqError):
        c.plan([300, 0])
    stale = c.plan([130, 0], pages=torch.tensor([6, 2], dtype=torch.int32, device=DEV))
    c.clear()
    with pytest.raises(kvq.KvqError):
        c.extend(stale, k, v)
    c.prefill(1, *rows)
    c.extend(c.plan([300, 0]), k, v)
    assert c.lengths(0)["T"] == 256 and c.lengths(1)["T"] == 128
    assert sorted(c.free + c.pages[0] + c.pages[1]) == list(range(8))
    assert c.table[0, :2].tolist() == c.pages[0] and c.table[1, :1].tolist() == c.pages[1]
    assert c.read_status() == 0


def test_refused_plan_leaves_a_capture_alone():
    """A plan that would take pages from the cache's list, or make a chunk, is refused while the
    stream is captured like any other, and the capture goes on."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(35)
    c = make_cache(rng, [100])
    q, k, v = chunk_inputs(rng, c, 40)
    ch = c.new_chunk(40)
    free = list(c.free)
    x = torch.zeros(4, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x += 1
        for call in (lambda: c.plan([40], ch), lambda: c.plan([4]), lambda: c.chunk_step([40], q, k, v)):
            with pytest.raises(kvq.KvqError) as e:
                call()
            assert e.value.code == -2
    graph.replay()
    assert x.tolist() == [1.0] * 4 and c.free == free and c.pages == [[]]
    c.extend(c.plan([40], ch), k, v)
    assert c.lengths(0)["T"] == 128 and c.read_status() == 0


def test_step_without_tokens():
    """A padded batch in which no slot has a token: no rows out, or the caller's left alone."""
    rng = np.random.default_rng(36)
    c = make_cache(rng, [100, 0])
    state = list(c.lens_host)
    q, k, v = chunk_inputs(rng, c, 0, 3)
    out, chunk = c.chunk_step([0, 0], q, k, v)
    assert out.shape == (0, c.cfg.H_q, 128) and out.dtype == torch.float16 and chunk.n_tokens == 0
    mine = torch.full((3, c.cfg.H_q, 128), 7.0, dtype=torch.float16, device=DEV)
    out, chunk = c.chunk_step([0, 0], q, k, v, chunk=chunk, out=mine)
    assert out is mine and (mine == 7.0).all()
    out, _ = c.chunk_step([2, 0], q, k, v, chunk=c.new_chunk(3))
    assert out.shape[0] == 2 and state != list(c.lens_host) and c.read_status() == 0


def test_values_not_finite_in_some_of_many_units():
    """Ranges of many short units, wide ones among them: an infinite or NaN value reaches the rows
    of its own slot that see it, in whichever unit of a range it lies."""
    rng = np.random.default_rng(37)
    new = [70 if b % 9 == 4 else 1 + b % 3 for b in range(90)]
    c = make_cache(rng, [int(x) for x in rng.integers(0, 120, 90)], H_q=16, H_kv=4, max_T=512)
    n = sum(new)
    q, k, v = (x.clone() for x in chunk_inputs(rng, c, n))
    at = np.cumsum([0] + new)
    for b in list(range(0, 90, 7)) + [4, 5, 6, 9, 13, 14]:
        v[at[b] + new[b] // 2, b % 4, b] = [float("inf"), float("nan"), float("-inf")][b % 3]
    c.view("v_res")[20, 1, 0, 3] = float("inf")
    assert c.lengths(20)["n_res"] > 0
    ch = c.plan(new)
    out = c.chunk_attn(ch, q, k, v)
    attn_check(c, new, q, k, v, out)
    assert torch.equal(out.view(torch.int16), c.chunk_attn(ch, q, k, v).view(torch.int16))


def test_default_device():
    """A cache made without a device index takes the tensors of the current device in every call,
    chunk calls and the others alike."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(38)
    with torch.cuda.device(0):
        c = kvq.KVQPagedCache(2, 8, 2, 128, 128, 2, n_pages=8, max_T=512)
        q, k, v = (x.contiguous() for x in chunk_inputs(rng, c, 4))
        c.prefill(0, randn(rng, 2, 200, 128), randn(rng, 2, 200, 128))
        out, _ = c.chunk_step([1, 3], q, k, v)
        attended = c.decode_attn(q[:2])
        c.append(k[:2], v[:2])
        dense = kvq.KVQCache(1, 8, 2, 128, 128, 2, max_T=512)
        dense.prefill(randn(rng, 1, 2, 200, 128), randn(rng, 1, 2, 200, 128))
        dense.decode_attn(q[:1])
    assert out.device == attended.device == torch.device(DEV)
    assert c.lengths(0) == dict(n_sink=0, T=128, n_res=74, active=1) and c.read_status() == 0
