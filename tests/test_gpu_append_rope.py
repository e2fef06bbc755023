"""One token per slot with norm and rotation on the way: against flush, qk_norm_rope and append
(bit for bit), against the formula in 64 bits, and in a run with decode attention."""
import math

import numpy as np
import pytest
import torch

import block_util
import chunk_util
from block_util import D, DEV, bound_of, cached_rows, randn, softmax_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def build(rng, lens, mode, spare=64, **kw):
    if mode in ("e4m3", "int8"):
        return block_util.make_cache(rng, lens, mode, spare=spare, **kw)
    kb, vb = mode
    return chunk_util.make_cache(rng, lens, bits=kb, v_bits=vb, spare=spare, **kw)


def two(lens, mode, seed=1, **kw):
    return [build(np.random.default_rng(seed), lens, mode, **kw) for _ in range(2)]


def full_residuals(c, slots, rng):
    """Fills the residuals of these slots by appends (the others take tokens as well, until theirs are full)."""
    while any(c.lengths(b)["n_res"] < c.cfg.R for b in slots):
        x = randn(rng, 2, c.cfg.B, c.cfg.H_kv, D)
        hold = {b: c.lens_host[4 * b + 3] for b in range(c.cfg.B)}
        for b in range(c.cfg.B):
            if c.lengths(b)["n_res"] == c.cfg.R:
                c.lens_host[4 * b + 3] = 0
        push(c)
        c.append(x[0], x[1])
        for b, on in hold.items():
            c.lens_host[4 * b + 3] = on
        push(c)


def push(c):
    c.lens.copy_(torch.tensor(list(c.lens_host), dtype=torch.int32).view(-1, 4))


def rows(rng, c):
    """q, k, v as views of one projection's rows; the rows of empty slots hold NaN."""
    H_q, H = c.cfg.H_q, c.cfg.H_kv
    x = randn(rng, c.cfg.B, H_q + 2 * H + 3, D)
    for b in range(c.cfg.B):
        if not c.lengths(b)["active"]:
            x[b] = float("nan")
    return x[:, :H_q], x[:, H_q:H_q + H], x[:, H_q + H:H_q + 2 * H]


def plain_steps(c, q, k, v, rope, w_q, w_k, **kw):
    """The same by the calls that there are for each part."""
    import bit_kv_cache_gb300 as kvq
    c.flush()
    pos = torch.tensor([sum(c.lens_host[4 * b: 4 * b + 3]) for b in range(c.cfg.B)], dtype=torch.int32, device=DEV)
    qr, kr = kvq.qk_norm_rope(q, k, w_q, w_k, pos, rope=rope, **kw)
    c.append(kr, v.contiguous())
    return qr


def same_state(a, b):
    assert list(a.lens_host) == list(b.lens_host) and torch.equal(a.lens, b.lens)
    for name in a.buf:
        assert torch.equal(a.buf[name], b.buf[name]), name
    for s in range(a.cfg.B):
        n = a.lengths(s)["T"] // a.cfg.G
        assert torch.equal(a.table[s, :n], b.table[s, :n])


ROPES = {
    "all": dict(rotary_dim=128),
    "halves_part_yarn": dict(rotary_dim=64, halves=True, base=500000.0, scaling=dict(kind="yarn", factor=16, original=4096)),
    "part16_bands": dict(rotary_dim=16, scaling=dict(kind="bands", factor=8, original=8192)),
    "halves_ntk": dict(rotary_dim=128, halves=True, scaling=dict(kind="ntk", factor=8)),
}


KINDS = [(mode, kw) for kw in [dict(G=128), dict(G=128, R=256, S=5), dict(G=256, R=512, S=3), dict(G=64), dict(G=64, R=192, S=70)]
         for mode in ["e4m3", "int8"] + ([] if kw["G"] == 64 else [(2, 2), (4, 8), (8, 2)])]  # pages of 64: the 8-bit modes'


@pytest.mark.parametrize("mode, kw", KINDS, ids=str)
def test_same_as_the_parts(mode, kw):
    import bit_kv_cache_gb300 as kvq
    R = kw.get("R", kw["G"])
    lens = [2 * R + 60, 0, 1, R + 1, 70, 0, 3 * R]
    a, b = two(lens, mode, **kw)
    for c in (a, b):
        full_residuals(c, [0, 3], np.random.default_rng(2))
    assert [a.lengths(s)["n_res"] == R for s in range(7)].count(True) >= 2
    rng = np.random.default_rng(3)
    for i, name in enumerate(list(ROPES) * 2):
        rope = kvq.Rope(**ROPES[name])
        q, k, v = rows(rng, a)
        w_q, w_k = (randn(rng, D), randn(rng, D)) if i % 2 else (None, randn(rng, D) if i == 2 else None)
        rot = dict(rotate_q=i != 4, rotate_k=i != 6)
        out = torch.full((7, a.cfg.H_q, D), 7.0, dtype=torch.float16, device=DEV)
        got = a.append_rope(q, k, v, rope, w_q, w_k, out=out, **rot)
        want = plain_steps(b, q, k, v, rope, w_q, w_k, **rot)
        for s in range(7):
            assert torch.all(got[s] == 7.0) if not lens[s] else torch.equal(got[s], want[s])
        same_state(a, b)
    assert a.read_status() == 0


@pytest.mark.parametrize("name", list(ROPES))
def test_against_the_formula(name):
    """Queries in 64 bits: the norm and sums of fp32 add 2^-20 of the row's size, the angle (2^-27
    turns, and what the frequency's own rounding makes) as much, the output half a step of fp16."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(4)
    rope = kvq.Rope(**ROPES[name])
    c = build(rng, [700, 64, 1], "e4m3", max_T=1 << 20)
    far = [0, (1 << 19) + 64, 64 * 5001]
    for s in range(3):
        if far[s]:
            c.lens_host[4 * s + 1] = far[s]
    push(c)
    q, k, v = rows(rng, c)
    w = randn(rng, D)
    pos = np.array([sum(c.lens_host[4 * s: 4 * s + 3]) for s in range(3)], np.float64)
    x = q.cpu().double().numpy()
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * w.cpu().double().numpy()
    n, y, a = rope.rotary_dim, x.copy(), pos[:, None] * np.array(rope.freq)
    lo, hi = (np.arange(n // 2), np.arange(n // 2) + n // 2) if rope.halves else (np.arange(0, n, 2), np.arange(1, n, 2))
    cs, sn = rope.amp * np.cos(a)[:, None], rope.amp * np.sin(a)[:, None]
    y[..., lo], y[..., hi] = x[..., lo] * cs - x[..., hi] * sn, x[..., lo] * sn + x[..., hi] * cs
    got = c.append_rope(q, k, v, rope, w, None, eps=1e-5).cpu().double().numpy()
    size = np.maximum(np.abs(x), 0)
    size[..., lo] = size[..., hi] = np.hypot(x[..., lo], x[..., hi]) * abs(rope.amp)
    assert np.all(np.abs(got - y) <= 2.0 ** -11 * np.abs(y) + size * 2.0 ** -20 + 2.0 ** -25)


def test_pages_of_the_caller_and_refusals():
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(5)
    c = build(rng, [64, 200], "int8", max_T=256)
    full_residuals(c, [1], rng)  # T = 192, residual full: fits once
    q, k, v = rows(rng, c)
    before = list(c.lens_host)
    for bad, code in (([], -3), ([c.n_pages], -1), ([-1], -1)):
        with pytest.raises(kvq.KvqError) as e:
            c.append_rope(q, k, v, pages=bad)
        assert e.value.code == code
    for kw in (dict(q=q[:1]), dict(k=k.float()), dict(v=v.transpose(0, 1)), dict(out=torch.zeros(2, 8, 2 * D, dtype=torch.float16, device=DEV)[..., :D])):
        with pytest.raises(ValueError):
            c.append_rope(**{**dict(q=q, k=k, v=v), **kw})
    whole = torch.zeros(2, 12, D, dtype=torch.float16, device=DEV)
    with pytest.raises(kvq.KvqError):  # the output lies over the keys
        c.append_rope(whole[:, :8], whole.view(-1, D)[16:].view(-1)[: 2 * 2 * D].view(2, 2, D), v, out=whole.view(-1)[: 2 * 8 * D + 0].view(2, 8, D))
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(q, memory_format=torch.contiguous_format)
    torch.cuda.synchronize()
    with pytest.raises(kvq.KvqError) as e:
        with torch.cuda.graph(g, stream=s):
            c.append_rope(q, k, v, pages=[3], out=out)
    assert e.value.code == -2
    torch.cuda.synchronize()
    assert list(c.lens_host) == before
    page = c.free[0]
    c.append_rope(q, k, v, pages=torch.tensor([page], dtype=torch.int32))
    assert c.lengths(1) == dict(n_sink=0, T=256, n_res=1, active=1) and c.table[1, 3].item() == page
    full_residuals(c, [1], rng)
    with pytest.raises(kvq.KvqError) as e:  # past max_T
        c.append_rope(q, k, v, pages=[page])
    assert e.value.code == -3
    with pytest.raises(kvq.KvqError):  # the caller maps
        c.append_rope(q, k, v)


def test_in_place_and_contiguous():
    rng = np.random.default_rng(6)
    a, b = two([100, 5], "e4m3")
    q, k, v = rows(rng, a)
    q = q.contiguous()
    want = a.append_rope(q, k, v)
    got = b.append_rope(q, k, v, out=q)
    assert got is q and torch.equal(got, want)


def test_no_sequence():
    c = build(np.random.default_rng(0), [0, 0], "e4m3")
    q, k, v = rows(np.random.default_rng(1), c)
    assert torch.all(c.append_rope(q, k, v) == 0)


def test_many_full_residuals_of_several_pages():
    """More pages than one launch packs."""
    B, G, R = 300, 64, 256
    a, b = two([R] * B, "int8", G=G, R=R, H_q=1, H_kv=1, spare=B * R // G + 8, max_T=1024)
    for c in (a, b):  # prompts leave no full residual: unpack them by hand
        for s in range(B):
            c.lens_host[4 * s: 4 * s + 4] = [0, 0, R, 1] if s % 50 else [0, R, 3, 1]
        push(c)
        x = randn(np.random.default_rng(9), B, 1, R, D)
        c.view("k_res").copy_(x)
        c.view("v_res").copy_(x.flip(2))
        c.free, c.pages = list(range(c.n_pages)), [[] for _ in range(B)]
        for s in range(0, B, 50):
            c.pages[s] = [c.free.pop() for _ in range(R // G)]
    q, k, v = rows(np.random.default_rng(10), a)
    got = a.append_rope(q, k, v)
    want = plain_steps(b, q, k, v, None, None, None)
    assert torch.equal(got, want)
    same_state(a, b)
    assert a.read_status() == 0


def test_bad_page_is_reported_and_the_token_kept():
    """A page-table entry that is no page, mapped by the caller of the C call."""
    import ctypes
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(11)
    c = build(rng, [128], "e4m3")
    full_residuals(c, [0], rng)
    c.table[0, 2] = c.n_pages + 5
    q, k, v = (x.contiguous() for x in rows(rng, c))
    out = torch.empty_like(q)
    qk = kvq.QkConfig(8, 2, D, 0, 0, 0, 1e-6, 0.0, 8 * D, 2 * D)
    st = torch.cuda.current_stream().cuda_stream
    assert kvq.lib.kvq_paged_append_rope(*c._refs, ctypes.byref(qk), None, 1.0, q.data_ptr(), k.data_ptr(), v.data_ptr(), 2 * D, None,
                                         None, out.data_ptr(), None, 0, st) == 0
    assert c.read_status() == 2
    assert torch.equal(out, q) and torch.equal(c.view("k_res")[0, :, 0], k[0]) and torch.equal(c.view("v_res")[0, :, 0], v[0])


@pytest.mark.parametrize("mode", ["e4m3", "int8", (2, 2)], ids=str)
def test_decode_run(mode):
    """Prompts, then steps over several flushes: append with rotation, attention of the step."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(12)
    G = 128 if mode == (2, 2) else 64
    c = build(rng, [300, 0, 61, 128], mode, G=G, S=2)
    rope = kvq.Rope(128, halves=True, scaling=dict(kind="linear", factor=4))
    w = randn(rng, D)
    attn = chunk_util.cached_rows if mode == (2, 2) else cached_rows
    for step in range(G + 5):
        q, k, v = rows(rng, c)
        pos = torch.tensor([sum(c.lens_host[4 * b: 4 * b + 3]) for b in range(4)], dtype=torch.int32, device=DEV)
        out = c.decode_step(q, k, v, rope, w, w)
        if step % 23 and step < G - 2:
            continue
        qr, _ = kvq.qk_norm_rope(q, k, w, w, pos, rope=rope)
        for b in (0, 2, 3):
            K, V = attn(c, b)
            for h in range(2):
                ref, size, mag = softmax_rows(qr[b, 4 * h: 4 * h + 4].cpu().double().numpy(), K[h], V[h])
                err = np.abs(out[b, 4 * h: 4 * h + 4].cpu().double().numpy() - ref)
                bound = 2e-3 + 2e-3 * np.abs(ref) if mode == (2, 2) else bound_of(ref, size, mag)
                assert np.all(err <= bound), (step, b, h)
    assert c.read_status() == 0


@pytest.mark.parametrize("name", list(ROPES))
def test_chunk_step_with_scaled_positions(name):
    """A prompt by chunk_step and by append_rope, token by token, leave the same state."""
    import bit_kv_cache_gb300 as kvq
    rng = np.random.default_rng(13)
    a, b = two([64, 3], "int8")
    rope = kvq.Rope(**ROPES[name])
    x = randn(rng, 2, 100, 12, D)
    w = randn(rng, D)
    y = x.reshape(200, 12, D)
    a.chunk_step([100, 100], y[:, :8], y[:, 8:10], y[:, 10:], None, w, rope=rope)
    for t in range(100):
        b.append_rope(x[:, t, :8], x[:, t, 8:10], x[:, t, 10:], rope, None, w)
    b.flush()
    assert list(a.lens_host) == list(b.lens_host)
    for s in range(2):
        for r, o in zip(cached_rows(a, s), cached_rows(b, s)):
            assert np.array_equal(r, o)
