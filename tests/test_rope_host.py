"""Frequencies of scaled positions, and the host checks of the calls that take them (no GPU)."""
import ctypes
import math

import pytest

INVALID, UNSUPPORTED, CAPACITY = -1, -2, -3


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_gb300 as m
    return m


def test_plain_and_linear(kvq):
    f = kvq.Rope(64, base=500000.0).freq
    assert f[0] == 1.0 and len(f) == 32
    assert all(abs(x - 500000.0 ** (-j / 32)) <= 1e-15 * x for j, x in enumerate(f))
    g = kvq.Rope(64, base=500000.0, scaling=dict(kind="linear", factor=4)).freq
    assert all(abs(4 * y - x) <= 1e-15 * x for x, y in zip(f, g))


def test_ntk_keeps_the_first_pair_and_slows_the_last(kvq):
    f, g = kvq.Rope(128).freq, kvq.Rope(128, scaling=dict(kind="ntk", factor=8)).freq
    assert g[0] == f[0] and abs(g[-1] * 8 / f[-1] - 1) < 1e-12 and all(y < x for x, y in zip(f[1:], g[1:]))


def test_bands_by_wavelength(kvq):
    r = kvq.Rope(128, base=500000.0, scaling=dict(kind="bands", factor=8, original=8192))
    f = kvq.Rope(128, base=500000.0).freq
    for x, y in zip(f, r.freq):
        turns = 8192 * x / (2 * math.pi)
        if turns >= 4:
            assert y == x
        elif turns <= 1:
            assert abs(8 * y / x - 1) < 1e-14
        else:
            assert x / 8 < y < x
    assert r.amp == 1.0


def test_yarn_by_index(kvq):
    r = kvq.Rope(128, scaling=dict(kind="yarn", factor=16, original=4096))
    f = kvq.Rope(128).freq
    ratio = [y / x for x, y in zip(f, r.freq)]
    assert ratio[0] == 1.0 and abs(ratio[-1] * 16 - 1) < 1e-12 and all(a >= b - 1e-15 for a, b in zip(ratio, ratio[1:]))
    # pairs that turn 32 times and more within the original length keep their frequency, below one turn all is scaled
    assert all(a > 1 - 1e-9 for x, a in zip(f, ratio) if 4096 * x / (2 * math.pi) > 32 * 1.2)
    assert all(abs(16 * a - 1) < 1e-9 for x, a in zip(f, ratio) if 4096 * x / (2 * math.pi) < 1 / 1.2)
    assert abs(r.amp - (0.1 * math.log(16) + 1)) < 1e-15
    assert kvq.Rope(128, scaling=dict(kind="yarn", factor=16, original=4096), amp=1.0).amp == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=0.0), dict(rotary_dim=64, base=float("inf")),
                                dict(rotary_dim=64, scaling=dict(kind="other", factor=2)), dict(rotary_dim=64, scaling=dict(factor=2)),
                                dict(rotary_dim=64, scaling=dict(kind="linear")), dict(rotary_dim=64, scaling=dict(kind="linear", factor=0)),
                                dict(rotary_dim=64, scaling=dict(kind="linear", factor=2, slow=1)),
                                dict(rotary_dim=64, scaling=dict(kind="bands", factor=2, original=100, low=4, high=4)),
                                dict(rotary_dim=2, scaling=dict(kind="ntk", factor=2)),
                                dict(rotary_dim=64, base=1.0, scaling=dict(kind="yarn", factor=2, original=100)),
                                dict(rotary_dim=64, freq=[1.0] * 31), dict(rotary_dim=4, freq=[1.0, -1.0]),
                                dict(rotary_dim=4, freq=[1.0, float("nan")]), dict(rotary_dim=4, freq=[1.0, 1.0], scaling=dict(kind="linear", factor=2)),
                                dict(rotary_dim=64, amp=float("nan"))], ids=str)
def test_refused_ropes(kvq, kw):
    with pytest.raises(ValueError):
        kvq.Rope(**kw)


B, H_q, H_kv, D = 4, 16, 2, 128


class Fake:
    """A paged cache whose device pointers are aligned placeholders (no refused call reads them)."""

    def __init__(self, kvq, lens, mode="e4m3", G=64, R=64, S=0, max_T=1024, n_pages=9):
        self.kvq = kvq
        self.cfg = kvq.make_config(B, H_q, H_kv, D, G, 8, S, R, 0, mode, max_T, 0)
        self.p = kvq.Paged()
        for i, name in enumerate(("k_codes", "k_meta", "v_codes", "v_meta", "page_table", "k_sink", "v_sink", "k_res", "v_res",
                                  "lens", "status")):
            setattr(self.p, name, 0x10000 * (i + 1))
        self.p.n_pages = n_pages
        self.lens = (ctypes.c_int32 * (4 * B))(*[x for l in lens for x in l])
        self.p.lens_host = ctypes.cast(self.lens, ctypes.c_void_p)
        self.qk = kvq.QkConfig(H_q, H_kv, D, 128, 0, 3, 1e-6, 10000.0, H_q * D, H_kv * D)

    def append(self, q=0x1000000, k=0x2000000, v=0x3000000, vs=H_kv * D, w=None, out=0x4000000, pages=(), freq=None, amp=1.0, qk=None):
        ids = None if pages is None else (ctypes.c_int32 * max(1, len(pages)))(*pages)
        freq = None if freq is None else (ctypes.c_double * 64)(*freq)
        return self.kvq.lib.kvq_paged_append_rope(ctypes.byref(self.cfg), ctypes.byref(self.p), ctypes.byref(qk or self.qk), freq, amp, q, k,
                                                  v, vs, w, None, out, ids, 0 if pages is None else len(pages), None)


LENS = [(0, 256, 40, 1), (0, 64, 64, 1), (0, 0, 0, 0), (0, 128, 64, 1)]


def test_append_rope_refusals(kvq):
    f = Fake(kvq, LENS)
    before = list(f.lens)
    assert f.append(pages=[1]) == CAPACITY                       # two residuals are full
    assert f.append(pages=[1, 9]) == INVALID and f.append(pages=[-1, 2]) == INVALID
    ok = dict(pages=[1, 2])
    for kw in (dict(q=None), dict(q=0x1000008), dict(k=None), dict(v=None), dict(vs=H_kv * D - 8), dict(vs=H_kv * D + 4), dict(w=0x5000002),
               dict(out=None), dict(out=0x4000004), dict(out=0x1000000 + 256), dict(out=0x2000000), dict(out=0x3000000 + 512), dict(out=0x5000000, w=0x5000010),
               dict(w=0x4000010),
               dict(amp=float("inf")), dict(freq=[-1.0] * 64), dict(freq=[float("nan")] * 64), dict(freq=[3e9] * 64)):
        assert f.append(**{**ok, **kw}) == INVALID, kw
    for name, bad, code in (("H_q", 8, INVALID), ("H_kv", 4, INVALID), ("D", 64, INVALID), ("rotary_dim", 136, INVALID),
                            ("rotary_dim", 24, UNSUPPORTED), ("halves", 2, INVALID), ("rotate", 4, INVALID), ("eps", -1.0, INVALID),
                            ("rope_base", -2.0, INVALID), ("q_stride", H_q * D - 8, INVALID), ("k_stride", 4, INVALID)):
        qk = kvq.QkConfig(H_q, H_kv, D, 128, 0, 3, 1e-6, 10000.0, H_q * D, H_kv * D)
        setattr(qk, name, bad)
        assert f.append(**ok, qk=qk) == code, name
    f.lens[4 + 1] = 1024  # a full slot at max_T
    assert f.append(**ok) == CAPACITY
    f.lens[4 + 1] = 65    # packed tokens that are not whole pages
    assert f.append(**ok) == INVALID
    f.lens[4 + 1] = 64
    f.p.n_pages = 0
    assert f.append(**ok) == CAPACITY
    f.p.n_pages = 9
    f.p.k_res = 0x8
    assert f.append(**ok) == INVALID
    assert list(f.lens) == before
    g = Fake(kvq, [(0, 0, 64 * 1025, 1)] + [(0, 0, 0, 0)] * 3, R=64 * 1025, max_T=64 * 4096, n_pages=5000)
    assert g.append(pages=list(range(1025))) == UNSUPPORTED


def test_block_mode_configurations(kvq):
    L = kvq.lib

    def paged(**kw):
        a = dict(dict(B=2, H_q=8, H_kv=2, D=128, G=64, bits=8, S=0, R=64, mode="e4m3", max_T=1024), **kw)
        return L.kvq_paged_bytes(ctypes.byref(kvq.make_config(**a)), 10, 0)

    for mode in ("e4m3", "int8"):
        assert paged(mode=mode) == 10 * 2 * 64 * 128 and paged(mode=mode, G=256, R=256) == 10 * 2 * 256 * 128
        assert paged(mode=mode, H_q=16) and paged(mode=mode, v_bits=8) and paged(mode=mode, R=192, S=7)
        for kw in (dict(G=32, R=64), dict(G=512, R=512, max_T=1024), dict(D=64), dict(H_q=18), dict(H_q=7), dict(bits=4), dict(v_bits=4), dict(R=96),
                   dict(R=0), dict(max_T=1000), dict(max_T=0), dict(B=513), dict(B=0), dict(S=-1), dict(n_boost=4), dict(rope_base=1e4)):
            assert paged(mode=mode, **kw) == 0, kw
        cfg = kvq.make_config(2, 8, 2, 128, 64, 8, 3, 64, 0, mode, 1024)
        size = lambda which: L.kvq_paged_bytes(ctypes.byref(cfg), 10, which)  # noqa: E731
        assert size(3) == size(5) == 10 * 2 * 16 and size(4) == size(0) and size(6) == 2 * 2 * 3 * 256 and size(7) == 2 * 2 * 64 * 256
        assert L.kvq_config_check(ctypes.byref(cfg)) == UNSUPPORTED  # no dense cache
        assert L.kvq_buffer_bytes(ctypes.byref(cfg), 0) == 0 and L.kvq_decode_attn_workspace_bytes(ctypes.byref(cfg)) == 0
        assert L.kvq_paged_workspace_bytes(ctypes.byref(cfg)) > 0 and L.kvq_paged_chunk_workspace_bytes(ctypes.byref(cfg)) > 0


def test_block_decode_refusals(kvq):
    f = Fake(kvq, LENS)
    L = kvq.lib
    size = L.kvq_paged_workspace_bytes(ctypes.byref(f.cfg))

    def decode(q=0x1000000, out=0x2000000, ws=0x3000000, n=size):
        return L.kvq_paged_decode_attn(ctypes.byref(f.cfg), ctypes.byref(f.p), q, out, ws, n, None)

    assert decode(q=None) == INVALID and decode(out=0x2000008) == INVALID and decode(q=0x1000002) == INVALID
    assert decode(out=0x1000000 + 256) == INVALID and decode(q=0x2000000 + 4 * H_q * D * 2 - 16) == INVALID
    assert decode(ws=None) == -4 and decode(n=size - 1) == -4 and decode(ws=0x3000004) == -4
    f.p.n_pages = 0
    assert decode() == INVALID  # packed tokens, and no page
