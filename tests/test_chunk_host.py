"""Host-side checks of the chunk operators' ABI (no GPU): sizes, and every argument,
capacity and consistency error before anything is enqueued."""
import ctypes

import pytest

INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_gb300 as m
    return m


B, H_q, H_kv, D, G = 4, 32, 8, 128, 128


class Fake:
    """A paged cache and a chunk whose device pointers are aligned placeholders (no host
    check dereferences them)."""

    def __init__(self, kvq, lens, S=0, R=128, max_T=4096, max_tokens=100, **kw):
        self.kvq = kvq
        self.cfg = kvq.make_config(B, H_q, H_kv, D, kw.get("G", G), 2, S, R, 0, "kivi", max_T, 0)
        self.p = kvq.Paged()
        for i, name in enumerate(("k_codes", "k_meta", "v_codes", "v_meta", "page_table", "k_sink", "v_sink",
                                  "k_res", "v_res", "lens", "status")):
            setattr(self.p, name, 0x10000 * (i + 1))
        self.p.n_pages = 64
        self.lens = (ctypes.c_int32 * (4 * B))(*[x for l in lens for x in l])
        self.p.lens_host = ctypes.cast(self.lens, ctypes.c_void_p)
        self.host = (ctypes.c_int32 * (8 * B))()
        self.ch = kvq.ChunkDesc(0x100000, 0x110000, 0x120000, 0x130000, ctypes.cast(self.host, ctypes.c_void_p), max_tokens, 0)
        self.S, self.R = S, R

    def planned(self, n_new):
        """The host side of a plan, as kvq_paged_plan leaves it."""
        cu = page = 0
        for b, n in enumerate(n_new):
            ns, T, nr, on = self.lens[4 * b: 4 * b + 4]
            if not on:
                ns = T = nr = 0
            sink = min(n, self.S - ns)
            pk = (nr + n - sink) // self.R * self.R if n else 0
            self.host[8 * b: 8 * b + 8] = [ns, T, nr, n, cu, sink, pk, page]
            cu += n
            page += pk // G
        self.ch.n_tokens = cu
        return self

    def plan(self, n_new, pages=0x500000, n_pages=64):
        n = (ctypes.c_int32 * B)(*n_new)
        return self.kvq.lib.kvq_paged_plan(ctypes.byref(self.cfg), ctypes.byref(self.p), n, pages, n_pages,
                                           ctypes.byref(self.ch), None)

    def attn(self, q=0x600000, qs=H_q * D, k=0x700000, ks=H_kv * D, v=0x800000, vs=H_kv * D, out=0x900000, ws=0xA00000, wsb=None):
        L = self.kvq.lib
        wsb = L.kvq_paged_chunk_workspace_bytes(ctypes.byref(self.cfg)) if wsb is None else wsb
        return L.kvq_paged_chunk_attn(ctypes.byref(self.cfg), ctypes.byref(self.p), ctypes.byref(self.ch), q, qs, k, ks, v, vs,
                                      out, ws, wsb, None)

    def extend(self, k=0x700000, ks=H_kv * D, v=0x800000, vs=H_kv * D):
        return self.kvq.lib.kvq_paged_extend(ctypes.byref(self.cfg), ctypes.byref(self.p), ctypes.byref(self.ch), k, ks, v, vs, None)


LENS = [(0, 256, 40, 1), (0, 0, 5, 1), (0, 0, 0, 0), (0, 128, 128, 1)]


def test_plan_refusals(kvq):
    f = Fake(kvq, LENS)
    before = list(f.lens), list(f.host)
    assert f.plan([1, -1, 0, 0]) == INVALID
    assert f.plan([60, 41, 0, 0]) == CAPACITY            # 101 tokens, room for 100
    assert f.plan([90, 0, 0, 1], n_pages=1) == CAPACITY  # two slots pack a page each
    f.ch.max_tokens = 1 << 30
    assert f.plan([4000, 0, 0, 0]) == CAPACITY           # past max_T
    assert f.plan([(1 << 31) - 1, 0, 0, 0]) == CAPACITY
    f.ch.max_tokens = 100
    assert kvq.lib.kvq_paged_plan(ctypes.byref(f.cfg), ctypes.byref(f.p), None, None, 0, ctypes.byref(f.ch), None) == INVALID
    assert f.plan([1, 0, 0, 0], pages=0x500002) == INVALID
    for name, bad in (("cu", None), ("slot", 0x110004), ("desc", 0x130008), ("host", None), ("max_tokens", -1)):
        keep = getattr(f.ch, name)
        setattr(f.ch, name, bad)
        assert f.plan([1, 0, 0, 0]) == INVALID, name
        setattr(f.ch, name, keep)
    f.lens[1] = 100  # packed tokens that are not whole pages
    assert f.plan([1, 0, 0, 0]) == INVALID
    f.lens[1] = 256
    assert (list(f.lens), list(f.host)) == before and f.ch.n_tokens == 0


@pytest.mark.parametrize("kw", [dict(H_q=40, H_kv=8), dict(D=64), dict(mode="kitty", R=64), dict(G=32, R=128), dict(rope_base=1e4)])
def test_unsupported_configurations(kvq, kw):
    a = dict(dict(B=B, H_q=H_q, H_kv=H_kv, D=D, G=G, bits=2, S=0, R=128, n_boost=0, mode="kivi", max_T=4096), **kw)
    cfg = kvq.make_config(**a)
    assert kvq.lib.kvq_paged_chunk_workspace_bytes(ctypes.byref(cfg)) == 0
    f = Fake(kvq, LENS)
    f.cfg = cfg
    assert f.plan([1, 1, 1, 1]) < 0
    f.planned([1, 1, 1, 1])
    assert f.attn(wsb=1 << 40) < 0 and f.extend() < 0


def test_attention_and_extend_refusals(kvq):
    f = Fake(kvq, LENS).planned([2, 3, 1, 1])
    for call in (f.attn, f.extend):
        for kw in (dict(k=None), dict(v=None), dict(k=0x700008), dict(ks=H_kv * D - 8), dict(vs=H_kv * D + 4), dict(vs=0)):
            assert call(**kw) == INVALID, kw
    for kw in (dict(q=None), dict(q=0x600002), dict(qs=H_kv * D), dict(out=None), dict(out=0x900004)):
        assert f.attn(**kw) == INVALID, kw
    for out in (0x600000, 0x600000 + H_q * D * 2 * 6, 0x700000 - 16, 0x800000 + H_kv * D * 2 * 7 - 16):
        assert f.attn(out=out) == INVALID  # seven rows overlap an input
    assert f.attn(ws=None) == WORKSPACE and f.attn(wsb=64) == WORKSPACE and f.attn(ws=0xA00004) == WORKSPACE
    state = list(f.lens)
    # a plan for other lengths, other counts, another residual size
    f.lens[2] += 1
    assert f.attn() == INVALID and f.extend() == INVALID
    f.lens[2] -= 1
    f.ch.n_tokens += 1
    assert f.attn() == INVALID and f.extend() == INVALID
    f.ch.n_tokens -= 1
    f.cfg.R = 256
    assert f.attn() == INVALID and f.extend() == INVALID
    f.cfg.R = 128
    f.host[3] = -1
    assert f.attn() == INVALID and f.extend() == INVALID
    assert list(f.lens) == state


def test_captured_chunk_is_not_planned_again(kvq):
    f = Fake(kvq, LENS).planned([2, 3, 1, 1])
    f.ch.captured = 1
    state = list(f.host)
    assert f.plan([1, 1, 1, 1]) == UNSUPPORTED
    assert list(f.host) == state


def test_empty_chunk_enqueues_nothing(kvq):
    f = Fake(kvq, LENS).planned([0, 0, 0, 0])
    assert f.attn(q=None) == 0 and f.extend(k=None) == 0
    assert [tuple(f.lens[4 * b: 4 * b + 4]) for b in range(B)] == LENS


def test_extend_needs_pages(kvq):
    f = Fake(kvq, LENS).planned([100, 0, 0, 0])
    f.p.n_pages = 0
    assert f.extend() in (CAPACITY, UNSUPPORTED)  # without a device the capture query comes first


def test_qk_norm_rope_refusals(kvq):
    L = kvq.lib

    def call(n=4, q=0x100000, k=0x200000, wq=0x300000, wk=0x310000, pos=0x320000, qo=0x400000, ko=0x500000, **kw):
        c = dict(dict(H_q=4, H_kv=2, D=128, rotary_dim=128, halves=0, rotate=3, eps=1e-6, rope_base=1e4,
                      q_stride=512, k_stride=256), **kw)
        return L.kvq_qk_norm_rope(ctypes.byref(kvq.QkConfig(**c)), q, k, wq, wk, pos, n, qo, ko, None)

    assert L.kvq_qk_norm_rope(None, 0, 0, 0, 0, 0, 1, 0, 0, None) == INVALID
    for kw in (dict(n=-1), dict(H_q=-1), dict(H_q=0, H_kv=0), dict(rotary_dim=-16), dict(rotary_dim=144), dict(halves=2),
               dict(rotate=4), dict(eps=-1.0), dict(eps=float("nan")), dict(rope_base=-1.0), dict(rope_base=float("inf")),
               dict(q=None), dict(q=0x100002), dict(qo=None), dict(ko=0x500004), dict(wq=0x300002), dict(pos=None),
               dict(pos=0x320002), dict(q_stride=511), dict(q_stride=504), dict(k_stride=260)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=96, q_stride=512), dict(rotary_dim=24), dict(n=1 << 31)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=0, pos=None) == 0
    # overlaps: the outputs, an output with the other input, with a strided input, or shifted
    for kw in (dict(qo=0x400000, ko=0x400000), dict(ko=0x100000), dict(qo=0x200100), dict(qo=0x100000, q_stride=1024),
               dict(qo=0x100100), dict(qo=0x0ff100)):  # the outputs are 0x1000 and 0x800 bytes
        assert call(**kw) == INVALID, kw


def test_python_refusals(kvq):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 128, dtype=torch.float16)
    for call in (lambda: kvq._rows(x.float(), 2, 128, 4, x.device, "x"), lambda: kvq._rows(x, 2, 128, 5, x.device, "x"),
                 lambda: kvq._rows(x, 4, 128, 4, x.device, "x"), lambda: kvq._rows(x[:, :, ::2], 2, 64, 4, x.device, "x"),
                 lambda: kvq._rows(x.view(4, 256), 2, 128, 4, x.device, "x"),
                 lambda: kvq._rows(x.transpose(0, 1), 4, 128, 2, x.device, "x")):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(4, 6, 128, dtype=torch.float16)
    assert kvq._rows(wide[:, 2:4], 2, 128, 4, wide.device, "x") == (wide.data_ptr() + 2 * 256, 6 * 128)
    assert kvq._rows(x[:1], 2, 128, 1, x.device, "x")[1] == 256


@pytest.mark.parametrize("G", [64, 128, 256])
def test_nvfp4_configurations_are_unsupported(kvq, G):
    """Paged pages hold min-max codes; the chunk kernels know pages of 128 and 256 tokens."""
    cfg = kvq.make_config(B, H_q, H_kv, D, G, 4, 0, 256, 0, "nvfp4", 4096)
    L = kvq.lib
    assert L.kvq_config_check(ctypes.byref(cfg)) == 0  # a dense cache has this mode
    assert L.kvq_paged_chunk_workspace_bytes(ctypes.byref(cfg)) == 0
    assert L.kvq_paged_workspace_bytes(ctypes.byref(cfg)) == 0 and L.kvq_paged_bytes(ctypes.byref(cfg), 4, 0) == 0
    f = Fake(kvq, [(0, 256, 40, 1)] * B, R=256)
    f.cfg = cfg
    assert f.plan([1, 1, 1, 1]) == UNSUPPORTED
    f.planned([1, 1, 1, 1])
    assert f.attn(wsb=1 << 40) == UNSUPPORTED and f.extend() == UNSUPPORTED


def test_attention_needs_pages(kvq):
    """Packed tokens without a page pool: there is nothing that a table entry could stand for."""
    f = Fake(kvq, LENS)
    f.p.n_pages = 0
    assert f.planned([2, 3, 1, 1]).attn() == INVALID
    assert f.planned([0, 0, 0, 1]).attn() == INVALID


def host_cache(kvq, B):
    """A paged cache without device memory, for checks that come before any device work."""
    torch = pytest.importorskip("torch")
    c = kvq.KVQPagedCache.__new__(kvq.KVQPagedCache)
    c.torch, c.cfg, c._dev = torch, kvq.make_config(B, H_q, H_kv, D, G, 2, 0, 128, 0, "kivi", 4096, 0), torch.device("cpu")
    c.p = kvq.Paged()
    for i, name in enumerate(("k_codes", "k_meta", "v_codes", "v_meta", "page_table", "k_res", "v_res", "lens", "status")):
        setattr(c.p, name, 0x10000 * (i + 1))
    c.lens_host = (ctypes.c_int32 * (4 * B))()
    c.p.lens_host = ctypes.cast(c.lens_host, ctypes.c_void_p)
    c.p.n_pages = 8
    c._refs = ctypes.byref(c.cfg), ctypes.byref(c.p)
    c.caller_pages, c.mapping = False, 0
    c.free, c.pages = list(range(8)), [[] for _ in range(B)]
    return c


@pytest.mark.parametrize("caller", [False, True])
def test_chunk_of_another_configuration(kvq, caller):
    """A chunk has arrays for its own number of slots; every call that reads them says so."""
    torch = pytest.importorskip("torch")
    c = host_cache(kvq, 6)
    c.caller_pages = caller
    rows = lambda h: torch.zeros(3, h, D, dtype=torch.float16)  # noqa: E731
    ch = kvq.KVQChunk(host_cache(kvq, 2).cfg, 3, "cpu")
    ch.cache = c
    for call in (lambda: c.plan([1, 1, 1, 0, 0, 0], ch), lambda: c.chunk_attn(ch, rows(H_q), rows(H_kv), rows(H_kv)),
                 lambda: c.extend(ch, rows(H_kv), rows(H_kv))):
        with pytest.raises(ValueError, match="another configuration"):
            call()
    ch = kvq.KVQChunk(c.cfg, 3, "meta")
    ch.cache = c
    with pytest.raises(ValueError, match="another configuration"):
        c.chunk_attn(ch, rows(H_q), rows(H_kv), rows(H_kv))


def test_no_page_needs_no_list(kvq):
    """A cache whose pages the caller maps refuses to hand out pages, not to hand out none."""
    c = host_cache(kvq, 2)
    c.caller_pages = True
    c._map(0, 0)
    with pytest.raises(kvq.KvqError):
        c._map(0, 1)
    assert len(c.free) == 8 and c.pages == [[], []]
