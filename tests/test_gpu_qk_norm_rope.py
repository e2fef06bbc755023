"""Norm and rotation of queries and keys on the GPU, against float64."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def reference(x, w, pos, base, rd, halves, rotate, eps):
    """float64 result, and the magnitude that its rounding errors scale with."""
    x = x.double().cpu()
    D = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double().cpu()
    y, mag = x.clone(), x.abs()
    if rotate:
        for j in range(rd // 2):
            a, b = (j, j + rd // 2) if halves else (2 * j, 2 * j + 1)
            ang = pos.cpu().double() * float(base) ** (-2.0 * j / rd)
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
            m = x[..., a].abs() + x[..., b].abs()
            mag[..., a], mag[..., b] = m, m
    return y, mag


def check(got, x, w, pos, base, rd, halves, rotate, eps):
    ref, mag = reference(x, w, pos, base, rd, halves, rotate, eps)
    # one rounding to fp16 (half a step, or half the subnormal step), and fp32 arithmetic: the
    # sum of D squares (D 2^-24 at most, halved by the root), a few products, and an angle
    # held to 2^-24 of half a turn
    tol = 2.0 ** -11 * ref.abs() + 2.0 ** -25 + mag * (x.shape[-1] * 2.0 ** -25 + 8 * 2.0 ** -24 + np.pi * 2.0 ** -24)
    err = (got.double().cpu() - ref).abs()
    assert torch.all(err <= tol), (err - tol).max().item()


CASES = [dict(n=1, H_q=1, H_kv=1, D=128), dict(n=8, H_q=32, H_kv=8, D=128), dict(n=37, H_q=5, H_kv=3, D=64, halves=True),
         dict(n=3, H_q=2, H_kv=1, D=256, rd=128), dict(n=300, H_q=6, H_kv=2, D=128, rd=48, halves=True),
         dict(n=5, H_q=4, H_kv=4, D=256, rd=256, halves=True), dict(n=7, H_q=12, H_kv=2, D=64, rd=16),
         dict(n=9, H_q=4, H_kv=2, D=128, norm=False), dict(n=4, H_q=4, H_kv=2, D=128, rd=0),
         dict(n=400, H_q=32, H_kv=8, D=128, far=1 << 30), dict(n=6, H_q=4, H_kv=2, D=128, base=1.0)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_norm_rope(i):
    import bit_kv_cache_gb300 as kvq
    c = dict(dict(rd=None, halves=False, norm=True, far=1 << 17, base=500000.0), **CASES[i])
    rd = c["D"] if c["rd"] is None else c["rd"]
    g = torch.Generator(device=DEV).manual_seed(i)
    x = torch.randn(c["n"], c["H_q"] + 2 * c["H_kv"], c["D"], generator=g, device=DEV) * 3
    x = x.half()
    q, k = x[:, : c["H_q"]], x[:, c["H_q"]: c["H_q"] + c["H_kv"]]
    w = [torch.randn(c["D"], generator=g, device=DEV).half() if c["norm"] else None for _ in range(2)]
    pos = torch.randint(0, c["far"], (c["n"],), generator=g, device=DEV, dtype=torch.int32)
    before = x.clone()
    qo, ko = kvq.qk_norm_rope(q, k, *w, pos, eps=1e-5, rope_base=c["base"], rotary_dim=c["rd"], halves=c["halves"])
    assert torch.equal(x, before)
    args = (pos, c["base"], rd, c["halves"], True, 1e-5)
    check(qo, q, w[0], *args)
    check(ko, k, w[1], *args)


def test_rotate_flags_queries_only_and_in_place():
    import bit_kv_cache_gb300 as kvq
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(20, 4, 128, generator=g, device=DEV).half()
    k = torch.randn(20, 2, 128, generator=g, device=DEV).half()
    w = torch.randn(128, generator=g, device=DEV).half()
    pos = torch.arange(20, dtype=torch.int32, device=DEV) * 1000
    qo, ko = kvq.qk_norm_rope(q, k, w, w, pos, rotate_k=False)
    check(qo, q, w, pos, 10000.0, 128, False, True, 1e-6)
    check(ko, k, w, pos, 10000.0, 128, False, False, 1e-6)
    only, none = kvq.qk_norm_rope(q, None, w, None, pos)
    assert none is None and torch.equal(only, qo)
    q2, k2 = q.clone(), k.clone()
    a, b = kvq.qk_norm_rope(q2, k2, w, w, pos, rotate_k=False, out=(q2, k2))
    assert a is q2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    empty = kvq.qk_norm_rope(q[:0], k[:0], w, w, pos[:0])
    assert empty[0].shape == (0, 4, 128)


def test_not_finite_and_zero_rows():
    import bit_kv_cache_gb300 as kvq
    q = torch.ones(3, 2, 128, device=DEV).half()
    q[0, 0] = 0
    q[1, 1, 5] = float("nan")
    w = torch.ones(128, device=DEV).half()
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    out, _ = kvq.qk_norm_rope(q, None, w, None, pos)
    assert (out[0, 0] == 0).all() and torch.isnan(out[1, 1]).all()
    keep = torch.ones(3, 2, dtype=torch.bool, device=DEV)
    keep[1, 1] = False
    assert torch.isfinite(out[keep]).all()


def test_matches_pre_rope_cache_rotation():
    """The interleaved rotation at base b is the one that a pre-RoPE cache's attention gives
    its keys: attending with a rotated query over raw keys equals attending over keys rotated
    here (both in fp16 buffers)."""
    import bit_kv_cache_gb300 as kvq
    g = torch.Generator(device=DEV).manual_seed(2)
    L, H_q, H = 20, 4, 2
    k = torch.randn(1, H, L, 128, generator=g, device=DEV).half()
    v = torch.randn(1, H, L, 128, generator=g, device=DEV).half()
    q = torch.randn(1, H_q, 128, generator=g, device=DEV).half()
    pos = torch.arange(L, dtype=torch.int32, device=DEV)
    qr, _ = kvq.qk_norm_rope(q, None, None, None, pos[-1:])
    _, kr = kvq.qk_norm_rope(k[0].transpose(0, 1).contiguous(), k[0].transpose(0, 1).contiguous(), None, None, pos)
    outs = []
    for base, keys in ((10000.0, k), (0.0, kr.transpose(0, 1).contiguous()[None])):
        c = kvq.KVQCache(1, H_q, H, 128, 128, 2, max_T=128, device=DEV, rope_base=base)
        c.prefill(keys.contiguous(), v)
        outs.append(c.decode_attn(qr).float())
    assert torch.all((outs[0] - outs[1]).abs() <= 2e-3 + 2e-3 * outs[1].abs())


def test_captured():
    import bit_kv_cache_gb300 as kvq
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(20, 4, 128, generator=g, device=DEV).half()
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    out = (torch.empty_like(q), None)
    kvq.qk_norm_rope(q, None, None, None, pos, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.qk_norm_rope(q, None, None, None, pos, out=out)
    q.copy_(torch.randn(20, 4, 128, generator=g, device=DEV))
    pos += 70000
    graph.replay()
    check(out[0], q, None, pos, 10000.0, 128, False, True, 1e-6)


def test_refusals():
    import bit_kv_cache_gb300 as kvq
    q = torch.zeros(4, 2, 128, device=DEV).half()
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    for kw, err in ((dict(pos=pos[:3]), ValueError), (dict(pos=pos.long()), ValueError), (dict(rotary_dim=20), kvq.KvqError),
                    (dict(rotary_dim=144), kvq.KvqError), (dict(eps=-1.0), kvq.KvqError),
                    (dict(w_q=torch.ones(64, device=DEV).half()), ValueError),
                    (dict(out=(q, q)), ValueError), (dict(k=q, out=(q, q)), kvq.KvqError),
                    (dict(k=q.float()), ValueError), (dict(k=q[:3]), ValueError)):
        with pytest.raises(err):
            kvq.qk_norm_rope(q, **{**dict(pos=pos), **kw})
    with pytest.raises(ValueError):
        kvq.qk_norm_rope(q.transpose(1, 2), pos=pos)
    big = torch.zeros(4, 4, 128, device=DEV).half()
    with pytest.raises(kvq.KvqError):  # an output inside a strided input
        kvq.qk_norm_rope(big[:, :2], pos=pos, out=(big.view(-1)[: 4 * 2 * 128].view(4, 2, 128), None))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rd", [0, 32, None])
@pytest.mark.parametrize("norm", [False, True])
def test_channels_that_do_not_rotate_stay_apart(D, halves, rd, norm):
    """An infinite or NaN channel behind rotary_dim, or of rows that do not rotate, reaches no
    other channel but through the norm; without a norm those rows pass through bit for bit."""
    import bit_kv_cache_gb300 as kvq
    g = torch.Generator(device=DEV).manual_seed(D)
    n, H = 12, 3
    q = torch.randn(n, H, D, generator=g, device=DEV).half()
    k = torch.randn(n, H, D, generator=g, device=DEV).half()
    bad = [float("inf"), float("-inf")] + ([] if norm else [float("nan")])
    for i in range(n):
        q[i, i % H, D - 1 - i % 3] = bad[i % len(bad)]  # rd <= 32 < D - 3
        k[i, (i + 1) % H, 5 * i % D] = bad[i % len(bad)]
    w = torch.randn(D, generator=g, device=DEV).half() if norm else None
    pos = torch.randint(1, 1000, (n,), generator=g, device=DEV, dtype=torch.int32)
    rotate_q = rd is not None
    qo, ko = kvq.qk_norm_rope(q, k, w, w, pos, rotary_dim=rd, halves=halves, rotate_q=rotate_q, rotate_k=False)
    for got, x, rotate in ((qo, q, rotate_q), (ko, k, False)):
        ref, mag = reference(x, w, pos, 10000.0, D if rd is None else rd, halves, rotate, 1e-6)
        got = got.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        fin = torch.isfinite(ref)
        assert torch.equal(got[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
        tol = 2.0 ** -11 * ref.abs() + 2.0 ** -25 + mag * (D * 2.0 ** -25 + 8 * 2.0 ** -24 + np.pi * 2.0 ** -24)
        assert torch.all((got - ref).abs()[fin] <= tol[fin])
        if not norm:
            first = (rd or 0) if rotate else 0
            assert torch.equal(got[..., first:].nan_to_num(7.0), x[..., first:].double().cpu().nan_to_num(7.0))


def test_weight_of_a_side_without_heads_is_not_read():
    import ctypes

    import bit_kv_cache_gb300 as kvq
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(9, 3, 128, generator=g, device=DEV).half()
    w = torch.randn(128, generator=g, device=DEV).half()
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    want, _ = kvq.qk_norm_rope(x, None, w, None, pos)
    stray = w.data_ptr() + 2  # aligned for no vector load
    got = torch.zeros_like(x)
    for heads, args in (((3, 0), (x.data_ptr(), None, w.data_ptr(), stray, got.data_ptr(), None)),
                        ((0, 3), (None, x.data_ptr(), stray, w.data_ptr(), None, got.data_ptr()))):
        got.zero_()
        c = kvq.QkConfig(*heads, 128, 128, 0, 3, 1e-6, 1e4, 384, 384)
        q, k, wq, wk, qo, ko = args
        assert kvq.lib.kvq_qk_norm_rope(ctypes.byref(c), q, k, wq, wk, pos.data_ptr(), 9, qo, ko,
                                        torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(got, want)
