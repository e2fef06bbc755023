"""Norm and rotation with given frequencies at every head dim, against float64."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("D, rd, halves, kw", [
    (64, 64, False, dict(base=10000.0, scaling=dict(kind="linear", factor=4))),
    (64, 32, True, dict(base=500000.0, scaling=dict(kind="bands", factor=8, original=8192))),
    (128, 128, True, dict(scaling=dict(kind="yarn", factor=16, original=4096))),
    (256, 256, False, dict(scaling=dict(kind="ntk", factor=8))),
    (256, 96, True, dict(scaling=dict(kind="yarn", factor=4, original=2048), amp=0.5)),
    (256, 16, False, dict(freq=[0.0, 3.0, 1e-3, 1e-9, 6.0, 0.1, 2.0, 100.0], amp=2.0)),
    (64, 64, True, dict(freq=[2.0 ** -j for j in range(32)])),
], ids=str)
def test_given_frequencies(D, rd, halves, kw):
    import bit_kv_cache_gb300 as kvq
    rope = kvq.Rope(rd, halves=halves, **kw)
    g = torch.Generator(device=DEV).manual_seed(D + rd)
    n, H_q, H = 70, 6, 2
    x = (torch.randn(n, H_q + 2 * H, D, generator=g, device=DEV) * 3).half()
    q, k = x[:, :H_q], x[:, H_q: H_q + H]
    w = torch.randn(D, generator=g, device=DEV).half()
    pos = torch.randint(0, 1 << 17, (n,), generator=g, device=DEV, dtype=torch.int32)
    pos[:3] = torch.tensor([0, 1, (1 << 31) - 1], dtype=torch.int32)
    outs = kvq.qk_norm_rope(q, k, w, None, pos, eps=1e-5, rope=rope)
    for got, y, wt in zip(outs, (q, k), (w, None)):
        y = y.double().cpu()
        if wt is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5) * wt.double().cpu()
        ref, mag, ang_err = y.clone(), y.abs(), torch.zeros_like(y)
        for j, f in enumerate(rope.freq):
            a, b = (j, j + rd // 2) if halves else (2 * j, 2 * j + 1)
            turns = pos.cpu().numpy().astype(object) * Fraction(f)  # exact
            ang = torch.tensor([float(t % (2 * PI)) for t in turns], dtype=torch.float64)
            c, s = torch.cos(ang)[:, None] * rope.amp, torch.sin(ang)[:, None] * rope.amp
            ref[..., a], ref[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
            m = (y[..., a].abs() + y[..., b].abs()) * max(abs(rope.amp), 1.0)
            mag[..., a], mag[..., b] = m, m
            # the table holds a frequency to a unit of 2^-64 turns (its relative 2^-62 beyond 2 pi)
            e = pos.cpu().double()[:, None] * (2 * np.pi * 2.0 ** -64 + f * 2.0 ** -62)
            ang_err[..., a], ang_err[..., b] = m * e, m * e
        # one rounding to fp16, the sum of D squares and a few products in fp32, an angle of 2^-24 of
        # half a turn
        tol = 2.0 ** -11 * ref.abs() + 2.0 ** -25 + mag * (D * 2.0 ** -25 + 8 * 2.0 ** -24 + np.pi * 2.0 ** -24) + ang_err
        err = (got.double().cpu() - ref).abs()
        assert torch.all(err <= tol), (err / tol).max().item()
