"""The softmax weights of the 8-bit caches with one scale per page and head: their precision beside
dominant tokens and beside pages of other scales."""
import math

import numpy as np
import pytest
import torch

from block_bounds import Errors, rows_of, worst
from block_util import D, DEV, U16, cached_rows, make_cache, randn

pytestmark = pytest.mark.gpu
MODES = ["e4m3", "int8"]
SIZES = [1.0, 0.1, 0.01, 0.001]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def aimed(rng, B, H_kv, g, height):
    """Queries whose heads of a group are alike, [B][H_kv g][D], and for each group the key whose
    score is `height` above 0 for the common part of them (the others' scores spread by about 1)."""
    q0 = rng.standard_normal((B, H_kv, 1, D))
    q = (q0 + 0.2 * rng.standard_normal((B, H_kv, g, D))).reshape(B, H_kv * g, D).astype(np.float16)
    key = (q0[:, :, 0] * (height * math.sqrt(D) / (q0[:, :, 0] ** 2).sum(-1, keepdims=True))).astype(np.float16)
    return torch.from_numpy(q).to(DEV), torch.from_numpy(key).to(DEV)


def fill(c, rng, lens, keys, size, at, zero=None):
    """Prefills the slots with Gaussian keys and values of `size`; token `at` has the slot's key of
    `keys` and, with the tokens of `zero`, values of zero."""
    for b, n in enumerate(lens):
        k, v = randn(rng, c.cfg.H_kv, n, D), randn(rng, c.cfg.H_kv, n, D, scale=size)
        k[:, at] = keys[b]
        v[:, at] = 0
        if zero is not None:
            v[:, zero] = 0
        c.prefill(b, k, v)


def decode_errors(c, q):
    e, g = Errors(), c.cfg.H_q // c.cfg.H_kv
    out = c.decode_attn(q).cpu().double().numpy()
    qd = q.cpu().double().numpy()
    for b in range(c.cfg.B):
        K, V = cached_rows(c, b)
        for h in range(c.cfg.H_kv):
            e.add(out[b, h * g: h * g + g], qd[b, h * g: h * g + g], K[h], V[h])
    assert c.read_status() == 0
    return e


def chunk_errors(c, rng, new, q0, size):
    """A chunk of new[b] tokens whose queries are those of q0 [B][H_q][D] with some noise."""
    e, g, n = Errors(), c.cfg.H_q // c.cfg.H_kv, sum(new)
    slot = np.repeat(np.arange(len(new)), new)
    q = (q0[torch.from_numpy(slot).to(DEV)].float() + 0.1 * randn(rng, n, c.cfg.H_q, D).float()).half()
    k, v = randn(rng, n, c.cfg.H_kv, D), randn(rng, n, c.cfg.H_kv, D, scale=size)
    out = c.chunk_attn(c.plan(new), q, k, v).cpu().double().numpy()
    qd, k, v = (x.cpu().double().numpy() for x in (q, k, v))
    at = 0
    for b, m in enumerate(new):
        K, V = cached_rows(c, b)
        L = K.shape[1]
        K = np.concatenate([K, k[at:at + m].transpose(1, 0, 2)], 1)
        V = np.concatenate([V, v[at:at + m].transpose(1, 0, 2)], 1)
        hid = np.arange(L + m)[None, :] > L + np.arange(m)[:, None]
        for h in range(c.cfg.H_q):
            e.add(out[at:at + m, h], qd[at:at + m, h], K[h // g], V[h // g], hid)
        at += m
    assert c.read_status() == 0
    return e


LENS = [4 + 960 + 5, 4 + 1024 + 9]  # slots in one part: 16 items of a CTA's four warps


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("height", [8.0, 11.0, 14.0])
@pytest.mark.parametrize("size", SIZES)
def test_decode_beside_a_sink(size, height, mode):
    """An fp16 sink token far above packed tokens of any size: their weights keep their bits."""
    rng = np.random.default_rng(21)
    q, keys = aimed(rng, 2, 2, 4, height)
    c = make_cache(rng, [0, 0], mode, S=4)
    fill(c, rng, LENS, keys, size, at=1)
    decode_errors(c, q).check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [[3, 1], [8, 5], [80, 20], [10, 30]], ids=str)
@pytest.mark.parametrize("size", SIZES)
def test_chunk_beside_a_sink(size, new, mode):
    """The same for few new tokens (their own kernel) and more."""
    rng = np.random.default_rng(22)
    q, keys = aimed(rng, 2, 2, 4, 9.0)
    c = make_cache(rng, [0, 0], mode, S=4)
    fill(c, rng, LENS, keys, size, at=1)
    chunk_errors(c, rng, new, q, size).check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("size", SIZES)
def test_decode_beside_a_page_of_zeros(size, mode):
    """A page whose values are all zero has a scale of 1: a token of it that takes most of the
    attention costs the weights of pages of small values nothing."""
    rng = np.random.default_rng(23)
    q, keys = aimed(rng, 2, 2, 4, 9.0)
    c = make_cache(rng, [0, 0], mode)
    fill(c, rng, [965, 1030], keys, size, at=70, zero=slice(64, 128))
    decode_errors(c, q).check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [[3, 1], [8, 5], [80, 20], [10, 30]], ids=str)
@pytest.mark.parametrize("size", SIZES)
def test_chunk_beside_a_page_of_zeros(size, new, mode):
    rng = np.random.default_rng(24)
    q, keys = aimed(rng, 2, 2, 4, 9.0)
    c = make_cache(rng, [0, 0], mode)
    fill(c, rng, [965, 1030], keys, size, at=70, zero=slice(64, 128))
    chunk_errors(c, rng, new, q, size).check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [None, [8, 5], [80, 20]], ids=str)
def test_a_block_of_small_values_that_counts(new, mode):
    """Attention that lies on a block of small values beside blocks of large ones: the output is
    that block's, and an output of zeros would be found out."""
    rng = np.random.default_rng(25)
    q, keys = aimed(rng, 2, 1, 4, 40.0)
    c = make_cache(rng, [0, 0], mode, H_q=4, H_kv=1)
    for b, n in enumerate((5 * 64 + 7, 6 * 64)):
        k, v = randn(rng, 1, n, D, scale=0.5), randn(rng, 1, n, D)
        for j, x in enumerate((200.0, 1.0, 2e-3, 1e-2, 300.0, 50.0)):
            v[:, 64 * j: 64 * j + 64] *= x
        k[:, 130] = keys[b]
        c.prefill(b, k, v)
    for b in range(2):
        K, V = cached_rows(c, b)
        p, ref, mag = rows_of(q[b].cpu().double().numpy(), K[0], V[0])
        assert p[:, 130].min() > 0.99 and np.median(np.abs(ref) / worst(p, V[0], ref, mag)) > 100
    (decode_errors(c, q) if new is None else chunk_errors(c, rng, new, q, 1.0)).check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("new", [None, [7, 2], [70, 25], [1, 200]], ids=str)
@pytest.mark.parametrize("seed", range(3))
def test_pages_of_any_sizes(seed, new, mode):
    """Every page with sizes of its own, keys by 16 times, values from 1e-4 to 300, some pages of
    zeros, and sink tokens of any weight and size."""
    rng = np.random.default_rng(100 + seed)
    G, S = ((64, 3), (128, 0), (256, 20))[seed]
    q, keys = aimed(rng, 2, 2, 4, 5.0)
    c = make_cache(rng, [0, 0], mode, G=G, S=S)
    for b, n in enumerate((S + 2500, S + 7 * G + 13)):
        k, v = randn(rng, 2, n, D), randn(rng, 2, n, D)
        for t in range(0, n, G):
            k[:, S + t: S + t + G] *= float(2.0 ** rng.uniform(-3, 1))
            v[:, S + t: S + t + G] *= float(rng.choice([0.0, 10.0 ** rng.uniform(-4, 2.5)], p=[0.15, 0.85]))
        if S:
            k[:, 1] = keys[b]
            v[:, :S] *= float(10.0 ** rng.uniform(-4, 1))
        k[:, S + 2 * G + 5] = keys[b]
        c.prefill(b, k, v)
    (decode_errors(c, q) if new is None else chunk_errors(c, rng, new, q, float(10.0 ** rng.uniform(-4, 1)))).check()
