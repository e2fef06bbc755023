"""Operators of the paged cache held in 8 bits: their measured cases and plain forms.

Keys and values are e4m3 or int8 codes with one scale for each block (a page of G tokens of one
head); the newest tokens are fp16 rows (sink, residual).
  decode  attention of one token per slot over the cache
  chunk   attention of many new tokens per slot over the cache and, causally, themselves
  extend  new tokens enter the cache: sink, fp16 residual, quantized pages
  append  one token per slot: norm and rotation of its query and key (positions scaled for long
          contexts), full residuals packed, key and value rows stored

Every case is a dict of plain values; ``op`` names the operator.  Pages follow include/kvq.h: a
key page is G rows of 128 codes, 16-byte chunk j of row t at position j ^ (4 * (t mod 2)); a value
page is G / 64 tiles of [128 channels][64 tokens].  scale = amax / M with M = 448 (e4m3) or 127
(int8), 1 for a block of zeros; code = x * (M / amax), rounded to nearest even.
"""
import ctypes
import math

import torch

own = False

D = 128
DEV = "cuda"
TOP = {"e4m3": 448.0, "int8": 127.0}


# ---------------------------------------------------------------- cases --------------
def listed():
    # slot lengths of a paged batch of eight grouped-query sequences around 32K tokens
    ragged = "36635,52857,16879,55910,22004,44176,27797,16948"
    heads = dict(H_q=32, H_kv=8)
    return [
        # one user's step after a short prompt
        dict(name="decode_small", op="decode", mode="e4m3", **heads, G=64, R=64, S=0, ctx="300"),
        # one step of eight long sequences
        dict(name="decode_ragged", op="decode", mode="e4m3", **heads, G=128, R=128, S=0, ctx=ragged),
        # a batch of many ordinary sequences, eight query heads to a key head, sink tokens
        dict(name="decode_many", op="decode", mode="int8", H_q=64, H_kv=8, G=64, R=128, S=4, ctx="", B=128, longest=4001, seed=3),
        # one step over a book
        dict(name="decode_long", op="decode", mode="int8", **heads, G=256, R=256, S=0, ctx="131136"),
        # drafted tokens of eight sequences, verified at once
        dict(name="chunk_verify", op="chunk", mode="int8", **heads, G=64, R=64, S=0, ctx="8200,6001,3333,129,12000,777,2500,300",
             new="8,5,8,1,7,8,3,6"),
        # decoding slots beside one slot that is still reading its prompt
        dict(name="chunk_mixed", op="chunk", mode="e4m3", **heads, G=128, R=128, S=8, ctx="8200,6001,3333,1", new="1,517,1,5"),
        # a chunk of a long prompt
        dict(name="chunk_long", op="chunk", mode="e4m3", **heads, G=128, R=128, S=0, ctx="49252", new="1025"),
        # a prompt in two odd chunks, the second starting inside a page
        dict(name="extend_chunk", op="extend", mode="e4m3", H_kv=8, G=128, R=128, S=0, first="1000", then="2048"),
        # four long prompts at once
        dict(name="extend_long", op="extend", mode="int8", H_kv=8, G=64, R=128, S=8, first="8191,4000,127,6000",
             then="8200,12345,1,2222"),
        # a small batch's step
        dict(name="append_small", op="append", mode="int8", **heads, G=64, R=64, S=4, B=8, full=0, far=8192, rotary=128,
             halves=True, norm=True, scaling="none", seed=1),
        # the largest batch's step, part of each head rotates, positions scaled
        dict(name="append_batch", op="append", mode="e4m3", **heads, G=128, R=128, S=0, B=511, full=4, far=131072, rotary=64,
             halves=True, norm=False, scaling="yarn", seed=2),
        # sequences that started together: every residual is full
        dict(name="append_full", op="append", mode="e4m3", **heads, G=128, R=128, S=0, B=256, full=256, far=32768, rotary=128,
             halves=False, norm=True, scaling="bands", seed=3),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "chunk", "extend", "append"])
    H_q, H_kv = rng.choice([(32, 8), (32, 32), (16, 4), (64, 8), (24, 8), (5, 1), (4, 2)])
    G = rng.choice([64, 128, 128, 256])
    common = dict(mode=rng.choice(["e4m3", "int8"]), G=G, R=G * rng.choice([1, 1, 2]), S=rng.choice([0, 0, 4, 33]))
    if op == "decode":
        B = rng.choice([1, 1, 3, 8, 61])
        most = max(2, min(131136, 8 * 55000 * 8 // (B * H_kv)))
        return dict(op=op, H_q=H_q, H_kv=H_kv, **common, ctx=",".join(str(_spread(rng, 1, most)) for _ in range(B)))
    if op == "chunk":
        B = rng.choice([1, 1, 2, 3, 8])
        ctx = [_spread(rng, 1, 49252) for _ in range(B)]
        most = max(1, min(2048, int(1025 * 50000 * 32 / (H_q * (max(ctx) + 2048) * B))))
        return dict(op=op, H_q=H_q, H_kv=H_kv, **common, ctx=",".join(map(str, ctx)),
                    new=",".join(str(_spread(rng, 1, most)) for _ in range(B)))
    if op == "extend":
        B = rng.choice([1, 2, 4, 9])
        most = min(12345, 40000 * 8 // (B * H_kv))
        return dict(op=op, H_kv=H_kv, **common, first=",".join(str(_spread(rng, 1, most // 2)) for _ in range(B)),
                    then=",".join(str(_spread(rng, 1, most // 2)) for _ in range(B)))
    B = _spread(rng, 1, 511)
    # (a second pass packs the first one's rotated key: int8 codes next to a border would tell its last bit)
    full = rng.choice([0, 1, B // 3, B * H_kv <= 2048 and B or 0]) if common["mode"] == "e4m3" else 0
    return dict(op=op, H_q=H_q, H_kv=H_kv, **common, B=B, full=min(full, B), far=_spread(rng, 600, 1 << 20),
                rotary=rng.choice([128, 128, 64, 32]), halves=rng.random() < 0.5, norm=rng.random() < 0.6,
                scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), seed=rng.randrange(1 << 20))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _contexts(case):
    """Tokens of every slot: given, or plain integers of the case's own seed."""
    if case["ctx"]:
        return _ints(case["ctx"])
    import random
    r = random.Random(case["seed"])
    return [_spread(r, 8, case["longest"]) for _ in range(case["B"])]


def _split(L, S, G):
    """A sequence of L tokens as a prefill leaves it: (sink, packed, residual)."""
    ns = min(S, L)
    T = (L - ns) // G * G
    return ns, T, L - ns - T


def _grown(lens, n, S, R):
    """(sink, packed, residual, tokens to the sink, tokens packed) after n more tokens."""
    ns, T, nr = lens
    to_sink = min(n, S - ns)
    tot = nr + n - to_sink
    pk = tot // R * R if n else 0
    return ns + to_sink, T + pk, tot - pk, to_sink, pk


def _append_lengths(case):
    """Slot lengths of an append case; the first `full` slots have a full residual."""
    import random
    r = random.Random(case["seed"])
    S, G, R = case["S"], case["G"], case["R"]
    lens = []
    for b in range(case["B"]):
        L = r.randrange(0, case["far"] // G) * G + S  # positions in earnest; few of the pages are held
        lens.append((S, L - S, R) if b < case["full"] else _split(r.randrange(0, S + 1), S, G) if S and r.random() < 0.1
                    else (S, L - S, r.randrange(0, R)))
    return lens


def _scaling(case):
    return {"none": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=8.0),
            "bands": dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192),
            "yarn": dict(kind="yarn", factor=16.0, fast=32.0, slow=1.0, original=4096)}[case["scaling"]]


def _frequencies(n, base, s):
    """(radians per position of every pair, factor of the rotated channels)."""
    f = [base ** (-2.0 * j / n) for j in range(n // 2)]
    if s is None:
        return f, 1.0
    k = s["factor"]
    if s["kind"] == "linear":
        return [x / k for x in f], 1.0
    if s["kind"] == "ntk":  # a larger base: the last pair turns `factor` times slower, the first as before
        b = base * k ** (n / (n - 2))
        return [b ** (-2.0 * j / n) for j in range(n // 2)], 1.0
    if s["kind"] == "bands":  # long wavelengths are scaled, short ones kept, a ramp over wavelengths between
        part = [min(1.0, max(0.0, (s["original"] * x / (2 * math.pi) - s["low"]) / (s["high"] - s["low"]))) for x in f]
        return [x * p + x / k * (1 - p) for x, p in zip(f, part)], 1.0
    at = lambda turns: n * math.log(s["original"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(s["fast"])), 0), min(math.ceil(at(s["slow"])), n - 1)  # a ramp over the pairs' indices
    part = [min(1.0, max(0.0, (j - lo) / max(hi - lo, 0.001))) for j in range(n // 2)]
    return [x * (1 - p) + x / k * p for x, p in zip(f, part)], 0.1 * math.log(k) + 1.0


# ---------------------------------------------------------------- inputs -------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _kv(g, *shape, channels=None):
    x = torch.randn(*shape, D, generator=g, device=DEV)
    if channels is not None:
        x[..., channels] *= 5.0  # a few key channels carry large magnitudes
    return x.half()


def _codes(x, mode):
    """fp32 values within the codes' range -> codes, as bytes."""
    if mode == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.int8)
    return x.clamp(-127.0, 127.0).round().to(torch.int8)


def _pool(g, mode, span, P, H, *shape, channels=None):
    """A pool's codes of Gaussians whose blocks reach about `span` deviations, and their scales;
    of keys if there are channels of five times the size."""
    out = torch.empty(P, H, *shape, dtype=torch.int8, device=DEV)
    step = max(1, (1 << 26) // (H * math.prod(shape)))
    for i in range(0, P, step):
        x = torch.randn(min(step, P - i), H, *shape, generator=g, device=DEV)
        if channels is not None:
            x[..., channels] *= 5.0
            x = _swap(x)
        out[i:i + step] = _codes(x * (TOP[mode] / span), mode)
    return out, (0.9 + 0.2 * torch.rand(P, H, generator=g, device=DEV)) * (span / TOP[mode])


def _cache(case, B, max_T, n_pages):
    """The framework's cache of a case (empty)."""
    import bit_kv_cache_gb300 as kvq
    return kvq.KVQPagedCache(B, case.get("H_q", case["H_kv"]), case["H_kv"], D, case["G"], 8, n_pages=n_pages,
                             max_T=max_T, S=case["S"], R=case["R"], device=DEV, mode=case["mode"])


def _host(lens):
    """Lengths as the library's host copy."""
    return (ctypes.c_int32 * (4 * len(lens)))(*[x for l in lens for x in (*l, int(sum(l) > 0))])


def _device(lens):
    return torch.tensor([[*l, int(sum(l) > 0)] for l in lens], dtype=torch.int32, device=DEV)


def _fill(cache, host, device):
    """Sets the cache's lengths."""
    ctypes.memmove(cache.lens_host, host, ctypes.sizeof(host))
    cache.lens.copy_(device)


def _shown(held, mode):
    """The codes as the values they stand for, apart from their block's scale."""
    as_value = lambda n, x: x.view(torch.float8_e4m3fn) if n.endswith("codes") and mode == "e4m3" else x  # noqa: E731
    return {n: as_value(n, x) for n, x in held.items()}


def _own_held(c, held):
    """The framework's buffers by the names of `held`."""
    name = {"k_scale": "k_meta", "v_scale": "v_meta"}
    return {n: c.lens if n == "lens" else c.table if n == "table" else c.view(name.get(n, n)) for n in held}


def _fp16_rows(g, case, B, fill):
    S, R, H = case["S"], case["R"], case["H_kv"]
    held = {"k_res": fill(g, B, H, R, "k"), "v_res": fill(g, B, H, R, "v")}
    if S:
        held["k_sink"], held["v_sink"] = fill(g, B, H, S, "k"), fill(g, B, H, S, "v")
    return held


def prepare(case, seed):
    g = _gen(seed)
    op, mode, H, S, G, R = (case[x] for x in ("op", "mode", "H_kv", "S", "G", "R"))
    s = {"case": case, "op": op}
    i32 = dict(dtype=torch.int32, device=DEV)
    ch = torch.randperm(D, generator=g, device=DEV)[:4]
    if op in ("decode", "chunk"):
        ctx = _contexts(case)
        new = _ints(case["new"]) if op == "chunk" else [1] * len(ctx)
        B, N = len(ctx), sum(new)
        lens = [_split(L, S, G) for L in ctx]
        max_T = max(max(l[1] for l in lens) + R * (2 + max(new) // R), R)
        P = sum(l[1] for l in lens) // G + 1
        held = _fp16_rows(g, case, B, lambda g, B, H, n, side: _kv(g, B, H, n, channels=ch if side == "k" else None))
        held["k_codes"], held["k_scale"] = _pool(g, mode, 22.0, P, H, G, D, channels=ch)
        held["v_codes"], held["v_scale"] = _pool(g, mode, 4.7, P, H, G // 64, D, 64)
        order, table, at = torch.randperm(P, generator=g, device=DEV).to(torch.int32), torch.zeros(B, max_T // G, **i32), 0
        for b, l in enumerate(lens):
            table[b, :l[1] // G] = order[at:at + l[1] // G]
            at += l[1] // G
        s.update(held=held, table=table, lens=torch.tensor(lens, **i32), T=max(l[1] for l in lens), N=N, most=max(new),
                 new=torch.tensor(new, **i32), q=torch.randn(N, case["H_q"], D, generator=g, device=DEV).half(),
                 out=torch.empty(N, case["H_q"], D, dtype=torch.float16, device=DEV))
        if op == "chunk":
            s["k"], s["v"] = _kv(g, N, H, channels=ch), _kv(g, N, H)
        if own:
            c = s["cache"] = _cache(case, B, max_T, P)
            for name, x in _own_held(c, held).items():
                x.copy_(held[name].view(x.dtype) if name.endswith("codes") else held[name])
            c.table.copy_(table)
            _fill(c, _host(lens), _device(lens))
            if op == "chunk":
                s["chunk"] = c.plan(new, c.new_chunk(N), pages=torch.zeros(sum(n // R + 2 for n in new) * R // G, **i32))
            s["held"] = None
        return s
    zeros = lambda g, B, H, n, side: torch.zeros(B, H, n, D, dtype=torch.float16, device=DEV)  # noqa: E731
    if op == "append":
        lens, B, F = _append_lengths(case), case["B"], case["full"]
        H_q, J = case["H_q"], R // G
        P = max(1, F * J)
        max_T = max(l[1] for l in lens) // R * R + 2 * R
        held = _fp16_rows(g, case, B, lambda g, B, H, n, side: _kv(g, B, H, n, channels=ch if side == "k" else None))
        held["k_codes"], held["v_codes"] = (torch.zeros(P, H, *sh, dtype=torch.int8, device=DEV) for sh in ((G, D), (G // 64, D, 64)))
        held["k_scale"], held["v_scale"] = torch.zeros(P, H, device=DEV), torch.zeros(P, H, device=DEV)
        held["table"], held["lens"] = torch.zeros(B, max_T // G, **i32), _device([(1, 0, 0)] * B)
        qkv = torch.randn(B, H_q + 2 * H, D, generator=g, device=DEV)
        s["qkv"] = (qkv * torch.exp(0.3 * torch.randn(B, 1, 1, generator=g, device=DEV))).half()  # one projection's rows
        s["q"], s["k"], s["v"] = s["qkv"][:, :H_q], s["qkv"][:, H_q:H_q + H], s["qkv"][:, H_q + H:]
        w = lambda: (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).half() if case["norm"] else None  # noqa: E731
        s["wq"], s["wk"] = w(), w()
        pages = torch.randperm(P, generator=g, device=DEV)[:F * J].to(torch.int32)
        s.update(held=held, pages=pages, out=torch.empty(B, H_q, D, dtype=torch.float16, device=DEV), max_T=max_T)
        lens = [(ns, T, nr) if ns + T + nr else (min(1, S), 0, 1 - min(1, S)) for ns, T, nr in lens]  # every slot is active
        s["lens0"] = _device(lens)
        if own:
            import bit_kv_cache_gb300 as kvq
            c = s["cache"] = _cache(case, B, max_T, P)
            for name, x in _own_held(c, held).items():
                x.copy_(held[name].view(x.dtype) if name.endswith("codes") else held[name])
            s["held"] = _own_held(c, held)
            s["lens_host"], s["pages"] = _host(lens), pages.cpu()
            s["rope"] = kvq.Rope(case["rotary"], base=500000.0, halves=case["halves"], scaling=_scaling(case))
            return s
        f, s["amp"] = _frequencies(case["rotary"], 500000.0, _scaling(case))
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        s["pos"] = torch.tensor([sum(l) for l in lens], device=DEV)
        idx = lambda it: torch.tensor(list(it), dtype=torch.long, device=DEV)  # noqa: E731
        s["full"] = idx(range(F))
        s["to_sink"] = idx(b for b, l in enumerate(lens) if l[0] < S)
        s["to_res"] = idx(b for b, l in enumerate(lens) if l[0] >= S)
        s["sink_row"] = idx(l[0] for l in lens if l[0] < S)
        s["res_row"] = idx(l[2] % R for l in lens if l[0] >= S)
        s["page_row"] = idx(l[1] // G for l in lens[:F])
        s["after"] = _device([(l[0] + 1, l[1], l[2]) if l[0] < S else (l[0], l[1] + l[2] // R * R, l[2] % R + 1) for l in lens])
        return s
    first, then = _ints(case["first"]), _ints(case["then"])
    B = len(first)
    lens = [[(0, 0, 0)] * B]
    for n in (first, then):
        lens.append([_grown(l, x, S, R)[:3] for l, x in zip(lens[-1], n)])
    max_T = max(max(l[1] for l in lens[-1]), R)
    P = max(sum(l[1] for l in lens[-1]) // G, 1)
    held = _fp16_rows(g, case, B, zeros)
    held["k_codes"], held["v_codes"] = (torch.zeros(P, H, *sh, dtype=torch.int8, device=DEV) for sh in ((G, D), (G // 64, D, 64)))
    held["k_scale"], held["v_scale"] = torch.zeros(P, H, device=DEV), torch.zeros(P, H, device=DEV)
    held["lens"] = torch.zeros(B, 4, **i32)
    s["k"], s["v"] = [_kv(g, sum(n), H, channels=ch) for n in (first, then)], [_kv(g, sum(n), H) for n in (first, then)]
    order, table, at = torch.randperm(P, generator=g, device=DEV).to(torch.int32), torch.zeros(B, max_T // G, **i32), 0
    for b, l in enumerate(lens[-1]):
        table[b, :l[1] // G] = order[at:at + l[1] // G]
        at += l[1] // G
    s.update(held=held, table=table, new=[torch.tensor(n, **i32) for n in (first, then)],
             most=[max(l[2] + n for l, n in zip(a, x)) for a, x in zip(lens, (first, then))])
    if own:
        c = s["cache"] = _cache(case, B, max_T, P)
        for x in _own_held(c, held).values():
            x.zero_()
        s["held"] = _own_held(c, held)
        s["chunks"] = []
        for l, n in zip(lens, (first, then)):  # a plan follows from the lengths before its chunk
            _fill(c, _host(l), _device(l))
            s["chunks"].append(c.plan(n, c.new_chunk(sum(n)), pages=order))
        c.table.copy_(table)  # the pages of both chunks
    return s


# ---------------------------------------------------------------- plain forms --------
def _swap(x):
    """A key page's rows from logical to stored order, or back: odd rows swap their halves."""
    y = x.reshape(*x.shape[:-2], x.shape[-2] // 2, 2, 2, D // 2)
    return torch.stack([y[..., 0, :, :], y[..., 1, :, :].flip(-2)], -3).reshape(x.shape)


def _value(codes, mode):
    return (codes.view(torch.float8_e4m3fn) if mode == "e4m3" else codes).float()


def _plain_rows(s):
    """The cached keys and values of every slot in 32 bits: [B][H][S + T + R][D] each."""
    c, held = s["case"], s["held"]
    G, H, mode = c["G"], c["H_kv"], c["mode"]
    B, J = s["table"].shape[0], s["T"] // c["G"]
    pages = s["table"][:, :J].long()
    scale = lambda n: held[n][pages].transpose(1, 2)[..., None, None]  # noqa: E731
    keys = _swap(_value(held["k_codes"][pages], mode)).transpose(1, 2) * scale("k_scale")
    vals = _value(held["v_codes"][pages], mode).permute(0, 2, 1, 3, 5, 4).reshape(B, H, J, G, D) * scale("v_scale")
    keys, vals = [keys.reshape(B, H, J * G, D)], [vals.reshape(B, H, J * G, D)]
    if c["S"]:
        keys.insert(0, held["k_sink"].float())
        vals.insert(0, held["v_sink"].float())
    return torch.cat(keys + [held["k_res"].float()], 2), torch.cat(vals + [held["v_res"].float()], 2)


def _plain_attn(s):
    c, lens, new, most = s["case"], s["lens"], s["new"], s["most"]
    H, g, B = c["H_kv"], c["H_q"] // c["H_kv"], s["lens"].shape[0]
    keys, vals = _plain_rows(s)
    end = new.cumsum(0)
    i = torch.arange(most, device=DEV)
    at = ((end - new)[:, None] + i).clamp(max=s["N"] - 1)  # [B][most] rows of the queries
    seen = [torch.arange(n, device=DEV) < lens[:, k, None] for k, n in enumerate((c["S"], s["T"], c["R"]))]
    mask = torch.cat(seen, 1)[:, None, :].expand(B, most, -1)
    if "k" in s:
        keys = torch.cat([keys, s["k"][at].transpose(1, 2).float()], 2)
        vals = torch.cat([vals, s["v"][at].transpose(1, 2).float()], 2)
        mask = torch.cat([mask, (i[None, :] <= i[:, None]).expand(B, most, most)], 2)  # [B][most][keys]
    q = s["q"][at].view(B, most, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * most, D).float()
    x = (q @ keys.transpose(2, 3) / math.sqrt(D)).view(B, H, g, most, -1)
    x = x.masked_fill(~mask[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p.view(B, H, g * most, -1) @ vals) / p.sum(-1).view(B, H, g * most, 1)
    o = o.view(B, H, g, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, c["H_q"], D).half()
    slot = torch.repeat_interleave(torch.arange(B, device=DEV), new.long(), output_size=s["N"])
    return o[slot, torch.arange(s["N"], device=DEV) - (end - new)[slot]]


def _plain_pack(x, mode):
    """Blocks [..., G, D] -> (codes as bytes, logical order; scales)."""
    x = x.float()
    amax = x.abs().amax((-2, -1))
    top = torch.full((), TOP[mode], device=DEV)
    scale = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    return _codes(x * torch.where(amax > 0, top / amax, torch.zeros_like(amax))[..., None, None], mode), scale


def _plain_store(held, side, pages, x, mode):
    """Blocks [pages][H][G][D] into the pool."""
    code, held[side + "_scale"][pages] = _plain_pack(x, mode)
    if side == "k":
        held["k_codes"][pages] = _swap(code)
    else:
        held["v_codes"][pages] = code.view(*code.shape[:2], -1, 64, D).transpose(3, 4)


def _plain_extend(s, lens, k):
    """Chunk k enters the cache: returns the lengths after it (all slots at once)."""
    c, held, new, most = s["case"], s["held"], s["new"][k], s["most"][k]
    S, G, R, H = c["S"], c["G"], c["R"], c["H_kv"]
    B = lens.shape[0]
    ns, T, nr = lens.unbind(1)
    to_sink = torch.minimum(new, S - ns)
    tot = nr + new - to_sink
    pk = tot // R * R * (new > 0)
    cu = new.cumsum(0) - new
    j = torch.arange(-(-most // R) * R, device=DEV)
    from_new = (cu + to_sink - nr)[:, None] + j
    J = j.numel() // G
    p = torch.arange(J, device=DEV)
    b, p = torch.nonzero(p[None] < (pk // G)[:, None], as_tuple=True)
    pages = s["table"][b, T[b] // G + p].long()
    i = torch.arange(R, device=DEV)
    tail = (i[None] >= torch.where(pk > 0, 0, nr)[:, None]) & (i[None] < (tot - pk)[:, None])
    src = (pk[:, None] + i).clamp(max=j.numel() - 1)
    for side, x in (("k", s["k"][k]), ("v", s["v"][k])):
        res = held[side + "_res"]
        old = res[:, :, j.clamp(max=R - 1)]
        all_ = torch.where((j[None] < nr[:, None])[:, None, :, None], old, x[from_new.clamp(0, x.shape[0] - 1)].transpose(1, 2))
        rows = all_.gather(2, src[:, None, :, None].expand(B, H, R, D))
        _plain_store(held, side, pages, all_.view(B, H, J, G, D)[b, :, p], c["mode"])
        res.copy_(torch.where(tail[:, None, :, None], rows, res))
        if S:
            t = torch.arange(S, device=DEV)
            got = x[((cu - ns)[:, None] + t).clamp(0, x.shape[0] - 1)].transpose(1, 2)
            put = (t[None] >= ns[:, None]) & (t[None] < (ns + to_sink)[:, None])
            held[side + "_sink"].copy_(torch.where(put[:, None, :, None], got, held[side + "_sink"]))
    return torch.stack([ns + to_sink, T + pk, tot - pk], 1)


def _plain_rope(s, x, w):
    """RMS norm of each head's row in 32 bits, then its rotation; angles in 64 bits."""
    c, x = s["case"], x.float()
    n = c["rotary"]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    ang = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = (torch.cos(ang) * s["amp"]).float(), (torch.sin(ang) * s["amp"]).float()
    a, b = (x[..., :n // 2], x[..., n // 2:n]) if c["halves"] else (x[..., 0:n:2], x[..., 1:n:2])
    y = a * cos - b * sin, a * sin + b * cos
    y = torch.cat(y, -1) if c["halves"] else torch.stack(y, -1).flatten(-2)
    return torch.cat([y, x[..., n:]], -1).half()


def _plain_append(s):
    c, held, full = s["case"], s["held"], s["full"]
    G, H, J, F = c["G"], c["H_kv"], c["R"] // c["G"], c["full"]
    held["table"][full[:, None], s["page_row"][:, None] + torch.arange(J, device=DEV)] = s["pages"].view(F, J)
    rows = {"k": _plain_rope(s, s["k"], s["wk"]), "v": s["v"]}
    for side, x in rows.items():
        if F:
            _plain_store(held, side, s["pages"].long(), held[side + "_res"][full].view(F, H, J, G, D).transpose(1, 2).flatten(0, 1),
                         c["mode"])
        held[side + "_res"][s["to_res"], :, s["res_row"]] = x[s["to_res"]]
        if c["S"]:
            held[side + "_sink"][s["to_sink"], :, s["sink_row"]] = x[s["to_sink"]]
    held["lens"].copy_(s["after"])
    return {"q": _plain_rope(s, s["q"], s["wq"]), **_shown(held, c["mode"])}


def run(s):
    op, mode = s["op"], s["case"]["mode"]
    if own:
        cache = s["cache"]
        if op == "decode":
            return cache.decode_attn(s["q"], out=s["out"])
        if op == "chunk":
            return cache.chunk_attn(s["chunk"], s["q"], s["k"], s["v"], out=s["out"])
        if op == "append":
            _fill(cache, s["lens_host"], s["lens0"])  # the step before this one
            q = cache.append_rope(s["q"], s["k"], s["v"], s["rope"], s["wq"], s["wk"], eps=1e-6, pages=s["pages"], out=s["out"])
            return {"q": q, **s["held"]}
        cache.clear(unmap=False)
        cache.extend(s["chunks"][0], s["k"][0], s["v"][0])
        cache.extend(s["chunks"][1], s["k"][1], s["v"][1])
        return s["held"]
    if op in ("decode", "chunk"):
        return _plain_attn(s)
    if op == "append":
        return _plain_append(s)
    lens = torch.zeros_like(s["held"]["lens"][:, :3])
    lens = _plain_extend(s, lens, 0)
    lens = _plain_extend(s, lens, 1)
    s["held"]["lens"].copy_(torch.cat([lens, (lens.sum(1, keepdim=True) > 0).to(torch.int32)], 1))
    return _shown(s["held"], mode)


# ---------------------------------------------------------------- work ---------------
def work(case):
    op, S, G, R, H = (case[x] for x in ("op", "S", "G", "R", "H_kv"))
    page = H * (2 * G * D + 8)  # codes and scales of keys and values
    row = H * D * 4             # an fp16 key and value of every head
    if op in ("decode", "chunk"):
        ctx = _contexts(case)
        new = _ints(case["new"]) if op == "chunk" else [1] * len(ctx)
        read = pairs = 0
        for L, n in zip(ctx, new):
            ns, T, nr = _split(L, S, G)
            read += T // G * page + (ns + nr) * row + (n * row if op == "chunk" else 0)
            pairs += n * L + (n * (n + 1) // 2 if op == "chunk" else 0)
        return {"bytes": read + 4 * sum(new) * case["H_q"] * D, "flops": 4 * pairs * case["H_q"] * D}
    if op == "append":
        n = case["B"] * (case["H_q"] + H) * D
        packed = case["full"] * (R * row + R // G * (page + 4))
        return {"bytes": 4 * n + case["B"] * (row + 32) + packed, "flops": 8 * n}
    moved, lens = 0, [(0, 0, 0)] * len(_ints(case["first"]))
    for text in (case["first"], case["then"]):
        for b, n in enumerate(_ints(text)):
            ns, T, nr, to_sink, pk = _grown(lens[b], n, S, R)
            kept = to_sink + (nr if pk else nr - lens[b][2])  # rows written in fp16
            moved += n * row + (lens[b][2] * row if pk else 0) + pk // G * page + kept * row
            lens[b] = (ns, T, nr)
    return {"bytes": moved, "flops": 0}


# ---------------------------------------------------------------- exact --------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_extend(s) if case["op"] == "extend" else _exact_attn(s)


def _exact_block(s, side, page, h):
    """One head's block [G][D] in 64 bits."""
    c, held = s["case"], s["held"]
    G = c["G"]
    code = held[side + "_codes"][page, h]
    code = (code.view(torch.float8_e4m3fn).float() if c["mode"] == "e4m3" else code).double().reshape(-1)
    t, d = torch.arange(G, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    at = 128 * t + ((d // 16) ^ (4 * (t % 2))) * 16 + d % 16 if side == "k" else t // 64 * 8192 + 64 * d + t % 64
    return code[at] * held[side + "_scale"][page, h].double()


def _exact_attn(s):
    c = s["case"]
    g, G, out, at = c["H_q"] // c["H_kv"], c["G"], torch.zeros(s["N"], c["H_q"], D, dtype=torch.float64, device=DEV), 0
    for b, n in enumerate(s["new"].tolist()):
        ns, T, nr = s["lens"][b].tolist()
        pages = s["table"][b, :T // G].tolist()
        for h in range(c["H_kv"]):
            both = []
            for side in "kv":
                x = [s["held"][side + "_sink"][b, h, :ns].double()] if ns else []
                x += [_exact_block(s, side, p, h) for p in pages]
                x.append(s["held"][side + "_res"][b, h, :nr].double())
                both.append(torch.cat(x + ([s[side][at:at + n, h].double()] if "k" in s else [])))
            K, V = both
            for i in range(0, n, 512):
                m = min(512, n - i)
                ahead = torch.arange(len(K), device=DEV)[None] > ns + T + nr + i + torch.arange(m, device=DEV)[:, None]
                for e in range(g * h, g * h + g):
                    x = s["q"][at + i:at + i + m, e].double() @ K.T / D ** 0.5
                    out[at + i:at + i + m, e] = torch.softmax(x.masked_fill_(ahead, -math.inf), -1) @ V
        at += n
    return out


def _exact_scale(x, mode):
    amax = x.double().abs().max().item()
    return amax / TOP[mode] if amax else 1.0


def _exact_extend(s):
    """Scales and fp16 rows from the definition, slot by slot; codes follow from rounded
    products and have no value here."""
    c, held = s["case"], s["held"]
    S, G, R, mode = c["S"], c["G"], c["R"], c["mode"]
    want = {n: None if n.endswith("codes") or x.dtype == torch.int32 else torch.zeros_like(x, dtype=torch.float64) for n, x in held.items()}
    B = len(s["new"][0])
    lens, at = [(0, 0, 0)] * B, [0, 0]
    for k in range(2):
        for b, n in enumerate(s["new"][k].tolist()):
            ns, T, nr = lens[b]
            after = _grown(lens[b], n, S, R)
            to_sink, pk = after[3:]
            for side in "kv":
                x = s[side][k][at[k]:at[k] + n].transpose(0, 1).double()
                if to_sink:
                    want[side + "_sink"][b, :, ns:ns + to_sink] = x[:, :to_sink]
                x = torch.cat([want[side + "_res"][b, :, :nr], x[:, to_sink:]], 1)
                for j in range(pk // G):
                    m = x[:, j * G:(j + 1) * G].abs().amax((1, 2))
                    want[side + "_scale"][s["table"][b, T // G + j].item()] = torch.where(m > 0, m / TOP[mode], torch.ones_like(m))
                i0 = 0 if pk else nr
                want[side + "_res"][b, :, i0:after[2]] = x[:, pk + i0:]
            lens[b] = after[:3]
            at[k] += n
    return want


def _exact_append(s):
    """Rotated rows pair by pair as complex numbers turned by their angles, and the scales."""
    c, held = s["case"], s["held"]
    R, G, H, mode, n = c["R"], c["G"], c["H_kv"], c["mode"], c["rotary"]
    want = {m: None if m.endswith("codes") or x.dtype == torch.int32 else x.double() for m, x in held.items()}

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x * w.double() * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + 1e-6)
        y = x.clone()
        for j, f in enumerate(s["freq"].tolist()):
            a, b = (j, j + n // 2) if c["halves"] else (2 * j, 2 * j + 1)
            turn = torch.polar(torch.full_like(s["pos"], s["amp"], dtype=torch.float64), s["pos"].double() * f)
            z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        return y

    k = turned(s["k"], s["wk"])
    for b, (ns, T, nr, _) in enumerate(s["lens0"].tolist()):
        for side, x in (("k", k[b]), ("v", s["v"][b].double())):
            if nr == R:
                for j in range(R // G):
                    for h in range(H):
                        want[side + "_scale"][s["pages"][b * (R // G) + j], h] = _exact_scale(held[side + "_res"][b, h, j * G:(j + 1) * G], mode)
            if ns < c["S"]:
                want[side + "_sink"][b, :, ns] = x
            else:
                want[side + "_res"][b, :, nr % R] = x
    return {"q": turned(s["q"], s["wq"]), **want}
