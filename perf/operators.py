"""The chunk operators of the paged low-bit KV cache: their measured cases and plain forms.

A serving step adds a few or many new tokens to every slot of a paged cache at once:
the tokens of a prompt's next chunk, drafted tokens to verify, or one token each.
  plan    slot maps, positions and block-table rows from the slots' request lengths
  rope    RMS norm of every query and key head, then the rotary position embedding
  attn    attention of the new tokens over the packed cache and, causally, themselves
  extend  the new tokens enter the cache: sink, fp16 residual, quantized pages

Every case is a dict of plain values; ``op`` names the operator.  Packed pages follow
include/kvq.h: 32 / bits codes to a word, element j at bit bits * j; key words along
tokens with the word of channel d of word row r at position d ^ (4 * (r mod 8)); value
words along channels in tiles of 256 / (key bits) tokens, the word of token j of row m at
position j ^ (4 * (m mod 8)).
"""
import math

import torch

own = False

D = 128
DEV = "cuda"


# ---------------------------------------------------------------- cases --------------
def listed():
    # slot lengths of a paged batch of eight grouped-query sequences around 32K tokens
    ragged = "36635,52857,16879,55910,22004,44176,27797,16948"
    return [
        # the smallest attention call: four tokens after a short prompt
        dict(name="attn_small", op="attn", H_q=32, H_kv=8, bits=2, v_bits=2, G=128, R=128, S=0, ctx="300", new="4"),
        # drafted tokens of eight long sequences, verified at once
        dict(name="attn_verify", op="attn", H_q=32, H_kv=8, bits=2, v_bits=2, G=128, R=128, S=0, ctx=ragged,
             new="8,5,8,1,7,8,3,6"),
        # decoding slots beside one slot that is still reading its prompt; sink tokens, 4-bit keys
        dict(name="attn_mixed", op="attn", H_q=32, H_kv=8, bits=4, v_bits=2, G=128, R=128, S=8,
             ctx="8200,6001,3333,1", new="1,517,1,5"),
        # one key head per query head, 8-bit codes, pages of 256 tokens: a chunk of an ordinary prompt
        dict(name="attn_mha_k8", op="attn", H_q=32, H_kv=32, bits=8, v_bits=8, G=256, R=256, S=0, ctx="4096,1000",
             new="512,301"),
        # a 2048-token chunk of a long prompt
        dict(name="attn_chunk", op="attn", H_q=32, H_kv=8, bits=2, v_bits=2, G=128, R=128, S=0, ctx="32868", new="2048"),
        # one decode step's queries and keys, and a prefill's
        dict(name="rope_step", op="rope", H_q=32, H_kv=8, N=8, far=131072, rotary=128, halves=False, norm=True),
        dict(name="rope_prefill", op="rope", H_q=32, H_kv=8, N=8191, far=131072, rotary=128, halves=True, norm=True),
        # a small batch's plan, and that of the largest batch with long prompts
        dict(name="plan_small", op="plan", B=8, G=128, R=128, S=0, longest=16, seed=1),
        dict(name="plan_large", op="plan", B=512, G=128, R=128, S=8, longest=1000, seed=2),
        # eight slots near a full residual take a few tokens each, and most of them flush
        dict(name="extend_step", op="extend", H_kv=8, bits=2, v_bits=2, G=128, R=128, S=0,
             first="125,127,120,121,3,124,126,122", then="8,5,8,7,1,8,3,6"),
        # a prompt in two odd chunks, the second starting inside a page
        dict(name="extend_chunk", op="extend", H_kv=8, bits=2, v_bits=2, G=128, R=128, S=0, first="1000", then="2048"),
        # four long prompts at once, 4-bit keys and 8-bit values, sink tokens
        dict(name="extend_long", op="extend", H_kv=8, bits=4, v_bits=8, G=128, R=128, S=8, first="8191,4000,127,6000",
             then="8200,12345,1,2222"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "plan", "extend"])
    H_q, H_kv = rng.choice([(32, 8), (32, 32), (16, 4), (8, 8), (24, 8), (4, 2)])
    G = rng.choice([128, 128, 256])
    common = dict(H_kv=H_kv, bits=rng.choice([2, 4, 8]), v_bits=rng.choice([2, 4, 8]), G=G,
                  R=G * rng.choice([1, 1, 2]), S=rng.choice([0, 0, 4, 33]))
    if op == "attn":
        B = rng.choice([1, 1, 2, 3, 8])
        ctx = [_spread(rng, 1, 32768) for _ in range(B)]
        most = max(1, min(2048, int(2048 * 32868 * 32 / (H_q * (max(ctx) + 2048) * B))))
        new = [min(most, _spread(rng, 1, 2048)) for _ in range(B)]
        return dict(op=op, H_q=H_q, **common, ctx=",".join(map(str, ctx)), new=",".join(map(str, new)))
    if op == "rope":
        return dict(op=op, H_q=H_q, H_kv=H_kv, N=_spread(rng, 1, 8191 * 40 // (H_q + H_kv)), far=_spread(rng, 100, 1 << 20),
                    rotary=rng.choice([128, 128, 64]), halves=rng.random() < 0.5, norm=rng.random() < 0.8)
    if op == "plan":
        return dict(op=op, B=_spread(rng, 1, 512), G=G, R=common["R"], S=common["S"], longest=_spread(rng, 1, 1000),
                    seed=rng.randrange(1 << 20))
    B = rng.choice([1, 2, 4, 9])
    most = min(12345, 40000 * 8 // (B * H_kv))
    return dict(op=op, **common, first=",".join(str(_spread(rng, 1, most // 2)) for _ in range(B)),
                then=",".join(str(_spread(rng, 1, most // 2)) for _ in range(B)))


def _ints(text):
    return [int(x) for x in text.split(",")]


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


def _plan_lengths(case):
    """Slot lengths and request lengths of a plan case: plain integers of its own seed."""
    import random
    r = random.Random(case["seed"])
    lens = [_split(r.randrange(0, 4000), case["S"], case["G"]) for _ in range(case["B"])]
    return lens, [r.randrange(0, case["longest"] + 1) if b else case["longest"] for b in range(case["B"])]


# ---------------------------------------------------------------- inputs -------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _kv(g, *shape, channels=None):
    x = torch.randn(*shape, D, generator=g, device=DEV)
    if channels is not None:
        x[..., channels] *= 5.0  # a few key channels carry large magnitudes
    return x.half()


def _words(g, bits, *shape):
    """Random words whose codes gather around the middle, as a Gaussian's do."""
    rnd = lambda: torch.randint(-(1 << 31), 1 << 31, shape, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)  # noqa: E731
    top = sum(1 << (bits * j + bits - 1) for j in range(32 // bits))
    nxt = sum(1 << (bits * j + bits - 2) for j in range(32 // bits))
    sgn = lambda v: v - (1 << 32) if v >= 1 << 31 else v  # noqa: E731
    w, flip = rnd(), rnd() & rnd()
    other = ~((w & sgn(top)).bitwise_right_shift(1)) & sgn(nxt)  # the second bit mostly against the first
    return (w & ~sgn(nxt)) | (other ^ (flip & sgn(nxt)))


def _meta(g, bits, *shape):
    """(scale, min) of groups whose values span about 2.6 deviations to each side."""
    sd = 0.9 + 0.2 * torch.rand(*shape, generator=g, device=DEV)
    return sd, lambda sd: torch.stack([5.2 * sd / ((1 << bits) - 1), -2.6 * sd], -1).half()


def _cache(case, B, max_T, n_pages):
    """The framework's cache of a case (empty)."""
    import bit_kv_cache_gb300 as kvq
    return kvq.KVQPagedCache(B, case.get("H_q", case.get("H_kv", 1)), case.get("H_kv", 1), D, case["G"],
                             case.get("bits", 2), n_pages=n_pages, max_T=max_T, S=case["S"], R=case["R"],
                             v_bits=case.get("v_bits", 0), device=DEV)


def _fill(cache, lens, active):
    """Sets the cache's lengths, as a prefill of those lengths leaves them."""
    flat = [x for l, a in zip(lens, active) for x in (*l, a)]
    cache.lens.copy_(torch.tensor(flat, dtype=torch.int32).view(-1, 4))
    for i, x in enumerate(flat):
        cache.lens_host[i] = x


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "rope":
        H_q, H_kv, N = case["H_q"], case["H_kv"], case["N"]
        qkv = torch.randn(N, H_q + 2 * H_kv, D, generator=g, device=DEV)
        s["qkv"] = (qkv * torch.exp(torch.randn(N, 1, 1, generator=g, device=DEV))).half()  # one projection's rows
        s["q"], s["k"] = s["qkv"][:, :H_q], s["qkv"][:, H_q:H_q + H_kv]
        w = lambda: (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).half() if case["norm"] else None  # noqa: E731
        s["wq"], s["wk"] = w(), w()
        s["pos"] = torch.randint(0, case["far"], (N,), generator=g, device=DEV, dtype=torch.int32)
        s["out"] = torch.empty(N, H_q, D, dtype=torch.float16, device=DEV), torch.empty(N, H_kv, D, dtype=torch.float16, device=DEV)
        return s
    S, G, R = case["S"], case["G"], case["R"]
    if case["op"] == "plan":
        lens, new = _plan_lengths(case)
        B = case["B"]
        more = torch.randint(0, 16, (B,), generator=g, device=DEV).tolist()  # further pages of the sequences past their sink
        lens = [(ns, T + G * m * (ns == S), nr) for (ns, T, nr), m in zip(lens, more)]
        grown = [_grown(l, n, S, R) for l, n in zip(lens, new)]
        max_T = -(-(4000 + 16 * G + R + case["longest"]) // R) * R
        total = sum(x[4] for x in grown) // G
        s.update(new=torch.tensor(new, dtype=torch.int32, device=DEV), N=sum(new), n_pages=total,
                 new_host=torch.tensor(new, dtype=torch.int32), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 pages=torch.randperm(total + 64, generator=g, device=DEV)[:max(total, 1)].to(torch.int32),
                 table=torch.zeros(B, max_T // G, dtype=torch.int32, device=DEV))
        if own:
            c = s["cache"] = _cache(case, B, max_T, total + 64)
            _fill(c, lens, [int(sum(l) > 0) for l in lens])
            s["chunk"], s["table"] = c.new_chunk(max(s["N"], 1)), c.table
        return s
    if case["op"] == "attn":
        ctx, new = _ints(case["ctx"]), _ints(case["new"])
        H, B, N = case["H_kv"], len(ctx), sum(new)
        kb, vb = case["bits"], case["v_bits"]
        lens = [_split(L, S, G) for L in ctx]
        max_T = max(max(l[1] for l in lens) + R * (2 + max(new) // R), R)
        J, P = max_T // G, sum(l[1] for l in lens) // G + 1
        ch = torch.randperm(D, generator=g, device=DEV)[:4]
        sd, km = _meta(g, kb, P, H, D)
        sd[..., ch] *= 5.0
        sv, vm = _meta(g, vb, P, H, G, 1)
        sv = sv * (1.0 + 9.0 * (torch.rand(P, H, G, 1, generator=g, device=DEV) < 0.001))
        TV = 256 // kb
        held = {"k_codes": _words(g, kb, P, H, G * kb // 32, D), "k_meta": km(sd),
                "v_codes": _words(g, vb, P, H, G // TV, D * vb // 32, TV), "v_meta": vm(sv),
                "k_res": _kv(g, B, H, R, channels=ch), "v_res": _kv(g, B, H, R)}
        if S:
            held["k_sink"], held["v_sink"] = _kv(g, B, H, S, channels=ch), _kv(g, B, H, S)
        order, table, at = torch.randperm(P, generator=g, device=DEV).to(torch.int32), torch.zeros(B, J, dtype=torch.int32, device=DEV), 0
        for b, l in enumerate(lens):
            table[b, :l[1] // G] = order[at:at + l[1] // G]
            at += l[1] // G
        s.update(held=held, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), N=N, most=max(new),
                 T=max(l[1] for l in lens), new=torch.tensor(new, dtype=torch.int32, device=DEV),
                 q=torch.randn(N, case["H_q"], D, generator=g, device=DEV).half(), k=_kv(g, N, H, channels=ch), v=_kv(g, N, H),
                 out=torch.empty(N, case["H_q"], D, dtype=torch.float16, device=DEV))
        if own:
            c = s["cache"] = _cache(case, B, max_T, P)
            for name, x in held.items():
                c.view(name).copy_(x)
            c.table.copy_(table)
            _fill(c, lens, [1] * B)
            s["chunk"] = c.plan(new, c.new_chunk(N), pages=torch.zeros(sum(max(new) // R + 1 for _ in new) * R // G, dtype=torch.int32, device=DEV))
        return s
    first, then = _ints(case["first"]), _ints(case["then"])
    H, B, kb, vb = case["H_kv"], len(first), case["bits"], case["v_bits"]
    lens = [[(0, 0, 0)] * B]
    for n in (first, then):
        lens.append([_grown(l, x, S, R)[:3] for l, x in zip(lens[-1], n)])
    max_T = max(max(l[1] for l in lens[-1]), R)
    J, P = max_T // G, max(sum(l[1] for l in lens[-1]) // G, 1)
    TV = 256 // kb
    zeros = lambda dt, *sh: torch.zeros(*sh, dtype=dt, device=DEV)  # noqa: E731
    held = {"k_codes": zeros(torch.int32, P, H, G * kb // 32, D), "k_meta": zeros(torch.float16, P, H, D, 2),
            "v_codes": zeros(torch.int32, P, H, G // TV, D * vb // 32, TV), "v_meta": zeros(torch.float16, P, H, G, 1, 2),
            "k_res": zeros(torch.float16, B, H, R, D), "v_res": zeros(torch.float16, B, H, R, D)}
    if S:
        held["k_sink"], held["v_sink"] = zeros(torch.float16, B, H, S, D), zeros(torch.float16, B, H, S, D)
    ch = torch.randperm(D, generator=g, device=DEV)[:4]
    s["k"], s["v"] = [_kv(g, sum(n), H, channels=ch) for n in (first, then)], [_kv(g, sum(n), H) for n in (first, then)]
    order, table, at = torch.randperm(P, generator=g, device=DEV).to(torch.int32), zeros(torch.int32, B, J), 0
    for b, l in enumerate(lens[-1]):
        table[b, :l[1] // G] = order[at:at + l[1] // G]
        at += l[1] // G
    held["lens"] = zeros(torch.int32, B, 4)
    s.update(held=held, table=table, new=[torch.tensor(n, dtype=torch.int32, device=DEV) for n in (first, then)],
             most=[max(l[2] + n for l, n in zip(a, x)) for a, x in zip(lens, (first, then))])
    if own:
        c = s["cache"] = _cache(case, B, max_T, P)
        s["held"] = {n: c.view(n) for n in held if n != "lens"} | {"lens": c.lens}
        s["chunks"] = []
        for l, n in zip(lens, (first, then)):  # a plan follows from the lengths before its chunk
            _fill(c, l, [int(sum(x) > 0) for x in l])
            s["chunks"].append(c.plan(n, c.new_chunk(sum(n)), pages=order))
        c.table.copy_(table)  # the pages of both chunks
    return s


# ---------------------------------------------------------------- plain forms --------
def _unpack(words, bits):
    """[..., W] int32 -> [..., 32 / bits, W]: element j of each word."""
    sh = torch.arange(0, 32, bits, device=words.device, dtype=torch.int32)[:, None]
    return (words[..., None, :] >> sh) & ((1 << bits) - 1)


def _key_order(rows):
    """Where the word of channel d sits in word row r of a page."""
    r = torch.arange(rows, device=DEV)[:, None]
    return torch.arange(D, device=DEV)[None, :] ^ (4 * (r % 8))


def _value_order(rows, TV):
    m = torch.arange(rows, device=DEV)[:, None]
    j = torch.arange(TV, device=DEV)[None, :]
    return j ^ (4 * (m % 8)) if TV % 32 == 0 else j.expand(rows, TV)


def _plain_rows(s):
    """The cached keys and values of every slot in 32 bits: [B][H][S + T + R][D] each."""
    c, held = s["case"], s["held"]
    kb, vb, G, H = c["bits"], c["v_bits"], c["G"], c["H_kv"]
    B, J = s["table"].shape[0], s["T"] // G
    pages = s["table"][:, :J].long()
    kw = held["k_codes"][pages].transpose(1, 2)  # [B][H][J][rows][D]
    kw = kw.gather(-1, _key_order(kw.shape[3]).expand_as(kw))
    km = held["k_meta"][pages].transpose(1, 2).float()
    keys = _unpack(kw, kb).reshape(B, H, J, G, D).float() * km[:, :, :, None, :, 0] + km[:, :, :, None, :, 1]
    vw = held["v_codes"][pages].transpose(1, 2)  # [B][H][J][tiles][rows][TV]
    vw = vw.gather(-1, _value_order(*vw.shape[-2:]).expand_as(vw))
    vals = _unpack(vw, vb).permute(0, 1, 2, 3, 6, 4, 5).reshape(B, H, J, G, D)  # tile, token, row, element
    vm = held["v_meta"][pages].transpose(1, 2).float()
    vals = vals.float() * vm[..., 0] + vm[..., 1]
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
    at = ((end - new)[:, None] + i).clamp(max=s["N"] - 1)  # [B][most] rows of the chunk
    keys = torch.cat([keys, s["k"][at].transpose(1, 2).float()], 2)
    vals = torch.cat([vals, s["v"][at].transpose(1, 2).float()], 2)
    seen = [torch.arange(n, device=DEV) < lens[:, k, None] for k, n in enumerate((c["S"], s["T"], c["R"]))]
    cached = torch.cat(seen, 1)[:, None, :].expand(B, most, -1)
    mask = torch.cat([cached, (i[None, :] <= i[:, None]).expand(B, most, most)], 2)  # [B][most][keys]
    q = s["q"][at].view(B, most, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * most, D).float()
    x = (q @ keys.transpose(2, 3) / math.sqrt(D)).view(B, H, g, most, -1)
    x = x.masked_fill(~mask[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p.view(B, H, g * most, -1) @ vals) / p.sum(-1).view(B, H, g * most, 1)
    o = o.view(B, H, g, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, c["H_q"], D).half()
    slot = torch.repeat_interleave(torch.arange(B, device=DEV), new.long(), output_size=s["N"])
    return o[slot, torch.arange(s["N"], device=DEV) - (end - new)[slot]]


def _plain_rope(x, w, pos, c):
    """RMS norm of each head's row in 32 bits, then its rotation; angles in 64 bits."""
    x, n = x.float(), c["rotary"]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    inv = 500000.0 ** (-torch.arange(0, n, 2, device=DEV, dtype=torch.float64) / n)
    ang = pos.double()[:, None, None] * inv
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    a, b = (x[..., :n // 2], x[..., n // 2:n]) if c["halves"] else (x[..., 0:n:2], x[..., 1:n:2])
    y = a * cos - b * sin, a * sin + b * cos
    y = torch.cat(y, -1) if c["halves"] else torch.stack(y, -1).flatten(-2)
    return torch.cat([y, x[..., n:]], -1).half()


def _plain_plan(s):
    c, lens, new = s["case"], s["lens"], s["new"]
    S, G, R, B = c["S"], c["G"], c["R"], c["B"]
    cu = torch.cat([new.new_zeros(1), new.cumsum(0, dtype=torch.int32)])
    ids = torch.arange(B, device=DEV, dtype=torch.int32)
    slot = torch.repeat_interleave(ids, new.long(), output_size=s["N"])
    pos = lens.sum(1, dtype=torch.int32)[slot] + torch.arange(s["N"], device=DEV, dtype=torch.int32) - cu[slot]
    to_sink = torch.minimum(new, S - lens[:, 0])
    n = (lens[:, 2] + new - to_sink) // R * (new > 0) * (R // G)
    row = torch.repeat_interleave(ids, n.long(), output_size=s["n_pages"])
    j = torch.arange(s["n_pages"], device=DEV) - (n.cumsum(0) - n)[row]
    s["table"][row, lens[:, 1][row] // G + j] = s["pages"][:s["n_pages"]]
    return {"cu": cu, "slot": slot, "pos": pos, "table": s["table"]}


def _plain_quant(x, dim, bits):
    """Codes and fp16 (scale, min) of groups along `dim`, in 32 bits."""
    x = x.float()
    mn, mx = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    mn, mx = mn + 0.0, mx + 0.0
    top = torch.full((), (1 << bits) - 1, dtype=torch.float32, device=DEV)
    s = ((mx - mn) / top).half()
    q = torch.where(s == 0, torch.zeros_like(x), torch.round((x - mn) / s.float())).clamp(max=float(top))
    return q.to(torch.int32), torch.stack([s, mn.half()], -1)


def _pack(codes, bits):
    """[..., 32 / bits, W] -> [..., W] words."""
    sh = torch.arange(0, 32, bits, device=DEV, dtype=torch.int64)[:, None]
    w = (codes.long() << sh).sum(-2)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _plain_extend(s, lens, k):
    """Chunk k enters the cache: returns the lengths after it (all slots at once)."""
    c, held, new, most = s["case"], s["held"], s["new"][k], s["most"][k]
    S, G, R, H, kb, vb = c["S"], c["G"], c["R"], c["H_kv"], c["bits"], c["v_bits"]
    B, TV = lens.shape[0], 256 // c["bits"]
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
        full = all_.view(B, H, J, G, D)[b, :, p]  # [pages][H][G][D]
        if side == "k":
            code, meta = _plain_quant(full, 2, kb)
            w = _pack(code.view(-1, H, G * kb // 32, 32 // kb, D), kb)
            held["k_codes"][pages] = w.gather(-1, _key_order(w.shape[2]).expand_as(w))  # the order is its own inverse
            held["k_meta"][pages] = meta[:, :, 0]
        else:
            code, meta = _plain_quant(full, 3, vb)
            code = code.view(-1, H, G // TV, TV, D * vb // 32, 32 // vb).permute(0, 1, 2, 4, 5, 3)
            w = _pack(code, vb)
            held["v_codes"][pages] = w.gather(-1, _value_order(*w.shape[-2:]).expand_as(w))
            held["v_meta"][pages] = meta
        res.copy_(torch.where(tail[:, None, :, None], rows, res))
        if S:
            t = torch.arange(S, device=DEV)
            got = x[((cu - ns)[:, None] + t).clamp(0, x.shape[0] - 1)].transpose(1, 2)
            put = (t[None] >= ns[:, None]) & (t[None] < (ns + to_sink)[:, None])
            held[side + "_sink"].copy_(torch.where(put[:, None, :, None], got, held[side + "_sink"]))
    return torch.stack([ns + to_sink, T + pk, tot - pk], 1)


def run(s):
    op = s["op"]
    if own:
        if op == "rope":
            import bit_kv_cache_gb300 as kvq
            c = s["case"]
            return kvq.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], eps=1e-6, rope_base=500000.0,
                                    rotary_dim=c["rotary"], halves=c["halves"], out=s["out"])
        cache = s["cache"]
        if op == "plan":
            ch = cache.plan(s["new_host"], s["chunk"], pages=s["pages"])
            return {"cu": ch.cu, "slot": ch.slot[:s["N"]], "pos": ch.pos[:s["N"]], "table": s["table"]}
        if op == "attn":
            return cache.chunk_attn(s["chunk"], s["q"], s["k"], s["v"], out=s["out"])
        cache.clear(unmap=False)
        cache.extend(s["chunks"][0], s["k"][0], s["v"][0])
        cache.extend(s["chunks"][1], s["k"][1], s["v"][1])
        return s["held"]
    if op == "rope":
        return _plain_rope(s["q"], s["wq"], s["pos"], s["case"]), _plain_rope(s["k"], s["wk"], s["pos"], s["case"])
    if op == "plan":
        return _plain_plan(s)
    if op == "attn":
        return _plain_attn(s)
    lens = torch.zeros_like(s["held"]["lens"][:, :3])
    lens = _plain_extend(s, lens, 0)
    lens = _plain_extend(s, lens, 1)
    s["held"]["lens"].copy_(torch.cat([lens, (lens.sum(1, keepdim=True) > 0).to(torch.int32)], 1))
    return s["held"]


# ---------------------------------------------------------------- work ---------------
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["N"] * (case["H_q"] + case["H_kv"]) * D
        return {"bytes": 4 * n + 4 * case["N"], "flops": 8 * n}
    S, G, R = case["S"], case["G"], case["R"]
    if op == "plan":
        lens, new = _plan_lengths(case)
        pages = sum(_grown(l, n, S, R)[4] for l, n in zip(lens, new)) // G
        return {"bytes": 8 * sum(new) + 8 * pages + 20 * case["B"], "flops": 0}
    H = case["H_kv"]
    page = H * (G * D * (case["bits"] + case["v_bits"]) // 8 + 4 * D + 4 * G)  # codes, (scale, min)
    row = H * D * 4  # an fp16 key and value of every head
    if op == "attn":
        ctx, new = _ints(case["ctx"]), _ints(case["new"])
        read = pairs = 0
        for L, n in zip(ctx, new):
            ns, T, nr = _split(L, S, G)
            read += T // G * page + (ns + nr + n) * row
            pairs += n * L + n * (n + 1) // 2
        return {"bytes": read + 4 * sum(new) * case["H_q"] * D, "flops": 4 * pairs * case["H_q"] * D}
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
    op = case["op"]
    if op == "plan":
        return None  # whole numbers only
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if op == "rope":
        return tuple(_exact_rope(s[x], s["w" + x], s["pos"], case) for x in "qk")
    return _exact_attn(s) if op == "attn" else _exact_extend(s)


def _exact_rope(x, w, pos, c):
    n, x = c["rotary"], x.double()
    if w is not None:
        x = x * w.double() * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + 1e-6)
    y = x.clone()
    for j in range(n // 2):  # pair by pair, as a complex number turned by its angle
        a, b = (j, j + n // 2) if c["halves"] else (2 * j, 2 * j + 1)
        turn = torch.polar(torch.ones_like(pos, dtype=torch.float64), pos.double() * 500000.0 ** (-2.0 * j / n))
        z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_page(s, side, page, h):
    """One head's page [G][D] in 64 bits."""
    c = s["case"]
    bits, G, TV = c["bits" if side == "k" else "v_bits"], c["G"], 256 // c["bits"]
    w = s["held"][side + "_codes"][page, h].long() & 0xFFFFFFFF
    n = 32 // bits
    t, d = torch.arange(G, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    if side == "k":
        word, j = w[t // n, d ^ (4 * ((t // n) % 8))], t % n
    else:
        at = (t % TV) ^ (4 * ((d // n) % 8)) if TV % 32 == 0 else t % TV + 0 * d
        word, j = w[(t // TV).expand(G, D), (d // n).expand(G, D), at], d % n
    m = s["held"][side + "_meta"][page, h].double()
    return ((word >> (bits * j)) % (1 << bits)).double() * m[..., 0] + m[..., 1]


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
                x += [_exact_page(s, side, p, h) for p in pages]
                both.append(torch.cat(x + [s["held"][side + "_res"][b, h, :nr].double(), s[side][at:at + n, h].double()]))
            K, V = both
            for i in range(0, n, 512):
                m = min(512, n - i)
                ahead = torch.arange(len(K), device=DEV)[None] > ns + T + nr + i + torch.arange(m, device=DEV)[:, None]
                for e in range(g * h, g * h + g):
                    x = s["q"][at + i:at + i + m, e].double() @ K.T / D ** 0.5
                    out[at + i:at + i + m, e] = torch.softmax(x.masked_fill_(ahead, -math.inf), -1) @ V
        at += n
    return out


def _exact_extend(s):
    """Scales, minima and fp16 rows from the definition, slot by slot; codes are whole
    numbers and have no value here."""
    c, held = s["case"], s["held"]
    S, G, R = c["S"], c["G"], c["R"]
    want = {n: None if x.dtype == torch.int32 else torch.zeros_like(x, dtype=torch.float64) for n, x in held.items()}
    B = len(s["new"][0])
    lens, at = [(0, 0, 0)] * B, [0, 0]
    for k in range(2):
        for b, n in enumerate(s["new"][k].tolist()):
            ns, T, nr = lens[b]
            after = _grown(lens[b], n, S, R)
            to_sink, pk = after[3:]
            for side, bits, dim in (("k", c["bits"], 1), ("v", c["v_bits"], 2)):
                x = s[side][k][at[k]:at[k] + n].transpose(0, 1).double()
                if to_sink:
                    want[side + "_sink"][b, :, ns:ns + to_sink] = x[:, :to_sink]
                x = torch.cat([want[side + "_res"][b, :, :nr], x[:, to_sink:]], 1)
                for j in range(pk // G):
                    y = x[:, j * G:(j + 1) * G]
                    lo, hi = y.min(dim).values, y.max(dim).values
                    m = torch.stack([(hi - lo) / (2 ** bits - 1), lo], -1)
                    want[side + "_meta"][s["table"][b, T // G + j].item()] = m if side == "k" else m[:, :, None]
                i0 = 0 if pk else nr
                want[side + "_res"][b, :, i0:after[2]] = x[:, pk + i0:]
            lens[b] = after[:3]
            at[k] += n
    return want
