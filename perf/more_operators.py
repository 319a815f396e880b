"""Operators of a KV cache that lives in pages, and the cases they are measured on.

paged_attention   attention of each sequence's new tokens (one, a chunk, a whole prompt) over
                  the pages of its cache, causal, with a sliding window and first tokens that
                  stay visible, the pages in bf16 or in 8 bits;
rope_append_e4m3  per-head norms and rotary positions, and the append of keys and values to
                  8-bit pages, quantised as they are written;
kv_write_pages    rows of a contiguous cache saved to pages, as they are or quantised;
kv_read_pages     rows of pages restored to a contiguous cache.

An 8-bit row is held as e4m3 codes with a power of two for each 32 elements (a byte, the
exponent + 127): 2^e is the smallest with max|x| <= 448 * 2^e, e in [-100, 7].

Cases are dicts of plain values; `own` selects the library's kernels, otherwise `run` computes
the same with elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a single sequence over a short context: latency only
        dict(name="attend one token", op="attend", seqs=1, new=1, new_spread=0, heads=32, kv_heads=8, head_dim=64,
             type="f32", cache="bf16", page=16, length=192, spread=0, window=0, sinks=0, pad=0),
        # a serving batch decoding, contexts of all lengths, in a launch padded to 40 tokens
        dict(name="attend decode batch", op="attend", seqs=32, new=1, new_spread=0, heads=32, kv_heads=8, head_dim=64,
             type="bf16", cache="bf16", page=16, length=4099, spread=3900, window=0, sinks=0, pad=8),
        # long contexts held in 8 bits
        dict(name="attend decode 8 bits", op="attend", seqs=8, new=1, new_spread=0, heads=24, kv_heads=8, head_dim=128,
             type="bf16", cache="e4m3", page=64, length=32768, spread=5001, window=0, sinks=0, pad=0),
        # drafted or chunked tokens far out, a sliding window and four first tokens
        dict(name="attend window", op="attend", seqs=4, new=33, new_spread=9, heads=32, kv_heads=8, head_dim=128,
             type="bf16", cache="bf16", page=32, length=20001, spread=7000, window=4096, sinks=4, pad=3),
        # a whole prompt
        dict(name="attend prompt", op="attend", seqs=1, new=4096, new_spread=0, heads=32, kv_heads=8, head_dim=64,
             type="bf16", cache="bf16", page=16, length=4096, spread=0, window=0, sinks=0, pad=0),
        # chunks of prompts behind a cached prefix in 8 bits, fp32 queries
        dict(name="attend chunks 8 bits", op="attend", seqs=3, new=301, new_spread=200, heads=24, kv_heads=8,
             head_dim=64, type="f32", cache="e4m3", page=128, length=6001, spread=3333, window=0, sinks=0, pad=0),
        # one token of a decode step
        dict(name="append one token", op="append", seqs=1, tokens=1, heads=32, kv_heads=8, head_dim=64, rot=64,
             type="f32", norm=False, interleaved=False, page=16, base=128),
        # the tokens of two long prompts, normed heads, half of the head rotated
        dict(name="append prompts", op="append", seqs=2, tokens=2047, heads=24, kv_heads=8, head_dim=128, rot=64,
             type="bf16", norm=True, interleaved=False, page=64, base=30000),
        # the rows of one short sequence to bf16 pages
        dict(name="save one", op="write", layers=16, slots=1, kv_heads=8, head_dim=64, room=512, length=130, spread=0,
             page=16, cache="bf16"),
        # the caches of a batch quantised to 8-bit pages (and read back: what they hold is the result)
        dict(name="save batch 8 bits", op="write", layers=16, slots=8, kv_heads=8, head_dim=64, room=2048, length=2000,
             spread=777, page=64, cache="e4m3"),
        # a short prefix of one sequence restored from 8-bit pages
        dict(name="restore one 8 bits", op="read", layers=16, slots=1, kv_heads=8, head_dim=64, room=512, length=130,
             spread=0, page=16, cache="e4m3"),
        # a batch restored from bf16 pages, heads of 128
        dict(name="restore batch", op="read", layers=28, slots=4, kv_heads=8, head_dim=128, room=2100, length=2050,
             spread=601, page=32, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "write", "read"])
    head_dim, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    page, cache, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "e4m3"]), rng.choice(["f32", "bf16"])
    if op == "attend":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
        seqs, new = _log(rng, 1, 32), rng.choice([1, _log(rng, 2, 64), _log(rng, 64, 4096)])
        new = min(new, max(1, 4096 // seqs))
        length = new + _log(rng, 1, 32768) - 1
        length = max(new, min(length, int(5e8 / (4 * seqs * new * heads)), int(2e8 / (seqs * kv_heads * head_dim))))
        return dict(op=op, seqs=seqs, new=new, new_spread=rng.randint(0, new - 1), heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, type=dtype, cache=cache, page=page, length=length,
                    spread=rng.randint(0, length - new), window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                    sinks=rng.choice([0, 4, rng.randint(1, 200)]), pad=rng.choice([0, rng.randint(1, 9)]))
    if op == "append":
        seqs = _log(rng, 1, 16)
        rot = rng.choice([head_dim, head_dim // 2, head_dim // 4, 2 * rng.randint(1, head_dim // 2)])
        return dict(op=op, seqs=seqs, tokens=max(1, _log(rng, 1, 4094) // seqs), heads=kv_heads * rng.choice([1, 2, 3, 4]),
                    kv_heads=kv_heads, head_dim=head_dim, rot=rot, type=dtype, norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, page=page, base=_log(rng, 1, 120000))
    slots, layers = _log(rng, 1, 8), rng.randint(1, 28)
    length = min(_log(rng, 1, 8000), int(1.2e8 / (slots * layers * kv_heads * head_dim)))
    return dict(op=op, layers=layers, slots=slots, kv_heads=kv_heads, head_dim=head_dim, room=length + rng.randint(0, 99),
                length=length, spread=rng.randint(0, length - 1), page=page, cache=cache)


def _ragged(value, spread, n):
    """n whole numbers falling from value to value - spread."""
    return [value - (spread * i) // max(1, n - 1) for i in range(n)]


def _news(c):
    """Each sequence's new tokens."""
    return _ragged(c["new"], c["new_spread"], c["seqs"])


def _lens(c):
    return _ragged(c["length"], c["spread"], c.get("seqs") or c["slots"])


def _row_bytes(c, cache):
    return c["kv_heads"] * c["head_dim"] * 2 * (2 if cache == "bf16" else 1 + 1 / 32)


def work(case):
    c, size = case, {"f32": 4, "bf16": 2}
    if c["op"] == "attend":
        rows = pairs = 0
        for n, length in zip(_news(c), _lens(c)):
            window = c["window"] or length
            first = max(0, length - n - window + 1)
            rows += length - first + min(c["sinks"], first)
            for p in range(length - n, length):
                pairs += min(p + 1, window) + min(c["sinks"], max(0, p + 1 - window))
        qo = 2 * sum(_news(c)) * c["heads"] * c["head_dim"] * size[c["type"]]
        return {"bytes": rows * _row_bytes(c, c["cache"]) + qo, "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    if c["op"] == "append":
        n, d = c["seqs"] * c["tokens"], c["head_dim"]
        per = (2 * c["heads"] + 2 * c["kv_heads"]) * d * size[c["type"]] + _row_bytes(c, "e4m3") + 12
        back = _append_pages(c) * c["page"] * (_row_bytes(c, "e4m3") + _row_bytes(c, "bf16"))
        return {"bytes": n * per + back, "flops": n * (c["heads"] + 2 * c["kv_heads"]) * d * 6}
    n = sum(_lens(c)) * c["layers"]
    there = n * (_row_bytes(c, "bf16") + _row_bytes(c, c["cache"]))
    if c["op"] == "write" and c["cache"] == "e4m3":
        there += c["layers"] * _pool_pages(c) * c["page"] * (_row_bytes(c, "e4m3") + _row_bytes(c, "bf16"))
    return {"bytes": there, "flops": 0}


# ---------------------------------------------------------------- inputs
def _normal(g, dev, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _power(e):
    """2^e in fp32, for whole numbers e in [-126, 127], by its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """fp32 rows as e4m3 codes and the exponents' bytes."""
    x = x.unflatten(-1, (-1, 32))
    most = x.abs().amax(-1)
    m, e = torch.frexp(most)  # most = m 2^e, m in [0.5, 1): over 448 = 1.75 * 2^8 takes one more
    e = torch.where(most > 0, e - 9 + (m > 0.875), -100).clamp(-100, 7)
    codes = (x * _power(-e)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """The fp32 values of 8-bit rows."""
    return (codes.float().unflatten(-1, (-1, 32)) * _power(scales.int() - 127)[..., None]).flatten(-2)


def _pool(g, dev, cache, *shape):
    """A layer's (or all layers') pages with rows of normal values: (codes or bf16, scales or None)."""
    x = _normal(g, dev, *shape)
    return (x, None) if cache == "bf16" else _quantise(x.float())


def _append_pages(c):
    return c["seqs"] * ((c["tokens"] + c["page"] - 2) // c["page"] + 1)


def _pool_pages(c):
    return sum(-(-n // c["page"]) for n in _lens(c)) + 1


def _tables(lens, page, total, h):
    """Each sequence's pages in random places of the pool, -1 behind the last."""
    order, at = torch.randperm(total, generator=h), 0
    table = torch.full((len(lens), max(-(-n // page) for n in lens)), -1)
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = order[at: at + need]
        at += need
    return table


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    h = torch.Generator().manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device=dev)
    s, K, D, ps = {"case": c}, c["kv_heads"], c["head_dim"], c["page"]
    if c["op"] == "append":
        n, B, dt = c["tokens"], c["seqs"], DTYPES[c["type"]]
        pages, per = _append_pages(c), (n + ps - 2) // ps + 1
        s["qkv"] = _normal(g, dev, B * n, (c["heads"] + 2 * K) * D, dtype=dt)
        s["q_out"] = torch.empty(B * n, c["heads"], D, dtype=dt, device=dev)
        s["k"], s["ks"] = _pool(g, dev, "e4m3", pages, K, ps, D)
        s["v"], s["vs"] = _pool(g, dev, "e4m3", pages, K, ps, D)
        table = torch.randperm(pages, generator=h).view(B, per)
        first = torch.randint(0, ps, (B, 1), generator=h).clamp(max=per * ps - n)  # the row of the first token
        row = first + torch.arange(n)[None]
        s["slots"] = table.gather(1, row // ps).reshape(-1).to(**i32)
        s["rows"] = (row % ps).reshape(-1).to(**i32)
        s["positions"] = (c["base"] + row).reshape(-1).to(**i32)
        s["freq"] = (5e5 ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64) / c["rot"])).to(dev)
        for name in ("q_norm", "k_norm"):
            s[name] = (1 + 0.05 * _normal(g, dev, D, dtype=torch.float32)).to(torch.bfloat16) if c["norm"] else None
    elif c["op"] == "attend":
        lens, news, G = _lens(c), _news(c), c["heads"] // K
        total = sum(news) + c["pad"]
        pages = sum(-(-n // ps) for n in lens) + 2
        s["q"] = (1.5 * _normal(g, dev, total, c["heads"], D, dtype=torch.float32)).to(DTYPES[c["type"]])
        s["out"] = torch.zeros(total, c["heads"], D, dtype=DTYPES[c["type"]], device=dev)
        s["k"], s["ks"] = _pool(g, dev, c["cache"], pages, K, ps, D)
        s["v"], s["vs"] = _pool(g, dev, c["cache"], pages, K, ps, D)
        s["table"] = _tables(lens, ps, pages, h).to(**i32)
        s["starts"] = torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], **i32)
        s["lengths"] = torch.tensor(lens, **i32)
        return s
    else:
        L, B, lens, pages = c["layers"], c["slots"], _lens(c), _pool_pages(c)
        s["ck"], s["cv"] = _normal(g, dev, L, B, K, c["room"], D), _normal(g, dev, L, B, K, c["room"], D)
        s["k"], s["ks"] = _pool(g, dev, c["cache"], L, pages, K, ps, D)
        s["v"], s["vs"] = _pool(g, dev, c["cache"], L, pages, K, ps, D)
        s["table"] = _tables(lens, ps, pages, h).to(**i32)
        s["lengths"] = torch.tensor(lens, **i32)
    if c["op"] == "append" or (c["op"] == "write" and c["cache"] == "e4m3"):
        # to read the whole pool back, each page as a sequence of its own
        shape = (c.get("layers", 1), pages, K, ps, D)
        s["k_back"], s["v_back"] = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        s["each"] = torch.arange(pages, **i32)[:, None]
        s["full"] = torch.full((pages,), ps, **i32)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return {"attend": _attend, "append": _append, "write": _write, "read": _read}[state["case"]["op"]](state)


def _sequence_pages(pool, scales, table, length):
    """Rows [0, length) of a sequence in a layer's pool, [kv heads][length][head dim], fp32."""
    ids = table[: -(-length // pool.shape[2])].long()
    if scales is None:
        x = pool[ids].float()
    else:
        x = _values(pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn), scales[ids])
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def _attend(s):
    c = s["case"]
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.paged_attention(s["q"], s["k"], s["v"], s["table"], s["starts"], s["lengths"], s["out"],
                             window=c["window"], sinks=c["sinks"], k_scales=s["ks"], v_scales=s["vs"],
                             max_new=c["new"], max_len=c["length"])
        return s["out"]
    H, K, D, at = c["heads"], c["kv_heads"], c["head_dim"], 0
    for b, (n, length) in enumerate(zip(_news(c), _lens(c))):
        k = _sequence_pages(s["k"], s["ks"], s["table"][b], length)
        v = _sequence_pages(s["v"], s["vs"], s["table"][b], length)
        q = s["q"][at: at + n].float().view(n, K, H // K, D).permute(1, 0, 2, 3).reshape(K, -1, D)
        score = (q @ k.transpose(-1, -2)) * (D ** -0.5)
        j = torch.arange(length, device=k.device)[None]
        p = torch.arange(length - n, length, device=k.device)[:, None]
        seen = j <= p
        if c["window"]:
            seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
        seen = seen[:, None].expand(n, H // K, length).reshape(1, -1, length)
        score = torch.where(seen, score, float("-inf"))
        w = torch.exp(score - score.amax(-1, keepdim=True))
        o = (w @ v) / w.sum(-1, keepdim=True)
        s["out"][at: at + n] = o.view(K, n, H // K, D).permute(1, 0, 2, 3).reshape(n, H, D).to(s["out"].dtype)
        at += n
    return s["out"]


def _append(s):
    c = s["case"]
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.rope_append_e4m3(s["qkv"], s["q_out"], s["k"], s["v"], s["ks"], s["vs"], s["positions"], s["rows"],
                              s["freq"], slots=s["slots"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-5,
                              interleaved=c["interleaved"])
        return s["q_out"], *_back(s)
    H, K, D, r = c["heads"], c["kv_heads"], c["head_dim"], c["rot"]
    x = s["qkv"].float().view(-1, H + 2 * K, D)
    q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-5) * s["q_norm"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-5) * s["k_norm"].float()
    angle = s["positions"].double()[:, None] * s["freq"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(y):
        if c["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., r:]], -1)
        a, b = y[..., : r // 2], y[..., r // 2: r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., r:]], -1)

    s["q_out"].copy_(rotate(q))
    slots, rows = s["slots"].long(), s["rows"].long()
    for x, pool, scales in ((rotate(k), s["k"], s["ks"]), (v, s["v"], s["vs"])):
        codes, e = _quantise(x)
        pool.view(torch.uint8)[slots, :, rows] = codes.view(torch.uint8)
        scales[slots, :, rows] = e
    return s["q_out"], *_back(s)


def _back(s):
    """What the 8-bit pages hold, in bf16 (exactly)."""
    if own:
        from decode_megakernel_llama_gb300 import _lib
        k, v, ks, vs = ((s[x] if s[x].dim() == 5 else s[x][None]) for x in ("k", "v", "ks", "vs"))
        _lib.kv_read_pages(k, v, s["k_back"], s["v_back"], s["each"], s["full"], k_scales=ks, v_scales=vs)
    else:
        s["k_back"].copy_(_values(s["k"], s["ks"]))
        s["v_back"].copy_(_values(s["v"], s["vs"]))
    return s["k_back"], s["v_back"]


def _places(s, b, n):
    """(page, row of the page) of a sequence's first n rows."""
    j = torch.arange(n, device=s["table"].device)
    return s["table"][b].long()[j // s["case"]["page"]], j % s["case"]["page"]


def _write(s):
    c = s["case"]
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.kv_write_pages(s["ck"], s["cv"], s["k"], s["v"], s["table"], s["lengths"], k_scales=s["ks"],
                            v_scales=s["vs"])
    else:
        for cache, pool, scales in ((s["ck"], s["k"], s["ks"]), (s["cv"], s["v"], s["vs"])):
            for b, n in enumerate(_lens(c)):
                page, row = _places(s, b, n)
                x = cache[:, b, :, :n].permute(2, 0, 1, 3)  # (the indexed dimensions come first)
                if scales is None:
                    pool[:, page, :, row] = x
                else:
                    codes, e = _quantise(x.float())
                    pool.view(torch.uint8)[:, page, :, row] = codes.view(torch.uint8)
                    scales[:, page, :, row] = e
    return _back(s) if c["cache"] == "e4m3" else (s["k"], s["v"])


def _read(s):
    c = s["case"]
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.kv_read_pages(s["k"], s["v"], s["ck"], s["cv"], s["table"], s["lengths"], k_scales=s["ks"],
                           v_scales=s["vs"])
        return s["ck"], s["cv"]
    for cache, pool, scales in ((s["ck"], s["k"], s["ks"]), (s["cv"], s["v"], s["vs"])):
        for b, n in enumerate(_lens(c)):
            page, row = _places(s, b, n)
            if scales is None:
                x = pool[:, page, :, row]
            else:
                x = _values(pool.view(torch.uint8)[:, page, :, row].view(torch.float8_e4m3fn), scales[:, page, :, row])
            cache[:, b, :, :n] = x.permute(1, 2, 0, 3).to(torch.bfloat16)
    return s["ck"], s["cv"]


# ---------------------------------------------------------------- 64 bits
def _code_values(device):
    """The value of each e4m3 code, by its bits."""
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(math.nan if c & 127 == 127 else -v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=device)


def _exact_power(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales):
    power = _exact_power(scales.long() - 127)
    return _code_values(codes.device)[codes.view(torch.uint8).long()] * power.repeat_interleave(32, -1)


def _exact_quantised(x):
    """The values that 64-bit rows keep in 8 bits: the nearest multiple of the code's step, ties to even."""
    y = x.reshape(*x.shape[:-1], -1, 32)
    most = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(most.clamp(min=448 * 2.0 ** -100) / 448))
    e = e - (most <= 448 * _exact_power(e - 1)).double() + (most > 448 * _exact_power(e)).double()
    e = e.clamp(-100, 7)
    z = (y / _exact_power(e)).clamp(-448, 448)
    step = _exact_power(torch.frexp(z.abs().clamp(min=2.0 ** -6))[1] - 4)  # 2^(floor(log2 |z|) - 3)
    return (torch.round(z / step) * step * _exact_power(e)).reshape(x.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "attend":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
        G, ps, at = c["heads"] // c["kv_heads"], c["page"], 0
        for b, length in enumerate(s["lengths"].tolist()):
            n = int(s["starts"][b + 1]) - at
            ids = [int(x) for x in s["table"][b] if x >= 0]
            for h in range(c["kv_heads"]):
                k, v = [], []
                for pool, scales, to in ((s["k"], s["ks"], k), (s["v"], s["vs"], v)):
                    for i in ([ids] if len(ids) > 64 else ids):  # (many pages at once)
                        x = pool.view(torch.uint8)[i, h].view(pool.dtype) if scales is not None else pool[i, h]
                        x = x.double() if scales is None else _exact_values(x, scales[i, h])
                        to.append(x.reshape(-1, c["head_dim"]))
                k, v = torch.cat(k)[:length], torch.cat(v)[:length]
                behind = torch.arange(length - n, length, device=k.device)[:, None] - torch.arange(length, device=k.device)
                hidden = behind < 0
                if c["window"]:
                    hidden |= (behind >= c["window"]) & (torch.arange(length, device=k.device) >= c["sinks"])
                for x in range(h * G, (h + 1) * G):
                    score = (s["q"][at: at + n, x].double() @ k.T / math.sqrt(c["head_dim"])).masked_fill(hidden, -math.inf)
                    out[at: at + n, x] = torch.softmax(score, -1) @ v
            at += n
        return out
    if c["op"] == "append":
        H, K, D, r = c["heads"], c["kv_heads"], c["head_dim"], c["rot"]
        x = s["qkv"].double().reshape(-1, H + 2 * K, D).clone()
        if c["norm"]:
            for part, gain in ((slice(0, H), s["q_norm"]), (slice(H, H + K), s["k_norm"])):
                ms = x[:, part].pow(2).sum(-1, keepdim=True) / D
                x[:, part] = x[:, part] / (ms + 1e-5).sqrt() * gain.double()
        angle = torch.outer(s["positions"].double(), s["freq"])
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        first = torch.arange(r // 2, device=x.device) * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else r // 2)
        z = torch.complex(x[:, : H + K, first], x[:, : H + K, second]) * turn
        x[:, : H + K, first], x[:, : H + K, second] = z.real, z.imag
        back = []
        for rows, codes, scales in ((x[:, H:H + K], s["k"], s["ks"]), (x[:, H + K:], s["v"], s["vs"])):
            pool = _exact_values(codes, scales)
            kept = _exact_quantised(rows)
            for i, (page, row) in enumerate(zip(s["slots"].tolist(), s["rows"].tolist())):
                pool[page, :, row] = kept[i]
            back.append(pool[None])
        return x[:, :H].contiguous(), *back
    out = []
    for cache, pool, scales in ((s["ck"], s["k"], s["ks"]), (s["cv"], s["v"], s["vs"])):
        cache = cache.double()
        pool = pool.double() if scales is None else _exact_values(pool, scales)
        for b, n in enumerate(s["lengths"].tolist()):
            for i in range(0, n, c["page"]):
                m, page = min(c["page"], n - i), int(s["table"][b, i // c["page"]])
                if c["op"] == "read":
                    cache[:, b, :, i: i + m] = pool[:, page, :, :m]
                else:
                    rows = cache[:, b, :, i: i + m]
                    pool[:, page, :, :m] = rows if scales is None else _exact_quantised(rows)
        out.append(cache if c["op"] == "read" else pool)
    return tuple(out)
