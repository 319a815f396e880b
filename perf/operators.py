"""Operators of verifying a tree of drafted tokens, and the cases they are measured on.

rope_append      per-head norms of queries and keys, rotary positions, and the
                 append of keys and values to the cache, in one pass;
tree_attention   attention of a tree of drafted tokens over a KV cache;
kv_compact       the accepted path's cache rows moved behind the committed ones;
kv_reorder       cache slots copied, forked and swapped.

Cases are dicts of plain values; `own` selects the library's kernels, otherwise
`run` computes the same with elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a single-sequence decode step: latency only
        dict(name="rope decode", op="rope", seqs=1, tokens=1, heads=32, kv_heads=8, head_dim=64, rot=64, type="f32",
             norm=False, interleaved=False, scaling="none", base=128, room=256),
        # eight drafted trees of 27 nodes, normed heads, a quarter of the head rotated in adjacent pairs
        dict(name="rope trees", op="rope", seqs=8, tokens=27, heads=24, kv_heads=8, head_dim=128, rot=32, type="bf16",
             norm=True, interleaved=True, scaling="none", base=2000, room=2048),
        # a long prompt far out in a scaled context
        dict(name="rope prompt", op="rope", seqs=1, tokens=8192, heads=32, kv_heads=8, head_dim=64, rot=64, type="f32",
             norm=True, interleaved=False, scaling="yarn", base=120000, room=8192),
        # one token over a short context: the smallest attention call
        dict(name="attend one token", op="attend", seqs=1, nodes=1, heads=32, kv_heads=8, head_dim=64, type="f32",
             length=191, spread=0, count_spread=0, room=256),
        # a tree of 16 over the long single-sequence context
        dict(name="attend tree 8k", op="attend", seqs=1, nodes=16, heads=32, kv_heads=8, head_dim=64, type="f32",
             length=8192, spread=0, count_spread=0, room=8256),
        # a ragged serving batch with large trees, some of them not full
        dict(name="attend ragged batch", op="attend", seqs=8, nodes=61, heads=32, kv_heads=8, head_dim=64, type="bf16",
             length=8192, spread=6001, count_spread=17, room=8256),
        # three query heads per kv head, odd tree and length, heads of 128
        dict(name="attend odd groups", op="attend", seqs=2, nodes=33, heads=24, kv_heads=8, head_dim=128, type="f32",
             length=2047, spread=300, count_spread=2, room=2304),
        # a small tree at the end of a very long context
        dict(name="attend long context", op="attend", seqs=1, nodes=8, heads=24, kv_heads=8, head_dim=128, type="bf16",
             length=131071, spread=0, count_spread=0, room=131136),
        # the accepted path of one sequence
        dict(name="compact one", op="compact", layers=16, slots=1, kv_heads=8, head_dim=64, room=1024, nodes=16,
             accepted=5, start=800),
        # the accepted paths of eight sequences with heads of 128
        dict(name="compact batch", op="compact", layers=28, slots=8, kv_heads=8, head_dim=128, room=1024, nodes=64,
             accepted=40, start=900),
        # four hypotheses of a small model exchanged
        dict(name="reorder small", op="reorder", layers=2, slots=4, kv_heads=2, head_dim=64, room=256, length=100,
             spread=31, moved=3),
        # a prompt's cache forked over a batch of eight
        dict(name="reorder batch", op="reorder", layers=16, slots=8, kv_heads=8, head_dim=64, room=2048, length=2000,
             spread=301, moved=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "compact", "reorder"])
    head_dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        seqs, total = _log(rng, 1, 8), _log(rng, 1, 4096)
        tokens = max(1, total // seqs)
        rot = rng.choice([head_dim, head_dim // 2, head_dim // 4, 2 * rng.randint(1, head_dim // 2)])
        return dict(op=op, seqs=seqs, tokens=tokens, heads=kv_heads * min(group, 4), kv_heads=kv_heads,
                    head_dim=head_dim, rot=rot, type=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "wavelength", "yarn"]),
                    base=_log(rng, 1, 120000), room=tokens + rng.randint(0, 300))
    if op == "attend":
        seqs, nodes, length = _log(rng, 1, 8), _log(rng, 1, 64), _log(rng, 1, 32768)
        length = min(length, int(18e9 / (4 * seqs * nodes * kv_heads * group * head_dim)))
        return dict(op=op, seqs=seqs, nodes=nodes, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim,
                    type=rng.choice(["f32", "bf16"]), length=length, spread=rng.randint(0, length),
                    count_spread=rng.randint(0, nodes - 1), room=length + nodes + rng.randint(0, 100))
    if op == "compact":
        nodes = _log(rng, 1, 64)
        start = _log(rng, 1, 2000)
        return dict(op=op, layers=rng.randint(1, 28), slots=_log(rng, 1, 8), kv_heads=kv_heads, head_dim=head_dim,
                    room=start + nodes + rng.randint(0, 50), nodes=nodes, accepted=rng.randint(1, nodes), start=start)
    slots, layers = rng.randint(2, 8), rng.randint(1, 16)
    length = min(_log(rng, 1, 8000), int(3.6e8 / (4 * slots * layers * kv_heads * head_dim)))
    return dict(op=op, layers=layers, slots=slots, kv_heads=kv_heads, head_dim=head_dim,
                room=length + rng.randint(0, 100), length=length, spread=rng.randint(0, length - 1),
                moved=rng.randint(1, slots))


def _ragged(value, spread, n):
    """n whole numbers falling from value to value - spread."""
    return [value - (spread * i) // max(1, n - 1) for i in range(n)]


def work(case):
    c, size = case, {"f32": 4, "bf16": 2}
    if c["op"] == "rope":
        n, e = c["seqs"] * c["tokens"], size[c["type"]]
        rows = c["heads"] + 2 * c["kv_heads"]
        per = rows * c["head_dim"] * e + c["heads"] * c["head_dim"] * e + 4 * c["kv_heads"] * c["head_dim"] + 12
        return {"bytes": n * per, "flops": n * rows * c["head_dim"] * 6}
    if c["op"] == "attend":
        lens = _ragged(c["length"], c["spread"], c["seqs"])
        counts = _ragged(c["nodes"], c["count_spread"], c["seqs"])
        kv = sum(a + t for a, t in zip(lens, counts)) * c["kv_heads"] * c["head_dim"] * 4
        qo = 2 * sum(counts) * c["heads"] * c["head_dim"] * size[c["type"]]
        flops = sum(4 * t * (a + t) for a, t in zip(lens, counts)) * c["heads"] * c["head_dim"]
        return {"bytes": kv + qo, "flops": flops}
    row = c["layers"] * c["kv_heads"] * c["head_dim"] * 4
    if c["op"] == "compact":
        return {"bytes": 2 * c["slots"] * _accepted(c) * row, "flops": 0}
    lens = _ragged(c["length"], c["spread"], c["slots"])
    return {"bytes": 2 * sum(lens[: c["moved"]]) * row, "flops": 0}


def _accepted(c):
    return min(c["accepted"], c["nodes"])


# ---------------------------------------------------------------- inputs
def _scaling(c):
    """Frequencies (radians a position) of the rotated pairs, in 64 bits, and the factor on the rotated values."""
    half, theta, factor, original = c["rot"] // 2, 5e5, 8.0, 8192
    i = torch.arange(half, dtype=torch.float64)
    f = theta ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "wavelength":
        turns = original * f / (2 * math.pi)
        s = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * ((1 - s) / factor + s), 1.0
    if c["scaling"] == "yarn":
        at = [c["rot"] * math.log(original / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(c["rot"] - 1, math.ceil(at[1]))
        ramp = ((i - lo) / max(1e-3, hi - lo)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _parents(n, gen):
    """A tree in node order: node 0 the root, each other node below one of the last few before it."""
    back = torch.randint(1, 9, (n,), generator=gen)
    t = torch.arange(n)
    return torch.where(t == 0, torch.full_like(t, -1), (t - back).clamp(min=0))


def _mask_words(parents):
    """Bit j of word t: node j is node t or one of its ancestors (the closure of `parents`)."""
    n = len(parents)
    step = torch.eye(n, dtype=torch.float64)
    step[torch.arange(1, n), parents[1:]] = 1
    seen = torch.linalg.matrix_power(step, n) > 0
    return (seen.long() << torch.arange(n)).sum(-1)


def _normal(g, dev, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    h = torch.Generator().manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device=dev)
    s = {"case": c}
    if c["op"] == "rope":
        B, n, D = c["seqs"], c["tokens"], c["head_dim"]
        dt = DTYPES[c["type"]]
        s["qkv"] = _normal(g, dev, B * n, (c["heads"] + 2 * c["kv_heads"]) * D, dtype=dt)
        s["q_out"] = torch.empty(B * n, c["heads"], D, dtype=dt, device=dev)
        s["k"] = _normal(g, dev, B, c["kv_heads"], c["room"], D)
        s["v"] = _normal(g, dev, B, c["kv_heads"], c["room"], D)
        # a sequence's tokens sit in consecutive rows; their positions are those of a tree's depths or of a prompt
        first = torch.randint(0, c["room"] - n + 1, (B,), generator=h)
        depth = torch.arange(n) // (4 if n <= 64 else 1)
        s["rows"] = (first[:, None] + torch.arange(n)[None]).reshape(-1).to(**i32)
        s["positions"] = (c["base"] + first[:, None] + depth[None]).reshape(-1).to(**i32)
        s["slots"] = torch.arange(B).repeat_interleave(n).to(**i32)
        freq, s["mscale"] = _scaling(c)
        s["freq"] = freq.to(dev)
        if c["norm"]:
            s["q_norm"] = (1 + 0.05 * _normal(g, dev, D, dtype=torch.float32)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.05 * _normal(g, dev, D, dtype=torch.float32)).to(torch.bfloat16)
        else:
            s["q_norm"] = s["k_norm"] = None
    elif c["op"] == "attend":
        B, T, D = c["seqs"], c["nodes"], c["head_dim"]
        s["q"] = 1.5 * _normal(g, dev, B, T, c["heads"], D, dtype=torch.float32)
        s["q"] = s["q"].to(DTYPES[c["type"]])
        s["out"] = torch.zeros(B, T, c["heads"], D, dtype=DTYPES[c["type"]], device=dev)
        s["k"] = _normal(g, dev, B, c["kv_heads"], c["room"], D)
        s["v"] = _normal(g, dev, B, c["kv_heads"], c["room"], D)
        s["lengths"] = torch.tensor(_ragged(c["length"], c["spread"], B), **i32)
        s["counts"] = torch.tensor(_ragged(T, c["count_spread"], B), **i32)
        s["masks"] = torch.stack([_mask_words(_parents(T, h)) for _ in range(B)]).to(dev)
    else:
        L, B = c["layers"], c["slots"]
        s["k"] = _normal(g, dev, L, B, c["kv_heads"], c["room"], c["head_dim"])
        s["v"] = _normal(g, dev, L, B, c["kv_heads"], c["room"], c["head_dim"])
        if c["op"] == "compact":
            nodes = [torch.randperm(c["nodes"], generator=h)[: _accepted(c)].sort().values for _ in range(B)]
            pad = torch.zeros(c["nodes"] - _accepted(c), dtype=torch.int64)
            s["nodes"] = torch.stack([torch.cat([x, pad]) for x in nodes]).to(**i32)
            s["counts"] = torch.full((B,), _accepted(c), **i32)
            s["starts"] = torch.tensor([max(0, c["start"] - int(x)) for x in torch.randint(0, 40, (B,), generator=h)],
                                       **i32)
        else:
            # the first `moved` slots take another slot's rows: forks and exchanges among them
            src = torch.arange(B)
            src[: c["moved"]] = (src[: c["moved"]] + torch.randint(1, B, (c["moved"],), generator=h)) % B
            s["sources"] = src.to(**i32)
            s["lengths"] = torch.tensor(_ragged(c["length"], c["spread"], B), **i32)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return {"rope": _rope, "attend": _attend, "compact": _compact, "reorder": _reorder}[state["case"]["op"]](state)


def _rope(s):
    c = s["case"]
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.rope_append(s["qkv"], s["q_out"], s["k"], s["v"], s["positions"], s["rows"], s["freq"], slots=s["slots"],
                         q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-5, mscale=s["mscale"],
                         interleaved=c["interleaved"])
        return s["q_out"], s["k"], s["v"]
    H, K, D, r = c["heads"], c["kv_heads"], c["head_dim"], c["rot"]
    x = s["qkv"].float().view(-1, H + 2 * K, D)
    q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-5) * s["q_norm"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-5) * s["k_norm"].float()
    angle = s["positions"].double()[:, None] * s["freq"][None]
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]

    def rotate(y):
        if c["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., r:]], -1)
        a, b = y[..., : r // 2], y[..., r // 2: r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., r:]], -1)

    s["q_out"].copy_(rotate(q))
    slots, rows = s["slots"].long(), s["rows"].long()
    s["k"][slots, :, rows] = rotate(k).to(torch.bfloat16)
    s["v"][slots, :, rows] = v.to(torch.bfloat16)
    return s["q_out"], s["k"], s["v"]


def _attend(s):
    c = s["case"]
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.tree_attention(s["q"], s["k"], s["v"], s["lengths"], s["masks"], s["out"], counts=s["counts"],
                            max_len=c["length"])
        return s["out"]
    B, T, H, K, D = c["seqs"], c["nodes"], c["heads"], c["kv_heads"], c["head_dim"]
    n = c["length"] + T
    k, v = s["k"][:, :, :n].float(), s["v"][:, :, :n].float()
    q = s["q"].float().view(B, T, K, H // K, D).permute(0, 2, 1, 3, 4).reshape(B, K, T * (H // K), D)
    score = (q @ k.transpose(-1, -2)) * (D ** -0.5)
    at = torch.arange(n, device=k.device)[None, None] - s["lengths"].long()[:, None, None]
    bit = (s["masks"][:, :, None] >> at.clamp(0, 63)) & 1
    seen = (at < 0) | ((at < s["counts"][:, None, None]) & (bit == 1))
    seen = seen[:, None, :, None].expand(B, 1, T, H // K, n).reshape(B, 1, T * (H // K), n)
    score = torch.where(seen, score, float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    o = o.view(B, K, T, H // K, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    live = (torch.arange(T, device=k.device)[None] < s["counts"][:, None])[:, :, None, None]
    s["out"].copy_(torch.where(live, o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _compact(s):
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.kv_compact(s["k"], s["v"], s["starts"], s["nodes"], s["counts"])
        return s["k"], s["v"]
    c = s["case"]
    n = _accepted(c)
    start = s["starts"].long()[:, None]
    source = start + s["nodes"].long()[:, :n]
    target = start + torch.arange(n, device=source.device)[None]
    slot = torch.arange(c["slots"], device=source.device)[:, None]
    s["k"][:, slot, :, target] = s["k"][:, slot, :, source]
    s["v"][:, slot, :, target] = s["v"][:, slot, :, source]
    return s["k"], s["v"]


def _reorder(s):
    if own:
        from decode_megakernel_llama_gb300 import _lib
        _lib.kv_reorder(s["k"], s["v"], s["sources"], s["lengths"])
        return s["k"], s["v"]
    c = s["case"]
    m = c["moved"]  # the slots behind the moved ones keep their own rows
    take = (torch.arange(c["length"], device=s["k"].device)[None] < s["lengths"][:m, None])[None, :, None, :, None]

    def taken(x):
        old = x[:, :, :, : c["length"]]
        return torch.where(take, old.index_select(1, s["sources"][:m]), old[:, :m])

    s["k"][:, :m, :, : c["length"]] = taken(s["k"])
    s["v"][:, :m, :, : c["length"]] = taken(s["v"])
    return s["k"], s["v"]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        H, K, D, r = c["heads"], c["kv_heads"], c["head_dim"], c["rot"]
        x = s["qkv"].double().reshape(-1, H + 2 * K, D).clone()
        if c["norm"]:
            for part, gain in ((slice(0, H), s["q_norm"]), (slice(H, H + K), s["k_norm"])):
                ms = x[:, part].pow(2).sum(-1, keepdim=True) / D
                x[:, part] = x[:, part] / (ms + 1e-5).sqrt() * gain.double()
        angle = torch.outer(s["positions"].double(), s["freq"])
        turn = torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None]
        first = torch.arange(r // 2, device=x.device) * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else r // 2)
        z = torch.complex(x[:, : H + K, first], x[:, : H + K, second]) * turn
        x[:, : H + K, first], x[:, : H + K, second] = z.real, z.imag
        k, v = s["k"].double(), s["v"].double()
        for b in range(c["seqs"]):
            of = (s["slots"] == b).nonzero()[:, 0]
            rows = s["rows"][of].long()
            k[b, :, rows] = x[of, H:H + K].transpose(0, 1)
            v[b, :, rows] = x[of, H + K:].transpose(0, 1)
        return x[:, :H].contiguous(), k, v
    if c["op"] == "attend":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
        G = c["heads"] // c["kv_heads"]
        for b in range(c["seqs"]):
            n, t = int(s["lengths"][b]), int(s["counts"][b])
            seen = torch.ones(t, n + t, dtype=torch.bool)
            for i, w in enumerate(s["masks"][b, :t].tolist()):
                seen[i, n:] = torch.tensor([bool((w >> j) & 1) for j in range(t)])
            seen = seen.to(out.device)
            for h in range(c["heads"]):
                k, v = s["k"][b, h // G, : n + t].double(), s["v"][b, h // G, : n + t].double()
                score = (s["q"][b, :t, h].double() @ k.T / math.sqrt(c["head_dim"])).masked_fill(~seen, -math.inf)
                out[b, :t, h] = torch.softmax(score, -1) @ v
        return out
    k, v = s["k"].double(), s["v"].double()
    if c["op"] == "compact":
        for x in (k, v):
            for b in range(c["slots"]):
                a = int(s["starts"][b])
                rows = [a + i for i in s["nodes"][b, : int(s["counts"][b])].tolist()]
                x[:, b, :, a: a + len(rows)] = x[:, b][:, :, rows].clone()
        return k, v
    for x in (k, v):
        old = x.clone()
        for b, src in enumerate(s["sources"].tolist()):
            x[:, b, :, : int(s["lengths"][b])] = old[:, src, :, : int(s["lengths"][b])]
    return k, v
