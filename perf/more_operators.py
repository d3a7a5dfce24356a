"""Cases for further operators on the paged FP8 latent cache: dense decode with capped, biased and masked scores, decode of
a batch that shares a long prefix, attention weights accumulated per cached position, and eviction by those weights.

`run` computes them with elementary torch operations in 32 bits (`own` false) or calls the package (`own` true).
The cache record is 656 bytes: 512 E4M3 codes, 4 float32 scales (one per 128 dims), 64 bf16 rope values; pages of 64.
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, REC = 64, 512, 64, 656


def listed():
    return [
        # one session of a few hundred tokens on a slice of 16 heads, scores capped: latency
        dict(name="masked_b1_h16_500", op="masked", requests=1, heads=16, queries=1, ctx=500, spread=1.0, cap=30.0,
             slopes=False, mask="none", window=0, prefix=0),
        # a batch of layers with a sliding window that also keeps the first tokens
        dict(name="masked_b32_h64_window", op="masked", requests=32, heads=64, queries=1, ctx=32768, spread=8.0, cap=0.0,
             slopes=False, mask="window", window=4096, prefix=64),
        # scores capped and biased by distance over whole contexts, two tokens per request to verify
        dict(name="masked_b8_h64_q2_bias", op="masked", requests=8, heads=64, queries=2, ctx=20011, spread=1.0, cap=50.0,
             slopes=True, mask="none", window=0, prefix=0),
        # several documents packed into each request behind a common prompt, 128 heads
        dict(name="masked_b16_h128_docs", op="masked", requests=16, heads=128, queries=1, ctx=16384, spread=2.0, cap=0.0,
             slopes=False, mask="document", window=0, prefix=700),
        # four samples of one prompt of a thousand tokens
        dict(name="shared_b4_h16_1k", op="shared", requests=4, groups=1, heads=16, queries=1, prefix=1000, suffix=60,
             spread=4.0),
        # a batch of 64 on a slice of 16 heads behind one long system prompt
        dict(name="shared_b64_h16_32k", op="shared", requests=64, groups=1, heads=16, queries=1, prefix=32768, suffix=600,
             spread=30.0),
        # the benchmark's batch of 32 and 64 heads, over one shared document
        dict(name="shared_b32_h64_32k", op="shared", requests=32, groups=1, heads=64, queries=1, prefix=32768, suffix=1024,
             spread=64.0),
        # four prompts with eight samples each, two tokens per request to verify, odd lengths
        dict(name="shared_b32_g4_q2_9k", op="shared", requests=32, groups=4, heads=32, queries=2, prefix=9001, suffix=333,
             spread=9.0),
        # one session's step
        dict(name="weights_b1_h16_300", op="weights", requests=1, heads=16, queries=1, ctx=300, spread=1.0, decay=1.0),
        # the benchmark's batch, weights that fade
        dict(name="weights_b32_h64_32k", op="weights", requests=32, heads=64, queries=1, ctx=32768, spread=1.0, decay=0.98),
        # one request that is a little over its budget
        dict(name="evict_b1_4k", op="evict", requests=1, ctx=4160, spread=1.0, keep=4096, sinks=4, recent=128),
        # a batch cut to half of its cache
        dict(name="evict_b32_32k", op="evict", requests=32, ctx=32768, spread=2.0, keep=16384, sinks=16, recent=1024),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["masked", "masked", "shared", "shared", "weights", "evict"])
    heads = rng.choice([1, 5, 8, 16, 24, 32, 64, 128])
    queries = rng.choice([1, 1, 2, 3])
    if op == "masked":
        requests = _log(rng, 1, 64)
        most = (1 << 19) // (requests * max(1, heads * queries // 64))
        mask = rng.choice(["none", "window", "document"])
        return dict(op=op, requests=requests, heads=heads, queries=queries, ctx=_log(rng, 3, max(3, min(most, 131072))),
                    spread=rng.choice([1.0, 4.0, 100.0]), cap=rng.choice([0.0, 20.0, 50.0]), slopes=rng.random() < 0.4,
                    mask=mask, window=_log(rng, 1, 8192) if mask == "window" else 0,
                    prefix=rng.choice([0, 4, 777]) if mask != "none" else 0)
    if op == "shared":
        groups = rng.choice([1, 1, 1, 2, 5])
        requests = groups * _log(rng, 1, 64 // groups)
        most = (1 << 26) // (requests * heads * queries)
        return dict(op=op, requests=requests, groups=groups, heads=heads, queries=queries,
                    prefix=_log(rng, 40, max(40, min(most, 65536 // groups))), suffix=_log(rng, 1, 1024),
                    spread=rng.choice([1.0, 5.0, 64.0]))
    if op == "weights":
        requests = _log(rng, 1, 64)
        most = (1 << 19) // (requests * max(1, heads * queries // 64))
        return dict(op=op, requests=requests, heads=heads, queries=queries, ctx=_log(rng, 3, max(3, min(most, 131072))),
                    spread=rng.choice([1.0, 4.0, 100.0]), decay=rng.choice([1.0, 0.9, 0.0]))
    requests = _log(rng, 1, 64)
    ctx = _log(rng, 70, (1 << 19) // requests)
    return dict(op=op, requests=requests, ctx=ctx, spread=rng.choice([1.0, 3.0]), keep=max(1, int(ctx * rng.random())),
                sinks=rng.choice([0, 4, 50]), recent=rng.choice([0, 17, 256]))


def _lengths(n, ctx, spread):
    """Length of each request: fixed, or log-uniform from ctx / spread to ctx in a mixed order."""
    if spread == 1.0:
        return [ctx] * n
    lens = [max(1, int(ctx * spread ** (-(i + 0.5) / n))) for i in range(n)]
    lens[0] = ctx
    return [lens[(i * 37 + 11) % n] if math.gcd(37, n) == 1 else lens[i] for i in range(n)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _records(n, g):
    """n records of unit-variance latents (one channel in a hundred eight times larger) and rope values."""
    out = torch.empty((n, REC), dtype=torch.uint8, device="cuda")
    gain = torch.where(torch.rand(LATENT, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    for at in range(0, n, 1 << 18):
        m = min(1 << 18, n - at)
        x = (torch.randn((m, LATENT), generator=g, device="cuda") * gain).view(m, 4, 128)
        scale = x.abs().amax(-1) / 448.0
        out[at:at + m, :512] = (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(m, 512).view(torch.uint8)
        out[at:at + m, 512:528] = scale.view(torch.uint8)
        out[at:at + m, 528:] = torch.randn((m, ROPE), generator=g, device="cuda").to(torch.bfloat16).view(torch.uint8)
    return out


def _tables(lens, g, first=0):
    """Block table of requests of these lengths over pages first, first + 1, ... in a random order; pages used."""
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    total = sum(pages)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32) + first
    begin = torch.tensor([0] + pages, device="cuda").cumsum(0)
    col = torch.arange(max(1, max(pages)), device="cuda")
    at = begin[:-1, None] + col
    used = col < torch.tensor(pages, device="cuda")[:, None]
    return torch.where(used, perm[at.clamp_max(max(0, total - 1))] if total else at.to(torch.int32), -1).contiguous(), total


def _query_lengths(lens, nq):
    back = torch.arange(nq - 1, -1, -1, device="cuda")
    return (torch.tensor(lens, device="cuda")[:, None] - back).clamp_min(0).reshape(-1).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "scale": 1.0 / math.sqrt(LATENT + ROPE)}
    R = case["requests"]
    if case["op"] == "evict":
        return _prepare_evict(s, case, g)
    nq, H = case["queries"], case["heads"]
    rows = R * nq
    s["q"] = torch.randn((rows, H, LATENT + ROPE), generator=g, device="cuda").to(torch.bfloat16)
    s["out"] = torch.empty((rows, H, LATENT), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((rows, H), device="cuda")
    if case["op"] == "shared":
        s["pbt"], n0 = _tables([case["prefix"] - 3 * i for i in range(case["groups"])], g)
        s["plens"] = torch.tensor([case["prefix"] - 3 * i for i in range(case["groups"])], dtype=torch.int32, device="cuda")
        lens = _lengths(R, case["suffix"], case["spread"])
        s["bt"], n1 = _tables(lens, g, n0)
        s["lens"] = _query_lengths(lens, nq)
        s["cache"] = _records((n0 + n1) * PAGE, g).view(n0 + n1, PAGE, REC)
        if own:      # the workspace that a program keeps for its decode calls
            from sparse_mla_decode_paged_gb300 import api
            s["ws"] = api.alloc_shared_workspace(s["q"], s["cache"], s["pbt"], s["bt"])
        return s
    lens = _lengths(R, case["ctx"], case["spread"])
    s["bt"], n = _tables(lens, g)
    s["lens"] = _query_lengths(lens, nq)
    s["cache"] = _records(n * PAGE, g).view(n, PAGE, REC)
    if case["op"] == "weights":
        s["lse"] = _lse(s)                                  # as the step's decode gave it
        s["weights"] = 0.01 * torch.rand((R, s["bt"].shape[1] * PAGE), generator=g, device="cuda")
        return s
    if case["cap"]:
        s["q"] = (s["q"].float() * 6).to(torch.bfloat16)    # scores that reach the cap
    s["slopes"] = s["starts"] = s["prefix"] = None
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    if case["mask"] == "window":
        s["starts"] = (s["lens"] - case["window"]).clamp_min(0)
    elif case["mask"] == "document":                        # the last document begins somewhere in the request
        at = torch.rand(R, generator=g, device="cuda") * torch.tensor(lens, device="cuda")
        s["starts"] = at.to(torch.int32).repeat_interleave(nq)
    if case["prefix"]:
        s["prefix"] = torch.full((rows,), case["prefix"], dtype=torch.int32, device="cuda")
    if own:          # the workspace that a program keeps for its decode calls
        from sparse_mla_decode_paged_gb300 import api
        s["ws"] = api.alloc_dense_workspace(api.dense_dims_of(s["q"], s["cache"], s["bt"]), s["q"].device)
    return s


def _prepare_evict(s, case, g):
    R = case["requests"]
    lens = _lengths(R, case["ctx"], case["spread"])
    s["bt"], n = _tables(lens, g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cache"] = _records(n * PAGE, g).view(n, PAGE, REC)
    cols = s["bt"].shape[1] * PAGE
    # heavy-tailed sums, one slot in twenty never looked at (ties at 0)
    w = torch.exp(2.0 * torch.randn((R, cols), generator=g, device="cuda"))
    s["weights"] = torch.where(torch.rand((R, cols), generator=g, device="cuda") < 0.05, 0.0, w)
    # positions with gaps, the first half of the slots mixed by earlier evictions
    pos = torch.randint(1, 3, (R, cols), generator=g, device="cuda").cumsum(1) - 1
    half = max(1, min(lens) // 2)
    mixed = torch.rand((R, half), generator=g, device="cuda").argsort(1)
    s["positions"] = torch.cat([pos[:, :half].gather(1, mixed), pos[:, half:]], 1).to(torch.int32)
    s["next"] = (pos.gather(1, (s["lens"].long() - 1)[:, None])[:, 0] + 1).to(torch.int32)
    if own:          # the workspace that a program keeps for its evictions
        from sparse_mla_decode_paged_gb300 import api
        s["ws"] = api.alloc_evict_workspace(s["weights"])
    return s


def _unpack(rec):
    """Records [.., 656] -> latent * scale [.., 512], rope [.., 64] in float32."""
    lat = rec[..., :512].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    lat = (lat * rec[..., 512:528].contiguous().view(torch.float32)[..., None]).flatten(-2)
    return lat, rec[..., 528:].contiguous().view(torch.bfloat16).float()


def _scores(s, table, q, per):
    """Scores [rows of the table, per, positions] of q (per rows of q for each row of the table), and the latents."""
    lat, rope = _unpack(s["cache"][table.long().clamp_min(0)].flatten(1, 2))
    k = torch.cat([lat, rope], -1)
    return (q.float().view(table.shape[0], per, LATENT + ROPE) @ k.transpose(1, 2)) * s["scale"], lat


def _lse(s):
    """lse of a plain decode, a few requests at a time."""
    c = s["case"]
    nq, H, R = c["queries"], c["heads"], c["requests"]
    out = []
    for r in range(R):
        sc, _ = _scores(s, s["bt"][r:r + 1], s["q"][r * nq:(r + 1) * nq], nq * H)
        sc = sc.view(nq, H, -1)
        t = torch.arange(sc.shape[-1], device="cuda")
        sc = sc.masked_fill(t >= s["lens"][r * nq:(r + 1) * nq].view(nq, 1, 1), -math.inf)
        m = sc.amax(-1, keepdim=True).clamp_min(-3e38)
        out.append((m + torch.log(torch.exp(sc - m).sum(-1, keepdim=True))).squeeze(-1))
    return torch.cat(out)


def _softmax(sc):
    """Weights over the last dim, 0 in rows without positions, and lse."""
    m = sc.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    return p / z.clamp_min(1e-38), (m + torch.log(z)).squeeze(-1)


def _plain_masked(s):
    c = s["case"]
    R, nq, H = c["requests"], c["queries"], c["heads"]
    sc, lat = _scores(s, s["bt"], s["q"], nq * H)
    sc = sc.view(R, nq, H, -1)
    n = s["lens"].view(R, nq, 1, 1)
    t = torch.arange(sc.shape[-1], device="cuda")
    if c["cap"]:
        sc = c["cap"] * torch.tanh(sc / c["cap"])
    if s["slopes"] is not None:
        sc = sc + s["slopes"].view(1, 1, H, 1) * (t - (n - 1)).float()
    seen = t < n
    if s["starts"] is not None:
        late = t >= s["starts"].view(R, nq, 1, 1)
        seen = seen & (late if s["prefix"] is None else late | (t < s["prefix"].view(R, nq, 1, 1)))
    p, lse = _softmax(sc.masked_fill(~seen, -math.inf))
    return (p.view(R, nq * H, -1) @ lat).view(R * nq, H, LATENT).to(torch.bfloat16), lse.view(R * nq, H)


def _plain_shared(s):
    c = s["case"]
    R, G, nq, H = c["requests"], c["groups"], c["queries"], c["heads"]
    a, lat_a = _scores(s, s["pbt"], s["q"], R // G * nq * H)               # [G, rows, prefix]
    b, lat_b = _scores(s, s["bt"], s["q"], nq * H)                         # [R, rows, own]
    n0 = a.shape[-1]
    a = a.masked_fill(torch.arange(n0, device="cuda") >= s["plens"].view(G, 1, 1), -math.inf).view(R, nq, H, n0)
    b = b.view(R, nq, H, -1)
    b = b.masked_fill(torch.arange(b.shape[-1], device="cuda") >= s["lens"].view(R, nq, 1, 1), -math.inf)
    p, lse = _softmax(torch.cat([a, b], -1))
    o = (p[..., :n0].reshape(G, -1, n0) @ lat_a).view(R, nq * H, LATENT) + p[..., n0:].reshape(R, nq * H, -1) @ lat_b
    return o.view(R * nq, H, LATENT).to(torch.bfloat16), lse.view(R * nq, H)


def _plain_weights(s):
    c = s["case"]
    R, nq, H = c["requests"], c["queries"], c["heads"]
    sc, _ = _scores(s, s["bt"], s["q"], nq * H)
    sc = sc.view(R, nq, H, -1)
    n = s["lens"].view(R, nq, 1, 1)
    t = torch.arange(sc.shape[-1], device="cuda")
    p = torch.exp(sc - s["lse"].view(R, nq, H, 1)).masked_fill(t >= n, 0.0)
    return torch.where(t < n.amax((1, 2, 3))[:, None], c["decay"] * s["weights"] + p.sum((1, 2)), s["weights"])


def _cache_parts(cache):
    """The whole cache as the values it stands for: codes, scales and rope (views)."""
    return {"codes": cache[..., :512].view(torch.float8_e4m3fn), "scales": cache[..., 512:528].view(torch.float32),
            "rope": cache[..., 528:].view(torch.bfloat16)}


def _slots(table, r, t):
    return table[r, t // PAGE].long() * PAGE + t % PAGE


def _plain_evict(s, w, pos):
    c = s["case"]
    n, t = s["lens"].long()[:, None], torch.arange(w.shape[1], device="cuda")
    held = (t < n) & ((pos < c["sinks"]) | (pos >= s["next"][:, None] - c["recent"]))
    bits = w.view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits)                   # the order of the values as whole numbers
    key = torch.where(held, 1 << 40, torch.where(t < n, key, -(1 << 40)))
    order = key.sort(dim=1, descending=True, stable=True).indices              # equal keys: the lower slot first
    keep = torch.minimum(n, held.sum(1, keepdim=True).clamp_min(c["keep"]))
    kept = torch.zeros_like(held).scatter_(1, order, t < keep)
    (r0, src), (r1, dst) = (kept & (t >= keep)).nonzero(as_tuple=True), (~kept & (t < keep)).nonzero(as_tuple=True)
    flat = s["cache"].view(-1, REC)
    flat[_slots(s["bt"], r1, dst)] = flat[_slots(s["bt"], r0, src)]
    w[r1, dst] = w[r0, src]
    pos[r1, dst] = pos[r0, src]
    w.masked_fill_((t >= keep) & (t < n), 0.0)
    return keep[:, 0].to(torch.int32)


def run(s):
    c = s["case"]
    if own:
        from sparse_mla_decode_paged_gb300 import api
        if c["op"] == "masked":
            return api.sparse_mla_masked_decode(s["q"], s["cache"], s["bt"], s["lens"], s["scale"], softcap=c["cap"],
                                                slopes=s["slopes"], starts=s["starts"], prefix_lens=s["prefix"],
                                                out=s["out"], lse=s["lse"], workspace=s["ws"])
        if c["op"] == "shared":
            return api.sparse_mla_shared_decode(s["q"], s["cache"], s["pbt"], s["plens"], s["bt"], s["lens"], s["scale"],
                                                out=s["out"], lse=s["lse"], workspace=s["ws"])
        if c["op"] == "weights":
            return api.sparse_mla_attention_weights(s["q"], s["cache"], s["bt"], s["lens"], s["lse"], s["scale"],
                                                    s["weights"].clone(), decay=c["decay"])
    elif c["op"] == "masked":
        return _plain_masked(s)
    elif c["op"] == "shared":
        return _plain_shared(s)
    elif c["op"] == "weights":
        return _plain_weights(s)
    # a pass evicts by the same weights again: the records that move are the same ones each time
    w, pos = s["weights"].clone(), s["positions"].clone()
    if own:
        n = api.sparse_mla_kv_evict(w, pos, s["next"], s["lens"], c["keep"], s["cache"], s["bt"], sinks=c["sinks"],
                                    recent=c["recent"], workspace=s["ws"])
    else:
        n = _plain_evict(s, w, pos)
    return {"lens": n, "weights": w, "positions": pos, **_cache_parts(s["cache"])}


def work(case):
    R = case["requests"]
    if case["op"] == "evict":
        lens = _lengths(R, case["ctx"], case["spread"])
        slots = sum(lens)
        # a kept record moves when its slot is behind the kept ones
        moved = sum(min(n, case["keep"]) * max(0, n - case["keep"]) / n for n in lens)
        return {"bytes": slots * 4 + moved * 2 * (REC + 8) + sum(max(0, n - case["keep"]) for n in lens) * 4, "flops": slots}
    nq, H = case["queries"], case["heads"]
    rows = R * nq * H
    if case["op"] == "shared":
        G = case["groups"]
        pre, lens = [case["prefix"] - 3 * i for i in range(G)], _lengths(R, case["suffix"], case["spread"])
        pairs = sum(pre) * (rows // G) + sum(max(0, n - j) for n in lens for j in range(nq)) * H
        return {"bytes": (sum(pre) + sum(lens)) * REC + rows * (1152 + 1024 + 4), "flops": 2 * 1088 * pairs}
    lens = _lengths(R, case["ctx"], case["spread"])
    if case["op"] == "weights":
        pairs = sum(max(0, n - j) for n in lens for j in range(nq)) * H
        return {"bytes": sum(lens) * (REC + 4 + (4 if case["decay"] else 0)) + rows * (1152 + 4), "flops": 2 * 576 * pairs}
    seen = lens                                             # positions that a request's rows see
    if case["mask"] == "window":
        seen = [min(n, case["window"] + min(case["prefix"], max(0, n - case["window"]))) for n in lens]
    elif case["mask"] == "document":                        # on average
        seen = [n / 2 + min(case["prefix"], n / 2) for n in lens]
    return {"bytes": sum(seen) * REC + rows * (1152 + 1024 + 4), "flops": 2 * 1088 * sum(seen) * nq * H}


# --------------------------------------------------------------------------- the definitions in 64 bits

def _exact_code_values():
    c = torch.arange(256, device="cuda")
    e, m = (c >> 3 & 15).double(), (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    v[(c & 127) == 127] = math.nan
    return torch.where(c >= 128, -v, v)


def _exact_records(rec):
    v = _exact_code_values()[rec[:, :512].long()]
    scale = rec[:, 512:528].contiguous().view(torch.float32).double()
    rope = rec[:, 528:].contiguous().view(torch.bfloat16).double()
    return v * scale.repeat_interleave(128, 1), rope


def _exact_keys(s, row, n):
    """Latents and ropes of the first n positions of a block-table row."""
    t = torch.arange(n, device="cuda")
    return _exact_records(s["cache"].view(-1, REC)[row[t // PAGE].long() * PAGE + t % PAGE])


def _exact_dots(s, b, lat, rope):
    q = s["q"][b].double()
    return (q[:, :LATENT] @ lat.T + q[:, LATENT:] @ rope.T) * s["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s, case)
    R, nq, H = case["requests"], case["queries"], case["heads"]
    most = s["lens"].view(R, nq).amax(1).tolist()
    if case["op"] == "weights":
        w = s["weights"].double()
        for r in range(R):
            lat, rope = _exact_keys(s, s["bt"][r], most[r])
            w[r, :most[r]] *= case["decay"]
            for b in range(r * nq, (r + 1) * nq):
                n = int(s["lens"][b])
                z = _exact_dots(s, b, lat[:n], rope[:n]) - s["lse"][b].double()[:, None]
                w[r, :n] += torch.exp(z).sum(0)
        return w
    out = torch.zeros((R * nq, H, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((R * nq, H), -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "shared":
        each = R // case["groups"]
        pre = [_exact_keys(s, s["pbt"][g], int(s["plens"][g])) for g in range(case["groups"])]
    for r in range(R):
        lat, rope = _exact_keys(s, s["bt"][r], most[r])
        for b in range(r * nq, (r + 1) * nq):
            n = int(s["lens"][b])
            z, v = _exact_dots(s, b, lat[:n], rope[:n]), lat[:n]
            if case["op"] == "shared":
                z = torch.cat([_exact_dots(s, b, *pre[r // each]), z], 1)
                v = torch.cat([pre[r // each][0], v])
            else:
                t = torch.arange(n, device="cuda")
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    z = z - s["slopes"].double()[:, None] * (n - 1 - t).double()
                if s["starts"] is not None:
                    see = t >= s["starts"][b]
                    if s["prefix"] is not None:
                        see |= t < s["prefix"][b]
                    z, v = z[:, see], v[see]
            if z.shape[1]:
                lse[b] = torch.logsumexp(z, -1)
                out[b] = torch.softmax(z, -1) @ v
    return out, lse


def _exact_evict(s, case):
    """Slot by slot in lists, from the definition."""
    w, pos = s["weights"].double(), s["positions"].clone()
    flat, lens = s["cache"].view(-1, REC), []
    for r, n in enumerate(s["lens"].tolist()):
        at, value, last = pos[r, :n].tolist(), s["weights"][r, :n].tolist(), int(s["next"][r])
        held = [p < case["sinks"] or p >= last - case["recent"] for p in at]
        order = sorted(range(n), key=lambda t: (not held[t], 0.0 if held[t] else -value[t], t))
        m = min(n, max(case["keep"], sum(held)))
        kept = set(order[:m])
        src = [t for t in range(m, n) if t in kept]
        dst = [t for t in range(m) if t not in kept]
        if src:
            a, b = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
            row = s["bt"][r].long()
            flat[row[b // PAGE] * PAGE + b % PAGE] = flat[row[a // PAGE] * PAGE + a % PAGE]
            w[r, b], pos[r, b] = w[r, a], pos[r, a]
        w[r, m:n] = 0
        lens.append(m)
    return {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "weights": w, "positions": pos,
            **{k: v.double() for k, v in _cache_parts(s["cache"]).items()}}
