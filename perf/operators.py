"""Cases for the operators around the paged FP8 latent cache: dense decode over every cached position, the fused
norm + rotation + FP8 append that writes the cache, reading records back, and the per-head norm with rotation.

`run` computes them with elementary torch operations in 32 bits (`own` false) or calls the package (`own` true).
The cache record is 656 bytes: 512 E4M3 codes, 4 float32 scales (one per 128 dims), 64 bf16 rope values; pages of 64.
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, REC = 64, 512, 64, 656
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one request of a few tokens on one tensor-parallel slice of 16 heads: pure latency
        dict(name="dense_b1_h16_77", op="dense", requests=1, heads=16, queries=1, ctx=77, spread=1.0),
        # a single interactive session, 64 heads
        dict(name="dense_b1_h64_8k", op="dense", requests=1, heads=64, queries=1, ctx=8192, spread=1.0),
        # the benchmark's batch of 32 requests of 32768 positions each
        dict(name="dense_b32_h64_32k", op="dense", requests=32, heads=64, queries=1, ctx=32768, spread=1.0),
        # a ragged batch of 96 on 16 heads: lengths log-uniform from 64 to 32768
        dict(name="dense_b96_h16_ragged", op="dense", requests=96, heads=16, queries=1, ctx=32768, spread=512.0),
        # two tokens per request to verify, 128 heads, an odd length
        dict(name="dense_b4_h128_q2_20011", op="dense", requests=4, heads=128, queries=2, ctx=20011, spread=1.0),
        # one request over a long document
        dict(name="dense_b1_h64_512k", op="dense", requests=1, heads=64, queries=1, ctx=524288, spread=1.0),
        # a decode step's new tokens, one per request of a batch of 32
        dict(name="append_32", op="append", tokens=32, dtype="bf16", interleaved=True),
        # a chunk of prompts being written, an odd count
        dict(name="append_65521", op="append", tokens=65521, dtype="bf16", interleaved=True),
        # the queries of a decode step: 64 heads of 128 + 64 dims
        dict(name="norm_rope_32", op="norm_rope", tokens=32, heads=64, dim=192, rope_offset=128, dtype="bf16",
             interleaved=True),
        # the queries of a prompt chunk
        dict(name="norm_rope_8192", op="norm_rope", tokens=8192, heads=64, dim=192, rope_offset=128, dtype="bf16",
             interleaved=True),
        # a short prefix read back
        dict(name="read_100", op="read", tokens=100, dtype="bf16"),
        # the earlier context of a chunked prompt read back
        dict(name="read_131071", op="read", tokens=131071, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["dense", "dense", "dense", "append", "norm_rope", "read"])
    if op == "dense":
        heads = rng.choice([1, 5, 8, 16, 24, 32, 64, 128])
        queries = rng.choice([1, 1, 2, 3])
        requests = _log(rng, 1, 96)
        most = (1 << 20) // (requests * max(1, heads * queries // 64))
        return dict(op=op, requests=requests, heads=heads, queries=queries, ctx=_log(rng, 3, max(3, min(most, 524288))),
                    spread=rng.choice([1.0, 1.0, 8.0, 300.0]))
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 32768), dtype=dtype, interleaved=rng.random() < 0.5)
    if op == "norm_rope":
        dim, off = rng.choice([(64, 0), (128, 0), (128, 64), (192, 128), (576, 512)])
        heads = _log(rng, 1, 128)
        return dict(op=op, tokens=_log(rng, 1, max(1, (1 << 25) // (heads * dim))), heads=heads, dim=dim, rope_offset=off,
                    dtype=dtype, interleaved=rng.random() < 0.5)
    return dict(op=op, tokens=_log(rng, 1, 65536), dtype=dtype)


def _lengths(case):
    """Context length of each request: fixed, or log-uniform from ctx / spread to ctx in a mixed order."""
    n, ctx, spread = case["requests"], case["ctx"], case["spread"]
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


def _table(positions, base=10000.0):
    """cos (first half) and sin (second half) of the rotation angles, one row per position, float32."""
    freq = base ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], -1).float().contiguous()


def _paged_tokens(case, g):
    """Tokens of a few requests at consecutive positions: (requests, positions, block table, pages)."""
    n = case["tokens"]
    per = 1 if n <= 64 else (n + 7) // 8                     # a decode step's tokens, or prompts of up to eight requests
    i = torch.arange(n, device="cuda")
    rows = (n + per - 1) // per
    start = torch.randint(0, 500, (rows,), generator=g, device="cuda")
    req = i // per
    pos = i % per + start[req]
    width = (per + 500 + PAGE - 1) // PAGE
    bt = torch.randperm(rows * width, generator=g, device="cuda").view(rows, width).to(torch.int32)
    return req.to(torch.int32), pos.to(torch.int32), bt, rows * width


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "dense":
        lens = _lengths(case)
        pages = [(n + PAGE - 1) // PAGE for n in lens]
        total = sum(pages)
        s["cache"] = _records(total * PAGE, g).view(total, PAGE, REC)
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + pages, device="cuda").cumsum(0)
        col = torch.arange(max(pages), device="cuda")
        at = first[:-1, None] + col
        s["bt"] = torch.where(col < torch.tensor(pages, device="cuda")[:, None], perm[at.clamp_max(total - 1)], -1).contiguous()
        nq = case["queries"]
        back = torch.arange(nq - 1, -1, -1, device="cuda")
        s["lens"] = (torch.tensor(lens, device="cuda")[:, None] - back).clamp_min(0).reshape(-1).to(torch.int32)
        s["q"] = torch.randn((len(lens) * nq, case["heads"], LATENT + ROPE), generator=g, device="cuda").to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(LATENT + ROPE)
        if own:      # the workspace that a program keeps for its decode calls, and its output buffers
            from sparse_mla_decode_paged_gb300 import api
            s["ws"] = api.alloc_dense_workspace(api.dense_dims_of(s["q"], s["cache"], s["bt"]), s["q"].device)
        s["out"] = torch.empty((len(lens) * nq, case["heads"], LATENT), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((len(lens) * nq, case["heads"]), device="cuda")
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        n = case["tokens"]
        s["req"], s["pos"], s["bt"], pages = _paged_tokens(case, g)
        s["cache"] = _records(pages * PAGE, g).view(pages, PAGE, REC)
        # the key projection's output: latent and rope side by side in one row
        kv = torch.randn((n, LATENT + ROPE), generator=g, device="cuda")
        kv[:, :LATENT] *= torch.where(torch.rand(LATENT, generator=g, device="cuda") < 0.01, 8.0, 1.0)
        s["kv"] = kv.to(dt)
        s["w"] = (1 + 0.2 * torch.randn(LATENT, generator=g, device="cuda")).to(dt)
        s["table"] = _table(s["bt"].shape[1] * PAGE)
    elif case["op"] == "norm_rope":
        n = case["tokens"]
        s["x"] = torch.randn((n, case["heads"], case["dim"]), generator=g, device="cuda").to(dt)
        s["w"] = (1 + 0.2 * torch.randn(case["dim"], generator=g, device="cuda")).to(dt)
        s["table"] = _table(131072)
        s["pos"] = torch.randint(0, 131072, (n,), generator=g, device="cuda").to(torch.int32)
        s["out"] = torch.empty_like(s["x"])
    else:
        s["req"], s["pos"], s["bt"], pages = _paged_tokens(case, g)
        s["cache"] = _records(pages * PAGE, g).view(pages, PAGE, REC)
        s["out"] = torch.empty((case["tokens"], LATENT + ROPE), dtype=dt, device="cuda")
    return s


def _unpack(rec):
    """Records [.., 656] -> latent * scale [.., 512], rope [.., 64] in float32."""
    lat = rec[..., :512].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    lat = (lat * rec[..., 512:528].contiguous().view(torch.float32)[..., None]).flatten(-2)
    return lat, rec[..., 528:].contiguous().view(torch.bfloat16).float()


def _rotate(x, table, pos, interleaved):
    """Rotation of the last dim (64) of x [T, .., 64] by the angles of pos."""
    cs = table[pos.long()]
    cs = cs.view(cs.shape[0], *[1] * (x.dim() - 2), ROPE)
    c, s = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y = (a * c - b * s, a * s + b * c)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _cache_parts(cache):
    """The whole cache as the values it stands for: codes, scales and rope (views)."""
    return {"codes": cache[..., :512].view(torch.float8_e4m3fn), "scales": cache[..., 512:528].view(torch.float32),
            "rope": cache[..., 528:].view(torch.bfloat16)}


def _rows(s):
    page = s["bt"][s["req"].long(), s["pos"].long() // PAGE].long()
    return page * PAGE + s["pos"].long() % PAGE


def _plain_dense(s):
    R, nq, H = s["bt"].shape[0], s["case"]["queries"], s["case"]["heads"]
    rec = s["cache"][s["bt"].long().clamp_min(0)].flatten(1, 2)             # [R, positions, 656]
    lat, rope = _unpack(rec)
    k = torch.cat([lat, rope], -1)
    q = s["q"].float().view(R, nq * H, LATENT + ROPE)
    sc = (q @ k.transpose(1, 2)).view(R, nq, H, -1) * s["scale"]
    t = torch.arange(sc.shape[-1], device="cuda")
    sc = sc.masked_fill(t >= s["lens"].view(R, nq, 1, 1), -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    o = (p / z.clamp_min(1e-38)).view(R, nq * H, -1) @ lat
    return o.view(R * nq, H, LATENT).to(torch.bfloat16), (m + torch.log(z)).view(R * nq, H)


def run(s):
    case = s["case"]
    if own:
        from sparse_mla_decode_paged_gb300 import api
        if case["op"] == "dense":
            return api.sparse_mla_dense_decode(s["q"], s["cache"], s["bt"], s["lens"], s["scale"], out=s["out"],
                                               lse=s["lse"], workspace=s["ws"])
        if case["op"] == "append":
            api.sparse_mla_kv_norm_append(s["kv"][:, :LATENT], s["kv"][:, LATENT:], s["w"], 1e-6, s["table"], s["bt"],
                                          s["pos"], s["cache"], requests=s["req"], interleaved=case["interleaved"])
            return _cache_parts(s["cache"])
        if case["op"] == "norm_rope":
            return api.sparse_mla_norm_rope(s["x"], s["pos"], s["table"], weight=s["w"], eps=1e-6,
                                            rope_offset=case["rope_offset"], interleaved=case["interleaved"], out=s["out"])
        return api.sparse_mla_kv_read(s["cache"], s["bt"], s["pos"], requests=s["req"], out=s["out"])
    if case["op"] == "dense":
        return _plain_dense(s)
    if case["op"] == "append":
        x = s["kv"][:, :LATENT].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
        blk = x.view(-1, 4, 128)
        amax = blk.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        codes = (blk / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1, LATENT)
        rope = _rotate(s["kv"][:, LATENT:].float(), s["table"], s["pos"], case["interleaved"]).to(torch.bfloat16)
        s["cache"].view(-1, REC)[_rows(s)] = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8),
                                                        rope.view(torch.uint8)], -1)
        return _cache_parts(s["cache"])
    if case["op"] == "norm_rope":
        x = s["x"].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
        at = case["rope_offset"]
        y = _rotate(x[..., at:at + ROPE], s["table"], s["pos"], case["interleaved"])
        s["out"].copy_(torch.cat([x[..., :at], y, x[..., at + ROPE:]], -1))
        return s["out"]
    lat, rope = _unpack(s["cache"].view(-1, REC)[_rows(s)])
    s["out"].copy_(torch.cat([lat, rope], -1))
    return s["out"]


def work(case):
    if case["op"] == "dense":
        lens, rows = _lengths(case), case["requests"] * case["queries"] * case["heads"]
        tokens, pages = sum(lens), sum((n + PAGE - 1) // PAGE for n in lens)
        # query j of a request sees the context less the queries after it
        pairs = sum(max(0, n - j) for n in lens for j in range(case["queries"])) * case["heads"]
        return {"bytes": tokens * REC + pages * 4 + rows * (1152 + 1024 + 4), "flops": 2 * 1088 * pairs}
    size = 4 if case["dtype"] == "fp32" else 2
    n = case["tokens"]
    if case["op"] == "append":
        return {"bytes": n * (576 * size + 256 + 12 + REC) + 512 * size, "flops": n * 512 * 6}
    if case["op"] == "norm_rope":
        return {"bytes": n * (2 * case["heads"] * case["dim"] * size + 260) + case["dim"] * size,
                "flops": n * case["heads"] * case["dim"] * 5}
    return {"bytes": n * (REC + 576 * size + 12), "flops": n * 512}


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


def _exact_rotation(x, pos, interleaved):
    """x [T, .., 64] as complex numbers times exp(i angle); the angles as the float32 table gives them."""
    i = torch.arange(32, dtype=torch.float64, device="cuda")
    ang = pos.double()[:, None] * 10000.0 ** (-2 * i / 64)
    turn = torch.complex(ang.cos().float().double(), ang.sin().float().double())
    turn = turn.view(turn.shape[0], *[1] * (x.dim() - 2), 32)
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :32], x[..., 32:])
    z = z * turn
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def _exact_e4m3(x):
    """Nearest E4M3 value, ties to even: multiples of 2^(exponent - 3), of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 4).clamp_min(-9))
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    flat = s["cache"].view(-1, REC) if "cache" in s else None
    if case["op"] == "dense":
        H, nq = case["heads"], case["queries"]
        out = torch.zeros((case["requests"] * nq, H, LATENT), dtype=torch.float64, device="cuda")
        lse = torch.full((case["requests"] * nq, H), -math.inf, dtype=torch.float64, device="cuda")
        for r in range(case["requests"]):
            most = int(s["lens"][r * nq:(r + 1) * nq].max())
            parts = [([], []) for _ in range(nq)]
            for at in range(0, most, 1 << 17):
                t = torch.arange(at, min(most, at + (1 << 17)), device="cuda")
                lat, rope = _exact_records(flat[s["bt"][r, t // PAGE].long() * PAGE + t % PAGE])
                for j in range(nq):
                    n = int(s["lens"][r * nq + j]) - at
                    if n <= 0:
                        continue
                    q = s["q"][r * nq + j].double()
                    z = (q[:, :LATENT] @ lat[:n].T + q[:, LATENT:] @ rope[:n].T) * s["scale"]
                    parts[j][0].append(torch.logsumexp(z, -1))
                    parts[j][1].append(torch.softmax(z, -1) @ lat[:n])
            for j in range(nq):
                if parts[j][0]:
                    each = torch.stack(parts[j][0])
                    lse[r * nq + j] = torch.logsumexp(each, 0)
                    out[r * nq + j] = (torch.exp(each - lse[r * nq + j])[..., None] * torch.stack(parts[j][1])).sum(0)
        return out, lse
    if case["op"] == "append":
        x = s["kv"][:, :LATENT].double()
        x = s["w"].double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / LATENT + 1e-6)
        blk = x.view(-1, 4, 128)
        scale = blk.abs().amax(-1) / 448.0
        parts = {k: v.double() for k, v in _cache_parts(s["cache"]).items()}
        rows = _rows(s)
        parts["codes"].view(-1, LATENT)[rows] = _exact_e4m3(blk / scale[..., None]).view(-1, LATENT)
        parts["scales"].view(-1, 4)[rows] = scale
        parts["rope"].view(-1, ROPE)[rows] = _exact_rotation(s["kv"][:, LATENT:].double(), s["pos"], case["interleaved"])
        return parts
    if case["op"] == "norm_rope":
        x = s["x"].double()
        x = s["w"].double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6)
        at = case["rope_offset"]
        x[..., at:at + ROPE] = _exact_rotation(x[..., at:at + ROPE].clone(), s["pos"], case["interleaved"])
        return x
    return torch.cat(_exact_records(flat[_rows(s)]), -1)
