"""Measured cases of the 8-bit paged cache and of what writes, reads and fills it.

Four operators that a serving loop uses around its cache:

* ``norm``   - RMS norms of new tokens' query and key heads, rotary positions and
  the write into the 16-bit paged cache;
* ``write``  - the same into a cache held in 8 bits, with a power-of-two scale
  for each block of 16 tokens, kv head and array (K or V);
* ``attend`` - decode attention over the 8-bit cache;
* ``pages``  - blocks of a 16-bit pool parked in an 8-bit pool and brought back.

``run`` computes a case in plain torch operations (32 bits, rounded once) or,
where ``own`` is true, with the library's entry points.  Lengths follow from
the case alone, values and block placement from the seed.
"""
import math
import statistics

import torch

own = False

BS, D = 16, 128  # tokens of a cache block, elements of a head
EPS = 1e-6
TOP = {"e4m3": 448.0, "int8": 127.0}  # largest code


def listed():
    return [
        # One decode step of 64 running conversations on a model that norms its query and key heads: latency.
        dict(name="norm decode b64", op="norm", tokens=64, hq=32, hkv=8, dtype="bf16", rot=128, axes=1,
             interleaved=False, fused=True, norms="both", far=1 << 17),
        # A prompt of 8,192 tokens, rows sliced from one fused q|k|v projection.
        dict(name="norm prompt 8k", op="norm", tokens=8192, hq=32, hkv=8, dtype="bf16", rot=128, axes=1,
             interleaved=False, fused=True, norms="both", far=8192),
        # A video clip on a small model: fp16, partial rotary width, adjacent pairs, an odd number of tokens.
        dict(name="norm clip 1531", op="norm", tokens=1531, hq=12, hkv=2, dtype="fp16", rot=64, axes=3,
             interleaved=True, fused=False, norms="both", far=4096),
        # The decode step of 64 conversations with an 8-bit cache: one token each, in the middle of a block.
        dict(name="write decode b64", op="write", batch=64, new=1, held=600, sigma=0.8, pad=0, hq=32, hkv=8,
             dtype="bf16", rot=128, axes=1, interleaved=False, fused=True, norms="both"),
        # Chunks of 24 prompts, ragged, behind what earlier chunks left; the batch padded with rows that go nowhere.
        dict(name="write chunks 8k", op="write", batch=24, new=312, held=200, sigma=0.4, pad=37, hq=32, hkv=8,
             dtype="bf16", rot=128, axes=1, interleaved=False, fused=True, norms="both"),
        # Drafted tokens of 16 requests on a small model: five each, adjacent pairs, partial width.
        dict(name="write drafts b16", op="write", batch=16, new=5, held=300, sigma=0.3, pad=0, hq=12, hkv=2,
             dtype="fp16", rot=64, axes=1, interleaved=True, fused=False, norms="both"),
        # Four requests on a small model: latency, six query heads per kv head.
        dict(name="attend tiny b4", op="attend", batch=4, hq=12, hkv=2, dtype="fp16", out="fp16", kind="e4m3",
             median=160, sigma=1.2, empty=0),
        # Batch 64 with ragged chat lengths.
        dict(name="attend chat b64", op="attend", batch=64, hq=32, hkv=8, dtype="bf16", out="bf16", kind="e4m3",
             median=600, sigma=0.8, empty=0),
        # Multi-head layout (one query head per kv head), integer codes, 32-bit output, two slots of the batch unused.
        dict(name="attend mha b16", op="attend", batch=16, hq=40, hkv=40, dtype="fp16", out="fp32", kind="int8",
             median=2000, sigma=0.3, empty=2),
        # Four long documents, 8K to 32K tokens.
        dict(name="attend long b4", op="attend", batch=4, hq=32, hkv=8, dtype="bf16", out="bf16", kind="int8",
             median=18000, sigma=0.5, empty=0),
        # One paused request of a small model parked and brought back.
        dict(name="pages request", op="pages", blocks=121, hkv=2, dtype="fp16", kind="e4m3", partial=1),
        # 64 paused conversations of about 1,000 tokens.
        dict(name="pages batch", op="pages", blocks=4096, hkv=8, dtype="bf16", kind="int8", partial=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    hq, hkv = rng.choice([(32, 8), (12, 2), (40, 40), (16, 2), (8, 8), (24, 8), (10, 2)])
    dtype = rng.choice(["bf16", "fp16"])
    op = rng.choice(["norm", "write", "attend", "attend", "pages"])
    turn = dict(rot=rng.choice([128, 128, 64, 32, 96]), interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                norms=rng.choice(["both", "both", "both", "q", "k"]))
    most = 8000 if hq < 40 else 3000  # tokens of a call
    if op == "norm":
        return dict(op=op, tokens=log(1, most), hq=hq, hkv=hkv, dtype=dtype, axes=rng.choice([1, 2, 3, 4]),
                    far=log(64, 1 << 21), **turn)
    if op == "write":
        batch = log(1, 100)
        return dict(op=op, batch=batch, new=log(1, most // (2 * batch)), held=log(1, 50000 // (batch * hkv)),
                    sigma=round(rng.uniform(0.0, 0.8), 2), pad=rng.choice([0, 0, 1, 19]), hq=hq, hkv=hkv, dtype=dtype,
                    axes=rng.choice([1, 2, 3]), **turn)
    kind = rng.choice(["e4m3", "int8"])
    if op == "attend":
        batch = log(1, 100)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]), kind=kind,
                    median=log(1, 500000 // (batch * hkv)), sigma=round(rng.uniform(0.0, 0.9), 2),
                    empty=rng.choice([0, 0, 1]) if batch > 1 else 0)
    blocks = log(1, 32000 // hkv)
    return dict(op=op, blocks=blocks, hkv=hkv, dtype=dtype, kind=kind, partial=rng.randint(0, min(blocks, 40)))


def _type(name):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn,
            "int8": torch.int8}[name]


def _lengths(n, median, sigma):
    """n lengths at the quantiles of a lognormal distribution: ragged, and the same for every seed."""
    z = statistics.NormalDist()
    return [max(1, round(median * math.exp(sigma * z.inv_cdf((i + 0.5) / n)))) for i in range(n)]


def _attended(case):
    """Lengths of an attend case: the last of them are unused slots of the batch."""
    lens = _lengths(case["batch"], case["median"], case["sigma"])
    return lens[:case["batch"] - case["empty"]] + [0] * case["empty"]


def _up(n, m):
    return -(-n // m)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _shuffled(values, g):
    t = _ints(values)
    return t[torch.randperm(len(values), generator=g, device="cuda")]


def _tables(lens, g):
    """Block tables [B][W] (-1 past each sequence's end) at random places of a pool, and the pool's size."""
    nb = (lens + BS - 1) // BS
    need, width = int(nb.sum()), max(1, int(nb.max()))
    n = int(need * 1.25) + 1
    perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    inside = torch.arange(width, device="cuda")[None, :] < nb[:, None]
    tables = torch.full((lens.numel(), width), -1, dtype=torch.int32, device="cuda")
    tables[inside] = perm[:need]
    return tables, n


def _exponent(amax, kind):
    """Biased exponent of the smallest power of two 2^x >= 2^-126 with amax <= TOP * 2^x; 255 (NaN) if amax is not finite."""
    m, e = torch.frexp(amax)
    tm, te = math.frexp(TOP[kind])
    x = (e - te + (m > tm).to(e.dtype)).clamp(min=-126)
    x = torch.where(amax > 0, x, torch.full_like(x, -126)) + 127
    return torch.where(torch.isfinite(amax), x, torch.full_like(x, 255)).to(torch.uint8)


def _power(e):
    """2^(e - 127) in 64 bits, NaN for 255."""
    p = torch.ldexp(torch.ones((), dtype=torch.float64, device=e.device), e.int() - 127)
    return torch.where(e == 255, torch.full_like(p, torch.nan), p)


def _code(x, kind):
    """Codes nearest to x (even ones for ties)."""
    if kind == "e4m3":
        return x.float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.round(x).clamp(-127.0, 127.0).to(torch.int8)


def _pick(codes, at):
    """codes[at] for 8-bit floats and integers."""
    return codes.view(torch.uint8)[at].view(codes.dtype)


def _cache8(s, g, n_blocks, hkv, kind):
    """An 8-bit cache [n_blocks][hkv][16][128] of rows whose size varies from block to block and head to head, and its
    exponents [n_blocks][hkv]; with the library, its pool's own."""
    if own:
        import paged_kv_cache_227_gb300 as pa
        s["pool8"] = pa.Pool8(n_blocks, hkv, _type(kind))
    for x in ("k", "v"):
        codes = torch.empty(n_blocks, hkv, BS, D, dtype=_type(kind), device="cuda")
        exps = torch.empty(n_blocks, hkv, dtype=torch.uint8, device="cuda")
        for b in range(0, n_blocks, 4096):
            rows = _randn(g, min(4096, n_blocks - b), hkv, BS, D)
            rows *= torch.exp(0.4 * _randn(g, rows.shape[0], hkv, 1, 1))
            e = _exponent(rows.abs().amax((2, 3)), kind)
            codes[b:b + 4096] = _code(rows / _power(e).float()[:, :, None, None], kind)
            exps[b:b + 4096] = e
        if own:
            mine, scale = (s["pool8"].k, s["pool8"].k_scale) if x == "k" else (s["pool8"].v, s["pool8"].v_scale)
            mine.copy_(codes)
            scale.view(torch.uint8).copy_(exps)
            codes, exps = mine, scale.view(torch.uint8)
        s[x], s["e" + x] = codes, exps


def _axis_of_pair(rot, axes):
    """Frequency pairs dealt out to the axes in runs, the first axis (time) taking what is left over."""
    share = (rot // 2) // axes
    rest = rot // 2 - share * (axes - 1)
    return [0] * rest + [a for a in range(1, axes) for _ in range(share)]


def _new_tokens(s, c, g, n, positions):
    """The rows of n new tokens and what norms and turns them."""
    hq, hkv, rot, dtype = c["hq"], c["hkv"], c["rot"], _type(c["dtype"])
    if c["fused"]:  # rows of one projection: q | k | v
        qkv = _randn(g, n, (hq + 2 * hkv) * D).mul_(1.5).to(dtype).view(n, hq + 2 * hkv, D)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"], s["k_new"], s["v_new"] = (_randn(g, n, h, D).mul_(1.5).to(dtype) for h in (hq, hkv, hkv))
    for x in ("q", "k"):
        s["w" + x] = (1.0 + 0.25 * _randn(g, D)).to(dtype) if c["norms"] in ("both", x) else None
    s["positions"] = positions
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float()
    s["axis_of_pair"] = _axis_of_pair(rot, c["axes"])
    s["axis_dev"] = _ints(s["axis_of_pair"], torch.int64)
    s["q_out"] = torch.zeros(n, hq, D, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    c, s = case, {"case": case, "scale": 1.0 / math.sqrt(D)}
    hkv = c["hkv"]
    if c["op"] == "norm":
        n = c["tokens"]
        n_blocks = _up(n, BS) + 4
        dtype = _type(c["dtype"])
        if own:
            import paged_kv_cache_227_gb300 as pa
            s["pool"] = pa.Pool(n_blocks, hkv, dtype)
        for x in ("k", "v"):
            rows = _randn(g, n_blocks, hkv, BS, D).to(dtype)
            s[x] = getattr(s["pool"], x).copy_(rows) if own else rows
        _new_tokens(s, c, g, n, torch.randint(0, c["far"], (c["axes"], n), generator=g, device="cuda", dtype=torch.int32))
        s["slots"] = torch.randperm(n_blocks * BS, generator=g, device="cuda")[:n].to(torch.int64)
        return s
    if c["op"] == "write":
        # (the shortest chunks behind the longest contexts, in an order of the seed's)
        order = torch.randperm(c["batch"], generator=g, device="cuda")
        new = _ints(_lengths(c["batch"], c["new"], c["sigma"]))[order]
        held = _ints(_lengths(c["batch"], c["held"], c["sigma"])[::-1])[order]
        tables, n_blocks = _tables(held + new, g)
        _cache8(s, g, n_blocks, hkv, "e4m3")
        n, pad = int(new.sum()), c["pad"]
        seq = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), new.long())
        start = torch.cumsum(new, 0) - new
        pos = torch.arange(n, device="cuda") - start[seq] + held[seq]
        slots = tables[seq, pos // BS].long() * BS + pos % BS
        s["slots"] = torch.cat([slots, torch.full((pad,), -1, dtype=torch.int64, device="cuda")])
        at = torch.cat([pos, torch.zeros(pad, dtype=torch.int64, device="cuda")]).int()
        _new_tokens(s, c, g, n + pad, torch.stack([at // (1 + a) for a in range(c["axes"])]).contiguous())
        return s
    if c["op"] == "attend":
        lens = _shuffled(_attended(c), g)
        s["tables"], n_blocks = _tables(lens, g)
        s["lens"] = lens
        _cache8(s, g, n_blocks, hkv, c["kind"])
        s["q"] = _randn(g, c["batch"], c["hq"], D).to(_type(c["dtype"]))
        s["out"] = torch.zeros(c["batch"], c["hq"], D, dtype=_type(c["out"]), device="cuda")
        if own:  # the workspace that a serving loop keeps
            import paged_kv_cache_227_gb300 as pa
            s["workspace"] = pa.decode8_workspace_for(s["pool8"], s["q"], s["tables"])
        return s
    n, dtype = c["blocks"], _type(c["dtype"])
    n_blocks, n8 = 2 * n + 3, n + 2  # the blocks of the requests, those they come back to, and spare ones
    if own:
        import paged_kv_cache_227_gb300 as pa
        s["pool"], s["pool8"] = pa.Pool(n_blocks, hkv, dtype), pa.Pool8(n8, hkv, _type(c["kind"]))
    for x in ("k", "v"):
        rows = (_randn(g, n_blocks, hkv, BS, D) * torch.exp(0.4 * _randn(g, n_blocks, hkv, 1, 1))).to(dtype)
        s[x] = getattr(s["pool"], x).copy_(rows) if own else rows
        if not own:
            s["c" + x] = torch.zeros(n8, hkv, BS, D, dtype=_type(c["kind"]), device="cuda")
            s["e" + x] = torch.zeros(n8, hkv, dtype=torch.uint8, device="cuda")
    perm = torch.randperm(n_blocks, generator=g, device="cuda").int()
    s["src"], s["back"] = perm[:n].contiguous(), perm[n:2 * n].contiguous()
    s["parked"] = torch.randperm(n8, generator=g, device="cuda")[:n].int()
    s["rows"] = torch.full((n,), BS, dtype=torch.int32, device="cuda")
    part = c["partial"]
    s["rows"][n - part:] = torch.randint(1, BS, (part,), generator=g, device="cuda", dtype=torch.int32)
    return s


def run(s):
    return {"norm": _norm, "write": _write, "attend": _attend, "pages": _pages}[s["case"]["op"]](s)


def _rotate(x, cos, sin, rot, interleaved):
    """x [n][h][128] in fp32, cos and sin [n][rot/2]."""
    c, z = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * z, b * c + a * z
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * z, b * c + a * z
    return y


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _turned(s):
    """The normed and turned query and key rows, fp32."""
    c = s["case"]
    angle = s["positions"].double()[s["axis_dev"]].t() * s["inv_freq"].double()  # [n][rot/2]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return (_rotate(_normed(s[x], s[w]), cos, sin, c["rot"], c["interleaved"]) for x, w in (("q", "wq"), ("k_new", "wk")))


def _norm(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_norm_rope_append(s["pool"], s["q"], s["k_new"], s["v_new"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                               s["axis_of_pair"], s["slots"], s["q_out"], eps=EPS, interleaved=c["interleaved"])
    else:
        q, k = _turned(s)
        s["q_out"] = q.to(s["q"].dtype)
        blk, off = s["slots"] // BS, s["slots"] % BS
        s["k"][blk, :, off] = k.to(s["k"].dtype)
        s["v"][blk, :, off] = s["v_new"]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _write(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_norm_rope_append8(s["pool8"], s["q"], s["k_new"], s["v_new"], s["wq"], s["wk"], s["positions"],
                                s["inv_freq"], s["axis_of_pair"], s["slots"], s["q_out"], eps=EPS,
                                interleaved=c["interleaved"])
    else:
        q, k = _turned(s)
        s["q_out"] = q.to(s["q"].dtype)
        real = s["slots"] >= 0
        blk, off = s["slots"][real] // BS, s["slots"][real] % BS
        n = s["k"].shape[0]
        touched = torch.zeros(n, dtype=torch.bool, device="cuda").index_fill_(0, blk, True)
        fresh = torch.zeros(n, dtype=torch.bool, device="cuda").index_fill_(0, blk[off == 0], True)
        for x, rows in (("k", k[real]), ("v", s["v_new"][real].float())):
            amax = torch.zeros(n, c["hkv"], device="cuda")
            amax.scatter_reduce_(0, blk[:, None].expand(-1, c["hkv"]), rows.abs().amax(2), "amax")
            need, was = _exponent(amax, "e4m3"), s["e" + x]
            e = torch.where(fresh[:, None], need, torch.maximum(need, was))
            e = torch.where(touched[:, None], e, was)
            # what the block holds moves to the new scale
            less = torch.where(fresh[:, None], torch.ones_like(_power(e)), _power(was) / _power(e)).float()
            codes = _code(s[x].float() * less[:, :, None, None], "e4m3")
            mine = _code(rows / _power(e).float()[blk][:, :, None], "e4m3")
            codes.view(torch.uint8)[blk, :, off] = mine.view(torch.uint8)
            s[x], s["e" + x] = codes, e
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["ek"].view(torch.float8_e8m0fnu),
            "v_scale": s["ev"].view(torch.float8_e8m0fnu)}


def _gathered(codes, exps, tables):
    """The values of each table row in order, fp32: [rows][hkv][W*16][128]."""
    at = tables.clamp(min=0).long()
    x = _pick(codes, at).float() * _power(exps[at]).float()[..., None, None]  # [rows][W][hkv][16][128]
    r, w, h = x.shape[:3]
    return x.transpose(1, 2).reshape(r, h, w * BS, D)


def _attend(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_decode8(s["pool8"], s["q"], s["tables"], s["lens"], s["scale"], s["out"], workspace=s["workspace"])
        return s["out"]
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    k, v = _gathered(s["k"], s["ek"], s["tables"]), _gathered(s["v"], s["ev"], s["tables"])
    inside = (torch.arange(k.shape[2], device="cuda")[None, :] < s["lens"][:, None])[:, None, None, :]
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    sc = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    sc = torch.where(inside, sc, torch.full_like(sc[:1, :1, :1, :1], -torch.inf))
    m = sc.amax(3, keepdim=True)
    p = torch.exp(sc - torch.where(m == -torch.inf, torch.zeros_like(m), m))
    v = torch.where(inside.transpose(2, 3), v, torch.zeros_like(v[:1, :1, :1, :1]))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.view(B, hq, D).to(s["out"].dtype)


def _pages(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_quantize_blocks(s["pool"], s["src"], s["pool8"], s["parked"], rows=s["rows"])
        pa.pa_dequantize_blocks(s["pool8"], s["parked"], s["pool"], s["back"])
    else:
        held = (torch.arange(BS, device="cuda")[None, :] < s["rows"][:, None])[:, None, :, None]
        src, parked, back = (s[x].long() for x in ("src", "parked", "back"))
        top = torch.finfo(s["k"].dtype).max
        for x in ("k", "v"):
            rows = s[x][src].float()
            e = _exponent(torch.where(held, rows.abs(), torch.zeros_like(rows)).amax((2, 3)), c["kind"])
            scale = _power(e).float()[:, :, None, None]
            was = _pick(s["c" + x], parked)
            codes = torch.where(held, _code(rows / scale, c["kind"]).view(torch.uint8), was.view(torch.uint8))
            s["c" + x].view(torch.uint8)[parked] = codes
            s["e" + x][parked] = e
            s[x][back] = (codes.view(was.dtype).float() * scale).clamp(-top, top).to(s[x].dtype)
    return {"k": s["k"], "v": s["v"]}


def _rows_of(case):
    """New tokens of a norm or write case, those that go nowhere among them, and those that reach the cache."""
    if case["op"] == "norm":
        return case["tokens"], case["tokens"]
    n = sum(_lengths(case["batch"], case["new"], case["sigma"]))
    return n + case["pad"], n


def work(case):
    hkv, e = case["hkv"], 2
    if case["op"] in ("norm", "write"):
        n, kept = _rows_of(case)
        hq, to = case["hq"], 2 if case["op"] == "norm" else 1
        return {"bytes": n * (2 * hq * D * e + 8 + 4 * case["axes"]) + 2 * kept * hkv * D * (e + to),
                "flops": n * (hq + hkv) * (4 * D + 3 * case["rot"])}
    if case["op"] == "attend":
        lens, hq = _attended(case), case["hq"]
        out = 4 if case["out"] == "fp32" else 2
        tiles = sum(_up(n, BS) for n in lens)
        return {"bytes": sum(lens) * hkv * 2 * D + tiles * (2 * hkv + 4) + case["batch"] * hq * D * (e + out),
                "flops": 4 * D * hq * sum(lens)}
    rows = case["blocks"] * BS - case["partial"] * BS // 2
    return {"bytes": 2 * hkv * D * (rows * (e + 1) + case["blocks"] * BS * (1 + e)), "flops": 2 * hkv * D * 3 * rows}


def _turn64(x, w, pos, s, case):
    """Norm and rotation of rows [n][h][128] in 64 bits, the rotation as a product of complex numbers."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(2, keepdim=True) / D + EPS) * w.double()
    rot = case["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos * s["inv_freq"].double()[None, :])
    first = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if case["interleaved"] else rot // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _near(x, kind):
    """The nearest values that codes stand for, ties to the even one, from their spacing at each x (64 bits)."""
    if kind == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _least(amax, kind):
    """The least power of two of at least 2^-126 that holds amax (a number): counted up from below."""
    x = max(-126, math.floor(math.log2(amax / TOP[kind])) - 1) if amax > 0 else -126
    while TOP[kind] * 2.0 ** x < amax:
        x += 1
    return 2.0 ** x


def exact(case, seed):
    """The operators' definitions in 64 bits, block by block or sequence by sequence."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    hkv = case["hkv"]
    if case["op"] in ("norm", "write"):
        pos = torch.stack([s["positions"][a] for a in s["axis_of_pair"]], 1).double()
        q, k = _turn64(s["q"], s["wq"], pos, s, case), _turn64(s["k_new"], s["wk"], pos, s, case)
        new = {"k": k, "v": s["v_new"].double()}
        slots = s["slots"].tolist()
        if case["op"] == "norm":
            got = {"q": q}
            for x in ("k", "v"):
                rows = s[x].double().transpose(1, 2).reshape(-1, hkv, D).clone()
                rows[s["slots"]] = new[x]
                got[x] = rows.view(-1, BS, hkv, D).transpose(1, 2)
            return got
        runs = {}
        for r, slot in enumerate(slots):
            if slot >= 0:
                runs.setdefault(slot // BS, []).append((slot % BS, r))
        if len(runs) * hkv > 6000:
            return None
        got = {"q": q}
        for x in ("k", "v"):
            codes, scale = s[x].double(), _power(s["e" + x])
            for b, run_ in runs.items():
                off, r = (torch.tensor(t, device="cuda") for t in zip(*run_))
                tops = new[x][r].abs().amax((0, 2)).tolist()
                for h, top in enumerate(tops):
                    p = _least(top, "e4m3")
                    if run_[0][0]:
                        p = max(p, float(scale[b, h]))
                        codes[b, h] = _near(codes[b, h] * (float(scale[b, h]) / p), "e4m3")
                    scale[b, h] = p
                    codes[b, h, off] = _near(new[x][r, h] / p, "e4m3")
            got[x], got[x + "_scale"] = codes, scale
        return got
    if case["op"] == "attend":
        hq, outs = case["hq"], []
        for i, n in enumerate(s["lens"].tolist()):
            if n == 0:
                outs.append(torch.zeros(hq, D, dtype=torch.float64, device="cuda"))
                continue
            at = s["tables"][i, :_up(n, BS)].long()
            k, v = ((_pick(s[x], at).double() * _power(s["e" + x][at])[..., None, None]).permute(1, 0, 2, 3)
                    .reshape(hkv, -1, D)[:, :n] for x in ("k", "v"))
            q = s["q"][i].double().view(hkv, hq // hkv, D)
            p = torch.softmax(torch.einsum("hgd,htd->hgt", q, k) * s["scale"], dim=2)
            outs.append(torch.einsum("hgt,htd->hgd", p, v).reshape(hq, D))
        return torch.stack(outs)
    if case["blocks"] * hkv > 4000:
        return None
    got = {}
    for x in ("k", "v"):
        pool = s[x].double()
        for a, n, b in zip(s["src"].tolist(), s["rows"].tolist(), s["back"].tolist()):
            tile = s[x][a, :, :n].double()
            p = torch.tensor([_least(t, case["kind"]) for t in tile.abs().amax((1, 2)).tolist()], dtype=torch.float64,
                             device="cuda")[:, None, None]
            pool[b, :, :n] = _near(tile / p, case["kind"]) * p
            pool[b, :, n:] = 0
        got[x] = pool
    return got
