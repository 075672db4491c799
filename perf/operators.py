"""Measured cases of the cache operators around paged decode attention.

Four operators that a serving loop uses next to the decode step:

* ``rope``    - rotary positions with several axes on new tokens' queries and
  keys, with the write of the rotated keys and the values into the paged cache;
* ``shared``  - decode attention of a batch whose sequences share long
  prefixes, each prefix attended once for all of its members;
* ``weights`` - decode attention that also accumulates, per kv head and cached
  token, the attention weight the token received;
* ``evict``   - eviction from the cache by that accumulated weight: the
  heaviest tokens of each kv head stay, in order, and the cache closes up.

``run`` computes a case in plain torch operations (32 bits, rounded once) or,
where ``own`` is true, with the library's entry points.  Lengths follow from
the case alone, values and block placement from the seed.
"""
import math
import statistics

import torch

own = False

BS, D = 16, 128  # tokens of a cache block, elements of a head


def listed():
    return [
        # One decode step of 64 running conversations, text and video mixed, far into their contexts: latency.
        dict(name="rope decode b64", op="rope", tokens=64, hq=32, hkv=8, dtype="bf16", rot=128, axes=3,
             interleaved=False, fused=True, far=1 << 20),
        # A prompt of images and text, 8,192 tokens, rows sliced from one fused q|k|v projection.
        dict(name="rope prompt 8k", op="rope", tokens=8192, hq=32, hkv=8, dtype="bf16", rot=128, axes=3,
             interleaved=False, fused=True, far=8192),
        # A video clip on a small model: fp16, partial rotary width, adjacent pairs, an odd number of tokens.
        dict(name="rope clip 1531", op="rope", tokens=1531, hq=12, hkv=2, dtype="fp16", rot=64, axes=4,
             interleaved=True, fused=False, far=4096),
        # Four requests behind a short system prompt on a small model: latency.
        dict(name="shared tiny b4", op="shared", batch=4, hq=12, hkv=2, dtype="fp16", out="fp16", groups=1,
             prefix=256, suffix=17, sigma=0.9),
        # 64 chats behind one 2,048-token system prompt, ragged own turns.
        dict(name="shared chat b64", op="shared", batch=64, hq=32, hkv=8, dtype="bf16", out="bf16", groups=1,
             prefix=2048, suffix=200, sigma=0.8),
        # Multi-head layout (one query head per kv head), two prompts, 16 sequences, 32-bit output.
        dict(name="shared mha b16", op="shared", batch=16, hq=40, hkv=40, dtype="fp16", out="fp32", groups=2,
             prefix=2064, suffix=300, sigma=0.5),
        # 256 samples of one 16K-token document.
        dict(name="shared document b256", op="shared", batch=256, hq=32, hkv=8, dtype="bf16", out="bf16", groups=1,
             prefix=16384, suffix=150, sigma=0.6),
        # Batch 64 with ragged chat lengths, weights gathered every step.
        dict(name="weights chat b64", op="weights", batch=64, hq=32, hkv=8, dtype="bf16", out="bf16", median=600,
             sigma=0.8, decay=1.0),
        # Four long documents, 8K to 32K tokens, decaying weights, 32-bit output.
        dict(name="weights long b4", op="weights", batch=4, hq=32, hkv=8, dtype="bf16", out="fp32", median=18000,
             sigma=0.5, decay=0.96875),
        # A small model's four requests: latency, six query heads per kv head.
        dict(name="weights tiny b4", op="weights", batch=4, hq=12, hkv=2, dtype="fp16", out="fp16", median=160,
             sigma=1.2, decay=1.0),
        # 64 sequences of about 4K tokens cut back to 1,024.
        dict(name="evict batch b64", op="evict", batch=64, hkv=8, dtype="bf16", median=4000, sigma=0.2, keep=1024,
             sink=4, recent=128),
        # Four long documents cut back to 4,001 tokens.
        dict(name="evict long b4", op="evict", batch=4, hkv=8, dtype="fp16", median=18000, sigma=0.5, keep=4001,
             sink=16, recent=512),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    hq, hkv = rng.choice([(32, 8), (12, 2), (40, 40), (16, 2), (8, 8), (24, 8), (10, 2)])
    dtype = rng.choice(["bf16", "fp16"])
    out = rng.choice([dtype, dtype, "fp32"])
    op = rng.choice(["rope", "shared", "weights", "evict"])
    if op == "rope":
        return dict(op=op, tokens=log(1, 7000 if hq < 40 else 2900), hq=hq, hkv=hkv, dtype=dtype,
                    rot=rng.choice([128, 128, 64, 32, 96]), axes=rng.choice([1, 2, 3, 4]),
                    interleaved=rng.random() < 0.4, fused=rng.random() < 0.5, far=log(64, 1 << 21))
    if op == "shared":
        batch = log(2, 200)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, out=out, groups=rng.randint(1, min(3, batch)),
                    prefix=BS * log(1, min(1024, 4096 // hkv, 200000 // batch)),
                    suffix=log(1, min(400, 150000 // (batch * hkv))), sigma=round(rng.uniform(0.1, 0.9), 2))
    if op == "weights":
        batch = log(1, 100)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, dtype=dtype, out=out, median=log(1, 320000 // (batch * hkv)),
                    sigma=round(rng.uniform(0.0, 0.9), 2), decay=rng.choice([1.0, 0.5, 0.9375]))
    batch, hkv = log(1, 48), min(hkv, 8)
    median = log(2, 90000 // batch)
    return dict(op=op, batch=batch, hkv=hkv, dtype=dtype, median=median, sigma=round(rng.uniform(0.0, 0.5), 2),
                keep=max(1, int(median * rng.uniform(0.1, 0.8))), sink=rng.choice([0, 1, 4, 16]),
                recent=rng.choice([0, 1, 31, 256]))


def _type(name):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _lengths(n, median, sigma):
    """n lengths at the quantiles of a lognormal distribution: ragged, and the same for every seed."""
    z = statistics.NormalDist()
    return [max(1, round(median * math.exp(sigma * z.inv_cdf((i + 0.5) / n)))) for i in range(n)]


def _up(n, m):
    return -(-n // m)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, dtype, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _shuffled(values, g):
    t = _ints(values)
    return t[torch.randperm(len(values), generator=g, device="cuda")]


def _tables(lens, g, spare=1.25):
    """Block tables [B][W] (-1 past each sequence's end) at random places of a pool, and the blocks left free."""
    nb = (lens + BS - 1) // BS
    need, width = int(nb.sum()), int(nb.max())
    n = int(need * spare) + 1
    perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    inside = torch.arange(width, device="cuda")[None, :] < nb[:, None]
    tables = torch.full((lens.numel(), width), -1, dtype=torch.int32, device="cuda")
    tables[inside] = perm[:need]
    return tables, perm[need:], n


def _cache(s, g, n_blocks, hkv, dtype):
    """The K and V arrays [n_blocks][hkv][16][128]; with the library, its pool's own."""
    if own:
        import paged_kv_cache_227_gb300 as pa
        s["pool"] = pa.Pool(n_blocks, hkv, dtype)
        s["k"], s["v"] = s["pool"].k, s["pool"].v
        s["k"].copy_(_rand(g, dtype, n_blocks, hkv, BS, D))
        s["v"].copy_(_rand(g, dtype, n_blocks, hkv, BS, D))
    else:
        s["k"] = _rand(g, dtype, n_blocks, hkv, BS, D)
        s["v"] = _rand(g, dtype, n_blocks, hkv, BS, D)


def _axis_of_pair(rot, axes):
    """Frequency pairs dealt out to the axes in runs, the first axis (time) taking what is left over."""
    share = (rot // 2) // axes
    rest = rot // 2 - share * (axes - 1)
    return [0] * rest + [a for a in range(1, axes) for _ in range(share)]


def prepare(case, seed):
    g = _gen(seed)
    dtype = _type(case["dtype"])
    hkv = case["hkv"]
    s = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "rope":
        n, hq, rot = case["tokens"], case["hq"], case["rot"]
        n_blocks = _up(n, BS) + 4
        _cache(s, g, n_blocks, hkv, dtype)
        if case["fused"]:  # rows of one projection: q | k | v
            qkv = _rand(g, dtype, n, (hq + 2 * hkv) * D).view(n, hq + 2 * hkv, D)
            s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = _rand(g, dtype, n, hq, D), _rand(g, dtype, n, hkv, D), _rand(g, dtype, n, hkv, D)
        s["positions"] = torch.randint(0, case["far"], (case["axes"], n), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float()
        s["axis_of_pair"] = _axis_of_pair(rot, case["axes"])
        s["axis_dev"] = _ints(s["axis_of_pair"], torch.int64)
        slots = torch.randperm(n_blocks * BS, generator=g, device="cuda")[:n]
        s["slots"] = slots.to(torch.int64)
        s["q_out"] = torch.zeros(n, hq, D, dtype=dtype, device="cuda")
        return s
    if case["op"] == "shared":
        B, G = case["batch"], case["groups"]
        suffix = _shuffled(_lengths(B, case["suffix"], case["sigma"]), g)
        group_of = torch.arange(B, device="cuda") % G
        pre = _ints([max(1, case["prefix"] // BS // (1 + k)) for k in range(G)])
        lens = (pre[group_of] * BS + suffix).to(torch.int32)
        tables, _, n_blocks = _tables(lens, g)
        first = tables[:G][group_of]  # group k's first member is sequence k
        width = tables.shape[1]
        shared = torch.arange(width, device="cuda")[None, :] < pre[group_of][:, None]
        s["tables"] = torch.where(shared, first, tables).contiguous()
        _cache(s, g, n_blocks, hkv, dtype)
        members = torch.argsort(group_of, stable=True).to(torch.int32)
        count = torch.bincount(group_of, minlength=G)
        s["group_start"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)]).to(torch.int32)
        s["members"], s["prefix_blocks"], s["lens"] = members, pre, lens
        # plans of the plain form: members by place in their group, padded
        most = int(count.max())
        place = torch.arange(most, device="cuda")[None, :]
        s["member_at"] = members.long()[(s["group_start"][:-1, None].long() + place).clamp(max=B - 1)]
        s["member_in"] = place < count[:, None]
        s["pre_max"] = int(pre.max())
        s["suffix_max"] = int(suffix.max())
        s["group_of"] = group_of
        hq = case["hq"]
    elif case["op"] == "weights":
        B, hq = case["batch"], case["hq"]
        lens = _shuffled(_lengths(B, case["median"], case["sigma"]), g)
        s["tables"], _, n_blocks = _tables(lens, g)
        s["lens"] = lens
        _cache(s, g, n_blocks, hkv, dtype)
        span = s["tables"].shape[1] * BS
        s["weights"] = torch.rand(B, hkv, span, generator=g, device="cuda") * (4.0 / case["median"])
    else:
        B = case["batch"]
        lens = _shuffled(_lengths(B, case["median"], case["sigma"]), g)
        keep = min(case["keep"], int(lens.max()))
        # room for the sequences and for the closed-up copies
        s["tables"], free, n_blocks = _tables(lens, g, spare=1.0 + 1.0 * B * (_up(keep, BS) + 1) / int(((lens + BS - 1) // BS).sum()))
        s["lens"] = lens
        s["keep"] = _ints([keep] * B)
        wd = _up(keep, BS)
        s["dst"] = free[:B * wd].view(B, wd).contiguous()
        _cache(s, g, n_blocks, hkv, dtype)
        span = s["tables"].shape[1] * BS
        # heavy-tailed sums of attention weights on a grid coarse enough that some of them are equal
        w = torch.exp(1.5 * torch.randn(B, hkv, span, generator=g, device="cuda"))
        s["weights"] = torch.round(w * 1024.0) / 1024.0
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["kept"] = torch.full((B, hkv, span), -1, dtype=torch.int32, device="cuda")
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    s["q"] = _rand(g, dtype, B, hq, D)
    s["out"] = torch.zeros(B, hq, D, dtype=_type(case["out"]), device="cuda")
    if own:  # the workspace that a serving loop keeps
        import paged_kv_cache_227_gb300 as pa
        if case["op"] == "shared":
            s["workspace"] = pa.shared_workspace_for(s["pool"], s["q"], s["tables"], s["prefix_blocks"])
        else:
            s["workspace"] = pa.weights_workspace_for(s["pool"], s["q"], s["tables"])
    return s


def run(s):
    return {"rope": _rope, "shared": _shared, "weights": _weights, "evict": _evict}[s["case"]["op"]](s)


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


def _rope(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_rope_append(s["pool"], s["q"], s["k_new"], s["v_new"], s["positions"], s["inv_freq"], s["axis_of_pair"],
                          s["slots"], s["q_out"], interleaved=c["interleaved"])
    else:
        angle = s["positions"].double()[s["axis_dev"]].t() * s["inv_freq"].double()  # [n][rot/2]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        s["q_out"] = _rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
        k = _rotate(s["k_new"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["k"].dtype)
        blk, off = s["slots"] // BS, s["slots"] % BS
        s["k"][blk, :, off] = k
        s["v"][blk, :, off] = s["v_new"]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _gathered(pool, tables):
    """The cache of each table row in order, fp32: [rows][hkv][W*16][128]."""
    x = pool[tables.clamp(min=0).long()].float()          # [rows][W][hkv][16][128]
    r, w, h = x.shape[:3]
    return x.transpose(1, 2).reshape(r, h, w * BS, D)


def _attend(q, k, v, inside, scale):
    """q [r][h][x][128], k and v [r][h][t][128], inside [r][t]: unnormalised sums with their maxima and weights."""
    sc = torch.matmul(q, k.transpose(2, 3)) * scale
    sc = torch.where(inside[:, None, None, :], sc, torch.full_like(sc[:1, :1, :1, :1], -torch.inf))
    m = sc.amax(3, keepdim=True)
    p = torch.exp(sc - torch.where(m == -torch.inf, torch.zeros_like(m), m))
    v = torch.where(inside[:, None, :, None], v, torch.zeros_like(v[:1, :1, :1, :1]))
    return torch.matmul(p, v), m, p.sum(3, keepdim=True), p


def _shared(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_decode_shared(s["pool"], s["q"], s["tables"], s["lens"], s["scale"], s["out"], s["group_start"],
                            s["members"], s["prefix_blocks"], workspace=s["workspace"])
        return s["out"]
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    G, ng = hq // hkv, c["groups"]
    q = s["q"].float().view(B, hkv, G, D)
    # each prefix once: all members' query heads of a kv head against it
    first = s["member_at"][:, 0]
    k, v = (_gathered(s[x], s["tables"][first, :s["pre_max"]]) for x in ("k", "v"))
    inside = torch.arange(s["pre_max"] * BS, device="cuda")[None, :] < s["prefix_blocks"][:, None] * BS
    most = s["member_at"].shape[1]
    qg = q[s["member_at"]].transpose(1, 2).reshape(ng, hkv, most * G, D)
    o1, m1, l1, _ = _attend(qg, k, v, inside, s["scale"])

    def back(x):  # [ng][hkv][most*G][..] -> [B][hkv][G][..]
        x = x.view(ng, hkv, most, G, -1).transpose(1, 2)
        y = torch.empty(B, hkv, G, x.shape[-1], device="cuda")
        y[s["member_at"][s["member_in"]]] = x[s["member_in"]]
        return y

    o1, m1, l1 = back(o1), back(m1), back(l1)
    # the sequences' own tokens
    pre = s["prefix_blocks"][s["group_of"]].long()
    at = pre[:, None] + torch.arange(_up(s["suffix_max"], BS), device="cuda")[None, :]
    own_tables = s["tables"].gather(1, at.clamp(max=s["tables"].shape[1] - 1))
    k, v = _gathered(s["k"], own_tables), _gathered(s["v"], own_tables)
    inside = torch.arange(k.shape[2], device="cuda")[None, :] < (s["lens"] - pre * BS)[:, None]
    o2, m2, l2, _ = _attend(q, k, v, inside, s["scale"])
    m = torch.maximum(m1, m2)
    a, b = torch.exp(m1 - m), torch.exp(m2 - m)
    return ((a * o1 + b * o2) / (a * l1 + b * l2)).view(B, hq, D).to(s["out"].dtype)


def _weights(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_decode_weights(s["pool"], s["q"], s["tables"], s["lens"], s["scale"], s["out"], s["weights"],
                             decay=c["decay"], workspace=s["workspace"])
        return {"out": s["out"], "weights": s["weights"]}
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    k, v = _gathered(s["k"], s["tables"]), _gathered(s["v"], s["tables"])
    inside = torch.arange(k.shape[2], device="cuda")[None, :] < s["lens"][:, None]
    o, _, l, p = _attend(s["q"].float().view(B, hkv, hq // hkv, D), k, v, inside, s["scale"])
    grown = s["weights"] * c["decay"] + (p / l).sum(2)
    s["weights"] = torch.where(inside[:, None, :], grown, s["weights"])
    return {"out": (o / l).view(B, hq, D).to(s["out"].dtype), "weights": s["weights"]}


def _evict(s):
    c = s["case"]
    if own:
        import paged_kv_cache_227_gb300 as pa
        pa.pa_evict(s["pool"], s["weights"], s["tables"], s["lens"], s["keep"], s["lens_out"], s["kept"],
                    n_sink=c["sink"], n_recent=c["recent"], dst_tables=s["dst"], weights_out=s["weights_out"])
    else:
        w = s["weights"]
        B, hkv, span = w.shape
        L = s["lens"].long()[:, None]
        n = torch.minimum(s["keep"].long()[:, None], L)
        sink = torch.clamp(n, max=c["sink"])
        recent = torch.clamp(n - sink, max=c["recent"])
        t = torch.arange(span, device="cuda")[None, :]
        # rank: protected tokens first, then by weight, the earlier of two equals first, tokens past the end last
        always = (t < sink) | ((t >= L - recent) & (t < L))
        key = torch.where(always[:, None], torch.full_like(w, torch.inf), w)
        key = torch.where((t < L)[:, None], key, torch.full_like(w, -torch.inf))
        order = torch.sort(key, dim=2, descending=True, stable=True).indices
        left = torch.where((t < n)[:, None], order, torch.full_like(order, span)).sort(dim=2).values  # ascending, span past n
        stays = (t < n)[:, None].expand(B, hkv, span)
        src = left.clamp(max=span - 1)
        s["kept"] = torch.where(stays, left.int(), s["kept"])
        grown = torch.where(stays, w.gather(2, src), torch.zeros_like(w))
        s["weights_out"] = torch.where((t < L)[:, None], grown, s["weights_out"])
        s["lens_out"] = n[:, 0].int()
        # the rows move: token j of head h of sequence i comes from position left[i][h][j]
        i, h, j = stays.nonzero(as_tuple=True)
        p = left[i, h, j]
        blk, to = s["tables"][i, p // BS].long(), s["dst"][i, j // BS].long()
        for x in ("k", "v"):
            s[x][to, h, j % BS] = s[x][blk, h, p % BS]
    return {"k": s["k"], "v": s["v"], "weights": s["weights_out"], "kept": s["kept"], "lens": s["lens_out"]}


def work(case):
    hkv, e = case["hkv"], 2
    if case["op"] == "rope":
        n, hq = case["tokens"], case["hq"]
        return {"bytes": 2 * n * (hq + 2 * hkv) * D * e + n * (8 + 4 * case["axes"]),
                "flops": 3 * n * (hq + hkv) * case["rot"]}
    out = {"fp32": 4}.get(case.get("out"), 2)
    if case["op"] == "shared":
        B, hq, ng = case["batch"], case["hq"], case["groups"]
        pre = [BS * max(1, case["prefix"] // BS // (1 + k)) for k in range(ng)]
        suffix = sum(_lengths(B, case["suffix"], case["sigma"]))
        seen = suffix + sum(pre[i % ng] for i in range(B))
        return {"bytes": (sum(pre) + suffix) * hkv * D * 2 * e + B * hq * D * (e + out) + 4 * (sum(pre) + suffix) // BS,
                "flops": 4 * D * hq * seen}
    lens = _lengths(case["batch"], case["median"], case["sigma"])
    if case["op"] == "weights":
        B, hq = case["batch"], case["hq"]
        return {"bytes": sum(lens) * hkv * (D * 2 * e + 8) + B * hq * D * (e + out), "flops": 4 * D * hq * sum(lens)}
    kept = sum(min(case["keep"], x) for x in lens)
    return {"bytes": sum(lens) * hkv * 8 + kept * hkv * (2 * D * 2 * e + 4), "flops": sum(lens) * hkv}


def exact(case, seed):
    """The operators' definitions in 64 bits, token by token or sequence by sequence."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        rot, half = case["rot"], case["rot"] // 2
        pos = torch.stack([s["positions"][a] for a in s["axis_of_pair"]], 1).double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos * s["inv_freq"].double()[None, :])

        def turned(x):
            x = x.double()
            y = x.clone()
            at = (torch.arange(0, rot, 2), torch.arange(1, rot, 2)) if case["interleaved"] else (
                torch.arange(half), torch.arange(half, rot))
            z = torch.complex(x[..., at[0].cuda()], x[..., at[1].cuda()]) * turn[:, None, :]
            y[..., at[0].cuda()], y[..., at[1].cuda()] = z.real, z.imag
            return y

        k, v = s["k"].double(), s["v"].double()
        hkv = case["hkv"]
        rows = k.transpose(1, 2).reshape(-1, hkv, D).clone()
        rows[s["slots"]] = turned(s["k_new"])
        vrows = v.transpose(1, 2).reshape(-1, hkv, D).clone()
        vrows[s["slots"]] = s["v_new"].double()
        back = lambda r: r.view(-1, BS, hkv, D).transpose(1, 2)  # noqa: E731
        return {"q": turned(s["q"]), "k": back(rows), "v": back(vrows)}
    if case["op"] in ("shared", "weights"):
        hq, hkv = case["hq"], case["hkv"]
        outs, w = [], s["weights"].double() if case["op"] == "weights" else None
        lens = s["lens"].tolist()
        for i, L in enumerate(lens):
            blocks = s["tables"][i, :_up(L, BS)].long()
            k = s["k"][blocks].double().permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :L]
            v = s["v"][blocks].double().permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :L]
            q = s["q"][i].double().view(hkv, hq // hkv, D)
            p = torch.softmax(torch.einsum("hgd,htd->hgt", q, k) * s["scale"], dim=2)
            outs.append(torch.einsum("hgt,htd->hgd", p, v).reshape(hq, D))
            if w is not None:
                w[i, :, :L] = w[i, :, :L] * case["decay"] + p.sum(1)
        out = torch.stack(outs)
        return out if w is None else {"out": out, "weights": w}
    B, hkv, span = s["weights"].shape
    if B * hkv > 600:
        return None
    w = s["weights"].double().cpu()
    k, v = s["k"].double(), s["v"].double()
    k0, v0 = k.clone(), v.clone()
    grown = s["weights_out"].double().cpu()
    for i, L in enumerate(s["lens"].tolist()):
        n = min(case["keep"], L)
        a = min(case["sink"], n)
        b = min(case["recent"], n - a)
        for h in range(hkv):
            rest = w[i, h, a:L - b]
            order = torch.argsort(-rest, stable=True)[:n - a - b] + a
            at = torch.cat([torch.arange(a), order.sort().values, torch.arange(L - b, L)])
            grown[i, h, :n] = w[i, h, at]
            grown[i, h, n:L] = 0
            at = at.cuda()
            j = torch.arange(n, device="cuda")
            blk, to = s["tables"][i].long()[at // BS], s["dst"][i].long()[j // BS]
            k[to, h, j % BS] = k0[blk, h, at % BS]
            v[to, h, j % BS] = v0[blk, h, at % BS]
    return {"k": k, "v": v, "weights": grown, "kept": None, "lens": None}
