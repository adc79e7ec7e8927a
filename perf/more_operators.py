"""Measured cases of rotary positions and of the latent cache: rotation alone and fused with the
store into a pool of K/V heads, the store of normalised latents with their rotary key, and
attention over a pool of one latent vector a token.

Where ``own`` is true ``run`` makes the framework's calls; where it is false it computes the same
values with elementary torch operations in 32 bits (angles in 64).

Operators (``case["op"]``):
    rope          rotates the first ``rot`` elements of every head by its token's position
    rope_store    rotates q and k of a fused projection's rows and stores k and v into pool slots
    latent_store  RMS norm of a token's latent, its rotary key rotated, both written as one row
    latent        attention of each request's newest tokens over its latents (the absorbed form:
                  keys are whole rows, values their first ``r`` elements)
"""

import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
EPS = 1e-6
YARN = dict(factor=32.0, original=4096, beta_fast=32.0, beta_slow=1.0)


# ----------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step's queries: the rotary part of 128 absorbed heads, a slice of each row
        dict(name="rope 256x128 slice", op="rope", n=256, heads=128, dim=64, rot=64, row=576, inter=True, scaled=True, far=100000, seed=1),
        # a prompt batch's queries, whole heads
        dict(name="rope 16384x32", op="rope", n=16384, heads=32, dim=128, rot=128, row=128, inter=False, scaled=False, far=8192, seed=2),
        # a tiny interactive batch: latency counts
        dict(name="rope_store 4", op="rope_store", n=4, hq=8, hkv=2, d=64, rot=64, inter=False, scaled=False, fp8=False, far=80, seed=3),
        # chunks of long prompts into an 8-bit pool, positions far out, half of the head rotated
        dict(name="rope_store 65536 fp8", op="rope_store", n=65536, hq=32, hkv=8, d=128, rot=64, inter=False, scaled=True, fp8=True, far=1000000, seed=4),
        # one decode step's append
        dict(name="latent_store 256", op="latent_store", n=256, r=512, inter=True, scaled=True, far=100000, seed=5),
        # long prompts stored at once
        dict(name="latent_store 131072", op="latent_store", n=131072, r=512, inter=True, scaled=False, far=8192, seed=6),
        # a tiny interactive batch
        dict(name="latent tiny 4x80", op="latent", batch=4, heads=16, r=512, page=16, shared=64, new_lo=1, new_hi=1, len_lo=80, len_hi=80, seed=7),
        # one long document
        dict(name="latent 1x100001", op="latent", batch=1, heads=16, r=512, page=1, shared=0, new_lo=1, new_hi=1, len_lo=100001, len_hi=100001, seed=8),
        # batched decode of wide groups after a shared system prompt
        dict(name="latent 256 shared, 128 heads", op="latent", batch=256, heads=128, r=512, page=16, shared=1024, new_lo=1, new_hi=1, len_lo=1200, len_hi=3000, seed=9),
        # many long unrelated contexts
        dict(name="latent 64 ragged long, 32 heads", op="latent", batch=64, heads=32, r=512, page=64, shared=0, new_lo=1, new_hi=1, len_lo=500, len_hi=16384, seed=10),
        # a few tokens to verify after long contexts
        dict(name="latent 32x4 after 8000", op="latent", batch=32, heads=64, r=512, page=1, shared=0, new_lo=4, new_hi=4, len_lo=7000, len_hi=8000, seed=11),
        # short suffixes behind cached prefixes
        dict(name="latent 16x60 suffixes", op="latent", batch=16, heads=128, r=512, page=16, shared=1792, new_lo=40, new_hi=80, len_lo=1900, len_hi=3000, seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "rope_store", "latent_store", "latent", "latent"])
    seed = rng.randrange(1 << 30)
    rotary = dict(inter=rng.choice([False, True]), scaled=rng.choice([False, True]), far=_log_int(rng, 16, 1000000), seed=seed)
    if op == "rope":
        dim, rot, row = rng.choice([(128, 128, 128), (64, 64, 64), (64, 64, 576), (128, 64, 128), (64, 32, 64), (128, 96, 136), (256, 64, 256)])
        heads = rng.choice([1, 5, 8, 32, 128])
        return dict(op=op, n=_log_int(rng, 1, max(1, 16384 * 32 * 128 // (heads * row))), heads=heads, dim=dim, rot=rot, row=row, **rotary)
    if op == "rope_store":
        hq, hkv, d = rng.choice([(32, 8, 128), (8, 2, 64), (16, 16, 64), (8, 1, 128), (10, 5, 128), (64, 8, 128)])
        rot = rng.choice([d, d, d // 2, 32])
        return dict(op=op, n=_log_int(rng, 1, max(1, 65536 * 48 // (hq + 2 * hkv) // (d // 64) * 2)), hq=hq, hkv=hkv, d=d, rot=rot,
                    fp8=rng.choice([False, True]), **rotary)
    if op == "latent_store":
        return dict(op=op, n=_log_int(rng, 1, 131072), r=rng.choice([256, 512]), **rotary)
    heads, r, page = rng.choice([8, 16, 20, 32, 64, 96, 128]), rng.choice([256, 512, 512]), rng.choice([1, 16, 64])
    keys = _log_int(rng, 64, 500000)
    batch = _log_int(rng, 1, min(keys, 512))
    new = rng.choice([1, 1, 1, _log_int(rng, 1, 80)])
    hi = max(1, keys // batch // max(1, new * heads // 128))
    lo = rng.choice([0, 1, max(1, hi // 8), hi])
    shared = rng.choice([0, 0, lo // (2 * page) * page])
    return dict(op=op, batch=batch, heads=heads, r=r, page=page, shared=shared, new_lo=max(1, new // 2), new_hi=new, len_lo=lo, len_hi=hi,
                seed=seed)


# ----------------------------------------------------------------------------------------
# shapes (from the case alone: every seed of a case has the same lengths and pages)


def _lengths(case):
    """(context lengths, new tokens) of a latent case's requests."""
    rs = np.random.RandomState(case["seed"] % (1 << 31))
    seq = rs.randint(case["len_lo"], case["len_hi"] + 1, case["batch"])
    new = np.minimum(rs.randint(case["new_lo"], case["new_hi"] + 1, case["batch"]), seq)
    if case["new_hi"] == 1:
        new[:] = 1     # one query a request, of the empty ones too
    return seq, new


def _pages(case, blocks, shared_blocks):
    """Page ids of every request's blocks (padded rows) and the pages in all.  The first
    ``shared_blocks`` are the same pages for all requests."""
    rs = np.random.RandomState((case["seed"] + 17) % (1 << 31))
    own_blocks = blocks - shared_blocks
    total = int(own_blocks.sum()) + shared_blocks + 1
    perm = rs.permutation(total)
    table = np.zeros((len(blocks), max(int(blocks.max()), 1)), np.int32)
    table[:, :shared_blocks] = perm[:shared_blocks]
    at = shared_blocks
    for r, n in enumerate(own_blocks):
        table[r, shared_blocks:shared_blocks + n] = perm[at:at + n]
        at += n
    return table, total


# ----------------------------------------------------------------------------------------
# inputs


def _frequencies(rot, scaled):
    """(float64 angle per position of each pair, magnitude) of the case's rotation."""
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if not scaled:
        return f, 1.0
    # between the pairs that turn often within the original context and those that hardly do,
    # a ramp from the plain frequency to the interpolated one
    def edge(turns):
        return rot * math.log(YARN["original"] / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    lo, hi = max(math.floor(edge(YARN["beta_fast"])), 0), min(math.ceil(edge(YARN["beta_slow"])), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return f * (1 - ramp) + f / YARN["factor"] * ramp, 0.1 * math.log(YARN["factor"]) + 1.0


def _rope(case):
    import prefix_shared_kv_token_gb300 as pkv
    scaling = dict(kind="yarn", **YARN) if case["scaled"] else None
    return pkv.Rope(case.get("rot", 64), base=10000.0, layout="interleaved" if case["inter"] else "half", scaling=scaling)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "latent":
        return _prepare_latent(case, s, normal)
    n, rot = case["n"], case.get("rot", 64)
    f, s["magnitude"] = _frequencies(rot, case["scaled"])
    s["freq"] = torch.from_numpy(f).cuda()
    s["positions"] = torch.randint(0, case["far"], (n,), device="cuda", generator=gen, dtype=torch.int32)
    if own:
        s["rope"] = _rope(case)
    if case["op"] == "rope":
        rows = normal(n, case["heads"], case["row"]).to(torch.bfloat16)
        s["x"] = rows[..., case["row"] - case["dim"]:]
        s["out"] = torch.empty((n, case["heads"], case["dim"]), dtype=torch.bfloat16, device="cuda")
        return s
    slots = n + n // 8 + 3
    s["loc"] = torch.randperm(slots, device="cuda", generator=gen)[:n].to(torch.int32)
    s["ws"] = torch.zeros(64, dtype=torch.int32, device="cuda")
    if case["op"] == "latent_store":
        # a projection's rows: the latent, then the rotary key
        rows = (normal(n, case["r"] + 64) * torch.exp2(normal(n, 1))).to(torch.bfloat16)
        s["c"], s["pe"] = rows[:, :case["r"]], rows[:, case["r"]:]
        s["w"] = (1 + normal(case["r"]) / 4).to(torch.bfloat16)
        s["rows"] = torch.zeros((slots, case["r"] + 64), dtype=torch.bfloat16, device="cuda")
        if own:
            import prefix_shared_kv_token_gb300 as pkv
            s["pool"] = pkv.LatentPool(s["rows"], case["r"])
        return s
    # a fused projection's rows: q heads, k heads, v heads
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    qkv = normal(n, hq + 2 * hkv, d).to(torch.bfloat16)
    s["q"], s["kn"], s["vn"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    s["k"], s["v"] = (torch.zeros((slots, hkv, d), dtype=torch.uint8 if case["fp8"] else torch.bfloat16, device="cuda") for _ in range(2))
    s["scales"] = (0.02, 0.011) if case["fp8"] else (1.0, 1.0)
    if own:
        import prefix_shared_kv_token_gb300 as pkv
        s["pool"] = pkv.Pool(s["k"], s["v"], "fp8_e4m3" if case["fp8"] else "bf16", *s["scales"])
    return s


def _prepare_latent(case, s, normal):
    seq, new = _lengths(case)
    page, batch, heads, r = case["page"], case["batch"], case["heads"], case["r"]
    blocks = (seq + page - 1) // page
    table, total = _pages(case, blocks, case["shared"] // page)
    rows = np.random.RandomState(case["seed"] % 1000).permutation(batch)
    by_row = np.zeros_like(table)
    by_row[rows] = table
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    qo = np.concatenate([[0], np.cumsum(new)])
    s |= dict(table=dev(by_row), rows=dev(rows), seq=dev(seq), qo=dev(qo), lens=seq.tolist(), starts=qo.tolist(), row_list=rows.tolist())
    pool = normal(total * page, r + 64).to(torch.bfloat16)
    # what lies behind a sequence in its last page is nobody's
    ends = np.nonzero(seq % page)[0]
    dead = [np.arange(table[e, blocks[e] - 1] * page + seq[e] % page, (table[e, blocks[e] - 1] + 1) * page) for e in ends]
    pool[torch.from_numpy(np.concatenate(dead + [np.zeros(0, np.int64)]).astype(np.int64)).cuda()] = float("nan")
    s["pool_rows"] = pool
    s["q"] = normal(int(qo[-1]), heads, r + 64).to(torch.bfloat16)
    s["o"] = torch.empty((int(qo[-1]), heads, r), dtype=torch.bfloat16, device="cuda")
    s["scale"] = (128 + 64) ** -0.5
    if own:
        import prefix_shared_kv_token_gb300 as pkv
        s["pool"] = pkv.LatentPool(pool, r)
        s["batch"] = pkv.Batch(s["table"], s["rows"], s["seq"], page)
        s["ws"] = torch.zeros(pkv.latent_workspace(s["pool"], heads) // 4, dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------------------------------
# one pass


def _rotate(s, x, positions):
    """float32 x [n, heads, dim] with its first rot elements rotated."""
    case, x = s["case"], x.float()
    rot = case.get("rot", 64)
    a = positions.double()[:, None] * s["freq"]
    cos, sin = ((s["magnitude"] * t).float()[:, None] for t in (a.cos(), a.sin()))
    turned = x[..., :rot]
    x1, x2 = (turned[..., 0::2], turned[..., 1::2]) if case["inter"] else (turned[..., :rot // 2], turned[..., rot // 2:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if case["inter"] else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _held(x, scale, fp8):
    if not fp8:
        return x.to(torch.bfloat16)
    return (x / scale).clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def _attend(s):
    c, page = s["case"], s["case"]["page"]
    out = torch.zeros(s["o"].shape, device="cuda")
    for b, length in enumerate(s["lens"]):
        i, j = s["starts"][b], s["starts"][b + 1]
        if i == j or length == 0:
            continue
        t = torch.arange(length, device="cuda")
        keys = s["pool_rows"][s["table"][s["row_list"][b], t // page].long() * page + t % page].float()
        w = torch.matmul(s["q"][i:j].float(), keys.T) * s["scale"]
        seen = t[None] <= length - (j - i) + torch.arange(j - i, device="cuda")[:, None]
        w = w.masked_fill_(~seen[:, None], float("-inf"))
        w = torch.exp(w - w.amax(-1, keepdim=True))
        out[i:j] = torch.matmul(w, keys[:, :c["r"]]) / w.sum(-1, keepdim=True)
    return out.to(torch.bfloat16)


def run(s):
    op = s["case"]["op"]
    if own:
        import prefix_shared_kv_token_gb300 as pkv
        if op == "rope":
            return pkv.rope(s["x"], s["positions"], s["rope"], out=s["out"])
        if op == "rope_store":
            pkv.rope_store(s["pool"], s["q"], s["kn"], s["vn"], s["positions"], s["loc"], s["rope"], q_out=s["q_out"], workspace=s["ws"])
        elif op == "latent_store":
            pkv.latent_store(s["pool"], s["c"], s["pe"], s["positions"], s["loc"], s["rope"], norm_weight=s["w"], eps=EPS, workspace=s["ws"])
        else:
            pkv.attn_latent(s["pool"], s["batch"], s["q"], s["o"], s["scale"], s["ws"], qo_indptr=None if s["case"]["new_hi"] == 1 else s["qo"])
            return s["o"]
    elif op == "rope":
        return _rotate(s, s["x"], s["positions"]).to(torch.bfloat16)
    elif op == "rope_store":
        loc, fp8 = s["loc"].long(), s["case"]["fp8"]
        s["q_out"].copy_(_rotate(s, s["q"], s["positions"]))
        s["k"][loc] = _held(_rotate(s, s["kn"], s["positions"]), s["scales"][0], fp8)
        s["v"][loc] = _held(s["vn"].float(), s["scales"][1], fp8)
    elif op == "latent_store":
        c = s["c"].float()
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["w"].float()
        s["rows"][s["loc"].long()] = torch.cat((c, _rotate(s, s["pe"][:, None], s["positions"])[:, 0]), -1).to(torch.bfloat16)
    else:
        return _attend(s)
    if op == "latent_store":
        return s["rows"]
    fp8 = s["case"]["fp8"]
    return dict(q=s["q_out"], k=s["k"].view(F8) if fp8 else s["k"], v=s["v"].view(F8) if fp8 else s["v"])


# ----------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "latent":
        seq, new = _lengths(case)
        r, heads, shared = case["r"], case["heads"], case["shared"]
        keys = int(np.maximum(seq - shared, 0).sum()) + min(shared, int(seq.max()))
        pairs = int((new * np.maximum(seq - new, 0) + new * (new + 1) // 2)[seq > 0].sum())
        return {"bytes": 2 * keys * (r + 64) + 4 * keys // case["page"] + 2 * int(new.sum()) * heads * (2 * r + 64),
                "flops": 2 * pairs * heads * (2 * r + 64)}
    n = case["n"]
    if op == "rope":
        return {"bytes": 4 * n * case["heads"] * case["dim"] + 4 * n, "flops": 3 * n * case["heads"] * case["rot"]}
    if op == "latent_store":
        return {"bytes": 4 * n * (case["r"] + 64) + 8 * n + 2 * case["r"], "flops": n * (4 * case["r"] + 3 * 64)}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    kv = 2 * hkv * d * (3 if case["fp8"] else 4)
    return {"bytes": n * (4 * hq * d + kv + 8), "flops": 3 * n * (hq + hkv) * case["rot"]}


# ----------------------------------------------------------------------------------------
# the operators' definitions in 64 bits


def _turned(case, x, positions):
    """float64 x [n, heads, dim] rotated as complex numbers."""
    rot = case.get("rot", 64)
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f, magnitude = torch.exp(-2 * i / rot * math.log(10000.0)), 1.0
    if case["scaled"]:
        turns = [rot / 2 * (math.log(YARN["original"]) - math.log(2 * math.pi * b)) / math.log(10000.0)
                 for b in (YARN["beta_fast"], YARN["beta_slow"])]
        lo, hi = max(math.floor(turns[0]), 0), min(math.ceil(turns[1]), rot - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (keep + (1 - keep) / YARN["factor"])
        magnitude = 1 + math.log(YARN["factor"]) / 10
    a = positions.double()[:, None] * f
    unit = torch.polar(torch.full_like(a, magnitude), a)[:, None]
    out = x.double().clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(out[..., first].contiguous(), out[..., second].contiguous()) * unit
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(case, s["x"], s["positions"])
    if op == "rope_store":
        k, v = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        loc = s["loc"].long()
        k[loc] = _turned(case, s["kn"], s["positions"]) / float(np.float32(s["scales"][0]))
        v[loc] = s["vn"].double() / float(np.float32(s["scales"][1]))
        if case["fp8"]:
            k, v = k.clamp(-448, 448), v.clamp(-448, 448)
        return dict(q=_turned(case, s["q"], s["positions"]), k=k, v=v)
    if op == "latent_store":
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
        c = s["c"].double()
        c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / case["r"] + EPS) * s["w"].double()
        rows[s["loc"].long()] = torch.cat((c, _turned(case, s["pe"][:, None], s["positions"])[:, 0]), -1)
        return rows
    if work(case)["flops"] > 3e12:
        return None
    seq, new = _lengths(case)
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["batch"]):
        n, length = int(new[b]), int(seq[b])
        if n and length:
            pages = s["table"][s["rows"][b].long()].long()
            held = s["pool_rows"].view(-1, case["page"], case["r"] + 64)[pages].reshape(-1, case["r"] + 64)[:length].double()
            for i in range(n):
                a = held[:length - n + i + 1]
                out[at + i] = torch.softmax(s["q"][at + i].double() @ a.T * s["scale"], -1) @ a[:, :case["r"]]
        at += n
    return out
