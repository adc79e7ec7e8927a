"""Measured cases of the block-scaled 8-bit KV cache: page tables and slot maps built on the
GPU, the store that quantises new rows, and the attention that reads them.

The cache holds e4m3 codes in pages of ``page_size`` tokens.  Each page has one exponent byte
per KV head for K and one for V: a code c under byte b stands for c * 2^(b - 127).  Where
``own`` is true ``run`` makes the framework's calls; where it is false it computes the same
values with elementary torch operations in 32 bits.

Operators (``case["op"]``):
    tables   a step's page table entries, slot map, positions and offsets from request lengths
    store    new K/V rows quantised into their pages (a page's exponent may have to grow)
    decode   one query token per request over its whole context
    extend   causal attention of each request's new tokens over its context
"""

import numpy as np
import torch

own = False

E_MIN, E_MAX = -117, 118     # exponents a page may have
F8 = torch.float8_e4m3fn


# ----------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step of a running batch: every request grows by a token
        dict(name="tables decode 256", op="tables", batch=256, page=16, old_lo=100, old_hi=4000, new_lo=1, new_hi=1, seed=1),
        # admission of many prompts whose prefixes are cached in part
        dict(name="tables prefill 1000", op="tables", batch=1000, page=64, old_lo=0, old_hi=1800, new_lo=1, new_hi=400, seed=2),
        # one decode step's append: one token per request, mostly into half-filled pages
        dict(name="store append 256", op="store", batch=256, hkv=8, d=128, page=16, old_lo=100, old_hi=3000, new_lo=1, new_hi=1, seed=3),
        # the few-shot prefill: 64 requests of about 200 new tokens
        dict(name="store prompts 64x200", op="store", batch=64, hkv=8, d=128, page=16, old_lo=1700, old_hi=1900, new_lo=150, new_hi=250, seed=4),
        # long prompts stored at once, in larger pages
        dict(name="store prompts 16x8192", op="store", batch=16, hkv=8, d=128, page=64, old_lo=0, old_hi=0, new_lo=8100, new_hi=8192, seed=5),
        # a tiny interactive batch: latency counts
        dict(name="decode tiny 4x80", op="decode", batch=4, hq=8, hkv=2, d=64, page=16, shared=64, len_lo=80, len_hi=80, seed=6),
        # one long document
        dict(name="decode 1x100001", op="decode", batch=1, hq=32, hkv=8, d=128, page=16, shared=0, len_lo=100001, len_hi=100001, seed=7),
        # batched decode after a shared system prompt
        dict(name="decode 256 shared 2048", op="decode", batch=256, hq=32, hkv=8, d=128, page=16, shared=2048, len_lo=2176, len_hi=3000, seed=8),
        # many long unrelated contexts, wide groups
        dict(name="decode 64 ragged long", op="decode", batch=64, hq=64, hkv=8, d=128, page=64, shared=0, len_lo=500, len_hi=16384, seed=9),
        # a few tokens to verify after a long context
        dict(name="extend 4x5 after 9000", op="extend", batch=4, hq=32, hkv=8, d=128, page=16, shared=0, old_lo=8000, old_hi=9000, new_lo=5, new_hi=5, seed=10),
        # the few-shot prefill behind a shared prefix
        dict(name="extend 64x200 shared 1792", op="extend", batch=64, hq=32, hkv=8, d=128, page=16, shared=1792, old_lo=1792, old_hi=1800, new_lo=150, new_hi=250, seed=11),
        # the last 1,024-token chunk of long prompts
        dict(name="extend 16x1024 chunk", op="extend", batch=16, hq=32, hkv=8, d=128, page=64, shared=0, old_lo=6900, old_hi=7168, new_lo=1000, new_hi=1024, seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tables", "store", "decode", "extend"])
    page = rng.choice([16, 32, 64, 128])
    hkv, g, d = rng.choice([(8, 4, 128), (8, 8, 128), (2, 4, 64), (16, 1, 64), (1, 8, 128), (5, 2, 128), (4, 4, 64)])
    seed = rng.randrange(1 << 30)
    if op == "tables":
        b = _log_int(rng, 1, 1000)
        new = _log_int(rng, 1, max(1, min(8192, 200000 // b)))
        return dict(op=op, batch=b, page=page, old_lo=0, old_hi=_log_int(rng, 1, 16384), new_lo=rng.choice([0, 1]), new_hi=new, seed=seed)
    if op == "store":
        n = _log_int(rng, 1, 120000)
        b = _log_int(rng, 1, min(n, 512))
        new = max(1, n // b)
        old = _log_int(rng, 1, max(1, min(4000, 120000 // b)))
        return dict(op=op, batch=b, hkv=hkv, d=d, page=page, old_lo=0, old_hi=old, new_lo=max(1, new // 2), new_hi=new, seed=seed)
    if op == "decode":
        n = _log_int(rng, 64, 300000)
        b = _log_int(rng, 1, min(n, 512))
        hi = max(1, n // b)
        lo = rng.choice([0, 1, max(1, hi // 8), hi])
        shared = rng.choice([0, 0, lo // (2 * page) * page])
        return dict(op=op, batch=b, hq=hkv * g, hkv=hkv, d=d, page=page, shared=shared, len_lo=lo, len_hi=hi, seed=seed)
    b = _log_int(rng, 1, 64)
    new = _log_int(rng, 1, max(1, 16384 // b))
    old = _log_int(rng, 1, max(1, min(8192, 100000 // b, 60000000 // (b * new))))
    shared = rng.choice([0, old // (2 * page) * page])
    return dict(op=op, batch=b, hq=hkv * g, hkv=hkv, d=d, page=page, shared=shared, old_lo=max(shared, old // 2), old_hi=old,
                new_lo=max(1, new // 2), new_hi=new, seed=seed)


# ----------------------------------------------------------------------------------------
# shapes (from the case alone: every seed of a case has the same lengths and pages)


def _lengths(case):
    """(lengths before, new tokens) of the case's requests."""
    rs = np.random.RandomState(case["seed"] % (1 << 31))
    b = case["batch"]
    if case["op"] == "decode":
        return np.zeros(b, np.int64), rs.randint(case["len_lo"], case["len_hi"] + 1, b)
    old = rs.randint(case["old_lo"], case["old_hi"] + 1, b)
    return old, rs.randint(case["new_lo"], case["new_hi"] + 1, b)


def _pages(case, blocks, shared_blocks):
    """Page ids of every request's blocks (padded rows) and the pages in all.  The first
    ``shared_blocks`` are the same pages for all requests."""
    rs = np.random.RandomState((case["seed"] + 17) % (1 << 31))
    own_blocks = blocks - shared_blocks
    total = int(own_blocks.sum()) + shared_blocks + 1
    perm = rs.permutation(total)
    stride = max(int(blocks.max()), 1)
    table = np.zeros((len(blocks), stride), np.int32)
    table[:, :shared_blocks] = perm[:shared_blocks]
    at = shared_blocks
    for r, n in enumerate(own_blocks):
        table[r, shared_blocks:shared_blocks + n] = perm[at:at + n]
        at += n
    return table, total


# ----------------------------------------------------------------------------------------
# inputs


def _exponent(amax):
    """The smallest exponent under which amax is at most 448, as torch.frexp gives it."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    """2^e in float32, exactly (exp2 may be an ulp off, which would break ties the wrong way)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x):
    return x.clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def _cache(pages, page, hkv, d, gen):
    """Codes [pages * page, hkv, d] and exponent bytes [pages, hkv] of rows that a model might
    have stored: normal values whose size differs by head and page."""
    size = torch.exp2(torch.randn((pages, 1, hkv, 1), device="cuda", generator=gen))
    x = torch.randn((pages, page, hkv, d), device="cuda", generator=gen) * size
    e = _exponent(x.abs().amax(dim=(1, 3)))
    codes = _encode(x * _pow2(-e)[:, None, :, None])
    return codes.view(pages * page, hkv, d), (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    old, new = _lengths(case)
    seq, page, batch = old + new, case["page"], case["batch"]
    blocks = (seq + page - 1) // page
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    s = dict(case=case, seq=dev(seq), new=dev(new), max_len=int(seq.max()), max_new=int(new.max()))
    rows = np.random.RandomState(case["seed"] % 1000).permutation(batch)
    s["rows"] = dev(rows)
    qo = np.concatenate([[0], np.cumsum(new)])
    if case["op"] == "tables":
        had = (old + page - 1) // page
        ids = torch.randperm(int(blocks.sum()) + 40, device="cuda", generator=gen).to(torch.int32)
        table = torch.full((batch, int(blocks.max()) + 1), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(table.shape[1], device="cuda")[None] < dev(had)[:, None]
        first = dev(np.cumsum(had) - had)
        pos = first[:, None] + torch.arange(table.shape[1], device="cuda", dtype=torch.int32)[None]
        table[s["rows"].long()] = torch.where(held, ids[pos.clamp(max=len(ids) - 1).long()], -1)
        n = int(new.sum())
        s |= dict(table=table, free=ids[int(had.sum()):].contiguous(),
                  head=torch.full((1,), 3, dtype=torch.int32, device="cuda"),
                  head_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
                  loc=torch.zeros(n + 7, dtype=torch.int32, device="cuda"),
                  pos=torch.zeros(n + 7, dtype=torch.int32, device="cuda"),
                  qo=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"),
                  ws=torch.zeros(64, dtype=torch.int32, device="cuda"))
        return s
    hkv, d = case["hkv"], case["d"]
    table, total = _pages(case, blocks, case.get("shared", 0) // page)
    by_row = np.zeros_like(table)
    by_row[rows] = table
    s["table"] = dev(by_row)
    (s["k"], s["k_exp"]), (s["v"], s["v_exp"]) = (_cache(total, page, hkv, d, gen) for _ in range(2))
    # what lies behind a sequence in its last page is nobody's: codes of NaN
    ends = np.nonzero(seq % page)[0]
    last = table[ends, blocks[ends] - 1].astype(np.int64) * page
    dead = np.concatenate([np.arange(a + n % page, a + page) for a, n in zip(last, seq[ends])] or [np.zeros(0, np.int64)])
    dead = torch.from_numpy(dead).cuda()
    s["k"][dead] = 0x7F
    s["v"][dead] = 0x7F
    req = np.repeat(np.arange(batch), new)
    pos = np.arange(len(req)) - qo[req] + old[req]
    if case["op"] == "store":
        size = torch.exp2(torch.randn((len(req), hkv, 1), device="cuda", generator=gen))
        s["k_new"], s["v_new"] = (
            (torch.randn((len(req), hkv, d), device="cuda", generator=gen) * size).to(torch.bfloat16) for _ in range(2))
        s["loc"] = dev(table[req, pos // page].astype(np.int64) * page + pos % page)
        s["first"] = dev(qo[:-1])
        s["ws"] = torch.zeros(64, dtype=torch.int32, device="cuda")
        if own:
            import prefix_shared_kv_token_gb300 as pkv
            s["pool"] = pkv.BlockPool(s["k"], s["v"], s["k_exp"], s["v_exp"], page)
        return s
    hq = case["hq"]
    tokens = batch if case["op"] == "decode" else len(req)
    s["scale"] = d ** -0.5
    s["q"] = (2 * torch.randn((tokens, hq, d), device="cuda", generator=gen)).to(torch.bfloat16)
    s["o"] = torch.empty_like(s["q"])
    s |= dict(req=dev(req), pos=dev(pos), qo=dev(qo))
    if own:
        import prefix_shared_kv_token_gb300 as pkv
        s["pool"] = pkv.BlockPool(s["k"], s["v"], s["k_exp"], s["v_exp"], page)
        s["batch"] = pkv.Batch(s["table"], s["rows"], s["seq"], page)
        if case["op"] == "decode":
            size = pkv.decode_block_workspace(s["pool"], hq)
        else:
            shared, cascade = case["shared"], None
            if shared and batch > 1:
                cascade = pkv.Cascade(*(np.asarray(a, np.int32) for a in ([0], [0], [shared], [0, batch], np.arange(batch))))
            s["plan"] = pkv.plan_extend(seq, new, qo, hq, hkv, d, cascade)
            s["plan_dev"] = torch.from_numpy(s["plan"].blob).cuda()
            size = s["plan"].info.workspace_bytes
        s["ws"] = torch.zeros((size + 3) // 4, dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------------------------------
# one pass


def _tables(s):
    page, table = s["case"]["page"], s["table"]
    seq, new, rows = s["seq"].long(), s["new"].long(), s["rows"].long()
    old = seq - new
    had, has = (old + page - 1) // page, (seq + page - 1) // page
    need = has - had
    taken = need.cumsum(0) - need
    block = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (block >= had[:, None]) & (block < has[:, None])
    at = s["head"].long() + taken[:, None] + block - had[:, None]
    here = table[rows]
    here = torch.where(fresh, s["free"][at.clamp(0, len(s["free"]) - 1)], here)
    table[rows] = here
    qo = s["qo"]
    qo[1:] = new.cumsum(0)
    i = torch.arange(len(s["loc"]), device="cuda")
    r = torch.searchsorted(qo[1:].long(), i, right=True)
    in_use = r < len(seq)
    r = r.clamp(max=len(seq) - 1)
    t = i - qo.long()[r] + old[r]
    slot = here[r, (t // page).clamp(0, table.shape[1] - 1)].long() * page + t % page
    s["loc"].copy_(torch.where(in_use, slot, -1))
    s["pos"].copy_(torch.where(in_use, t, -1))
    s["head_out"].copy_(s["head"] + need.sum())
    return dict(table=table, loc=s["loc"], pos=s["pos"], qo=qo, head=s["head_out"])


def _store(codes, exps, x, loc, first, page):
    x = x.float()
    block = loc // page
    amax = torch.zeros(exps.shape, device="cuda").scatter_reduce_(
        0, block[:, None].expand(-1, exps.shape[1]), x.abs().amax(2), "amax")
    written = torch.zeros(len(exps), dtype=torch.bool, device="cuda")
    written[block] = True
    begun = torch.zeros_like(written)   # pages that held rows of the request before
    lead = loc[first]
    begun[lead // page] = lead % page > 0
    e_old, e_new = exps.int() - 127, _exponent(amax)
    e = torch.where(begun[:, None], torch.maximum(e_old, e_new), torch.where(written[:, None], e_new, e_old))
    # rows that were there before the new ones
    rows = (lead // page * page)[:, None] + torch.arange(page, device="cuda")[None]
    live = rows < lead[:, None]
    was = codes[rows]
    shift = _pow2((e_old - e).clamp(min=-126))[lead // page][:, None, :, None]
    codes[rows] = torch.where(live[..., None, None], _encode(was.view(F8).float() * shift), was)
    codes[loc] = _encode(x * _pow2(-e)[block][..., None])
    exps.copy_(e + 127)


def _rows(s, codes, exps):
    """float32 [batch, max_len, hkv, d]: every request's rows, zeros behind its end."""
    page = s["case"]["page"]
    t = torch.arange(s["max_len"], device="cuda")
    pages = s["table"][s["rows"].long()][:, t // page].long()
    x = codes[pages * page + t % page].view(F8).float()
    x *= _pow2(exps[pages].int() - 127)[..., None]
    return x.masked_fill_(t[None, :, None, None] >= s["seq"][:, None, None, None], 0.0)


def _attend(s):
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    k, v = _rows(s, s["k"], s["k_exp"]), _rows(s, s["v"], s["v_exp"])
    q = s["q"].float().view(-1, hkv, c["hq"] // hkv, d)
    t = torch.arange(s["max_len"], device="cuda")
    if c["op"] == "decode":
        q = q[:, None]
        seen = t[None, None] < s["seq"][:, None, None]
    else:
        i = torch.arange(s["max_new"], device="cuda")
        q = q[(s["qo"][:-1, None] + i[None]).clamp(max=len(s["q"]) - 1).long()]
        seen = t[None, None] < (s["seq"] - s["new"] + 1)[:, None, None] + i[None, :, None]
    w = torch.einsum("bighd,btgd->bghit", q, k) * s["scale"]
    w = w.masked_fill_(~seen[:, None, None], float("-inf"))
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == float("-inf"), 0.0, top))
    total = w.sum(-1, keepdim=True)
    o = torch.einsum("bghit,btgd->bghid", w, v) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(len(s["seq"]), -1, c["hq"], d)
    if c["op"] == "extend":
        r = s["req"].long()
        return o[r, (s["pos"] - (s["seq"] - s["new"])[r]).long()].to(torch.bfloat16)
    return o[:, 0].to(torch.bfloat16)


def run(s):
    op = s["case"]["op"]
    if op == "tables":
        if own:
            import prefix_shared_kv_token_gb300 as pkv
            pkv.build_block_tables(s["table"], s["rows"], s["seq"], s["new"], s["free"], s["head"], s["head_out"], s["loc"],
                                   s["pos"], s["qo"], s["case"]["page"], s["ws"])
            return dict(table=s["table"], loc=s["loc"], pos=s["pos"], qo=s["qo"], head=s["head_out"])
        return _tables(s)
    if op == "store":
        if own:
            import prefix_shared_kv_token_gb300 as pkv
            pkv.kv_store_block(s["pool"], s["k_new"], s["v_new"], s["loc"], s["ws"])
        else:
            loc, first = s["loc"].long(), s["first"].long()
            _store(s["k"], s["k_exp"], s["k_new"], loc, first, s["case"]["page"])
            _store(s["v"], s["v_exp"], s["v_new"], loc, first, s["case"]["page"])
        return dict(k=s["k"].view(F8), v=s["v"].view(F8), k_exp=s["k_exp"], v_exp=s["v_exp"])
    if own:
        import prefix_shared_kv_token_gb300 as pkv
        if op == "decode":
            pkv.attn_decode_block(s["pool"], s["batch"], s["q"], s["o"], s["scale"], s["ws"])
        else:
            pkv.attn_extend_block(s["pool"], s["batch"], s["q"], s["o"], s["scale"], s["plan"], s["plan_dev"], s["ws"])
        return s["o"]
    return _attend(s)


# ----------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    old, new = _lengths(case)
    seq, page, n = old + new, case["page"], int(new.sum())
    blocks = (seq + page - 1) // page
    if case["op"] == "tables":
        fresh = blocks - (old + page - 1) // page
        begun = int(((old % page > 0) & (new > 0)).sum())
        return {"bytes": 4 * (4 * case["batch"] + 2 * int(fresh.sum()) + begun + 2 * n), "flops": 0}
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "store":
        # bf16 rows in, codes and exponents out
        pages = int((blocks - old // page).sum())
        return {"bytes": 2 * n * hkv * d * 3 + 4 * n + 4 * pages * hkv, "flops": 0}
    shared = case["shared"]
    keys = int(np.maximum(seq - shared, 0).sum()) + min(shared, int(seq.max()))
    q = case["batch"] if case["op"] == "decode" else n
    if case["op"] == "decode":
        pairs = int(seq.sum())
    else:
        pairs = int((new * old + new * (new + 1) // 2).sum())
    return {"bytes": 2 * keys * hkv * d + 2 * (keys // page) * hkv + 4 * q * case["hq"] * d, "flops": 4 * pairs * case["hq"] * d}


# ----------------------------------------------------------------------------------------
# the operators' definitions in 64 bits


def _two_to(e):
    """2^e in float64, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), at most 448 in size, in float64."""
    size = x.abs().clamp(max=448.0)
    step = _two_to(torch.frexp(size.clamp(min=2.0 ** -6)).exponent - 4)
    return torch.sign(x) * torch.round(size / step) * step


def _exact_store(codes, exps, x, loc, new, page):
    values = codes.view(F8).double()
    loc, at = loc.cpu().numpy().astype(np.int64), 0
    for n in new:
        for a in range(at - loc[at] % page, at + n, page):   # a page's first row, as if all were new
            i, j = max(a, at), min(a + page, at + n)
            block, off = loc[i] // page, int(loc[i] % page)
            rows = x[i:j].double()
            amax = rows.abs().amax(dim=(0, 2))
            part, e = torch.frexp(amax / 448.0)   # part in [0.5, 1): amax <= 448 * 2^e, the smallest such e
            e = torch.where(amax > 0, e - (part == 0.5).to(e.dtype), E_MIN).clamp(E_MIN, E_MAX).long()
            if off:
                e_old = exps[block].long() - 127
                e = torch.maximum(e, e_old)
                s0 = slice(loc[i] - off, loc[i])
                values[s0] = _e4m3(values[s0] * _two_to(e_old - e)[None, :, None])
            values[loc[i]:loc[i] + j - i] = _e4m3(rows * _two_to(-e)[None, :, None])
            exps[block] = (e + 127).to(torch.uint8)
        at += n
    return values


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    old, new = _lengths(case)
    page = case["page"]
    if case["op"] == "store":
        if int(new.sum()) // page + case["batch"] > 3000:
            return None
        k = _exact_store(s["k"], s["k_exp"], s["k_new"], s["loc"], new, page)
        v = _exact_store(s["v"], s["v_exp"], s["v_new"], s["loc"], new, page)
        return dict(k=k, v=v, k_exp=None, v_exp=None)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if work(case)["flops"] > 3e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r in range(case["batch"]):
        n = 1 if case["op"] == "decode" else int(new[r])
        length = int(old[r] + new[r])
        pages = s["table"][s["rows"][r].long()].long()
        kv = []
        for codes, exps in ((s["k"], s["k_exp"]), (s["v"], s["v_exp"])):
            paged = codes.view(-1, page, hkv, d)[pages].view(F8).double()
            paged = paged * _two_to(exps[pages].long() - 127)[:, None, :, None]
            kv.append(paged.reshape(-1, hkv, d)[:length])
        ask = s["q"][at:at + n].double()
        if length:
            for h in range(hq):
                a = ask[:, h] @ kv[0][:, h * hkv // hq].T * s["scale"]
                hidden = torch.ones_like(a, dtype=torch.bool).triu(length - n + 1)
                a = torch.softmax(a.masked_fill(hidden, float("-inf")), -1)
                out[at:at + n, h] = a @ kv[1][:, h * hkv // hq]
        at += n
    return out
