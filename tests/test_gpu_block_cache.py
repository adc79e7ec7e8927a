"""The block-scaled cache on the GPU against its plain 64-bit forms: page tables and slot maps
built on the device, the quantising store, decode and extend attention, and a run of them
together captured in a graph.  The error bounds are derived in block_reference.attend."""

import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import prefix_shared_kv_token_gb300 as m
    return m


def dev(a, t=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, t)).cuda()


def host(t):
    return t.cpu().numpy()


def bf16(x):
    """(device bf16 tensor, its float64 values) of an array."""
    bits = ref.bf16_bits(x)
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), ref.bf16_values(bits)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def words(n=64):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


def error(pkv, ws):
    return pkv.get_device_error(ws)


# ----------------------------------------------------------------------------------------
# tables


def table_inputs(rng, b, page, longest, most_new):
    seq = rng.integers(0, longest + 1, b)
    new = np.minimum(rng.integers(0, most_new + 1, b), seq)
    blocks = -(-seq // page)
    had = -(-(seq - new) // page)
    stride = int(max(blocks.max(), 1)) + 2
    ids = rng.permutation(int(blocks.sum()) + 9)
    rows = rng.permutation(b + 3)[:b]
    table, at = np.full((b + 3, stride), -7), 0
    for r, n in zip(rows, had):
        table[r, :n] = ids[at:at + n]
        at += n
    return seq, new, rows, table, ids[at:]


def build(pkv, page, seq, new, rows, table, free, head, cap, ws=None, in_place=False):
    t, h = dev(table), dev([head])
    out = h if in_place else words(1)
    loc, pos, qo = words(cap), words(cap), words(len(seq) + 1)
    ws = words() if ws is None else ws
    pkv.build_block_tables(t, dev(rows), dev(seq), dev(new), dev(free), h, out, loc, pos, qo, page, ws)
    return [host(x) for x in (t, loc, pos, qo, out)], ws


@pytest.mark.parametrize("b,page,longest,most_new", [
    (1, 16, 1, 1), (1, 16, 5000, 4000), (3, 1, 40, 40), (33, 2, 70, 3), (256, 16, 4000, 1), (257, 64, 1000, 300),
    (1500, 128, 700, 90), (16384, 16, 100, 2), (5, 4096, 9000, 9000)])
def test_tables(pkv, b, page, longest, most_new):
    rng = np.random.default_rng(b + page)
    seq, new, rows, table, free = table_inputs(rng, b, page, longest, most_new)
    cap = int(new.sum()) + 5
    want = ref.tables(table, rows, seq, new, np.concatenate([[0, 0], free]), 2, page, cap)
    for in_place in (False, True):
        got, ws = build(pkv, page, seq, new, rows, table, np.concatenate([[0, 0], free]), 2, cap, in_place=in_place)
        assert error(pkv, ws) == 0
        for g, w in zip(got, want):
            assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1))
        assert int(ws[16]) == 0   # the workspace is ready for the next call


def test_tables_empty_batch(pkv):
    got, ws = build(pkv, 16, [], [], [], np.full((2, 3), 5), [1, 2], 1, 4)
    assert error(pkv, ws) == 0 and np.all(got[0] == 5) and np.all(got[1] == -1) and np.all(got[2] == -1)
    assert got[3].tolist() == [0] and got[4].tolist() == [1]


@pytest.mark.parametrize("case,code", [("few pages", 0x800), ("cap", 0x400), ("length", 0x400), ("row", 0x400),
                                       ("negative", 0x400), ("more new than all", 0x400), ("head", 0x800),
                                       ("huge", 0x400)])
@pytest.mark.parametrize("b", [5, 700])
def test_tables_refuse_a_bad_step_whole(pkv, case, code, b):
    rng = np.random.default_rng(b)
    seq, new, rows, table, free = table_inputs(rng, b, 16, 300, 60)
    head, cap = 0, int(new.sum())
    need = int((-(-seq // 16) - -(-(seq - new) // 16)).sum())
    seq, new, rows = seq.copy(), new.copy(), rows.copy()
    if case == "few pages":
        free = free[:need - 1]
    elif case == "cap":
        cap -= 1
    elif case == "length":
        seq[b // 2] = table.shape[1] * 16 + 1
    elif case == "row":
        rows[b - 1] = len(table)
    elif case == "negative":
        new[0] = -1
    elif case == "more new than all":
        new[0] = seq[0] + 1
    elif case == "head":
        head = -1
    else:
        seq[:] = new[:] = 2**31 - 1     # their sum passes 2^31
    got, ws = build(pkv, 16, seq, new, rows, table, free, head, cap)
    assert error(pkv, ws) == code
    assert np.array_equal(got[0], table) and np.all(got[1] == -1) and np.all(got[2] == -1)
    assert np.all(got[3] == 0) and got[4].tolist() == [head]


@pytest.mark.parametrize("page", [1, 16, 4096])
def test_tables_flag_pages_that_no_pool_has(pkv, page):
    """Page ids whose slots do not fit 32 bits, where they are read: in a row and in the free list."""
    last = 2**31 // page - 1    # the last that fits
    for bad in (-1, 2**31 // page, 2**31 - 1, -2**31):
        if bad == last or bad >= 2**31:
            continue
        table = np.array([[last, 7], [bad, 8]])
        half = max(page // 2, 1)
        # request 0: the rest of page `last`, then a bad page; request 1: the rest of a bad page (a page of
        # one token leaves no rest)
        old = half if page > 1 else 0
        seq, new = [page + 1, page], [page + 1 - old, page - old]
        if page == 1:
            table[:] = -5
        free = [last, bad, bad] if page == 1 else [bad]
        got, ws = build(pkv, page, seq, new, [0, 1], table, free, 0, sum(new))
        assert error(pkv, ws) == 0x100
        ok = new[0] - 1
        assert got[0][0, 1] == bad and got[4].tolist() == [len(free)]
        assert got[0][1, 0] == bad
        assert np.array_equal(got[2], [*range(old, page + 1), *range(old, page)])
        assert np.array_equal(got[1], [last * page + old + i for i in range(ok)] + [-1] * (1 + new[1]))


# ----------------------------------------------------------------------------------------
# the pool and its store


def random_pool(pkv, rng, pages, page, hkv, d, layout="separate", spread=2):
    pool = pkv.BlockPool.allocate(pages, page, hkv, d, layout=layout)
    out = []
    for codes_t, exps_t in ((pool.k, pool.k_exp), (pool.v, pool.v_exp)):
        codes = rng.integers(0, 256, (pages * page, hkv, d)).astype(np.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x30
        codes = np.where((codes & 0x7F) > 0x58, codes & 0xD7, codes)   # mostly of size 1
        exps = (127 + rng.integers(-spread, spread + 1, (pages, hkv))).astype(np.uint8)
        codes_t.copy_(dev(codes, np.uint8))
        exps_t.copy_(dev(exps, np.uint8))
        out += [codes, exps]
    return pool, out


def state(pool):
    return [host(t) for t in (pool.k, pool.k_exp, pool.v, pool.v_exp)]


def same_codes(got, want):
    nan = ((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)
    return np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want))


def check_store(pkv, pool, was, k, v, loc, page, ws):
    kt, kv = bf16(k)
    vt, vv = bf16(v)
    pkv.kv_store_block(pool, kt, vt, dev(loc), ws)
    with np.errstate(invalid="ignore"):
        ref.store(was[0], was[1], kv, loc, page)
        ref.store(was[2], was[3], vv, loc, page)
    got = state(pool)
    for g, w in zip(got, was):
        assert same_codes(g, w) if g.ndim == 3 else np.array_equal(g, w)


@pytest.mark.parametrize("hkv,d,page,layout", [(8, 128, 16, "separate"), (8, 128, 16, "interleaved"), (2, 64, 32, "separate"),
                                               (1, 64, 256, "separate"), (5, 128, 64, "interleaved"),
                                               (16, 64, 128, "separate"), (3, 64, 16, "interleaved")])
def test_store_appends_and_rescales(pkv, hkv, d, page, layout):
    """Prompts of ragged lengths, then single tokens, some far larger than what their page holds:
    codes and exponents equal the plain form's bit for bit, other rows stay."""
    rng = np.random.default_rng(hkv * d + page)
    lens = [1, page - 1, page, page + 1, 3 * page + 7, 2]
    pages = sum(-(-(n + 40) // page) for n in lens) + 3
    pool, was = random_pool(pkv, rng, pages, page, hkv, d, layout)
    ids, at, table = rng.permutation(pages), 0, []
    for n in lens:
        c = -(-(n + 40) // page)
        table.append(ids[at:at + c])
        at += c
    ws = words()
    done = [0] * len(lens)
    for step in range(6):
        add = lens if step == 0 else [1, 1, int(rng.integers(1, 6)), 1, 2, 1]
        loc = np.concatenate([[int(table[r][t // page]) * page + t % page for t in range(done[r], done[r] + n)]
                              for r, n in enumerate(add)]).astype(np.int64)
        done = [a + n for a, n in zip(done, add)]
        k, v = (rng.standard_normal((len(loc), hkv, d)) * 2.0 ** rng.integers(-3, 3 + 3 * step, (len(loc), hkv, 1))
                for _ in range(2))
        check_store(pkv, pool, was, k, v, loc, page, ws)
    assert error(pkv, ws) == 0


def test_store_extreme_values(pkv):
    """Zeros, subnormals, infinities, NaN and the format's ends."""
    rng = np.random.default_rng(1)
    page, hkv, d = 16, 4, 64
    pool, was = random_pool(pkv, rng, 12, page, hkv, d)
    rows = []
    for scale in (0.0, 1e-40, 2.0 ** -126, 1e-30, 1.0, 448.0, 3e38):
        x = rng.standard_normal((page, hkv, d))
        x = x / np.abs(x).max() * scale if scale else x * 0
        rows.append(x)
    x = np.concatenate(rows)
    k, v = x.copy(), x.copy()
    k[4 * page + 3, 1, 5], k[4 * page + 4, 1, 6], k[5 * page, 2, 7] = 448.0, 449.0, 450.0
    kb, vb = ref.bf16_bits(k), ref.bf16_bits(v)
    kb[4 * page + 5, 0, :4] = [0x7F80, 0xFF80, 0x7FC0, 0xFFC1]   # inf, -inf, NaN, -NaN
    vb[4 * page:5 * page, 3] = 0x7FC0                            # a page of nothing but NaN
    vb[5 * page:6 * page, 3] = 0x7F80
    loc = np.arange(len(x)) + 2 * page
    kt, vt = (torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16) for b in (kb, vb))
    ws = words()
    pkv.kv_store_block(pool, kt, vt, dev(loc), ws)
    ref.store(was[0], was[1], ref.bf16_values(kb), loc, page)
    ref.store(was[2], was[3], ref.bf16_values(vb), loc, page)
    for g, w in zip(state(pool), was):
        assert same_codes(g, w) if g.ndim == 3 else np.array_equal(g, w)
    assert error(pkv, ws) == 0


@pytest.mark.parametrize("n", [3, 5000])
def test_store_skips_padding_and_reports_bad_slots(pkv, n):
    rng = np.random.default_rng(n)
    page, hkv, d = 16, 2, 64
    pool, was = random_pool(pkv, rng, n // page + 6, page, hkv, d)
    loc = np.arange(n) + page
    loc[n - 1] = -1
    if n > 10:
        loc[40:60] = -1
    x = rng.standard_normal((n, hkv, d))
    ws = words()
    check_store(pkv, pool, was, x, x[::-1].copy(), loc, page, ws)
    assert error(pkv, ws) == 0
    for bad in (pool.k.shape[0], -2, 2**31 - 1):
        loc[1] = bad
        ws = words()
        check_store(pkv, pool, was, x, x, loc, page, ws)
        assert error(pkv, ws) == 0x100
    check_store(pkv, pool, was, x, x, loc, page, None)    # no workspace: skipped all the same


# ----------------------------------------------------------------------------------------
# attention


def paged_batch(pkv, rng, lens, page, pages, shared=0, extra_rows=2):
    """Batch over random distinct pages (the first `shared` blocks the same ones for all)."""
    blocks = [-(-n // page) for n in lens]
    ids, at = rng.permutation(pages), shared
    table = np.full((len(lens) + extra_rows, max(blocks + [1]) + 1), -5)
    rows = rng.permutation(len(table))[:len(lens)]
    for r, n in zip(rows, blocks):
        s = min(shared, n)
        table[r, :s] = ids[:s]
        table[r, s:n] = ids[at:at + n - s]
        at += max(n - s, 0)
    assert at <= pages
    return table, rows, pkv.Batch(dev(table), dev(rows), dev(lens), page)


def kill_tails(pool, was, table, rows, lens, page):
    """What lies behind a sequence's end in its last page becomes NaN."""
    for r, n in zip(rows, lens):
        if n % page:
            first = int(table[r, n // page]) * page
            for codes, t in ((was[0], pool.k), (was[2], pool.v)):
                codes[first + n % page:first + page] = 0x7F
                t[first + n % page:first + page] = 0x7F


def decode(pkv, pool, batch, q, hq, scale, ws=None):
    o = torch.full_like(q, float("nan"))
    ws = torch.zeros(pkv.decode_block_workspace(pool, hq) // 4, dtype=torch.int32, device="cuda") if ws is None else ws
    pkv.attn_decode_block(pool, batch, q, o, scale, ws)
    return o, ws


# weights are f16 (half a step is 2^-11); their sum takes them unrounded
DECODE_EPS = 2.0 ** -11


def check_decode(pkv, pool, was, table, rows, lens, page, hq, scale, q=None, seed=0, only=None):
    rng = np.random.default_rng(seed)
    b, d = len(lens), pool.k.shape[2]
    qt, qv = bf16(rng.standard_normal((b, hq, d)) * 2 if q is None else q)
    o, ws = decode(pkv, pool, pkv.Batch(dev(table), dev(rows), dev(lens), page), qt, hq, scale)
    got = values(o)
    for r in range(b) if only is None else only:
        k = ref.rows_of(was[0], was[1], table[rows[r]], lens[r], page)
        v = ref.rows_of(was[2], was[3], table[rows[r]], lens[r], page)
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        want, bound = ref.attend(qv[r:r + 1], k, v, scale, [lens[r] - 1], DECODE_EPS, v_exp=e)
        off = np.abs(got[r:r + 1] - want)
        assert np.all(off <= bound), (r, lens[r], float((off - bound).max()))
    return o, ws


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 300, 0, 1000, 1]


@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("hkv,d,page,layout", [(8, 128, 16, "separate"), (2, 64, 16, "interleaved"), (5, 128, 64, "interleaved"),
                                               (1, 128, 32, "separate"), (16, 64, 128, "separate"), (3, 64, 256, "separate")])
def test_decode(pkv, g, hkv, d, page, layout):
    rng = np.random.default_rng(g * 100 + hkv)
    pages = sum(-(-n // page) for n in LENS) + 2
    pool, was = random_pool(pkv, rng, pages, page, hkv, d, layout)
    table, rows, _ = paged_batch(pkv, rng, LENS, page, pages)
    kill_tails(pool, was, table, rows, LENS, page)
    o, ws = check_decode(pkv, pool, was, table, rows, LENS, page, hkv * g, d ** -0.5)
    assert error(pkv, ws) == 0
    assert torch.all(o[0] == 0) and torch.all(o[14] == 0)


@pytest.mark.parametrize("b,length", [(1, 1), (1, 100), (1, 70000), (3, 9001), (40, 2300), (700, 40), (4100, 3), (9000, 30)])
def test_decode_batches(pkv, b, length):
    """One long request split over the GPU, and more requests than warps."""
    rng = np.random.default_rng(b)
    page, hkv, g, d = 16, 4, 4, 64
    lens = np.maximum(1, length - rng.integers(0, max(length // 3, 1), b))
    pages = int((-(-lens // page)).sum())
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    table, rows, _ = paged_batch(pkv, rng, lens.tolist(), page, pages)
    kill_tails(pool, was, table, rows, lens, page)
    only = range(b) if b < 10 else rng.permutation(b)[:8]
    o, ws = check_decode(pkv, pool, was, table, rows, lens, page, hkv * g, d ** -0.5, only=only)
    assert error(pkv, ws) == 0 and torch.isfinite(o).all()


@pytest.mark.parametrize("b,g,hkv", [(16385, 8, 1), (65536, 8, 1), (65537, 8, 1), (40000, 4, 2), (131073, 4, 1)])
def test_decode_of_very_many_requests(pkv, b, g, hkv):
    """Batches around the most whose shared pages and tile sums are kept (65,536 streams), rows of the
    same table many times."""
    rng = np.random.default_rng(b)
    page, d, n = 16, 64, 500
    pool, was = random_pool(pkv, rng, 3 * n, page, hkv, d)
    table, rows = rng.permutation(3 * n).reshape(n, 3), rng.integers(0, n, b)
    lens = rng.integers(0, 49, b)
    lens[-1] = 48
    only = [0, b - 1, *rng.permutation(b)[:10]]
    q = np.zeros((b, hkv * g, d), np.float32)
    q[:] = rng.standard_normal((1, hkv * g, d))
    o, ws = check_decode(pkv, pool, was, table, rows, lens.tolist(), page, hkv * g, 0.1, q=q, only=only)
    assert error(pkv, ws) == 0 and torch.isfinite(o).all()
    assert torch.equal((o == 0).all(2).all(1).cpu(), torch.from_numpy(lens == 0))


@pytest.mark.parametrize("g,hkv,d,page", [(1, 8, 64, 16), (2, 3, 128, 32), (4, 8, 128, 16), (4, 2, 64, 64), (8, 4, 128, 16)])
@pytest.mark.parametrize("b", [2, 9, 70])
def test_decode_with_shared_pages(pkv, g, hkv, d, page, b):
    """Requests behind a common prefix (attended once for neighbours), some shorter than it, some
    empty, some that leave it early, some that meet again behind a difference, and a page of it
    that is outside the pool."""
    rng = np.random.default_rng(b + g)
    shared = 640 // page
    lens = rng.integers(640, 1500, b)
    lens[0] = 1400            # (the table is long enough to be looked through)
    if b > 2:
        lens[3], lens[4], lens[6] = 90, 0, 640
    pages = int((-(-lens // page)).sum()) + shared
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    table, rows, _ = paged_batch(pkv, rng, lens.tolist(), page, pages, shared)
    kill_tails(pool, was, table, rows, [n if n > 640 else 0 for n in lens], page)
    if b > 2:
        table[rows[8], 2] = table[rows[8], shared]     # another page in place of the third
        table[rows[1], 0] = table[rows[1], shared]     # the first differs, the rest is common
    only = range(b) if b < 10 else [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, b - 2, b - 1]
    o, ws = check_decode(pkv, pool, was, table, rows, lens.tolist(), page, hkv * g, d ** -0.5, only=only)
    assert error(pkv, ws) == 0
    table[rows, 1] = pages
    o, ws = check_decode(pkv, pool, was, table, rows, lens.tolist(), page, hkv * g, d ** -0.5, only=only)
    assert error(pkv, ws) == 0x100


@pytest.mark.parametrize("g,hkv,d", [(1, 2, 64), (4, 8, 128), (2, 1, 128), (8, 2, 64)])
@pytest.mark.parametrize("shared", [0, 64])
def test_decode_keeps_a_nan_to_its_request(pkv, g, hkv, d, shared):
    """NaN codes among one request's keys or values: its rows are NaN where the definition's are, and
    the requests attended beside it are not touched."""
    rng = np.random.default_rng(d)
    page, lens = 16, [1100, 1090, 1300, 70, 1200, 1024, 1111, 1040, 1500]
    pages = sum(-(-n // page) for n in lens) + shared
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    table, rows, _ = paged_batch(pkv, rng, lens, page, pages, shared)
    for r, codes, t in ((1, was[0], pool.k), (4, was[2], pool.v), (6, was[2], pool.v), (6, was[0], pool.k)):
        slot = int(table[rows[r], (lens[r] - 7) // page]) * page + (lens[r] - 7) % page
        codes[slot, 0, 3] = 0xFF
        t[slot, 0, 3] = 0xFF
    q, qv = bf16(rng.standard_normal((len(lens), hkv * g, d)))
    o, ws = decode(pkv, pool, pkv.Batch(dev(table), dev(rows), dev(lens), page), q, hkv * g, d ** -0.5)
    got = values(o)
    for r in range(len(lens)):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        with np.errstate(invalid="ignore"):
            want, bound = ref.attend(qv[r:r + 1], k, v, d ** -0.5, [lens[r] - 1], DECODE_EPS, v_exp=e)
        assert np.array_equal(np.isnan(got[r:r + 1]), np.isnan(want)), r
        fine = np.isfinite(want)
        assert np.all(np.abs(got[r:r + 1] - want)[fine] <= np.where(np.isfinite(bound), bound, np.inf)[fine]), r
    assert np.isfinite(got[[0, 2, 3, 5, 7, 8]]).all()


def test_extend_streams_keep_a_later_nan_from_earlier_tokens(pkv):
    """A NaN in a new token's row reaches the tokens that see it, not those before it."""
    rng = np.random.default_rng(0)
    page, hkv, g, d, lens, ext = 16, 2, 2, 64, [75, 40], [6, 3]
    pool, was = random_pool(pkv, rng, 9, page, hkv, d)
    table, rows, batch = paged_batch(pkv, rng, lens, page, 9)
    for codes, t in ((was[0], pool.k), (was[2], pool.v)):
        slot = int(table[rows[0], 72 // page]) * page + 72 % page     # token 3 of 6
        codes[slot] = 0x7F
        t[slot] = 0x7F
    qo = np.array([0, 6, 9])
    plan = pkv.plan_extend(lens, ext, qo, hkv * g, hkv, d)
    plan.info.offsets[18] = 1
    q, qv = bf16(rng.standard_normal((9, hkv * g, d)))
    o, ws = torch.empty_like(q), words(plan.info.workspace_bytes // 4 + 1)
    pkv.attn_extend_block(pool, batch, q, o, 0.1, plan, dev(plan.blob, np.uint8), ws)
    got = values(o)
    assert np.isnan(got[3:6]).all()
    for r, rows_ in ((0, range(3)), (1, range(6, 9))):
        k, v = (np.nan_to_num(ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page)) for j in (0, 2))
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        for i in rows_:
            want, bound = ref.attend(qv[i:i + 1], k, v, 0.1, [lens[r] - ext[r] + i - qo[r]], DECODE_EPS, v_exp=e)
            assert np.all(np.abs(got[i:i + 1] - want) <= bound)


@pytest.mark.parametrize("hkv,d", [(8, 128), (2, 64)])
def test_decode_exponents_far_apart(pkv, hkv, d):
    """Pages whose V exponents differ by up to 40 binades, K logits of several hundred, queries of
    very different sizes, and shared pages."""
    rng = np.random.default_rng(d)
    page, lens = 16, [400, 90, 650, 17]
    pool, was = random_pool(pkv, rng, 90, page, hkv, d, spread=20)
    pool.k_exp.copy_(dev(was[1] // 8 + 110, np.uint8))
    was[1] = host(pool.k_exp)
    table, rows, _ = paged_batch(pkv, rng, lens, page, 90, shared=1)
    q = rng.standard_normal((4, hkv * 4, d)) * 2.0 ** rng.integers(-60, 6, (4, hkv * 4, 1))
    q[0, 0] = 0.0
    q[1, 1, 1:] *= 2.0 ** -40     # one element far above the others
    o, ws = check_decode(pkv, pool, was, table, rows, lens, page, hkv * 4, d ** -0.5, q=q)
    assert error(pkv, ws) == 0


@pytest.mark.parametrize("byte", [10, 245])
def test_decode_at_the_ends_of_the_exponents(pkv, byte):
    """V pages all at the smallest or the largest exponent keep their values."""
    rng = np.random.default_rng(byte)
    page, hkv, d, lens = 16, 2, 64, [3000, 5]
    pool, was = random_pool(pkv, rng, 190, page, hkv, d)
    pool.v_exp.fill_(byte)
    was[3][:] = byte
    table, rows, _ = paged_batch(pkv, rng, lens, page, 190)
    check_decode(pkv, pool, was, table, rows, lens, page, 8, d ** -0.5)


def test_decode_reports_bad_pages_rows_and_lengths(pkv):
    rng = np.random.default_rng(3)
    page, hkv, d, lens = 16, 2, 64, [70, 40, 33, 50]
    pool, was = random_pool(pkv, rng, 30, page, hkv, d)
    table, rows, _ = paged_batch(pkv, rng, lens, page, 30)
    for bad in (30, -1, 2**31 - 1):
        t = table.copy()
        t[rows[1], 1] = bad      # its keys read as zero rows
        o, ws = check_decode(pkv, pool, was, t, rows, lens, page, 8, d ** -0.5)
        assert error(pkv, ws) == 0x100
    for change in ("row", "negative row", "length", "negative length"):
        rr, ll = rows.copy(), list(lens)
        if change.endswith("row"):
            rr[2] = len(table) if change == "row" else -1
        else:
            ll[2] = table.shape[1] * page + 1 if change == "length" else -4
        q, qv = bf16(rng.standard_normal((4, 8, d)))
        o, ws = decode(pkv, pool, pkv.Batch(dev(table), dev(rr), dev(ll), page), q, 8, 0.125)
        assert error(pkv, ws) == 0x400 and torch.all(o[2] == 0)
        # the other requests are attended all the same (the work is divided over the whole batch, so
        # a request's rounding may move with the others' lengths)
        for r in (0, 1, 3):
            k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
            e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
            want, bound = ref.attend(qv[r:r + 1], k, v, 0.125, [lens[r] - 1], DECODE_EPS, v_exp=e)
            assert np.all(np.abs(values(o[r:r + 1]) - want) <= bound)


@pytest.mark.parametrize("g,hkv,d", [(1, 64, 64), (4, 8, 128), (8, 1, 128)])
def test_decode_of_the_same_row_more_than_once(pkv, g, hkv, d):
    """Several queries of one row (samples of one prompt) at the same and at different lengths, and
    rows that fill their table to its last position."""
    rng = np.random.default_rng(g)
    page = 32
    lens = [40 * page, 40 * page, 1000, 40 * page, 999, 1, 40 * page]
    pool, was = random_pool(pkv, rng, 80, page, hkv, d)
    table = rng.permutation(80).reshape(2, 40)
    rows = [0, 0, 0, 1, 0, 1, 1]
    q = rng.standard_normal((len(lens), hkv * g, d))
    q[1] = q[0]
    o, ws = check_decode(pkv, pool, was, table, rows, lens, page, hkv * g, d ** -0.5, q=q)
    assert error(pkv, ws) == 0


def test_decode_is_the_same_every_time_and_on_any_stream(pkv):
    rng = np.random.default_rng(8)
    page, hkv, d, lens = 32, 8, 128, [5000, 1, 777, 2048]
    pool, was = random_pool(pkv, rng, 260, page, hkv, d)
    table, rows, batch = paged_batch(pkv, rng, lens, page, 260)
    q, _ = bf16(rng.standard_normal((4, 32, d)))
    first, ws = decode(pkv, pool, batch, q, 32, 0.1)
    for _ in range(3):
        assert torch.equal(decode(pkv, pool, batch, q, 32, 0.1, ws)[0], first)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for _ in range(2)]
    spaces = [torch.zeros_like(ws) for _ in range(2)]
    for _ in range(4):            # two calls at once, each with its own workspace
        for s, o, w in zip((side, other), outs, spaces):
            pkv.attn_decode_block(pool, batch, q, o, 0.1, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


def test_decode_past_32_bit_offsets(pkv):
    """Pages behind the first 4 GB of codes."""
    rng = np.random.default_rng(9)
    page, hkv, d = 64, 8, 128
    pages = (9 << 30) // 2 // (page * hkv * d)      # 4.5 GB of K, as much V
    pool = pkv.BlockPool.allocate(pages, page, hkv, d)
    lens = [200, 64]
    ids = np.array([pages - 1, 0, pages - 3, pages - 7, pages // 2])
    table = np.zeros((2, 4), np.int64)
    table[0], table[1, 0] = ids[:4], ids[4]
    small, was = random_pool(pkv, rng, 5, page, hkv, d)
    for i, at in enumerate(ids):
        for a, b in ((pool.k, small.k), (pool.v, small.v)):
            a[at * page:(at + 1) * page] = b[i * page:(i + 1) * page]
        pool.k_exp[at], pool.v_exp[at] = small.k_exp[i], small.v_exp[i]
    q, qv = bf16(rng.standard_normal((2, 32, d)))
    o, ws = decode(pkv, pool, pkv.Batch(dev(table), dev([0, 1]), dev(lens), page), q, 32, 0.1)
    local = np.array([[0, 1, 2, 3], [4, 0, 0, 0]])
    for r in range(2):
        k, v = (ref.rows_of(was[j], was[j + 1], local[r], lens[r], page) for j in (0, 2))
        e = ref.exponents_of(was[3], local[r], lens[r], page)
        want, bound = ref.attend(qv[r:r + 1], k, v, 0.1, [lens[r] - 1], DECODE_EPS, v_exp=e)
        assert np.all(np.abs(values(o[r:r + 1]) - want) <= bound)
    # and a store there
    x = rng.standard_normal((3, hkv, d))
    kt, kv = bf16(x)
    loc = (pages - 1) * page + 5 + np.arange(3)
    pkv.kv_store_block(pool, kt, kt, dev(loc), ws)
    ref.store(was[0], was[1], kv, 5 + np.arange(3), page)
    assert same_codes(host(pool.k[(pages - 1) * page:]), was[0][:page])
    assert error(pkv, ws) == 0


# the extend kernel's weights: their exponent is rounded to bf16 (2^-9 of it), the exponential and
# the lazily rescaled product to bf16 (2^-9 each, 8 bits of significand): 2^-8 and 2^-9 |ln w|; the
# sum takes the rounded weights, which doubles neither
EXTEND_EPS, EXTEND_LOG_EPS = 2.0 ** -7, 2.0 ** -8


@pytest.mark.parametrize("hkv,g,d,page,shared,old,new", [
    (8, 4, 128, 16, 0, [0, 50, 333], [40, 1, 17]), (8, 4, 128, 16, 256, [256, 300, 260, 256], [30, 5, 64, 8]),
    (2, 4, 64, 32, 0, [0, 31], [1, 2]), (5, 2, 128, 64, 0, [100], [190]), (16, 1, 64, 128, 128, [128, 200], [33, 3]),
    (1, 8, 128, 16, 0, [1000, 7], [3, 100]), (3, 8, 64, 256, 0, [5, 255], [251, 2])])
@pytest.mark.parametrize("layout", ["separate", "interleaved"])
@pytest.mark.parametrize("streams", [0, 1])
def test_extend(pkv, hkv, g, d, page, shared, old, new, layout, streams):
    """Both ways an extend call has (the plan chooses one): gathered rows on the tensor cores, and
    few tokens at a time over the pages."""
    rng = np.random.default_rng(d + page)
    lens = [a + b for a, b in zip(old, new)]
    pages = sum(-(-n // page) for n in lens) + 1
    pool, was = random_pool(pkv, rng, pages, page, hkv, d, layout)
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages, shared // page)
    kill_tails(pool, was, table, rows, lens, page)
    qo = np.concatenate([[0], np.cumsum(new)])
    cascade = None
    if shared:
        cascade = pkv.Cascade(*(np.asarray(a, np.int32) for a in ([0], [0], [shared], [0, len(old)], range(len(old)))))
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d, cascade)
    plan.info.offsets[18] = streams
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    o = torch.full_like(qt, float("nan"))
    ws = words((plan.info.workspace_bytes + 3) // 4)
    scale = 0.5 * d ** -0.5
    pkv.attn_extend_block(pool, batch, qt, o, scale, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0
    got = values(o)
    for r in range(len(old)):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        at = np.arange(old[r], lens[r])
        if streams:
            e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
            want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, scale, at, DECODE_EPS, v_exp=e)
        else:
            want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, scale, at, EXTEND_EPS, EXTEND_LOG_EPS)
        assert np.all(np.abs(got[qo[r]:qo[r + 1]] - want) <= bound), r


def test_extend_chooses_by_the_tokens(pkv):
    """A few tokens after a long context are streams; many are gathered."""
    few = pkv.plan_extend([9000] * 4, [5] * 4, np.arange(5) * 5, 32, 8, 128)
    many = pkv.plan_extend([2000] * 64, [200] * 64, np.arange(65) * 200, 32, 8, 128)
    assert few.info.offsets[18] == 1 and many.info.offsets[18] == 0


@pytest.mark.parametrize("hkv,g,d,page", [(2, 4, 128, 16), (3, 8, 64, 32), (8, 1, 128, 64)])
def test_gathered_extend_keeps_a_nan_to_the_rows_that_see_it(pkv, hkv, g, d, page):
    """Requests whose gathered rows meet in a 128-key tile, later tokens of the same request, and a
    prefix that two share: a NaN code of K or V reaches what sees it, element by element."""
    rng = np.random.default_rng(hkv + d)
    old, new = [30, 0, 260, 256, 7], [20, 40, 33, 50, 1]
    lens = [a + b for a, b in zip(old, new)]
    pages = sum(-(-n // page) for n in lens) + 1
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages)
    qo = np.concatenate([[0], np.cumsum(new)])
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d)
    plan.info.offsets[18] = 0
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    ws = words((plan.info.workspace_bytes + 3) // 4)
    blob = dev(plan.blob, np.uint8)

    def slot(r, j):
        return int(table[rows[r], j // page]) * page + j % page
    # (tensor, request, position, head, element): in order of how many rows see it
    plants = [None, (2, 1, 0, 0, 3), (2, 0, 45, hkv - 1, d - 1), (0, 3, 280, 0, 0), (2, 2, 0, hkv - 1, 17), (2, 4, 7, 0, 1), None]
    last = None
    for plant in plants:
        if last is not None:   # what was there before the last one
            (pool.k, None, pool.v)[last[0]][last[1]] = int(last[2])
            was[last[0]][last[1]] = last[2]
        last = None
        if plant is not None:
            t, r, j, h, i = plant
            at = (slot(r, j), h, i)
            last = (t, at, was[t][at])
            (pool.k, None, pool.v)[t][at] = 0xFF
            was[t][at] = 0xFF
        o = torch.full_like(qt, 5.0)
        pkv.attn_extend_block(pool, batch, qt, o, 0.1, plan, blob, ws)
        assert error(pkv, ws) == 0 and int(ws[20]) == 0
        got = values(o)
        for r in range(len(old)):
            k, v = (ref.rows_of(was[x], was[x + 1], table[rows[r]], lens[r], page) for x in (0, 2))
            with np.errstate(invalid="ignore"):
                want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, 0.1, np.arange(old[r], lens[r]), EXTEND_EPS, EXTEND_LOG_EPS)
            mine = got[qo[r]:qo[r + 1]]
            assert np.array_equal(np.isnan(mine), np.isnan(want)), (plant, r)
            assert np.all((np.abs(mine - want) <= bound) | np.isnan(want)), (plant, r)


@pytest.mark.parametrize("b,g,hkv", [(512, 4, 2), (513, 8, 2), (1025, 2, 3), (3000, 4, 1)])
def test_extend_streams_of_many_requests(pkv, b, g, hkv):
    """Around the batch from which the tiles before each request are written down (512)."""
    rng = np.random.default_rng(b)
    page, d, n = 16, 64, 400
    new, old = rng.integers(1, 5, b), rng.integers(0, 60, b)
    old[-1], new[-1] = 59, 4
    lens = old + new
    pool, was = random_pool(pkv, rng, 4 * n, page, hkv, d)
    table, rows = rng.permutation(4 * n).reshape(n, 4), rng.integers(0, n, b)
    qo = np.concatenate([[0], np.cumsum(new)])
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d)
    plan.info.offsets[18] = 1
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    o, ws = torch.full_like(qt, float("nan")), words((plan.info.workspace_bytes + 3) // 4)
    batch = pkv.Batch(dev(table), dev(rows), dev(lens), page)
    pkv.attn_extend_block(pool, batch, qt, o, 0.1, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0 and torch.isfinite(o).all()
    got = values(o)
    for r in [0, 1, 510, 511, b - 2, b - 1, *rng.permutation(b)[:10]]:
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, 0.1, np.arange(old[r], lens[r]), DECODE_EPS, v_exp=e)
        assert np.all(np.abs(got[qo[r]:qo[r + 1]] - want) <= bound), r


@pytest.mark.parametrize("hkv,g,d", [(1, 1, 64), (8, 4, 128), (3, 8, 64), (16, 2, 128)])
@pytest.mark.parametrize("old,new", [([0], [1]), ([1], [1]), ([0, 3], [5, 1]), ([15] * 7, [1] * 7)])
def test_extend_of_short_contexts(pkv, hkv, g, d, old, new):
    """A few keys in all, by the way that the plan chooses in the workspace that it asks for."""
    rng = np.random.default_rng(hkv + len(old))
    page, lens = 16, [a + b for a, b in zip(old, new)]
    pool, was = random_pool(pkv, rng, 12, page, hkv, d)
    table, rows, batch = paged_batch(pkv, rng, lens, page, 12)
    qo = np.concatenate([[0], np.cumsum(new)])
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d)
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    o = torch.full_like(qt, float("nan"))
    ws = words((plan.info.workspace_bytes + 3) // 4)
    pkv.attn_extend_block(pool, batch, qt, o, 0.1, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0
    got = values(o)
    for r in range(len(old)):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, 0.1, np.arange(old[r], lens[r]), EXTEND_EPS, EXTEND_LOG_EPS)
        if plan.info.offsets[18]:
            e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
            want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, 0.1, np.arange(old[r], lens[r]), DECODE_EPS, v_exp=e)
        assert np.all(np.abs(got[qo[r]:qo[r + 1]] - want) <= bound), r


@pytest.mark.parametrize("b,old,new", [(2, 20000, 3), (60, 700, 9), (300, 1, 2)])
def test_extend_streams_over_many_ranges(pkv, b, old, new):
    """Streams cut into many ranges, and more streams than ranges."""
    rng = np.random.default_rng(b)
    page, hkv, g, d = 16, 8, 4, 128
    old = np.maximum(old - rng.integers(0, old // 3 + 1, b), 0)
    ext = rng.integers(1, new + 1, b)
    lens = (old + ext).tolist()
    pages = sum(-(-n // page) for n in lens)
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages)
    kill_tails(pool, was, table, rows, lens, page)
    qo = np.concatenate([[0], np.cumsum(ext)])
    plan = pkv.plan_extend(lens, ext, qo, hkv * g, hkv, d)
    plan.info.offsets[18] = 1
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    o = torch.full_like(qt, float("nan"))
    ws = words((plan.info.workspace_bytes + 3) // 4)
    pkv.attn_extend_block(pool, batch, qt, o, d ** -0.5, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0 and torch.isfinite(o).all()
    got = values(o)
    for r in (range(b) if b < 5 else rng.permutation(b)[:6]):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, d ** -0.5, np.arange(old[r], lens[r]), DECODE_EPS, v_exp=e)
        assert np.all(np.abs(got[qo[r]:qo[r + 1]] - want) <= bound), r

@pytest.mark.parametrize("what", ["decode", "streams"])
def test_a_short_wait_limit_gives_up_and_the_next_call_is_right(pkv, what):
    """Only the limit is cut: waits for tiles that are on their way give up, every copy lands, the
    error word says so, and the same call with the default limit is right."""
    rng = np.random.default_rng(12)
    page, hkv, d, lens = 16, 8, 128, [900, 300, 200000, 17]   # 410 MB of codes: tiles have to be waited for
    pages = sum(-(-n // page) for n in lens)
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages)
    ext = [1] * 4 if what == "decode" else [3, 2, 5, 1]
    qo = np.concatenate([[0], np.cumsum(ext)])
    plan = pkv.plan_extend(lens, ext, qo, hkv * 4, hkv, d)
    plan.info.offsets[18] = 1
    q, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * 4, d)))
    o = torch.zeros_like(q)
    ws = words(max(pkv.decode_block_workspace(pool, hkv * 4), plan.info.workspace_bytes) // 4 + 1)
    blob = dev(plan.blob, np.uint8)

    def call():
        if what == "decode":
            pkv.attn_decode_block(pool, batch, q, o, 0.1, ws)
        else:
            pkv.attn_extend_block(pool, batch, q, o, 0.1, plan, blob, ws)
    try:
        pkv.set_wait_limit_ns(1)
        for _ in range(3):
            call()
        assert error(pkv, ws) & 0x200
    finally:
        pkv.set_wait_limit_ns(0)
    ws.zero_()
    call()
    assert error(pkv, ws) == 0 and torch.isfinite(o).all()
    for r in (0, 1, 3):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, 0.1, np.arange(lens[r] - ext[r], lens[r]), DECODE_EPS, v_exp=e)
        assert np.all(np.abs(values(o[qo[r]:qo[r + 1]]) - want) <= bound)


def test_python_calls_check_their_tensors(pkv):
    rng = np.random.default_rng(0)
    pool, _ = random_pool(pkv, rng, 4, 16, 2, 64)
    table, rows, batch = paged_batch(pkv, rng, [20], 16, 4)
    q, _ = bf16(rng.standard_normal((1, 8, 64)))
    o, ws = decode(pkv, pool, batch, q, 8, 0.1)
    bad = [dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.cpu()), dict(o=o[:, :4]), dict(o=o.half()),
           dict(q=torch.cat([q, q])), dict(batch=pkv.Batch(dev(table, np.int64), dev(rows), dev([20]), 16)),
           dict(batch=pkv.Batch(dev(table), dev(rows), dev([20, 20]), 16)),
           dict(batch=pkv.Batch(dev(table).T, dev(rows), dev([20]), 16)), dict(ws=ws.cpu())]
    for kw in bad:
        a = {**dict(pool=pool, batch=batch, q=q, o=o, sm_scale=0.1, ws=ws), **kw}
        with pytest.raises(ValueError):
            pkv.attn_decode_block(a["pool"], a["batch"], a["q"], a["o"], a["sm_scale"], a["ws"])
    with pytest.raises(pkv.PkvError):
        pkv.attn_decode_block(pool, batch, q, o, 0.1, ws[:8])
    x, _ = bf16(rng.standard_normal((3, 2, 64)))
    for args in ((x.float(), x, words(3)), (x, x[:2], words(3)), (x, x, words(3).long()), (x, x, words(2)),
                 (x.transpose(0, 1).contiguous().transpose(0, 1), x, words(3))):
        with pytest.raises(ValueError):
            pkv.kv_store_block(pool, *args)


# ----------------------------------------------------------------------------------------
# together


def test_a_serving_run_in_a_graph(pkv):
    """Prompts admitted through the device-built tables, stored and extended; then decode steps
    replayed from one captured graph (tables, store, attention) with a request that leaves, one
    that is padding from the start, and pages taken from one free list.  Every output is checked
    against attention over the values the pages stand for, and those against the inputs."""
    rng = np.random.default_rng(42)
    page, hkv, g, d, scale = 16, 4, 4, 64, 0.125
    hq, b, most = hkv * g, 5, 200
    prompts = np.array([37, 16, 1, 64, 0])
    pool = pkv.BlockPool.allocate(60, page, hkv, d)
    free, head = dev(rng.permutation(60)), words(1)
    table = torch.full((8, most // page + 1), -1, dtype=torch.int32, device="cuda")
    rows, ws = dev([6, 0, 3, 2, 5]), words()
    k_all, v_all = (ref.bf16_values(ref.bf16_bits(rng.standard_normal((b, most, hkv, d)) * 2.0 ** (np.arange(most) / 16)[:, None, None]))
                    for _ in range(2))

    def new_rows(x, spans):
        return bf16(np.concatenate([x[r, a:z] for r, (a, z) in enumerate(spans)] or [np.zeros((0, hkv, d))]))[0]

    def check(outs, q, lens, at):
        """outs, q [n, hq, d]; at: (request, position) of each row."""
        t = host(table)
        codes = state(pool)
        kv = {}
        for r in set(r for r, _ in at):
            kv[r] = [ref.rows_of(codes[j], codes[j + 1], t[int(rows[r])], lens[r], page) for j in (0, 2)]
            for x, y in zip(kv[r], (k_all, v_all)):
                # a code is off by half a step, 2^-4 of its value, or half the smallest step of its page
                # (2^-10 of 2^e, e the exponent that the page's largest value needs); rescaled rows by as much again
                top = np.abs(y[r, :lens[r]]).max()
                assert np.all(np.abs(x - y[r, :lens[r]]) <= 2.0 ** -4 * np.abs(y[r, :lens[r]]) + 2 * 2.0 ** -10 * top / 224)
        for i, (r, p) in enumerate(at):
            want, bound = ref.attend(q[i:i + 1], *kv[r], scale, [p], EXTEND_EPS, EXTEND_LOG_EPS)
            assert np.all(np.abs(values(outs[i:i + 1]) - want) <= bound), (r, p)

    # admission
    n = int(prompts.sum())
    loc, pos, qo = words(n), words(n), words(b + 1)
    pkv.build_block_tables(table, rows, dev(prompts), dev(prompts), free, head, head, loc, pos, qo, page, ws)
    spans = [(0, int(x)) for x in prompts]
    pkv.kv_store_block(pool, new_rows(k_all, spans), new_rows(v_all, spans), loc, ws)
    live = [0, 1, 2, 3]
    q, qv = bf16(rng.standard_normal((n, hq, d)))
    plan = pkv.plan_extend(prompts[live], prompts[live], host(qo)[:5], hq, hkv, d)
    o = torch.empty_like(q)
    big = words((plan.info.workspace_bytes + 3) // 4)
    pkv.attn_extend_block(pool, pkv.Batch(table, rows[:4].contiguous(), dev(prompts[live]), page), q, o, scale, plan,
                          dev(plan.blob, np.uint8), big)
    assert error(pkv, big) == 0 and error(pkv, ws) == 0
    check(o, qv, prompts, [(r, t) for r in live for t in range(prompts[r])])

    # decode steps from a graph
    seq, new = dev(prompts), words(b)
    loc, pos, qo = words(b), words(b), words(b + 1)
    k_new, v_new = (torch.zeros((b, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((b, hq, d), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    space = torch.zeros(pkv.decode_block_workspace(pool, hq) // 4, dtype=torch.int32, device="cuda")

    def step():
        pkv.build_block_tables(table, rows, seq, new, free, head, head, loc, pos, qo, page, ws)
        pkv.kv_store_block(pool, k_new, v_new, loc, ws)
        pkv.attn_decode_block(pool, pkv.Batch(table, rows, seq, page), q, o, scale, space)

    step()   # nothing new: tables, pool and head stay (and the kernels are loaded before capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = prompts.copy()
    for i in range(40):
        on = np.array([1, 1, 1, i < 20, 0])
        lens = lens + on
        seq.copy_(dev(np.where(on, lens, 0)))
        new.copy_(dev(on))
        at = [r for r in range(b) if on[r]]
        fill = lambda x: new_rows(x, [(lens[r] - 1, lens[r]) if on[r] else (0, 0) for r in range(b)])  # noqa: E731
        k_new[:len(at)], v_new[:len(at)] = fill(k_all), fill(v_all)
        qt, qv = bf16(rng.standard_normal((b, hq, d)))
        q.copy_(qt)
        graph.replay()
        torch.cuda.synchronize()
        assert error(pkv, ws) == 0 and error(pkv, space) == 0
        for r in range(b):
            if not on[r]:
                assert torch.all(o[r] == 0)
        if i % 8 == 7 or i in (0, 20):
            check(o[at], qv[at], lens, [(r, int(lens[r]) - 1) for r in at])
    pages = sum(-(-int(n) // page) for n in lens)
    assert int(head) == pages and len(set(host(table)[host(table) >= 0].tolist())) == pages


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("captured", [False, True])
def test_tables_feed_the_calls_over_a_plain_pool(pkv, page, captured):
    """The step's tables and slots are any pool's: steps of tables, kv_store and attn_extend over a bf16
    pool, one behind the other with nothing in between that waits, also in one graph."""
    rng = np.random.default_rng(page)
    b, hkv, d, steps, grow = 120, 2, 64, 12, 3
    stride = -(-steps * grow // page)
    slots = b * stride * page
    pool = pkv.Pool(*(torch.zeros((slots, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    free, head = dev(rng.permutation(b * stride)), dev([0])
    table, rows, new = torch.full((b, stride), -1, dtype=torch.int32, device="cuda"), dev(rng.permutation(b)), dev([grow] * b)
    loc, pos, qo, ws = words(b * grow), words(b * grow), words(b + 1), words()
    qo_host = np.arange(b + 1) * grow
    xs, outs, calls = [], [], []
    for s in range(steps):
        lens = [(s + 1) * grow] * b
        plan = pkv.plan_extend(lens, [grow] * b, qo_host, hkv * 4, hkv, d)
        x = [bf16(rng.standard_normal((b * grow, n, d)))[0] for n in (hkv, hkv, hkv * 4)]
        calls.append((dev(lens), plan, dev(plan.blob, np.uint8), words((plan.info.workspace_bytes + 3) // 4)))
        xs.append(x)
        outs.append(torch.zeros_like(x[2]))
    torch.cuda.synchronize()

    def run():
        for (k, v, q), o, (lens, plan, blob, space) in zip(xs, outs, calls):
            pkv.build_block_tables(table, rows, lens, new, free, head, head, loc, pos, qo, page, ws)
            pkv.kv_store(pool, k, v, loc, ws)
            pkv.attn_extend(pool, pkv.Batch(table, rows, lens, page), q, o, 0.2, plan, blob, space)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
    else:
        run()
    assert error(pkv, ws) == 0 and int(head[0]) == b * stride
    # what request r should hold is what its steps gave it, in order
    k, v = (np.concatenate([values(x[i]).reshape(b, grow, hkv, d) for x in xs], 1) for i in (0, 1))
    t = host(table)[host(rows)]
    at = np.arange(steps * grow)
    assert np.array_equal(values(pool.k)[t[:, at // page] * page + at % page], k)
    assert np.array_equal(values(pool.v)[t[:, at // page] * page + at % page], v)
    for s in (0, 5, steps - 1):
        assert error(pkv, calls[s][3]) == 0
        q, got = values(xs[s][2]).reshape(b, grow, -1, d), values(outs[s]).reshape(b, grow, -1, d)
        for r in range(0, b, 17):
            n = (s + 1) * grow
            want, bound = ref.attend(q[r], k[r, :n], v[r, :n], 0.2, np.arange(n - grow, n), EXTEND_EPS, EXTEND_LOG_EPS)
            assert np.all(np.abs(got[r] - want) <= bound)
