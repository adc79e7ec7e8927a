"""Edges of the block-scaled cache's calls: batches at a launch limit, workspaces with old contents, exponents
and logits at their ends, pools at any 16-byte address, large batches of few-head groups."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import block_reference as ref
from test_gpu_block_cache import (DECODE_EPS, EXTEND_EPS, EXTEND_LOG_EPS, bf16, check_decode, check_store, dev,
                                  error, host, paged_batch, random_pool, table_inputs, values, words)

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import prefix_shared_kv_token_gb300 as m
    return m


# ----------------------------------------------------------------------------------------
# tables

RISING = """
import numpy as np
import block_reference as ref
import prefix_shared_kv_token_gb300 as pkv
from test_gpu_block_cache import build, error, table_inputs
for b in (6111, 6112, 6143, 6144, 16384, 7000):
    seq, new, rows, table, free = table_inputs(np.random.default_rng(b), b, 16, 100, 2)
    cap = int(new.sum()) + 5
    got, ws = build(pkv, 16, seq, new, rows, table, free, 0, cap)
    assert error(pkv, ws) == 0, b
    for g, w in zip(got, ref.tables(table, rows, seq, new, free, 0, 16, cap)):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), b
print("done")
"""


def test_tables_of_rising_batches_in_a_process_of_their_own():
    """8 bytes a request and one more in shared memory, and 256 bytes beside them: 6,112 requests are
    the first to pass 48 KB with both, 6,144 without those."""
    path = os.pathsep.join([HERE, os.path.dirname(HERE), os.environ.get("PYTHONPATH", "")])
    run = subprocess.run([sys.executable, "-c", RISING], env={**os.environ, "PYTHONPATH": path}, capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.strip() == "done", run.stderr[-2000:]


def test_tables_of_different_batches_from_two_threads(pkv):
    """Two host threads, each with its own stream and workspace: a small batch's launch takes nothing
    from a large one's."""
    def inputs(b):
        seq, new, rows, table, free = table_inputs(np.random.default_rng(b), b, 16, 100, 2)
        cap = int(new.sum())
        out = [words(cap), words(cap), words(b + 1), words(1)]
        want = ref.tables(table, rows, seq, new, free, 0, 16, cap)
        return [dev(x) for x in (table, rows, seq, new, free, [0])], out, words(), torch.cuda.Stream(), want
    sets, failed = [inputs(16384), inputs(7000)], []
    torch.cuda.synchronize()

    def calls(args, out, ws, stream, want):
        try:
            table, rows, seq, new, free, head = args
            loc, pos, qo, head_out = out
            for _ in range(400):
                pkv.build_block_tables(table, rows, seq, new, free, head, head_out, loc, pos, qo, 16, ws, stream=stream)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))
    threads = [threading.Thread(target=calls, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (table, *_), (loc, pos, qo, head), ws, _, want in sets:
        assert error(pkv, ws) == 0
        for g, w in zip((table, loc, pos, qo, head), want):
            assert np.array_equal(host(g).reshape(-1), np.asarray(w).reshape(-1))


# ----------------------------------------------------------------------------------------
# gathered extend: what a refused request leaves in the workspace

OLD_NAN = 0x7FC07FC0    # two bf16 NaN


def bad_neighbours(rng, pages_a_row=40):
    """(lengths, new tokens, their offsets, table, rows): requests of which several meet in a 128-key tile."""
    lens, new = [30, 40, 300, 20], [10, 12, 40, 20]
    return lens, new, np.concatenate([[0], np.cumsum(new)]), rng.permutation(5 * pages_a_row).reshape(5, pages_a_row), rng.permutation(5)[:4]


@pytest.mark.parametrize("change", ["row", "negative row", "position"])
@pytest.mark.parametrize("bad", [1, 3])
def test_gathered_extend_beside_a_refused_request(pkv, change, bad):
    """A request whose row or positions are out of range gets an error; the keys it would have gathered are
    zeros and not what the workspace held, which a neighbour in the same tile would see as NaN."""
    rng = np.random.default_rng(bad)
    page, hkv, g, d = 16, 2, 4, 64
    lens, new, qo, table, rows = bad_neighbours(rng)
    pool, was = random_pool(pkv, rng, table.size, page, hkv, d)
    rr, t = rows.copy(), table
    if change == "position":
        t = table[:, :2] if bad == 1 else table[:, :1]    # too short for request 1, and for 2; or for all but the last
        lens = [30, 40, 28, 20] if bad == 1 else [10, 12, 16, 20]
        new = [10, 12, 8, 20] if bad == 1 else [5, 6, 8, 20]
        qo = np.concatenate([[0], np.cumsum(new)])
    else:
        rr[bad] = len(table) if change == "row" else -1
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d)
    plan.info.offsets[18] = 0
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    o = torch.full_like(qt, float("nan"))
    ws = words((plan.info.workspace_bytes + 3) // 4)
    ws[64:] = OLD_NAN
    pkv.attn_extend_block(pool, pkv.Batch(dev(t), dev(rr), dev(lens), page), qt, o, 0.1, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0x400
    got = values(o)
    assert np.isfinite(got).all()
    for r in range(4):
        if r == bad:
            continue
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, 0.1, np.arange(lens[r] - new[r], lens[r]), EXTEND_EPS, EXTEND_LOG_EPS)
        assert np.all(np.abs(got[qo[r]:qo[r + 1]] - want) <= bound), r


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 16])
def test_extend_of_a_plain_pool_beside_a_refused_request(pkv, fp8, page):
    """The same over the pools without block scales."""
    rng = np.random.default_rng(page)
    hkv, g, d = 2, 4, 64
    lens, new, qo, table, rows = bad_neighbours(rng, 320 if page == 1 else 40)
    x = [rng.standard_normal((table.size * page, hkv, d)) for _ in range(2)]
    t = [bf16(a)[0] for a in x]
    if fp8:
        t = [a.to(torch.float8_e4m3fn) for a in t]
        pool = pkv.Pool(*(a.view(torch.uint8) for a in t), "fp8_e4m3")
    else:
        pool = pkv.Pool(*t)
    kv = [values(a) for a in t]
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d)
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), hkv * g, d)))
    o = torch.full_like(qt, float("nan"))
    ws = words((plan.info.workspace_bytes + 3) // 4)
    ws[64:] = OLD_NAN
    rr = rows.copy()
    rr[1] = len(table)
    pkv.attn_extend(pool, pkv.Batch(dev(table), dev(rr), dev(lens), page), qt, o, 0.1, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0x400
    got = values(o)
    assert np.isfinite(got).all()
    for r in (0, 2, 3):
        at = np.arange(lens[r])
        slots = table[rows[r]][at // page] * page + at % page
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], kv[0][slots], kv[1][slots], 0.1, np.arange(lens[r] - new[r], lens[r]),
                                 EXTEND_EPS, EXTEND_LOG_EPS)
        assert np.all(np.abs(got[qo[r]:qo[r + 1]] - want) <= bound), r


# ----------------------------------------------------------------------------------------
# a pool's address


@pytest.mark.parametrize("g,d,layer", [(4, 64, 1), (8, 64, 2), (1, 128, 1)])
def test_a_layer_of_a_cache_of_many(pkv, g, d, layer):
    """K and V are a layer's view of [slots, layers, 1, d]: rows 16-byte aligned, one behind the other at
    the stride of all layers.  Store, decode and both ways of extend."""
    rng = np.random.default_rng(d + g)
    page, layers, pages = 16, 3, 40
    was_pool, was = random_pool(pkv, rng, pages, page, 1, d)
    k, v = (torch.full((pages * page, layers, 1, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    k[:, layer], v[:, layer] = was_pool.k, was_pool.v
    pool = pkv.BlockPool(k[:, layer], v[:, layer], was_pool.k_exp, was_pool.v_exp, page)
    assert d == 128 or layer % 2 == 0 or pool.k.data_ptr() % 128 == 64
    lens, new = [200, 33, 300], [5, 33, 2]
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages)
    loc = np.concatenate([[int(table[rows[r], t // page]) * page + t % page for t in range(n - e, n)]
                          for r, (n, e) in enumerate(zip(lens, new))])
    x = [rng.standard_normal((len(loc), 1, d)) for _ in range(2)]
    ws = words()
    check_store(pkv, pool, was, *x, loc, page, ws)
    assert error(pkv, ws) == 0
    o, ws = check_decode(pkv, pool, was, table, rows, lens, page, g, d ** -0.5)
    assert error(pkv, ws) == 0
    qo = np.concatenate([[0], np.cumsum(new)])
    qt, qv = bf16(rng.standard_normal((int(qo[-1]), g, d)))
    for streams in (0, 1):
        plan = pkv.plan_extend(lens, new, qo, g, 1, d)
        plan.info.offsets[18] = streams
        o, ws = torch.full_like(qt, float("nan")), words((plan.info.workspace_bytes + 3) // 4)
        pkv.attn_extend_block(pool, batch, qt, o, 0.1, plan, dev(plan.blob, np.uint8), ws)
        assert error(pkv, ws) == 0
        for r in range(3):
            kk, vv = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
            e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
            at = np.arange(lens[r] - new[r], lens[r])
            want, bound = ref.attend(qv[qo[r]:qo[r + 1]], kk, vv, 0.1, at, *((DECODE_EPS, 0.0, e) if streams else
                                                                             (EXTEND_EPS, EXTEND_LOG_EPS)))
            assert np.all(np.abs(values(o[qo[r]:qo[r + 1]]) - want) <= bound), (streams, r)
    for t in (k, v):    # the other layers are as they were
        assert torch.all(t[:, [i for i in range(layers) if i != layer]] == 0x7F)


# ----------------------------------------------------------------------------------------
# exponents and logits at their ends


def steep_keys(pool, was, rng, page, top):
    """K rows whose logits (for queries of whole numbers over d) are up to `top` apart in log2 units, page
    by page; V pages at the ends of the exponents and between."""
    pages, hkv = was[1].shape
    level = rng.choice([0.0, 0.03125, 0.25, 0.75, 1.0], (pages * page, hkv, 1)) * np.where(rng.random((pages * page, hkv, 1)) < 0.2, 1, 0)
    codes = np.broadcast_to(ref.e4m3_encode(level), was[0].shape).astype(np.uint8).copy()
    was[0][:], was[1][:] = codes, 127
    was[3][:] = rng.choice([10, 60, 127, 190, 245], (pages, hkv))
    for t, w in zip((pool.k, pool.k_exp, pool.v_exp), (was[0], was[1], was[3])):
        t.copy_(dev(w, np.uint8))
    return top * np.log(2.0)


@pytest.mark.parametrize("g,hkv,d", [(1, 3, 64), (2, 8, 128), (4, 2, 64), (8, 1, 128), (8, 4, 64)])
@pytest.mark.parametrize("top", [100, 300, 1000])
@pytest.mark.parametrize("lens", [[900, 33, 5000, 16, 1, 130, 2600, 64], [30000], [40] * 9])
def test_decode_sums_of_steep_logits_over_far_exponents(pkv, g, hkv, d, top, lens):
    """A key far above the others in logit may lie far below them in s + e (V's exponent 235 lower): the
    sum of the weights without V's exponents then passes fp32's range over the reference of the others."""
    rng = np.random.default_rng(top + d + len(lens))
    page = 16
    pages = sum(-(-n // page) for n in lens) + 64
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    scale = steep_keys(pool, was, rng, page, top)
    table, rows, _ = paged_batch(pkv, rng, lens, page, pages, 2 if len(lens) == 8 else 0)
    q = np.broadcast_to(rng.choice([1.0, 0.5, -1.0], (len(lens), hkv * g, 1)), (len(lens), hkv * g, d)) / d
    o, ws = check_decode(pkv, pool, was, table, rows, lens, page, hkv * g, scale, q=q)
    assert error(pkv, ws) == 0


@pytest.mark.parametrize("first", ["near", "far"])
@pytest.mark.parametrize("gap", [119, 126, 127, 128, 140, 200, 235])
def test_decode_of_two_pages_far_apart(pkv, first, gap):
    """One page whose V exponent is `gap` binades above the other's; the other's keys are `gap` - 1 above it in
    logits, so that both reach the result, or far more, so that only they do."""
    page, hkv, g, d = 16, 1, 8, 64
    rng = np.random.default_rng(gap)
    pool, was = random_pool(pkv, rng, 4, page, hkv, d)
    lo, hi = (245 - gap, 245) if gap > 200 else (127 - gap // 2, 127 - gap // 2 + gap)
    order = [0, 1] if first == "near" else [1, 0]
    was[0][:page], was[0][page:2 * page] = 0, 0x38          # logits 0 and q * 64 scale
    was[1][:], was[3][0], was[3][1] = 127, hi, lo
    for t, w in zip((pool.k, pool.k_exp, pool.v_exp), (was[0], was[1], was[3])):
        t.copy_(dev(w, np.uint8))
    table = np.array([order + [0, 0]])
    q = np.broadcast_to(np.array([1.0, 0.5, 2.0, 4.0, 0.25, -1.0, 1.5, 0.75])[None, :, None], (1, 8, d)) / d
    o, ws = check_decode(pkv, pool, was, table, [0], [2 * page], page, 8, (gap - 1) * np.log(2.0), q=q)
    assert error(pkv, ws) == 0


@pytest.mark.parametrize("hkv,g,d", [(2, 4, 64), (1, 8, 128), (8, 1, 64)])
def test_extend_streams_of_steep_logits_over_far_exponents(pkv, hkv, g, d):
    rng = np.random.default_rng(d + g)
    page, lens, new = 16, [700, 20, 3000, 5], [5, 20, 3, 1]
    pages = sum(-(-n // page) for n in lens) + 1
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    scale = steep_keys(pool, was, rng, page, 300)
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages)
    qo = np.concatenate([[0], np.cumsum(new)])
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d)
    plan.info.offsets[18] = 1
    n = int(qo[-1])
    qt, qv = bf16(np.broadcast_to(rng.choice([1.0, 0.5, -1.0], (n, hkv * g, 1)), (n, hkv * g, d)) / d)
    o, ws = torch.full_like(qt, float("nan")), words((plan.info.workspace_bytes + 3) // 4)
    pkv.attn_extend_block(pool, batch, qt, o, scale, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0
    for r in range(len(lens)):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        e = ref.exponents_of(was[3], table[rows[r]], lens[r], page)
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, scale, np.arange(lens[r] - new[r], lens[r]), DECODE_EPS, v_exp=e)
        assert np.all(np.abs(values(o[qo[r]:qo[r + 1]]) - want) <= bound), r


@pytest.mark.parametrize("g,hkv", [(8, 1), (2, 2)])
@pytest.mark.parametrize("length,listed", [(1109248, 70000), (100016, 16 * 6251)])
def test_decode_of_the_smallest_values_over_long_contexts(pkv, g, hkv, length, listed):
    """Equal weights over one page named many times, a power of two in each column of V: every sum is a whole
    number of that power, below 2^24, so that the result is the value itself, at the smallest exponent too.  Only the
    output's rounding and five fp32 roundings are left: the weights' sum, its reciprocal (2 ulp), two factors."""
    page, d = 16, 64
    pool = pkv.BlockPool.allocate(2, page, hkv, d)
    codes = np.broadcast_to(0x50 + 8 * (np.arange(d) % 6), (page, hkv, d)).astype(np.uint8)     # 8 to 256
    pool.v[page:] = dev(codes, np.uint8)
    pool.v_exp.fill_(10)
    blocks = -(-length // page)
    table = torch.ones((1, blocks), dtype=torch.int32, device="cuda")
    q, _ = bf16(np.ones((1, hkv * g, d)))
    o = torch.full_like(q, float("nan"))
    ws = words(pkv.decode_block_workspace(pool, hkv * g) // 4)
    for n in (length, length - 5, listed):
        pkv.attn_decode_block(pool, pkv.Batch(table, dev([0]), dev([n]), page), q, o, 0.1, ws)
        assert error(pkv, ws) == 0
        want = ref.e4m3_decode(codes[:1]) * 2.0 ** -117
        got = values(o).reshape(1, hkv, g, d)
        assert np.all(np.abs(got - want[:, :, None]) <= (2.0 ** -8 + 5 * 2.0 ** -24) * want[:, :, None])


@pytest.mark.parametrize("choice", [[10], [245], [10, 127, 245], [205, 215, 225]])
@pytest.mark.parametrize("hkv,g,d,shared", [(2, 4, 64, 0), (1, 8, 128, 128), (8, 1, 128, 0)])
def test_gathered_extend_at_the_ends_of_the_exponents(pkv, choice, hkv, g, d, shared):
    """V pages at the smallest exponent, the largest and both.  Values of one sign, so that a sum of the largest
    ones passes fp32's range where their mean does not; none so small that a product with its weight
    (2^-12 or more) would be below fp32's normal numbers."""
    rng = np.random.default_rng(len(choice) + d)
    page, old, new = 16, [0, 900, 130, 300], [60, 30, 200, 3]
    lens = [a + b for a, b in zip(old, new)]
    if shared:
        old[0], lens[0] = 200, 260
    pages = sum(-(-n // page) for n in lens) + 1
    pool, was = random_pool(pkv, rng, pages, page, hkv, d)
    was[2][:] = rng.integers(0x50, 0x7F, was[2].shape)    # 8 to 448
    was[3][:] = rng.choice(choice, was[3].shape)
    pool.v.copy_(dev(was[2], np.uint8))
    pool.v_exp.copy_(dev(was[3], np.uint8))
    table, rows, batch = paged_batch(pkv, rng, lens, page, pages, shared // page)
    qo = np.concatenate([[0], np.cumsum(new)])
    cascade = None
    if shared:
        cascade = pkv.Cascade(*(np.asarray(a, np.int32) for a in ([0], [0], [shared], [0, 4], range(4))))
    plan = pkv.plan_extend(lens, new, qo, hkv * g, hkv, d, cascade)
    plan.info.offsets[18] = 0
    x = rng.standard_normal((int(qo[-1]), hkv * g, d))
    qt, qv = bf16(x)
    scale = 0.01
    o, ws = torch.full_like(qt, float("nan")), words((plan.info.workspace_bytes + 3) // 4)
    for _ in range(2):
        pkv.attn_extend_block(pool, batch, qt, o, scale, plan, dev(plan.blob, np.uint8), ws)
    assert error(pkv, ws) == 0 and int(ws[20]) == 0
    for r in range(len(lens)):
        k, v = (ref.rows_of(was[j], was[j + 1], table[rows[r]], lens[r], page) for j in (0, 2))
        want, bound = ref.attend(qv[qo[r]:qo[r + 1]], k, v, scale, np.arange(lens[r] - new[r], lens[r]), EXTEND_EPS, EXTEND_LOG_EPS)
        assert np.all(np.abs(values(o[qo[r]:qo[r + 1]]) - want) <= bound), r


# ----------------------------------------------------------------------------------------
# large batches of few-head groups


@pytest.mark.parametrize("b,g,hkv,stride", [(4097, 1, 2, 4), (5000, 1, 1, 70), (2049, 2, 3, 70), (9000, 2, 1, 4)])
def test_decode_of_many_requests_of_own_tiles(pkv, b, g, hkv, stride):
    """With 4 or 8 requests a stream results and records go by a request's own tiles; past 512 streams the
    tiles before each are written down.  Both at once, with and without shared pages (rows long enough to
    be looked through), lengths that cross ranges, and empty requests."""
    rng = np.random.default_rng(b)
    page, d, n = 16, 64, 100
    pool, was = random_pool(pkv, rng, stride * n, page, hkv, d)
    table, rows = rng.permutation(stride * n).reshape(n, stride), np.repeat(rng.integers(0, n, b), 3)[:b]
    if stride > 4:
        table[50:, :40] = table[0, :40]     # a prefix of half of the rows
    lens = rng.integers(0, stride * page + 1, b)
    lens[rng.random(b) < 0.1] = 0
    lens[-1] = stride * page
    q = np.zeros((b, hkv * g, d), np.float32)
    q[:] = rng.standard_normal((1, hkv * g, d))
    only = [0, 1, b // 2, b - 1, *rng.permutation(b)[:16]]
    o, ws = check_decode(pkv, pool, was, table, rows, lens.tolist(), page, hkv * g, 0.1, q=q, only=only)
    assert error(pkv, ws) == 0 and torch.isfinite(o).all()
    assert torch.equal((o == 0).all(2).all(1).cpu(), torch.from_numpy(lens == 0))


@pytest.mark.parametrize("g", [1, 4, 8])
def test_a_captured_step_holds_decodes_own_bound(pkv, g):
    """Tables, store and decode in one graph, replayed as lengths grow, with attention held to decode's bound."""
    rng = np.random.default_rng(g)
    page, hkv, d, b, scale = 16, 2, 64, 9, 0.125
    hq = hkv * g
    pool = pkv.BlockPool.allocate(80, page, hkv, d)
    free, head, table = dev(rng.permutation(80)), words(1), torch.full((b, 6), -1, dtype=torch.int32, device="cuda")
    rows, seq, new = dev(rng.permutation(b)), words(b), words(b)
    most = 30
    loc, pos, qo = words(b * most), words(b * most), words(b + 1)
    k, v = (torch.zeros((b * most, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, o = (torch.zeros((b, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, space = words(), words(pkv.decode_block_workspace(pool, hq) // 4)

    def step():
        pkv.build_block_tables(table, rows, seq, new, free, head, head, loc, pos, qo, page, ws)
        pkv.kv_store_block(pool, k, v, loc, ws)
        pkv.attn_decode_block(pool, pkv.Batch(table, rows, seq, page), q, o, scale, space)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = np.zeros(b, np.int64)
    for i in range(4):
        add = rng.integers(0, most + 1, b) if i == 0 else rng.integers(0, 2, b)
        lens += add
        for t, a in zip((seq, new), (lens, add)):
            t.copy_(dev(a))
        for t in (k, v):
            t.copy_(bf16(rng.standard_normal(t.shape) * 2.0 ** rng.integers(-2, 3, (b * most, hkv, 1)))[0])
        qt, qv = bf16(rng.standard_normal((b, hq, d)))
        q.copy_(qt)
        graph.replay()
        assert error(pkv, ws) == 0 and error(pkv, space) == 0
        codes, t = [host(x) for x in (pool.k, pool.k_exp, pool.v, pool.v_exp)], host(table)[host(rows)]
        for r in range(b):
            kk, vv = (ref.rows_of(codes[j], codes[j + 1], t[r], lens[r], page) for j in (0, 2))
            e = ref.exponents_of(codes[3], t[r], lens[r], page)
            want, bound = ref.attend(qv[r:r + 1], kk, vv, scale, [lens[r] - 1], DECODE_EPS, v_exp=e)
            assert np.all(np.abs(values(o[r:r + 1]) - want) <= bound), (i, r)


# ----------------------------------------------------------------------------------------
# the store's error word


def test_store_refuses_a_workspace_without_an_error_word(pkv):
    pool, was = random_pool(pkv, np.random.default_rng(0), 4, 16, 2, 64)
    x, _ = bf16(np.ones((3, 2, 64)))
    raw = torch.zeros(64, dtype=torch.uint8, device="cuda")
    for ws in (raw[:0], raw[:3]):
        with pytest.raises(ValueError):
            pkv.kv_store_block(pool, x, x, dev([0, 1, 2]), ws)
    for at in (1, 2, 3):
        with pytest.raises(pkv.PkvError):
            pkv.kv_store_block(pool, x, x, dev([0, 1, 2]), raw[at:])
    for t, w in zip((pool.k, pool.k_exp, pool.v, pool.v_exp), was):
        assert np.array_equal(host(t), w)
    pkv.kv_store_block(pool, x, x, dev([0, 1, -2]), raw[4:])
    assert error(pkv, raw[4:]) == 0x100 and torch.all(raw[8:] == 0) and torch.all(raw[:4] == 0)


# ----------------------------------------------------------------------------------------
# pages given back


def test_pages_given_back_are_taken_again(pkv):
    """A request that left has its row's pages written below the list's head, which drops by as many; the next
    step takes them first, and the other requests' pages stay theirs."""
    page, b = 16, 3
    free, head = dev(np.arange(20, 40)), words(1)
    table = torch.full((b, 8), -1, dtype=torch.int32, device="cuda")
    loc, pos, qo, ws = words(200), words(200), words(b + 1), words()

    def step(seq, new):
        pkv.build_block_tables(table, dev([0, 1, 2]), dev(seq), dev(new), free, head, head, loc, pos, qo, page, ws)
        assert error(pkv, ws) == 0
        return host(table), host(loc), int(head)
    t, _, h = step([33, 20, 0], [33, 20, 0])
    assert t[0, :3].tolist() == [20, 21, 22] and t[1, :2].tolist() == [23, 24] and h == 5
    free[h - 3:h] = table[0, :3]
    head -= 3
    t, slots, h = step([0, 33, 20], [0, 13, 20])     # request 1 grows into a third page, request 2 arrives
    assert t[1, :3].tolist() == [23, 24, 20] and t[2, :2].tolist() == [21, 22] and h == 5
    want = [24 * 16 + i for i in range(4, 16)] + [20 * 16] + [21 * 16 + i for i in range(16)] + [22 * 16 + i for i in range(4)]
    assert slots[:33].tolist() == want and np.all(slots[33:] == -1)
