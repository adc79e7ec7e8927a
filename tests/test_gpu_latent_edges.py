"""Rotary positions and the latent pool where they can go wrong: logits and rows that are not finite, sizes past one pass
of a grid, ranges of many requests, joins of many records, waits that run out, rows of few keys, other streams."""

import numpy as np
import pytest
import torch

import latent_reference as ref
from test_gpu_latent import SLOT_RANGE, POSITION, TIMEOUT, YARN, Case, dev, draws, e4m3_near, near, values, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import prefix_shared_kv_token_gb300 as m
    return m


@pytest.fixture(scope="module")
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ----------------------------------------------------------------------------------------
# logits that are not finite


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("length,new,at", [(128, 1, 70), (128, 1, 3), (100, 1, 99), (100, 1, 3), (65, 1, 64), (64, 1, 5), (63, 1, 62),
                                           (200, 10, 195), (200, 10, 20), (700, 1, 690), (9000, 1, 8999), (9000, 1, 4444)])
def test_an_infinite_rotary_key_weighs_the_same_anywhere(pkv, heads, length, new, at):
    """Odd heads see it with a logit of -inf, and so as if it were not there; even ones with +inf, and get NaN."""
    c = Case(pkv, heads, 512, 1, [length], [new], seed=at)
    c.pool.rows[int(c.slots(0)[at]), 520] = float("inf")
    sign = np.where(np.arange(heads) % 2, -1.0, 1.0)
    c.q[:, :, 520] = torch.from_numpy(sign).cuda().to(torch.bfloat16)
    c.qv[:, :, 520] = sign
    o = values(c.run())
    rows, seen = c.data[c.slots(0)], length - new + np.arange(new) + 1
    blind = seen <= at
    want, bound = ref.attend(c.qv, np.delete(rows, at, 0), 512, float(np.float32(c.scale)), seen - ~blind)
    assert np.all(np.abs(o[:, 1::2] - want[:, 1::2]) <= bound[:, 1::2])
    assert np.isnan(o[~blind, ::2]).all() and np.all(np.abs(o[blind, ::2] - want[blind, ::2]) <= bound[blind, ::2])


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("length", [1, 63, 64, 65, 700, 9000])
def test_logits_that_are_all_minus_infinity_give_nan(pkv, heads, length):
    """The largest of them is -inf too, and their differences NaN.  Zeros are for tokens that see nothing."""
    c = Case(pkv, heads, 512, 1, [length, 2, 0], [1, 4, 1], seed=length)
    c.pool.rows[torch.from_numpy(c.slots(0)).cuda(), 530] = float("inf")
    c.pool.rows[torch.from_numpy(c.slots(1)).cuda(), 530] = float("inf")
    c.q[:, :, 530] = -1.0
    o = values(c.run())
    assert np.isnan(o[0]).all() and np.isnan(o[3:5]).all()
    assert np.all(o[1:3] == 0) and np.all(o[5] == 0)


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("length,loud", [(150, 70), (700, 600), (9000, 6000)])
def test_a_nan_survives_the_join(pkv, heads, length, loud):
    """A latent with an infinity under a logit of -inf: 0 times it is NaN, in that element alone, and stays so beside a key of
    another range whose logit leaves all others without weight."""
    c = Case(pkv, heads, 512, 1, [length], seed=length)
    rows = c.slots(0)
    c.pool.rows[int(rows[10]), 7] = float("inf")
    c.q[:, :, 7] = -1.0
    c.pool.rows[int(rows[loud]), 530] = 1024.0
    c.q[:, :, 530] = 128.0
    o = values(c.run())
    rest = np.arange(512) != 7
    assert np.isnan(o[:, :, 7]).all()
    # the others' weights are below e^-5000: the output is the loud key's latent
    assert np.array_equal(o[..., rest], np.broadcast_to(c.data[rows[loud], :512][rest], o[..., rest].shape))


# ----------------------------------------------------------------------------------------
# other streams


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("call", ["rope", "rope_store"])
def test_an_output_made_for_another_stream_is_that_streams(pkv, call, raw):
    """The current stream still reads memory that it has given back: the call on the other stream takes none of it."""
    n, heads, dim = 3000, 16, 64
    rope, side = pkv.Rope(dim), torch.cuda.Stream()
    x, xv = draws((n, heads, dim), 1)
    k, _ = draws((n, 1, dim), 2)
    pool, pos, loc = pkv.Pool.allocate(n, 1, dim), dev(np.arange(n)), dev(np.arange(n))
    want, slack = ref.rotate(xv, np.arange(n), rope.inv_freq, False)
    handle = side.cuda_stream if raw else side
    side.wait_stream(torch.cuda.current_stream())
    for turn in range(4):
        old = torch.full((n, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda")
        kept = torch.empty_like(old)
        torch.cuda._sleep(100_000_000)     # some 50 ms
        kept.copy_(old)
        del old
        if call == "rope":
            got = pkv.rope(x, pos, rope, stream=handle)
        else:
            got = pkv.rope_store(pool, x, k, k, pos, loc, rope, stream=handle)
        side.synchronize()
        # the read has not been made yet (but for the first time, when memory and kernels were new, which waits for it)
        assert turn == 0 or not torch.cuda.current_stream().query()
        near(values_on(got, side), want, slack)
        assert bool((kept == 5.0).all())
        del got


def values_on(t, stream):
    with torch.cuda.stream(stream):
        return values(t)


def test_the_default_stream_by_its_handle(pkv):
    """Handle 0, from a stream of one's own."""
    rope = pkv.Rope(64)
    x, xv = draws((50, 4, 64), 1)
    pos = dev(np.arange(50))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = pkv.rope(x, pos, rope, stream=0)
    torch.cuda.synchronize()
    want, slack = ref.rotate(xv, np.arange(50), rope.inv_freq, False)
    near(values(out), want, slack)


def test_every_call_runs_on_the_stream_it_is_given(pkv):
    """Behind work of that stream, which makes its inputs."""
    side = torch.cuda.Stream()
    rope = pkv.Rope(64)
    c = Case(pkv, 16, 512, 1, [100, 80], seed=8)
    clean = c.run()
    q, qv = draws((90, 16, 64), 3)
    rows, rv = draws((90, 576), 4)
    pool, pos, loc = pkv.LatentPool.allocate(90), dev(np.arange(90)), dev(np.arange(90)[::-1].copy())
    batch, o = c.batch(), torch.zeros_like(clean)
    late = [torch.full_like(t, float("nan")) for t in (q, rows, c.q)]
    turned = torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for t, x in zip(late, (q, rows, c.q)):
            t.copy_(x)
    pkv.rope(late[0], pos, rope, out=turned, stream=side)
    pkv.latent_store(pool, late[1][:, :512], late[1][:, 512:], pos, loc, rope, stream=side)
    pkv.attn_latent(c.pool, batch, late[2], o, c.scale, c.ws, stream=side.cuda_stream)
    side.synchronize()
    want, slack = ref.rotate(qv, np.arange(90), rope.inv_freq, False)
    near(values(turned), want, slack)
    assert torch.equal(pool.rows.flip(0)[:, :512], rows[:, :512]) and torch.equal(o, clean)


@pytest.mark.parametrize("n", [1, 31, 33, 5000, 400000])
def test_padded_rows_alone_are_zeroed(pkv, n):
    from prefix_shared_kv_token_gb300 import _lib
    rng = np.random.default_rng(n)
    loc = rng.integers(-2, 3, n)
    for heads, dim, wide in ((3, 64, 72), (1, 24, 24)):
        held = torch.full((n, heads + 1, wide), 7.0, dtype=torch.bfloat16, device="cuda")
        at, st = dev(loc), held.stride()
        rc = _lib.lib.pkv_zero_padded(held.data_ptr(), st[0], st[1], heads, dim, at.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        want = torch.full_like(held, 7.0)
        want[at == -1, :heads, :dim] = 0
        assert torch.equal(held, want)


@pytest.mark.parametrize("aside", [False, True])
def test_rows_of_padded_tokens_are_zeros_in_a_new_output(pkv, aside):
    rope = pkv.Rope(64)
    q, qv = draws((300, 4, 64), 3)
    k, _ = draws((300, 1, 64), 4)
    loc = np.arange(300)
    loc[::3] = -1
    pool, side = pkv.Pool.allocate(300, 1, 64), torch.cuda.Stream()
    pos, at = dev(np.arange(300)), dev(loc)
    torch.cuda.synchronize()
    for _ in range(3):                     # memory that held something else
        for s in (side, torch.cuda.current_stream()):
            with torch.cuda.stream(s):
                torch.full((300, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        out = pkv.rope_store(pool, q, k, k, pos, at, rope, stream=side if aside else None)
        torch.cuda.synchronize()
        want, slack = ref.rotate(qv, np.arange(300), rope.inv_freq, False)
        got = values(out)
        assert np.all(got[loc < 0] == 0)
        near(got[loc >= 0], want[loc >= 0], slack[loc >= 0])
        del out


# ----------------------------------------------------------------------------------------
# what is copied


def test_what_is_not_rotated_keeps_its_bits(pkv):
    """NaNs with their payloads among them, in the rest of a head and in v, as kv_store keeps them."""
    rope = pkv.Rope(16)
    odd = torch.tensor([0x7FA1, -0x3D, 0x7FFF, 0x7F81, 0x0001, -0x8000, 0x7F80, 0x1234], dtype=torch.int16, device="cuda")
    for n, heads, dim in ((3, 5, 64), (200, 2, 72), (1, 1, 24)):
        x = torch.zeros((n, heads, dim), dtype=torch.bfloat16, device="cuda")
        x.view(torch.int16)[..., 16:] = odd.repeat(dim // 8 - 2)
        out = pkv.rope(x, words(n), rope)
        assert torch.equal(out.view(torch.int16)[..., 16:], x.view(torch.int16)[..., 16:])
    pool, plain = pkv.Pool.allocate(12, 3, 64), pkv.Pool.allocate(12, 3, 64)
    q, _ = draws((9, 4, 64), 1)
    k, _ = draws((9, 3, 64), 2)
    v = odd.repeat(9 * 3 * 8).view(9, 3, 64).view(torch.bfloat16)
    k.view(torch.int16)[..., 16:] = odd.repeat(6)
    pos, loc = dev(np.arange(9)), dev(np.arange(9) + 1)
    pkv.rope_store(pool, q, k, v, pos, loc, rope)
    pkv.kv_store(plain, pkv.rope(k, pos, rope), v, loc)
    assert torch.equal(pool.v.view(torch.int16), plain.v.view(torch.int16)) and torch.equal(pool.k.view(torch.int16), plain.k.view(torch.int16))
    assert torch.equal(pool.v[1:10].view(torch.int16), v.view(torch.int16))


# ----------------------------------------------------------------------------------------
# waits that run out


@pytest.mark.parametrize("heads,seq", [(16, [20000]), (128, [3000, 100, 900]), (32, [500] * 300)])
def test_a_timeout_shows_behind_an_earlier_error(pkv, heads, seq):
    """It takes the place of the lesser error in the word, and what it kept from being computed is left as it was: no records of
    an earlier call are joined."""
    c = Case(pkv, heads, 512, 1, seq, seed=3)
    other = Case(pkv, heads, 512, 1, seq, seed=4)
    other.run(ws=c.ws)                     # records of other rows
    torch.cuda.synchronize()
    c.ws[0] = SLOT_RANGE
    pkv.set_wait_limit_ns(1)
    try:
        o = values(c.run())
    finally:
        pkv.set_wait_limit_ns(0)
    assert pkv.get_device_error(c.ws) & TIMEOUT
    for i in range(len(seq)):
        w, bound = c.want(i)
        left = (o[i] == 11.0).all(-1)
        assert np.all(left | (np.abs(o[i] - w[0]) <= bound[0]).all(-1)), i
    again = c.run()                        # the word still holds the error: it is the caller's to clear
    assert pkv.get_device_error(c.ws) & TIMEOUT
    c.ws[0] = 0
    c.check(again)


# ----------------------------------------------------------------------------------------
# rows of few keys


def few_keys(q, rows, latent, scale, seen):
    """(o, bound) as latent_reference.attend, for rows of fewer than 32 keys: their weights are two bf16 numbers, the second
    the rounding of what the first leaves, and so within 2^-16 of themselves (2^-8 of the 2^-8 that is left)."""
    n, heads, width = q.shape
    o, bound = np.zeros((n, heads, latent)), np.zeros((n, heads, latent))
    for i in range(n):
        k = rows[:int(seen[i])]
        v = k[:, :latent]
        s = q[i] @ k.T * scale
        w = np.exp(s - s.max(-1, keepdims=True))
        p = w / w.sum(-1, keepdims=True)
        o[i] = p @ v
        logit = (width + 4) * 2.0 ** -24 * scale * (np.abs(q[i]) @ np.abs(k).T).max(-1)
        err = 2.0 ** -16 + 2 * logit + 2.0 ** -21
        spread = np.stack([p[h] @ np.abs(v - o[i, h]) for h in range(heads)])
        bound[i] = 2.0 ** -8 * np.abs(o[i]) + err[:, None] * spread + (len(k) + 8) * 2.0 ** -24 * (p @ np.abs(v)) + 1e-37
    return o, bound


@pytest.mark.parametrize("heads,latent", [(16, 512), (20, 256), (128, 512), (1, 512)])
def test_weights_of_rows_of_few_keys(pkv, heads, latent):
    """Decode over short contexts, and the first tokens of prompts."""
    lengths = np.arange(1, 34)
    for c in (Case(pkv, heads, latent, 16, lengths, seed=heads), Case(pkv, heads, latent, 1, [40, 3, 100], [40, 3, 90], seed=heads)):
        o = values(c.run())
        assert pkv.get_device_error(c.ws) == 0
        for i in range(len(c.seq)):
            seen = c.seq[i] - c.new[i] + np.arange(c.new[i]) + 1
            few = np.flatnonzero(seen < 32)
            want, bound = few_keys(c.qv[c.qo[i] + few], c.data[c.slots(i)], latent, float(np.float32(c.scale)), seen[few])
            assert np.all(np.abs(o[c.qo[i] + few] - want) <= bound), i
        c.check(torch.from_numpy(o).cuda())


# ----------------------------------------------------------------------------------------
# sizes that take other code


@pytest.mark.parametrize("heads,dim,rot,layout", [(32, 64, 64, "half"), (3, 72, 16, "interleaved"), (1, 64, 64, "interleaved"), (2, 16, 16, "half")])
@pytest.mark.parametrize("times", [1, 2])
def test_rope_past_one_pass_of_the_grid(pkv, sms, heads, dim, rot, layout, times):
    """32 blocks an SM of 8 warps, a token or several each: the next ones after them."""
    units = rot // 16 + ((dim - rot) // 8 + 1) // 2
    lanes = 1 << (units - 1).bit_length()
    per = min(32 // lanes, 1 << (heads - 1).bit_length())
    n = sms * 256 * (32 // (lanes * per)) * times + 5
    rope = pkv.Rope(rot, layout=layout)
    x, xv = draws((n, heads, dim), n)
    pos = np.random.default_rng(n).integers(0, 2 ** 18, n)
    got = values(pkv.rope(x, dev(pos), rope))
    for at in range(0, n, 65536):
        part = slice(at, at + 65536)
        want, slack = ref.rotate(xv[part], pos[part], rope.inv_freq, layout == "interleaved")
        near(got[part], want, slack)


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("hq,hkv,d,layout", [(4, 2, 64, "half"), (0, 1, 64, "interleaved")])
def test_rope_store_past_one_pass_of_the_grid(pkv, sms, dtype, hq, hkv, d, layout):
    rope = pkv.Rope(d, layout=layout)
    n = sms * 256 * (1 if hq else 4) + 77
    rng = np.random.default_rng(n)
    pool = pkv.Pool.allocate(n + 40, hkv, d, dtype, *((0.013, 0.5) if dtype != "bf16" else (1.0, 1.0)))
    qkv, xv = draws((n, hq + 2 * hkv, d), n, 4.0)
    loc = rng.permutation(n + 40)[:n]
    padded = rng.random(n) < 0.1
    loc[padded] = -1
    loc[n - 3] = n + 40                    # one out of range, in the last step
    live = ~padded
    live[n - 3] = False
    pos, ws = rng.integers(0, 2 ** 18, n), words()
    q_out = torch.full((n, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    pkv.rope_store(pool, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], dev(pos), dev(loc), rope, q_out=q_out, workspace=ws)
    assert pkv.get_device_error(ws) == SLOT_RANGE
    want, slack = ref.rotate(xv, pos, rope.inv_freq, layout == "interleaved")
    turned = live.copy()
    turned[n - 3] = True
    if hq:
        near(values(q_out)[turned], want[turned, :hq], slack[turned, :hq])
        assert np.all(values(q_out)[~turned] == 9.0)
    at = torch.from_numpy(loc[live]).cuda()
    for t, w, sl, scale in ((pool.k, want[:, hq:hq + hkv], slack[:, hq:hq + hkv], pool.k_scale), (pool.v, xv[:, hq + hkv:], 0 * xv[:, :hkv], pool.v_scale)):
        if dtype == "bf16":
            near(values(t[at]), w[live], sl[live])
        else:
            s32 = float(np.float32(scale))
            e4m3_near(t[at].contiguous(), w[live] / s32, sl[live] / s32 + 2.0 ** -23 * np.abs(w[live] / s32))
        rest = torch.ones(n + 40, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert bool((t[rest] == 0).all())


@pytest.mark.parametrize("latent,layout,normed,extra", [(512, "half", True, 5), (512, "interleaved", True, 20547), (256, "half", False, 0),
                                                        (256, "interleaved", True, 1), (512, "half", True, -1)])
def test_latent_store_of_many_tokens(pkv, sms, latent, layout, normed, extra):
    """Eight tokens a warp from 128 an SM on, the last warp's fewer; and one less."""
    n = sms * 128 + extra
    rope = pkv.Rope(64, layout=layout, scaling=YARN)
    rng = np.random.default_rng(n)
    pool, ws = pkv.LatentPool.allocate(n + 30, latent), words()
    pool.rows.fill_(5.0)
    rows, rv = draws((n, latent + 64), n, 3.0)
    w, wv = draws((latent,), 3)
    loc = rng.permutation(n + 30)[:n]
    padded = rng.random(n) < 0.1
    loc[padded] = -1
    loc[n - 2] = n + 30
    live = ~padded
    live[n - 2] = False
    pos = rng.integers(0, 10 ** 6, n)
    pkv.latent_store(pool, rows[:, :latent], rows[:, latent:], dev(pos), dev(loc), rope, norm_weight=w if normed else None, workspace=ws)
    assert pkv.get_device_error(ws) == SLOT_RANGE
    at = torch.from_numpy(loc[live]).cuda()
    got = values(pool.rows[at])
    want, slack = ref.normalise(rv[:, :latent], wv, 1e-6) if normed else (rv[:, :latent], 0 * rv[:, :latent])
    near(got[:, :latent], want[live], slack[live])
    turned, slack = ref.rotate(rv[:, None, latent:], pos, rope.inv_freq, layout == "interleaved", rope.magnitude)
    near(got[:, latent:], turned[live, 0], slack[live, 0])
    rest = torch.ones(n + 30, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((pool.rows[rest] == 5.0).all())


@pytest.mark.parametrize("heads", [16, 128])
def test_more_requests_than_a_range_keeps(pkv, heads):
    """Over a hundred requests a range, empty ones and short ones, and runs of requests without new tokens."""
    rng = np.random.default_rng(heads)
    seq = rng.integers(0, 4, 16000)
    seq[5000] = 300
    c = Case(pkv, heads, 256, 1, seq, seed=heads)
    c.check(c.run(), list(range(0, 16000, 41)) + [4999, 5000, 5001, 15999])
    new = np.minimum(rng.integers(0, 3, 16000), seq)
    new[2000:2300] = new[9000:12000] = new[-500:] = 0
    c = Case(pkv, heads, 256, 1, seq, new, seed=heads)
    c.check(c.run(), [i for i in range(0, 16000, 7) if new[i]] + [5000])


@pytest.mark.parametrize("heads,length", [(32, 60000), (16, 100001), (128, 9000), (200, 30000), (1, 700)])
def test_every_tile_of_a_long_request_counts(pkv, heads, length):
    """One key of each 64 outweighs the rest, all of them alike, and has a 1 in its own element of the latent: an element is the
    share of the tiles that have it, and a tile lost or counted twice changes its element by half of it or more."""
    c = Case(pkv, heads, 512, 64, [length, 10, 4000, 128], seed=9)
    tiles = -(-length // 64)
    rng = np.random.default_rng(1)
    rows = np.zeros((length, 576))
    own = [t * 64 + int(rng.integers(0, min(64, length - t * 64))) for t in range(tiles)]
    rows[own, np.arange(tiles) % 512] = 1.0
    rows[own, 512] = 100.0                 # a logit of 100 beside 0: e^-100 of the others' weights is left
    c.pool.rows[torch.from_numpy(c.slots(0)).cuda()] = torch.from_numpy(rows.astype(np.float32)).cuda().to(torch.bfloat16)
    q = np.zeros(576)
    q[512] = 1.0 / c.scale                 # 24: exact
    c.q[0] = torch.from_numpy(q.astype(np.float32)).cuda().to(torch.bfloat16)
    o = c.run()
    want = np.bincount(np.arange(tiles) % 512, minlength=512) / tiles
    got = values(o)[0]
    # equal weights of 1 and their sums are exact; what is left is the output's rounding, and the division's
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -20) * want + 1e-30)
    c.check(o, [1, 2, 3])


def test_a_request_left_out_leaves_the_others(pkv):
    """Offsets out of range: that request's rows stay as they were, the others are right."""
    c = Case(pkv, 16, 512, 16, [100, 80, 60], [2, 3, 4], seed=5)
    for qo, good in (([0, 2, 5, 40], [0, 1]), ([-4, 2, 5, 9], [1, 2]), ([0, 2, 1, 1], [0]), ([5, 2, 5, 9], [1, 2])):
        o = torch.full((9, 16, 512), 11.0, dtype=torch.bfloat16, device="cuda")
        ws = c.workspace()
        pkv.attn_latent(c.pool, c.batch(), c.q, o, c.scale, ws, qo_indptr=dev(qo))
        assert pkv.get_device_error(ws) == POSITION
        got, rest = values(o), np.ones(9, bool)
        for i in good:
            w, bound = c.want(i)
            assert np.all(np.abs(got[qo[i]:qo[i + 1]] - w) <= bound), (qo, i)
            rest[qo[i]:qo[i + 1]] = False
        assert np.all(got[rest] == 11.0), qo
