"""Rotary positions, the fused stores and attention over the latent pool on the GPU, against their plain 64-bit
forms.  The error bounds are derived in latent_reference."""

import numpy as np
import pytest
import torch

import latent_reference as ref

pytestmark = pytest.mark.gpu

SLOT_RANGE, TIMEOUT, POSITION = 0x100, 0x200, 0x400
YARN = dict(kind="yarn", factor=32.0, original=4096)


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


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def draws(shape, seed, size=1.0):
    """(device bf16 tensor, its float64 values) of normal draws."""
    x = ref.bf16(np.random.default_rng(seed).standard_normal(shape) * size)
    return torch.from_numpy(x.astype(np.float32)).cuda().to(torch.bfloat16), x


def words(n=64):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


def near(got, want, slack):
    """A bf16 result: its rounding, 2^-8 of it, beside the slack of what was rounded (which is rounded too)."""
    off = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + slack * (1 + 2.0 ** -8) + 1e-38)
    assert np.all(np.isfinite(got)) and np.all(off <= 0), float(off.max())


# ----------------------------------------------------------------------------------------
# rope


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,dim,rot", [(1, 1, 64, 64), (3, 5, 128, 128), (257, 8, 128, 64), (1000, 32, 64, 32), (7, 128, 64, 64),
                                             (33, 3, 72, 16), (5, 2, 512, 512), (64, 7, 256, 96), (2, 40, 16, 16), (9000, 3, 136, 128)])
def test_rope(pkv, layout, n, heads, dim, rot):
    rope = pkv.Rope(rot, layout=layout, scaling=YARN if rot == 64 else None)
    x, xv = draws((n, heads, dim), n + dim)
    pos = np.random.default_rng(n).integers(0, 2 ** 20, n)
    pos[:3] = [0, 2 ** 31 - 1, 131071][:n]
    want, slack = ref.rotate(xv, pos, rope.inv_freq, layout == "interleaved", rope.magnitude)
    near(values(pkv.rope(x, dev(pos), rope)), want, slack)
    assert np.array_equal(values(x), xv)               # not in place unless asked
    assert pkv.rope(x, dev(pos), rope, out=x) is x
    near(values(x), want, slack)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,dim,rot", [(1001, 1, 64, 64), (30001, 1, 16, 16), (777, 2, 64, 32), (95, 3, 32, 16), (5, 1, 128, 128), (7, 1, 24, 16)])
def test_rope_of_few_heads(pkv, layout, n, heads, dim, rot):
    """Several tokens to a warp, the last warp with fewer."""
    rope = pkv.Rope(rot, layout=layout)
    x, xv = draws((n, heads, dim), n)
    pos = np.random.default_rng(n).integers(0, 2 ** 18, n)
    want, slack = ref.rotate(xv, pos, rope.inv_freq, layout == "interleaved")
    near(values(pkv.rope(x, dev(pos), rope)), want, slack)


def test_rope_negative_positions_turn_back(pkv):
    rope = pkv.Rope(64)
    x, xv = draws((50, 4, 64), 1)
    pos = -np.arange(50) * 997
    want, slack = ref.rotate(xv, pos, rope.inv_freq, False)
    near(values(pkv.rope(x, dev(pos), rope)), want, slack)


def test_rope_of_slices(pkv):
    """Slices of longer rows in, a slice of longer rows out; what lies between them stays."""
    rope = pkv.Rope(64, layout="interleaved")
    rows, rv = draws((20, 6, 576), 2)
    out = torch.full((20, 8, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = np.arange(20) * 31
    want, slack = ref.rotate(rv[..., 512:], pos, rope.inv_freq, True)
    pkv.rope(rows[..., 512:], dev(pos), rope, out=out[:, 1:7, 8:72])
    near(values(out[:, 1:7, 8:72]), want, slack)
    out[:, 1:7, 8:72] = 7.0
    assert bool((out == 7.0).all()) and np.array_equal(values(rows), rv)
    by_heads = rows.transpose(0, 1)[..., :64]          # [heads, tokens, dim] as 6 tokens of 20 heads
    want, slack = ref.rotate(rv.transpose(1, 0, 2)[..., :64], np.arange(6), rope.inv_freq, True)
    near(values(pkv.rope(by_heads, dev(np.arange(6)), rope)), want, slack)


def test_rope_refuses(pkv):
    rope = pkv.Rope(64)
    x, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda"), words(4)
    for args in ((x.float(), pos), (x.cpu(), pos), (x, pos.cpu()), (x, pos[:3]), (x, pos.long()), (x[0], pos), (x.transpose(1, 2), pos)):
        with pytest.raises(ValueError):
            pkv.rope(*args, rope)
    with pytest.raises(ValueError):
        pkv.rope(x, pos, rope, out=x[:3])
    with pytest.raises(pkv.PkvError):
        pkv.rope(x, pos, rope, out=x[:1].expand(4, 2, 64))
    with pytest.raises(pkv.PkvError):
        pkv.rope(x[..., :32], pos, rope)               # fewer elements than turn
    odd = torch.zeros(4 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(4, 2, 64)
    with pytest.raises(pkv.PkvError):
        pkv.rope(odd, pos, rope)                       # not 16-byte aligned
    assert pkv.rope(x[:0], pos[:0], rope).shape == (0, 2, 64)


# ----------------------------------------------------------------------------------------
# rope_store


def e4m3_near(codes, want, slack):
    """Codes of want: half a step of their type, 2^-4 of the value or 2^-10 below its normal numbers, saturating."""
    got = codes.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
    want = np.clip(want, -448, 448)
    assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + slack * 1.1)


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("n,hq,hkv,d,rot,layout,pools", [
    (1, 8, 2, 64, 64, "half", "separate"), (4, 32, 8, 128, 128, "half", "interleaved"), (300, 5, 5, 64, 32, "interleaved", "separate"),
    (2001, 16, 1, 128, 64, "interleaved", "interleaved"), (700, 64, 8, 128, 96, "half", "separate"), (33, 0, 3, 64, 16, "half", "separate"),
    (4003, 0, 1, 64, 64, "half", "interleaved"), (901, 1, 1, 64, 48, "interleaved", "separate")])
def test_rope_store(pkv, dtype, n, hq, hkv, d, rot, layout, pools):
    rope = pkv.Rope(rot, layout=layout, scaling=YARN if rot == 64 else None)
    rng = np.random.default_rng(n)
    scales = (0.013, 0.5) if dtype != "bf16" else (1.0, 1.0)
    pool = pkv.Pool.allocate(n + 40, hkv, d, dtype, *scales, layout=pools)
    pool.k.fill_(3)
    pool.v.fill_(3)
    qkv, xv = draws((n, hq + 2 * hkv, d), n, 4.0)
    loc = rng.permutation(n + 40)[:n]
    padded = rng.random(n) < 0.1
    loc[padded] = -1
    pos = rng.integers(0, 10 ** 6, n)
    ws = words()
    q_out = torch.full((n, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    got = pkv.rope_store(pool, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], dev(pos), dev(loc), rope, q_out=q_out, workspace=ws)
    assert got is q_out and pkv.get_device_error(ws) == 0
    want, slack = ref.rotate(xv, pos, rope.inv_freq, layout == "interleaved", rope.magnitude)
    live = ~padded
    if hq and live.any():
        near(values(q_out)[live], want[live, :hq], slack[live, :hq])
    assert np.all(values(q_out)[padded] == 9.0)
    for t, w, sl, scale in ((pool.k, want[:, hq:hq + hkv], slack[:, hq:hq + hkv], scales[0]), (pool.v, xv[:, hq + hkv:], 0 * xv[:, :hkv], scales[1])):
        at = torch.from_numpy(loc[live]).cuda()
        if dtype == "bf16":
            if live.any():
                near(values(t[at]), w[live], sl[live])
        else:
            s32 = float(np.float32(scale))
            e4m3_near(t[at].contiguous(), w[live] / s32, sl[live] / s32 + 2.0 ** -23 * np.abs(w[live] / s32))
        rest = torch.ones(n + 40, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert bool((t[rest] == 3).all())


def test_rope_store_takes_q_in_place_and_matches_its_parts(pkv):
    """bf16: the pool holds the same bits as rope and kv_store one after the other."""
    rope = pkv.Rope(128)
    q, _ = draws((90, 4, 128), 5)
    k, _ = draws((90, 2, 128), 6)
    v, _ = draws((90, 2, 128), 7)
    pos, loc = dev(np.arange(90) * 11), dev(np.random.default_rng(0).permutation(100)[:90])
    one, two = pkv.Pool.allocate(100, 2, 128), pkv.Pool.allocate(100, 2, 128)
    want_q = pkv.rope(q, pos, rope)
    pkv.kv_store(one, pkv.rope(k, pos, rope), v, loc)
    assert pkv.rope_store(two, q, k, v, pos, loc, rope, q_out=q) is q
    for a, b in ((one.k, two.k), (one.v, two.v), (want_q, q)):
        assert torch.equal(a, b)


def test_rope_store_reports_a_slot_out_of_range(pkv):
    rope = pkv.Rope(64)
    q, qv = draws((3, 2, 64), 8)
    k, _ = draws((3, 1, 64), 9)
    for bad in (10, -2, 2 ** 31 - 1):
        pool, ws = pkv.Pool.allocate(10, 1, 64), words()
        out = pkv.rope_store(pool, q, k, k, dev([5, 6, 7]), dev([1, bad, 3]), rope, workspace=ws)
        assert pkv.get_device_error(ws) == SLOT_RANGE
        want, slack = ref.rotate(qv, [5, 6, 7], rope.inv_freq, False)
        near(values(out), want, slack)
        rest = torch.ones(10, dtype=torch.bool, device="cuda")
        rest[[1, 3]] = False
        assert bool((pool.k[rest] == 0).all()) and bool((pool.k[[1, 3]] != 0).any())


def test_rope_store_refuses(pkv):
    rope = pkv.Rope(64)
    pool = pkv.Pool.allocate(10, 2, 64)
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, pos = t(3, 4, 64), t(3, 2, 64), words(3)
    for args in ((q, t(3, 1, 64), k, pos, pos), (q, k, t(2, 2, 64), pos, pos), (t(3, 4, 128), k, k, pos, pos), (q, k, k, pos[:2], pos),
                 (q, k, k, pos, pos.long()), (q.cpu(), k, k, pos, pos), (q, t(3, 2, 128)[..., :64], k, pos, pos)):
        with pytest.raises(ValueError):
            pkv.rope_store(pool, *args, rope)
    with pytest.raises(ValueError):
        pkv.rope_store(pool, q, k, k, pos, pos, rope, workspace=torch.zeros(3, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pkv.PkvError):
        pkv.rope_store(pool, q, k, k, pos, pos, pkv.Rope(80))


# ----------------------------------------------------------------------------------------
# latent_store


@pytest.mark.parametrize("latent,n,layout,normed,far", [(512, 1, "half", True, 0), (512, 2, "interleaved", False, 9), (256, 77, "half", True, 0),
                                                        (512, 4001, "interleaved", True, 64), (256, 130, "interleaved", False, 0)])
def test_latent_store(pkv, latent, n, layout, normed, far):
    """far: elements between one row of the pool and the next, beyond the row."""
    rope = pkv.Rope(64, layout=layout, scaling=YARN)
    rng = np.random.default_rng(n)
    far = -(-far // 8) * 8
    held = torch.full((n + 30, latent + 64 + far), 5.0, dtype=torch.bfloat16, device="cuda")
    pool = pkv.LatentPool(held[:, :latent + 64], latent)
    rows, rv = draws((n, latent + 64), n, 3.0)
    rows[0, :latent] = 0
    rv[0, :latent] = 0
    w, wv = draws((latent,), 3)
    loc = rng.permutation(n + 30)[:n]
    padded = rng.random(n) < 0.1
    loc[padded] = -1
    pos = rng.integers(0, 10 ** 6, n)
    ws = words()
    pkv.latent_store(pool, rows[:, :latent], rows[:, latent:], dev(pos), dev(loc), rope, norm_weight=w if normed else None, eps=1e-5, workspace=ws)
    assert pkv.get_device_error(ws) == 0
    live = ~padded
    got = values(held[torch.from_numpy(loc[live]).cuda()])
    if live.any():
        want, slack = ref.normalise(rv[:, :latent], wv, float(np.float32(1e-5))) if normed else (rv[:, :latent], 0 * rv[:, :latent])
        near(got[:, :latent], want[live], slack[live])
        turned, slack = ref.rotate(rv[:, None, latent:], pos, rope.inv_freq, layout == "interleaved", rope.magnitude)
        near(got[:, latent:latent + 64], turned[live, 0], slack[live, 0])
        assert np.all(got[:, latent + 64:] == 5.0)
    rest = torch.ones(n + 30, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(loc[live]).cuda()] = False
    assert bool((held[rest] == 5.0).all())


def test_latent_store_reports_a_slot_out_of_range(pkv):
    pool, ws, rope = pkv.LatentPool.allocate(10, 256), words(), pkv.Rope(64)
    rows, _ = draws((4, 320), 1)
    pkv.latent_store(pool, rows[:, :256], rows[:, 256:], dev([0, 1, 2, 3]), dev([2, 10, -5, 4]), rope, workspace=ws)
    assert pkv.get_device_error(ws) == SLOT_RANGE
    assert torch.equal(pool.rows[[2, 4], :256], rows[[0, 3], :256])
    rest = torch.ones(10, dtype=torch.bool, device="cuda")
    rest[[2, 4]] = False
    assert bool((pool.rows[rest] == 0).all())


def test_latent_store_refuses(pkv):
    pool, rope, pos = pkv.LatentPool.allocate(10), pkv.Rope(64), words(2)
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for args, kw in (((t(2, 256), t(2, 64), pos, pos), {}), ((t(3, 512), t(2, 64), pos, pos), {}), ((t(2, 512), t(2, 32), pos, pos), {}),
                     ((t(2, 512), t(2, 64), pos[:1], pos), {}), ((t(2, 512), t(2, 64), pos, pos), dict(norm_weight=t(256))),
                     ((t(2, 512), t(2, 64), pos, pos), dict(norm_weight=t(512).float())), ((t(2, 512).float(), t(2, 64), pos, pos), {})):
        with pytest.raises(ValueError):
            pkv.latent_store(pool, *args, rope, **kw)
    with pytest.raises(pkv.PkvError):
        pkv.latent_store(pool, t(2, 512), t(2, 64), pos, pos, pkv.Rope(32))
    with pytest.raises(pkv.PkvError):
        pkv.latent_store(pool, t(2, 512), t(2, 64), pos, pos, rope, norm_weight=t(512), eps=-1.0)


# ----------------------------------------------------------------------------------------
# attn_latent


class Case:
    """A batch over a pool with shuffled slots or pages; rows that are nobody's hold NaN."""

    def __init__(self, pkv, heads, latent, page, seq, new=None, seed=0, spare_q=0, size=1.0, shared=0):
        rng = np.random.default_rng(seed)
        self.pkv, self.heads, self.latent, self.page = pkv, heads, latent, page
        self.seq, b = np.asarray(seq), len(seq)
        self.new = np.ones(b, np.int64) if new is None else np.asarray(new)
        blocks = -(-self.seq // page)
        total = int(blocks.sum()) + 3
        ids, at = rng.permutation(total), 0
        self.rows = rng.permutation(b + 2)[:b]
        self.table = np.full((b + 2, max(int(blocks.max()), 1) + 1), 2 ** 30)
        for r, n in zip(self.rows, blocks):
            self.table[r, :n] = ids[at:at + n]
            at += n
        if shared:
            self.table[self.rows, :shared // page] = self.table[self.rows[0], :shared // page]
        self.data = ref.bf16(rng.standard_normal((total * page, latent + 64)))
        live = np.zeros(total * page, bool)
        for i in range(b):
            live[self.slots(i)] = True
        self.data[~live] = np.nan
        self.pool = pkv.LatentPool(torch.from_numpy(self.data.astype(np.float32)).cuda().to(torch.bfloat16), latent)
        self.qo = np.concatenate([[0], np.cumsum(self.new)])
        self.q, self.qv = draws((int(self.qo[-1]) + spare_q, heads, latent + 64), seed + 1, size)
        self.scale = (latent + 64) ** -0.5
        self.ws = self.workspace()

    def workspace(self):
        return torch.zeros(self.pkv.latent_workspace(self.pool, self.heads) // 4, dtype=torch.int32, device="cuda")

    def slots(self, i):
        t = np.arange(self.seq[i])
        return self.table[self.rows[i], t // self.page] * self.page + t % self.page

    def batch(self, seq=None):
        return self.pkv.Batch(dev(self.table), dev(self.rows), dev(self.seq if seq is None else seq), self.page)

    def run(self, decode=None, ws=None, q=None):
        decode = bool(np.all(self.new == 1)) if decode is None else decode
        o = torch.full((len(self.q), self.heads, self.latent), 11.0, dtype=torch.bfloat16, device="cuda")
        self.pkv.attn_latent(self.pool, self.batch(), self.q if q is None else q, o, self.scale, self.ws if ws is None else ws,
                             qo_indptr=None if decode else dev(self.qo))
        return o

    def want(self, i, data=None):
        n, length = int(self.new[i]), int(self.seq[i])
        rows = (self.data if data is None else data)[self.slots(i)]
        return ref.attend(self.qv[self.qo[i]:self.qo[i + 1]], rows, self.latent, float(np.float32(self.scale)), length - n + np.arange(n) + 1)

    def check(self, o, requests=None):
        got = values(o)
        assert self.pkv.get_device_error(self.ws) == 0
        for i in range(len(self.seq)) if requests is None else requests:
            w, bound = self.want(i)
            off = np.abs(got[self.qo[i]:self.qo[i + 1]] - w) - bound
            assert np.all(np.isfinite(got[self.qo[i]:self.qo[i + 1]])) and (off.size == 0 or off.max() <= 0), (i, float(off.max()))
        assert np.all(got[self.qo[-1]:] == 11.0)


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [1, 8, 16, 17, 32, 40, 64, 96, 128, 200])
def test_decode_heads(pkv, heads, latent):
    c = Case(pkv, heads, latent, 16, [1, 300, 63, 64, 65, 129, 0, 500], seed=heads)
    c.check(c.run())


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 64, 128, 4096])
def test_decode_pages(pkv, page):
    c = Case(pkv, 16, 512, page, [5, 700, 64, 1000], seed=page)
    c.check(c.run())


@pytest.mark.parametrize("seq", [[1], [64], [0], [0, 0, 0], [9000], [12000, 3, 1, 0, 2500], [70] * 400, [1] * 1000])
@pytest.mark.parametrize("heads", [16, 128])
def test_decode_lengths(pkv, seq, heads):
    c = Case(pkv, heads, 512, 1, seq, seed=len(seq))
    c.check(c.run(), None if len(seq) < 20 else range(0, len(seq), 17))


@pytest.mark.parametrize("heads,latent", [(16, 512), (128, 512), (20, 256), (64, 512), (1, 256), (80, 512)])
def test_several_new_tokens(pkv, heads, latent):
    """Ragged counts of new tokens, none among them, all of a context, and rows of q behind the last request."""
    c = Case(pkv, heads, latent, 16, [200, 40, 1, 77, 130, 64, 0, 300], [4, 40, 1, 0, 9, 64, 0, 33], seed=heads, spare_q=5)
    c.check(c.run())


def test_more_new_tokens_than_positions(pkv):
    """The first of them see nothing, and get zeros."""
    c = Case(pkv, 16, 512, 1, [3, 5], [8, 5], seed=4)
    o = c.run()
    c.check(o)
    assert bool((o[:5] == 0).all()) and bool((o[5:8] != 0).any())


def test_a_long_request_beside_short_ones(pkv):
    """A request over all ranges: merged from every one of them, by many records and by few."""
    c = Case(pkv, 32, 512, 64, [60000, 10, 4000, 128], seed=9)
    c.check(c.run(), [1, 2, 3])
    got, (w, bound) = values(c.run())[:1], c.want(0)
    assert (np.abs(got - w) - bound).max() <= 0


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_steep_logits(pkv, heads):
    """Logits of several hundred in either direction, growing along the context: references that rise many times."""
    c = Case(pkv, heads, 512, 1, [3000, 700], seed=3, size=30.0)
    order = np.argsort(c.data[c.slots(0)] @ c.qv[0, 0])
    c.table[c.rows[0], :3000] = c.table[c.rows[0], :3000][order]
    c.check(c.run())
    c.table[c.rows[0], :3000] = c.table[c.rows[0], :3000][::-1].copy()
    c.check(c.run())


def test_one_key_gives_its_latent(pkv):
    c = Case(pkv, 16, 512, 1, [1, 1], seed=2)
    o = values(c.run())
    for i in range(2):
        assert np.array_equal(o[i], np.broadcast_to(c.data[c.slots(i)][:, :512], (16, 512)))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_far_out(pkv, sign):
    """Equal keys under logits of some 10^31 in size, above or below 0: the weights are equal, and the output is their latent."""
    c = Case(pkv, 16, 512, 1, [100, 70], [4, 1], seed=2)
    row = ref.bf16(np.random.default_rng(1).choice([-1.0, 1.0], 576) * 1e15)
    c.pool.rows.copy_(torch.from_numpy(np.broadcast_to(row, c.data.shape).astype(np.float32)))
    c.q.copy_(torch.from_numpy(np.broadcast_to(sign * row, c.q.shape).astype(np.float32)))
    o = values(c.run())
    assert np.array_equal(o, np.broadcast_to(row[:512], o.shape))


def test_shared_prefixes(pkv):
    c = Case(pkv, 16, 512, 16, [300, 260, 400, 257], [1, 3, 2, 1], seed=6, shared=256)
    c.check(c.run())


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("where", [0, 200, 511, 520])
def test_a_value_that_is_not_finite_reaches_the_tokens_that_see_it(pkv, bad, where):
    """In the latent and in the rotary key of the last token, of one in the middle of the new ones, and of an early one."""
    for at, first in ((99, 9), (95, 5), (40, 0)):
        c = Case(pkv, 16, 512, 1, [100, 80], [10, 3], seed=8)
        clean = values(c.run())
        c.pool.rows[int(c.slots(0)[at]), where] = bad
        o = values(c.run())
        assert np.array_equal(o[:first], clean[:first])
        assert np.array_equal(o[10:], clean[10:])
        # NaN or infinite somewhere in each head that sees it, unless the key's weight is 0 and its latent finite
        if np.isnan(bad) or where < 512:
            assert not np.isfinite(o[first:10]).all(-1).any()


def test_a_query_that_is_not_finite_stays_in_its_row(pkv):
    c = Case(pkv, 16, 512, 1, [100, 80], [10, 3], seed=8)
    clean = values(c.run())
    c.q[4, 7, 100] = float("nan")
    c.q[11, 2, 530] = float("inf")
    o = values(c.run())
    same = np.ones((13, 16), bool)
    same[4, 7] = same[11, 2] = False
    assert np.array_equal(o[same], clean[same])
    assert np.isnan(o[4, 7]).all() and np.isnan(o[11, 2]).any()


def test_bad_tables_are_reported_and_read_as_zeros(pkv):
    c = Case(pkv, 16, 512, 1, [100, 80, 60], seed=5)
    c.table[c.rows[1], 30] = len(c.data)              # a slot outside the pool
    c.table[c.rows[1], 31] = -1
    o = values(c.run())
    assert pkv.get_device_error(c.ws) == SLOT_RANGE
    rows = c.data[np.where(c.slots(1) == len(c.data), 0, c.slots(1))].copy()
    rows[[30, 31]] = 0
    w, bound = ref.attend(c.qv[1:2], rows, 512, float(np.float32(c.scale)), [80])
    assert np.all(np.abs(o[1:2] - w) <= bound)
    c.ws = c.workspace()
    c.check(torch.from_numpy(o).cuda(), [0, 2])


@pytest.mark.parametrize("what", ["row", "negative row", "length", "negative length"])
def test_a_request_out_of_range_gets_zeros(pkv, what):
    c = Case(pkv, 16, 512, 16, [100, 80, 60], seed=5)
    if what.endswith("row"):
        c.rows = c.rows.copy()
        c.rows[1] = len(c.table) if what == "row" else -1
    batch = c.batch([100, c.table.shape[1] * 16 + 1 if what == "length" else -3 if what == "negative length" else 80, 60])
    o = torch.full((3, 16, 512), 11.0, dtype=torch.bfloat16, device="cuda")
    pkv.attn_latent(c.pool, batch, c.q, o, c.scale, c.ws)
    assert pkv.get_device_error(c.ws) == POSITION
    assert bool((o[1] == 0).all())
    c.ws = c.workspace()
    c.check(o, [0, 2])


def test_offsets_out_of_range_leave_the_request_out(pkv):
    c = Case(pkv, 16, 512, 16, [100, 80, 60], [2, 3, 4], seed=5)
    for qo in ([0, 2, 1, 9], [0, 2, 5, 40], [-4, 2, 5, 9]):
        o = torch.full((9, 16, 512), 11.0, dtype=torch.bfloat16, device="cuda")
        c.ws = c.workspace()
        pkv.attn_latent(c.pool, c.batch(), c.q, o, c.scale, c.ws, qo_indptr=dev(qo))
        assert pkv.get_device_error(c.ws) == POSITION


def test_calls_repeat_exactly_and_workspaces_are_apart(pkv):
    a = Case(pkv, 32, 512, 1, [4000, 900, 10], seed=1)
    b = Case(pkv, 128, 512, 16, [700, 5000], [3, 1], seed=2)
    first = [x.run() for x in (a, b)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            again_b = b.run()
    again_a = a.run()
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(first[0], again_a) and torch.equal(first[1], again_b)
    a.check(again_a)
    b.check(again_b)


def test_slots_beyond_4_gib(pkv):
    """A pool of 4.7 GB: rows past 2^32 bytes, and elements past 2^31."""
    c = Case(pkv, 16, 512, 1, [200, 90], seed=7)
    slots = (1 << 32) // 1152 + 400000
    rows = torch.zeros((slots, 576), dtype=torch.bfloat16, device="cuda")
    far = slots - 1 - np.arange(len(c.data)) * 3
    rows[torch.from_numpy(far).cuda()] = c.pool.rows
    c.pool = pkv.LatentPool(rows, 512)
    data = c.data
    c.data = None
    table, c.table = c.table, np.where(c.table < len(data), far[np.minimum(c.table, len(data) - 1)], c.table)
    o = c.run()
    c.table, c.data = table, data
    c.check(o)


def test_a_pool_with_rows_apart(pkv):
    c = Case(pkv, 16, 256, 16, [200, 90], seed=7)
    held = torch.full((len(c.data), 328), float("nan"), dtype=torch.bfloat16, device="cuda")
    held[:, 8:] = c.pool.rows
    c.pool = pkv.LatentPool(held[:, 8:], 256)
    assert c.pool._c.slot_stride == 328
    c.check(c.run())


def test_a_captured_step_follows_lengths_and_tables(pkv):
    c = Case(pkv, 64, 512, 16, [400, 90, 1000], [1, 1, 1], seed=11)
    table, rows, seq, q = dev(c.table), dev(c.rows), dev([1, 0, 2]), torch.zeros_like(c.q)
    qo = dev([0, 1, 2, 3])
    o = torch.zeros((3, 64, 512), dtype=torch.bfloat16, device="cuda")
    run = lambda: pkv.attn_latent(c.pool, pkv.Batch(table, rows, seq, 16), q, o, c.scale, c.ws, qo_indptr=qo)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    q.copy_(c.q)
    for lengths in ([400, 90, 1000], [1, 64, 65], [0, 90, 3]):
        seq.copy_(dev(lengths))
        graph.replay()
        c.seq = np.asarray(lengths)
        c.check(o)


def test_a_wait_that_runs_out_is_reported(pkv):
    c = Case(pkv, 16, 512, 1, [20000], seed=1)
    pkv.set_wait_limit_ns(1)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_limit_ns(0)
    assert pkv.get_device_error(c.ws) & TIMEOUT
    c.ws = c.workspace()
    c.check(c.run())


def test_attn_latent_refuses(pkv):
    c = Case(pkv, 16, 512, 16, [100, 80], seed=5)
    o, b = torch.zeros((2, 16, 512), dtype=torch.bfloat16, device="cuda"), c.batch()
    for args in ((c.q.float(), o, c.scale, c.ws), (c.q[..., :512], o, c.scale, c.ws), (c.q, o[..., :256], c.scale, c.ws), (c.q, o[:1], c.scale, c.ws),
                 (c.q.cpu(), o, c.scale, c.ws), (c.q[0], o, c.scale, c.ws)):
        with pytest.raises(ValueError):
            pkv.attn_latent(c.pool, b, *args)
    with pytest.raises(ValueError):
        pkv.attn_latent(c.pool, b, c.q, o, c.scale, c.ws, qo_indptr=dev([0, 1]))
    for args, kw in (((c.q[:1], o[:1], c.scale, c.ws), {}), ((c.q, o, 0.0, c.ws), {}), ((c.q, o, c.scale, c.ws[:100]), {})):
        with pytest.raises(pkv.PkvError):
            pkv.attn_latent(c.pool, b, *args, **kw)


# ----------------------------------------------------------------------------------------
# a run of them together


@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_step(pkv, captured):
    """Prompts, then decode steps: tables on the device, the store of new rows, the queries' rotation in place, attention,
    each step against the 64-bit forms of what the pool holds; eager, and as one captured graph."""
    heads, latent, page, b, steps = 32, 512, 16, 3, 4
    rope = pkv.Rope(64, layout="interleaved", scaling=YARN)
    pool = pkv.LatentPool.allocate(64 * page, latent)
    width = latent + 64
    w, wv = draws((latent,), 1)
    prompt = np.array([37, 5, 100])
    most = int(prompt.sum())
    table, rows = torch.full((b, 16), -1, dtype=torch.int32, device="cuda"), dev(np.arange(b))
    seq, new = words(b), words(b)
    free, head = dev(np.random.default_rng(2).permutation(64)), words(1)
    tables_ws, store_ws = words(), words()
    held = [np.zeros((0, width)) for _ in range(b)]

    def buffers(cap):
        return dict(loc=words(cap), pos=words(cap), qo=words(b + 1), x=torch.zeros((cap, width), dtype=torch.bfloat16, device="cuda"),
                    q=torch.zeros((cap, heads, width), dtype=torch.bfloat16, device="cuda"),
                    o=torch.zeros((cap, heads, latent), dtype=torch.bfloat16, device="cuda"))

    attn_ws = torch.zeros(pkv.latent_workspace(pool, heads) // 4, dtype=torch.int32, device="cuda")

    def step(s):
        pkv.build_block_tables(table, rows, seq, new, free, head, head, s["loc"], s["pos"], s["qo"], page, tables_ws)
        pkv.latent_store(pool, s["x"][:, :latent], s["x"][:, latent:], s["pos"], s["loc"], rope, norm_weight=w, workspace=store_ws)
        pkv.rope(s["q"][..., latent:], s["pos"], rope, out=s["q"][..., latent:])
        pkv.attn_latent(pool, pkv.Batch(table, rows, seq, page), s["q"], s["o"], width ** -0.5, attn_ws, qo_indptr=s["qo"])

    graph = None
    lengths = np.zeros(b, np.int64)
    bufs = None
    for t in range(steps):
        counts = prompt if t == 0 else np.array([1, 1, 1] if t % 2 else [2, 1, 0])
        if t == 0:
            s = buffers(most + 3)
        elif bufs is None:
            s = bufs = buffers(b + 2)
        lengths = lengths + counts
        n = int(counts.sum())
        x, xv = draws((n, width), 100 + t, 2.0)
        q, qv = draws((n, heads, width), 200 + t)
        if captured and t == 1:
            # captured before the step's inputs are in place, on a step of no tokens
            new.zero_()
            step(s)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(s)
        s["x"][:n].copy_(x)
        s["q"][:n].copy_(q)
        seq.copy_(dev(lengths))
        new.copy_(dev(counts))
        graph.replay() if graph else step(s)
        for ws in (tables_ws, store_ws, attn_ws):
            assert pkv.get_device_error(ws) == 0
        o, at = values(s["o"]), 0
        turned = values(s["q"][:n])                    # what attention read
        for r in range(b):
            k = int(counts[r])
            pos = np.arange(lengths[r] - k, lengths[r])
            c, slack = ref.normalise(xv[at:at + k, :latent], wv, 1e-6)
            pe, pslack = ref.rotate(xv[at:at + k, None, latent:], pos, rope.inv_freq, True, rope.magnitude)
            slots = table.cpu().numpy()[r, np.arange(lengths[r]) // page].astype(np.int64) * page + np.arange(lengths[r]) % page
            stored = values(pool.rows[torch.from_numpy(slots).cuda()])
            near(stored[lengths[r] - k:, :latent], c, slack)
            near(stored[lengths[r] - k:, latent:], pe[:, 0], pslack[:, 0])
            assert np.array_equal(stored[:lengths[r] - k], held[r])   # what was there stays
            held[r] = stored
            if k:
                qt, qslack = ref.rotate(qv[at:at + k, :, latent:], pos, rope.inv_freq, True, rope.magnitude)
                near(turned[at:at + k, :, latent:], qt, qslack)
                assert np.array_equal(turned[at:at + k, :, :latent], qv[at:at + k, :, :latent])
                want, bound = ref.attend(turned[at:at + k], stored, latent, float(np.float32(width ** -0.5)), pos + 1)
                assert np.all(np.abs(o[at:at + k] - want) <= bound)
            at += k
