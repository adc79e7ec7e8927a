"""Plain 64-bit forms of the block-scaled cache's operators, and the error bounds their kernels
are held to.  Test infrastructure: it shares no code with the library."""

import numpy as np

from oracle.fp8 import e4m3_decode, e4m3_encode

E_MIN, E_MAX = -117, 118


def bf16_bits(x):
    """float -> bf16 bit patterns (round to nearest even; finite input)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def page_exponent(x):
    """The smallest exponent with max |x| <= 448 * 2^e over the finite values of x."""
    a = np.abs(x[np.isfinite(x)])
    amax = float(a.max()) if a.size else 0.0
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def store(codes, exps, x, loc, page):
    """In place: rows x [n, heads, d] (float64) into the slots loc.  A run is tokens at consecutive
    slots of a page; a token with no slot of the pool is skipped and leaves its row out of the run."""
    ok = [0 <= s < len(codes) for s in loc]
    done = [False] * len(loc)
    for i in range(len(loc)):
        if not ok[i] or done[i]:
            continue
        block, off = loc[i] // page, loc[i] % page
        run = [i]
        for j in range(i + 1, min(i + page - off, len(loc))):
            if ok[j] and loc[j] != loc[i] + j - i:
                break
            if ok[j]:
                run.append(j)
        for j in run:
            done[j] = True
        slots = [loc[j] for j in run]
        for h in range(codes.shape[1]):
            e = page_exponent(x[run, h])
            old = int(np.clip(exps[block, h], 10, 245)) - 127
            if off and old >= e:
                e = old
            elif off:
                rows = slice(loc[i] - off, loc[i])
                codes[rows, h] = e4m3_encode(e4m3_decode(codes[rows, h]) * 2.0 ** (old - e))
            exps[block, h] = e + 127
            # past 448 it saturates (infinities too)
            codes[slots, h] = e4m3_encode(np.clip(x[run, h] * 2.0 ** -e, -1024.0, 1024.0))


def rows_of(codes, exps, table_row, length, page):
    """float64 values [length, heads, d] of a request's positions."""
    t = np.arange(length)
    pages = np.asarray(table_row, np.int64)[t // page]
    ok = (pages >= 0) & (pages < len(exps))
    pages = np.where(ok, pages, 0)
    e = np.clip(exps[pages].astype(np.int64), 10, 245) - 127
    v = e4m3_decode(codes[pages * page + t % page]) * 2.0 ** e[..., None].astype(np.float64)
    return np.where(ok[:, None, None], v, 0.0)


def exponents_of(exps, table_row, length, page):
    """The exponent [length, heads] of each position's page (0 where the page is outside the pool)."""
    pages = np.asarray(table_row, np.int64)[np.arange(length) // page]
    ok = (pages >= 0) & (pages < len(exps))
    return np.where(ok[:, None], np.clip(exps[np.where(ok, pages, 0)].astype(np.int64), 10, 245) - 127, 0)


def tables(table, rows, seq, new, free, head, page, cap):
    """(table, out_cache_loc, positions, qo_indptr, head) after the step."""
    table = table.copy()
    loc, pos = np.full(cap, -1, np.int64), np.full(cap, -1, np.int64)
    indptr, i = [0], 0
    for row, s, n in zip(rows, seq, new):
        had, has = -(-(s - n) // page), -(-s // page)
        table[row, had:has] = free[head:head + has - had]
        head += has - had
        for t in range(s - n, s):
            loc[i], pos[i] = int(table[row, t // page]) * page + t % page, t
            i += 1
        indptr.append(i)
    return table, loc, pos, np.array(indptr), head


def attend(q, k, v, scale, positions, weight_eps, log_weight_eps=0.0, v_exp=None):
    """(o, bound): attention of queries q [n, Hq, d] at `positions` over k, v [L, Hkv, d] and how
    far a kernel's bf16 output may be from it, element by element.

    The kernel's errors: (1) its output's rounding, half a bf16 step, 2^-8 of the result;
    (2) each weight w_j carries a relative error of weight_eps plus log_weight_eps |ln(w_j / w_max)|
    (rounding the weight, and rounding the exponent it is computed from), which moves the result by
    at most sum_j p_j err_j |v_j - o|, the normalisation included, where the sum takes the same weights,
    and sum_j p_j err_j |v_j| where it takes them unrounded (the kernels that v_exp is given for:
    d(sum w v / l) = sum dw v / l with l as it is; a lone key's weight is then not cancelled); (3) a logit, an fp32 sum of d
    products, is off by at most (d + 4) 2^-24 sum |q_i k_i| times the scale, and so is ln w_j, with
    the fp32 exponential's 2^-22 beside it; (4) the fp32 sum over the keys: L 2^-24 sum p |v|;
    (5) where v_exp [L, hkv] (V's exponents) is given, weights are f16: 2^6 2^(s_j + e_j - R) with
    R <= max (s_j + e_j), s in log2 units, times the code v_j 2^-e_j.  f16's smallest step is 2^-24, so
    such a weight is also off by up to 2^-25, whatever its size, which moves the result by at most
    2^-31 2^R / sum 2^s_j times sum |code_j|, largest for the largest R."""
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    o, bound = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        m = min(int(positions[i]) + 1, length)
        if m <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:m, h * hkv // hq], v[:m, h * hkv // hq]
            s = kk @ q[i, h] * scale
            top = s.max()
            w = np.exp(s - top)
            p = w / w.sum()
            o[i, h] = p @ vv
            logit = (d + 4) * 2.0 ** -24 * (np.abs(kk) @ np.abs(q[i, h])) * abs(scale)
            err = weight_eps + log_weight_eps * (top - s) + 2 * logit.max() + 2.0 ** -21
            bound[i, h] = (2.0 ** -8 * np.abs(o[i, h]) + (p * err) @ np.abs(vv - (o[i, h] if v_exp is None else 0.0))
                           + m * 2.0 ** -24 * (p @ np.abs(vv)) + 1e-37)
            if v_exp is not None:
                e = v_exp[:m, h * hkv // hq].astype(np.float64)
                log2p = (s - top) / np.log(2.0) - np.log2(w.sum())
                bound[i, h] += 2.0 ** -31 * 2.0 ** (log2p + e).max() * np.abs(vv * 2.0 ** -e[:, None]).sum(0)
    return o, bound
