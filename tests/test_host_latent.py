"""Refusals of the rotary and latent-pool entry points, and their host parts, without a GPU: every call here returns
before anything is enqueued."""

import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import prefix_shared_kv_token_gb300 as pkv
from prefix_shared_kv_token_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
lib = _lib.lib
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = 0x10000   # stands for a device address (never read)
INF, NAN = float("inf"), float("nan")


def spec(**kw):
    return _lib.PkvRopeSpec(**{**dict(phases=P, rotary_dim=64, interleaved=0, magnitude=1.0), **kw})


def pool(**kw):
    return _lib.PkvLatentPool(**{**dict(rows=P, num_slots=100, latent_dim=512, rope_dim=64, slot_stride=0), **kw})


def heads_pool(**kw):
    a = dict(k=P, v=P, num_slots=64, num_kv_heads=8, head_dim=128, dtype=0, k_scale=1.0, v_scale=1.0, slot_stride=0)
    return _lib.PkvPool(**{**a, **kw})


def batch(**kw):
    a = dict(req_to_token=P, stride=4, num_rows=2, req_pool_indices=P, seq_lens=P, batch=2, page_size=16)
    return _lib.PkvBatch(**{**a, **kw})


# ----------------------------------------------------------------------------------------
# rotary positions

BAD_SPECS = [(dict(phases=None), INVALID), (dict(phases=P + 4), INVALID), (dict(rotary_dim=0), UNSUPPORTED),
             (dict(rotary_dim=24), UNSUPPORTED), (dict(rotary_dim=-16), UNSUPPORTED), (dict(interleaved=2), INVALID),
             (dict(magnitude=INF), INVALID), (dict(magnitude=NAN), INVALID)]


def rope(r=None, x=P, xt=1024, xh=128, out=P, ot=1024, oh=128, heads=8, dim=128, pos=P, n=4):
    return lib.pkv_rope(C.byref(spec() if r is None else r), x, xt, xh, out, ot, oh, heads, dim, pos, n, None)


def rope_store(p=None, r=None, q=P, qt=4096, qh=128, qo=P, qot=4096, qoh=128, hq=32, k=P, kt=1024, v=P, vt=1024, pos=P, loc=P,
               n=4, ws=None):
    return lib.pkv_rope_store(C.byref(heads_pool() if p is None else p), C.byref(spec() if r is None else r), q, qt, qh, qo, qot,
                              qoh, hq, k, kt, v, vt, pos, loc, n, ws, None)


def latent_store(p=None, r=None, c=P, ct=576, pe=P, pt=576, w=P, eps=1e-6, pos=P, loc=P, n=4, ws=None):
    return lib.pkv_latent_store(C.byref(pool() if p is None else p), C.byref(spec() if r is None else r), c, ct, pe, pt, w, eps,
                                pos, loc, n, ws, None)


@pytest.mark.parametrize("change,code", BAD_SPECS)
def test_bad_specs_are_refused_by_every_call(change, code):
    r = spec(**change)
    assert rope(r) == rope_store(r=r) == latent_store(r=r) == code


def test_rope_refusals():
    for kw in (dict(x=None), dict(x=P + 8), dict(out=None), dict(out=P + 2), dict(xt=1020), dict(xh=4), dict(ot=12), dict(oh=129),
               dict(pos=None), dict(n=-1), dict(heads=-1), dict(dim=48), dict(oh=0), dict(ot=0)):
        assert rope(**kw) == INVALID, kw
    for kw in (dict(dim=132), dict(dim=520), dict(heads=65537), dict(n=1 << 40)):
        assert rope(**kw) == UNSUPPORTED, kw
    assert lib.pkv_rope(None, P, 8, 8, P, 8, 8, 1, 64, P, 1, None) == INVALID
    assert rope(n=0) == 0 and rope(heads=0) == 0       # nothing to rotate


def test_rope_store_refusals():
    for kw in (dict(q=None), dict(q=P + 4), dict(qo=None), dict(qt=4), dict(qh=100), dict(qot=0), dict(qoh=0), dict(k=None),
               dict(k=P + 8), dict(v=None), dict(kt=1025), dict(vt=4), dict(pos=None), dict(loc=None), dict(n=-1), dict(hq=-1),
               dict(ws=P + 1), dict(ws=P + 2), dict(r=spec(rotary_dim=144))):
        assert rope_store(**kw) == INVALID, kw
    assert rope_store(p=heads_pool(head_dim=96)) == UNSUPPORTED
    assert rope_store(p=heads_pool(k=None)) == INVALID
    assert rope_store(p=heads_pool(dtype=1, k_scale=0.0)) == INVALID
    assert rope_store(hq=65537) == UNSUPPORTED and rope_store(n=1 << 40) == UNSUPPORTED
    assert rope_store(n=0, q=None, k=None, v=None) == 0


def test_rope_phases():
    """2^64ths of a turn: their product with any position, modulo 2^64, is the angle's fraction of a turn."""
    f = np.array([1.0, 0.1, 1e-4, 2 * np.pi, 0.0, -0.25, 7.0, 1e-9])
    out = np.zeros(len(f), np.uint64)
    at = lambda a: a.ctypes.data_as(C.c_void_p)  # noqa: E731
    assert lib.pkv_rope_phases(at(f), len(f), at(out)) == 0
    assert out[3] == 0 and out[4] == 0
    for i, x in enumerate(f):
        for pos in (1, 3, 1000003, 2 ** 31 - 1):
            turns = (int(out[i]) * pos % 2 ** 64) / 2.0 ** 64
            want = pos * x / (2 * np.pi) % 1.0
            off = abs(turns - want)
            # a double's rounding of f / 2 pi and of the wanted value, and the phase's own last bit: a phase is a
            # multiple of 2^-64, off by half of that a position
            assert min(off, 1 - off) <= 2.0 ** -51 * max(1.0, pos * abs(x)) + pos * 2.0 ** -65, (x, pos)
    for bad in (INF, NAN):
        assert lib.pkv_rope_phases(at(np.array([1.0, bad])), 2, at(out)) == INVALID
    assert lib.pkv_rope_phases(None, 2, at(out)) == INVALID and lib.pkv_rope_phases(at(f), -1, at(out)) == INVALID
    assert lib.pkv_rope_phases(at(f), 0, at(out)) == 0


def test_rope_frequencies():
    plain = pkv.Rope(64, base=10000.0, device="cpu")
    assert plain.magnitude == 1.0 and np.allclose(plain.inv_freq, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    assert plain.phases.dtype == torch.int64 and plain.phases.shape == (32,)
    assert np.allclose(pkv.Rope(64, scaling=dict(kind="linear", factor=4), device="cpu").inv_freq, plain.inv_freq / 4, rtol=1e-15)
    ntk = pkv.Rope(64, scaling=dict(kind="ntk", factor=4), device="cpu")
    assert ntk.inv_freq[0] == 1.0 and np.isclose(ntk.inv_freq[-1], plain.inv_freq[-1] / 4, rtol=1e-12)
    yarn = pkv.Rope(64, scaling=dict(kind="yarn", factor=32, original=4096), device="cpu")
    ratio = yarn.inv_freq / plain.inv_freq
    turns = 4096 * plain.inv_freq / (2 * np.pi)          # within the original context
    assert np.all(ratio[turns > 40] == 1.0) and np.allclose(ratio[turns < 0.7], 1 / 32) and np.all(np.diff(ratio) <= 1e-15)
    assert np.isclose(yarn.magnitude, 0.1 * np.log(32) + 1)
    own = pkv.Rope(32, inv_freq=np.linspace(1, 0.1, 16), magnitude=0.5, layout="interleaved", device="cpu")
    assert own.magnitude == 0.5 and own._c.interleaved == 1 and own._c.rotary_dim == 32


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=40), dict(layout="other"), dict(base=1.0), dict(base=NAN),
                                dict(scaling=dict(kind="none")), dict(scaling=dict(kind="linear")),
                                dict(scaling=dict(kind="linear", factor=0.5)), dict(scaling=dict(kind="linear", factor=2, extra=1)),
                                dict(scaling=dict(kind="yarn", factor=2)),
                                dict(scaling=dict(kind="yarn", factor=2, original=4096, beta_fast=1, beta_slow=2)),
                                dict(inv_freq=np.ones(31)), dict(inv_freq=np.full(32, INF)), dict(magnitude=INF),
                                dict(inv_freq=np.ones(32), scaling=dict(kind="linear", factor=2))])
def test_rope_refuses(kw):
    with pytest.raises(ValueError):
        pkv.Rope(**{**dict(rotary_dim=64, device="cpu"), **kw})


# ----------------------------------------------------------------------------------------
# the latent pool

BAD_POOLS = [(dict(rows=None), INVALID), (dict(rows=P + 8), INVALID), (dict(num_slots=0), INVALID),
             (dict(num_slots=1 << 31), UNSUPPORTED), (dict(latent_dim=384), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED),
             (dict(slot_stride=568), INVALID), (dict(slot_stride=580), INVALID), (dict(slot_stride=1 << 33), UNSUPPORTED)]


@pytest.mark.parametrize("change,code", BAD_POOLS)
def test_bad_latent_pools_are_refused_by_every_call(change, code):
    p, n = pool(**change), C.c_size_t(0)
    assert latent_store(p) == code
    assert lib.pkv_latent_workspace(C.byref(p), 16, C.byref(n)) == code
    assert lib.pkv_attn_latent(C.byref(p), C.byref(batch()), P, P, 2, None, 16, 0.1, P, 1 << 40, None) == code


def test_latent_store_refusals():
    for kw in (dict(c=None), dict(c=P + 8), dict(pe=None), dict(pe=P + 2), dict(ct=577), dict(pt=4), dict(w=P + 8), dict(eps=-1.0),
               dict(eps=NAN), dict(eps=INF), dict(pos=None), dict(loc=None), dict(n=-1), dict(ws=P + 3), dict(r=spec(rotary_dim=32)),
               dict(r=spec(rotary_dim=128))):
        assert latent_store(**kw) == INVALID, kw
    assert latent_store(n=1 << 40) == UNSUPPORTED
    assert latent_store(n=0, c=None) == 0


def test_attn_latent_refusals():
    p, need = pool(), C.c_size_t(0)
    assert lib.pkv_latent_workspace(C.byref(p), 16, C.byref(need)) == 0 and need.value > 256
    for heads, code in ((0, INVALID), (-1, INVALID), (1025, UNSUPPORTED)):
        assert lib.pkv_latent_workspace(C.byref(p), heads, C.byref(need)) == code
    assert lib.pkv_latent_workspace(C.byref(p), 16, None) == INVALID
    assert lib.pkv_latent_workspace(C.byref(p), 16, C.byref(need)) == 0

    def call(q=P, o=P, total=2, qo=None, heads=16, scale=0.1, ws=P, size=1 << 40, **kw):
        return lib.pkv_attn_latent(C.byref(p), C.byref(batch(**kw)), q, o, total, qo, heads, scale, ws, size, None)

    for kw in (dict(q=None), dict(q=P + 8), dict(o=None), dict(o=P + 2), dict(total=-1), dict(total=3), dict(heads=0), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(ws=None), dict(ws=P + 128), dict(req_to_token=None),
               dict(req_pool_indices=None), dict(seq_lens=None), dict(batch=-1), dict(stride=-1), dict(stride=1 << 31),
               dict(num_rows=-1), dict(page_size=12), dict(page_size=8192)):
        assert call(**kw) == INVALID, kw
    assert call(heads=1025) == UNSUPPORTED
    assert call(total=1 << 30, qo=P, heads=2) == UNSUPPORTED
    assert call(size=need.value - 1) == WORKSPACE
    assert call(batch=0, total=0) == 0 and call(total=0, qo=P) == 0
    assert lib.pkv_attn_latent(C.byref(p), None, P, P, 2, None, 16, 0.1, P, 1 << 40, None) == INVALID


def test_latent_pool_checks_its_tensor():
    good = pkv.LatentPool.allocate(10, 256, device="cpu")
    assert good.num_slots == 10 and good.rope_dim == 64 and good._c.slot_stride == 320
    wide = torch.zeros((10, 640), dtype=torch.bfloat16)
    assert pkv.LatentPool(wide[:, :576], 512)._c.slot_stride == 640
    assert pkv.latent_workspace(good, 16) > 256
    for rows in (torch.zeros((10, 576)), wide[:, ::2], torch.zeros(576, dtype=torch.bfloat16), torch.zeros((1, 576), dtype=torch.bfloat16).expand(4, 576)):
        with pytest.raises(ValueError):
            pkv.LatentPool(rows, 512)
    with pytest.raises(pkv.PkvError):
        pkv.latent_workspace(pkv.LatentPool(wide, 512), 16)      # a rotary key of 128
    with pytest.raises(ValueError):                              # no call takes a pool in host memory
        good.c(0)
    with pytest.raises(ValueError):
        pkv.Rope(64, device="cpu").c(0)


@pytest.mark.parametrize("cls,name", [(_lib.PkvLatentPool, "pkv_latent_pool"), (_lib.PkvRopeSpec, "pkv_rope_spec")])
def test_structs_match_the_header(tmp_path, cls, name):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "pkv.h"', "int main(void) {",
             f'printf("%zu", sizeof({name}));']
    lines += [f'printf(" %zu", offsetof({name}, {f}));' for f, _ in cls._fields_] + ["return 0;", "}"]
    (tmp_path / "layout.c").write_text("\n".join(lines))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", str(tmp_path / "layout")],
                   check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == [C.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
