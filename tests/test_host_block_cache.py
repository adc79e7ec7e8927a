"""Refusals of the block-scaled cache's entry points, on the host: every call here returns before
anything is enqueued, so none needs a GPU."""

import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

import prefix_shared_kv_token_gb300 as pkv
from prefix_shared_kv_token_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
lib = _lib.lib
INVALID, UNSUPPORTED, WORKSPACE, PLAN = -1, -2, -3, -8
P = 0x10000   # stands for a device address (never read)


def pool(**kw):
    a = dict(k=P, v=P, k_exp=P, v_exp=P, num_pages=8, page_size=16, num_kv_heads=8, head_dim=128, slot_stride=0)
    return _lib.PkvBlockPool(**{**a, **kw})


def batch(**kw):
    a = dict(req_to_token=P, stride=4, num_rows=2, req_pool_indices=P, seq_lens=P, batch=2, page_size=16)
    return _lib.PkvBatch(**{**a, **kw})


BAD_POOLS = [
    (dict(k=None), INVALID), (dict(v_exp=None), INVALID), (dict(num_pages=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED), (dict(num_pages=1 << 62), UNSUPPORTED),
    (dict(k=P + 8), INVALID), (dict(slot_stride=512), INVALID), (dict(slot_stride=1032), INVALID),
]


@pytest.mark.parametrize("change,code", BAD_POOLS)
def test_bad_pools_are_refused_by_every_call(change, code):
    p, b, info = pool(**change), batch(), _lib.PkvPlanInfo()
    n = C.c_size_t(0)
    assert lib.pkv_kv_store_block(C.byref(p), P, P, P, 4, None, None) == code
    assert lib.pkv_decode_block_workspace(C.byref(p), 32, C.byref(n)) == code
    assert lib.pkv_attn_decode_block(C.byref(p), C.byref(b), P, P, 32, 0.1, P, 1 << 40, None) == code
    assert lib.pkv_attn_extend_block(C.byref(p), C.byref(b), P, P, 0.1, C.byref(info), P, P, 1 << 40, None) == code


def test_store_refusals():
    p = pool()
    assert lib.pkv_kv_store_block(None, P, P, P, 4, None, None) == INVALID
    assert lib.pkv_kv_store_block(C.byref(p), P, P, P, -1, None, None) == INVALID
    assert lib.pkv_kv_store_block(C.byref(p), P, P, P, 1 << 31, None, None) == INVALID
    assert lib.pkv_kv_store_block(C.byref(p), P, P, None, 4, None, None) == INVALID
    assert lib.pkv_kv_store_block(C.byref(p), P + 2, P, P, 4, None, None) == INVALID
    assert lib.pkv_kv_store_block(C.byref(p), None, None, None, 0, None, None) == 0   # nothing to store


def test_decode_refusals():
    p = pool()
    need = C.c_size_t(0)
    assert lib.pkv_decode_block_workspace(C.byref(p), 32, C.byref(need)) == 0 and need.value > 256
    assert lib.pkv_decode_block_workspace(C.byref(p), 32, None) == INVALID

    def call(b=None, q=P, o=P, hq=32, ws=P, size=1 << 40, **kw):
        b = batch(**kw) if b is None else b
        return lib.pkv_attn_decode_block(C.byref(p), C.byref(b), q, o, hq, 0.1, ws, size, None)

    for hq, code in ((0, INVALID), (12, INVALID), (24, UNSUPPORTED), (128, UNSUPPORTED)):
        assert call(hq=hq) == code
        assert lib.pkv_decode_block_workspace(C.byref(p), hq, C.byref(need)) == code
    assert lib.pkv_decode_block_workspace(C.byref(p), 32, C.byref(need)) == 0
    assert call(size=need.value - 1) == WORKSPACE
    assert call(page_size=32) == INVALID          # not the pool's
    assert call(page_size=1) == INVALID
    assert call(batch=-1) == INVALID
    assert call(stride=-1) == INVALID and call(stride=1 << 31) == INVALID
    for name in ("req_to_token", "req_pool_indices", "seq_lens"):
        assert call(**{name: None}) == INVALID
    assert call(q=None) == INVALID and call(o=None) == INVALID and call(ws=None) == INVALID
    assert call(q=P + 8) == INVALID and call(o=P + 2) == INVALID and call(ws=P + 16) == INVALID
    assert call(batch=0) == 0                     # an empty batch is nothing to do


def test_extend_refusals():
    p = pool()
    plan = pkv.plan_extend([40], [8], [0, 8], 32, 8, 128)
    fused = pkv.plan_extend([40], [8], [0, 8], 32, 8, 128, opts={"fuse_store": 1})
    other = pkv.plan_extend([40], [8], [0, 8], 32, 4, 128)

    def call(plan=plan, size=1 << 40, **kw):
        b = batch(**{"batch": 1, **kw})
        return lib.pkv_attn_extend_block(C.byref(p), C.byref(b), P, P, 0.1, C.byref(plan.info), P, P, size, None)

    assert call(page_size=32) == INVALID
    assert call(plan=fused) == PLAN and call(plan=other) == PLAN and call(batch=2) == PLAN
    assert call(plan=pkv.plan_decode([40], 32, 8, 128)) == PLAN
    assert call(size=plan.info.workspace_bytes - 1) == WORKSPACE
    assert lib.pkv_attn_extend_block(C.byref(p), None, P, P, 0.1, C.byref(plan.info), P, P, 1 << 40, None) == INVALID


def test_extend_refuses_a_scale_that_is_not_positive():
    p, b = pool(), batch(batch=1)
    for tokens, seq in ((8, 40), (1, 9000)):      # gathered, streams
        plan = pkv.plan_extend([seq], [tokens], [0, tokens], 32, 8, 128)
        for scale in (0.0, -0.1, float("nan"), float("inf")):
            assert lib.pkv_attn_extend_block(C.byref(p), C.byref(b), P, P, scale, C.byref(plan.info), P, P, 1 << 40,
                                             None) == INVALID


@pytest.mark.parametrize("hkv,g,d", [(1, 1, 64), (1, 8, 128), (2, 4, 64), (3, 2, 128), (8, 1, 128), (16, 4, 64)])
def test_extend_streams_fit_the_plans_workspace(hkv, g, d):
    """Short contexts, whose gathered rows are smaller than one range's two records of 8 columns for a
    group of up to 8 heads: such a plan gathers."""
    hg = max(x for x in (8, 4, 2, 1) if hkv % x == 0)
    streams = 0
    for b in (1, 2, 7, 40):
        for seq, ext in ((1, 1), (2, 1), (5, 5), (17, 3), (130, 2), (1000, 1)):
            plan = pkv.plan_extend([seq] * b, [ext] * b, [i * ext for i in range(b + 1)], hkv * g, hkv, d)
            if plan.info.offsets[18]:
                streams += 1
                assert plan.info.workspace_bytes - 256 >= 2 * hg * 8 * (d + 4) * 4
    assert streams


def test_table_refusals():
    def call(new=P, free=P, num_free=5, head=P, head_out=P, loc=P, pos=P, cap=4, indptr=P, ws=P, size=256, **kw):
        b = batch(**kw)
        return lib.pkv_build_block_tables(C.byref(b), new, free, num_free, head, head_out, loc, pos, cap, indptr, ws,
                                          size, None)
    for kw in (dict(new=None), dict(free=None), dict(num_free=-1), dict(num_free=1 << 31), dict(head=None),
               dict(head_out=None), dict(loc=None), dict(pos=None), dict(cap=-1), dict(cap=1 << 31), dict(indptr=None),
               dict(ws=None), dict(ws=P + 2), dict(batch=-1), dict(stride=-1), dict(stride=1 << 31), dict(num_rows=-1),
               dict(req_to_token=None), dict(req_pool_indices=None), dict(seq_lens=None), dict(page_size=12),
               dict(page_size=8192)):
        assert call(**kw) == INVALID, kw
    assert call(size=255) == WORKSPACE
    assert call(batch=16385) == UNSUPPORTED


def test_block_pool_checks_its_tensors():
    good = pkv.BlockPool.allocate(4, 16, 2, 64, device="cpu")
    assert good.num_pages == 4 and good._c.slot_stride == 128
    both = pkv.BlockPool.allocate(4, 16, 2, 64, device="cpu", layout="interleaved")
    assert both._c.slot_stride == 256 and both._c.v == both._c.k + 128
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t)  # noqa: E731
    for args in ((z(64, 2, 64), z(64, 2, 64), z(4, 2), z(4, 3), 16), (z(64, 2, 64), z(48, 2, 64), z(4, 2), z(4, 2), 16),
                 (z(60, 2, 64), z(60, 2, 64), z(3, 2), z(3, 2), 16), (z(64, 128), z(64, 128), z(4, 2), z(4, 2), 16),
                 (z(64, 2, 64, t=torch.int8), z(64, 2, 64), z(4, 2), z(4, 2), 16),
                 (z(64, 2, 64), z(64, 2, 64), z(4, 2, t=torch.float32), z(4, 2), 16),
                 (z(64, 64, 2).transpose(1, 2), z(64, 64, 2).transpose(1, 2), z(4, 2), z(4, 2), 16),
                 (z(64, 2, 64), z(64, 2, 64), z(2, 4).T, z(4, 2), 16)):
        with pytest.raises(ValueError):
            pkv.BlockPool(*args)
    with pytest.raises(ValueError):
        pkv.BlockPool.allocate(4, 16, 2, 64, device="cpu", layout="striped")
    with pytest.raises(ValueError):    # no call takes a pool in host memory
        good.c(0)
    assert pkv.decode_block_workspace(good, 8) > 256
    with pytest.raises(pkv.PkvError):
        pkv.decode_block_workspace(good, 7)


def test_block_pool_struct_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    cls = _lib.PkvBlockPool
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "pkv.h"', "int main(void) {",
             'printf("%zu", sizeof(pkv_block_pool));']
    lines += [f'printf(" %zu", offsetof(pkv_block_pool, {f}));' for f, _ in cls._fields_] + ["return 0;", "}"]
    (tmp_path / "layout.c").write_text("\n".join(lines))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", str(tmp_path / "layout")],
                   check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == [C.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


@pytest.mark.parametrize("offset", [16, 64, 112])
def test_a_pool_at_any_16_byte_address_is_taken_by_every_call(offset):
    """Each call gets past the pool to the refusal of what comes after it."""
    p, b = pool(k=P + offset, v=P + offset, num_kv_heads=8), batch(batch=1)
    assert lib.pkv_kv_store_block(C.byref(p), P + 2, P, P, 4, None, None) == INVALID
    assert lib.pkv_kv_store_block(C.byref(p), None, None, None, 0, None, None) == 0
    need = C.c_size_t(0)
    assert lib.pkv_decode_block_workspace(C.byref(p), 32, C.byref(need)) == 0
    assert lib.pkv_attn_decode_block(C.byref(p), C.byref(b), P, P, 32, 0.1, P, need.value - 1, None) == WORKSPACE
    for tokens, seq in ((8, 40), (1, 9000)):      # gathered, streams
        plan = pkv.plan_extend([seq], [tokens], [0, tokens], 32, 8, 128)
        assert plan.info.offsets[18] == (tokens == 1)
        assert lib.pkv_attn_extend_block(C.byref(p), C.byref(b), P, P, 0.1, C.byref(plan.info), P, P,
                                         plan.info.workspace_bytes - 1, None) == WORKSPACE


def test_store_refuses_an_error_word_that_is_not_aligned():
    p = pool()
    for at in (1, 2, 3):
        assert lib.pkv_kv_store_block(C.byref(p), P, P, P, 4, P + at, None) == INVALID
