"""Refusals of the calls on 8-bit pools with a scale per block and head (no
GPU: every check here returns before the device is touched)."""
import ctypes
import os
import subprocess

import pytest
import torch

import paged_kv_cache_291_gb300 as pkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, HEADS, HEADDIM, BLOCKSIZE, ALIAS, WORKSPACE, ALIGN, DTYPE = 1, 2, 3, 4, 5, 6, 7, 8, 16
MB = 1 << 20
E4M3, INT8 = pkv.PKV_KV_E4M3_BLOCKS, pkv.PKV_KV_INT8_BLOCKS


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_291_gb300 import build
    build.build()
    return pkv.load()


def cache(**kw):
    a = dict(k_pool=64 * MB, v_pool=80 * MB, num_blocks=16, num_kv_heads=2, head_dim=64, block_size=16, kv_dtype=INT8,
             k_scale=0.0, v_scale=0.0, block_scales=96 * MB) | kw
    return pkv.Cache(*(a[f] for f, _ in pkv.Cache._fields_))


def append(lib, c=None, **kw):
    """A valid call of 4 rows (never reached: each test breaks one argument)."""
    a = dict(k=MB, ks=128, v=2 * MB, vs=128, T=4, start=3 * MB, lens=4 * MB, S=2, tables=5 * MB, wide=3) | kw
    return lib.pkv_cache_append(ctypes.byref(c or cache()), a["k"], a["ks"], a["v"], a["vs"], a["T"], a["start"],
                                a["lens"], a["S"], a["tables"], a["wide"], None)


def read(lib, c=None, **kw):
    a = dict(k=MB, v=2 * MB, T=4, start=3 * MB, lens=4 * MB, S=2, tables=5 * MB, wide=3) | kw
    return lib.pkv_cache_read(ctypes.byref(c or cache()), a["k"], a["v"], a["T"], a["start"], a["lens"], a["S"],
                              a["tables"], a["wide"], None)


DESCRIPTORS = [
    (dict(k_pool=None), NULL), (dict(v_pool=None), NULL), (dict(block_scales=None), NULL),
    (dict(block_scales=96 * MB + 8), ALIGN), (dict(k_pool=64 * MB + 8), ALIGN), (dict(block_size=32), BLOCKSIZE),
    (dict(num_blocks=-1), SHAPE), (dict(num_kv_heads=0), SHAPE), (dict(head_dim=96), HEADDIM), (dict(kv_dtype=4), DTYPE),
    (dict(kv_dtype=-1), DTYPE),
]


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("kw,want", DESCRIPTORS)
def test_descriptors(lib, kw, want, kind):
    kw = dict(kv_dtype=kind) | kw
    assert append(lib, cache(**kw)) == want
    assert read(lib, cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(start=None), NULL), (dict(lens=None), NULL),
    (dict(tables=None), NULL), (dict(T=-1), SHAPE), (dict(S=-1), SHAPE), (dict(wide=-1), SHAPE), (dict(ks=120), SHAPE),
    (dict(vs=132), SHAPE), (dict(ks=-128), SHAPE), (dict(k=MB + 8), ALIGN), (dict(v=2 * MB + 2), ALIGN),
    (dict(S=2 ** 30), SHAPE),
    (dict(k=64 * MB), ALIAS), (dict(v=80 * MB + 64), ALIAS), (dict(k=96 * MB), ALIAS),
])
def test_append_arguments(lib, kw, want):
    assert append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(start=None), NULL), (dict(lens=None), NULL),
    (dict(tables=None), NULL), (dict(T=-1), SHAPE), (dict(S=-1), SHAPE), (dict(wide=-1), SHAPE),
    (dict(k=MB + 8), ALIGN), (dict(k=2 * MB + 16), ALIAS), (dict(v=64 * MB), ALIAS), (dict(k=80 * MB), ALIAS),
    (dict(v=96 * MB), ALIAS),
])
def test_read_arguments(lib, kw, want):
    assert read(lib, **kw) == want


def test_nothing_to_do(lib):
    for kw in (dict(T=0), dict(S=0)):
        assert append(lib, k=None, v=None, start=None, **kw) == 0
        assert read(lib, k=None, v=None, start=None, **kw) == 0


def test_pools_that_overlap(lib):
    assert append(lib, cache(v_pool=64 * MB + 16)) == ALIAS
    assert append(lib, cache(block_scales=64 * MB)) == ALIAS


@pytest.mark.parametrize("kind", [pkv.PKV_KV_BF16, pkv.PKV_KV_E4M3])
def test_append_takes_pools_with_block_scales_only(lib, kind):
    assert append(lib, cache(kv_dtype=kind, k_scale=1.0, v_scale=1.0)) == DTYPE


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_calls_that_store_rows_one_by_one_refuse_the_pools(lib, kind):
    c = ctypes.byref(cache(kv_dtype=kind))
    assert lib.pkv_cache_write(c, MB, 2 * MB, 3 * MB, 4, None) == DTYPE
    assert lib.pkv_decode_step(c, MB, 2 * MB, 3 * MB, 4 * MB, 4, 5 * MB, 3, 6 * MB, 2, 40, 1.0, 7 * MB, 8 * MB, MB, 0,
                               None) == DTYPE
    r = pkv.Rotary(64 * MB, 65 * MB, 64, 1, (ctypes.c_int32 * 4)(32, 0, 0, 0), 0)
    assert lib.pkv_rotary_cache_write(c, ctypes.byref(r), MB, 256, 4, 2 * MB, 128, 3 * MB, 128, 4 * MB, 4, 5 * MB,
                                      None) == DTYPE


def test_chunked_prefill_still_refuses_a_pool_with_one_scale(lib):
    c = cache(kv_dtype=pkv.PKV_KV_E4M3, k_scale=1.0, v_scale=1.0)
    assert lib.pkv_chunked_prefill_attention(ctypes.byref(c), MB, 4, 4, 2 * MB, None, 3 * MB, 1, 4 * MB, 3, 40, 1.0,
                                             5 * MB, 6 * MB, MB, None) == DTYPE


def test_attention_heads_and_descriptor(lib):
    def decode(c, hq):
        return lib.pkv_decode_attention(ctypes.byref(c), MB, hq, 2 * MB, 3, 3 * MB, 0, 40, 1.0, 4 * MB, None, 0, 0, None)
    def decode_some(c):
        return lib.pkv_decode_attention(ctypes.byref(c), MB, 4, 2 * MB, 3, 3 * MB, 2, 40, 1.0, 4 * MB, None, 0, 0, None)
    assert decode_some(cache(num_blocks=0)) == SHAPE and decode_some(cache(num_blocks=2 ** 31 - 1)) == SHAPE
    assert decode(cache(), 4) == 0 and decode(cache(), 6) == HEADS and decode(cache(block_scales=None), 4) == NULL


def test_descriptor_struct_matches_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "pkv.h"', 'int main(void) {',
             'printf("size %zu\\n", sizeof(pkv_cache_t));']
    lines += [f'printf("{f} %zu\\n", offsetof(pkv_cache_t, {f}));' for f, _ in pkv.Cache._fields_]
    lines.append('printf("kinds %d\\n", PKV_KV_E4M3_BLOCKS * 10 + PKV_KV_INT8_BLOCKS); return 0; }')
    (tmp_path / "layout.c").write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o",
                    str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split("\n")
    got = {ln.split()[0]: int(ln.split()[1]) for ln in out if ln}
    assert got.pop("size") == ctypes.sizeof(pkv.Cache) and got.pop("kinds") == E4M3 * 10 + INT8
    assert got == {f: getattr(pkv.Cache, f).offset for f, _ in pkv.Cache._fields_}


def calls_without_block_scales(k, v):
    """Every call that takes a pool, with valid arguments but for int8 pools that come without their scales."""
    i32 = torch.zeros(2, dtype=torch.int32)
    tables, rows = torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    attend = (rows, tables, i32[:1], 16, 0.125)
    one = dict(k_scale=1.0, v_scale=1.0)
    host = torch.zeros(2 * 2 * 16 * 64, dtype=torch.int8)
    return {
        "cache_write": lambda: pkv.cache_write(k, v, rows, rows, i32[:1], **one),
        "cache_read": lambda: pkv.cache_read(k, v, i32, i32[:1], tables, 1, **one),
        "copy_blocks": lambda: pkv.copy_blocks(k, v, i32[:1], i32[:1]),
        "swap_out": lambda: pkv.swap_out(k, v, i32[:1], i32[:1], host),
        "swap_in": lambda: pkv.swap_in(k, v, i32[:1], i32[:1], host),
        "decode_attention": lambda: pkv.decode_attention(k, v, *attend, **one),
        "decode_step": lambda: pkv.decode_step(k, v, rows, rows, i32[:1], *attend, **one),
        "decode_attention_shared_prefix": lambda: pkv.decode_attention_shared_prefix(
            k, v, rows, tables, i32[:1], 16, 0, 0.125, **one),
        "chunked_prefill_attention": lambda: pkv.chunked_prefill_attention(k, v, rows, i32, i32[:1], tables, 16, 0.125),
        "rotary_cache_write": lambda: pkv.rotary_cache_write(
            k, v, rows, rows, rows, i32[:1], torch.zeros((1, 1), dtype=torch.int32), torch.zeros(32), 64, **one),
    }


@pytest.mark.parametrize("call", calls_without_block_scales(None, None))
@pytest.mark.parametrize("which", ["both", "k", "v"])
def test_int8_pools_without_their_scales(lib, monkeypatch, call, which):
    """int8 codes are not e4m3 codes, and a copy that leaves the scales behind has lost the rows."""
    monkeypatch.setattr(pkv, "_device", lambda: 0)
    k, v = (torch.zeros((1, 2, 16, 64), dtype=torch.int8 if which in ("both", x) else torch.uint8) for x in "kv")
    with pytest.raises(TypeError, match="int8 pool needs block_scales"):
        calls_without_block_scales(k, v)[call]()
