"""Refusals of the rotary and linear-attention calls (no GPU: every check
here returns before the device is touched), and the binding's structs."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import paged_kv_cache_291_gb300 as pkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, HEADS, HEADDIM, BLOCKSIZE, ALIAS, WORKSPACE, ALIGN = 1, 2, 3, 4, 5, 6, 7, 8
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_291_gb300 import build
    build.build()
    return pkv.load()


def rot(**kw):
    a = dict(inv_freq=64 * MB, positions=65 * MB, rot_dim=64, num_axes=1, sections=(32, 0, 0, 0), flags=0) | kw
    a["sections"] = (ctypes.c_int32 * 4)(*a["sections"])
    return pkv.Rotary(**a)


def call_rotary(lib, r=None, **kw):
    """A valid call of 4 tokens (never reached: each test breaks one argument)."""
    a = dict(q=MB, qs=512, hq=8, k=2 * MB, ks=128, hkv=2, d=64, T=4, q_out=3 * MB, k_out=4 * MB) | kw
    r = rot() if r is None else r
    return lib.pkv_rotary(ctypes.byref(r), a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["hkv"], a["d"], a["T"],
                          a["q_out"], a["k_out"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL),
    (dict(T=-1), SHAPE), (dict(qs=504), SHAPE), (dict(ks=132), SHAPE), (dict(qs=-512), SHAPE),
    (dict(hq=0), HEADS), (dict(hkv=0), HEADS), (dict(d=96), HEADDIM),
    (dict(q=MB + 8), ALIGN), (dict(k_out=4 * MB + 2), ALIGN),
    (dict(q_out=MB + 16), ALIAS),                  # overlaps q
    (dict(qs=1024, q_out=MB), ALIAS),              # in place, but q is not contiguous
    (dict(k_out=3 * MB), ALIAS),                   # the outputs overlap
    (dict(q_out=2 * MB), ALIAS),                   # q_out over k
    (dict(k_out=MB), ALIAS),                       # k_out over q
])
def test_rotary_arguments(lib, kw, want):
    assert call_rotary(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=128, sections=(64, 0, 0, 0)), dict(num_axes=0), dict(num_axes=5),
    dict(sections=(31, 0, 0, 0)), dict(num_axes=2, sections=(33, -1, 0, 0)), dict(flags=4), dict(flags=-1),
    dict(num_axes=1, sections=(16, 16, 0, 0)), dict(rot_dim=-16, sections=(-8, 0, 0, 0)),
])
def test_rotary_descriptor_shapes(lib, kw):
    assert call_rotary(lib, rot(**kw)) == SHAPE


def test_rotary_descriptor_pointers_and_empty_batch(lib):
    assert call_rotary(lib, rot(inv_freq=None)) == NULL
    assert call_rotary(lib, rot(positions=None)) == NULL
    assert lib.pkv_rotary(None, MB, 512, 8, MB, 128, 2, 64, 4, MB, MB, None) == NULL
    assert call_rotary(lib, T=0, q=None, k=None, q_out=None, k_out=None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(v=None), NULL), (dict(slots=None), NULL), (dict(q_out=None), NULL), (dict(vs=120), SHAPE),
    (dict(T=-2), SHAPE), (dict(v=5 * MB + 4), ALIGN), (dict(q_out=16 * MB), ALIAS), (dict(k=16 * MB), ALIAS),
    (dict(v_pool=16 * MB), ALIAS), (dict(q_out=5 * MB), ALIAS), (dict(bs=32), BLOCKSIZE), (dict(pd=80), HEADDIM),
])
def test_rotary_cache_write_arguments(lib, kw, want):
    a = dict(q=MB, qs=512, hq=8, k=2 * MB, ks=128, v=5 * MB, vs=128, T=4, q_out=3 * MB, slots=6 * MB,
             v_pool=17 * MB, bs=16, pd=64) | kw
    c = pkv.Cache(16 * MB, a["v_pool"], 16, 2, a["pd"], a["bs"], 0, 1.0, 1.0)
    r = rot()
    got = lib.pkv_rotary_cache_write(ctypes.byref(c), ctypes.byref(r), a["q"], a["qs"], a["hq"], a["k"], a["ks"],
                                     a["v"], a["vs"], a["slots"], a["T"], a["q_out"], None)
    assert got == want


LINEAR = [
    (dict(states=None), NULL), (dict(log_decay=None), NULL), (dict(q=None), NULL), (dict(k=None), NULL),
    (dict(v=None), NULL), (dict(slots=None), NULL), (dict(ctx=None), NULL), (dict(out=None), NULL),
    (dict(n=-1), SHAPE), (dict(num_slots=-1), SHAPE), (dict(qs=1016), SHAPE), (dict(ks=260), SHAPE),
    (dict(vs=128), SHAPE), (dict(hkv=0), SHAPE), (dict(hq=6), HEADS), (dict(hq=32), HEADS), (dict(d=32), HEADDIM),
    (dict(states=9 * MB + 4), ALIGN), (dict(q=MB + 2), ALIGN), (dict(out=7 * MB + 8), ALIGN),
]


def linear_args(kw):
    return dict(states=9 * MB, log_decay=8 * MB, num_slots=4, hkv=2, d=128, q=MB, qs=1024, hq=8, k=2 * MB, ks=256,
                v=3 * MB, vs=256, slots=4 * MB, new=None, ctx=5 * MB, n=3, out=7 * MB) | kw


@pytest.mark.parametrize("kw,want", LINEAR)
def test_linear_decode_arguments(lib, kw, want):
    a = linear_args(kw)
    s = pkv.States(a["states"], a["log_decay"], a["num_slots"], a["hkv"], a["d"])
    got = lib.pkv_linear_decode_attention(ctypes.byref(s), a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["v"], a["vs"],
                                          a["slots"], a["new"], a["ctx"], a["n"], 1.0, a["out"], None)
    assert got == want


@pytest.mark.parametrize("kw,want", LINEAR + [
    (dict(qsl=None), NULL), (dict(host=None), NULL), (dict(T=-1), SHAPE), (dict(host=[0, 5, 5, 11]), SHAPE),
    (dict(host=[1, 5, 5, 10]), SHAPE), (dict(host=[0, 6, 5, 10]), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(ws=10 * MB + 128), WORKSPACE), (dict(ws_bytes=255), WORKSPACE),
])
def test_linear_prefill_arguments(lib, kw, want):
    a = linear_args(kw) | dict(T=10, qsl=6 * MB, host=[0, 5, 5, 10], ws=10 * MB, ws_bytes=1 << 40) | kw
    s = pkv.States(a["states"], a["log_decay"], a["num_slots"], a["hkv"], a["d"])
    host = np.array(a["host"], np.int32) if a["host"] is not None else None
    got = lib.pkv_linear_prefill_attention(
        ctypes.byref(s), a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["qsl"],
        host.ctypes.data_as(ctypes.c_void_p) if host is not None else None, a["slots"], a["new"], a["ctx"], a["n"], 1.0,
        a["out"], a["ws"], a["ws_bytes"], None)
    assert got == want


def test_linear_empty_batches_and_null_descriptor(lib):
    s = pkv.States(9 * MB, 8 * MB, 4, 2, 128)
    none = [None] * 2
    assert lib.pkv_linear_decode_attention(ctypes.byref(s), None, 0, 8, None, 0, None, 0, None, None, None, 0, 1.0,
                                           None, None) == 0
    assert lib.pkv_linear_prefill_attention(ctypes.byref(s), None, 0, 8, None, 0, None, 0, 0, *none, None, None, None,
                                            3, 1.0, None, None, 0, None) == 0
    assert lib.pkv_linear_decode_attention(None, None, 0, 8, None, 0, None, 0, None, None, None, 0, 1.0, None,
                                           None) == NULL


@pytest.mark.parametrize("args", [(-1, 5, 8, 2, 128), (1, -5, 8, 2, 128), (1, 5, 6, 2, 128), (1, 5, 8, 2, 96)])
def test_linear_workspace_size_of_bad_shapes(lib, args):
    assert lib.pkv_linear_prefill_workspace_size(*args) == 0


def test_structs_match_the_header(tmp_path):
    structs = {"pkv_rotary_t": pkv.Rotary, "pkv_states_t": pkv.States}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "pkv.h"', 'int main(void) {']
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ['return 0; }']))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    got = {tuple(ln.split()[:2]): int(ln.split()[2]) for ln in out if ln}
    for cname, py in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset
