"""A library whose torch binding is missing, or built for another torch,
serves every call: the binding only shortens the host's part of some."""
import subprocess
import sys
import textwrap
import warnings

import pytest

from conftest import ROOT

HIDE = """
import sys
sys.modules["paged_kv_cache_291_gb300._binding"] = None  # its import raises ImportError
sys.path[:0] = [%r, %r]
import warnings
import numpy as np
import torch
import paged_kv_cache_291_gb300 as pkv
""" % (ROOT, ROOT + "/tests")


def run(body):
    r = subprocess.run([sys.executable, "-c", HIDE + textwrap.dedent(body)], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.split()[-1:] == ["done"], r.stdout + r.stderr


def test_the_library_loads_without_the_binding():
    from paged_kv_cache_291_gb300 import build
    build.build()
    run("""
        with warnings.catch_warnings():
            warnings.simplefilter("error")  # nothing is said to who does not need it
            assert pkv.version()
            assert pkv.common_prefix_blocks(np.zeros((2, 3), np.int32), np.array([48, 48], np.int32)) == 3
        print("done")
        """)


def test_the_calls_that_use_it_say_so_once_and_check_their_arguments():
    run("""
        q, k = torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 1, 64), dtype=torch.bfloat16)
        pos, f = torch.zeros(2, dtype=torch.int32), torch.zeros(32)
        pkv._device = lambda: 0
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            for _ in range(2):
                try:
                    pkv.rotary(q, k, pos, f)
                except ValueError as e:
                    assert "CUDA" in str(e), e
                else:
                    raise SystemExit("taken")
        assert [w.category for w in seen] == [RuntimeWarning] and "_binding" in str(seen[0].message), seen
        print("done")
        """)


def test_the_binding_is_used_where_it_is_there():
    import paged_kv_cache_291_gb300 as pkv
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert pkv._fast().__name__.endswith("_binding")


@pytest.mark.gpu
def test_results_are_the_same_without_the_binding():
    run("""
        from test_gpu_linear import Batch
        from gpu_helpers import dev_tensor
        warnings.simplefilter("ignore")
        f = dev_tensor((10000.0 ** (-np.arange(32) / 32.0)).astype(np.float32))

        def all_calls():
            a, b = Batch(600, [1] * 3, [2] * 3, 4, 2, 64), Batch(601, [90, 2, 300], [0, 3, 3], 4, 2, 64)
            pos = torch.arange(b.T, dtype=torch.int32, device="cuda")
            out = [a.decode(pkv), b.prefill(pkv), a.states, b.states]
            out += pkv.rotary(b.q, b.k, pos, f)
            pools = [torch.zeros((30, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            out += [pkv.rotary_cache_write(*pools, b.q, b.k, b.v, pos, pos, f)] + pools
            torch.cuda.synchronize()
            assert pkv.get_error() == (0, 0)
            return out

        without = all_calls()
        assert pkv._calls is pkv._NoCalls
        del sys.modules["paged_kv_cache_291_gb300._binding"]
        pkv._calls = None
        with_it = all_calls()
        assert pkv._calls is not pkv._NoCalls
        for x, y in zip(without, with_it):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
        print("done")
        """)


def test_the_library_builds_without_torch(tmp_path, monkeypatch):
    """With a compiler that only makes its output files."""
    from paged_kv_cache_291_gb300 import build
    cc = tmp_path / "nvcc"
    cc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n')
    cc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(cc))
    monkeypatch.setenv("CXX", "/bin/false")
    for name, to in (("BUILD", "objects"), ("LIB", "libpagedkv.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(build, name, str(tmp_path / to))
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert (tmp_path / "libpagedkv.so").exists() and not build.up_to_date()
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.up_to_date()
    (tmp_path / "libpagedkv.so").unlink()
    assert build.build() == str(tmp_path / "libpagedkv.so")
    assert build.up_to_date() and not (tmp_path / "_binding.so").exists()
