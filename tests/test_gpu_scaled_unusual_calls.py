"""Calls over pools with a scale per block that are allowed and unusual: empty
batches, empty contexts only, numpy scalars, uint8 codes, one output given, a
stream of the caller's, tables wider than the contexts, captured appends."""
import numpy as np
import pytest
import torch

from oracle import scaled as S
from scaled_batch import Batch, attention_tolerance, bf16_rows, to_dev
from test_gpu_scaled_attention import KINDS, check, decode, pkv, prefill  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("side", [False, True])
def test_empty_batches(pkv, kind, side):
    b = Batch(90, kind, [1], [20], 2, 64)
    k, v, sc, _, _, _ = b.dev()
    i32 = dict(dtype=torch.int32, device="cuda")
    none, zero, tables = torch.zeros(0, **i32), torch.zeros(1, **i32), torch.zeros((0, 2), **i32)
    rows, q = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (0, 4, 64), dtype=torch.bfloat16, device="cuda")
    kw = dict(stream=torch.cuda.Stream()) if side else {}
    pkv.cache_append(k, v, sc, rows, rows, zero, none, tables, **kw)
    ko, vo = pkv.cache_read(k, v, zero, none, tables, 0, block_scales=sc, **kw)
    assert ko.shape == vo.shape == (0, 2, 64)
    assert pkv.decode_attention(k, v, q, tables, none, 32, 0.1, block_scales=sc, **kw).shape == (0, 4, 64)
    got = pkv.chunked_prefill_attention(k, v, q, zero, none, tables, 32, 0.1, block_scales=sc,
                                        query_start_loc_host=np.zeros(1, np.int32), **kw)
    assert got.shape == (0, 4, 64)
    # sequences without rows
    lens, tables = torch.zeros(3, **i32), torch.zeros((3, 2), **i32)
    start = torch.zeros(4, **i32)
    pkv.cache_append(k, v, sc, rows, rows, start, lens, tables, **kw)
    pkv.cache_read(k, v, start, lens, tables, 0, block_scales=sc, **kw)
    pkv.chunked_prefill_attention(k, v, q, start, lens, tables, 32, 0.1, block_scales=sc,
                                  query_start_loc_host=[0, 0, 0, 0], **kw)
    torch.cuda.synchronize()
    assert torch.equal(k.view(torch.uint8).cpu(), torch.from_numpy(b.k.view(np.uint8)))
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_empty_contexts_only(pkv, kind):
    """No sequence has a key: zero rows, whatever the pools hold."""
    b = Batch(91, kind, [1] * 3, [40] * 3, 2, 128)
    _, qt = bf16_rows(b.rng, 3, 4, 128)
    k, v, sc, _, lens, tables = b.dev()
    for longest in (0, 41):
        out = torch.full((3, 4, 128), 7.0, device="cuda")
        pkv.decode_attention(k, v, qt, tables, torch.zeros_like(lens), longest, 0.1, out=out, block_scales=sc)
        assert not out.any()
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_numpy_scalars_and_a_stream(pkv, kind):
    """Arguments that the compiled binding hands back give the same bits through the wrapper."""
    b = Batch(92, kind, [1, 150, 1], [300, 70, 17], 2, 64)
    q, qt = bf16_rows(b.rng, b.T, 4, 64)
    k, v, sc, start, lens, tables = b.dev()
    longest = int(b.lens.max())
    want = prefill(pkv, b, qt, 0.125)
    check(b, want, q, 0.125)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        got = pkv.chunked_prefill_attention(k, v, qt, start, lens, tables, np.int64(longest), np.float32(0.125),
                                            query_start_loc_host=b.start.tolist(), block_scales=sc, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        rows = pkv.cache_read(k, v, start, lens, tables, np.int32(b.T), block_scales=sc, stream=stream,
                              k_out=torch.empty((b.T, 2, 64), dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
        for x, exact in zip(rows, S.read(b.k, b.v, b.scales, b.start, b.lens, b.tables, b.T)):
            assert np.array_equal(x.view(torch.int16).cpu().numpy().view(np.uint16), S.to_bf16_bits(exact))
    assert pkv.get_error()[0] == 0


def test_uint8_pools_and_wide_tables(pkv):
    """e4m3 codes as uint8 are those of float8_e4m3fn; entries past a context are never read."""
    b = Batch(93, np.uint8, [1] * 4, [5, 300, 0, 47], 2, 128)
    q, qt = bf16_rows(b.rng, 4, 4, 128)
    want = decode(pkv, b, qt, 0.1)
    check(b, want, q, 0.1)
    wide = np.full((4, 1000), 2 ** 31 - 1, np.int32)
    wide[:, :b.tables.shape[1]] = b.tables
    k, v, sc, _, lens, _ = b.dev()
    got = pkv.decode_attention(k.view(torch.uint8), v.view(torch.uint8), qt, torch.from_numpy(wide).cuda(), lens, 16000,
                               0.1, block_scales=sc)
    check(b, got, q, 0.1)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_captured_steps_replayed(pkv, kind):
    """Append and attention captured together, replayed as the context grows block by block: the scales grow, blocks
    begin, rows are encoded again, on one workspace."""
    hkv, d, hq = 2, 64, 4
    rng = np.random.default_rng(94)
    tables = rng.permutation(8).astype(np.int32)[:6].reshape(2, 3)
    x = rng.standard_normal((8, hkv, 16, d)).astype(np.float32) * 30
    host = [np.zeros((8, hkv, 16, d), kind) for _ in range(2)] + [np.full((8, hkv, 2), 0.01, np.float32)]
    host[0][:], host[1][:] = S.encode(x, host[0]), S.encode(x[::-1], host[1])
    k, v = (to_dev(x.copy()) for x in host[:2])
    sc, tab = torch.from_numpy(host[2]).cuda(), torch.from_numpy(tables).cuda()
    lens = torch.tensor([15, 31], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    kt, vt = (torch.zeros((2, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qt = torch.zeros((2, hq, d), dtype=torch.bfloat16, device="cuda")
    ws = pkv.new_workspace(pkv.decode_workspace_size(2, hq, hkv, d, 48))
    out = torch.empty((2, hq, d), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.cache_append(k, v, sc, kt, vt, start, lens, tab)
        pkv.decode_attention(k, v, qt, tab, lens, 48, 0.125, out=out, workspace=ws, block_scales=sc)
    n = np.array([15, 31], np.int32)
    for step in range(16):
        kn, x = bf16_rows(rng, 2, hkv, d, size=1.1 ** step)
        kt.copy_(x)
        vn, x = bf16_rows(rng, 2, hkv, d, size=1.2 ** step)
        vt.copy_(x)
        q, x = bf16_rows(rng, 2, hq, d)
        qt.copy_(x)
        lens.copy_(torch.from_numpy(n))
        graph.replay()
        torch.cuda.synchronize()
        S.append(*host, kn, vn, [0, 1, 2], n, tables)
        assert np.array_equal(sc.cpu().numpy(), host[2], equal_nan=True)
        exact = S.attention(*host, q, [0, 1, 2], n, tables, 0.125)
        tol = attention_tolerance(exact, int(n.max()), host[2])
        assert np.all(np.abs(out.double().cpu().numpy() - exact[0]) <= tol)
        n = n + 1
    assert pkv.get_error()[0] == 0
