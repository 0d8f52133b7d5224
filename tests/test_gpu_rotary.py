"""GPU parity of pkv_rotary and pkv_rotary_cache_write against the fp64 oracle.

Tolerance of one turned element z = x cos a -+ y sin a, derived: its bf16
rounding is at most half a step, 2^-8 |z|; before it, the fp32 work is off by
at most a few 2^-24 of |x| + |y| for the products and sum, cos and sin by
2^-22 together with the rounding of the angle's last 32 bits, and the angle by
2^-47 of its size (an fp32 pair), so (2^-20 + 2^-47 |position * frequency|)
(|x| + |y|).  An e4m3 code is off by at most half a step of 2^-3, 2^-4 |p|,
or half the subnormal step, 2^-10, of the product p.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import dev_tensor
from oracle import fp8
from oracle import rotary as R
import pkv_workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


def f64(t):
    return t.float().double().cpu().numpy()


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()


class Batch:
    def __init__(self, seed, T, hq, hkv, d, rot, sections, interleaved, adjacent, packed=True, far=5000):
        rng = np.random.default_rng(seed)
        self.T, self.hq, self.hkv, self.d = T, hq, hkv, d
        self.how = dict(sections=sections, interleaved=interleaved, adjacent=adjacent)
        self.call = dict(sections=sections, interleaved_axes=interleaved, adjacent_pairs=adjacent)
        self.pos = rng.integers(-far, far, (len(sections), T)).astype(np.int32)
        self.f = (10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32)
        if packed:
            x = bf16(rng, T, hq + 2 * hkv + 1, d).cuda()
            self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
        else:
            self.q, self.k, self.v = (bf16(rng, T, h, d).cuda() for h in (hq, hkv, hkv))

    def want(self, x):
        return R.rotate(f64(x), self.pos, self.f, **self.how)

    def slack(self, x):
        """(|x| + |y|) of each element's pair times the fp32 part of the tolerance; 0 where nothing turns."""
        a = np.abs(f64(x))
        p = len(self.f)
        out = np.zeros_like(a)
        axes = R.axis_of_pairs(self.how["sections"], self.how["interleaved"])
        for i in range(p):
            e0, e1 = (2 * i, 2 * i + 1) if self.how["adjacent"] else (i, i + p)
            far = np.abs(self.pos[axes[i]].astype(np.float64) * float(self.f[i]))[:, None]
            out[:, :, e0] = out[:, :, e1] = (a[:, :, e0] + a[:, :, e1]) * (2.0 ** -20 + 2.0 ** -47 * far)
        return out

    def check_bf16(self, got, x, what):
        want, s = self.want(x), self.slack(x)
        err = np.abs(f64(got) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + s), f"{what}: {np.max(err - s):.3g} off"
        same = s == 0
        assert np.array_equal(f64(got)[same], f64(x)[same]), f"{what}: a passed element changed"


SHAPES = [
    # T, hq, hkv, d, rot, sections, interleaved, adjacent
    (1, 1, 1, 64, 64, [32], False, False),
    (3, 32, 8, 64, 64, [32], False, True),
    (5, 16, 8, 128, 128, [16, 24, 24], False, False),
    (7, 16, 8, 128, 128, [24, 20, 20], True, False),
    (33, 3, 5, 128, 64, [16, 16], False, True),
    (17, 5, 1, 128, 16, [2, 2, 2, 2], True, False),
    (9, 7, 2, 64, 48, [0, 24], False, False),
    (2, 40, 40, 128, 112, [20, 18, 18], True, True),
    (300, 16, 2, 64, 32, [6, 5, 5], False, False),
    (6000, 2, 1, 64, 64, [11, 11, 10], True, False),
]


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotary_matches_the_oracle(pkv, shape, packed):
    b = Batch(1, *shape, packed=packed)
    q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f), **b.call)
    assert pkv.get_error() == (0, 0)
    b.check_bf16(q, b.q, "q")
    b.check_bf16(k, b.k, "k")


def test_one_axis_takes_a_plain_vector_of_positions(pkv):
    b = Batch(2, 5, 2, 1, 64, 64, [32], False, False)
    q, _ = pkv.rotary(b.q, b.k, dev_tensor(b.pos[0]), dev_tensor(b.f))
    b.check_bf16(q, b.q, "q")


@pytest.mark.parametrize("packed", [False])
def test_rotary_in_place(pkv, packed):
    for shape in SHAPES[:5]:
        b = Batch(3, *shape, packed=packed)
        q0, k0 = b.q.clone(), b.k.clone()
        q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f), q_out=b.q, k_out=b.k, **b.call)
        assert q.data_ptr() == b.q.data_ptr() and k.data_ptr() == b.k.data_ptr()
        b.check_bf16(q, q0, "q")
        b.check_bf16(k, k0, "k")


def test_rotary_extreme_positions_and_frequencies(pkv):
    """Positions up to the ends of int32, frequencies from 0 to tens of turns
    a step: the angle keeps its accuracy."""
    b = Batch(4, 9, 2, 2, 64, 64, [32], False, False)
    b.pos[0] = [0, 1, -1, 2 ** 20, -2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789]
    b.f = np.concatenate([[0.0, 1.0, -1.0, 3.1415927, 6.2831855, 100.7, 1e-30, 0.5],
                          np.linspace(1e-3, 2.0, 24)]).astype(np.float32)
    q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f))
    b.check_bf16(q, b.q, "q")
    b.check_bf16(k, b.k, "k")


def test_rotary_keeps_guards_and_non_finite_rows_apart(pkv):
    """Rows around the outputs stay; a NaN or infinite row does not reach others."""
    b = Batch(5, 37, 4, 2, 128, 128, [64], False, False)
    b.q[11, 2] = float("nan")
    b.k[12, 1] = float("inf")
    full = torch.full((39, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f), q_out=full[1:38])
    assert torch.all(full[0] == 7) and torch.all(full[38] == 7)
    assert torch.all(torch.isnan(q[11, 2])) and torch.isfinite(q[11, 1]).all() and torch.isfinite(q[12]).all()
    assert not torch.isfinite(k[12, 1]).any() and torch.isfinite(k[12, 0]).all() and torch.isfinite(k[13]).all()


def test_rotary_empty_batch(pkv):
    b = Batch(6, 0, 4, 2, 64, 64, [32], False, False, packed=False)
    q, k = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("shape", SHAPES[:9])
def test_cache_write_bf16_equals_the_two_calls(pkv, shape, packed):
    b = Batch(7, *shape, packed=packed)
    rng = np.random.default_rng(8)
    nb = b.T // 16 + 3
    slots = rng.permutation(nb * 16)[:b.T].astype(np.int32)
    slots[rng.random(b.T) < 0.2] = -1
    pools = [dev_tensor(W.normal_bf16(9, i, nb * b.hkv * 16 * b.d).reshape(nb, b.hkv, 16, b.d)) for i in (1, 2)]
    two = [p.clone() for p in pools]
    q2, k2 = pkv.rotary(b.q, b.k, dev_tensor(b.pos), dev_tensor(b.f), **b.call)
    pkv.cache_write(two[0], two[1], k2, b.v.contiguous(), dev_tensor(slots))
    q = pkv.rotary_cache_write(pools[0], pools[1], b.q, b.k, b.v, dev_tensor(slots), dev_tensor(b.pos),
                               dev_tensor(b.f), **b.call)
    assert pkv.get_error() == (0, 0)
    for got, ref in ((q, q2), (pools[0], two[0]), (pools[1], two[1])):
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
    b.check_bf16(q, b.q, "q")


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[3], SHAPES[4], SHAPES[6]])
def test_cache_write_e4m3(pkv, shape):
    b = Batch(10, *shape)
    rng = np.random.default_rng(11)
    nb = b.T // 16 + 2
    slots = rng.permutation(nb * 16)[:b.T].astype(np.int32)
    slots[0] = -3 if b.T > 3 else slots[0]
    ks, vs = np.float32(0.0123), np.float32(0.004)   # v: values saturate
    inv_k, inv_v = np.float32(1) / ks, np.float32(1) / vs
    k8, v8 = (torch.from_numpy(rng.integers(0, 127, (nb, b.hkv, 16, b.d)).astype(np.uint8)).cuda() for _ in range(2))
    k0, v0 = k8.cpu().numpy(), v8.cpu().numpy()
    q = pkv.rotary_cache_write(k8, v8, b.q, b.k, b.v, dev_tensor(slots), dev_tensor(b.pos), dev_tensor(b.f),
                               k_scale=float(ks), v_scale=float(vs), **b.call)
    assert pkv.get_error() == (0, 0)
    b.check_bf16(q, b.q, "q")
    want, slack = b.want(b.k) * float(inv_k), b.slack(b.k) * float(inv_k)
    codes_v = fp8.encode(np.float32(f64(b.v)) * inv_v)
    values = fp8.decode_codes()
    got_k, got_v = k8.cpu().numpy(), v8.cpu().numpy()
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        blk, row = slot // 16, slot % 16
        p = np.clip(want[t], -448, 448)
        err = np.abs(values[got_k[blk, :, row]] - p)
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(p), 2.0 ** -10) + slack[t] + 2.0 ** -24 * np.abs(p))
        assert np.array_equal(got_v[blk, :, row], codes_v[t])
        k0[blk, :, row], v0[blk, :, row] = got_k[blk, :, row], got_v[blk, :, row]
    assert np.array_equal(got_k, k0) and np.array_equal(got_v, v0), "a slot outside the mapping changed"


def test_cache_write_reports_a_slot_past_the_pool(pkv):
    b = Batch(12, 4, 2, 2, 64, 64, [32], False, False)
    k, v = (torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = np.array([0, 32, 5, 2 ** 31 - 1], np.int32)
    q = pkv.rotary_cache_write(k, v, b.q, b.k, b.v, dev_tensor(slots), dev_tensor(b.pos), dev_tensor(b.f))
    st, detail = pkv.get_error()
    assert st == 9 and detail in (1, 3)
    b.check_bf16(q, b.q, "q")
    assert torch.count_nonzero(k.float().abs().sum((1, 3))) == 2  # rows of slots 0 and 5


def test_rotary_replayed_from_a_graph_on_another_stream(pkv):
    b = Batch(13, 65, 8, 4, 128, 128, [22, 21, 21], True, False)
    pos, f = dev_tensor(b.pos), dev_tensor(b.f)
    q_out, k_out = torch.zeros((65, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (65, 4, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.rotary(b.q, b.k, pos, f, q_out=q_out, k_out=k_out, **b.call)
    b.q.copy_(bf16(np.random.default_rng(14), 65, 8, 128))
    g.replay()
    torch.cuda.synchronize()
    b.check_bf16(q_out, b.q, "q")
    b.check_bf16(k_out, b.k, "k")


def test_rotary_on_a_stream_of_the_callers(pkv):
    """The stream argument takes the same way as the call without it."""
    b = Batch(16, 40, 4, 2, 128, 128, [64], False, False)
    st = torch.cuda.Stream()
    pos, f = dev_tensor(b.pos), dev_tensor(b.f)
    pools = [torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    slots = dev_tensor(np.arange(40, dtype=np.int32))
    torch.cuda.synchronize()
    q, k = pkv.rotary(b.q, b.k, pos, f, stream=st)
    q1 = pkv.rotary_cache_write(pools[0], pools[1], b.q, b.k, b.v, slots, pos, f, stream=st)
    torch.cuda.synchronize()
    b.check_bf16(q, b.q, "q")
    b.check_bf16(k, b.k, "k")
    q2 = pkv.rotary_cache_write(pools[2], pools[3], b.q, b.k, b.v, slots, pos, f)
    assert torch.equal(q1, q) and torch.equal(q2, q)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_binding_refuses_what_it_cannot_pass_on(pkv):
    b = Batch(15, 4, 4, 2, 64, 64, [32], False, False, packed=False)
    pos, f = dev_tensor(b.pos), dev_tensor(b.f)
    with pytest.raises(TypeError):
        pkv.rotary(b.q.float(), b.k, pos, f)
    with pytest.raises(ValueError):
        pkv.rotary(b.q.transpose(0, 1).contiguous().transpose(0, 1), b.k, pos, f)
    with pytest.raises(ValueError):
        pkv.rotary(b.q, b.k, pos[:, :3], f)
    with pytest.raises(ValueError):
        pkv.rotary(b.q, b.k, pos.repeat(2, 1), f)
    with pytest.raises(ValueError):
        pkv.rotary(b.q, b.k.cpu(), pos, f)
    with pytest.raises(TypeError):
        pkv.rotary(b.q, b.k, pos.long(), f)
    with pytest.raises(pkv.PKVError) as e:
        pkv.rotary(b.q, b.k, pos, f, q_out=b.q, k_out=b.q.view(8, 2, 64)[:4])
    assert e.value.status == 6
