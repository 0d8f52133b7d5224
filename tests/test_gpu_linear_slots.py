"""Linear attention: which sequences count as users of a state slot in the
check of slots that several share."""
import pytest
import torch

from test_gpu_linear import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


def batch(seed, form):
    return Batch(seed, [1, 1, 1, 1] if form == "decode" else [3, 90, 1, 150], [5] * 4, 2, 1, 64)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("other", [0, 1])
@pytest.mark.parametrize("user", [2, 3])
def test_a_skipped_sequence_shares_nothing(pkv, form, other, user):
    """No state to go on from: its stale entry for the new state is not used."""
    b = batch(500, form)
    b.slots[other] = -1
    stale = int(b.new[other])
    b.new[other] = b.new[user]
    out = getattr(b, form)(pkv)
    assert pkv.get_error() == (0, 0)
    rows = slice(int(b.qsl[other]), int(b.qsl[other + 1]))
    assert torch.all(out[rows] == 0)
    b.new[other] = stale  # nothing goes there either
    b.check(out, "skipped")


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("other", [0, 1])
@pytest.mark.parametrize("kind", ["reads past the pool", "stores past the pool", "short context"])
def test_a_refused_sequence_shares_nothing(pkv, form, other, kind):
    """It is reported for what is wrong with it, and not for a shared slot."""
    b = batch(501, form)
    if kind == "reads past the pool":
        b.slots[other], b.new[other] = 99, b.new[2]
    elif kind == "stores past the pool":
        b.slots[other], b.new[other] = b.new[3], 99
    else:
        b.ctx[other], b.new[other] = (-1 if form == "decode" else b.lens[other] - 1), b.new[3]
    out = getattr(b, form)(pkv)
    assert pkv.get_error() == (9, other)
    assert torch.all(out[int(b.qsl[other]):int(b.qsl[other + 1])] == 0)
    want, after = b.oracle()
    bound, bound_after = b.oracle(absolute=True)
    got = f64(out)
    states = b.states.double().cpu().numpy()
    for s in range(4):
        if s == other:
            continue
        c = (40 + 4 * b.lens[s]) * 2.0 ** -24
        rows = slice(int(b.qsl[s]), int(b.qsl[s + 1]))
        assert (abs(got[rows] - want[rows]) <= c * bound[rows] + 1e-37).all()
        i = int(b.new[s])
        assert (abs(states[i] - after[i]) <= c * bound_after[i] + 1e-37).all()


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_a_fresh_sequence_uses_its_new_slot_only(pkv, form):
    """A first chunk reads no state, so the slot it names for reading may be
    another's; the slot it stores to may not."""
    b = batch(502, form)
    b.ctx[1] = b.lens[1]
    b.slots[1] = b.new[2]
    out = getattr(b, form)(pkv)
    assert pkv.get_error() == (0, 0)
    b.check(out, "fresh")
    b = batch(503, form)
    b.ctx[1] = b.lens[1]
    b.new[1] = b.new[2]
    getattr(b, form)(pkv)
    st, detail = pkv.get_error()
    assert st == 6 and detail in (1, 2)
