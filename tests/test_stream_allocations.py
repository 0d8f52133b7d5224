"""What a call allocates (outputs, workspaces) and reads back on the host
belongs to the stream it launches on, not to torch's current one: the memory
of a workspace that the call lets go of may otherwise be handed out while the
kernels still use it.  The CPU tests watch the wrappers with torch's allocating
functions, the library and the tensors' checks replaced."""
import contextlib

import pytest
import torch

import paged_kv_cache_291_gb300 as pkv


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeCuda:
    Stream = FakeStream

    def __init__(self, owner):
        self.owner = owner

    @contextlib.contextmanager
    def stream(self, s):
        before, self.owner.now = self.owner.now, s.cuda_stream
        yield
        self.owner.now = before

    def ExternalStream(self, handle):
        return FakeStream(handle)

    def default_stream(self):
        return FakeStream(0)


class FakeTorch:
    """torch, with the allocating functions and the device's reads noted."""

    def __init__(self):
        self.now, self.seen, self.cuda = "current", [], FakeCuda(self)

    def __getattr__(self, name):
        return getattr(torch, name)

    def _new(self, what, shape, kw):
        self.seen.append((what, self.now))
        return torch.zeros(shape, dtype=kw["dtype"])

    def empty(self, shape, **kw):
        return self._new("empty", shape, kw)

    def zeros(self, shape, **kw):
        return self._new("zeros", shape, kw)


class FakeLib:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_size") else 0


@pytest.fixture
def fake(monkeypatch):
    f = FakeTorch()

    class OnDevice:
        """An int32 device tensor whose reads are noted."""

        def __init__(self, values):
            self.values = torch.tensor(values, dtype=torch.int32)
            self.shape = self.values.shape

        def cpu(self):
            f.seen.append(("read", f.now))
            return self.values

    f.on_device = OnDevice
    cache = pkv.Cache(0, 0, 4, 1, 64, 16, 0, 1.0, 1.0)
    binding = type("NoBinding", (), {"__getattr__": lambda self, name: lambda *a: None})()
    for name, value in (("_torch", lambda: f), ("load", lambda: FakeLib()), ("_fast", lambda: binding),
                        ("_dev", lambda *a, **k: None), ("_out", lambda *a, **k: None),
                        ("_addr", lambda *a, **k: 0), ("_rows", lambda *a, **k: (0, 0)),
                        ("_out_addr", lambda *a, **k: 0), ("_device", lambda: -1), ("_cache", lambda *a, **k: cache),
                        ("_rotary", lambda *a, **k: pkv.Rotary()), ("_states", lambda *a: pkv.States(0, 0, 1, 1, 64))):
        monkeypatch.setattr(pkv, name, value)
    return f


def calls(f):
    i32 = dict(dtype=torch.int32)
    q, k = torch.zeros((2, 2, 64)), torch.zeros((2, 1, 64))
    pool = torch.zeros((4, 1, 16, 64))
    tables, lens, two = torch.zeros((2, 2), **i32), torch.ones(2, **i32), torch.zeros(2, **i32)
    blocks = object.__new__(pkv.Blocks)
    blocks.block_tables = tables
    blocks._state = lambda: pkv.BlocksState()
    return {
        "copy_blocks": lambda s: pkv.copy_blocks(pool, pool, f.on_device([0]), f.on_device([1]), stream=s),
        "decode_attention": lambda s: pkv.decode_attention(pool, pool, q, tables, lens, 16, 1.0, stream=s),
        "decode_step": lambda s: pkv.decode_step(pool, pool, k, k, two, q, tables, lens, 16, 1.0, stream=s),
        "decode_attention_shared_prefix": lambda s: pkv.decode_attention_shared_prefix(
            pool, pool, q, tables, lens, 16, 0, 1.0, stream=s),
        "chunked_prefill_attention": lambda s: pkv.chunked_prefill_attention(
            pool, pool, q, f.on_device([0, 1, 2]), lens, tables, 16, 1.0, stream=s),
        "rotary": lambda s: pkv.rotary(q, k, two, torch.zeros(32), stream=s),
        "rotary_cache_write": lambda s: pkv.rotary_cache_write(pool, pool, q, k, k, two, two, torch.zeros(32), stream=s),
        "linear_decode_attention": lambda s: pkv.linear_decode_attention(
            torch.zeros((2, 1, 64, 64)), torch.zeros(1), q, k, k, two, lens, 1.0, stream=s),
        "linear_prefill_attention": lambda s: pkv.linear_prefill_attention(
            torch.zeros((2, 1, 64, 64)), torch.zeros(1), q, k, k, f.on_device([0, 1, 2]), two, lens, 1.0, stream=s),
        "prefix_keys": lambda s: pkv.prefix_keys(torch.zeros(16, **i32), torch.zeros(2, **i32), 1, stream=s),
        "match": lambda s: blocks.match(torch.zeros((2, 1, 32)), two, stream=s),
        "append": lambda s: blocks.append(torch.zeros(3, **i32), 2, stream=s),
    }


NAMES = ["copy_blocks", "decode_attention", "decode_step", "decode_attention_shared_prefix",
         "chunked_prefill_attention", "rotary", "rotary_cache_write", "linear_decode_attention",
         "linear_prefill_attention", "prefix_keys", "match", "append"]


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_belongs_to_its_stream(fake, name):
    """A stream object, an object with a handle, a handle, the default
    stream's handle, and no stream."""
    call = calls(fake)[name]
    other = type("Foreign", (), {"cuda_stream": 23})()
    for stream, at in ((FakeStream(7), 7), (other, 23), (41, 41), (0, 0)):
        fake.seen.clear()
        call(stream)
        assert fake.seen and all(now == at for _, now in fake.seen), (stream, fake.seen)
        assert fake.now == "current"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_calls_on_two_streams_share_no_workspace(kind):
    """Prefills on streams that are held back, with nothing allocated by the
    caller and nothing waited for in between, while the current stream takes
    and fills memory of the same sizes."""
    from test_gpu_linear import Batch

    from gpu_helpers import dev_tensor
    pkv.load()
    batches = [Batch(300 + i, [700, 3, 260, 90], [4, 4, 0, 4], 8, 4, 128, separate=False) for i in range(2)]
    wants = []
    for b in batches:
        wants.append((b.prefill(pkv), b.states.clone()))
        b.check(*wants[-1][:1])
        b.states = dev_tensor(b.S0)
    args = [(b.states, dev_tensor(b.g), b.q, b.k, b.v, dev_tensor(b.qsl), dev_tensor(b.slots), dev_tensor(b.ctx),
             b.scale) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    need = pkv.linear_prefill_workspace_size(4, batches[0].T, 8, 4, 128)
    torch.cuda.synchronize()
    outs = []
    for st, a, b in zip(streams, args, batches):
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)
        outs.append(pkv.linear_prefill_attention(*a, query_start_loc_host=b.qsl,
                                                 stream=st if kind == "stream" else st.cuda_stream))
        filled = [torch.full((need,), 0, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    assert pkv.get_error() == (0, 0)
    assert all(not torch.any(x) for x in filled)
    for b, out, (want, after) in zip(batches, outs, wants):
        assert torch.equal(out, want)
        assert torch.equal(b.states[dev_tensor(b.slots).long()], after[dev_tensor(b.slots).long()])
