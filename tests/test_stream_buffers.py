"""Buffers that a call allocates while ``stream`` names another stream than the current one.

The allocator hands a block out again as soon as its last use has been queued on the stream that
the block belongs to.  A block of the current stream that another stream writes at once may
still be in use; so whatever a call allocates has to belong to the stream that runs it, and what
it returns has to be recorded on the caller's.  Shown here on the CPU with stand-ins for the
tensors, the allocator and the library; the test on the GPU looks at the blocks themselves.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import attention_backward_bwd_gb300 as ab
from attention_backward_bwd_gb300 import binding, cache


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle
        self.device = "cuda:0"


class FakeTensor:
    """What the bindings look at of a CUDA tensor."""

    is_cuda, device = True, SimpleNamespace(type="cuda")

    def __init__(self, shape, dtype=torch.float16, owner=None):
        self.shape, self.dtype, self.owner, self.seen_by = tuple(shape), dtype, owner, []

    def stride(self, i=None):
        s = [1] * len(self.shape)
        for k in range(len(s) - 2, -1, -1):
            s[k] = s[k + 1] * self.shape[k + 1]
        return tuple(s) if i is None else s[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def is_contiguous(self):
        return True

    def record_stream(self, stream):
        self.seen_by.append(stream.cuda_stream)


class FakeTorch:
    """torch, with streams and an allocator of its own."""

    def __init__(self):
        self.made, self.now = [], FakeStream(7)
        self.cuda = SimpleNamespace(
            Stream=FakeStream, stream=self._stream, default_stream=lambda device=None: FakeStream(0),
            # a handle of 0 gives a new stream there
            ExternalStream=lambda h, device=None: FakeStream(h if h > 1 else 555),
            current_stream=lambda device=None: self.now, current_device=lambda: 0,
            is_available=lambda: False)

    def __getattr__(self, name):
        return getattr(torch, name)

    @contextlib.contextmanager
    def _stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def _new(self, shape, dtype):
        t = FakeTensor(shape, dtype, self.now.cuda_stream)
        self.made.append(t)
        return t

    def empty(self, *shape, dtype=None, device=None, pin_memory=None):
        shape = tuple(shape[0]) if isinstance(shape[0], (tuple, list)) else shape
        if pin_memory is not None:  # host memory
            return torch.empty(shape, dtype=dtype)
        return self._new(shape, dtype)

    def empty_like(self, t):
        return self._new(t.shape, t.dtype)


class FakeLib:
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 1024

        def call(*a):
            s = a[-1]
            self.streams.append(s)
            return 0
        return call


I32, F32 = torch.int32, torch.float32


def _rope(**kw):
    q = FakeTensor((6, 2, 64))
    return ab.attn_rope(q, q, FakeTensor((6,), I32), FakeTensor((32,), F32), **kw)


def _append(**kw):
    x, c = FakeTensor((3, 2, 64)), FakeTensor((9, 16, 2, 64))
    return (ab.attn_cache_append(x, x, c, c, FakeTensor((3, 3), I32), FakeTensor((3,), I32), q=x,
                                 positions=FakeTensor((3,), I32), inv_freq=FakeTensor((32,), F32), **kw),)


def _decode(**kw):
    c = FakeTensor((90, 16, 2, 64))
    return ab.attn_decode(FakeTensor((3, 4, 64)), c, c, FakeTensor((3, 30), I32), FakeTensor((3,), I32), **kw)


def _evict(**kw):
    c = FakeTensor((9, 16, 2, 64))
    return ab.attn_cache_evict(c, c, FakeTensor((3, 3), I32), FakeTensor((3,), I32), FakeTensor((3, 2, 48), F32),
                               16, **kw)[:1]


def _fwd(**kw):
    q = FakeTensor((2, 64, 4, 64))
    return ab.attn_fwd(q, q, q, **kw)


def _bwd(**kw):
    q, k = FakeTensor((2, 64, 4, 64)), FakeTensor((2, 64, 2, 64))
    return ab.attn_bwd(q, k, k, q, FakeTensor((2, 4, 64), F32), q, **kw)


def _bwd_host(**kw):
    q, lse = torch.randn(2, 64, 4, 64).half(), torch.zeros(2, 4, 64)
    ab.attn_bwd_host(q, q, q, q, lse, q, **kw)
    return ()


def _bwd_host_varlen(**kw):
    q, lse, cu = torch.randn(64, 4, 64).half(), torch.zeros(4, 64), torch.tensor([0, 30, 64])
    ab.attn_bwd_host_varlen(q, q, q, q, lse, q, cu, cu, **kw)
    return ()


@pytest.fixture
def fake(monkeypatch):
    t, lib = FakeTorch(), FakeLib()
    for m in (binding, cache):
        monkeypatch.setattr(m, "torch", t)
        monkeypatch.setattr(m, "lib", lambda: lib)
    monkeypatch.setattr(cache, "_raw_stream", lambda index: t.now.cuda_stream)
    for f in (cache.decode_workspace_size, cache.evict_workspace_size):
        f.cache_clear()
    yield t, lib
    for f in (cache.decode_workspace_size, cache.evict_workspace_size):
        f.cache_clear()


# each call and how many buffers it allocates on the device
CALLS = [(_rope, 2), (_append, 1), (_decode, 3), (_evict, 2), (_fwd, 2), (_bwd, 4), (_bwd_host, 1),
         (_bwd_host_varlen, 1)]


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("call,allocated", CALLS)
def test_buffers_belong_to_the_stream_that_runs_the_call(fake, call, allocated, as_handle):
    t, lib = fake
    out = call(stream=99 if as_handle else FakeStream(99))
    assert lib.streams == [99] and t.now.cuda_stream == 7
    assert [x.owner for x in t.made] == [99] * allocated
    for x in out:
        assert 7 in x.seen_by  # the caller's stream reads it later


@pytest.mark.parametrize("call,allocated", CALLS)
def test_buffers_of_calls_on_the_current_stream(fake, call, allocated):
    t, lib = fake
    call()
    assert lib.streams == [7] and [x.owner for x in t.made] == [7] * allocated


@pytest.mark.parametrize("handle", [0, 1])
@pytest.mark.parametrize("call,allocated", CALLS)
def test_handles_of_the_default_stream(fake, call, allocated, handle):
    t, lib = fake
    call(stream=handle)
    assert lib.streams == [handle] and [x.owner for x in t.made] == [0] * allocated


# ------------------------------------------------------------------ on the GPU

@pytest.mark.gpu
def test_the_default_stream_by_its_handle():
    side, main = torch.cuda.Stream(), torch.cuda.default_stream()
    q = torch.randn(300, 4, 64, device="cuda").half()
    pos, inv = torch.arange(300, dtype=torch.int32, device="cuda"), torch.rand(32, device="cuda")
    want = ab.attn_rope(q, None, pos, inv)[0]
    assert binding._side(0, 0) == binding._side(1, 0) == main
    assert binding._side(side.cuda_stream, 0).cuda_stream == side.cuda_stream
    side.wait_stream(main)
    with torch.cuda.stream(side):
        for handle in (0, 1):
            got = ab.attn_rope(q, None, pos, inv, stream=handle)[0]
            side.wait_stream(main)
            assert torch.equal(got, want)


def _busy_block(nbytes, stream):
    """A block of ``nbytes`` that the current stream still has to read: its address, where it is
    copied to and what it holds.  It was given back to the allocator already."""
    block = torch.full((nbytes,), 77, dtype=torch.uint8, device="cuda")
    copy = torch.empty_like(block)
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(100_000_000)  # some 50 ms
    copy.copy_(block)
    at = block.data_ptr()
    del block
    return at, copy


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["forward", "backward"])
def test_a_block_in_use_is_not_taken_by_training_calls(call):
    b, n, hq, hk, d = 2, 512, 4, 2, 128
    side = torch.cuda.Stream()
    q, do = (torch.randn(b, n, hq, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(b, n, hk, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    o, lse = ab.attn_fwd(q, k, v, causal=True)
    run = {"forward": lambda **kw: ab.attn_fwd(q, k, v, causal=True, **kw),
           "backward": lambda **kw: ab.attn_bwd(q, k, v, o, lse, do, causal=True, deterministic=True, **kw)}[call]
    want = [t.clone() for t in run()]
    size = q.numel() * 2 if call == "forward" else ab.workspace_size(b, n, hq, d, True)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    _, copy = _busy_block(size, side)
    got = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    ab.check_device_status()
    assert (copy == 77).all()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["rope", "append", "decode", "evict"])
def test_a_block_in_use_is_not_taken_by_another_stream(call):
    batch, hq, hk, d, page, n, dt = 8, 16, 4, 128, 16, 2048, torch.float16
    per = n // page
    side = torch.cuda.Stream()
    kc, vc = (torch.randn(batch * per, page, hk, d, device="cuda").to(dt) for _ in range(2))
    table = torch.arange(batch * per, dtype=torch.int32, device="cuda").view(batch, per)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    x = torch.randn(n, hk, d, device="cuda").to(dt)
    pos, inv = torch.arange(n, dtype=torch.int32, device="cuda"), torch.rand(d // 2, device="cuda")
    q, w = torch.randn(batch, hq, d, device="cuda").to(dt), torch.rand(batch, hk, n, device="cuda")
    none, cu = lens * 0, torch.arange(0, n + 1, n // batch, dtype=torch.int32, device="cuda")
    runs = {
        "rope": lambda **kw: ab.attn_rope(x, None, pos, inv, **kw)[0],
        "append": lambda **kw: ab.attn_cache_append(x, x, kc, vc, table, none, cu, q=x, positions=pos,
                                                    inv_freq=inv, **kw),
        "decode": lambda **kw: ab.attn_decode(q, kc, vc, table, lens, max_seqlen=n, **kw)[0],
        "evict": lambda **kw: ab.attn_cache_evict(kc, vc, table, lens, w, 100, **kw)[0],
    }
    size = {"rope": x.numel() * 2, "append": x.numel() * 2,
            "decode": ab.decode_workspace_size(batch, hq, hk, d, n),
            "evict": ab.evict_workspace_size(batch, hk, 100, n)}[call]
    state = kc, vc, w
    saved = [t.clone() for t in state]
    want = [t.clone() for t in (runs[call](), *state)]
    for t, old in zip(state, saved):
        t.copy_(old)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    at, copy = _busy_block(size, side)
    got = runs[call](stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    ab.check_device_status()
    assert (copy == 77).all()
    assert all(torch.equal(x, y) for x, y in zip((got, *state), want))
    if call in ("rope", "append"):
        assert got.data_ptr() != at


@pytest.mark.gpu
def test_calls_on_a_forked_stream_are_captured_with_their_buffers():
    batch, hq, hk, d, page, n = 4, 8, 2, 64, 16, 800
    per = n // page
    kc, vc = (torch.randn(batch * per, page, hk, d, device="cuda").half() for _ in range(2))
    table = torch.arange(batch * per, dtype=torch.int32, device="cuda").view(batch, per)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(batch, hq, d, device="cuda").half()
    pos, inv = torch.arange(batch, dtype=torch.int32, device="cuda"), torch.rand(d // 2, device="cuda")

    def step(**kw):
        r, _ = ab.attn_rope(q, None, pos, inv, **kw)
        return ab.attn_decode(r, kc, vc, table, lens, **kw)

    step()  # loads the kernels
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        first = step(stream=side)
        second = step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        q.normal_()
        want = step()
        g.replay()
        torch.cuda.synchronize()
        for got in (first, second):
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    ab.check_device_status()
