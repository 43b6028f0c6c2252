"""The workspace that a call allocates by itself belongs to the stream that the call runs
on. Which stream is current when it is allocated is seen without a GPU; with one, the
current stream reuses memory of the same sizes meanwhile."""
import contextlib

import pytest
import torch

from structured_sparse_matmul_gb300 import vnm


class _Native:
    """Stands for the binding's C part: sizes, and calls that do nothing."""

    def __init__(self):
        self.given = []

    def rmsnorm_workspace(self, T, D):
        return 4 * T * D

    def rmsnorm_backward(self, *args):
        self.given.append(args[7])
        return 0


class _Side:
    cuda_stream = 64


@pytest.fixture
def allocations(monkeypatch):
    """(stream current at the time, size) of each torch.empty."""
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    empty = torch.empty

    def recorded(*a, **k):
        seen.append((current[-1], a[0]))
        return empty(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    return seen


@pytest.mark.parametrize("side", [None, _Side()])
def test_norm_backward_allocates_on_its_stream(monkeypatch, allocations, side):
    native = _Native()
    monkeypatch.setattr(vnm, "_native", lambda: native)
    x, rstd, dw = torch.zeros(3, 5), torch.zeros(3), torch.zeros(5)
    vnm.vnm_rmsnorm_backward(x, x, None, rstd, None, dw, stream=side)
    assert allocations == [(side, 60)] and native.given[0].nbytes == 60
    own = torch.zeros(60, dtype=torch.uint8)
    vnm.vnm_rmsnorm_backward(x, x, None, rstd, None, dw, workspace=own, stream=side)
    vnm.vnm_rmsnorm_backward(x, x, None, rstd, x, None, stream=side)
    assert len(allocations) == 1 and native.given[1] is own and native.given[2] is None


class _OnGpu:
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


class _Library:
    """Stands for libvnm: every call succeeds."""

    def __getattr__(self, name):
        return lambda *a: 0


@pytest.mark.parametrize("side", [None, _Side()])
@pytest.mark.parametrize("call", ["vnm_linear", "vnm_energy"])
def test_the_pruned_calls_allocate_on_their_stream(monkeypatch, allocations, call, side):
    monkeypatch.setattr(vnm, "lib", _Library)
    monkeypatch.setattr(vnm, "_stream_ptr", lambda stream: 0)
    monkeypatch.setattr(vnm, "vnm_linear_workspace_size", lambda A, T: 48)
    monkeypatch.setattr(vnm, "vnm_energy_workspace_size", lambda A: 48)
    A = vnm.VnmMatrix(0, 4, 8, 4, 4, None, None, None)
    X = _OnGpu(torch.zeros(4, 8, dtype=torch.float16))
    if call == "vnm_linear":
        vnm.vnm_linear(A, X, _OnGpu(torch.zeros(4, 4)), stream=side)
    else:
        vnm.vnm_energy(A, X, vnm.VNM_PATTERN_UNSTRUCTURED, stream=side)
    assert allocations == [(side, 48)]


def _busy(stream, a, b):
    """A few milliseconds of copies."""
    with torch.cuda.stream(stream):
        for _ in range(12):
            a.copy_(b)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(2000, 1024), (600, 6000), (300, 20000)])
def test_norm_backward_on_a_side_stream(T, D):
    g = torch.Generator(device="cuda").manual_seed(T)
    h, dy = (torch.randn(T, D, generator=g, device="cuda").half() for _ in range(2))
    rstd = torch.rsqrt(h.float().square().mean(1))
    dh, want = torch.empty_like(h), torch.empty(D, device="cuda")
    vnm.vnm_rmsnorm_backward(dy, h, None, rstd, dh, want)
    n = vnm.vnm_rmsnorm_backward_workspace_size(T, D)
    big = [torch.zeros(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks that the current stream takes after the call's return must not be the call's
    dw = torch.empty(D, device="cuda")
    torch.cuda.synchronize()
    _busy(side, *big)
    vnm.vnm_rmsnorm_backward(dy, h, None, rstd, dh, dw, stream=side)
    later = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(dw, want)
    del later
    # a block that the current stream has given back but not yet read must not be the call's
    kept, out = torch.full((n,), 7, dtype=torch.uint8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream(), *big)
    out.copy_(kept)
    del kept
    vnm.vnm_rmsnorm_backward(dy, h, None, rstd, dh, dw, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(dw, want) and (out == 7).all()


@pytest.mark.gpu
def test_linear_on_a_side_stream():
    g = torch.Generator(device="cuda").manual_seed(1)
    R, K, T = 1024, 4096, 64
    A = vnm.vnm_matrix_alloc(R, K, 64, 8)
    vnm.vnm_compress(A, (0.02 * torch.randn(R, K, generator=g, device="cuda")).half())
    X = torch.randn(T, K, generator=g, device="cuda").half()
    want, Y = torch.empty((T, R), device="cuda"), torch.empty((T, R), device="cuda")
    n = vnm.vnm_linear_workspace_size(A, T)
    assert n > 0
    vnm.vnm_linear(A, X, want)
    big = [torch.zeros(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(side, *big)
    vnm.vnm_linear(A, X, Y, stream=side)
    later = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(Y, want)
    del later
    kept, out = torch.full((n,), 7, dtype=torch.uint8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream(), *big)
    out.copy_(kept)
    del kept
    vnm.vnm_linear(A, X, Y, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and (out == 7).all()
    assert vnm.vnm_get_status(A) == vnm.VNM_OK


@pytest.mark.gpu
def test_bitmap_encode_on_a_side_stream():
    g = torch.Generator(device="cuda").manual_seed(2)
    W = torch.randn(1024, 4096, generator=g, device="cuda").half()
    W *= torch.rand(1024, 4096, generator=g, device="cuda") < 0.5
    want = vnm.bitmap_encode(W)
    big = [torch.zeros(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2)]
    parts = (want.bitmaps, want.offsets, want.bases, want._values_storage)
    # blocks of the arrays' sizes that the current stream has given back but not yet read
    kept = [torch.full((t.nbytes,), 7, dtype=torch.uint8, device="cuda") for t in parts]
    out = [torch.empty_like(t) for t in kept]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream(), *big)
    for o, k in zip(out, kept):
        o.copy_(k)
    del kept, k
    got = vnm.bitmap_encode(W, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(parts, (got.bitmaps, got.offsets, got.bases, got._values_storage)):
        assert torch.equal(a, b)
    assert all((o == 7).all() for o in out)


class _Waiting(_Side):
    def __init__(self):
        self.waits = []

    def wait_stream(self, other):
        self.waits.append(other)


class _Recorded:
    def __init__(self):
        self.streams = []
        self.device = None

    def record_stream(self, s):
        self.streams.append(s)


def test_tensors_that_another_stream_writes(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    side, t = _Waiting(), _Recorded()
    vnm._written_on(None, t)
    assert not side.waits and not t.streams
    vnm._written_on(side, t)
    assert side.waits == ["current"] and t.streams == [side]
