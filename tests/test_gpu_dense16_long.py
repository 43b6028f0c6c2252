"""Long sums of one sign, and the order that calls keep among streams."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import BF16, DEV, F16, F32, NONE, ULP, check, generator, pitched, whole  # noqa: E402

LONG = 262144 + 40


def _factors(g, rows, unit):
    """A rows x LONG matrix of positive numbers a[r] * c[k] that fp16 holds, and a and c."""
    a = 2.0 ** torch.randint(-1, 2, (rows,), generator=g, device=DEV).double()
    c = (torch.rand(LONG, generator=g, device=DEV) * 0.5 + 0.5).half().double() * unit
    return (a.half()[:, None] * c.half()[None]), a, c


def _loss(K):
    """What the tensor cores' truncated sums of one sign lose: 6e-9 of the sum for each element was measured,
    and up to 2^-23 for each 16 is what one truncation an MMA would lose; twice that."""
    return 2 * K / 16 * ULP


@pytest.mark.parametrize("T,R", [(9, 40), (40, 300), (300, 300), (2304, 2048), (4850, 1024)])
def test_dense(T, R):
    """16-bit outputs take the sums out every 32768 elements of K (without that, 1.6e-3 of them would be lost), fp32 ones
    every 1024."""
    g = generator(T, R, 21)
    (x, a, c), (w, b, d) = _factors(g, T, 1.0), _factors(g, R, 2.0 ** -6)
    want = torch.outer(a, b) * (c * d).sum()
    for out, chunk in ((F16, 32768), (F32, 1024)):
        Y = torch.empty((T, R), dtype=out, device=DEV)
        vnm.vnm_dense_linear(x, w, Y)
        check(Y, want, (_loss(chunk) + (LONG / chunk + 16) * ULP) * want)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("T,F", [(9, 40), (300, 300), (2304, 1024), (4850, 510)])
def test_gated(T, F):
    g = generator(T, F, 22)
    (x, a, c), (wg, b, d), (wu, e, f) = _factors(g, T, 1.0), _factors(g, F, 2.0 ** -12), _factors(g, F, 2.0 ** -12)
    G, U = torch.outer(a, b) * (c * d).sum(), torch.outer(a, e) * (c * f).sum()
    loss = _loss(32768) + (LONG / 32768 + 16) * ULP
    Y, p, q = (torch.empty((T, F), dtype=F16, device=DEV) for _ in range(3))
    vnm.vnm_gated_linear(x, wg, wu, Y, act=NONE, g=p, u=q)
    check(p, G, loss * G)
    check(q, U, loss * U)
    check(Y, G * U, (2 * loss + 2 * ULP) * G * U)
    vnm.vnm_gated_linear(x, wg, wu, Y, act=NONE)
    check(Y, G * U, (2 * loss + 2 * ULP) * G * U)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


# (few tokens, narrow tiles, pairs of CTAs, K over pairs)
@pytest.mark.parametrize("T,R,K", [(4, 512, 4096), (24, 512, 4096), (2000, 2048, 1024), (470, 1752, 2688)])
@pytest.mark.parametrize("captured", [False, True])
def test_joins(T, R, K, captured):
    """A call that follows a call on its own stream and work of another stream waits for both: the other
    stream's long chain of products ends in this call's W, the call before it made its X."""
    g = generator(T, R, 23)
    x, eye, w = whole(g, T, K, BF16, 1), torch.eye(K, device=DEV).bfloat16(), whole(g, R, K, BF16, 1)
    x1, Y = torch.empty_like(x), torch.empty((T, R), dtype=BF16, device=DEV)
    w1, w2 = torch.empty_like(w), torch.empty_like(w)
    side = torch.cuda.Stream()

    def run():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            vnm.vnm_dense_linear(w, eye, w1)
            for _ in range(10):
                vnm.vnm_dense_linear(w1, eye, w2)
                vnm.vnm_dense_linear(w2, eye, w1)
        vnm.vnm_dense_linear(x, eye, x1)
        here.wait_stream(side)
        vnm.vnm_dense_linear(x1, w1, Y)
        w1.zero_()  # (and what follows waits for the call)
        x1.zero_()

    run()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        w.copy_(whole(g, R, K, BF16, 1))
        Y.fill_(float("nan"))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
    assert torch.equal(Y, (x.double() @ w.double().t()).bfloat16())
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


def test_two_streams_at_once():
    """Calls of every kernel on two streams at the same time give the bits that they give one by one."""
    g = generator(24)
    sizes = [(4, 512, 4096), (24, 512, 4096), (470, 1752, 2688), (2000, 2048, 1024)]
    ins = [(whole(g, T, K, F16), whole(g, R, K, F16)) for T, R, K in sizes]
    want = [(x.double() @ w.double().t()).half() for x, w in ins]
    outs = [[torch.empty_like(y) for y in want] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for n in range(20):
        for i, s in enumerate(streams):
            for j in range(4):
                k = (j + i * (1 + n % 3)) % 4
                vnm.vnm_dense_linear(*ins[k], outs[i][k], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, v) for out in outs for y, v in zip(out, want))
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("T,R,K,skip", [(470, 1752, 2688, 3), (843, 1432, 3216, 0)])
def test_time_out_of_split_pairs(T, R, K, skip):
    """A stage that never arrives in one of a cluster's pairs: the waits run out, the others' copies land before a CTA
    leaves, the error is kept and the next call is right."""
    assert vnm.vnm_testing_dense_plan(0, T, R, K, 152)[2] > 1
    g = generator(T, 25)
    x, w = whole(g, T, K, F16), whole(g, R, K, F16)
    Y = torch.empty((T, R), dtype=F16, device=DEV)
    vnm.vnm_testing_dense_linear_skip_stage(x, w, Y, skip)
    assert vnm.vnm_dense_get_status() == vnm.VNM_ERR_TIMEOUT
    vnm.vnm_dense_linear(x, w, Y)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    assert torch.equal(Y, (x.double() @ w.double().t()).half())


# (both of dX and of dWg and dWu by narrow tiles; dX by narrow tiles, the others by pairs; both by pairs)
@pytest.mark.parametrize("T,F,K", [(42, 1576, 125), (1, 79, 125), (736, 1280, 149), (2042, 654, 684), (578, 1346, 1274), (1024, 4096, 1024)])
@pytest.mark.parametrize("captured", [False, True])
def test_backward_passes_in_a_row(T, F, K, captured):
    """Passes one behind the other with one workspace, on changing inputs, and what overwrites their
    inputs right behind: dX and the weights' gradients, whose grids run side by side, give the bits that they give alone."""
    g = generator(T, F, K, 26)
    ins = [[pitched(torch.randn(*s, generator=g, device=DEV).bfloat16()) for s in ((T, F), (T, K), (F, K), (F, K), (T, F), (T, F))]
           for _ in range(3)]
    ws = torch.empty(vnm.vnm_gated_linear_backward_workspace_size(T, F), dtype=torch.uint8, device=DEV)

    def outputs():
        return [torch.full(s, float("nan"), dtype=BF16, device=DEV) for s in ((T, K), (F, K), (F, K))]

    want, outs = [outputs() for _ in ins], [outputs() for _ in ins]
    for i, o in zip(ins, want):
        vnm.vnm_gated_linear_backward(*i, dx=o[0], workspace=ws)
        torch.cuda.synchronize()
        vnm.vnm_gated_linear_backward(*i, dwg=o[1], dwu=o[2], workspace=ws)
        torch.cuda.synchronize()
    held = [pitched(torch.empty_like(v)) for v in ins[0]]

    def run():
        for _ in range(5):
            for i, o in zip(ins, outs):
                for h, v in zip(held, i):
                    h.copy_(v)
                vnm.vnm_gated_linear_backward(*held, dx=o[0], dwg=o[1], dwu=o[2], workspace=ws)
                for h in held:
                    h.fill_(float("nan"))
            for i, o in zip(ins, outs):
                vnm.vnm_gated_linear_backward(*i, dx=o[0], dwg=o[1], dwu=o[2], workspace=ws)

    run()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for o in outs:
            for v in o:
                v.fill_(float("nan"))
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o, w in zip(outs, want) for p, q in zip(o, w))
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("T", [1, 8, 16])
def test_what_was_added_to_in_place_is_read_by_the_next_call(T):
    """Calls that add to Y in place, whose neighbouring CTAs read and write parts of the same 32 bytes (Y starts 16 bytes into
    them), each followed by calls that read Y: as X of few tokens, as X of narrow tiles, as dY of a backward pass. The next grid's CTAs are
    there before the sums are; they must not see what was cached before."""
    D, F = 4096, 512
    g = generator(T, 27)
    x = whole(g, T, 256, F16, 1)
    w, w2, wide = whole(g, D, 256, F16, 1), whole(g, F, D, F16, 1), whole(g, 300, D, F16, 1)
    buf = torch.zeros(T * D + 8, dtype=F16, device=DEV)
    Y = buf[8:].view(T, D)
    gg, uu = whole(g, T, D, F16, 1), whole(g, T, D, F16, 1)
    n = 6
    Z, V = (torch.empty((n, T, F), dtype=F32, device=DEV) for _ in range(2))
    dx, wg = torch.empty((n, T, 64), dtype=F16, device=DEV), whole(g, D, 64, F16, 1)
    ws = torch.empty(vnm.vnm_gated_linear_backward_workspace_size(T, D), dtype=torch.uint8, device=DEV)
    turned = torch.empty((n, 300, T), dtype=F32, device=DEV)

    def run(wait=lambda: None):
        Y.zero_()
        for i in range(n):
            vnm.vnm_dense_linear(x, w, Y, residual=Y)
            wait()
            vnm.vnm_dense_linear(Y, w2, Z[i])
            wait()
            vnm.vnm_dense_linear(x, w, Y, residual=Y)
            wait()
            vnm.vnm_gated_linear_backward(Y, None, wg, wg, gg, uu, dx=dx[i], workspace=ws)
            wait()
            vnm.vnm_dense_linear(x, w, Y, residual=Y)
            wait()
            vnm.vnm_dense_linear(wide, Y, turned[i])
            wait()
            vnm.vnm_dense_linear(Y, w2, V[i])
            wait()

    run(torch.cuda.synchronize)
    want = [v.clone() for v in (Z, V, dx, turned, Y)]
    total = 3 * (x.double() @ w.double().t())
    for i in range(n):
        assert torch.equal(V[i].double(), (i + 1) * total @ w2.double().t())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for way in [run] * 20 + [graph.replay] * 20:
        way()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (Z, V, dx, turned, Y)))


@pytest.mark.parametrize("T,F,K", [(42, 1576, 125), (5, 301, 77), (736, 1281, 149), (578, 1346, 1275)])
@pytest.mark.parametrize("w_type", [BF16, F32])
def test_gradients_added_up_over_passes(T, F, K, w_type):
    """The weights' gradients of passes one behind the other, added up in rows whose ends share 32 bytes with their
    neighbours': the bits of passes that each wait for the one before."""
    g = generator(T, F, K, 28)
    dy, x, wg, wu = (pitched(whole(g, *s, BF16, 1)) for s in ((T, F), (T, K), (F, K), (F, K)))
    gate, up = (whole(g, T, F, BF16, 1) for _ in range(2))
    ws = torch.empty(vnm.vnm_gated_linear_backward_workspace_size(T, F), dtype=torch.uint8, device=DEV)
    dx = torch.empty((T, K), dtype=BF16, device=DEV)
    dwg, dwu = (torch.empty((F, K), dtype=w_type, device=DEV) for _ in range(2))

    def run(wait=lambda: None):
        dwg.zero_()
        dwu.zero_()
        for _ in range(12):
            wait()
            vnm.vnm_gated_linear_backward(dy, x, wg, wu, gate, up, act=NONE, dx=dx, dwg=dwg, dwu=dwu, accumulate=True, workspace=ws)

    run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [v.clone() for v in (dx, dwg, dwu)]
    if w_type == F32:
        assert torch.equal(dwg.double(), 12 * ((dy * up).double().t() @ x.double()))
        assert torch.equal(dwu.double(), 12 * ((dy * gate).double().t() @ x.double()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for way in [run] * 20 + [graph.replay] * 20:
        way()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (dx, dwg, dwu)))
