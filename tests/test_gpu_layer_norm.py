"""Layer normalisation on the GPU against its 64-bit form (gated_ref), within
the error bounds derived there, and a run of it together with the scan and step."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from nonlinear_rnn_iteration_b200 import binding
from test_gpu_gated_scan import TYPES, f64, within

pytestmark = pytest.mark.gpu


def make(M, P, N, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, P, N)) * scale + 0.5).to(TYPES[dtype]).cuda()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal((P, N))).float().cuda()
    b = torch.from_numpy(rng.standard_normal((P, N))).float().cuda()
    dy = torch.from_numpy(rng.standard_normal((M, P, N))).to(TYPES[dtype]).cuda()
    return x, w, b, dy


# widths around a lane's, a warp's and a block's share, odd ones, heads, and rows of one value
SHAPES = [(1, 1, 1), (3, 2, 2), (5, 1, 7), (9, 24, 8), (200, 3, 16), (1000, 8, 64), (33, 1, 65), (17, 5, 100),
          (700, 1, 128), (4, 3, 255), (50, 2, 256), (3, 1, 1000), (300, 1, 1024), (6, 1, 1030), (2, 3, 2048),
          (5, 1, 4097), (8, 1, 8192), (2, 1, 20001), (1, 1, 70000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    M, P, N = shape
    x, w, b, dy = make(M, P, N, dtype, M + N, scale=2.0)
    if N % 3 == 0:
        b = None
    if N % 5 == 0:
        w = None
    eps = 1e-5
    y, mean, rstd = binding.layer_norm_forward(x, w, b, eps, want_stats=True) if w is not None or b is not None else \
        binding.layer_norm_forward(x, torch.ones(P, N, device="cuda"), None, eps, want_stats=True)
    dx, dw, db = binding.layer_norm_backward(x, dy, mean, rstd, w, param_shape=(P, N))
    n = [f64(t) for t in (x, w, b, dy)]
    yr, mr, rr = ref.norm(n[0], n[1], n[2], eps)
    ey, em, er, edx, ew, eb = ref.norm_bounds(n[0], n[1], n[2], eps, dtype, n[3])
    within(y, yr, ey, "y")
    within(mean, mr, em, "mean")
    within(rstd, rr, er, "rstd")
    dxr, dwr, dbr = ref.norm_backward(n[0], n[3], n[1], eps)
    within(dx, dxr, edx, "dx")
    within(dw, dwr, ew, "dweight")
    within(db, dbr, eb, "dbias")
    assert dw.shape == db.shape == (P, N)


# several batches of rows for each thread, at each count of threads to a row; the last piece of a row short
@pytest.mark.parametrize("M,P,N,dtype", [(1500, 3, 2048, "bf16"), (1111, 2, 1000, "bf16"), (2500, 1, 520, "f32"),
                                         (900, 5, 296, "bf16"), (600, 1, 8192, "f32"), (700, 1, 12344, "f32"),
                                         (700, 1, 9000, "bf16")])
def test_many_rows_a_thread_and_in_place(M, P, N, dtype):
    x, w, b, dy = make(M, P, N, dtype, M)
    n = [f64(t) for t in (x, w, b, dy)]
    y, mean, rstd = binding.layer_norm_forward(x, w, b, want_stats=True)
    dx, dw, db = binding.layer_norm_backward(x, dy, mean, rstd, w)
    ey, em, er, edx, ew, eb = ref.norm_bounds(n[0], n[1], n[2], 1e-5, dtype, n[3])
    for got, want, bound, name in zip((y, mean, rstd), ref.norm(n[0], n[1], n[2], 1e-5), (ey, em, er),
                                      ("y", "mean", "rstd")):
        within(got, want, bound, name)
    for got, want, bound, name in zip((dx, dw, db), ref.norm_backward(n[0], n[3], n[1], 1e-5), (edx, ew, eb),
                                      ("dx", "dweight", "dbias")):
        within(got, want, bound, name)
    # dx over dy and over x, and y over x: the same bits
    code = binding.BF16 if dtype == "bf16" else binding.F32
    ws = torch.empty(binding.pararnn_layer_norm_workspace_bytes(M, P, N), dtype=torch.uint8, device="cuda")
    for over in ("dy", "x"):
        xs, gs = x.clone(), dy.clone()
        to = gs if over == "dy" else xs
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        assert binding.pararnn_layer_norm_backward(M, P, N, code, xs, w, mean, rstd, gs, to, dw2, db2, ws, ws.numel(),
                                                   None) == binding.OK
        assert torch.equal(to, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    xs = x.clone()
    assert binding.pararnn_layer_norm_forward(M, P, N, code, xs, w, b, 1e-5, xs, None, None, None, 0,
                                              None) == binding.OK
    assert torch.equal(xs, y)


def test_shapes_of_the_parameters():
    x = torch.randn(2, 5, 3, 16, device="cuda")
    want, _, _ = ref.norm(f64(x).reshape(30, 1, 16), None, None, 1e-5)
    y, m, r = binding.layer_norm_forward(x)
    assert m is None and r is None
    assert np.abs(f64(y).reshape(30, 1, 16) - want).max() < 1e-5
    for shape in ((16,), (3, 16), (5, 3, 16), (2, 5, 3, 16)):
        w = torch.rand(shape, device="cuda") + 0.5
        y, m, r = binding.layer_norm_forward(x, w, want_stats=True)
        assert m.shape == (2, 5, 3) and np.abs(f64(y) - want.reshape(2, 5, 3, 16) * f64(w)).max() < 1e-5
        dx, dw, db = binding.layer_norm_backward(x, torch.ones_like(x), m, r, w)
        assert dw.shape == db.shape == shape and (db == 30 * 16 / w.numel()).all()
    assert binding.layer_norm_backward(x, x, m, r, want_dparams=False)[1:] == (None, None)


def test_directional_difference():
    x, w, b, dy = make(7, 2, 40, "f32", 3)
    n = [f64(t) for t in (x, w, b, dy)]
    _, m, r = binding.layer_norm_forward(x, w, b, 1e-3, want_stats=True)
    dx, dw, db = (f64(t) for t in binding.layer_norm_backward(x, dy, m, r, w))
    _, _, _, edx, ew, eb = ref.norm_bounds(n[0], n[1], n[2], 1e-3, "f32", n[3])
    rng = np.random.default_rng(4)
    v, vw, vb = (rng.standard_normal(a.shape) for a in (n[0], n[1], n[2]))
    e = 1e-5
    loss = lambda s: (ref.norm(n[0] + s * v, n[1] + s * vw, n[2] + s * vb, 1e-3)[0] * n[3]).sum()  # noqa: E731
    num = (loss(e) - loss(-e)) / (2 * e)
    got = (dx * v).sum() + (dw * vw).sum() + (db * vb).sum()
    assert abs(num - got) <= (edx * abs(v)).sum() + (ew * abs(vw)).sum() + (eb * abs(vb)).sum() + 1e-6 * abs(num)


def test_far_mean_constant_rows_and_not_finite():
    # a mean 4096 times the spread: the two-pass variance keeps its digits (exact inputs in float32)
    x = torch.randint(-8, 9, (40, 1, 512), device="cuda").float() / 8 + 4096.0
    y, m, r = binding.layer_norm_forward(x, eps=0.0, want_stats=True)
    yr, mr, rr = ref.norm(f64(x), None, None, 0.0)
    ey, em, er = ref.norm_bounds(f64(x), None, None, 0.0, "f32")
    within(y, yr, ey, "y")
    within(r.view(40, 1), rr, er, "rstd")
    # a constant row is all shift
    c = torch.full((3, 1, 200), 5.0, device="cuda", dtype=torch.bfloat16)
    b = torch.randn(1, 200, device="cuda")
    y, _, _ = binding.layer_norm_forward(c, None, b)
    assert torch.equal(y, b.bfloat16().expand(3, 1, 200))
    # a row that is not finite spoils itself only
    c = torch.randn(70, 2, 64, device="cuda")
    want, _, _ = binding.layer_norm_forward(c, torch.ones(2, 64, device="cuda"))
    c2 = c.clone()
    c2[3, 1, 5] = float("inf")
    with pytest.raises(binding.PararnnError) as e:
        binding.layer_norm_forward(c2, torch.ones(2, 64, device="cuda"))
    assert e.value.status == binding.ENONFINITE
    y, _, _ = binding.layer_norm_forward(c2, torch.ones(2, 64, device="cuda"), sync_status=False)
    assert torch.isnan(y[3, 1, 5]) and not torch.isfinite(y[3, 1]).all()
    y[3, 1] = want[3, 1]
    assert torch.equal(y, want)


def test_empty_in_place_graph_and_repeats():
    y, m, r = binding.layer_norm_forward(torch.zeros(0, 3, 8, device="cuda"), torch.ones(3, 8, device="cuda"),
                                         want_stats=True)
    dx, dw, db = binding.layer_norm_backward(torch.zeros(0, 3, 8, device="cuda"), torch.zeros(0, 3, 8, device="cuda"),
                                             m, r, torch.ones(3, 8, device="cuda"))
    assert y.shape == dx.shape == (0, 3, 8) and (dw == 0).all() and (db == 0).all()
    x, w, b, dy = make(500, 3, 136, "bf16", 6)

    def both():
        y, m, r = binding.layer_norm_forward(x, w, b, want_stats=True, sync_status=False)
        return (y,) + binding.layer_norm_backward(x, dy, m, r, w, sync_status=False)

    want = both()
    assert all(torch.equal(a, c) for a, c in zip(want, both()))
    z = x.clone()
    assert torch.equal(binding.layer_norm_forward(z, w, b, out=z)[0], want[0])
    side = torch.cuda.Stream()
    y, m, r = binding.layer_norm_forward(x, w, b, want_stats=True, stream=side)
    got = (y,) + binding.layer_norm_backward(x, dy, m, r, w, stream=side)
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, out))
    # a buffer that is aligned to its elements only
    off = torch.cat([x.new_zeros(1), x.reshape(-1)])[1:].view(x.shape)
    n = [f64(t) for t in (x, w, b)]
    within(binding.layer_norm_forward(off, w, b)[0], ref.norm(*n, 1e-5)[0], ref.norm_bounds(*n, 1e-5, "bf16")[0], "y")


def test_offsets_past_32_bits():
    M, N = 1_100_000, 2048
    x = torch.empty(M, 1, N, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    for lo in range(0, M, 100_000):
        x[lo:lo + 100_000] = torch.randn(100_000, 1, N, device="cuda", dtype=torch.bfloat16, generator=g)
    y, m, r = binding.layer_norm_forward(x, want_stats=True)
    dx, dw, db = binding.layer_norm_backward(x, x, m, r)
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    n = f64(x[rows])
    ey, _, _, edx, _, _ = ref.norm_bounds(n, None, None, 1e-5, "bf16", n)
    within(y[rows], ref.norm(n, None, None, 1e-5)[0], ey, "y")
    within(dx[rows], ref.norm_backward(n, n, None, 1e-5)[0], edx, "dx")
    s = torch.zeros(N, dtype=torch.float64, device="cuda")
    a = torch.zeros_like(s)
    for lo in range(0, M, 100_000):
        s += x[lo:lo + 100_000, 0].double().sum(0)
        a += x[lo:lo + 100_000, 0].double().abs().sum(0)
    within(db, f64(s), (M + 2) * ref.U * f64(a), "dbias")


def test_together_as_a_layer():
    """normalised pre-activations, the scan, heads of its output normalised, the gradients back through all three,
    and decoding that carries the prompt's state on"""
    B, T, D, heads = 2, 90, 64, 4
    rng = np.random.default_rng(9)
    dev = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    x, w1, b1 = dev(rng.standard_normal((B, T, 3, D))), dev(1 + 0.2 * rng.standard_normal((3, D))), dev(
        0.2 * rng.standard_normal((3, D)))
    lam, w2, dy = dev(rng.uniform(-7, 0, D)), dev(1 + 0.2 * rng.standard_normal((heads, D // heads))), dev(
        rng.standard_normal((B, T, heads, D // heads)))
    reset = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    reset[:, 40] = True
    px, m1, r1 = binding.layer_norm_forward(x, w1, b1, want_stats=True)
    H, last, ck = binding.gated_scan_forward(px, lam, 8.0, None, reset, want_grad=True)
    y, m2, r2 = binding.layer_norm_forward(H.view(B, T, heads, -1), w2, None, want_stats=True)
    dH, dw2, _ = binding.layer_norm_backward(H.view(B, T, heads, -1), dy, m2, r2, w2)
    dpx, dlam, _ = binding.gated_scan_backward(px, lam, ck, dH.view(B, T, D), 8.0, reset)
    dx, dw1, db1 = binding.layer_norm_backward(x, dpx, m1, r1, w1)
    # the whole layer in 64 bits, and its gradients by torch's autograd
    leaves = [t.cpu().double().requires_grad_() for t in (x, w1, b1, lam, w2)]
    X, W1, B1, L, W2 = leaves
    p = torch.nn.functional.layer_norm(X, (D,), None, None, 1e-5) * W1 + B1
    r, i = torch.sigmoid(p[:, :, 0]), torch.sigmoid(p[:, :, 1])
    la = -8.0 * torch.nn.functional.softplus(L) * r
    u = torch.sqrt(-torch.expm1(2 * la)) * i * p[:, :, 2]
    h, hs = torch.zeros(B, D, dtype=torch.float64), []
    for t in range(T):
        h = (0 if t == 40 else torch.exp(la[:, t]) * h) + u[:, t]
        hs.append(h)
    Hr = torch.stack(hs, 1)
    yr = torch.nn.functional.layer_norm(Hr.view(B, T, heads, -1), (D // heads,), None, None, 1e-5) * W2
    yr.backward(dy.cpu().double())
    # each of the five steps adds relative errors of a few 2^-20 (SIG) times the memory's and the norms' condition,
    # which the weights and the spread of the rows keep below 2^5
    tol = 2.0 ** -13
    for name, got, want in [("y", y, yr), ("dx", dx, X.grad), ("dw1", dw1, W1.grad), ("db1", db1, B1.grad),
                            ("dlam", dlam, L.grad), ("dw2", dw2, W2.grad)]:
        want = want.detach().numpy()
        assert np.abs(f64(got) - want).max() <= tol * np.abs(want).max(), name
    # decoding: the next two tokens on a cache whose slots hold the prompts' states
    cache = torch.zeros(6, D, device="cuda")
    slots = torch.tensor([5, 2], dtype=torch.int32, device="cuda")
    cache[slots.long()] = last
    h = Hr[:, -1].detach().numpy()
    for k in range(2):
        xt = dev(rng.standard_normal((B, 3, D)))
        pt, _, _ = binding.layer_norm_forward(xt, w1, b1)
        yt = binding.gated_scan_step(pt, lam, cache, 8.0, slots)
        pn = ref.norm(f64(xt), f64(w1), f64(b1), 1e-5)[0]
        h = ref.forward(pn[:, None], f64(lam), 8.0, h)[1]
        assert np.abs(f64(yt) - h).max() <= tol * np.abs(h).max()
    assert torch.equal(cache[slots.long()], yt)


# N whose float32 reciprocal times an exact sum misses the mean (56 to 1000), others, and each count of threads to a row
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [14, 56, 120, 1000, 3000, 6040, 12000])
def test_means_are_quotients(N, dtype):
    """Values of 8 bits: every partial sum of up to 2^14 of them is exact in float32, so a mean that is the rounded
    quotient is the value itself, and what is left of a constant row, forward and backward, is nothing."""
    value = torch.tensor([1.0, 101.0, -724.0, 15424.0, 9984.0], device="cuda")
    M = 5 * max(1, 800_000 // N)
    x = value.repeat(M // 5).view(M, 1, 1).expand(M, 1, N).to(TYPES[dtype]).contiguous()
    b = torch.randn(1, N, device="cuda")
    signs = torch.tensor([1.0, -1.0], device="cuda").repeat(M * N // 2).view(M, 1, N).to(TYPES[dtype])
    for off in (0, 1):  # with 16-byte accesses where N allows them, and of single values
        at = lambda t: torch.cat([t.new_zeros(off), t.reshape(-1)])[off:].view(t.shape)  # noqa: E731
        y, m, r = binding.layer_norm_forward(at(x), None, b, want_stats=True)
        assert torch.equal(m.view(-1), x[:, 0, 0].float())
        assert torch.equal(y, b.to(y.dtype).expand(M, 1, N))
        y, _, _ = binding.layer_norm_forward(at(x), None, b, eps=0.0, sync_status=False)
        assert torch.isnan(y).all()  # 0 times Inf
        # rows of 1 and -1 in turn: their xh add up to zero, whatever the order, as each has its opposite beside
        # it; a constant dL/dy less its own mean is then all of dL/dx
        _, m, r = binding.layer_norm_forward(at(signs), want_stats=True)
        assert (m == 0).all()
        dx, _, _ = binding.layer_norm_backward(at(signs), at(x), m, r)
        assert (dx == 0).all()


def test_mean_of_an_exact_sum_is_rounded_once():
    # multiples of 1/2 next to 4096: 14 bits, and 9 more for the sum of 500 of them, so the sum is exact
    x = torch.randint(-8, 9, (400, 1, 500), device="cuda").float() / 2 + 4096.0
    _, m, _ = binding.layer_norm_forward(x, want_stats=True)
    want = f64(x).mean(-1)
    within(m, want, ref.U * np.abs(want), "mean")
