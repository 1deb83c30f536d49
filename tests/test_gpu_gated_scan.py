"""The gated linear recurrence on the GPU against its 64-bit form (gated_ref),
within the error bounds derived there."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from nonlinear_rnn_iteration_b200 import binding

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DECAY = 8.0


def make(B, T, D, dtype, packed, seed, h0=True):
    """inputs as (torch on the GPU, the same values in numpy float64)"""
    rng = np.random.default_rng(seed)
    px = torch.from_numpy(np.clip(rng.standard_normal((B, T, 3, D)), -8, 8)).to(TYPES[dtype]).cuda()
    # from memories of thousands of steps to gates that close within one
    lam = torch.from_numpy(rng.uniform(-9, 1, D)).float().cuda()
    h = torch.from_numpy(rng.standard_normal((B, D))).float().cuda() if h0 else None
    reset = torch.from_numpy((rng.random((B, T)) < 0.02).astype(np.uint8)).cuda() if packed else None
    dH = torch.from_numpy(rng.standard_normal((B, T, D))).to(TYPES[dtype]).cuda()
    dl = torch.from_numpy(rng.standard_normal((B, D))).float().cuda()
    return px, lam, h, reset, dH, dl


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound + 1e-30)
    assert not bad.any(), "%s: %d of %d outside; worst %.3g of the bound" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / (bound + 1e-30)))


# lengths around the warps', tiles' and clusters' steps, widths around the tile's and not a multiple of 16 bytes
SHAPES = [(1, 1, 1), (2, 2, 8), (1, 7, 64), (3, 8, 5), (2, 9, 72), (1, 16, 130), (1, 17, 64), (2, 63, 24), (1, 64, 64),
          (1, 65, 128), (2, 127, 8), (1, 128, 66), (3, 129, 40), (1, 257, 16), (2, 500, 33), (1, 1025, 96),
          (4, 300, 200), (1, 2100, 8), (1, 4200, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, packed, dtype):
    B, T, D = shape
    px, lam, h0, reset, dH, dl = make(B, T, D, dtype, packed, 100 + T + D, h0=T != 64)
    n = [f64(t) for t in (px, lam, h0, dH, dl)]
    rs = None if reset is None else reset.cpu().numpy()
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True)
    dpx, dlam, dh0 = binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True)
    Hr, lr = ref.forward(n[0], n[1], DECAY, n[2], rs)
    eH, el = ref.forward_bound(n[0], n[1], DECAY, dtype, n[2], rs)
    within(H, Hr, eH, "H")
    within(last, lr, el, "h_last")
    assert torch.equal(H[:, -1], last.to(H.dtype))  # the state rounded once
    gp, gl, g0 = ref.backward(n[0], n[1], DECAY, n[3], n[2], rs, n[4])
    ep, ela, e0 = ref.backward_bound(n[0], n[1], DECAY, n[3], dtype, n[2], rs, n[4])
    within(dpx, gp, ep, "dpx")
    within(dlam, gl, ela, "dlam")
    within(dh0, g0, e0, "dh0")
    # without gradients the forward gives the same bits
    H2, last2, none = binding.gated_scan_forward(px, lam, DECAY, h0, reset)
    assert none is None and torch.equal(H, H2) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shape", [(1, 9000, 24), (1, 13001, 7), (3, 7000, 130)])
def test_few_long_channels(shape, packed, dtype):
    """T in ranges that run at once: within the bounds, the same bits again, and the state updated in place"""
    B, T, D = shape
    px, lam, h0, reset, dH, dl = make(B, T, D, dtype, packed, 300 + D)
    if packed:  # long sequences too, across the ranges
        reset[:, 1000:8000] = 0
        reset[0, 5000] = 1
    n = [f64(t) for t in (px, lam, h0, dH, dl)]
    rs = None if reset is None else reset.cpu().numpy()
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True)
    dpx, dlam, dh0 = binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True)
    Hr, lr = ref.forward(n[0], n[1], DECAY, n[2], rs)
    eH, el = ref.forward_bound(n[0], n[1], DECAY, dtype, n[2], rs)
    within(H, Hr, eH, "H")
    within(last, lr, el, "h_last")
    gp, gl, g0 = ref.backward(n[0], n[1], DECAY, n[3], n[2], rs, n[4])
    ep, ela, e0 = ref.backward_bound(n[0], n[1], DECAY, n[3], dtype, n[2], rs, n[4])
    within(dpx, gp, ep, "dpx")
    within(dlam, gl, ela, "dlam")
    within(dh0, g0, e0, "dh0")
    state = h0.clone()
    H2, _, _ = binding.gated_scan_forward(px, lam, DECAY, state, reset, h_last=state)
    assert torch.equal(H, H2) and torch.equal(state, last)
    again = binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True)
    assert all(torch.equal(a, b) for a, b in zip(again, (dpx, dlam, dh0)))
    # a workspace for the status alone: one pass, another order of joins
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    H3, last3, _ = binding.gated_scan_forward(px, lam, DECAY, h0, reset, workspace=small)
    within(H3, Hr, eH, "H in one pass")
    within(last3, lr, el, "h_last in one pass")


def test_directional_difference():
    """the kernels' gradients against central differences of the 64-bit form's loss"""
    px, lam, h0, reset, dH, dl = make(2, 150, 40, "f32", True, 5)
    n = [f64(t) for t in (px, lam, h0, dH, dl)]
    rs = reset.cpu().numpy()
    _, _, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True)
    dpx, dlam, dh0 = (f64(t) for t in binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True))
    ep, ela, e0 = ref.backward_bound(n[0], n[1], DECAY, n[3], "f32", n[2], rs, n[4])
    rng = np.random.default_rng(6)
    v, vl, vh = rng.standard_normal(n[0].shape), rng.standard_normal(n[1].shape), rng.standard_normal(n[2].shape)

    def loss(s):
        H, last = ref.forward(n[0] + s * v, n[1] + s * vl, DECAY, n[2] + s * vh, rs)
        return (H * n[3]).sum() + (last * n[4]).sum()

    e = 1e-5
    num = (loss(e) - loss(-e)) / (2 * e)
    got = (dpx * v).sum() + (dlam * vl).sum() + (dh0 * vh).sum()
    bound = (ep * np.abs(v)).sum() + (ela * np.abs(vl)).sum() + (e0 * np.abs(vh)).sum()
    assert abs(num - got) <= bound + 1e-6 * abs(num)  # the difference's own error is of order e^2


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 33)])
def test_reset_stops_nan_and_inf(dtype, D):
    """what is not finite before a marked step reaches nothing behind it, forward or backward"""
    px, lam, h0, _, dH, _ = make(2, 400, D, dtype, False, 7)
    reset = torch.zeros(2, 400, dtype=torch.bool, device="cuda")
    reset[0, 0] = reset[0, 150] = reset[1, 399] = True
    h0[0] = float("nan")
    px[0, 149, 2] = float("inf")
    px[1, 100, 2] = float("nan")
    dH[0, 150] = float("inf")  # its own step, not the ones before it
    with pytest.raises(binding.PararnnError) as e:
        binding.gated_scan_forward(px, lam, DECAY, h0, reset)
    assert e.value.status == binding.ENONFINITE
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True, sync_status=False)
    rs = reset.cpu().numpy().astype(np.uint8)
    clean = px.clone()
    clean[0, 149, 2] = 0
    clean[1, 100, 2] = 0
    h1 = h0.clone()
    h1[0] = 0
    want, lr = ref.forward(f64(clean), f64(lam), DECAY, f64(h1), rs)
    bound, el = ref.forward_bound(f64(clean), f64(lam), DECAY, dtype, f64(h1), rs)
    within(H[0, :149], want[0, :149], bound[0, :149], "before")
    within(H[0, 150:], want[0, 150:], bound[0, 150:], "behind")
    assert not torch.isfinite(H[0, 149]).any() and torch.isnan(H[1, 100:399]).all()
    within(H[1, 399], want[1, 399], bound[1, 399], "last step")
    within(last, lr, el, "h_last")
    dpx, _, dh0 = binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, want_dh0=True, sync_status=False)
    g = dH.clone()
    g[0, 150] = 0
    gp, _, _ = ref.backward(f64(clean), f64(lam), DECAY, f64(g), f64(h1), rs)
    ep, _, _ = ref.backward_bound(f64(clean), f64(lam), DECAY, f64(g), dtype, f64(h1), rs)
    within(dpx[0, :149], gp[0, :149], ep[0, :149], "dpx before")
    within(dpx[0, 151:], gp[0, 151:], ep[0, 151:], "dpx behind")
    assert (dh0[0] == 0).all()  # step 0 is marked


def test_every_step_marked_and_none():
    px, lam, h0, _, dH, _ = make(2, 130, 24, "f32", False, 8)
    none = torch.zeros(2, 130, dtype=torch.uint8, device="cuda")
    H0, l0, c0 = binding.gated_scan_forward(px, lam, DECAY, h0, None, want_grad=True)
    H1, l1, c1 = binding.gated_scan_forward(px, lam, DECAY, h0, none, want_grad=True)
    assert torch.equal(H0, H1) and torch.equal(l0, l1) and torch.equal(c0, c1)
    every = torch.full((2, 130), 7, dtype=torch.uint8, device="cuda")  # any non-zero byte marks
    H, _, _ = binding.gated_scan_forward(px, lam, DECAY, h0, every)
    want, _ = ref.forward(f64(px), f64(lam), DECAY, f64(h0), every.cpu().numpy())
    bound, _ = ref.forward_bound(f64(px), f64(lam), DECAY, "f32", f64(h0), every.cpu().numpy())
    within(H, want, bound, "H")


def test_closed_and_open_gates():
    """gates at their limits: r = 0 (a = 1, b = 0), i = 0, y from subnormal to far past the exponential's range"""
    px, lam, h0, _, dH, _ = make(1, 70, 64, "f32", False, 9)
    px[:, :, 0] *= 40  # |p_r| to about 120
    px[:, :, 1] *= 40
    lam[::2] = torch.linspace(-90, 30, 32, device="cuda")
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, want_grad=True)
    dpx, dlam, _ = binding.gated_scan_backward(px, lam, ck, dH, DECAY)
    # U |p| more for the exponential's argument (|p| to 160: 2^-16), and a gate below 2^-126 is zero
    want, _ = ref.forward(f64(px), f64(lam), DECAY, f64(h0))
    bound, _ = ref.forward_bound(f64(px), f64(lam), DECAY, "f32", f64(h0))
    within(H, want, 16 * bound + 2.0 ** -60, "H")
    gp, gl, _ = ref.backward(f64(px), f64(lam), DECAY, f64(dH), f64(h0))
    ep, el, _ = ref.backward_bound(f64(px), f64(lam), DECAY, f64(dH), "f32", f64(h0))
    fine = np.isfinite(gp) & np.isfinite(ep)
    gp, ep = np.where(fine, gp, 0), np.where(fine, ep, np.inf)  # where b underflows in 64 bits too
    assert torch.isfinite(dpx).all() and torch.isfinite(dlam).all()
    within(dpx, gp, 16 * ep + 2.0 ** -55, "dpx")


@pytest.mark.parametrize("B,T,D", [(0, 5, 8), (2, 0, 8), (2, 5, 0)])
def test_empty(B, T, D):
    px = torch.zeros(B, T, 3, D, device="cuda")
    lam, h0, dl = torch.zeros(D, device="cuda"), torch.full((B, D), 3.0, device="cuda"), torch.full((B, D), 2.0,
                                                                                                 device="cuda")
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, want_grad=True)
    assert H.shape == (B, T, D) and torch.equal(last, h0)
    assert (binding.gated_scan_forward(px, lam, DECAY)[1] == 0).all()
    dpx, dlam, dh0 = binding.gated_scan_backward(px, lam, ck, torch.zeros(B, T, D, device="cuda"), DECAY, None, dl,
                                                 want_dh0=True)
    assert dpx.shape == px.shape and (dlam == 0).all() and torch.equal(dh0, dl)


def test_last_state_carries_on():
    """a prompt in two parts, the state updated in place, equals the whole within the bounds"""
    px, lam, h0, reset, _, _ = make(2, 300, 72, "bf16", True, 10)
    want, lr = ref.forward(f64(px), f64(lam), DECAY, f64(h0), reset.cpu().numpy())
    bound, el = ref.forward_bound(f64(px), f64(lam), DECAY, "bf16", f64(h0), reset.cpu().numpy())
    state = h0.clone()
    parts = []
    for lo, hi in ((0, 131), (131, 132), (132, 300)):
        H, last, _ = binding.gated_scan_forward(px[:, lo:hi].contiguous(), lam, DECAY, state,
                                                reset[:, lo:hi].contiguous(), h_last=state)
        assert last is state
        parts.append(H)
    within(torch.cat(parts, 1), want, bound, "H")
    within(state, lr, el, "state")


def test_repeats_bit_for_bit_and_in_a_graph_on_another_stream():
    px, lam, h0, reset, dH, dl = make(3, 700, 136, "bf16", True, 11)
    side = torch.cuda.Stream()

    def both():
        H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True, sync_status=False)
        return (H, last) + binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True,
                                                       sync_status=False)

    want = both()
    torch.cuda.synchronize()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, both()))
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True, stream=side)
    got = (H, last) + binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with torch.cuda.stream(side):
        both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    keep = px.clone()
    px.zero_()
    graph.replay()
    px.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_views_that_start_off_16_bytes():
    """element-aligned buffers are enough"""
    px, lam, h0, _, dH, _ = make(2, 140, 64, "bf16", False, 12)
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, want_grad=True)
    ref_grads = binding.gated_scan_backward(px, lam, ck, dH, DECAY)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    out = torch.empty(H.numel() + 1, dtype=H.dtype, device="cuda")[1:].view(H.shape)
    H2, last2, ck2 = binding.gated_scan_forward(off(px), off(lam), DECAY, off(h0), want_grad=True, out=out)
    got = binding.gated_scan_backward(off(px), off(lam), off(ck2), off(dH), DECAY)
    # another path may order the joins of the scan differently: the bounds hold for both
    n = [f64(t) for t in (px, lam, h0, dH)]
    within(H2, *_pair(ref.forward(n[0], n[1], DECAY, n[2])[0], ref.forward_bound(n[0], n[1], DECAY, "bf16", n[2])[0]), "H")
    gp, gl, _ = ref.backward(n[0], n[1], DECAY, n[3], n[2])
    ep, el, _ = ref.backward_bound(n[0], n[1], DECAY, n[3], "bf16", n[2])
    for dpx, dlam, _ in (ref_grads, got):
        within(dpx, gp, ep, "dpx")
        within(dlam, gl, el, "dlam")


def _pair(a, b):
    return a, b


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,n_slots", [(1, 1, 1), (1, 4096, 3), (5, 33, 9), (70, 130, 200), (300, 64, 310)])
def test_step(N, D, n_slots, dtype):
    rng = np.random.default_rng(N + D)
    px = torch.from_numpy(np.clip(rng.standard_normal((N, 3, D)), -8, 8)).to(TYPES[dtype]).cuda()
    lam = torch.from_numpy(rng.uniform(-9, 1, D)).float().cuda()
    state = torch.from_numpy(rng.standard_normal((n_slots, D))).float().cuda()
    slots = rng.permutation(n_slots)[:N].astype(np.int32)
    if N > 2:
        slots[1] = -1
    y = torch.full((N, D), 7.0, dtype=TYPES[dtype], device="cuda")
    old = f64(state)
    got = binding.gated_scan_step(px, lam, state, DECAY, torch.from_numpy(slots).cuda(), out=y)
    assert got is y
    want, new = ref.step(f64(px), f64(lam), DECAY, old, slots)
    Hb, eb = ref.forward_bound(f64(px)[:, None], f64(lam), DECAY, dtype, old[np.maximum(slots, 0)])
    live = slots >= 0
    within(y[torch.from_numpy(live).cuda()], want[live], Hb[live, 0], "y")
    assert (y[torch.from_numpy(~live).cuda()] == 7.0).all()  # rows of padding are left as they were
    bound = np.zeros_like(new)
    bound[slots[live]] = eb[live]
    within(state, new, bound, "state")  # slots that no row names keep their bits


def test_step_rows_of_one_slot_in_order():
    """several tokens of a sequence in one call: the states that the scan gives"""
    px, lam, h0, _, _, _ = make(2, 40, 72, "f32", False, 13)
    state = torch.zeros(5, 72, device="cuda")
    state[1], state[4] = h0[0], h0[1]
    slots = torch.tensor([1, 4] * 40, dtype=torch.int32, device="cuda")
    rows = px.transpose(0, 1).reshape(80, 3, 72).contiguous()  # t-major: rows of both sequences in turn
    y = binding.gated_scan_step(rows, lam, state, DECAY, slots)
    want, lr = ref.forward(f64(px), f64(lam), DECAY, f64(h0))
    bound, el = ref.forward_bound(f64(px), f64(lam), DECAY, "f32", f64(h0))
    within(y.view(40, 2, 72).transpose(0, 1), want, bound, "y")
    within(state[[1, 4]], lr, el, "state")
    assert (state[[0, 2, 3]] == 0).all()


def test_step_of_many_rows():
    """more rows than one launch takes, a slot named on both sides of its end, slots off 16 bytes"""
    N, D, n_slots = 8203, 12, 9000
    rng = np.random.default_rng(16)
    px = torch.from_numpy(np.clip(rng.standard_normal((N, 3, D)), -8, 8)).float().cuda()
    lam = torch.from_numpy(rng.uniform(-6, 0, D)).float().cuda()
    state = torch.from_numpy(rng.standard_normal((n_slots, D))).float().cuda()
    slots = rng.permutation(n_slots)[:N].astype(np.int32)
    slots[8191] = slots[8192] = slots[8202] = slots[17] = slots[16]
    old = f64(state)
    dev = torch.from_numpy(np.concatenate([[0], slots]).astype(np.int32)).cuda()[1:]
    y = binding.gated_scan_step(px, lam, state, DECAY, dev)
    want, new = ref.step(f64(px), f64(lam), DECAY, old, slots)
    # five steps of the slot named five times; each step's bound is that of one step, and the decay only shrinks it
    Hb, _ = ref.forward_bound(f64(px)[:, None], f64(lam), DECAY, "f32", np.maximum(np.abs(old[slots]), 4.0))
    within(y, want, 5 * np.maximum(Hb[:, 0], Hb[[16, 17, 8191, 8192, 8202], 0].max()), "y")
    within(state, new, 5 * Hb.max(), "state")
    torch.cuda.synchronize()
    state2 = torch.from_numpy(old).float().cuda()
    y2 = binding.gated_scan_step(px, lam, state2, DECAY)  # without slots: row n on slot n
    want2, new2 = ref.step(f64(px), f64(lam), DECAY, old, np.arange(N))
    within(y2, want2, 2 * ref.forward_bound(f64(px)[:, None], f64(lam), DECAY, "f32", old[:N])[0][:, 0], "y2")


def test_two_streams_at_once():
    """calls that overlap on the GPU with buffers of their own give what they give alone"""
    cases = [make(2, 3000, 200, "bf16", True, 17), make(1, 9000, 48, "f32", False, 18)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def run(c, st):
        px, lam, h0, reset, dH, dl = c
        H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True, stream=st,
                                                 sync_status=False)
        return (H, last) + binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True, stream=st,
                                                       sync_status=False)

    alone = [run(c, None) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(c, st) for c, st in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_step_without_slots_and_bad_slots():
    px, lam, h0, _, _, _ = make(6, 1, 64, "f32", False, 14)
    state = torch.cat([h0, h0])
    y = binding.gated_scan_step(px[:, 0].contiguous(), lam, state, DECAY)
    H, last, _ = binding.gated_scan_forward(px, lam, DECAY, h0)
    bound, _ = ref.forward_bound(f64(px), f64(lam), DECAY, "f32", f64(h0))
    within(y, f64(H[:, 0]), 2 * bound[:, 0], "y")
    assert torch.equal(state[6:], h0) and torch.equal(state[:6], y)
    slots = torch.tensor([0, 12, 3, -7, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    before = state.clone()
    out = torch.full((6, 64), 9.0, device="cuda")
    with pytest.raises(binding.PararnnError) as e:
        binding.gated_scan_step(px[:, 0].contiguous(), lam, state, DECAY, slots, out=out)
    assert e.value.status == binding.EINVAL and "out of range" in str(e.value)
    assert (out[[1, 3, 4]] == 9.0).all() and (out[[0, 2, 5]] != 9.0).all()
    keep = [1, 2, 4, 6, 7, 8, 9, 10, 11]
    assert torch.equal(state[keep], before[keep])
    # padding alone, and no rows
    pad = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    assert (binding.gated_scan_step(px[:, 0].contiguous(), lam, state, DECAY, pad) == 0).all()
    assert binding.gated_scan_step(px[:0, 0].contiguous(), lam, state, DECAY).shape == (0, 64)


def test_offsets_past_32_bits():
    """2.6 thousand million pre-activations: the last rows of the last channels"""
    B, T, D = 1, 70000, 12296
    px = torch.empty(B, T, 3, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(15)
    for lo in range(0, T, 7000):
        px[:, lo:lo + 7000] = torch.randn(B, 7000, 3, D, device="cuda", dtype=torch.bfloat16, generator=g)
    lam = torch.rand(D, device="cuda", generator=g) * 6 - 7
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, want_grad=True)
    ch = torch.tensor([0, 1, 6000, D - 3, D - 1], device="cuda")
    n = [f64(px[:, :, :, ch].clamp(-8, 8)), f64(lam[ch])]
    want, lr = ref.forward(n[0], n[1], DECAY)
    bound, el = ref.forward_bound(n[0], n[1], DECAY, "bf16")
    within(H[:, :, ch], want, bound, "H")
    within(last[:, ch], lr, el, "h_last")
    dH = torch.zeros_like(H)
    dH[:, -1000:] = 1
    dH[:, 0] = 1
    dpx, _, _ = binding.gated_scan_backward(px, lam, ck, dH, DECAY)
    gp, _, _ = ref.backward(n[0], n[1], DECAY, f64(dH[:, :, ch]))
    ep, _, _ = ref.backward_bound(n[0], n[1], DECAY, f64(dH[:, :, ch]), "bf16")
    within(dpx[:, :, :, ch], gp, ep, "dpx")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 33])
def test_gradient_of_the_input_gate_that_overflows_is_reported(dtype, D):
    """dL/dp_i = l b i x (1 - i) = Inf while dL/dx = l b i and dL/dp_r (a^2 is 4e-18) are finite"""
    px = torch.zeros(1, 1, 3, D, device="cuda")
    px[:, :, 0], px[:, :, 2] = 20.0, 1e20
    lam = torch.full((D,), 2.4, device="cuda")  # y = 8 softplus(2.4) = 20
    px = px.to(TYPES[dtype])
    dH = torch.full((1, 1, D), 1e25, device="cuda").to(TYPES[dtype])
    _, _, ck = binding.gated_scan_forward(px, lam, DECAY, want_grad=True)
    dpx, _, _ = binding.gated_scan_backward(px, lam, ck, dH, DECAY, sync_status=False)
    assert torch.isinf(dpx[:, :, 1]).all() and torch.isfinite(dpx[:, :, [0, 2]]).all()
    with pytest.raises(binding.PararnnError) as e:
        binding.gated_scan_backward(px, lam, ck, dH, DECAY)
    assert e.value.status == binding.ENONFINITE


@pytest.mark.parametrize("dtype,D,off", [("f32", 64, 0), ("bf16", 64, 0), ("f32", 33, 0), ("bf16", 33, 0),
                                         ("f32", 64, 1), ("bf16", 130, 1)])
def test_gates_next_to_zero_and_large_inputs(dtype, D, off):
    """p_i down to -86 with x so large that i x is of order 1: the scan, its adjoint and the step agree there"""
    rng = np.random.default_rng(20)
    B, T = 2, 150
    p = np.clip(rng.standard_normal((B, T, 3, D)), -8, 8)
    p[:, :, 1] = rng.uniform(-86, 8, (B, T, D))
    px = torch.from_numpy(p).to(TYPES[dtype])
    px[:, :, 2] = (px[:, :, 2].double() * torch.exp(-px[:, :, 1].double().clamp(max=0))).to(px.dtype)  # to 2^124 N(0, 1)
    assert torch.isfinite(px).all()
    px = torch.cat([px.new_zeros(off), px.reshape(-1)]).cuda()[off:].view(px.shape)
    lam = torch.from_numpy(rng.uniform(-9, 1, D)).float().cuda()
    dH = torch.from_numpy(rng.standard_normal((B, T, D))).to(TYPES[dtype]).cuda()
    H, last, ck = binding.gated_scan_forward(px, lam, DECAY, want_grad=True)
    dpx, dlam, _ = binding.gated_scan_backward(px, lam, ck, dH, DECAY)
    # the exponential's argument is rounded: U |p| more, 2^-17 for |p| to 86 (and a half step of 2^-126 where a
    # gate or its product is next to that), so 16 times the bounds for |p| <= 8 holds
    n = [f64(t) for t in (px, lam, dH)]
    want, lr = ref.forward(n[0], n[1], DECAY)
    bound, el = ref.forward_bound(n[0], n[1], DECAY, dtype)
    within(H, want, 16 * bound, "H")
    within(last, lr, 16 * el, "h_last")
    gp, gl, _ = ref.backward(n[0], n[1], DECAY, n[2])
    ep, ela, _ = ref.backward_bound(n[0], n[1], DECAY, n[2], dtype)
    within(dpx, gp, 16 * ep + 2.0 ** -126, "dpx")
    within(dlam, gl, 16 * ela, "dlam")
    state = torch.zeros(B, D, device="cuda")
    for t in range(T):
        y = binding.gated_scan_step(px[:, t].contiguous(), lam, state, DECAY)
        within(y, want[:, t], 16 * bound[:, t], "step")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bits_do_not_follow_what_earlier_calls_left(dtype):
    """steps past the end of T, which rows off 16 bytes leave unread: whatever an earlier kernel's shared memory holds"""
    px, lam, h0, reset, dH, dl = make(2, 500, 33, dtype, True, 25)
    before = make(40, 1100, 33, dtype, False, 26)[0]
    got = []
    for p_i in (0.0, -80.0, float("nan")):
        before[:, :, 1] = p_i
        binding.gated_scan_forward(before, lam, DECAY, sync_status=False)
        H, last, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True, sync_status=False)
        got.append((H, last, ck) + binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True,
                                                               sync_status=False))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("decay,lam,scale", [(1e30, 0.5, 1e10), (3e38, 5.0, 1.0), (8.0, -1.0, 1e20)])
def test_gradients_overflow_only_where_they_are_large(decay, lam, scale, D):
    """decays so large that every state is its own step's input, and products of which only a factor overflows"""
    px, _, _, _, _, _ = make(2, 40, D, "f32", False, 21)
    px[:, :, 0].clamp_(-2, 2)
    if decay > 8.0:
        px[:, 5, 0] = -200.0  # r = 0: the state is kept (|x| beside it is within 1e20)
    dH = torch.full((2, 40, D), scale, device="cuda")
    if scale == 1e20:  # x (1 - i) is of order 1, x l is not
        px[:, :, 1] = 46.0
        px[:, :, 2] *= 1e20
        dH[:, :, ::2] = 1e18
    lam = torch.full((D,), lam, device="cuda")
    H, last, ck = binding.gated_scan_forward(px, lam, decay, want_grad=True)
    large = scale == 1e20  # there dL/dp_r, of order l x = 1e38 to 1e40, may be Inf, but nothing is NaN
    dpx, dlam, _ = binding.gated_scan_backward(px, lam, ck, dH, decay, sync_status=not large)
    assert torch.isfinite(H).all() and torch.isfinite(dpx[:, :, 1:]).all() and not torch.isnan(dpx).any()
    if not large:
        assert torch.isfinite(dpx).all() and torch.isfinite(dlam).all()
    if decay > 8.0:
        want = torch.sigmoid(px[:, :, 1].double()) * px[:, :, 2].double()
        want[:, 5] = want[:, 4]  # a = 1, b = 0
        assert (H.double() - want).abs().max() <= ref.GATE * want.abs().max()
        assert (dpx[:, :, 0] == 0).all() and (dlam == 0).all()
    state = torch.zeros(2, D, device="cuda")
    for t in range(7):
        y = binding.gated_scan_step(px[:, t].contiguous(), lam, state, decay)
        assert (y - H[:, t]).abs().max() <= 4 * ref.GATE * H[:, :7].abs().max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 64), (300, 40, 64), (2, 65, 33), (160, 130, 72), (5, 700, 640), (1, 2000, 64),
                                   (1, 2700, 130), (1, 9000, 24), (17, 3000, 64)])
def test_backward_stays_in_its_workspace(B, T, D, dtype):
    """a workspace of exactly the stated size, with a guard behind it, gives what the library's own gives"""
    px, lam, h0, reset, dH, dl = make(B, T, D, dtype, True, 22)
    _, _, ck = binding.gated_scan_forward(px, lam, DECAY, h0, reset, want_grad=True)
    want = binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True)
    size = binding.pararnn_gated_scan_workspace_bytes(B, T, D)
    buf = torch.full((size + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    got = binding.gated_scan_backward(px, lam, ck, dH, DECAY, reset, dl, want_dh0=True, workspace=buf[:size])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert (buf[size:] == 0xA5).all()
    H, last, _ = binding.gated_scan_forward(px, lam, DECAY, h0, reset)
    buf.fill_(0xA5)
    H2, last2, _ = binding.gated_scan_forward(px, lam, DECAY, h0, reset, workspace=buf[:size])
    assert torch.equal(H, H2) and torch.equal(last, last2) and (buf[size:] == 0xA5).all()


def test_decoding_steps_in_a_graph():
    """one captured step replayed per token, its inputs refilled between: the states that the scan gives"""
    px, lam, h0, _, _, _ = make(3, 30, 136, "bf16", False, 23)
    state = torch.zeros(7, 136, device="cuda")
    slots = torch.tensor([6, -1, 1, 4], dtype=torch.int32, device="cuda")
    state[slots[[0, 2, 3]].long()] = h0
    row = torch.zeros(4, 3, 136, dtype=torch.bfloat16, device="cuda")
    y = torch.full((4, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gated_scan_step(row, lam, state, DECAY, slots, out=y, sync_status=False)
    want, lr = ref.forward(f64(px), f64(lam), DECAY, f64(h0))
    bound, el = ref.forward_bound(f64(px), f64(lam), DECAY, "bf16", f64(h0))
    for t in range(30):
        row[[0, 2, 3]] = px[:, t]
        graph.replay()
        within(y[[0, 2, 3]], want[:, t], bound[:, t], "y")
    assert (y[1] == 5.0).all()
    within(state[slots[[0, 2, 3]].long()], lr, el, "state")


def test_overlapped_launches_beside_the_newton_solver():
    """calls whose launches overlap the end of the kernel before them, between cluster forwards of the Newton solver
    on one stream and each on the other's output: the bits of the same calls with the GPU idle between them"""
    B, T, D = 2, 1024, 64
    px, lam, _, _, dH, _ = make(B, T, D, "f32", False, 24)
    diag = torch.full((3, D), 0.5, device="cuda")

    def run(wait):
        out, x = [], px
        for _ in range(4):
            H = binding.newton_forward("diag_gru", x, diag, K=3, sync_status=False)[:, :, 0].contiguous()
            wait()
            z, _, _ = binding.layer_norm_forward(H, sync_status=False)
            wait()
            x = x + z.unsqueeze(2) * 0.1
            H2, _, ck = binding.gated_scan_forward(x, lam, DECAY, want_grad=True, sync_status=False)
            wait()
            dpx, dlam, _ = binding.gated_scan_backward(x, lam, ck, dH, DECAY, sync_status=False)
            wait()
            x = dpx.contiguous()
            out += [H, z, H2, dpx, dlam]
        torch.cuda.synchronize()
        return out

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, run(lambda: None)))
