"""The gated linear recurrence and layer normalisation on the CPU: sizes,
refusals before any launch, and the 64-bit forms that the GPU tests compare with,
against finite differences and torch's autograd."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from nonlinear_rnn_iteration_b200 import binding

FAKE = 1 << 40  # never dereferenced: the checks fail first
F32, BF16, EINVAL = binding.F32, binding.BF16, binding.EINVAL


def test_sizes():
    ck = binding.pararnn_gated_scan_checkpoint_bytes
    assert ck(2, 100, 8, F32) > 0 and ck(2, 100, 8, F32) % 4 == 0
    assert ck(2, 200, 8, BF16) > ck(2, 100, 8, BF16) > 0
    assert ck(0, 100, 8, F32) == ck(2, 0, 8, F32) == 0
    assert ck(2, 100, 8, 7) == 0 and ck(-1, 100, 8, F32) == 0
    ws = binding.pararnn_gated_scan_workspace_bytes
    assert ws(2, 100, 8) >= 256 + 8 * 4 and ws(1, 1 << 31, 8) == 0 and ws(1, -1, 8) == 0
    nw = binding.pararnn_layer_norm_workspace_bytes
    assert nw(100, 3, 64) >= 256 + 2 * 3 * 64 * 4
    assert nw(0, 1, 1) >= 256
    assert nw(1, 0, 1) == nw(1, 1, 0) == nw(-1, 1, 1) == nw(1 << 31, 1, 1) == 0


SCAN = dict(B=1, T=8, D=8, dtype=F32, preacts=FAKE, lam=FAKE, decay=8.0, h0=None, reset=None, H_out=FAKE,
            h_last=None, checkpoints=None, workspace=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change", [dict(B=-1), dict(T=1 << 31), dict(dtype=2), dict(decay=0.0),
                                    dict(decay=float("nan")), dict(decay=float("inf")), dict(decay=-1.0),
                                    dict(preacts=None), dict(lam=None), dict(H_out=None), dict(preacts=FAKE + 2),
                                    dict(h0=FAKE + 1), dict(checkpoints=FAKE + 2), dict(preacts=FAKE)])
def test_scan_refuses(change):
    # the last one is not memory that a GPU reaches
    assert binding.pararnn_gated_scan_forward(**dict(SCAN, **change)) == EINVAL
    assert "pararnn_gated_scan_forward" in binding.pararnn_last_error()


@pytest.mark.parametrize("change", [dict(T=-1), dict(dtype=9), dict(decay=0.0), dict(checkpoints=None),
                                    dict(dL_dH=None), dict(dL_dpx=None), dict(dL_dH=FAKE + 1), dict(workspace=None)])
def test_scan_backward_refuses(change):
    args = dict(B=1, T=8, D=8, dtype=F32, preacts=FAKE, lam=FAKE, decay=8.0, reset=None, checkpoints=FAKE,
                dL_dH=FAKE, dL_dh_last=None, dL_dpx=FAKE, dL_dlam=None, dL_dh0=None, workspace=FAKE,
                ws_bytes=1 << 20, stream=None)
    assert binding.pararnn_gated_scan_backward(**dict(args, **change)) == EINVAL
    assert "pararnn_gated_scan_backward" in binding.pararnn_last_error()


@pytest.mark.parametrize("change", [dict(N=-1), dict(dtype=9), dict(decay=0.0), dict(n_slots=3), dict(n_slots=-1),
                                    dict(state=None), dict(y=None), dict(slots=FAKE + 2)])
def test_step_refuses(change):
    args = dict(N=4, D=8, dtype=F32, preacts=FAKE, lam=FAKE, decay=8.0, n_slots=4, slots=None, state=FAKE, y=FAKE,
                workspace=None, ws_bytes=0, stream=None)
    assert binding.pararnn_gated_scan_step(**dict(args, **change)) == EINVAL
    assert "pararnn_gated_scan_step" in binding.pararnn_last_error()


@pytest.mark.parametrize("change", [dict(M=-1), dict(P=0), dict(N=0), dict(dtype=9), dict(eps=-1.0),
                                    dict(eps=float("nan")), dict(x=None), dict(y=None), dict(mean=FAKE + 1)])
def test_norm_refuses(change):
    args = dict(M=4, P=1, N=8, dtype=F32, x=FAKE, weight=None, bias=None, eps=1e-5, y=FAKE, mean=None, rstd=None,
                workspace=None, ws_bytes=0, stream=None)
    assert binding.pararnn_layer_norm_forward(**dict(args, **change)) == EINVAL
    assert "pararnn_layer_norm_forward" in binding.pararnn_last_error()


@pytest.mark.parametrize("change", [dict(N=0), dict(dtype=9), dict(x=None), dict(mean=None), dict(dL_dx=None),
                                    dict(workspace=None)])
def test_norm_backward_refuses(change):
    args = dict(M=4, P=1, N=8, dtype=F32, x=FAKE, weight=None, mean=FAKE, rstd=FAKE, dL_dy=FAKE, dL_dx=FAKE,
                dL_dweight=None, dL_dbias=None, workspace=FAKE, ws_bytes=1 << 20, stream=None)
    assert binding.pararnn_layer_norm_backward(**dict(args, **change)) == EINVAL
    assert "pararnn_layer_norm_backward" in binding.pararnn_last_error()


def test_helpers_refuse():
    px, lam = torch.zeros(1, 4, 3, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="preacts"):
        binding.gated_scan_forward(torch.zeros(1, 4, 2, 8), lam)
    with pytest.raises(ValueError, match="lam"):
        binding.gated_scan_forward(px, torch.zeros(7))
    with pytest.raises(ValueError, match="reset"):
        binding.gated_scan_forward(px, lam, reset=torch.zeros(1, 3, dtype=torch.bool))
    with pytest.raises(ValueError, match="CUDA"):
        binding.gated_scan_forward(px, lam)
    with pytest.raises(TypeError):
        binding.gated_scan_forward(px.half(), lam)
    with pytest.raises(ValueError, match="dL_dH"):
        binding.gated_scan_backward(px, lam, torch.zeros(8), torch.zeros(1, 4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="slots"):
        binding.gated_scan_step(px[0], lam, torch.zeros(4, 8), slots=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="state"):
        binding.gated_scan_step(px[0], lam, torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="weight"):
        binding.layer_norm_forward(torch.zeros(4, 8), torch.zeros(7))
    with pytest.raises(ValueError, match="weight"):
        binding.layer_norm_forward(torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="last dimension"):
        binding.layer_norm_forward(torch.zeros(4, 0))


def _case(B, T, D, seed, packed=True):
    rng = np.random.default_rng(seed)
    px, lam = rng.standard_normal((B, T, 3, D)), rng.uniform(-6, 0, D)
    reset = (rng.random((B, T)) < 0.2).astype(np.uint8) if packed else None
    return rng, px, lam, rng.standard_normal((B, D)), reset


@pytest.mark.parametrize("packed", [False, True])
def test_reference_gradients_match_differences(packed):
    rng, px, lam, h0, reset = _case(2, 9, 3, 1, packed)
    dH, dl = rng.standard_normal((2, 9, 3)), rng.standard_normal((2, 3))

    def loss(px, lam, h0):
        H, last = ref.forward(px, lam, 8.0, h0, reset)
        return (H * dH).sum() + (last * dl).sum()

    dpx, dlam, dh0 = ref.backward(px, lam, 8.0, dH, h0, reset, dl)
    e = 1e-5
    for k in range(4):
        v, vl, vh = rng.standard_normal(px.shape), rng.standard_normal(3), rng.standard_normal(h0.shape)
        num = (loss(px + e * v, lam + e * vl, h0 + e * vh) - loss(px - e * v, lam - e * vl, h0 - e * vh)) / (2 * e)
        got = (dpx * v).sum() + (dlam * vl).sum() + (dh0 * vh).sum()
        assert abs(num - got) <= 1e-7 * max(1.0, abs(got))


def test_reference_recurrence_matches_torch():
    rng, px, lam, h0, reset = _case(2, 7, 4, 2)
    p = torch.from_numpy(px)
    r, i = torch.sigmoid(p[:, :, 0]), torch.sigmoid(p[:, :, 1])
    log_a = -8.0 * torch.nn.functional.softplus(torch.from_numpy(lam)) * r
    h = torch.from_numpy(h0)
    H, _ = ref.forward(px, lam, 8.0, h0, reset)
    for t in range(7):
        h = h * (1 - torch.from_numpy(reset[:, t, None]).double())
        h = torch.exp(log_a[:, t]) * h + torch.sqrt(1 - torch.exp(2 * log_a[:, t])) * i[:, t] * p[:, t, 2]
        assert np.abs(h.numpy() - H[:, t]).max() < 1e-12


def test_reference_norm_matches_torch():
    rng = np.random.default_rng(3)
    x, w, b, dy = (rng.standard_normal(s) for s in ((5, 1, 11), (1, 11), (1, 11), (5, 1, 11)))
    tx, tw, tb = (torch.from_numpy(a).requires_grad_() for a in (x[:, 0], w[0], b[0]))
    y = torch.nn.functional.layer_norm(tx, (11,), tw, tb, 1e-3)
    y.backward(torch.from_numpy(dy[:, 0]))
    dx, dw, db = ref.norm_backward(x, dy, w, 1e-3)
    for got, want in ((ref.norm(x, w, b, 1e-3)[0][:, 0], y), (dx[:, 0], tx.grad), (dw[0], tw.grad), (db[0], tb.grad)):
        assert np.abs(got - want.detach().numpy()).max() < 1e-12


def test_workspace_follows_the_launch():
    """a row of partial sums for each block that a channel group can have: no more than tiles of 64 steps, and one
    where the groups alone fill a device"""
    ws = binding.pararnn_gated_scan_workspace_bytes
    row = 65536 * 1024 * 4
    assert row <= ws(65536, 32, 1024) <= row + 4096
    assert ws(65536, 64, 1024) == ws(65536, 32, 1024) == ws(65536, 4096, 1024)
    assert ws(20, 128, 64) - ws(20, 64, 64) == 20 * 64 * 4
    sizes = [ws(20, T, 64) for T in (1, 64, 65, 129, 300, 520, 4000, 100000)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2] == 256 + 8 * 20 * 64 * 4
    assert ws(0, 10, 64) == ws(10, 0, 64) == ws(10, 10, 0) == 256
