"""Work over the gated linear recurrence and layer normalisation, as programs that use this package do it.

Three operators in five uses.

The gated linear recurrence takes pre-activations px (B, T, 3, D) in the order (p_r, p_i, x), a decay parameter lam (D)
and a scale c:

    r = sig(p_r),  i = sig(p_i),  y = c softplus(lam) r,  a = e^-y,
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,          h_{-1} = h0,

with the state set to zero before the steps that a reset mask (B, T) marks (the first steps of packed sequences).

* "scan": the forward pass of a prompt, H and the last state;
* "scan_train": the forward pass and the gradients of px, lam and h0;
* "step": one token for each row of a batch, on the slots of a cache of states, with rows of padding (slot -1).

Layer normalisation takes x (M, P, N): M positions of P gates or heads of N values, each with its own scale and shift:

* "norm": the forward pass; "norm_train": the forward pass and the gradients of x, the scale and the shift.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DECAY = 8.0
EPS = 1e-5


# ---- the cases --------------------------------------------------------------


def listed():
    return [
        # one short prompt of a narrow layer: latency (the sizes of the small workload)
        {"name": "scan 1x1024x64 f32", "op": "scan", "B": 1, "T": 1024, "D": 64, "dtype": "f32", "packed": False},
        # a batch of packed prompts whose width is odd: rows that no 16-byte access fits
        {"name": "scan 3x2777x515 bf16 packed", "op": "scan", "B": 3, "T": 2777, "D": 515, "dtype": "bf16", "packed": True},
        # a full batch of prompts (the sizes of the batched workload)
        {"name": "scan 8x4096x2048 bf16", "op": "scan", "B": 8, "T": 4096, "D": 2048, "dtype": "bf16", "packed": False},
        # one training step's layer on a small batch of packed documents, ragged in every size
        {"name": "scan_train 2x1500x1000 bf16 packed", "op": "scan_train", "B": 2, "T": 1500, "D": 1000, "dtype": "bf16",
         "packed": True},
        # training in full precision (the sizes of the LSTM workload)
        {"name": "scan_train 4x32768x1024 f32", "op": "scan_train", "B": 4, "T": 32768, "D": 1024, "dtype": "f32",
         "packed": False},
        # training on one very long sequence (the sizes of the headline workload)
        {"name": "scan_train 1x131072x4096 bf16", "op": "scan_train", "B": 1, "T": 131072, "D": 4096, "dtype": "bf16",
         "packed": False},
        # decoding one sequence
        {"name": "step 1x4096 bf16", "op": "step", "rows": 1, "D": 4096, "slots": 8, "dtype": "bf16"},
        # decoding a batch of 250 of up to 1024 sequences
        {"name": "step 250x2048 f32", "op": "step", "rows": 250, "D": 2048, "slots": 1024, "dtype": "f32"},
        # the rows of one decoding step
        {"name": "norm 8x1x4096 bf16", "op": "norm", "M": 8, "P": 1, "N": 4096, "dtype": "bf16"},
        # the pre-activations of the batched workload, a scale and a shift for each gate
        {"name": "norm 32768x3x2048 bf16", "op": "norm", "M": 32768, "P": 3, "N": 2048, "dtype": "bf16"},
        # the outputs of 8 heads of 64 channels, each normalised by itself, in training
        {"name": "norm_train 32768x8x64 bf16", "op": "norm_train", "M": 32768, "P": 8, "N": 64, "dtype": "bf16"},
        # a layer's input in full precision, in training
        {"name": "norm_train 131072x1x1024 f32", "op": "norm_train", "M": 131072, "P": 1, "N": 1024, "dtype": "f32"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "step", "norm", "norm_train"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("scan", "scan_train"):
        most = 1 << 26  # elements B T D
        B, D = log_int(1, 32), log_int(17, 5000)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        T = log_int(1, 100000)
        while B * T * D > most:
            if B > 1:
                B = max(1, B // 2)
            else:
                T = max(1, T // 2)
        return {"op": op, "B": B, "T": T, "D": D, "dtype": dtype, "packed": rng.random() < 0.5}
    if op == "step":
        rows = log_int(1, 1500)
        return {"op": op, "rows": rows, "D": log_int(17, 8000), "slots": rows + log_int(1, 1000), "dtype": dtype}
    P = rng.choice([1, 1, 2, 3, 4, 8, 24])
    N = log_int(8, 12000 // P)
    M = log_int(1, 200000)
    while M * P * N > 1 << 27:
        M //= 2
    return {"op": op, "M": M, "P": P, "N": N, "dtype": dtype}


# ---- the inputs ---------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = {"op": case["op"]}
    if case["op"] in ("scan", "scan_train", "step"):
        # memories of 2 to 1000 steps at a full gate: softplus(lam) = -log(a) / c
        away = torch.exp(math.log(1e-3) + rand(case["D"]) * (math.log(0.5) - math.log(1e-3)))
        s["lam"] = torch.log(torch.expm1(-torch.log1p(-away) / DECAY))
    if case["op"] in ("scan", "scan_train"):
        B, T, D = case["B"], case["T"], case["D"]
        s["px"] = randn(B, T, 3, D, dtype=dt)
        s["h0"] = randn(B, D)
        s["reset"] = None
        if case["packed"]:  # sequences of 500 steps on average; a row of the batch may go on with an earlier state
            s["reset"] = (rand(B, T) < 1 / 500).to(torch.uint8)
        if case["op"] == "scan_train":
            s["dH"] = randn(B, T, D, dtype=dt)
    elif case["op"] == "step":
        n, D = case["rows"], case["D"]
        s["px"] = randn(n, 3, D, dtype=dt)
        s["state"] = randn(case["slots"], D)
        slots = torch.randperm(case["slots"], generator=g, device=dev)[:n]
        if n > 1:
            slots = torch.where(rand(n) < 0.05, -1, slots)
        s["slots"] = slots.to(torch.int32)
        s["y"] = torch.zeros((n, D), device=dev, dtype=dt)
    else:
        M, P, N = case["M"], case["P"], case["N"]
        s["x"] = torch.empty((M, P, N), device=dev, dtype=dt).normal_(0.5, 2.0, generator=g)
        s["weight"] = 1 + 0.2 * randn(P, N)
        s["bias"] = 0.2 * randn(P, N)
        if case["op"] == "norm_train":
            s["dy"] = randn(M, P, N, dtype=dt)
    return s


# ---- one pass -----------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return {"scan": _scan, "scan_train": _scan_train, "step": _step, "norm": _norm, "norm_train": _norm_train}[s["op"]](s)


def _run_own(s):
    from nonlinear_rnn_iteration_b200 import binding

    op = s["op"]
    if op == "scan":
        H, last, _ = binding.gated_scan_forward(s["px"], s["lam"], decay=DECAY, h0=s["h0"], reset=s["reset"],
                                                sync_status=False)
        return {"H": H, "last": last}
    if op == "scan_train":
        H, last, ck = binding.gated_scan_forward(s["px"], s["lam"], decay=DECAY, h0=s["h0"], reset=s["reset"],
                                                 want_grad=True, sync_status=False)
        dpx, dlam, dh0 = binding.gated_scan_backward(s["px"], s["lam"], ck, s["dH"], decay=DECAY, reset=s["reset"],
                                                     want_dh0=True, sync_status=False)
        return {"H": H, "last": last, "dpx": dpx, "dlam": dlam, "dh0": dh0}
    if op == "step":
        y = binding.gated_scan_step(s["px"], s["lam"], s["state"], decay=DECAY, slots=s["slots"], out=s["y"],
                                    sync_status=False)
        return {"y": y, "state": s["state"]}
    if op == "norm":
        y, _, _ = binding.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS, sync_status=False)
        return {"y": y}
    y, mean, rstd = binding.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS, want_stats=True,
                                               sync_status=False)
    dx, dw, db = binding.layer_norm_backward(s["x"], s["dy"], mean, rstd, s["weight"], sync_status=False)
    return {"y": y, "dx": dx, "dweight": dw, "dbias": db}


# ---- the plain forms ------------------------------------------------------------


def _gates(px, lam):
    """r, i, x, y = -log a, a and b = sqrt(1 - a^2), in 32 bits; gates are dimension -2 of px.  Most a are next to 1,
    where an error of e^-y that leans to one side adds up over the memory: 1 + expm1(-y) rounds to nearest."""
    p = px.float()
    r, i, x = torch.sigmoid(p.select(-2, 0)), torch.sigmoid(p.select(-2, 1)), p.select(-2, 2)
    y = DECAY * torch.log1p(torch.exp(lam)) * r
    return r, i, x, y, 1 + torch.expm1(-y), torch.sqrt(-torch.expm1(-2 * y))


def _linear(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1, h_{-1} = 0: after k doublings (a, u) spans the last 2^k steps."""
    k = 1
    while k < a.shape[1]:
        u = torch.cat([u[:, :k], u[:, k:] + a[:, k:] * u[:, :-k]], dim=1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], dim=1)
        k *= 2
    return u


def _decays(a, reset):
    return a if reset is None else a * (reset == 0).unsqueeze(-1)


def _scan(s):
    _, i, x, _, a, b = _gates(s["px"], s["lam"])
    a = _decays(a, s["reset"])
    u = b * i * x
    u[:, 0] += a[:, 0] * s["h0"]
    H = _linear(a, u)
    return {"H": H.to(s["px"].dtype), "last": H[:, -1].clone()}


def _scan_train(s):
    r, i, x, y, a, b = _gates(s["px"], s["lam"])
    keep = _decays(torch.ones_like(y), s["reset"])
    u = b * i * x
    u[:, 0] += a[:, 0] * keep[:, 0] * s["h0"]
    H = _linear(a * keep, u)
    del u
    before = torch.cat([s["h0"].unsqueeze(1), H[:, :-1]], dim=1) * keep
    # adj_t = dH_t + a_{t+1} adj_{t+1}: the same recurrence in reversed time
    later = torch.cat([(a * keep)[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    adj = _linear(later.flip(1), s["dH"].float().flip(1)).flip(1)
    dx = adj * b * i
    # dL/dy = -adj (a h_{t-1} - a^2 / b i x), and y / b where y = 0 has the limit 0
    dy = -adj * (a * before - torch.where(b > 0, a * a / b, 0 * b) * i * x)
    dpx = torch.stack([dy * y * (1 - r), dx * x * (1 - i), dx], dim=2)
    sp = torch.log1p(torch.exp(s["lam"]))
    dlam = (dy * y).sum(dim=(0, 1), dtype=torch.float64) * (torch.sigmoid(s["lam"]) / sp)
    dt = s["px"].dtype
    return {"H": H.to(dt), "last": H[:, -1].clone(), "dpx": dpx.to(dt), "dlam": dlam.float(),
            "dh0": a[:, 0] * keep[:, 0] * adj[:, 0]}


def _step(s):
    _, i, x, _, a, b = _gates(s["px"], s["lam"])
    rows = s["slots"].long()
    live = (rows >= 0).unsqueeze(-1)
    # a row of padding adds nothing to the slot that it is sent to
    at = rows.clamp(min=0)
    old = s["state"][at]
    h = a * old + b * i * x
    s["state"].index_add_(0, at, torch.where(live, h - old, 0 * h))
    s["y"].copy_(torch.where(live, h.to(s["y"].dtype), s["y"]))
    return {"y": s["y"], "state": s["state"]}


def _norm(s):
    return {"y": _normed(s)[0]}


def _normed(s):
    x = s["x"].float()
    mean = x.mean(dim=-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(dim=-1, keepdim=True) + EPS)
    xh = xc * rstd
    return (xh * s["weight"] + s["bias"]).to(s["x"].dtype), xh, rstd


def _norm_train(s):
    y, xh, rstd = _normed(s)
    dy = s["dy"].float()
    d = dy * s["weight"]
    dx = rstd * (d - d.mean(dim=-1, keepdim=True) - xh * (d * xh).mean(dim=-1, keepdim=True))
    return {"y": y, "dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(dim=0, dtype=torch.float64).float(),
            "dbias": dy.sum(dim=0, dtype=torch.float64).float()}


# ---- bytes and operations -------------------------------------------------------


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op in ("scan", "scan_train"):
        B, T, D = case["B"], case["T"], case["D"]
        n = B * T * D
        masks = B * T if case["packed"] else 0
        if op == "scan":  # px and the mask in, H out; lam, h0 and the last state
            return {"bytes": 4 * n * e + masks + 4 * D + 8 * B * D, "flops": 20 * n}
        # and back: px, dH and the mask in, dpx out; lam and its gradient, dh0
        return {"bytes": 11 * n * e + 2 * masks + 12 * D + 12 * B * D, "flops": 70 * n}
    if op == "step":  # px, the state and the slots in, the state and y out
        n = case["rows"] * case["D"]
        return {"bytes": 4 * n * e + 8 * n + 4 * case["rows"] + 4 * case["D"], "flops": 25 * n}
    n, p = case["M"] * case["P"] * case["N"], case["P"] * case["N"]
    if op == "norm":
        return {"bytes": 2 * n * e + 8 * p, "flops": 8 * n}
    # x in and y out; x and dy in and dx out; the scale twice, the shift, both gradients
    return {"bytes": 5 * n * e + 20 * p, "flops": 24 * n}


# ---- the definition in 64 bits --------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    lam = s["lam"].double()
    k = DECAY * torch.nn.functional.softplus(lam)
    pr, pi, x = (t.double() for t in s["px"].unbind(-2))
    r, i = 1 / (1 + torch.exp(-pr)), 1 / (1 + torch.exp(-pi))
    del pr, pi
    a = torch.exp(-k * r)
    b = torch.sqrt((1 - a) * (1 + a))
    if case["op"] == "step":
        y, state = s["y"].double(), s["state"].double()
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                state[slot] = a[row] * state[slot] + b[row] * i[row] * x[row]
                y[row] = state[slot]
        return {"y": y, "state": state}
    B, T, D = case["B"], case["T"], case["D"]
    stays = torch.ones((B, T, 1), dtype=torch.float64, device=x.device)
    if s["reset"] is not None:
        stays = (1 - s["reset"].double()).unsqueeze(-1)
    a *= stays  # d/dy of a stays 0 where the state is set to zero
    H = b * i
    H *= x
    h = s["h0"].double()
    for at, hh in zip(a.unbind(1), H.unbind(1)):
        h = hh.addcmul_(at, h)
    if case["op"] == "scan":
        return {"H": H, "last": h.clone()}
    adj = s["dH"].double()
    later = None
    for t in range(T - 1, -1, -1):
        now = adj[:, t]
        if later is not None:
            now.addcmul_(a[:, t + 1], later)
        later = now
    dx = adj * b * i
    dpi = dx * x * (1 - i)
    # b'(y) = e^{-2y} / b; the decay of a reset step still scales its input
    dy = adj * torch.exp(-2 * k * r) / b * i * x
    dy[:, 0] -= adj[:, 0] * a[:, 0] * s["h0"].double()
    dy[:, 1:] -= adj[:, 1:] * a[:, 1:] * H[:, :-1]
    dlam = (dy * r).sum(dim=(0, 1)) * DECAY / (1 + torch.exp(-lam))
    dpr = dy * k * r * (1 - r)
    return {"H": H, "last": h.clone(), "dpx": torch.stack([dpr, dpi, dx], dim=2), "dlam": dlam,
            "dh0": a[:, 0] * adj[:, 0]}


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    N = x.shape[-1]
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    xh = (x - mean) / sd
    y = xh * w + s["bias"].double()
    if "dy" not in s:
        return {"y": y}
    dy = s["dy"].double()
    dxh = dy * w
    dx = (N * dxh - dxh.sum(-1, keepdim=True) - xh * (dxh * xh).sum(-1, keepdim=True)) / (N * sd)
    return {"y": y, "dx": dx, "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
