"""What is measured of the state space layer's operators: their cases, inputs, plain forms and definitions.

Six operators, each over ranges of sizes and types: layer normalisation and its gradient, the short causal
convolution and its gradient, the selective scan and its gradient.  Convolution and scan run as prompts (many
steps), as single tokens (one step with the state carried over) and backward.

Where ``own`` is true ``run`` calls the library's operators through ``StateSpaceLayer``; where it is false it
computes the same outputs from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F32 = torch.float32
EPSILON = 1e-5


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's normalisation: one row for each of 64 requests, latency counts
        dict(name="norm_token", op="norm", rows=64, cols=1024, dtype="bf16"),
        # the normalisation in front of the library's largest layer (512 steps of 64 rows of 1024)
        dict(name="norm_layer", op="norm", rows=32768, cols=1024, dtype="bf16"),
        # the same in a training step
        dict(name="norm_grad_layer", op="norm_grad", rows=32768, cols=1024, dtype="bf16"),
        # float32 training on odd sizes: rows that no vector load divides
        dict(name="norm_grad_odd", op="norm_grad", rows=1999, cols=777, dtype="f32"),
        # one decode step of 64 requests, twice 1024 channels, state carried over
        dict(name="conv_token", op="conv", seq=1, batch=64, channels=2048, width=4, dtype="bf16", layout=0,
             silu=True, ragged=False, state=True),
        # eight prompts of different lengths in one padded batch, batch-major, the input a slice of a wider row
        dict(name="conv_prompt", op="conv", seq=512, batch=8, channels=2048, width=4, dtype="f16", layout=1,
             silu=True, ragged=True, state=False),
        # a training batch of eight sequences of 512 steps
        dict(name="conv_grad", op="conv_grad", seq=512, batch=8, channels=2048, width=4, dtype="bf16", layout=1,
             silu=True, ragged=False, state=False),
        # one decode step of 64 requests: state read and written once
        dict(name="scan_token", op="scan", seq=1, batch=64, channels=2048, states=16, groups=1, dtype="bf16",
             layout=0, gate=True, ragged=False, state=True),
        # one long prompt alone: a single sequence has to fill the card
        dict(name="scan_prompt", op="scan", seq=4096, batch=1, channels=2048, states=16, groups=1, dtype="bf16",
             layout=0, gate=True, ragged=False, state=False),
        # float32 prompts of different lengths, odd sizes, two groups, states of an earlier prompt carried over
        dict(name="scan_ragged", op="scan", seq=777, batch=8, channels=1030, states=16, groups=2, dtype="f32",
             layout=1, gate=False, ragged=True, state=True),
        # a training batch of eight sequences of 512 steps
        dict(name="scan_grad", op="scan_grad", seq=512, batch=8, channels=2048, states=16, groups=1, dtype="bf16",
             layout=1, gate=True, ragged=False, state=False),
        # truncated back-propagation on odd sizes: ragged float16 sequences, three groups, the state's gradients too
        dict(name="scan_grad_odd", op="scan_grad", seq=201, batch=3, channels=519, states=24, groups=3, dtype="f16",
             layout=0, gate=False, ragged=True, state=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n - 1 if n == 3072 else n


def _even(rng, n):
    """Half of the sizes keep to multiples of 8, as a model's do; the others stay odd or even as they came."""
    return max(8, n // 8 * 8) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "conv", "conv_grad", "scan", "scan", "scan_grad", "scan_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm", "norm_grad"):
        cols = _even(rng, _spread(rng, 16, 4096))
        return dict(op=op, rows=_spread(rng, 1, max(1, min(32768, (1 << 25) // cols))), cols=cols, dtype=dtype)
    case = dict(op=op, dtype=dtype, layout=rng.randrange(2), ragged=rng.random() < 0.4, state=rng.random() < 0.5)
    channels = _even(rng, _spread(rng, 16, 2048))
    if op in ("conv", "conv_grad"):
        room = (1 << 23) // channels
        case.update(width=rng.choice([2, 3, 4, 4, 4, 5, 8]), silu=rng.random() < 0.8)
    else:
        states = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        groups = rng.choice([g for g in (1, 1, 1, 2, 4) if channels % g == 0])
        room = (1 << 27) // (channels * states)
        case.update(states=states, groups=groups, gate=rng.random() < 0.5)
    batch = _spread(rng, 1, max(1, min(64, room)))
    token = op in ("conv", "scan") and rng.random() < 0.3
    case.update(batch=batch, seq=1 if token else _spread(rng, 2, max(2, min(4096, room // batch))), channels=channels)
    if token:
        case.update(state=True, ragged=False)
    return case


def _tokens(case):
    """Tokens that hold work: lengths are uniform in 1..seq where the batch is ragged."""
    return case["batch"] * (case["seq"] + 1) / 2 if case["ragged"] else case["batch"] * case["seq"]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "norm":
        n, c = case["rows"], case["cols"]
        return {"bytes": 2 * n * c * e + 2 * c * e + 8 * n, "flops": 8 * n * c}
    if op == "norm_grad":
        n, c = case["rows"], case["cols"]
        return {"bytes": 3 * n * c * e + c * e + 8 * c + 8 * n, "flops": 14 * n * c}
    t, full, c = _tokens(case), case["batch"] * case["seq"], case["channels"]
    if op == "conv":
        w = case["width"]
        state = case["batch"] * (w - 1) * c * e
        return {"bytes": (t + full) * c * e + (w + 1) * c * e + state * (2 if case["state"] else 1),
                "flops": t * c * (2 * w + (5 if case["silu"] else 1))}
    if op == "conv_grad":
        w = case["width"]
        state = case["batch"] * (w - 1) * c * e
        return {"bytes": (2 * t + full) * c * e + (w + 1) * c * (e + 4) + (3 * state if case["state"] else 0),
                "flops": t * c * (6 * w + (12 if case["silu"] else 1))}
    n, g = case["states"], case["groups"]
    state = case["batch"] * c * n * 4
    gate = 1 if case["gate"] else 0
    if op == "scan":
        return {"bytes": (t * (2 + gate) + full) * c * e + 2 * t * g * n * e + c * (n + 2) * 4 + state * (2 if case["state"] else 1),
                "flops": t * c * (7 * n + 10 + 6 * gate)}
    return {"bytes": (t * (3 + gate) + full * (2 + gate)) * c * e + 2 * (t + full) * g * n * e + 2 * c * (n + 2) * 4
            + (3 * state if case["state"] else 0),
            "flops": t * c * (21 * n + 24 + 14 * gate)}


# ---- inputs -----------------------------------------------------------------------------------

_handle = []


def _layer():
    """The program's one handle: it keeps the scratch that the operators grow on demand."""
    if not _handle:
        import onnx_lstm_gru_gb300 as rk
        _handle.append(rk.StateSpaceLayer())
    return _handle[0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=F32)
        return x.mul_(scale).add_(mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=F32).mul_(hi - lo).add_(lo)

    s = {"case": case, "op": op}
    if op in ("norm", "norm_grad"):
        n, c = case["rows"], case["cols"]
        # a residual stream: every channel has its own offset and size
        X = (normal(n, c, dtype=F32) * uniform(c, lo=0.5, hi=1.5) + normal(c, scale=0.3, dtype=F32)).to(dt)
        t = dict(X=X, Scale=normal(c, scale=0.1, mean=1.0))
        if op == "norm":
            t["B"] = normal(c, scale=0.1)
        else:
            x = X.float()
            mean = x.mean(1)
            t.update(Mean=mean, InvStdDev=((x - mean[:, None]).square().mean(1) + EPSILON).rsqrt(),
                     dY=normal(n, c, scale=0.1))
        s["tensors"] = t
        if own:
            import onnx_lstm_gru_gb300 as rk
            s.update(layer=_layer(), problem=rk.NormProblem(rows=n, cols=c, dtype=case["dtype"], epsilon=EPSILON))
        return s

    S, N, C = case["seq"], case["batch"], case["channels"]
    rows = (S, N) if case["layout"] == 0 else (N, S)
    t = {}
    if case["ragged"]:
        t["sequence_lens"] = torch.randint(1, S + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    if op in ("conv", "conv_grad"):
        w = case["width"]
        # the input projection's rows hold the convolution's input and the gate side by side
        t["X"] = normal(*rows, 2 * C)[..., :C]
        t["W"] = uniform(C, w, lo=-1 / math.sqrt(w), hi=1 / math.sqrt(w)).to(dt)
        t["B"] = normal(C, scale=0.1)
        if case["state"]:
            t["initial_state"] = normal(N, w - 1, C)
        if op == "conv_grad":
            t["dY"] = normal(*rows, C, scale=0.1)
            if case["state"]:
                t["d_final_state"] = normal(N, w - 1, C, scale=0.1)
        s["tensors"] = t
        if own:
            import onnx_lstm_gru_gb300 as rk
            s.update(layer=_layer(), problem=rk.ConvProblem(
                seq=S, batch=N, channels=C, width=w, dtype=case["dtype"], layout=case["layout"],
                activation="silu" if case["silu"] else "none"))
        return s

    K, G = case["states"], case["groups"]
    # the convolution's output after its SiLU
    x = normal(*rows, C, dtype=F32)
    t["X"] = (x * torch.sigmoid(x)).to(dt)
    t["Delta"] = normal(*rows, C, scale=0.5)
    # step sizes from 0.001 to 0.1 before the input moves them, as the bias whose softplus they are
    step = torch.exp(uniform(C, lo=math.log(1e-3), hi=math.log(1e-1)))
    t["delta_bias"] = step + torch.log(-torch.expm1(-step))
    # decay rates -1 .. -K of each channel, somewhat apart
    t["A"] = -torch.arange(1, K + 1, device="cuda", dtype=F32) * uniform(C, K, lo=0.8, hi=1.2)
    bc = normal(*rows, 2 * G * K)
    t["B"], t["C"] = bc[..., :G * K], bc[..., G * K:]
    t["D"] = normal(C, scale=0.1, mean=1.0, dtype=F32)
    if case["gate"]:
        t["Z"] = normal(*rows, 2 * C)[..., C:]
    if case["state"]:
        t["initial_state"] = normal(N, C, K, scale=0.2, dtype=F32)
    if op == "scan_grad":
        t["dY"] = normal(*rows, C, scale=0.1)
        if case["state"]:
            t["d_final_state"] = normal(N, C, K, scale=0.1, dtype=F32)
    s["tensors"] = t
    if own:
        import onnx_lstm_gru_gb300 as rk
        s.update(layer=_layer(), problem=rk.ScanProblem(
            seq=S, batch=N, channels=C, state=K, groups=G, dtype=case["dtype"], layout=case["layout"], softplus=True))
    return s


def _names(case):
    """The outputs of a case, by the names that the library's operators give them."""
    op = case["op"]
    if op == "norm":
        return ("Y", "Mean", "InvStdDev")
    if op == "norm_grad":
        return ("dX", "dScale", "dB")
    if op in ("conv", "scan"):
        return ("Y", "final_state")
    if op == "conv_grad":
        names = ("dX", "dW", "dB")
    else:
        names = ("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias") + (("dZ",) if case["gate"] else ())
    return names + (("d_initial_state",) if case["state"] else ())


def run(s):
    case = s["case"]
    if own:
        return getattr(s["layer"], s["op"])(s["problem"], want=_names(case), **s["tensors"])
    return {"norm": _norm, "norm_grad": _norm_grad, "conv": _conv, "conv_grad": _conv_grad,
            "scan": _scan, "scan_grad": _scan_grad}[s["op"]](case, **s["tensors"])


# ---- plain forms: elementary torch operations in 32 bits, rounded once at the end ----------------

def _norm(case, X, Scale, B):
    x = X.float()
    mean = x.mean(1)
    d = x - mean[:, None]
    inv = (d.square().mean(1) + EPSILON).rsqrt()
    return {"Y": (d * inv[:, None] * Scale.float() + B.float()).to(X.dtype), "Mean": mean, "InvStdDev": inv}


def _norm_grad(case, X, Scale, Mean, InvStdDev, dY):
    x, dy = X.float(), dY.float()
    xhat = (x - Mean[:, None]) * InvStdDev[:, None]
    g = dy * Scale.float()
    dx = InvStdDev[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return {"dX": dx.to(X.dtype), "dScale": (dy * xhat).sum(0), "dB": dy.sum(0)}


def _steps_first(x, layout):
    return x if layout == 0 else x.transpose(0, 1)


def _rows(x, layout, dtype):
    """Back to the case's layout and type."""
    return _steps_first(x, layout).contiguous().to(dtype)


def _live(case, sequence_lens, device):
    """[S, N, 1] truth values: steps within each row's length."""
    S, N = case["seq"], case["batch"]
    if sequence_lens is None:
        return torch.ones(S, N, 1, dtype=torch.bool, device=device)
    return (torch.arange(S, device=device)[:, None] < sequence_lens[None, :])[..., None]


def _padded(case, X, initial_state):
    """[width - 1 + S, N, C]: the state's rows, then the input's."""
    x = _steps_first(X, case["layout"]).float()
    w = case["width"]
    before = x.new_zeros(w - 1, case["batch"], case["channels"]) if initial_state is None \
        else initial_state.float().transpose(0, 1)
    return torch.cat([before, x])


def _last_rows(case, sequence_lens, device):
    """[N, width - 1]: the rows of _padded that are the state after each sequence's end."""
    lens = torch.full((case["batch"],), case["seq"], device=device) if sequence_lens is None else sequence_lens.long()
    return lens[:, None] + torch.arange(case["width"] - 1, device=device)


def _conv(case, X, W, B, sequence_lens=None, initial_state=None):
    xp = _padded(case, X, initial_state)
    pre = (xp.unfold(0, case["width"], 1) * W.float()).sum(-1) + B.float()
    y = pre * torch.sigmoid(pre) if case["silu"] else pre
    y = torch.where(_live(case, sequence_lens, X.device), y, torch.zeros((), device=X.device))
    last = _last_rows(case, sequence_lens, X.device)
    final = xp[last, torch.arange(case["batch"], device=X.device)[:, None]]
    return {"Y": _rows(y, case["layout"], X.dtype), "final_state": final.to(X.dtype)}


def _conv_grad(case, X, W, B, dY, sequence_lens=None, initial_state=None, d_final_state=None):
    w, layout = case["width"], case["layout"]
    xp = _padded(case, X, initial_state)
    windows = xp.unfold(0, w, 1)
    dp = _steps_first(dY, layout).float()
    if case["silu"]:
        pre = (windows * W.float()).sum(-1) + B.float()
        sig = torch.sigmoid(pre)
        dp = dp * sig * (1 + pre * (1 - sig))
    dp = torch.where(_live(case, sequence_lens, X.device), dp, torch.zeros((), device=X.device))
    dW = (dp[..., None] * windows).sum((0, 1))
    side = dp.new_zeros(w - 1, case["batch"], case["channels"])
    dxp = (torch.cat([side, dp, side]).unfold(0, w, 1) * W.float().flip(1)).sum(-1)
    out = {"dW": dW, "dB": dp.sum((0, 1))}
    if d_final_state is not None:
        last, n = _last_rows(case, sequence_lens, X.device), torch.arange(case["batch"], device=X.device)[:, None]
        dxp[last, n] = dxp[last, n] + d_final_state.float()
    if case["state"]:
        out["d_initial_state"] = dxp[:w - 1].transpose(0, 1).contiguous().to(X.dtype)
    out["dX"] = _rows(dxp[w - 1:], layout, X.dtype)
    return out


def _recurrence(a, b):
    """h[t] = a[t] h[t-1] + b[t] along the first dimension, by doubling the span that each step covers."""
    k = 1
    while k < a.shape[0]:
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _scan_terms(case, X, Delta, A, B, C, delta_bias, sequence_lens):
    layout, per = case["layout"], case["channels"] // case["groups"]
    live = _live(case, sequence_lens, X.device)
    raw = _steps_first(Delta, layout).float() + delta_bias
    zero = torch.zeros((), device=X.device)
    dt = torch.where(live, torch.where(raw > 20, raw, torch.log1p(torch.exp(raw))), zero)
    u = _steps_first(X, layout).float()
    shape = (case["seq"], case["batch"], case["groups"], case["states"])
    b = _steps_first(B, layout).float().reshape(shape).repeat_interleave(per, 2)
    c = _steps_first(C, layout).float().reshape(shape).repeat_interleave(per, 2)
    a = torch.exp(dt[..., None] * A)
    return live, raw, dt, u, a, b, c


def _states(a, b, dt, u, initial_state):
    add = (dt * u)[..., None] * b
    if initial_state is not None:
        add[0] += a[0] * initial_state
    return _recurrence(a, add)


def _scan(case, X, Delta, A, B, C, D, delta_bias, Z=None, sequence_lens=None, initial_state=None):
    live, raw, dt, u, a, b, c = _scan_terms(case, X, Delta, A, B, C, delta_bias, sequence_lens)
    h = _states(a, b, dt, u, initial_state)
    y = (h * c).sum(-1) + D * u
    if Z is not None:
        z = _steps_first(Z, case["layout"]).float()
        y = y * z * torch.sigmoid(z)
    y = torch.where(live, y, torch.zeros((), device=X.device))
    return {"Y": _rows(y, case["layout"], X.dtype), "final_state": h[-1].clone()}


def _scan_grad(case, X, Delta, A, B, C, D, delta_bias, dY, Z=None, sequence_lens=None, initial_state=None,
               d_final_state=None):
    layout, groups, per = case["layout"], case["groups"], case["channels"] // case["groups"]
    live, raw, dt, u, a, b, c = _scan_terms(case, X, Delta, A, B, C, delta_bias, sequence_lens)
    zero = torch.zeros((), device=X.device)
    h = _states(a, b, dt, u, initial_state)
    dy = torch.where(live, _steps_first(dY, layout).float(), zero)
    out = {}
    if Z is not None:
        z = _steps_first(Z, layout).float()
        sig = torch.sigmoid(z)
        y = (h * c).sum(-1) + D * u
        out["dZ"] = _rows(dy * y * sig * (1 + z * (1 - sig)), layout, X.dtype)
        dy = dy * z * sig
    # the state's gradient runs from the last step to the first
    back = dy[..., None] * c
    if d_final_state is not None:
        back[-1] += d_final_state
    g = _recurrence(torch.cat([a[1:], a[:1]]).flip(0), back.flip(0)).flip(0)
    before = torch.cat([(torch.zeros_like(h[0]) if initial_state is None else initial_state)[None], h[:-1]])
    through = g * a * before                      # d loss / d (dt A), by state
    gb = (g * b).sum(-1)
    ddt = (through * A).sum(-1) + gb * u
    ddelta = torch.where(live, ddt * torch.sigmoid(raw), zero)
    out["dX"] = _rows(torch.where(live, gb * dt + D * dy, zero), layout, X.dtype)
    out["dDelta"] = _rows(ddelta, layout, X.dtype)
    out["dA"] = (through * dt[..., None]).sum((0, 1))
    grouped = (case["seq"], case["batch"], groups, per, case["states"])
    flat = (case["seq"], case["batch"], groups * case["states"])
    out["dB"] = _rows((g * (dt * u)[..., None]).reshape(grouped).sum(3).reshape(flat), layout, X.dtype)
    out["dC"] = _rows((h * dy[..., None]).reshape(grouped).sum(3).reshape(flat), layout, X.dtype)
    out["dD"] = (dy * u).sum((0, 1))
    out["d_delta_bias"] = ddelta.sum((0, 1))
    if case["state"]:
        out["d_initial_state"] = a[0] * g[0]
    return out


# ---- the definitions in 64 bits, step by step ----------------------------------------------------

def exact(case, seed):
    t = {k: v if v.dtype == torch.int32 else v.double() for k, v in prepare(case, seed)["tensors"].items()}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _norm_exact(case, op, t)
    lens = t["sequence_lens"].tolist() if "sequence_lens" in t else [case["seq"]] * case["batch"]
    rows = {k: t[k] if case["layout"] == 1 else t[k].permute(1, 0, 2) for k in ("X", "Delta", "B", "C", "Z", "dY")
            if k in t and t[k].dim() == 3}
    out = (_conv_exact if op.startswith("conv") else _scan_exact)(case, op, t, rows, lens)
    for k in ("Y", "dX", "dDelta", "dZ") + (("dB", "dC") if op == "scan_grad" else ()):
        if k in out and case["layout"] == 0:
            out[k] = out[k].permute(1, 0, 2).contiguous()
    return {k: out[k] for k in _names(case)}


def _norm_exact(case, op, t):
    n = case["cols"]
    if op == "norm":
        mean = t["X"].sum(1) / n
        var = (t["X"] ** 2).sum(1) / n - mean ** 2
        inv = 1 / torch.sqrt(var + EPSILON)
        return {"Y": (t["X"] - mean[:, None]) * inv[:, None] * t["Scale"] + t["B"], "Mean": mean, "InvStdDev": inv}
    inv = t["InvStdDev"][:, None]
    xhat = (t["X"] - t["Mean"][:, None]) * inv
    g = t["dY"] * t["Scale"]
    dx = inv / n * (n * g - g.sum(1, keepdim=True) - xhat * (g * xhat).sum(1, keepdim=True))
    return {"dX": dx, "dScale": torch.einsum("rc,rc->c", t["dY"], xhat), "dB": t["dY"].sum(0)}


def _conv_exact(case, op, t, rows, lens):
    """One sequence at a time, tap by tap."""
    w, N, S, C = case["width"], case["batch"], case["seq"], case["channels"]
    x, W, dev = rows["X"], t["W"], t["W"].device
    Y = torch.zeros(N, S, C, dtype=torch.float64, device=dev)
    final = torch.zeros(N, w - 1, C, dtype=torch.float64, device=dev)
    dX, dI, dW, dB = torch.zeros_like(Y), torch.zeros_like(final), torch.zeros_like(W), torch.zeros_like(t["B"])
    for n in range(N):
        L = lens[n]
        before = t["initial_state"][n] if "initial_state" in t else torch.zeros_like(final[n])
        seq = torch.cat([before, x[n, :L]])
        pre = t["B"].expand(L, C).clone()
        for j in range(w):
            pre += W[:, j] * seq[j:j + L]
        sig = 1 / (1 + torch.exp(-pre))
        if op == "conv":
            Y[n, :L] = pre * sig if case["silu"] else pre
            final[n] = seq[L:]
            continue
        dp = rows["dY"][n, :L] * ((sig + pre * sig * (1 - sig)) if case["silu"] else 1.0)
        dseq = torch.zeros_like(seq)
        if "d_final_state" in t:
            dseq[L:] += t["d_final_state"][n]
        for j in range(w):
            dseq[j:j + L] += W[:, j] * dp
            dW[:, j] += (dp * seq[j:j + L]).sum(0)
        dB += dp.sum(0)
        dI[n], dX[n, :L] = dseq[:w - 1], dseq[w - 1:]
    return {"Y": Y, "final_state": final, "dX": dX, "dW": dW, "dB": dB, "d_initial_state": dI}


def _scan_exact(case, op, t, rows, lens):
    """All sequences one step at a time, forward and then backward."""
    N, S, C, G, K = case["batch"], case["seq"], case["channels"], case["groups"], case["states"]
    dev, f64 = t["A"].device, torch.float64
    group = torch.arange(C, device=dev) // (C // G)
    end = torch.tensor(lens, device=dev)
    A, D, bias = t["A"], t["D"], t["delta_bias"]
    Bs, Cs = rows["B"].reshape(N, S, G, K), rows["C"].reshape(N, S, G, K)

    def step(i):
        on = (i < end).to(f64)[:, None]
        dt = torch.logaddexp(rows["Delta"][:, i] + bias, torch.zeros((), dtype=f64, device=dev)) * on
        return on, dt, rows["X"][:, i], Bs[:, i][:, group], Cs[:, i][:, group], torch.exp(dt[..., None] * A)

    start = t["initial_state"] if "initial_state" in t else torch.zeros(N, C, K, dtype=f64, device=dev)
    h, kept = start, []
    Y = torch.zeros(N, S, C, dtype=f64, device=dev)
    for i in range(S):
        on, dt, u, b, c, a = step(i)
        kept.append(h if op == "scan_grad" else None)
        h = a * h + (dt * u)[..., None] * b
        Y[:, i] = (torch.einsum("nck,nck->nc", h, c) + D * u) * on
    if op == "scan":
        if "Z" in rows:
            Y = Y * rows["Z"] / (1 + torch.exp(-rows["Z"]))
        return {"Y": Y, "final_state": h}

    out = {k: torch.zeros(N, S, C, dtype=f64, device=dev) for k in ("dX", "dDelta", "dZ")}
    out.update({k: torch.zeros(N, S, G, K, dtype=f64, device=dev) for k in ("dB", "dC")})
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(D), torch.zeros_like(bias)
    g = t["d_final_state"] if "d_final_state" in t else torch.zeros_like(start)
    for i in reversed(range(S)):
        on, dt, u, b, c, a = step(i)
        dy = rows["dY"][:, i] * on
        if "Z" in rows:
            z = rows["Z"][:, i]
            sig = 1 / (1 + torch.exp(-z))
            out["dZ"][:, i] = dy * Y[:, i] * (sig + z * sig * (1 - sig))
            dy = dy * z * sig
        before = kept[i]
        now = a * before + (dt * u)[..., None] * b
        g = g + dy[..., None] * c
        out["dC"][:, i].index_add_(1, group, dy[..., None] * now)
        out["dB"][:, i].index_add_(1, group, g * (dt * u)[..., None])
        drive = torch.einsum("nck,nck->nc", g, b)
        out["dX"][:, i] = (drive * dt + D * dy) * on
        ddt = torch.einsum("nck,nck,ck->nc", g, a * before, A) + drive * u
        ddelta = ddt * on / (1 + torch.exp(-(rows["Delta"][:, i] + bias)))
        out["dDelta"][:, i] = ddelta
        dA += torch.einsum("nck,nc->ck", g * a * before, dt)
        dD += (dy * u).sum(0)
        dbias += ddelta.sum(0)
        g = g * a
    out["dB"], out["dC"] = out["dB"].reshape(N, S, G * K), out["dC"].reshape(N, S, G * K)
    out.update(dA=dA, dD=dD, d_delta_bias=dbias, d_initial_state=g)
    return out
