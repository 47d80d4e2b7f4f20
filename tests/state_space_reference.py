"""Plain 64-bit definitions of the state space operators, for the tests.

Everything is a float64 CPU tensor; rows are [batch, seq, ...].  The gradients
are the formulas written out; ``tests/test_state_space_host.py`` holds them
against differences of the forward definitions.
"""
import torch

F64 = torch.float64


def norm(X, Scale=None, B=None, epsilon=1e-5):
    mean = X.mean(1)
    inv = 1 / torch.sqrt(((X - mean[:, None]) ** 2).mean(1) + epsilon)
    y = (X - mean[:, None]) * inv[:, None]
    if Scale is not None:
        y = y * Scale
    return dict(Y=y if B is None else y + B, Mean=mean, InvStdDev=inv)


def norm_grad(X, dY, Mean, InvStdDev, Scale=None):
    xh = (X - Mean[:, None]) * InvStdDev[:, None]
    g = dY if Scale is None else dY * Scale
    dX = InvStdDev[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dict(dX=dX, dScale=(dY * xh).sum(0), dB=dY.sum(0))


def _len(lens, n, S):
    return S if lens is None else min(max(int(lens[n]), 0), S)


def _silu_slope(z):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def conv(X, W, B=None, lens=None, initial_state=None, silu=True, dY=None, d_final_state=None):
    """The outputs, and with dY the gradients."""
    N, S, C = X.shape
    w = W.shape[1]
    out = dict(Y=torch.zeros(N, S, C, dtype=F64), final_state=torch.zeros(N, w - 1, C, dtype=F64))
    if dY is not None:
        out.update(dX=torch.zeros_like(X), dW=torch.zeros_like(W), dB=torch.zeros(C, dtype=F64),
                   d_initial_state=torch.zeros(N, w - 1, C, dtype=F64))
    for n in range(N):
        L = _len(lens, n, S)
        before = torch.zeros(w - 1, C, dtype=F64) if initial_state is None else initial_state[n]
        x = torch.cat([before, X[n, :L]])
        dx = torch.zeros_like(x)
        if d_final_state is not None:
            dx[L:] += d_final_state[n]
        for s in range(L):
            pre = (x[s:s + w] * W.t()).sum(0)
            if B is not None:
                pre = pre + B
            out["Y"][n, s] = pre * torch.sigmoid(pre) if silu else pre
            if dY is not None:
                dp = dY[n, s] * _silu_slope(pre) if silu else dY[n, s]
                dx[s:s + w] += W.t() * dp
                out["dW"] += (x[s:s + w] * dp).t()
                out["dB"] += dp
        out["final_state"][n] = x[L:]
        if dY is not None:
            out["d_initial_state"][n], out["dX"][n, :L] = dx[:w - 1], dx[w - 1:]
    return out


def scan(X, Delta, A, B, C, D=None, Z=None, delta_bias=None, lens=None, initial_state=None, softplus=True,
         groups=1, dY=None, d_final_state=None):
    """The outputs, and with dY the gradients."""
    N, S, ch = X.shape
    K = A.shape[1]
    group = torch.arange(ch) // (ch // groups)
    out = dict(Y=torch.zeros(N, S, ch, dtype=F64), final_state=torch.zeros(N, ch, K, dtype=F64))
    if dY is not None:
        out.update({k: torch.zeros(N, S, ch, dtype=F64) for k in ("dX", "dDelta", "dZ")})
        out.update({k: torch.zeros(N, S, groups, K, dtype=F64) for k in ("dB", "dC")})
        out.update(dA=torch.zeros_like(A), dD=torch.zeros(ch, dtype=F64), d_delta_bias=torch.zeros(ch, dtype=F64),
                   d_initial_state=torch.zeros(N, ch, K, dtype=F64))
    for n in range(N):
        L = _len(lens, n, S)
        h = torch.zeros(ch, K, dtype=F64) if initial_state is None else initial_state[n].clone()
        kept = []
        for s in range(L):
            raw = Delta[n, s] if delta_bias is None else Delta[n, s] + delta_bias
            dt = torch.logaddexp(raw, torch.zeros((), dtype=F64)) if softplus else raw
            u, b, c = X[n, s], B[n, s].view(groups, K)[group], C[n, s].view(groups, K)[group]
            a = torch.exp(dt[:, None] * A)
            before, h = h, a * h + (dt * u)[:, None] * b
            y = (h * c).sum(1)
            if D is not None:
                y = y + D * u
            kept.append((raw, dt, u, b, c, a, before, h, y))
            out["Y"][n, s] = y if Z is None else y * Z[n, s] * torch.sigmoid(Z[n, s])
        out["final_state"][n] = h
        if dY is None:
            continue
        e = torch.zeros(ch, K, dtype=F64) if d_final_state is None else d_final_state[n].clone()
        for s in reversed(range(L)):
            raw, dt, u, b, c, a, before, h, y = kept[s]
            dy = dY[n, s]
            if Z is not None:
                out["dZ"][n, s] = dy * y * _silu_slope(Z[n, s])
                dy = dy * Z[n, s] * torch.sigmoid(Z[n, s])
            g = e + dy[:, None] * c
            out["dC"][n, s].index_add_(0, group, dy[:, None] * h)
            out["dB"][n, s].index_add_(0, group, (dt * u)[:, None] * g)
            gb = (g * b).sum(1)
            e = a * g
            x = e * before
            out["dX"][n, s] = gb * dt + (0 if D is None else D * dy)
            dd = ((x * A).sum(1) + gb * u) * (torch.sigmoid(raw) if softplus else 1.0)
            out["dDelta"][n, s] = dd
            out["dA"] += x * dt[:, None]
            out["dD"] += dy * u
            out["d_delta_bias"] += dd
        out["d_initial_state"][n] = e
    if dY is not None:
        out["dB"], out["dC"] = out["dB"].view(N, S, -1), out["dC"].view(N, S, -1)
    return out
