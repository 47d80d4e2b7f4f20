"""A selective state space layer, trained and then run token by token.

    python examples/state_space_layer.py [steps]

The layer is the usual one: normalisation, an input projection that makes the
layer's input and its gate, the short causal convolution, projections that make
each step's size (Delta) and its B and C, the selective scan, an output
projection, and the sum with what came in.  The projections are torch products;
everything else, forward and backward, is ``StateSpaceLayer``.

The task is to remember: the target of every step is the input of a few steps
before.  After training, the sequence's second half is run one token at a time
on the carried states, and gives what the whole sequence gave.
"""
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import onnx_lstm_gru_gb300 as rk  # noqa: E402


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layer, problem, x, scale, bias):
        out = layer.norm(problem, x, Scale=scale, B=bias)
        ctx.layer, ctx.problem = layer, problem
        ctx.save_for_backward(x, scale, out["Mean"], out["InvStdDev"])
        return out["Y"]

    @staticmethod
    def backward(ctx, dy):
        x, scale, mean, inv = ctx.saved_tensors
        g = ctx.layer.norm_grad(ctx.problem, x, Scale=scale, Mean=mean, InvStdDev=inv, dY=dy.contiguous())
        return None, None, g["dX"], g["dScale"].to(scale.dtype), g["dB"].to(scale.dtype)


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layer, problem, x, w, b):
        ctx.layer, ctx.problem = layer, problem
        ctx.save_for_backward(x, w, b)
        return layer.conv(problem, x, W=w, B=b, want=("Y",))["Y"]

    @staticmethod
    def backward(ctx, dy):
        x, w, b = ctx.saved_tensors
        g = ctx.layer.conv_grad(ctx.problem, x, W=w, B=b, dY=dy.contiguous())
        return None, None, g["dX"], g["dW"].to(w.dtype), g["dB"].to(b.dtype)


class Scan(torch.autograd.Function):
    NAMES = ("X", "Delta", "B", "C", "Z", "A", "D", "delta_bias")

    @staticmethod
    def forward(ctx, layer, problem, *tensors):
        ctx.layer, ctx.problem = layer, problem
        ctx.save_for_backward(*tensors)
        return layer.scan(problem, **dict(zip(Scan.NAMES, tensors)), want=("Y",))["Y"]

    @staticmethod
    def backward(ctx, dy):
        want = tuple("d_delta_bias" if n == "delta_bias" else "d" + n for n in Scan.NAMES)
        g = ctx.layer.scan_grad(ctx.problem, **dict(zip(Scan.NAMES, ctx.saved_tensors)), dY=dy.contiguous(), want=want)
        return (None, None, *(g[n] for n in want))


class Layer(torch.nn.Module):
    def __init__(self, width, channels, states=16, taps=4, rank=8):
        super().__init__()
        self.width, self.channels, self.states, self.taps, self.rank = width, channels, states, taps, rank
        f32 = dict(device="cuda", dtype=torch.float32)

        def weight(out, inp):
            return torch.nn.Parameter(torch.randn(out, inp, **f32) / math.sqrt(inp))
        self.scale = torch.nn.Parameter(torch.ones(width, **f32))
        self.bias = torch.nn.Parameter(torch.zeros(width, **f32))
        self.proj_in, self.proj_out = weight(2 * channels, width), weight(width, channels)
        self.taps_w = torch.nn.Parameter(torch.randn(channels, taps, **f32) / math.sqrt(taps))
        self.taps_b = torch.nn.Parameter(torch.zeros(channels, **f32))
        self.proj_x, self.proj_dt = weight(rank + 2 * states, channels), weight(channels, rank)
        self.rates = torch.nn.Parameter(torch.log(torch.arange(1.0, states + 1, **f32)).repeat(channels, 1))
        self.skip = torch.nn.Parameter(torch.ones(channels, **f32))
        step = torch.exp(torch.rand(channels, **f32) * math.log(100.0) + math.log(1e-3))
        self.step_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.ops = rk.StateSpaceLayer()

    def mix(self, x):
        """What the scan takes of the convolution's output: Delta, B and C."""
        low, B, C = (x @ self.proj_x.t()).split((self.rank, self.states, self.states), dim=-1)
        return low @ self.proj_dt.t(), B, C

    def forward(self, x):
        """x [batch, seq, width]: a whole sequence, for training."""
        N, S, _ = x.shape
        y = Norm.apply(self.ops, rk.NormProblem(N * S, self.width), x.reshape(N * S, -1), self.scale, self.bias)
        u, z = (y @ self.proj_in.t()).view(N, S, -1).split(self.channels, dim=-1)
        u = Conv.apply(self.ops, rk.ConvProblem(S, N, self.channels, self.taps, layout=1), u, self.taps_w, self.taps_b)
        delta, B, C = self.mix(u)
        y = Scan.apply(self.ops, rk.ScanProblem(S, N, self.channels, self.states, layout=1), u, delta, B, C, z,
                       -torch.exp(self.rates), self.skip, self.step_bias)
        return x + y @ self.proj_out.t()

    @torch.no_grad()
    def step(self, x, state):
        """x [batch, seq, width], a prompt or a single token after what ``state`` has seen (None: nothing)."""
        N, S, _ = x.shape
        conv, scan = state if state is not None else (None, None)
        y = self.ops.norm(rk.NormProblem(N * S, self.width), x.reshape(N * S, -1), Scale=self.scale, B=self.bias,
                          want=("Y",))["Y"]
        u, z = (y @ self.proj_in.t()).view(N, S, -1).split(self.channels, dim=-1)
        # given a state the same tensors are updated in place
        c = self.ops.conv(rk.ConvProblem(S, N, self.channels, self.taps, layout=1), u, W=self.taps_w, B=self.taps_b,
                          initial_state=conv, **({} if conv is None else dict(final_state=conv)))
        delta, B, C = self.mix(c["Y"])
        s = self.ops.scan(rk.ScanProblem(S, N, self.channels, self.states, layout=1), c["Y"], Delta=delta, B=B, C=C,
                          Z=z, A=-torch.exp(self.rates), D=self.skip, delta_bias=self.step_bias, initial_state=scan,
                          **({} if scan is None else dict(final_state=scan)))
        return x + s["Y"] @ self.proj_out.t(), (c["final_state"], s["final_state"])


def main(steps=200, batch=16, seq=48, width=32, channels=64, delay=3, seed=0):
    """Trains, prints, and returns (first loss, last loss, largest difference of the token-by-token run)."""
    torch.manual_seed(seed)
    layer, read = Layer(width, channels), torch.nn.Linear(width, width, device="cuda")
    opt = torch.optim.Adam([*layer.parameters(), *read.parameters()], lr=3e-3)
    losses = []
    for i in range(steps):
        x = torch.randn(batch, seq, width, device="cuda")
        loss = (read(layer(x))[:, delay:] - x[:, :-delay]).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if i % 50 == 0 or i == steps - 1:
            print(f"step {i}: loss {float(losses[-1]):.4f}")
    x = torch.randn(batch, seq, width, device="cuda")
    with torch.no_grad():
        whole = layer(x)
    y, state = layer.step(x[:, :seq // 2], None)
    parts = [y]
    for t in range(seq // 2, seq):
        y, state = layer.step(x[:, t:t + 1], state)
        parts.append(y)
    off = float((torch.cat(parts, 1) - whole).abs().max())
    print(f"prompt of {seq // 2} and {seq - seq // 2} single tokens: largest difference {off:.2e}")
    return float(losses[0]), float(losses[-1]), off


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
