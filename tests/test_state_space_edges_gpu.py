"""GPU tests of the state space operators where they can go wrong: nothing to
do, values that are not numbers, and sizes that take the forms which the shapes
of ``test_state_space_gpu.py`` leave out.  Inputs, checks and tolerances are
that file's where a test does not state its own."""
import pytest
import torch

import onnx_lstm_gru_gb300 as rk
from test_state_space_gpu import DTYPES, conv_inputs, layer  # noqa: F401  (layer: the fixture)

pytestmark = pytest.mark.gpu


# ---- nothing to do -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [1, 5, 20, 33, 64])
@pytest.mark.parametrize("width", [1, 4, 8])
def test_conv_no_steps_any_channels(layer, channels, width, dtype):
    """The state after no steps is the state before them, of channels that
    16-byte pieces divide or not; and nothing else is written."""
    p = rk.ConvProblem(0, 3, channels, width, dtype)
    t, _ = conv_inputs(p, channels + width)
    size = 3 * (width - 1) * channels
    room = torch.full((size + 64,), 7.0, dtype=rk.torch_dtype(dtype), device="cuda")
    final = room[32:32 + size].view(3, width - 1, channels)
    assert torch.equal(layer.conv(p, **t, final_state=final)["final_state"], t["initial_state"])
    assert bool((room[:32] == 7).all()) and bool((room[32 + size:] == 7).all())
    del t["initial_state"]
    assert not layer.conv(p, **t, final_state=final)["final_state"].any()
    state = final.fill_(3.0)
    assert bool((layer.conv(p, **t, initial_state=state, final_state=state)["final_state"] == 3).all())
