"""GPU tests of the linear attention where its chunks can go wrong: chunks run
step by step beside others.  Inputs, checks and tolerances are those of
``test_linear_attention_gpu.py`` where a test does not state its own."""
import pytest

from test_linear_attention_gpu import DTYPES, Case, cut, layer  # noqa: F401  (layer: the fixture)

pytestmark = pytest.mark.gpu


# ---- chunks run step by step beside others ------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,S,H", [(80, 260, 2), (40, 260, 4), (1, 700, 2), (1, 700, 4)])
def test_attn_decays_that_are_none_in_the_second_head(layer, N, S, H, dtype):
    """Two heads share a block; whichever of them has the NaN, it is where the
    definition has it, in sequences whole and cut."""
    for at in (100, 128, 150, 191, 192):
        c = Case(S, N, H, 64, 64, dtype, ragged=False, layout=1)
        assert cut(c) == (N == 1)
        c.t["Decay"][:, at, 1::2] = float("nan")
        c.compare(layer.attn(c.p, **c.t), f"{at}")
