"""Row widths that the norms around a block cannot run are refused when they,
or a layer with them, are built."""
import pytest

from mixture_experts_ffn_histogram_gb300.layer import BlockNorm, DecodeLayer


@pytest.mark.parametrize("D", [0, -1, 8193, 16384])
@pytest.mark.parametrize("train", [True, False])
def test_the_norms_refuse(D, train):
    with pytest.raises(ValueError, match="unsupported sizes"):
        BlockNorm(4, D, train=train, device="cpu")


def test_a_layer_refuses():
    with pytest.raises(ValueError, match="unsupported sizes"):
        DecodeLayer(4, 8256, 8, 2, 64, 64, device="cpu")


@pytest.mark.parametrize("D", [1, 8192])
def test_the_borders_are_taken(D):
    assert BlockNorm(4, D, device="cpu").D == D
