"""The example's two layers together: prompt, single tokens and a training step agree with each other and with torch."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,steps,page", [((150, 77, 300), 5, 64), ((1, 64), 3, 16)])
def test_hybrid_layers(lens, steps, page):
    """Decoding differs from the prompt form by roundings to bf16 only: of the absorbed query (2^-9), of the latent output
    and of the weights, against the expanded key, value and output; the gradients by those of their inputs."""
    from examples.hybrid_layers import main
    worst = main(lens=lens, steps=steps, page=page, say=lambda *_: None)
    assert set(worst) == {"gradient of down", "gradient of q", "gradient of norm", "decoded tokens"}
    for k, v in worst.items():
        assert v <= 1e-2, (k, v)
