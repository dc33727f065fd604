"""The example's state-space layers: prompts, single tokens, the 8-bit norm and a training step agree with each other and with
torch."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,steps,N", [((70, 33, 128), 6, 16), ((1, 64), 3, 32)])
def test_state_space_layers(lens, steps, N):
    """Every activation between two operators is rounded to bf16 once, at most 2^-8 and in norm about 2^-9.3 of it; a
    layer rounds six of them in a row forwards (norm, projection, convolution, vectors, scan, projection) and as many more
    backwards, and independent roundings add in squares: 4 x 2^-9.3 = 6e-3 for twelve in a row, twice that allowed, because
    step sizes pass an exponential.  An 8-bit value is off by at most 2^-4 of itself, 2^-4.8 = 3.6e-2 in norm."""
    from examples.state_space_layer import main
    worst = main(lens=lens, steps=steps, N=N, say=lambda *_: None)
    assert len(worst) == 13
    for k, v in worst.items():
        assert v <= (3.6e-2 if k == "8-bit norm" else 1.2e-2), (k, v)
