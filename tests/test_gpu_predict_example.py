"""The token operators and the rasterizer together, as the example trains them."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_training_lowers_the_error_and_reaches_every_weight():
    import predict_gaussians as example
    model, losses = example.train(steps=60, say=lambda line: print(line, flush=True))
    for name, p in model.named_parameters():
        assert torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name
    assert losses[-1] < 0.7 * losses[0]


def test_scenes_of_a_packed_row_do_not_see_each_other():
    """Other patches in the second scene and in the padding change nothing of the first."""
    import predict_gaussians as example
    torch.manual_seed(1)
    model, data = example.Predictor().cuda(), example.make_data("cuda")
    draws = example.Draws(seed=3)
    hi = data["goals"][0][1]

    def first(patches):
        draws.offset = 0
        with torch.no_grad():
            out = model(patches, data["rays"], data["spans"], data["positions"], draws)
        return [t[:hi].clone() for t in out]

    a = first(data["patches"])
    other = data["patches"].clone()
    other[hi:] = other[hi:].flip(0) + 3.0
    for x, y in zip(a, first(other)):
        assert torch.equal(x, y)
