"""The short convolution's gradients on the GPU where rows hold infinities."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("C", [8, 7])
@pytest.mark.parametrize("row", [29, 30, 31, 32, 63, 127])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_an_infinite_row_makes_the_taps_gradients_infinite(C, row, kind):
    """Without an activation the gradient of a tap is the sum of dy x: with one row of x infinite and dy
    positive it is infinite, wherever the row lies in the tiles (32 rows here); dx and dbias do not depend on x."""
    import chunked_gated_delta_kda_amd as kda

    g = torch.Generator(device="cuda").manual_seed(row)
    x = torch.randn(200, C, generator=g, device="cuda").to(kind)
    dy = (0.5 + torch.rand(200, C, generator=g, device="cuda")).to(kind)
    w, b = torch.randn(C, 4, generator=g, device="cuda"), torch.zeros(C, device="cuda")
    ref = kda.conv_bwd(x, w, dy, b, activation=None)
    x[row, ::2] = float("inf")
    x[row, 1::2] = -float("inf")
    got = kda.conv_bwd(x, w, dy, b, activation=None)
    assert (got["dweight"] == x[row].float()[:, None]).all(), got["dweight"]
    assert torch.equal(got["dx"], ref["dx"]) and torch.equal(got["dbias"], ref["dbias"])
