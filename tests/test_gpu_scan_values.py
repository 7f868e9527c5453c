"""The selective scan on the GPU at values and sizes where its sums, joins and launches could go wrong."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_lanes_that_store_one_sum_agree():
    """dB and dC sum over 16 channels with four lanes to a sum, which all store it. With quarters of 2^24, 1,
    -2^24 and 1 the order decides: halves first, the same in every lane, give 2; two neighbouring
    quarters first, another pair of them in lanes 4 apart, give 1."""
    import chunked_gated_delta_kda_amd as kda

    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    dy = torch.zeros(1, 16, device="cuda")
    dy[0, ::4] = torch.tensor([2.0 ** 24, 1.0, -2.0 ** 24, 1.0])
    got = kda.ssm_bwd(one(1, 16), one(1, 16), torch.zeros(16, 16, device="cuda"), one(1, 1, 16), one(1, 1, 16), dy,
                      delta_softplus=False)
    assert (got["dB"] == 2).all() and (got["dC"] == 2).all()
