"""The convolution and the scan on the GPU over more than 2^31 elements (outputs and workspaces past 4 GiB): the
first and the last sequence of a packed batch against the same rows run by themselves."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

T, CH, EDGE = 66000, 32776, 50


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def big(g):
    return torch.randn(T, CH, generator=g, device="cuda", dtype=torch.bfloat16)


def edges(t):
    return (t[:EDGE], t[T - EDGE:])


def near(got, want):
    """Within one bf16 rounding of each (their fp32 sums may run in another order): 2^-7 of a value, and of the
    largest value of the rows 2^-12 where terms cancel (fp32 leaves 2^-24 of each of some hundred terms)."""
    got, want = got.float(), want.float()
    return bool(((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12 * want.abs().max()).all())


def test_convolution():
    import chunked_gated_delta_kda_amd as kda

    assert T * CH > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = big(g), big(g)
    w, b = torch.randn(CH, 4, generator=g, device="cuda") / 2, torch.randn(CH, generator=g, device="cuda") / 8
    cu = torch.tensor([0, EDGE, T - EDGE, T], dtype=torch.int32, device="cuda")
    y, fin = kda.conv_fwd(x, w, b, cu)
    dx = kda.conv_bwd(x, w, dy, b, cu)["dx"]
    for i, seq in enumerate((0, 2)):
        rows = edges(x)[i]
        want, last = kda.conv_fwd(rows, w, b)
        assert torch.equal(edges(y)[i], want) and torch.equal(fin[seq], last[0])
        assert torch.equal(edges(dx)[i], kda.conv_bwd(rows, w, edges(dy)[i], b)["dx"])


def test_scan():
    import chunked_gated_delta_kda_amd as kda

    g = torch.Generator(device="cuda").manual_seed(2)
    u, delta, dy, N = big(g), big(g), big(g), 16
    delta *= 0.5
    A = -torch.exp(torch.randn(CH, N, generator=g, device="cuda"))
    B, C = (torch.randn(T, 1, N, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    bias, D = torch.full((CH,), -3.0, device="cuda"), torch.ones(CH, device="cuda")
    cu = torch.tensor([0, EDGE, T - EDGE, T], dtype=torch.int32, device="cuda")
    y, fin = kda.ssm_fwd(u, delta, A, B, C, D, None, bias, cu)
    got = kda.ssm_bwd(u, delta, A, B, C, dy, D, None, bias, cu)
    for i, seq in enumerate((0, 2)):
        rows = [edges(t)[i] for t in (u, delta, B, C, dy)]
        want, last = kda.ssm_fwd(*rows[:2], A, *rows[2:4], D, None, bias)
        assert near(edges(y)[i], want) and near(fin[seq], last[0])
        ref = kda.ssm_bwd(*rows[:2], A, *rows[2:], D, None, bias)
        for name in ("du", "ddelta", "dB", "dC"):
            assert near(edges(got[name])[i], ref[name]), name
        assert near(got["d_initial_state"][seq], ref["d_initial_state"][0])
