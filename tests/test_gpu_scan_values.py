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


def test_gradients_of_as_many_groups_as_fill_a_launch():
    """2^18 groups of one channel with 129 states, one token: everything has a closed form. A rounding or two an
    operation: exponents up to 1 (8), products (4), sums over states (a rounding a term)."""
    import chunked_gated_delta_kda_amd as kda

    D, N = 1 << 18, 129
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = 0.1 + 0.9 * torch.rand(1, D, generator=g, device="cuda")
    u, dy, h0 = r(1, D), r(1, D), r(1, D, N)
    A, B, C = -torch.rand(D, N, generator=g, device="cuda"), r(1, D, N), r(1, D, N)
    got = kda.ssm_bwd(u, s, A, B, C, dy, initial_state=h0, delta_softplus=False)
    s, u, dy, h0, A, B, C = (t.double() for t in (s[0], u[0], dy[0], h0[0], A, B[0], C[0]))
    a = torch.exp(s[:, None] * A)
    x, dh = (s * u)[:, None], C * dy[:, None]
    h, hs = a * h0 + x * B, a * h0.abs() + (x * B).abs()
    into, size = (dh * B).sum(1), (dh * B).abs().sum(1)
    decay = dh * a * h0
    U = 2.0 ** -24
    for name, want, err in (("dB", dh * x, 4 * (dh * x).abs()), ("dC", h * dy[:, None], 14 * hs * dy[:, None].abs()),
                            ("dA", decay * s[:, None], 16 * (decay * s[:, None]).abs()),
                            ("d_initial_state", dh * a, 12 * (dh * a).abs()),
                            ("du", s * into, (N + 8) * s * size),
                            ("ddelta", (decay * A).sum(1) + u * into,
                             (N + 20) * ((decay * A).abs().sum(1) + u.abs() * size))):
        off = (got[name].double().reshape(want.shape) - want).abs() - U * err - 2.0 ** -126
        assert (off <= 0).all(), (name, off.max().item())


def test_tokens_of_rows_further_apart_than_the_scan_takes():
    """One token of two sequences whose rows lie 2^27 + 8 elements apart: as from rows side by side."""
    import chunked_gated_delta_kda_amd as kda

    g = torch.Generator(device="cuda").manual_seed(6)
    D, N, stride = 40, 16, (1 << 27) + 8
    buf = torch.empty(stride + 4096, dtype=torch.bfloat16, device="cuda")
    near, far = {}, {}
    for i, (name, shape) in enumerate(dict(u=(2, D), delta=(2, D), z=(2, D), B=(2, 1, N), C=(2, 1, N)).items()):
        near[name] = torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
        far[name] = buf.as_strided(shape, (stride,) + near[name].stride()[1:], 256 * i)
        far[name].copy_(near[name])
    A, state = -torch.rand(D, N, generator=g, device="cuda"), torch.randn(2, D, N, generator=g, device="cuda")
    want, got = state.clone(), state.clone()
    y, _ = kda.ssm_decode(A=A, state=want, **near)
    x, _ = kda.ssm_decode(A=A, state=got, **far)
    assert torch.equal(x, y) and torch.equal(got, want)


def test_malformed_offsets_without_tokens_raise_the_error_bit():
    import chunked_gated_delta_kda_amd as kda

    row, rows = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 1, 16, device="cuda")
    A, last = -torch.ones(8, 16, device="cuda"), torch.randn(2, 8, 16, device="cuda")
    for cu, bits in (([0, 0, 0], 0), ([0, 3, 0], 2), ([0, 0, 4], 2), ([1, 0, 0], 2)):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.device_errors()
        got = kda.ssm_bwd(row, row, A, rows, rows, row, cu_seqlens=cu, d_final_state=last)
        assert kda.device_errors() == bits, cu
        assert torch.equal(got["d_initial_state"], last) and not got["dA"].any()
        kda.ssm_fwd(row, row, A, rows, rows, cu_seqlens=cu)
        assert kda.device_errors() == bits, cu
        kda.conv_fwd(row, A[:, :4].contiguous(), cu_seqlens=cu)
        assert kda.device_errors() == bits, cu
        kda.conv_bwd(row, A[:, :4].contiguous(), row, cu_seqlens=cu)
        assert kda.device_errors() == bits, cu
