"""The short causal convolution on the GPU against a plain 64-bit form: forward, one row per
sequence, gradients; odd channel counts, strides, widths, lengths of zero and one, tiles that
sequences start and end in, states, streams and graphs.

Tolerances, per element: one rounding to the output's type, plus roundings of 2^-24 counted
against the sum of absolute terms: the W products and the bias (W + 1 additions), the sigmoid
(exponent's argument, exponential, sum, reciprocal, two products: 8, with |f'| <= 1.1), so
2 (W + 9); gradients pass through e_t and another W products: 4 (W + 9). Sums over tokens add
a rounding per addition in sequence: at most 128 + 8 in a tile, T / (16 * 32) + 16 over tiles.
"""
import numpy as np
import pytest

import ops_oracle as oo

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def np64(t):
    return t.detach().to("cpu").double().numpy()


def make(lengths, C, W, kind, seed, init=True, wide=1, bias=True):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[kind]
    T, N = sum(lengths), len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=r(T, wide * C).to(dt).cuda()[:, (wide - 1) * C:], weight=(r(C, W) / W ** 0.5).cuda(),
             bias=(0.3 * r(C)).cuda() if bias else None,
             cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda(),
             initial_state=r(N, W - 1, C).to(dt).cuda() if init else None)
    g = dict(dy=r(T, wide * C).to(dt).cuda()[:, :C], d_final_state=r(N, W - 1, C).cuda())
    return d, g


def oracle(d, lengths, act, g=None):
    opt = lambda t: np64(t) if t is not None else None  # noqa: E731
    return oo.conv(np64(d["x"]), np64(d["weight"]), opt(d["bias"]), lengths, opt(d["initial_state"]), act,
                   np64(g["dy"]) if g else None, opt(g["d_final_state"]) if g else None)


# lengths, channels, width, type, initial state, row stride / channels, activation, bias
CASES = [
    ([1], 1, 4, "bf16", False, 1, "silu", True),
    ([7], 8, 4, "bf16", False, 1, "silu", True),
    ([300], 64, 4, "bf16", True, 2, "silu", True),
    ([0, 3, 0, 0, 40, 1, 2, 0], 130, 4, "fp16", True, 1, "silu", True),
    ([5, 64, 8, 8, 1], 136, 4, "bf16", False, 3, None, False),
    ([129, 0, 17], 33, 2, "fp32", True, 1, "silu", True),
    ([100, 31], 257, 3, "fp32", False, 2, "silu", False),
    ([2, 9, 1, 70], 40, 8, "fp16", True, 1, "silu", True),
    ([33, 2], 24, 5, "bf16", True, 1, None, True),
    ([6, 6, 200], 1030, 6, "bf16", True, 1, "silu", True),
    ([11, 0, 54], 16, 7, "fp32", True, 1, "silu", True),
    ([0, 0], 20, 4, "bf16", True, 1, "silu", True),
    ([1500, 700], 2056, 4, "bf16", True, 1, "silu", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{sum(c[0])}x{c[1]}w{c[2]}{c[3]}")
def test_forward(case):
    import chunked_gated_delta_kda_amd as kda

    lengths, C, W, kind, init, wide, act, bias = case
    d, _ = make(lengths, C, W, kind, 1, init, wide, bias)
    y, fin = kda.conv_fwd(**d, activation=act, check=True)
    ref = oracle(d, lengths, act is not None)
    oo.check("y", np64(y), ref["y"], ref["y_size"], kind, 2 * (W + 9))
    np.testing.assert_array_equal(np64(fin), ref["final"])


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{sum(c[0])}x{c[1]}w{c[2]}{c[3]}")
def test_gradients(case):
    import chunked_gated_delta_kda_amd as kda

    lengths, C, W, kind, init, wide, act, bias = case
    d, g = make(lengths, C, W, kind, 2, init, wide, bias)
    got = kda.conv_bwd(**d, **g, activation=act)
    ref = oracle(d, lengths, act is not None, g)
    steps = 4 * (W + 9)
    over = steps + 136 + sum(lengths) / 512 + 16
    oo.check("dx", np64(got["dx"]), ref["dx"], ref["dx_size"], kind, steps)
    oo.check("d_initial_state", np64(got["d_initial_state"]), ref["d_initial_state"], ref["d_initial_state_size"], "fp32", steps)
    oo.check("dweight", np64(got["dweight"]), ref["dweight"], ref["dweight_size"], "fp32", over)
    if bias:
        oo.check("dbias", np64(got["dbias"]), ref["dbias"], ref["dbias_size"], "fp32", over)
    else:
        assert got["dbias"] is None
    again = kda.conv_bwd(**d, **g, activation=act)
    assert all(torch.equal(got[k], again[k]) for k in got if got[k] is not None)


def test_gradient_against_differences():
    """Central differences of the forward in fp32: L = <dy, y> + <dfin, fin>. A step h = 1/16 leaves a
    third-derivative term h^2/6 |f'''| |w|^3 (|f'''| < 1/2 here, at most W rows of it) and roundings of L
    over h: 1e-2 of the largest gradient covers both."""
    import chunked_gated_delta_kda_amd as kda

    lengths, C, W = [5, 1, 9], 3, 4
    d, g = make(lengths, C, W, "fp32", 3)
    got = kda.conv_bwd(**d, **g)
    dyc, dfc = np64(g["dy"]), np64(g["d_final_state"])

    def loss(e):
        y, fin = kda.conv_fwd(**e)
        return float((np64(y) * dyc).sum() + (np64(fin) * dfc).sum())

    for name, key in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("initial_state", "d_initial_state")):
        flat = d[name].contiguous().reshape(-1)
        want = got[key].double().reshape(-1).cpu().numpy()
        for i in range(0, flat.numel(), 5):
            side = []
            for sign in (1, -1):
                moved = flat.clone()
                moved[i] += sign / 16
                side.append(loss({**d, name: moved.reshape(d[name].shape)}))
            assert abs((side[0] - side[1]) * 8 - want[i]) <= 1e-2 * max(1.0, np.abs(want).max()), (name, i)


@pytest.mark.parametrize("N,C,W,kind,act,wide", [(1, 1, 4, "bf16", "silu", 1), (5, 130, 4, "fp16", "silu", 2),
                                                 (3, 33, 2, "fp32", None, 1), (256, 1032, 4, "bf16", "silu", 1),
                                                 (4, 28, 8, "fp32", "silu", 3)])
def test_decode(N, C, W, kind, act, wide):
    import chunked_gated_delta_kda_amd as kda

    d, _ = make([1] * N, C, W, kind, 4, True, wide)
    ref = oracle(d, [1] * N, act is not None)
    state = d["initial_state"].clone()
    y, out = kda.conv_decode(d["x"], d["weight"], d["bias"], state, activation=act)
    assert out is state
    oo.check("y", np64(y), ref["y"], ref["y_size"], kind, 2 * (W + 9))
    np.testing.assert_array_equal(np64(state), ref["final"])
    other = torch.empty_like(state)
    y2, out = kda.conv_decode(d["x"], d["weight"], d["bias"], d["initial_state"], activation=act, state_out=other)
    assert out is other and torch.equal(y2, y) and torch.equal(other, state)
    y3, none = kda.conv_decode(d["x"], d["weight"], d["bias"], None, activation=act, state_out=None)
    assert none is None
    d["initial_state"] = None
    ref = oracle(d, [1] * N, act is not None)
    oo.check("y", np64(y3), ref["y"], ref["y_size"], kind, 2 * (W + 9))


def test_prompt_then_tokens_is_the_whole():
    """A sequence in pieces (prompt, prompt with its state, tokens) gives the same rows, bit for bit."""
    import chunked_gated_delta_kda_amd as kda

    d, _ = make([90], 72, 4, "bf16", 5, False)
    whole, fin = kda.conv_fwd(**d)
    p = (d["weight"], d["bias"])
    a, s = kda.conv_fwd(d["x"][:50], *p)
    b, s = kda.conv_fwd(d["x"][50:83], *p, None, s)
    parts = [a, b]
    for t in range(83, 90):
        y, s = kda.conv_decode(d["x"][t:t + 1], *p, s)
        parts.append(y)
    assert torch.equal(torch.cat(parts), whole) and torch.equal(s, fin)


def test_nothing_is_written_beside_the_outputs():
    import chunked_gated_delta_kda_amd as kda

    lengths, C = [9, 0, 30], 50
    d, _ = make(lengths, C, 4, "bf16", 6)
    guard = torch.full((41, C), 7.0, dtype=torch.bfloat16, device="cuda")
    fin = torch.full((5, 3, C), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.conv_fwd(**d, out=guard[1:40], final_state=fin[1:4])
    assert (guard[0] == 7).all() and (guard[40] == 7).all() and (fin[0] == 7).all() and (fin[4] == 7).all()


def test_malformed_offsets_raise_the_error_bit():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    d, _ = make([20, 30, 14], 24, 4, "bf16", 7)
    for bad in ([0, 40, 20, 64], [5, 20, 50, 64], [0, 20, 50, 60], [0, -9, 900, 64]):
        d["cu_seqlens"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        with pytest.raises(native.KdaDeviceError) as e:
            kda.conv_fwd(**d, check=True)
        assert e.value.bits == 2


def test_another_stream_and_a_graph():
    import chunked_gated_delta_kda_amd as kda

    d, g = make([70, 3, 200], 264, 4, "bf16", 8)
    ref, fin = kda.conv_fwd(**d)
    gref = kda.conv_bwd(**d, **g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, f = kda.conv_fwd(**d, stream=side)
    gr = kda.conv_bwd(**d, **g, stream=side)
    side.synchronize()
    assert torch.equal(y, ref) and torch.equal(f, fin) and all(torch.equal(gr[k], gref[k]) for k in gr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, f = kda.conv_fwd(**d)
        gr = kda.conv_bwd(**d, **g)
    for _ in range(3):
        for t in (y, f, *gr.values()):
            t.zero_()
        kda.conv_fwd(**d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(f, fin) and all(torch.equal(gr[k], gref[k]) for k in gr)
