"""The selective state space scan on the GPU against a plain 64-bit form: prompts over packed
batches, one token per sequence; every state-size form, odd sizes and strides, the largest strides, groups, lengths of
zero and one, tiles that sequences start and end in, streams and graphs. Tolerances: one rounding
to the output's type, plus the fp32 roundings that ops_oracle.scan counts."""
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
    return t.detach().to("cpu").double().numpy() if t is not None else None


def make(lengths, D, N, kind, seed, groups=1, init=True, gate=True, wide=1, skip=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[kind]
    T, S = sum(lengths), len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    row = lambda n, k: r(T, wide * n).to(dt).cuda()[:, k % wide * n:(k % wide + 1) * n]  # noqa: E731
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    return dict(u=row(D, 0), delta=(r(T, D) * 0.5).to(dt).cuda() if bias else (r(T, D) - 2).to(dt).cuda(),
                A=-torch.exp(torch.log(torch.arange(1, N + 1).float()) + 0.1 * r(D, N)).cuda(),
                B=row(groups * N, 1).unflatten(1, (groups, N)), C=row(groups * N, 2).unflatten(1, (groups, N)),
                D=(1 + 0.1 * r(D)).cuda() if skip else None, z=row(D, 1) if gate else None,
                delta_bias=(step + torch.log(-torch.expm1(-step))).cuda() if bias else None,
                cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda(),
                initial_state=(0.3 * r(S, D, N)).cuda() if init else None)


def oracle(d, lengths, softplus=True):
    return oo.scan(*(np64(d[k]) for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")), lengths,
                   np64(d["initial_state"]), softplus)


def compare(y, fin, ref, kind):
    oo.check("y", np64(y), ref[0], ref[1], kind, 1)
    oo.check("final", np64(fin), ref[2], ref[3] + np.abs(ref[2]), "fp32", 1)


# lengths, channels, states, type, groups, initial state, gate, row stride, skip, bias
CASES = [
    ([1], 1, 1, "bf16", 1, False, False, 1, True, True),
    ([8], 64, 16, "bf16", 1, False, True, 1, True, True),
    ([7], 3, 16, "fp32", 1, True, True, 1, True, True),
    ([16, 17], 65, 16, "fp16", 1, True, True, 2, True, True),
    ([100], 70, 16, "fp32", 1, True, True, 1, True, True),
    ([0, 3, 0, 0, 40, 1, 2, 0], 130, 16, "bf16", 2, True, True, 2, True, True),
    ([33, 31, 0, 64, 1, 1, 1, 90], 24, 4, "fp32", 3, True, False, 1, False, True),
    ([29, 5], 40, 21, "fp32", 1, True, True, 3, True, True),
    ([16, 3, 50], 48, 32, "bf16", 3, False, True, 1, True, True),
    ([37], 18, 33, "fp16", 1, True, True, 1, True, True),
    ([64, 12], 20, 64, "fp32", 5, True, True, 2, True, True),
    ([19, 0, 41], 17, 100, "fp32", 1, True, False, 1, True, True),
    ([25, 25], 16, 128, "bf16", 2, True, True, 1, True, True),
    ([50, 2], 9, 200, "fp32", 1, True, True, 1, True, True),
    ([21], 5, 256, "bf16", 1, True, True, 1, True, True),
    ([60], 32, 16, "fp32", 1, True, True, 1, False, False),
    ([0, 0], 20, 16, "bf16", 1, True, True, 1, True, True),
    ([1200, 1, 700, 0, 99], 1030, 16, "bf16", 1, True, True, 2, True, True),
    ([700, 0, 200, 97], 70, 30, "fp32", 2, True, True, 1, True, True),
    ([96, 192, 1, 0, 95, 400], 33, 16, "bf16", 1, True, True, 1, True, True),
    ([3] * 40, 50, 16, "fp32", 1, True, True, 1, True, True),
    ([2] * 30 + [50], 36, 25, "bf16", 3, True, True, 2, True, True),
    ([90, 20], 24, 6, "fp32", 24, True, True, 1, True, True),
]


def ident(c):
    return f"{sum(c[0])}x{c[1]}n{c[2]}g{c[4]}{c[3]}"


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_prompt(case):
    import chunked_gated_delta_kda_amd as kda

    lengths, D, N, kind, groups, init, gate, wide, skip, bias = case
    d = make(lengths, D, N, kind, 1, groups, init, gate, wide, skip, bias)
    y, fin = kda.ssm_fwd(**d, check=True)
    compare(y, fin, oracle(d, lengths), kind)
    again, fagain = kda.ssm_fwd(**d)
    assert torch.equal(y, again) and torch.equal(fin, fagain)


def test_steps_without_softplus():
    import chunked_gated_delta_kda_amd as kda

    d = make([70, 9], 40, 16, "fp32", 2)
    d["delta"] = (d["delta"].abs() * 0.1).contiguous()
    d["delta_bias"] = d["delta_bias"].abs() * 0.01
    y, fin = kda.ssm_fwd(**d, delta_softplus=False)
    compare(y, fin, oracle(d, [70, 9], False), "fp32")


@pytest.mark.parametrize("rows,D,N,kind,groups,gate,wide", [(1, 1, 1, "bf16", 1, True, 1), (3, 65, 16, "bf16", 1, True, 2),
                                                            (5, 34, 21, "fp32", 2, False, 1), (2, 8, 200, "fp16", 1, True, 1),
                                                            (4, 12, 2, "fp32", 3, True, 3), (64, 520, 16, "bf16", 1, True, 1),
                                                            (2, 7, 100, "fp32", 1, True, 1), (2, 16, 40, "bf16", 4, True, 1)])
def test_token(rows, D, N, kind, groups, gate, wide):
    import chunked_gated_delta_kda_amd as kda

    d = make([1] * rows, D, N, kind, 3, groups, True, gate, wide)
    init = d["initial_state"]
    ref = oracle(d, [1] * rows)
    call = {k: v for k, v in d.items() if k not in ("cu_seqlens", "initial_state")}
    state = init.clone()
    y, out = kda.ssm_decode(**call, state=state)
    assert out is state
    compare(y, state, ref, kind)
    other = torch.empty_like(state)
    y2, _ = kda.ssm_decode(**call, state=init, state_out=other)
    assert torch.equal(y, y2) and torch.equal(other, state)
    y3, none = kda.ssm_decode(**call, state=init, state_out=None)
    assert none is None and torch.equal(y3, y)
    y4, fresh = kda.ssm_decode(**call)
    d["initial_state"] = None
    compare(y4, fresh, oracle(d, [1] * rows), kind)


def test_extreme_steps_and_values():
    """Steps from 0 to far past e^{sA} = 0, and inputs up to the type's largest: no NaN arises, states stay
    exact zeros where everything decays; what follows a sequence whose rows are not finite is untouched."""
    import chunked_gated_delta_kda_amd as kda

    lengths = [5, 13, 6]
    d = make(lengths, 20, 16, "fp32", 4, gate=False)
    ref, rfin = kda.ssm_fwd(**d)
    for name in ("u", "B", "C", "delta"):
        e = dict(d)
        e[name] = d[name].clone()
        e[name][5:18] = float("nan") if name != "B" else float("inf")
        y, fin = kda.ssm_fwd(**e)
        assert torch.equal(y[:5], ref[:5]) and torch.equal(y[18:], ref[18:]), name
        assert torch.equal(fin[0], rfin[0]) and torch.equal(fin[2], rfin[2]), name
        assert not torch.isfinite(y[5:18]).any(), name
    e = dict(d)
    e["delta"] = d["delta"].clone()
    e["delta"][::2], e["delta"][1::2] = -200.0, 300.0
    y, fin = kda.ssm_fwd(**e)
    compare(y, fin, oracle(e, lengths), "fp32")


def test_prompt_then_tokens_is_the_whole():
    """Pieces carry the state in fp32 and differ from the whole only in how tiles join."""
    import chunked_gated_delta_kda_amd as kda

    d = make([90], 72, 16, "fp32", 5, init=False)
    ref = oracle(d, [90])
    rows = lambda a, b: {k: v[a:b] if k in ("u", "delta", "B", "C", "z") else v  # noqa: E731
                         for k, v in d.items() if k not in ("cu_seqlens", "initial_state")}
    a, s = kda.ssm_fwd(**rows(0, 50))
    b, s = kda.ssm_fwd(**rows(50, 83), initial_state=s)
    parts = [a, b]
    for t in range(83, 90):
        y, s = kda.ssm_decode(**rows(t, t + 1), state=s)
        parts.append(y)
    compare(torch.cat(parts), s, ref, "fp32")


def test_nothing_is_written_beside_the_outputs():
    import chunked_gated_delta_kda_amd as kda

    lengths, D, N = [9, 0, 30], 50, 50      # over 32 states: tiles joined in the workspace
    d = make(lengths, D, N, "bf16", 6)
    out = torch.full((41, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fin = torch.full((5, D, N), 7.0, device="cuda")
    need = kda.native.load_library().kda_ssm_workspace_bytes(3, 39, D, N, 1)
    assert need > 0
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    kda.ssm_fwd(**d, out=out[1:40], final_state=fin[1:4], workspace=ws[256:256 + need])
    for t in (out[0], out[40], fin[0], fin[4], ws[:256], ws[256 + need:]):
        assert (t == 7).all()


def test_malformed_offsets_raise_the_error_bit():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    for T in (12, 64):     # one tile, several
        d = make([T // 2, T // 4, T - T // 2 - T // 4], 24, 16, "bf16", 7)
        for bad in ([0, T - 1, 3, T], [5, 6, 8, T], [0, 4, 6, T - 1], [0, -9, 900, T]):
            d["cu_seqlens"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
            with pytest.raises(native.KdaDeviceError) as e:
                kda.ssm_fwd(**d, check=True)
            assert e.value.bits == 2


def test_another_stream_and_a_graph():
    import chunked_gated_delta_kda_amd as kda

    d = make([70, 3, 200], 264, 16, "bf16", 8)
    ref, fin = kda.ssm_fwd(**d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, f = kda.ssm_fwd(**d, stream=side)
    side.synchronize()
    assert torch.equal(y, ref) and torch.equal(f, fin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, f = kda.ssm_fwd(**d)
    for _ in range(3):
        y.zero_(), f.zero_()
        kda.ssm_fwd(**make([50, 9], 100, 16, "bf16", 9))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(f, fin)


def grads_of(d, lengths, seed, kind, wide=1):
    g = torch.Generator().manual_seed(seed)
    T, D = d["u"].shape
    return dict(dy=torch.randn(T, wide * D, generator=g).to(TYPES[kind]).cuda()[:, :D],
                d_final_state=(0.2 * torch.randn(len(lengths), D, d["A"].shape[1], generator=g)).cuda())


def compare_grads(got, d, g, lengths, kind, softplus=True):
    ref, err = oo.scan_grads(*(np64(d[k]) for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")), lengths,
                             np64(d["initial_state"]), softplus, np64(g["dy"]), np64(g["d_final_state"]))
    for name in ("du", "ddelta", "dz", "dA", "dB", "dC", "dD", "ddelta_bias", "d_initial_state"):
        of = dict(dz="z", dD="D", ddelta_bias="delta_bias").get(name)
        if of and d[of] is None:
            assert got[name] is None
            continue
        t = kind if name in ("du", "ddelta", "dz", "dB", "dC") else "fp32"
        oo.check(name, np64(got[name]), ref[name], err[name] + 2 * np.abs(ref[name]), t, 1)


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_gradients(case):
    import chunked_gated_delta_kda_amd as kda

    lengths, D, N, kind, groups, init, gate, wide, skip, bias = case
    d = make(lengths, D, N, kind, 11, groups, init, gate, wide, skip, bias)
    g = grads_of(d, lengths, 12, kind, wide)
    got = kda.ssm_bwd(**d, **g)
    compare_grads(got, d, g, lengths, kind)
    again = kda.ssm_bwd(**d, **g)
    assert all(torch.equal(got[k], again[k]) for k in got if got[k] is not None)


def test_gradients_without_softplus_or_final_gradient():
    import chunked_gated_delta_kda_amd as kda

    lengths = [70, 9]
    d = make(lengths, 40, 16, "fp32", 13)
    d["delta"] = (d["delta"].abs() * 0.1).contiguous()
    d["delta_bias"] = d["delta_bias"].abs() * 0.01
    g = grads_of(d, lengths, 14, "fp32")
    g["d_final_state"] = None
    got = kda.ssm_bwd(**d, **g, delta_softplus=False, need_d_initial_state=False)
    assert got["d_initial_state"] is None
    got["d_initial_state"] = kda.ssm_bwd(**d, **g, delta_softplus=False)["d_initial_state"]
    compare_grads(got, d, g, lengths, "fp32", False)


def test_gradients_against_differences():
    """Central differences of the forward in fp32 with a step of 1/32: the third derivative's h^2/6 and the
    roundings of the loss (values of a few, over h) stay within 2e-2 of each input's largest gradient."""
    import chunked_gated_delta_kda_amd as kda

    lengths = [5, 1, 19]
    d = make(lengths, 3, 5, "fp32", 15)
    g = grads_of(d, lengths, 16, "fp32")
    got = kda.ssm_bwd(**d, **g)
    dyc, dfc = np64(g["dy"]), np64(g["d_final_state"])

    def loss(e):
        y, fin = kda.ssm_fwd(**e)
        return float((np64(y) * dyc).sum() + (np64(fin) * dfc).sum())

    for name, key in (("u", "du"), ("delta", "ddelta"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                      ("delta_bias", "ddelta_bias"), ("initial_state", "d_initial_state")):
        flat = d[name].contiguous().reshape(-1)
        want = got[key].double().reshape(-1).cpu().numpy()
        for i in range(0, flat.numel(), 1 + flat.numel() // 12):
            side = []
            for sign in (1, -1):
                moved = flat.clone()
                moved[i] += sign / 32
                side.append(loss({**d, name: moved.reshape(d[name].shape)}))
            assert abs((side[0] - side[1]) * 16 - want[i]) <= 2e-2 * max(1.0, np.abs(want).max()), (name, i)


def test_gradients_stay_in_their_sequences():
    import chunked_gated_delta_kda_amd as kda

    lengths = [21, 13, 30]
    d = make(lengths, 20, 16, "fp32", 17)
    g = grads_of(d, lengths, 18, "fp32")
    ref = kda.ssm_bwd(**d, **g)
    for name in ("u", "B", "C", "delta", "z", "dy"):
        e, f = dict(d), dict(g)
        src = f if name == "dy" else e
        src[name] = src[name].clone()
        src[name][21:34] = float("nan")
        got = kda.ssm_bwd(**e, **f)
        for k in ("du", "ddelta", "dB", "dC", "dz"):
            assert torch.equal(got[k][:21], ref[k][:21]) and torch.equal(got[k][34:], ref[k][34:]), (name, k)
        assert torch.equal(got["d_initial_state"][::2], ref["d_initial_state"][::2]), name


def test_gradients_on_a_stream_in_a_graph_and_within_their_buffers():
    import chunked_gated_delta_kda_amd as kda

    lengths = [70, 0, 3, 200]
    d = make(lengths, 100, 16, "bf16", 19)
    g = grads_of(d, lengths, 20, "bf16")
    need = kda.native.load_library().kda_ssm_bwd_workspace_bytes(273, 100, 16, 1)
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    ref = kda.ssm_bwd(**d, **g, workspace=ws[256:256 + need])
    assert (ws[:256] == 7).all() and (ws[256 + need:] == 7).all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kda.ssm_bwd(**d, **g, stream=side)
    side.synchronize()
    assert all(torch.equal(got[k], ref[k]) for k in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.ssm_bwd(**d, **g)
    for _ in range(3):
        for t in got.values():
            t.zero_()
        e = make([50, 9], 64, 16, "bf16", 9)
        kda.ssm_bwd(**e, **grads_of(e, [50, 9], 3, "bf16"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], ref[k]) for k in ref)


def test_gradients_of_malformed_offsets_stay_in_bounds():
    import chunked_gated_delta_kda_amd as kda

    for T in (12, 64):
        d = make([T // 2, T // 4, T - T // 2 - T // 4], 24, 16, "bf16", 21)
        g = grads_of(d, [1, 1, 1], 22, "bf16")
        for bad in ([0, T - 1, 3, T], [5, 6, 8, T], [0, 4, 6, T - 1], [0, -9, 900, T]):
            d["cu_seqlens"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
            kda.device_errors()
            kda.ssm_bwd(**d, **g)
            assert kda.device_errors() == 2


@pytest.mark.parametrize("N", [5, 16, 40], ids="states{}".format)
def test_the_largest_strides(N):
    """Rows 2^27 elements apart (20 of fp32 are 10 GiB): the same results as from rows one after another, by
    blocks (up to 32 states) and by waves, forward, one token and backward."""
    T, D, stride = 20, 24, 1 << 27
    d = make([13, 7], D, N, "fp32", 77)
    dy = torch.randn(T, D, generator=torch.Generator().manual_seed(78)).cuda()
    near = dict(d, dy=dy)
    for k in ("B", "C"):
        near[k] = near[k].contiguous()
    buf = torch.empty(T * stride, device="cuda")        # never filled: only the rows are touched
    far, at = dict(near), 0
    for k in ("u", "delta", "B", "C", "z", "dy"):
        t = near[k]
        inner = (t.stride(1),) if t.dim() == 2 else (t.stride(1), t.stride(2))
        far[k] = buf.as_strided(t.shape, (stride,) + inner, at)
        far[k].copy_(t)
        at += 4096
    for a, b in zip(all_calls(near), all_calls(far)):
        assert torch.equal(a, b)


def all_calls(d):
    """The outputs of the three calls, in one list."""
    import chunked_gated_delta_kda_amd as kda
    fwd = {k: v for k, v in d.items() if k != "dy"}
    step = {k: v for k, v in fwd.items() if k not in ("cu_seqlens", "initial_state")}
    state = torch.ones(d["u"].shape[0], d["u"].shape[1], d["A"].shape[1], device="cuda")
    return [*kda.ssm_fwd(**fwd), *kda.ssm_decode(**step, state=state), *kda.ssm_bwd(**d).values()]
