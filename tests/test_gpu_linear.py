"""The linear attention with a decay for each head on the GPU against its recurrence in 64 bits (linear_oracle): prompts over
packed batches, gradients, single tokens; lengths of zero, one and around a chunk, segments that sequences start, end and
pass in, strides, resets, far decays, values that are not finite, streams and graphs. Tolerances: one rounding to
the output's type, plus what linear_oracle counts; and, as those are worst cases, a bound on the relative error of whole
fp32 results: roundings of 2^-24 with random signs over sums of n terms add up to about sqrt(n) of them, which for
the hundreds of terms here stays under 2^-20."""
import numpy as np
import pytest

import linear_oracle as lo
import ops_oracle as oo

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def np64(t):
    return t.detach().to("cpu").double().numpy() if t is not None else None


def make(lengths, H, K, V, kind, seed, fixed=False, init=True, joint=False, slope=0.1):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[kind]
    T, S = sum(lengths), len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if joint:
        q, k, v = (x.unflatten(1, (H, -1)) for x in r(T, H * (2 * K + V)).to(dt).cuda().split([H * K, H * K, H * V], 1))
    else:
        q, k, v = r(T, H, K).to(dt).cuda(), r(T, H, K).to(dt).cuda(), r(T, H, V).to(dt).cuda()
    per = slope * torch.exp(r(H))
    return dict(q=q, k=k, v=v, g=(-per if fixed else -per * torch.rand(T, H, generator=g) * 2).cuda(),
                cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda(),
                initial_state=(0.3 * r(S, H, K, V)).cuda() if init else None)


def decays(d):
    g = np64(d["g"])
    return g if g.ndim == 2 else np.broadcast_to(g, (d["q"].shape[0], len(g)))


def near(name, got, ref, bound=2.0 ** -20):
    n = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= bound * n + 1e-30, f"{name}: relative error {np.linalg.norm(got - ref) / n:.3g}"


def check_forward(d, lengths, kind, scale=None, **kw):
    import chunked_gated_delta_kda_amd as kda

    out, fin = kda.lin_fwd(**d, scale=scale, **kw)
    s = d["q"].shape[2] ** -0.5 if scale is None else scale
    ro, eo, rf, ef = lo.forward(np64(d["q"]), np64(d["k"]), np64(d["v"]), decays(d), s, lengths, np64(d["initial_state"]))
    oo.check("out", np64(out), ro, eo, kind, 1)
    oo.check("final", np64(fin), rf, ef, "fp32", 1)
    near("final", np64(fin), rf)
    return out, fin


# lengths, heads, K, V, type, g of [H], initial state, one tensor
CASES = [
    ([1], 1, 64, 64, "bf16", False, False, False),
    ([7], 2, 128, 128, "bf16", True, True, False),
    ([63, 64, 65], 1, 128, 128, "bf16", False, True, True),
    ([0, 3, 0, 0, 70, 1, 2, 0], 3, 64, 128, "fp16", False, True, False),
    ([130, 0, 200], 2, 128, 64, "bf16", False, False, True),
    ([16, 17, 300], 2, 64, 64, "fp16", True, True, True),
    ([129, 128], 2, 128, 128, "fp16", False, True, False),
    ([400], 5, 128, 128, "bf16", False, True, False),
    ([0], 2, 64, 128, "bf16", False, True, False),
    ([5] * 40, 2, 128, 64, "fp16", False, True, False),
]
IDS = lambda c: f"{len(c[0])}x{max(c[0])}h{c[1]}k{c[2]}v{c[3]}{c[4]}{'f' if c[5] else ''}{'i' if c[6] else ''}{'j' if c[7] else ''}"  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    import chunked_gated_delta_kda_amd as kda

    lengths, H, K, V, kind, fixed, init, joint = case
    d = make(lengths, H, K, V, kind, 1, fixed, init, joint)
    out, fin = check_forward(d, lengths, kind, check=True)
    again, fagain = kda.lin_fwd(**d)
    assert torch.equal(out, again) and torch.equal(fin, fagain)
    only, none = kda.lin_fwd(**d, output_final_state=False)
    assert none is None and torch.equal(only, out)


def check_backward(d, lengths, kind, seed, scale=None, dfin=True, **kw):
    import chunked_gated_delta_kda_amd as kda

    T, H, V = d["v"].shape
    S, K = len(lengths), d["q"].shape[2]
    g = torch.Generator().manual_seed(seed)
    do = torch.randn(T, 2, H, V, generator=g).to(TYPES[kind]).cuda()[:, 0]
    df = (0.2 * torch.randn(S, H, K, V, generator=g)).cuda() if dfin else None
    got = kda.lin_bwd(**d, d_out=do, d_final_state=df, scale=scale, **kw)
    s = K ** -0.5 if scale is None else scale
    ref, err = lo.backward(np64(d["q"]), np64(d["k"]), np64(d["v"]), decays(d), s, lengths, np64(do), np64(d["initial_state"]), np64(df))
    if d["g"].dim() == 1:
        ref["dg"], err["dg"] = ref["dg"].sum(0), (err["dg"] + 8 * np.abs(ref["dg"])).sum(0)
    for n in ("dq", "dk", "dv"):
        oo.check(n, np64(got[n]), ref[n], err[n], kind, 1)
    for n in ("dg", "d_initial_state"):
        if got[n] is not None:
            oo.check(n, np64(got[n]), ref[n], err[n], "fp32", 1)
            if ref[n].size:
                near(n, np64(got[n]), ref[n])
    return do, df, got


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    import chunked_gated_delta_kda_amd as kda

    lengths, H, K, V, kind, fixed, init, joint = case
    d = make(lengths, H, K, V, kind, 2, fixed, init, joint)
    do, df, got = check_backward(d, lengths, kind, 3, check=True)
    again = kda.lin_bwd(**d, d_out=do, d_final_state=df)
    without = kda.lin_bwd(**d, d_out=do, d_final_state=df, need_d_initial_state=False)
    assert without.pop("d_initial_state") is None
    for n in got:
        assert torch.equal(got[n], again[n]), n
        assert n not in without or torch.equal(got[n], without[n]), n


def test_backward_without_a_final_states_gradient():
    d = make([70, 200], 2, 128, 128, "bf16", 4, init=False)
    check_backward(d, [70, 200], "bf16", 5, dfin=False)


@pytest.mark.parametrize("scale", [0.0, -0.5, 1.0])
def test_scales(scale):
    lengths = [100, 9]
    d = make(lengths, 2, 64, 64, "bf16", 6)
    check_forward(d, lengths, "bf16", scale)
    check_backward(d, lengths, "bf16", 7, scale)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_decays_of_every_size(kind):
    """No decay at all, resets (-infinity, the lowest number), decays past the range of sums, and mixtures of them."""
    import chunked_gated_delta_kda_amd as kda

    lengths = [150, 60]
    g = torch.Generator().manual_seed(8)
    for how in ("none", "resets", "far", "mixed"):
        d = make(lengths, 3, 64, 128, kind, 9)
        x = {"none": torch.zeros(210, 3), "resets": torch.where(torch.rand(210, 3, generator=g) < 0.1, float("-inf"), -0.05),
             "far": -100.0 * torch.rand(210, 3, generator=g),
             "mixed": torch.tensor([0.0, -1e-3, -3.0, -88.0, torch.finfo(torch.float32).min])[torch.randint(0, 5, (210, 3), generator=g)]}
        d["g"] = x[how].cuda()
        out, fin = kda.lin_fwd(**d)
        gd = np.maximum(decays(d), -1e5)      # exp of either is 0
        s = 64 ** -0.5
        ro, eo, rf, ef = lo.forward(np64(d["q"]), np64(d["k"]), np64(d["v"]), gd, s, lengths, np64(d["initial_state"]))
        oo.check(how, np64(out), ro, eo, kind, 1)
        oo.check(how, np64(fin), rf, ef, "fp32", 1)
        e = dict(d, g=torch.from_numpy(gd.copy()).float().cuda())
        check_backward(e, lengths, kind, 10)
        a = kda.lin_bwd(**d, d_out=d["v"])
        b = kda.lin_bwd(**e, d_out=d["v"])
        assert all(torch.equal(a[n], b[n]) for n in a), how


def test_gradients_agree_with_differences():
    """Central differences of <out, c> + <final, f> in 64 bits against the kernel's gradients, along random directions."""
    import chunked_gated_delta_kda_amd as kda

    lengths, H, K, V = [70, 3], 2, 64, 64
    d = make(lengths, H, K, V, "bf16", 11)
    rng = np.random.Generator(np.random.PCG64(12))
    do = torch.from_numpy(rng.standard_normal((73, H, V))).to(torch.bfloat16).cuda()
    df = torch.from_numpy(rng.standard_normal((2, H, K, V))).float().cuda()
    got = kda.lin_bwd(**d, d_out=do, d_final_state=df)
    base = {n: np64(d[n]) for n in ("q", "k", "v", "g", "initial_state")}

    def loss(x):
        o, _, f, _ = lo.forward(x["q"], x["k"], x["v"], x["g"], K ** -0.5, lengths, x["initial_state"])
        return (o * np64(do)).sum() + (f * np64(df)).sum()

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("initial_state", "d_initial_state")):
        way = rng.standard_normal(base[name].shape)
        h = 1e-4
        up, down = (loss({**base, name: base[name] + s * h * way}) for s in (1, -1))
        want = (up - down) / (2 * h)
        have = (np64(got[grad]) * way).sum()
        # 16-bit gradients: a rounding of 2^-9 on average each, with random signs; differences: h^2 of the third derivative
        size = np.linalg.norm(np64(got[grad]) * way)
        assert abs(have - want) <= 2.0 ** -8 * size + 1e-5 * abs(want) + 1e-4, name


@pytest.mark.parametrize("lengths,H", [([3000], 2), ([700, 1, 0, 1500, 64, 300], 3), ([1] * 300 + [900], 1),
                                       ([1, 0, 0, 2, 3] * 30 + [400] + [0, 1] * 40, 2)])
def test_many_segments(lengths, H):
    """Long enough for many segments; against the recurrence on the card in 64 bits."""
    import chunked_gated_delta_kda_amd as kda

    K = V = 128
    d = make(lengths, H, K, V, "bf16", 13, slope=0.01)
    out, fin = kda.lin_fwd(**d, check=True)
    q, k, v, g, h0 = (d[n].double() for n in ("q", "k", "v", "g", "initial_state"))
    do = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    df = 0.1 * torch.ones_like(d["initial_state"])
    got = kda.lin_bwd(**d, d_out=do, d_final_state=df)
    scale, at, x = K ** -0.5, 0, do.double()
    ref = {n: torch.zeros_like(t).double() for n, t in (("o", v), ("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    fins, dinit = [], []
    for n, length in enumerate(lengths):
        S, trail = h0[n], []
        for t in range(at, at + length):
            S = S * torch.exp(g[t])[:, None, None]
            trail.append(S)
            S = S + k[t][:, :, None] * v[t][:, None]
            ref["o"][t] = scale * (q[t][:, None] @ S)[:, 0]
            ref["dq"][t] = scale * (S @ x[t][:, :, None])[:, :, 0]
        fins.append(S)
        Y = df[n].double()
        for t in range(at + length - 1, at - 1, -1):
            Y = Y + scale * q[t][:, :, None] * x[t][:, None]
            ref["dk"][t], ref["dv"][t] = (Y @ v[t][:, :, None])[:, :, 0], (k[t][:, None] @ Y)[:, 0]
            ref["dg"][t] = (trail[t - at] * Y).sum((1, 2))
            Y = Y * torch.exp(g[t])[:, None, None]
        dinit.append(Y)
        at += length
    # whole results: one rounding to bf16 is 2^-8 / sqrt(3) at most on average; fp32 as said above
    for name, a, b, bound in (("out", out, ref["o"], 2.0 ** -8), ("final", fin, torch.stack(fins), 2.0 ** -20),
                              ("dq", got["dq"], ref["dq"], 2.0 ** -8), ("dk", got["dk"], ref["dk"], 2.0 ** -8),
                              ("dv", got["dv"], ref["dv"], 2.0 ** -8), ("dg", got["dg"], ref["dg"], 2.0 ** -19),
                              ("d_initial_state", got["d_initial_state"], torch.stack(dinit), 2.0 ** -20)):
        near(name, np64(a), np64(b), bound)


def test_sequences_and_heads_do_not_meet():
    """Whatever a sequence or head holds, the others' results are the same bits."""
    import chunked_gated_delta_kda_amd as kda

    lengths = [100, 30, 200]
    d = make(lengths, 2, 128, 128, "bf16", 14)
    do = torch.randn(330, 2, 128, device="cuda").to(torch.bfloat16)
    out, fin = kda.lin_fwd(**d)
    got = kda.lin_bwd(**d, d_out=do)
    for bad in (float("nan"), float("inf")):
        e = {k: x.clone() for k, x in d.items()}
        for n in ("q", "k", "v"):
            e[n][110, 1] = bad
        e["g"][120, 1] = bad
        e["initial_state"][1, 1] = bad
        o, f = kda.lin_fwd(**e)
        b = kda.lin_bwd(**e, d_out=do)
        rest = torch.ones(330, 2, dtype=torch.bool, device="cuda")
        rest[100:130, 1] = False
        keep = torch.ones(3, 2, dtype=torch.bool, device="cuda")
        keep[1, 1] = False
        assert torch.equal(o[rest], out[rest]) and torch.equal(f[keep], fin[keep])
        assert all(torch.equal(b[n][rest], got[n][rest]) for n in ("dq", "dk", "dv", "dg"))
        assert torch.equal(b["d_initial_state"][keep], got["d_initial_state"][keep])
        assert not torch.isfinite(o[110:130, 1]).any()


def test_malformed_offsets_raise_and_stay_inside():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    for bad in ([0, 150, 100, 400], [5, 100, 200, 400], [0, 100, 200, 390], [0, -5, 2 ** 31 - 1, 400], [0, 400, 400, -2 ** 31]):
        d = make([100, 100, 200], 2, 64, 64, "bf16", 15)
        d["cu_seqlens"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda: kda.lin_fwd(**d, check=True), lambda: kda.lin_bwd(**d, d_out=d["v"], check=True)):
            with pytest.raises(native.KdaDeviceError) as err:
                call()
            assert err.value.bits == 2


def test_malformed_offsets_of_many_sequences_stay_inside():
    """Where blocks share the parts of a segment: offsets in no order, with values outside, raise; inputs and guards stay."""
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    T, H = 500, 2
    g = torch.Generator().manual_seed(40)
    d = make([T // 50] * 50, H, 128, 128, "bf16", 41)
    held = torch.full((T + 128, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    for i in range(6):
        cu = torch.randint(-20, T + 40, (51,), generator=g, dtype=torch.int32)
        if i % 2:
            cu = cu.sort().values      # in order, with an end that is not the batch's
        d["cu_seqlens"] = cu.cuda()
        with pytest.raises(native.KdaDeviceError):
            kda.lin_fwd(**d, out=held[64:T + 64], check=True)
        assert (held[:64] == 7).all() and (held[T + 64:] == 7).all()


@pytest.mark.parametrize("K,V,kind,fixed", [(64, 64, "bf16", False), (64, 128, "fp16", True), (128, 64, "bf16", True), (128, 128, "fp16", False)])
def test_one_token(K, V, kind, fixed):
    import chunked_gated_delta_kda_amd as kda

    N, H = 5, 3
    d = make([1] * N, H, K, V, kind, 16, fixed, joint=True)
    s = d["initial_state"]
    args = (d["q"], d["k"], d["v"], d["g"], None)
    out, new = kda.lin_decode(*args, s.clone())
    ro, eo, rf, ef = lo.forward(np64(d["q"]), np64(d["k"]), np64(d["v"]), decays(d), K ** -0.5, [1] * N, np64(s))
    oo.check("out", np64(out), ro, eo, kind, 1)
    oo.check("state", np64(new), rf, ef, "fp32", 1)
    mine = s.clone()
    o2, same = kda.lin_decode(*args, mine)
    assert same is mine and torch.equal(mine, new) and torch.equal(o2, out)
    o3, none = kda.lin_decode(*args, s, state_out=None)
    assert none is None and torch.equal(o3, out)
    to = torch.empty_like(s)
    o4, t4 = kda.lin_decode(*args, s, state_out=to)
    assert t4 is to and torch.equal(to, new) and torch.equal(o4, out)
    o5, fresh = kda.lin_decode(*args)
    ro, eo, rf, ef = lo.forward(np64(d["q"]), np64(d["k"]), np64(d["v"]), decays(d), K ** -0.5, [1] * N, None)
    oo.check("out", np64(o5), ro, eo, kind, 1)
    oo.check("state", np64(fresh), rf, ef, "fp32", 1)


def test_prompt_continued_by_prompts_and_tokens():
    import chunked_gated_delta_kda_amd as kda

    n = 150
    d = make([n], 2, 128, 128, "bf16", 17, slope=0.02)
    ro, eo, rf, ef = lo.forward(np64(d["q"]), np64(d["k"]), np64(d["v"]), decays(d), 128 ** -0.5, [n], np64(d["initial_state"]))
    state, outs = d["initial_state"], []
    for a, b in ((0, 70), (70, 71), (71, 140)):
        o, state = kda.lin_fwd(d["q"][a:b], d["k"][a:b], d["v"][a:b], d["g"][a:b], None, None, state)
        outs.append(o)
    for t in range(140, n):
        o, state = kda.lin_decode(d["q"][t:t + 1], d["k"][t:t + 1], d["v"][t:t + 1], d["g"][t:t + 1], None, state)
        outs.append(o)
    oo.check("out", np64(torch.cat(outs)), ro, eo, "bf16", 1)
    oo.check("final", np64(state), rf, ef, "fp32", 1)


def test_gradients_of_parts_are_those_of_the_whole():
    """A sequence cut where its state is known: d_initial_state of what follows is d_final_state of what precedes."""
    import chunked_gated_delta_kda_amd as kda

    n, cut = 200, 75
    d = make([n], 2, 64, 128, "bf16", 18)
    do = torch.randn(n, 2, 128, device="cuda").to(torch.bfloat16)
    whole = kda.lin_bwd(**d, d_out=do)
    one = lambda a, b, s: dict(q=d["q"][a:b], k=d["k"][a:b], v=d["v"][a:b], g=d["g"][a:b], initial_state=s)  # noqa: E731
    _, mid = kda.lin_fwd(**one(0, cut, d["initial_state"]))
    late = kda.lin_bwd(**one(cut, n, mid), d_out=do[cut:])
    early = kda.lin_bwd(**one(0, cut, d["initial_state"]), d_out=do[:cut], d_final_state=late["d_initial_state"])
    for name in ("dq", "dk", "dv"):
        near(name, np64(torch.cat([early[name], late[name]])), np64(whole[name]), 2.0 ** -8)
    near("dg", np64(torch.cat([early["dg"], late["dg"]])), np64(whole["dg"]), 2.0 ** -19)
    near("d_initial_state", np64(early["d_initial_state"]), np64(whole["d_initial_state"]))


def test_captured_and_on_another_stream():
    """A captured prompt, gradients and token, replayed with new inputs between eager calls; the same on a side stream."""
    import chunked_gated_delta_kda_amd as kda

    lengths = [300, 0, 77]
    d = make(lengths, 2, 128, 128, "bf16", 19)
    do = torch.randn(377, 2, 128, device="cuda").to(torch.bfloat16)
    tok = make([1] * 3, 2, 128, 128, "bf16", 20, init=False)
    state = torch.zeros(3, 2, 128, 128, device="cuda")

    def step(d, do, tok, state):
        out, fin = kda.lin_fwd(**d)
        state.copy_(fin)
        o1, _ = kda.lin_decode(tok["q"], tok["k"], tok["v"], tok["g"], None, state)
        return dict(kda.lin_bwd(**d, d_out=do, d_final_state=fin), out=out, fin=fin, o1=o1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step(d, do, tok, state.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(d, do, tok, state)
    eager = step(d, do, tok, state.clone())
    assert all(torch.equal(on_side[n], eager[n]) for n in eager)
    g = torch.Generator().manual_seed(21)
    for i in range(4):
        for n in ("q", "k", "v"):
            d[n].copy_(torch.randn(d[n].shape, generator=g))
        d["cu_seqlens"].copy_(torch.tensor([0, 100 + i, 100 + i, 377], dtype=torch.int32))
        graph.replay()
        want = step(d, do, tok, state.clone())
        mine = step(d, do, tok, state.clone())
        assert all(torch.equal(held[n], want[n]) and torch.equal(mine[n], want[n]) for n in want), i


def test_caller_workspace_and_buffers():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    d = make([900], 2, 128, 128, "bf16", 22)
    out, fin = kda.lin_fwd(**d)
    lib = native.load_library()
    need = lib.kda_lin_workspace_bytes(900, 2, 128, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")        # NaN wherever it is read before it is written
    o, f = torch.empty_like(out), torch.empty_like(fin)
    r = kda.lin_fwd(**d, out=o, final_state=f, workspace=ws)
    assert r[0] is o and r[1] is f and torch.equal(o, out) and torch.equal(f, fin)
    got = kda.lin_bwd(**d, d_out=out)
    need = lib.kda_lin_bwd_workspace_bytes(1, 900, 2, 128, 128, 0, 1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    mine = kda.lin_bwd(**d, d_out=out, workspace=ws)
    assert all(torch.equal(got[n], mine[n]) for n in got)
    with pytest.raises(native.KdaError):
        kda.lin_bwd(**d, d_out=out, workspace=ws[:-4])


def test_no_tokens_without_offsets():
    """One sequence of no tokens: the final state is the initial one, and its gradient goes straight through."""
    import chunked_gated_delta_kda_amd as kda

    d = make([0], 3, 64, 128, "bf16", 30)
    d["cu_seqlens"] = None
    fin = torch.full_like(d["initial_state"], float("nan"))
    out, fin = kda.lin_fwd(**d, final_state=fin, check=True)
    assert out.shape == (0, 3, 128) and torch.equal(fin, d["initial_state"])
    _, none = kda.lin_fwd(**dict(d, initial_state=None), final_state=torch.full_like(fin, float("nan")))
    assert not none.any()
    for fixed in (False, True):
        g = d["g"] if not fixed else torch.full((3,), -0.1, device="cuda")
        got = kda.lin_bwd(**dict(d, g=g), d_out=out, d_final_state=fin)
        assert torch.equal(got["d_initial_state"], fin) and not got["dg"].any() and got["dg"].shape == g.shape


def test_shared_rows_and_rows_far_apart():
    """Keys that all heads share (stride 0), a query that all tokens share, and values as far apart as they may lie (rows past
    2^32 bytes): the same results as copies, bit by bit."""
    import chunked_gated_delta_kda_amd as kda

    T, H, D, far = 200, 4, 128, 1 << 24
    d = make([90, 110], H, D, D, "bf16", 31)
    d["k"] = d["k"][:, :1].expand(T, H, D)
    d["q"] = d["q"][:1].expand(T, H, D)
    wide = torch.empty(T * far, dtype=torch.bfloat16, device="cuda").view(T, far)[:, far - H * D:].unflatten(1, (H, D))
    wide.copy_(d["v"])
    apart = dict(d, v=wide)
    copies = {n: t.clone(memory_format=torch.contiguous_format) for n, t in d.items()}
    do = torch.randn(T, H, D, generator=torch.Generator().manual_seed(32)).to(torch.bfloat16).cuda()
    for a, b in zip(kda.lin_fwd(**apart, check=True), kda.lin_fwd(**copies)):
        assert torch.equal(a, b)
    a, b = kda.lin_bwd(**apart, d_out=do), kda.lin_bwd(**copies, d_out=do)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    tok = lambda x: [x[n][:1] for n in ("q", "k", "v", "g")]  # noqa: E731
    assert torch.equal(kda.lin_decode(*tok(apart))[0], kda.lin_decode(*tok(copies))[0])


def test_a_long_prompt_is_its_parts():
    """65536 tokens in one call and in four that hand on their states, and the gradients likewise: whole results to what
    fp32 states and one rounding of the outputs leave."""
    import chunked_gated_delta_kda_amd as kda

    n, part, H = 65536, 16384, 2
    d = make([n], H, 128, 128, "bf16", 33, slope=0.002)
    d.pop("cu_seqlens")
    do = torch.randn(n, H, 128, generator=torch.Generator().manual_seed(34)).to(torch.bfloat16).cuda()
    out, fin = kda.lin_fwd(**d)
    whole = kda.lin_bwd(**d, d_out=do)
    states, outs = [d["initial_state"]], []
    cut = lambda i: {x: d[x][i * part:(i + 1) * part] for x in ("q", "k", "v", "g")}  # noqa: E731
    for i in range(4):
        o, s = kda.lin_fwd(**cut(i), initial_state=states[-1])
        outs.append(o)
        states.append(s)
    near("out", np64(torch.cat(outs)), np64(out), 2.0 ** -8)
    near("final", np64(states[-1]), np64(fin), 2.0 ** -19)
    grads, back = [], None
    for i in (3, 2, 1, 0):
        grads.insert(0, kda.lin_bwd(**cut(i), d_out=do[i * part:(i + 1) * part], initial_state=states[i], d_final_state=back))
        back = grads[0]["d_initial_state"]
    for name in ("dq", "dk", "dv"):
        near(name, np64(torch.cat([x[name] for x in grads])), np64(whole[name]), 2.0 ** -8)
    near("dg", np64(torch.cat([x["dg"] for x in grads])), np64(whole["dg"]), 2.0 ** -18)
    near("d_initial_state", np64(back), np64(whole["d_initial_state"]), 2.0 ** -19)


def test_few_chunks_and_many_sequences_in_as_many_tokens():
    """256 tokens as one sequence, as four and as 256, with no more workspace than is asked for."""
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    need = native.load_library().kda_lin_workspace_bytes(256, 3, 128, 128)
    for lengths in ([256], [64] * 4, [65, 63, 128], [1] * 256):
        d = make(lengths, 3, 128, 128, "bf16", 42)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        out, fin = check_forward(d, lengths, "bf16", check=True, workspace=ws)
        again, fagain = kda.lin_fwd(**d)
        assert torch.equal(out, again) and torch.equal(fin, fagain)


def test_two_calls_at_once():
    """Calls on two streams side by side, each with workspaces of its own."""
    import chunked_gated_delta_kda_amd as kda

    jobs = [make([3000, 200], 8, 128, 128, "bf16", 35), make([1500], 12, 64, 128, "fp16", 36)]
    dos = [torch.randn(j["v"].shape, generator=torch.Generator().manual_seed(37)).to(j["v"].dtype).cuda() for j in jobs]
    run = lambda j, do: [*kda.lin_fwd(**j), *kda.lin_bwd(**j, d_out=do).values()]  # noqa: E731
    want = [run(j, do) for j, do in zip(jobs, dos)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for j, do, s in zip(jobs, dos, streams):
            with torch.cuda.stream(s):
                got.append(run(j, do))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2])), i


def test_a_captured_token_of_a_hybrid_block():
    """What one token of a model of both kinds of layers runs: a step of the linear attention, new keys and values into a 4-bit
    cache, attention over it; captured once, replayed while inputs and lengths change, every replay against eager calls."""
    import chunked_gated_delta_kda_amd as kda

    B, H, hq, hkv, D, page, W = 4, 4, 8, 2, 128, 16, 6
    g = torch.Generator().manual_seed(38)
    half = torch.arange(W * page)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
    rope = torch.cat([half.cos(), half.sin()], 1).float().cuda()
    table = torch.randperm(B * W, generator=g).to(torch.int32).view(B, W).cuda()
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, 3 * H * D, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(B, (hq + 2 * hkv) * D, dtype=torch.bfloat16, device="cuda")
    decay = -0.1 * torch.rand(H, generator=g).cuda()

    def step(state, cache, outs=(None, None, None)):
        q, k, v = (t.unflatten(1, (H, D)) for t in x.chunk(3, 1))
        o, _ = kda.lin_decode(q, k, v, decay, None, state, out=outs[0])
        q, k, v = (t.unflatten(1, (-1, D)) for t in y.split([hq * D, hkv * D, hkv * D], 1))
        kc, vc, ks, vs = cache
        q = kda.kv_append(k, v, kc, vc, table, lens, rope=rope, q=q, k_scale=ks, v_scale=vs, q_out=outs[1])
        return o, q, kda.attn_decode_fp4(q, kc, vc, ks, vs, table, lens, out=outs[2])

    state = lambda: torch.zeros(B, H, D, D, device="cuda")  # noqa: E731
    cache = lambda: kda.kv_cache_fp4(B * W, page, hkv, D)  # noqa: E731
    outs = [t.clone() for t in step(state(), cache())]
    mine, theirs, sm, st = cache(), cache(), state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(sm, mine, outs)
    for i in range(12):
        lens.copy_(torch.tensor([i + 1, i + 30, i + 60, 0 if i % 4 == 3 else i + 2], dtype=torch.int32))
        x.copy_(torch.randn(x.shape, generator=g))
        y.copy_(torch.randn(y.shape, generator=g))
        graph.replay()
        want = step(st, theirs, [None, outs[1].clone(), None])
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
        assert torch.equal(sm, st) and all(torch.equal(a, b) for a, b in zip(mine, theirs)), i
