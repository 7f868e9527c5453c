"""The linear attention where segments of the time axis hold several chunks (more than 256 heads times chunks), against the
recurrence in 64 bits, element by element: strong decays, resets inside a segment, stretches of tokens a thousand times
larger than the rest in each of the inputs, gradients that end before the batch does.

Tolerances: one rounding to the output's type, plus what linear_oracle_card counts (worst cases). Gradients of decays are
also held to 2^-20 of |X| |Y|, the most that <X, Y> can be: they are sums of what passes their token and of nothing else, so that
their roundings are 2^-24 of that times the root of the number of sums behind a result, which stays under 16: a state
of 64 tokens rounded three times each (14), of which all that does not lie along the other one drops out."""
import pytest

import linear_oracle_card as lc
import ops_oracle as oo

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(lengths, H, K, V, kind, seed, fixed=False, init=True):
    g = torch.Generator().manual_seed(seed)
    dt, T, S = TYPES[kind], sum(lengths), len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32).cuda()
    slope = 0.1 + 0.2 * torch.rand(H, generator=g)
    d = dict(q=r(T, H, K).to(dt).cuda(), k=r(T, H, K).to(dt).cuda(), v=r(T, H, V).to(dt).cuda(),
             g=(-slope if fixed else -slope * (0.5 + torch.rand(T, H, generator=g))).cuda(), cu_seqlens=cu,
             initial_state=(0.3 * r(S, H, K, V)).cuda() if init else None)
    return d, r(T, H, V).to(dt).cuda(), (0.2 * r(S, H, K, V)).cuda()


def check(d, lengths, kind, do, df):
    import chunked_gated_delta_kda_amd as kda

    T, H, K = d["q"].shape
    assert T * H > 256 * 64, "segments of one chunk"
    out, fin = kda.lin_fwd(**d, check=True)
    got = dict(kda.lin_bwd(**d, d_out=do, d_final_state=df, check=True), out=out, final=fin)
    ref, err, most = lc.forward_and_backward(d, lengths, do, df, K ** -0.5)
    if d["g"].dim() == 1:
        ref["dg"], err["dg"], most = ref["dg"].sum(0), (err["dg"] + 8 * ref["dg"].abs()).sum(0), most.sum(0)
    for n, x in got.items():
        fp32 = n in ("final", "dg", "d_initial_state")
        half, tiny = oo.HALF["fp32" if fp32 else kind], oo.TINY["fp32" if fp32 else kind]
        off = (x.double() - ref[n]).abs()
        bound = half * ref[n].abs() + tiny + oo.U * err[n] * (1 + half)
        assert (off <= bound).all(), f"{n}: {(off / bound).max().item():.3g} of the bound, at {(off / bound).argmax().item()}"
    off = (got["dg"].double() - ref["dg"]).abs()
    bound = 2.0 ** -20 * most + 1e-30
    assert (off <= bound).all(), f"dg: {(off / bound).max().item():.3g} of the bound, at {(off / bound).argmax().item()}"
    again = kda.lin_bwd(**d, d_out=do, d_final_state=df)
    assert all(torch.equal(again[n], got[n]) for n in again)
    return got


# lengths, heads, K, V, type, g of [H], initial state: segments of two to eleven chunks, sequences of one segment and of several
CASES = [
    ([700], 64, 128, 128, "bf16", False, True),
    ([5, 300, 0, 1, 63, 200, 131], 64, 64, 128, "fp16", False, True),
    ([190, 510], 64, 128, 64, "bf16", True, False),
    ([150, 50], 300, 64, 64, "fp16", False, True),
    ([400], 96, 64, 64, "bf16", True, True),
    ([1100], 160, 64, 64, "bf16", False, True),
    ([90, 0, 610], 128, 64, 128, "fp16", False, True),
]
IDS = lambda c: f"{len(c[0])}x{max(c[0])}h{c[1]}k{c[2]}v{c[3]}{c[4]}{'f' if c[5] else ''}{'i' if c[6] else ''}"  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_several_chunks_a_segment(case):
    lengths, H, K, V, kind, fixed, init = case
    d, do, df = make(lengths, H, K, V, kind, 1, fixed, init)
    check(d, lengths, kind, do, df)


@pytest.mark.parametrize("name", ["q", "k", "v", "do", "all"])
def test_a_stretch_of_large_tokens(name):
    """Tokens a thousand times larger than the rest: what they leave in the sums of the decays' gradients goes with them."""
    lengths = [700]
    d, do, df = make(lengths, 64, 128, 128, "bf16", 2)
    for n, x in (("q", d["q"]), ("k", d["k"]), ("v", d["v"]), ("do", do)):
        if name in (n, "all"):
            x[200:264] *= 1000
    check(d, lengths, "bf16", do, df)


@pytest.mark.parametrize("at", [[64], [128], [256], [300], [255, 320], list(range(192, 256))], ids=lambda a: f"{len(a)}at{a[0]}")
@pytest.mark.parametrize("smaller", [1, 64])
def test_resets_inside_a_segment(at, smaller):
    """A reset on a chunk's first token, inside one and on a segment's: nothing of what was before it is left behind it."""
    lengths = [700]
    d, do, df = make(lengths, 64, 64, 128, "bf16", 3)
    d["g"][at] = -1e5       # (exp of it is 0)
    for x in (d["q"], d["k"], d["v"], do):
        x[at[0]:] /= smaller
    got = check(d, lengths, "bf16", do, df)
    d["g"][at] = float("-inf")
    import chunked_gated_delta_kda_amd as kda
    mine = kda.lin_bwd(**d, d_out=do, d_final_state=df)
    assert all(torch.equal(mine[n], got[n]) for n in mine)
    assert not got["dg"][at].any()


def test_gradients_that_end_before_the_batch():
    """No gradient after token 330: those of the decays there are 0, not what rounding left before."""
    lengths = [700]
    d, do, _ = make(lengths, 64, 128, 128, "bf16", 4)
    do[330:] = 0
    got = check(d, lengths, "bf16", do, None)
    assert not got["dg"][330:].any()


def test_slow_decays_and_a_query_that_takes_all():
    """With hardly any decay: queries and their gradients a thousand times larger in the middle leave what passes them by exact."""
    lengths = [300, 400]
    d, do, df = make(lengths, 64, 128, 128, "bf16", 5)
    d["g"] *= 0.01
    d["q"][130:190] *= 1000
    do[130:190] *= 1000
    check(d, lengths, "bf16", do, df)


@pytest.mark.parametrize("K,V", [(128, 128), (64, 128)])
def test_more_blocks_than_the_handed_on_states_hold(K, V):
    """Where the walks take the segments a range at a time: each head as in a call of its own (other segments: whole results, to
    what fp32 states and one rounding of the outputs leave), and the same bits from run to run and in a workspace full of NaN."""
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    lengths, H = ([70000, 70000] if K == 128 else [200000, 80000]), 8
    T = sum(lengths)
    d, do, df = make(lengths, H, K, V, "bf16", 6)
    d["g"] *= 0.1
    got = kda.lin_bwd(**d, d_out=do, d_final_state=df)
    need = native.load_library().kda_lin_bwd_workspace_bytes(2, T, H, K, V, 0, 1)
    assert need < 1.3 * 2 ** 30
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    again = kda.lin_bwd(**d, d_out=do, d_final_state=df, workspace=ws)
    assert all(torch.equal(again[n], got[n]) for n in got)
    for h in range(H):
        one = {n: d[n][:, h:h + 1].contiguous() for n in ("q", "k", "v", "g", "initial_state")}
        own = kda.lin_bwd(**one, cu_seqlens=d["cu_seqlens"], d_out=do[:, h:h + 1], d_final_state=df[:, h:h + 1].contiguous())
        for n, bound in (("dq", 2.0 ** -8), ("dk", 2.0 ** -8), ("dv", 2.0 ** -8), ("dg", 2.0 ** -18), ("d_initial_state", 2.0 ** -19)):
            a, b = got[n][:, h].double(), own[n][:, 0].double()
            assert (a - b).norm() <= bound * b.norm(), f"{n} of head {h}: {((a - b).norm() / b.norm()).item():.3g}"


def test_captured_gradients_whose_states_are_handed_on():
    """Segments of several chunks in a graph: replays with other inputs and offsets, eager calls between them, a value that is not
    finite in one of the prompts."""
    import chunked_gated_delta_kda_amd as kda

    lengths = [300, 0, 400]
    d, do, df = make(lengths, 64, 64, 64, "bf16", 7)
    step = lambda: [*kda.lin_fwd(**d), *kda.lin_bwd(**d, d_out=do, d_final_state=df).values()]  # noqa: E731
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    g = torch.Generator().manual_seed(8)
    for i in range(5):
        for n in ("q", "k", "v"):
            d[n].copy_(torch.randn(d[n].shape, generator=g))
        if i == 2:
            d["v"][100, 5, 7] = float("inf")
        d["cu_seqlens"].copy_(torch.tensor([0, 100 * i, 100 * i + 70, 700], dtype=torch.int32))
        graph.replay()
        want = step()
        for x, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)), (i, x)
            assert bool(torch.isfinite(a).all()) == (i != 2 or x in (4, 6)), (i, x)     # (dv and d_initial_state do not hang on v)
