"""Infinities and NaN among the inputs of the linear attention: what comes before them keeps its bits, and of what comes from them
on, what does not hang on them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(lengths, H, K, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    T, dt = sum(lengths), TYPES[kind]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(q=r(T, H, K).to(dt).cuda(), k=r(T, H, K).to(dt).cuda(), v=r(T, H, V).to(dt).cuda(),
                g=(-0.05 * torch.rand(T, H, generator=g)).cuda(), initial_state=r(len(lengths), H, K, V).cuda(),
                cu_seqlens=torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32).cuda())


# one launch, segments, segments whose sequences blocks share, a chunk in the middle of a long segment
BATCHES = [([100, 150], 2), ([700, 1, 900], 2), ([9] * 60 + [300], 3), ([1200], 64)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lengths,H", BATCHES, ids=lambda b: str(len(b)) if isinstance(b, list) else f"h{b}")
def test_values_reach_their_column_from_their_token_on(lengths, H, K, V, kind):
    import chunked_gated_delta_kda_amd as kda

    d = make(lengths, H, K, V, kind, 1)
    T = sum(lengths)
    out, fin = kda.lin_fwd(**d)
    g = torch.Generator().manual_seed(2)
    e = dict(d, v=d["v"].clone())
    hit = torch.zeros(T, H, V, dtype=torch.bool)
    last = torch.zeros(len(lengths), H, V, dtype=torch.bool)
    places = [(0, 0, 0), (T - 1, H - 1, V - 1)] + [[int(torch.randint(0, n, (1,), generator=g)) for n in (T, H, V)] for _ in range(30)]
    for x, (t, h, c) in enumerate(places):
        e["v"][t, h, c] = (INF, -INF, float("nan"))[x % 3]
        end = next(n for n in range(len(lengths)) if t < sum(lengths[:n + 1]))
        hit[t:sum(lengths[:end + 1]), h, c] = True
        last[end, h, c] = True
    hit, last = hit.cuda(), last.cuda()[:, :, None].expand_as(fin)
    o, f = kda.lin_fwd(**e)
    assert torch.equal(o[~hit], out[~hit]) and torch.equal(f[~last], fin[~last])
    assert not torch.isfinite(o[hit]).any() and not torch.isfinite(f[last]).any()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["q", "k", "g"])
def test_what_comes_before_keeps_its_bits(name, kind):
    import chunked_gated_delta_kda_amd as kda

    lengths, H = [300, 130], 2
    d = make(lengths, H, 128, 128, kind, 3)
    out, fin = kda.lin_fwd(**d)
    for bad in (INF, -INF, float("nan")) if name != "g" else (INF, float("nan")):
        for t in (0, 63, 64, 100, 299, 300, 429):
            e = dict(d, **{name: d[name].clone()})
            at = (t, 1, 5) if name != "g" else (t, 1)
            e[name][at] = bad
            o, f = kda.lin_fwd(**e)
            rest = torch.ones(430, H, dtype=torch.bool, device="cuda")
            end = 300 if t < 300 else 430
            rest[t:t + 1 if name == "q" else end, 1] = False
            assert torch.equal(o[rest], out[rest]), (bad, t)
            assert not torch.isfinite(o[~rest]).any(1).any(), (bad, t)
            assert torch.equal(f[:, 0], fin[:, 0]) and torch.equal(f[int(t < 300), 1], fin[int(t < 300), 1])
            assert torch.equal(f, fin) == (name == "q")
