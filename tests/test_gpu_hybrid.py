"""The operators together, as a hybrid decoder runs them: the convolution in front of the delta rule and of
the scan, prompts continued token by token, a whole token step (convolution, scan, delta rule, attention
over a growing paged cache) captured and replayed, and the gradients of a chain. Every operator's output
is checked against its own 64-bit form on the inputs that it really got."""
import numpy as np
import pytest

import ops_oracle as oo

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from chunked_gated_delta_kda_amd import synth  # noqa: E402

pytestmark = pytest.mark.gpu

H, D = 2, 128
C = H * D


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def np64(t):
    return t.detach().to("cpu").double().numpy()


def unit(x):
    """Rows of one head at length one, as the delta rule wants its queries and keys."""
    x = x.float().view(-1, H, D)
    return (x / x.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(torch.bfloat16)


def test_convolution_and_delta_rule_prompt_then_tokens():
    import chunked_gated_delta_kda_amd as kda

    lengths, extra = [45, 1, 130], 3
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N = len(lengths)
    total = [n + extra for n in lengths]
    cut = np.concatenate([[0], np.cumsum(total)])
    # one projection for q, k and v; every sequence has `extra` tokens after its prompt
    proj = r(sum(total), 3 * C).to(torch.bfloat16).cuda()
    weight, bias = (r(3, C, 4) / 2).cuda(), (0.1 * r(3, C)).cuda()
    gate = torch.clamp(-torch.nn.functional.softplus(r(sum(total), H, D)), min=-5.0).cuda()
    beta = torch.sigmoid(r(sum(total), H)).cuda()
    prompt = torch.tensor(np.concatenate([np.arange(cut[i], cut[i] + n) for i, n in enumerate(lengths)])).cuda()
    token = lambda j: torch.tensor([int(cut[i]) + n + j for i, n in enumerate(lengths)]).cuda()  # noqa: E731
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()

    rows = proj[prompt]
    made, states = [], []
    for i in range(3):
        y, s = kda.conv_fwd(rows[:, i * C:(i + 1) * C], weight[i], bias[i], cu)
        made.append(y), states.append(s)
    q, k, v = unit(made[0]), unit(made[1]), made[2].view(-1, H, D).contiguous()
    o, S = kda.fwd(q, k, v, gate[prompt].contiguous(), beta[prompt].contiguous(), cu_seqlens=cu)
    seen = {n: [t] for n, t in dict(q=q, k=k, v=v, o=o).items()}
    for j in range(extra):
        at = token(j)
        step = []
        for i in range(3):
            y, states[i] = kda.conv_decode(proj[at][:, i * C:(i + 1) * C], weight[i], bias[i], states[i])
            step.append(y)
        q, k, v = unit(step[0]), unit(step[1]), step[2].view(-1, H, D).contiguous()
        o, S = kda.decode(q, k, v, gate[at].contiguous(), beta[at].contiguous(), state=S)
        for n, t in dict(q=q, k=k, v=v, o=o).items():
            seen[n].append(t)

    # the convolution of the whole sequences gives the same rows, bit for bit
    whole = torch.tensor(cut, dtype=torch.int32).cuda()
    order = torch.cat([prompt] + [token(j) for j in range(extra)])
    for i, n in enumerate(("q", "k", "v")):
        y, s = kda.conv_fwd(proj[:, i * C:(i + 1) * C], weight[i], bias[i], whole)
        want = y.view(-1, H, D) if n == "v" else unit(y)
        assert torch.equal(torch.cat(seen[n]), want[order]), n
        assert torch.equal(s, states[i]), n
    # the delta rule over them, against its oracle
    back = torch.argsort(order)
    full = {n: np64(torch.cat(seen[n])[back]) for n in ("q", "k", "v")}
    ro, rS = oracle.kda_forward(full["q"].astype(np.float32), full["k"].astype(np.float32), full["v"].astype(np.float32),
                                gate.cpu().numpy(), beta.cpu().numpy(), scale=1 / np.sqrt(D), cu_seqlens=cut.astype(np.int32))
    assert synth.passes(synth.parity(torch.cat(seen["o"])[back].cpu().numpy(), ro))
    assert synth.passes(synth.parity(S.cpu().numpy(), rS))


def test_a_captured_token_step_of_all_operators():
    """convolution -> scan -> (delta rule) -> attention, one graph for the step: replayed for four tokens, with
    the cache, its lengths and the states moving on in place, against the same steps run one by one."""
    import chunked_gated_delta_kda_amd as kda

    N, page, pages, width = 3, 16, 40, 8
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16).cuda()  # noqa: E731
    p = dict(w=(r(C, 4) / 2).cuda(), b=(0.1 * r(C)).cuda(), A=-torch.exp(r(C, 16) * 0.5).cuda(), Ds=torch.ones(C).cuda(),
             Win=bf(r(C, 2 * C + 32 + C) / C ** 0.5), Wq=bf(r(C, 3 * C) / C ** 0.5), db=(r(C) - 3).cuda())
    beta, gate = torch.full((N, H), 0.5).cuda(), (-0.1 * torch.ones(N, H, D)).cuda()
    start = [20, 31, 0]

    def fresh():
        return dict(x=bf(torch.zeros(N, C)), conv=bf(torch.zeros(N, 3, C)), ssm=torch.zeros(N, C, 16).cuda(),
                    S=torch.zeros(N, H, D, D).cuda(), k=bf(torch.zeros(pages, page, H, D)), v=bf(torch.zeros(pages, page, H, D)),
                    table=torch.arange(N * width, dtype=torch.int32).view(N, width).cuda(),
                    lens=torch.tensor(start, dtype=torch.int32).cuda(), out=bf(torch.zeros(N, C)))

    def step(s):
        z = s["x"] @ p["Win"]
        u, gt, B, Cm, dl = z[:, :C], z[:, C:2 * C], z[:, 2 * C:2 * C + 16], z[:, 2 * C + 16:2 * C + 32], z[:, 2 * C + 32:]
        a, _ = kda.conv_decode(u, p["w"], p["b"], s["conv"])
        y, _ = kda.ssm_decode(a, dl, p["A"], B.unflatten(1, (1, 16)), Cm.unflatten(1, (1, 16)), p["Ds"], gt, p["db"], s["ssm"])
        qkv = y @ p["Wq"]
        q, k, v = (qkv[:, i * C:(i + 1) * C].view(N, H, D) for i in range(3))
        o, _ = kda.decode(unit(q), unit(k), v.contiguous(), gate, beta, state=s["S"])
        at = s["lens"].long()
        where = torch.gather(s["table"], 1, (at // page)[:, None])[:, 0].long()
        s["k"][where, at % page] = k
        s["v"][where, at % page] = v
        s["lens"] += 1
        att = kda.attn_decode(q, s["k"], s["v"], s["table"], s["lens"])
        s["out"].copy_(att.reshape(N, C) + o.reshape(N, C).to(torch.bfloat16))
        return a, y, att

    prefix_k, prefix_v = bf(r(pages, page, H, D)), bf(r(pages, page, H, D))
    tokens = [bf(r(N, C)) for _ in range(4)]

    def begin(s):
        for n, t in fresh().items():
            s[n].copy_(t)
        s["k"].copy_(prefix_k), s["v"].copy_(prefix_v)

    eager = fresh()
    begin(eager)
    want = []
    for x in tokens:
        eager["x"].copy_(x)
        step(eager)
        want.append({n: eager[n].clone() for n in ("out", "conv", "ssm", "S", "lens")})
    live = fresh()
    begin(live)
    step(live)                      # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, y, att = step(live)
    for _ in range(2):
        begin(live)
        for x, ref in zip(tokens, want):
            live["x"].copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            for n, t in ref.items():
                assert torch.equal(live[n], t), n
            kda.attn_decode(bf(r(1, 2, D)), prefix_k, prefix_v, live["table"][:1], live["lens"][:1])   # eager work between
    # the last step's attention against its oracle
    q = (y @ p["Wq"])[:, :C].view(N, H, D)
    lens = live["lens"].tolist()
    ro, oe, _, _ = oo.attention(np64(q), np64(live["k"]), np64(live["v"]), live["table"].cpu().numpy(), lens, D ** -0.5, "bf16")
    oo.check("attention", np64(att), ro, oe / oo.U, "bf16", 1)


def test_gradients_of_a_chain():
    """conv -> scan in fp32: each backward against its oracle on what the forward and the other backward
    really gave it, and the chain against central differences (a step of 1/32; third derivatives and the
    loss's roundings stay within 2e-2 of the largest gradient)."""
    import chunked_gated_delta_kda_amd as kda

    lengths, ch, n = [9, 0, 30, 2], 6, 4
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, N = sum(lengths), len(lengths)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    x, w, b = r(T, ch).cuda(), (r(ch, 4) / 2).cuda(), (0.1 * r(ch)).cuda()
    delta, A = (0.5 * r(T, ch) - 1).cuda(), -torch.exp(0.3 * r(ch, n)).cuda()
    B, Cm, z, Ds = r(T, 1, n).cuda(), r(T, 1, n).cuda(), r(T, ch).cuda(), torch.ones(ch).cuda()
    dy = r(T, ch).cuda()

    def forward(x):
        a, _ = kda.conv_fwd(x, w, b, cu)
        y, _ = kda.ssm_fwd(a, delta, A, B, Cm, Ds, z, None, cu)
        return a, y

    a, _ = forward(x)
    gs = kda.ssm_bwd(a, delta, A, B, Cm, dy, Ds, z, None, cu)
    gc = kda.conv_bwd(x, w, gs["du"], b, cu)
    ref, err = oo.scan_grads(*(np64(t) for t in (a, delta, A, B, Cm, Ds, z)), None, lengths, None, True, np64(dy), None)
    oo.check("du", np64(gs["du"]), ref["du"], err["du"] + 2 * np.abs(ref["du"]), "fp32", 1)
    cref = oo.conv(np64(x), np64(w), np64(b), lengths, None, True, np64(gs["du"]), np.zeros((N, 3, ch)))
    oo.check("dx", np64(gc["dx"]), cref["dx"], cref["dx_size"], "fp32", 4 * 13)
    dyc = np64(dy)
    want = np64(gc["dx"]).reshape(-1)
    for i in range(0, T * ch, 11):
        side = []
        for sign in (1, -1):
            moved = x.clone().reshape(-1)
            moved[i] += sign / 32
            side.append(float((np64(forward(moved.view(T, ch))[1]) * dyc).sum()))
        assert abs((side[0] - side[1]) * 16 - want[i]) <= 2e-2 * max(1.0, np.abs(want).max()), i
