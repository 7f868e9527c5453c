"""Attention of one new token on the GPU where probabilities or values are far from each other, against
the plain 64-bit form: one token that draws nearly all of the attention beside many with little."""
import numpy as np
import pytest

import ops_oracle as oo
from test_gpu_attn import make, np64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def place(d, seq, token):
    """The page and the row in it of a cached token."""
    page = d["k_cache"].shape[1]
    return int(d["block_table"][seq, token // page]), token % page


def oracle(d, lens, kind, scale=1.0):
    """ops_oracle.attention; in fp16 with what the split may lose of a probability put at 2^-40 of the
    largest one instead of 2^-25: probabilities are multiplied by 2^15 before they are split, and what is
    left after two parts is at most half of fp16's last step, 2^-25 of 2^15."""
    v = np.nan_to_num(np64(d["v_cache"]))
    table = d["block_table"].cpu().numpy()
    out, oe, lse, le = oo.attention(np64(d["q"]), np.nan_to_num(np64(d["k_cache"])), v, table, lens, scale, kind)
    if kind == "fp16":
        group, page = d["q"].shape[1] // v.shape[2], v.shape[1]
        for b, n in enumerate(lens):
            if n == 0:
                continue
            t = np.arange(n)
            size = np.abs(v[table[b, t // page], t % page]).sum(0).repeat(group, 0)
            k = np.nan_to_num(np64(d["k_cache"]))[table[b, t // page], t % page].repeat(group, 1)
            s = scale * np.einsum("thd,hd->ht", k, np64(d["q"])[b])
            L = np.exp(s - s.max(1, keepdims=True)).sum(1, keepdims=True)
            oe[b] -= (2.0 ** -25 - 2.0 ** -40) * size / L
    return out, oe, lse, le


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [10, 14, 16, 18, 21])
def test_small_probabilities_beside_a_large_one(kind, gap):
    """A token with a score `gap` above the others and value 0: the output is what the others add up
    to, each with a probability of e^-gap."""
    import chunked_gated_delta_kda_amd as kda

    lens = [256, 2000, 33, 700]
    d = make(lens, 8, 2, 64, 16, kind, 11)
    g = torch.Generator().manual_seed(gap)
    used = ~torch.isnan(d["k_cache"][..., :1])
    k = torch.zeros_like(d["k_cache"])
    k[..., 1] = (torch.randn(k.shape[:-1], generator=g) / 4).to(k.dtype).cuda()
    v = (100 + torch.randn(k.shape, generator=g)).to(k.dtype).cuda()
    for seq, token in enumerate((0, 1999, 5, 350)):
        at = place(d, seq, token)
        k[at[0], at[1], :, 0] = gap
        v[at[0], at[1]] = 0
    nan = torch.tensor(float("nan"), dtype=k.dtype, device="cuda")
    d["k_cache"], d["v_cache"] = torch.where(used, k, nan), torch.where(used, v, nan)
    d["q"] = torch.zeros_like(d["q"])
    d["q"][..., :2] = 1
    out, lse = kda.attn_decode(**d, scale=1.0, return_lse=True, check=True)
    ro, oe, rl, le = oracle(d, lens, kind)
    oo.check("out", np64(out), ro, oe / oo.U, kind, 1)
    oo.check("lse", np64(lse), rl, le / oo.U, "fp32", 1)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_values_that_are_not_finite(kind, dh):
    """An infinite value of a cached token makes its element infinite in every head that reads it, whatever the
    token's probability; infinities of both signs, or a NaN, make it NaN. Other elements keep theirs."""
    import chunked_gated_delta_kda_amd as kda

    lens, hkv, group, page = [40, 3000, 300, 129], 2, 3, 16
    d = make(lens, hkv * group, hkv, dh, page, kind, 21)
    k, v = d["k_cache"], d["v_cache"]
    at = place(d, 2, 17)                # beside a token with all but e^-30 of the attention
    k[at[0], at[1]] = 0
    k[at[0], at[1], :, 0] = 40
    d["q"][2] = 0
    d["q"][2, :, 0] = 1
    for t in range(lens[2]):
        if t != 17:
            p = place(d, 2, t)
            k[p[0], p[1], :, 0] = 10
    inf, nan = float("inf"), float("nan")
    want = {}                           # (sequence, cache head, element): what the output holds
    for seq, head, element, values in ((0, 0, 3, {7: inf}), (0, 1, 0, {39: -inf}), (1, 0, 5, {0: inf, 2999: inf}),
                                       (1, 0, dh - 1, {1500: -inf}), (1, 1, 8, {100: inf, 2000: -inf}), (1, 1, 9, {64: nan}),
                                       (2, 0, 1, {200: inf}), (2, 1, 2, {299: -inf}), (3, 0, 33, {128: inf})):
        for token, x in values.items():
            p = place(d, seq, token)
            v[p[0], p[1], head, element] = x
        want[seq, head, element] = sum(values.values())
    out, lse = kda.attn_decode(**d, scale=1.0, return_lse=True, check=True)
    got = np64(out)
    plain = dict(d, v_cache=torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0))
    ro, oe, rl, le = oracle(plain, lens, kind)
    for (seq, head, element), x in want.items():
        rows = got[seq, head * group:(head + 1) * group, element]
        assert (np.isnan(rows) if np.isnan(x) else rows == x).all(), (seq, head, element, x, rows)
        got[seq, head * group:(head + 1) * group, element] = ro[seq, head * group:(head + 1) * group, element]
    oo.check("out", got, ro, oe / oo.U, kind, 1)
    oo.check("lse", np64(lse), rl, le / oo.U, "fp32", 1)
