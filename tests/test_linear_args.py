"""The linear attention with a decay for each head: what its entry points refuse before anything is launched, and its
64-bit recurrence's gradients against differences. No GPU needed."""
import ctypes
import os

import numpy as np
import pytest

import linear_oracle as lo
from chunked_gated_delta_kda_amd import native

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(1 << 30)
MB = 1 << 20
T, H, K, V, S = 6, 3, 64, 128, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(native.LIB_PATH):
        pytest.skip("libkda.so not built")
    return native.load_library()


def test_the_recurrences_gradients_agree_with_differences():
    rng = np.random.Generator(np.random.PCG64(1))
    lengths = [4, 0, 3]
    x = {n: rng.standard_normal(s) for n, s in (("q", (7, 2, 3)), ("k", (7, 2, 3)), ("v", (7, 2, 5)), ("init", (3, 2, 3, 5)))}
    x["g"] = -rng.random((7, 2))
    do, df = rng.standard_normal((7, 2, 5)), rng.standard_normal((3, 2, 3, 5))

    def loss(x):
        o, _, f, _ = lo.forward(x["q"], x["k"], x["v"], x["g"], 0.7, lengths, x["init"])
        return (o * do).sum() + (f * df).sum()

    r, _ = lo.backward(x["q"], x["k"], x["v"], x["g"], 0.7, lengths, do, x["init"], df)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("init", "d_initial_state")):
        way = rng.standard_normal(x[name].shape)
        up, down = (loss({**x, name: x[name] + s * 1e-5 * way}) for s in (1, -1))
        assert abs((up - down) / 2e-5 - (r[grad] * way).sum()) < 1e-6, name


def _args(dt=torch.bfloat16, per_head=False):
    return dict(q=torch.zeros(T, H, K, dtype=dt), k=torch.zeros(T, H, K, dtype=dt), v=torch.zeros(T, H, V, dtype=dt),
                g=torch.zeros(H) if per_head else torch.zeros(T, H), cu_seqlens=torch.zeros(S + 1, dtype=torch.int32),
                initial_state=torch.zeros(S, H, K, V))


def test_good_arguments():
    from chunked_gated_delta_kda_amd.linear import check_lin_bwd_args, check_lin_decode_args, check_lin_fwd_args
    s = check_lin_fwd_args(**_args())
    assert (s.T, s.H, s.K, s.V, s.S, s.per_head, s.strides) == (T, H, K, V, S, False, [H * K, K, H * K, K, H * V, V])
    assert check_lin_fwd_args(**_args(torch.float16, True)).per_head
    wide = torch.zeros(T, H * (2 * K + V), dtype=torch.bfloat16)
    a = _args()
    a["q"], a["k"], a["v"] = (x.unflatten(1, (H, -1)) for x in wide.split([H * K, H * K, H * V], 1))
    assert check_lin_fwd_args(**a).strides == [H * (2 * K + V), K] * 2 + [H * (2 * K + V), V]
    s, d = check_lin_bwd_args(**_args(), d_out=torch.zeros(T, H, 2 * V, dtype=torch.bfloat16)[..., :V])
    assert d == [2 * H * V, 2 * V]
    a = _args()
    a.pop("cu_seqlens"), a.pop("initial_state")
    assert check_lin_decode_args(**a, state=torch.zeros(T, H, K, V)).S == T


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(T, H, 32, dtype=torch.bfloat16)), ("q", torch.zeros(T, H, K)), ("q", torch.zeros(T, K, dtype=torch.bfloat16)),
    ("k", torch.zeros(T, H, 128, dtype=torch.bfloat16)), ("k", torch.zeros(T, H + 1, K, dtype=torch.bfloat16)),
    ("v", torch.zeros(T, H, 96, dtype=torch.bfloat16)), ("v", torch.zeros(T, H, V, dtype=torch.float16)),
    ("v", torch.zeros(T + 1, H, V, dtype=torch.bfloat16)), ("k", torch.zeros(T, H, K + 4, dtype=torch.bfloat16)[..., :K]),
    ("g", torch.zeros(T, H, dtype=torch.bfloat16)), ("g", torch.zeros(T)), ("g", torch.zeros(H, T).t()), ("scale", float("inf")),
    ("scale", float("nan")), ("cu_seqlens", torch.zeros(S + 1, dtype=torch.int64)), ("cu_seqlens", torch.zeros(1, dtype=torch.int32)),
    ("initial_state", torch.zeros(S, H, V, K)), ("initial_state", torch.zeros(S, H, K, V, dtype=torch.bfloat16)),
    ("initial_state", torch.zeros(S + 1, H, K, V)),
])
def test_rejects(name, bad):
    from chunked_gated_delta_kda_amd.linear import check_lin_bwd_args, check_lin_fwd_args
    a = _args()
    a[name] = bad
    with pytest.raises(ValueError):
        check_lin_fwd_args(**a)
    with pytest.raises(ValueError):
        check_lin_bwd_args(**a, d_out=torch.zeros(T, H, V, dtype=torch.bfloat16))


def test_rejects_outputs_states_and_places():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd.linear import check_lin_bwd_args, check_lin_decode_args, check_lin_fwd_args
    with pytest.raises(ValueError, match="out"):
        check_lin_fwd_args(**_args(), out=torch.zeros(T, H, V))
    with pytest.raises(ValueError, match="final_state"):
        check_lin_fwd_args(**_args(), final_state=torch.zeros(S, H, K, V, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="d_out"):
        check_lin_bwd_args(**_args(), d_out=torch.zeros(T, H, V))
    with pytest.raises(ValueError, match="d_final_state"):
        check_lin_bwd_args(**_args(), d_out=torch.zeros(T, H, V, dtype=torch.bfloat16), d_final_state=torch.zeros(S, H, K))
    a = _args()
    a.pop("cu_seqlens"), a.pop("initial_state")
    for kw in (dict(state=torch.zeros(S, H, K, V)), dict(state_out="copy"), dict(state_out=torch.zeros(1)), dict(out=torch.zeros(1))):
        with pytest.raises(ValueError):
            check_lin_decode_args(**a, **kw)
    with pytest.raises(ValueError, match="row"):
        check_lin_decode_args(a["q"][:0], a["k"][:0], a["v"][:0], torch.zeros(H))
    with pytest.raises(ValueError, match="device"):
        kda.lin_fwd(**_args())
    with pytest.raises(ValueError, match="device"):
        kda.lin_bwd(**_args(), d_out=torch.zeros(T, H, V, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device"):
        kda.lin_decode(**a)


def lin_args(**over):
    a = dict(q=1 * MB, k=2 * MB, v=3 * MB, g=4 * MB, cu_seqlens=5 * MB, initial_state=6 * MB, final_state=8 * MB, out=10 * MB,
             q_stride=H * K, q_head_stride=K, k_stride=H * K, k_head_stride=K, v_stride=H * V, v_head_stride=V, num_seqs=S,
             total_tokens=T, heads=H, key_dim=K, value_dim=V, dtype=1, g_per_head=0, scale=0.1)
    a.update(over)
    return native.KdaLinArgs(**a)


BAD = [(3, dict(dtype=0)), (3, dict(dtype=3)), (3, dict(key_dim=32)), (3, dict(value_dim=256)), (3, dict(g_per_head=2)),
       (3, dict(scale=float("nan"))), (3, dict(q_stride=H * K + 4)), (3, dict(v_head_stride=V + 1)), (3, dict(q=MB + 8)),
       (3, dict(initial_state=6 * MB + 4)), (2, dict(num_seqs=0)), (2, dict(total_tokens=-1)), (2, dict(heads=0)),
       (2, dict(heads=65536)), (2, dict(total_tokens=(1 << 27) + 1)), (2, dict(k_stride=-8)), (2, dict(num_seqs=1 << 27)),
       (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(g=None))]


@pytest.mark.parametrize("code,kw", BAD)
def test_abi_refusals(lib, code, kw):
    assert lib.kda_lin_fwd(ctypes.byref(lin_args(**kw)), None, None, 0) == code
    if "num_seqs" not in kw and "total_tokens" not in kw:
        assert lib.kda_lin_decode(ctypes.byref(lin_args(cu_seqlens=None, num_seqs=T, **kw)), None) == code
    assert lib.kda_lin_bwd(ctypes.byref(lin_args(**kw)), ctypes.byref(lin_grads()), None, None, 0) == code


def test_abi_refusals_of_outputs(lib):
    fwd = lambda ws=None, n=0, **kw: lib.kda_lin_fwd(ctypes.byref(lin_args(**kw)), None, ws, n)  # noqa: E731
    assert lib.kda_lin_fwd(None, None, None, 0) == 1 and fwd(out=None) == 1
    assert fwd(cu_seqlens=None) == 2                # two sequences without offsets
    assert fwd(out=10 * MB + 8) == 3 and fwd(final_state=8 * MB + 8) == 3
    for kw in (dict(out=1 * MB), dict(out=2 * MB + 16), dict(final_state=6 * MB), dict(final_state=3 * MB), dict(out=8 * MB),
               dict(out=4 * MB), dict(out=5 * MB), dict(final_state=6 * MB + 64)):
        assert fwd(**kw) == 7, kw
    need = lib.kda_lin_workspace_bytes(4096, 8, K, V)
    assert need > 0 and lib.kda_lin_workspace_bytes(4096, 8, 32, V) == 0 and lib.kda_lin_workspace_bytes(-1, 8, K, V) == 0
    far = dict(total_tokens=4096, heads=8, q=MB << 4, k=MB << 6, v=MB << 8, g=MB << 10, out=MB << 12, final_state=MB << 14)
    assert fwd(P, need - 1, **far) == 4
    assert fwd(ctypes.c_void_p((1 << 30) + 8), need, **far) == 4
    dec = lambda **kw: lib.kda_lin_decode(ctypes.byref(lin_args(**{**dict(cu_seqlens=None, num_seqs=T), **kw})), None)  # noqa: E731
    assert lib.kda_lin_decode(None, None) == 1
    assert dec(cu_seqlens=5 * MB) == 2 and dec(num_seqs=T + 1) == 2
    assert dec(final_state=6 * MB + 64) == 7 and dec(out=6 * MB) == 7


def lin_grads(**over):
    g = dict(d_out=20 * MB, d_final_state=21 * MB, dq=23 * MB, dk=24 * MB, dv=25 * MB, dg=26 * MB, d_initial_state=27 * MB,
             d_out_stride=H * V, d_out_head_stride=V)
    g.update(over)
    return native.KdaLinGrads(**g)


def test_abi_refusals_of_gradients(lib):
    def bwd(grads=None, ws=P, n=0, **kw):
        return lib.kda_lin_bwd(ctypes.byref(lin_args(**kw)), ctypes.byref(lin_grads(**(grads or {}))), None, ws, n)

    assert lib.kda_lin_bwd(None, None, None, None, 0) == 1
    assert lib.kda_lin_bwd(ctypes.byref(lin_args()), None, None, None, 0) == 1
    for name in ("d_out", "dq", "dk", "dv", "dg"):
        assert bwd({name: None}) == 1, name
    assert bwd(dict(dg=None), total_tokens=0, g_per_head=1) == 1
    assert bwd(dict(d_out_stride=-8)) == 2 and bwd(cu_seqlens=None) == 2
    for g in (dict(d_out_stride=H * V + 2), dict(dq=23 * MB + 8), dict(d_final_state=21 * MB + 4), dict(d_initial_state=27 * MB + 4)):
        assert bwd(g) == 3, g
    for g in (dict(dq=1 * MB), dict(dk=6 * MB), dict(dv=20 * MB), dict(dg=21 * MB), dict(d_initial_state=6 * MB), dict(dq=24 * MB),
              dict(dg=4 * MB), dict(dv=5 * MB)):
        assert bwd(g) == 7, g
    size = lambda *a: lib.kda_lin_bwd_workspace_bytes(*a)  # noqa: E731
    need = size(S, T, H, K, V, 0, 1)
    assert need > 0 and bwd(n=need - 1) == 4
    assert size(S, T, H, K, V, 0, 0) == need + S * H * K * V * 4        # the gradient that the caller does not take
    assert bwd(dict(d_initial_state=None), n=need) == 4
    assert size(S, T, H, K, V, 1, 1) > need and size(S, T, H, 32, V, 0, 1) == 0
