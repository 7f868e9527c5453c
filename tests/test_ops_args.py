"""Refusals of the operators beside the delta rule, on the CPU: the binding's checks of caller
tensors, and the C ABI's checks before anything is enqueued."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

from chunked_gated_delta_kda_amd import native  # noqa: E402
from chunked_gated_delta_kda_amd.short_conv import (check_conv_bwd_args, check_conv_decode_args,  # noqa: E402
                                                    check_conv_fwd_args)

P = 4096   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(native.LIB_PATH):
        pytest.skip("libkda.so not built")
    return native.load_library()


# ---------------------------------------------------------------- short convolution
T, C, W, N = 20, 12, 4, 3


def _conv():
    return dict(x=torch.zeros(T, C, dtype=torch.bfloat16), weight=torch.zeros(C, W), bias=torch.zeros(C),
                cu_seqlens=torch.tensor([0, 5, 5, T], dtype=torch.int32),
                initial_state=torch.zeros(N, W - 1, C, dtype=torch.bfloat16))


def test_conv_good_arguments():
    a = _conv()
    assert check_conv_fwd_args(**a) == (T, C, W, N, C)
    a["x"] = torch.zeros(T, 3 * C, dtype=torch.bfloat16)[:, C:2 * C]     # a slice of a projection
    assert check_conv_fwd_args(**a, out=torch.empty(T, C, dtype=torch.bfloat16)) == (T, C, W, N, 3 * C)
    assert check_conv_bwd_args(**a, dy=torch.zeros(T, C, dtype=torch.bfloat16))[4:] == (3 * C, C)
    assert check_conv_fwd_args(torch.zeros(0, C), torch.zeros(C, 2)) == (0, C, 2, 1, C)


@pytest.mark.parametrize("name,bad", [
    ("x", lambda: torch.zeros(T, C, dtype=torch.float64)),
    ("x", lambda: torch.zeros(T, 2, C // 2, dtype=torch.bfloat16)),
    ("x", lambda: torch.zeros(C, T, dtype=torch.bfloat16).t()),                  # columns contiguous
    ("x", lambda: torch.zeros(1, C, dtype=torch.bfloat16).expand(T, C)),         # rows overlap
    ("weight", lambda: torch.zeros(C, W, dtype=torch.bfloat16)),
    ("weight", lambda: torch.zeros(C, 9)),
    ("weight", lambda: torch.zeros(C, 1)),
    ("weight", lambda: torch.zeros(C + 1, W)),
    ("weight", lambda: torch.zeros(W, C).t()),
    ("bias", lambda: torch.zeros(C + 1)),
    ("cu_seqlens", lambda: torch.tensor([0, T])[:1]),
    ("cu_seqlens", lambda: torch.tensor([0, 5, 5, T])),
    ("initial_state", lambda: torch.zeros(N, W - 1, C)),
    ("initial_state", lambda: torch.zeros(N, W, C, dtype=torch.bfloat16)),
    ("activation", lambda: "gelu"),
])
def test_conv_rejects(name, bad):
    a = _conv()
    a[name] = bad()
    with pytest.raises(ValueError, match=name):
        check_conv_fwd_args(**a)


def test_conv_rejects_outputs_and_gradients():
    a = _conv()
    with pytest.raises(ValueError, match="out"):
        check_conv_fwd_args(**a, out=torch.empty(T, C))
    with pytest.raises(ValueError, match="final_state"):
        check_conv_fwd_args(**a, final_state=torch.empty(N + 1, W - 1, C, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dy"):
        check_conv_bwd_args(**a, dy=torch.zeros(T, C))
    with pytest.raises(ValueError, match="d_final_state"):
        check_conv_bwd_args(**a, dy=torch.zeros(T, C, dtype=torch.bfloat16), d_final_state=a["initial_state"])
    x, w = a["x"], a["weight"]
    with pytest.raises(ValueError, match="state"):
        check_conv_decode_args(x, w, None, torch.zeros(T, W - 1, C))
    with pytest.raises(ValueError, match="state_out"):
        check_conv_decode_args(x, w, None, None, state_out="elsewhere")
    with pytest.raises(ValueError, match="x"):
        check_conv_decode_args(x[:0], w)


def test_conv_needs_device_tensors():
    import chunked_gated_delta_kda_amd as kda
    a = _conv()
    with pytest.raises(ValueError, match="device"):
        kda.conv_fwd(**a)
    with pytest.raises(ValueError, match="device"):
        kda.conv_decode(a["x"], a["weight"])
    with pytest.raises(ValueError, match="device"):
        kda.conv_bwd(a["x"], a["weight"], a["x"])


def conv_args(**over):
    big = 1 << 30
    a = dict(x=P, weight=big, bias=None, cu_seqlens=None, initial_state=None, final_state=None, out=2 * big, x_stride=C,
             num_seqs=1, total_tokens=T, channels=C, width=W, dtype=1, activation=1)
    a.update(over)
    return native.KdaConvArgs(**a)


def test_conv_abi_refusals(lib):
    fwd = lambda **kw: lib.kda_conv_fwd(ctypes.byref(conv_args(**kw)), None)  # noqa: E731
    assert lib.kda_conv_fwd(None, None) == 1
    for kw in (dict(dtype=3), dict(dtype=-1), dict(width=1), dict(width=9), dict(activation=2)):
        assert fwd(**kw) == 3, kw
    for kw in (dict(num_seqs=0), dict(total_tokens=-1), dict(channels=0), dict(x_stride=C - 1), dict(num_seqs=2),
               dict(total_tokens=(1 << 27) + 1), dict(channels=(1 << 20) + 1, x_stride=1 << 21)):
        assert fwd(**kw) == 2, kw
    for kw in (dict(x=None), dict(weight=None), dict(out=None)):
        assert fwd(**kw) == 1, kw
    es = 2
    for kw in (dict(out=P + T * C * es - 2),                                     # out over x's last element
               dict(initial_state=1 << 20, final_state=1 << 20),                 # in place: a race over tiles
               dict(final_state=P), dict(out=1 << 20, final_state=1 << 20), dict(out=1 << 20, initial_state=1 << 20)):
        assert fwd(**kw) == 7, kw


def test_conv_decode_abi_refusals(lib):
    dec = lambda **kw: lib.kda_conv_decode(ctypes.byref(conv_args(num_seqs=T, **kw)), None)  # noqa: E731
    assert dec(cu_seqlens=P) == 2
    assert dec(total_tokens=T + 1) == 2
    assert dec(out=None) == 1
    state = T * (W - 1) * C * 2
    assert dec(initial_state=1 << 20, final_state=(1 << 20) + state - 2) == 7
    assert dec(out=P) == 7


def test_conv_bwd_abi_refusals(lib):
    big = 1 << 30

    def bwd(grads=(), ws=P, nbytes=0, **kw):
        g = dict(dy=3 * big, d_final_state=None, dx=4 * big, dweight=5 * big, dbias=None, d_initial_state=None, dy_stride=C)
        g.update(grads)
        return lib.kda_conv_bwd(ctypes.byref(conv_args(**kw)), ctypes.byref(native.KdaConvGrads(**g)), None, ws, nbytes)

    assert lib.kda_conv_bwd(None, None, None, None, 0) == 1
    for g in (dict(dy=None), dict(dx=None), dict(dweight=None)):
        assert bwd(g) == 1, g
    assert bwd(dict(dy_stride=C - 1)) == 2
    assert bwd(width=9) == 3
    assert bwd(num_seqs=2) == 2
    for g in (dict(dx=P), dict(dx=3 * big), dict(dweight=1 * big), dict(d_initial_state=3 * big), dict(dweight=4 * big),
              dict(dbias=5 * big)):
        assert bwd(g) == 7, g
    need = lib.kda_conv_bwd_workspace_bytes(T, C, W)
    assert need >= (W + 1) * C * 4 and bwd(nbytes=need - 1) == 4
    assert bwd(ws=P + 8, nbytes=need) == 4                                       # not aligned to 16 bytes
    assert lib.kda_conv_bwd_workspace_bytes(-1, C, W) == 0 and lib.kda_conv_bwd_workspace_bytes(T, C, 9) == 0


# ---------------------------------------------------------------- selective scan
Dn, Ns, G = 12, 5, 3


def _ssm():
    bf = torch.bfloat16
    return dict(u=torch.zeros(T, Dn, dtype=bf), delta=torch.zeros(T, Dn, dtype=bf), A=torch.zeros(Dn, Ns),
                B=torch.zeros(T, G, Ns, dtype=bf), C=torch.zeros(T, G, Ns, dtype=bf), D=torch.zeros(Dn),
                z=torch.zeros(T, Dn, dtype=bf), delta_bias=torch.zeros(Dn),
                cu_seqlens=torch.tensor([0, 5, 5, T], dtype=torch.int32), initial_state=torch.zeros(N, Dn, Ns))


def test_ssm_good_arguments():
    from chunked_gated_delta_kda_amd.scan import check_ssm_decode_args, check_ssm_fwd_args
    a = _ssm()
    s = check_ssm_fwd_args(**a)
    assert (s.T, s.D, s.N, s.G, s.S, s.strides) == (T, Dn, Ns, G, N, [Dn, Dn, G * Ns, G * Ns, Dn])
    proj = torch.zeros(T, 2 * Dn + 2 * G * Ns, dtype=torch.bfloat16)       # slices of one projection
    a.update(u=proj[:, :Dn], z=proj[:, Dn:2 * Dn], B=proj[:, 2 * Dn:2 * Dn + G * Ns].unflatten(1, (G, Ns)),
             C=proj[:, 2 * Dn + G * Ns:].unflatten(1, (G, Ns)))
    w = proj.shape[1]
    assert check_ssm_fwd_args(**a).strides == [w, Dn, w, w, w]
    a.update(D=None, z=None, delta_bias=None, cu_seqlens=None, initial_state=None)
    assert check_ssm_fwd_args(**a).S == 1
    del a["cu_seqlens"], a["initial_state"]
    assert check_ssm_decode_args(**a, state=torch.zeros(T, Dn, Ns)).S == T


@pytest.mark.parametrize("name,bad", [
    ("u", lambda: torch.zeros(T, Dn, dtype=torch.float64)),
    ("u", lambda: torch.zeros(T, G, 4, dtype=torch.bfloat16)),
    ("delta", lambda: torch.zeros(T, Dn)),
    ("delta", lambda: torch.zeros(T, 1, dtype=torch.bfloat16)),
    ("A", lambda: torch.zeros(Dn, 257)),
    ("A", lambda: torch.zeros(Dn, 0)),
    ("A", lambda: torch.zeros(Ns, Dn).t()),
    ("A", lambda: torch.zeros(Dn, Ns, dtype=torch.bfloat16)),
    ("B", lambda: torch.zeros(T, Ns, dtype=torch.bfloat16)),
    ("B", lambda: torch.zeros(T, 5, Ns, dtype=torch.bfloat16)),              # 5 groups do not divide 12 channels
    ("B", lambda: torch.zeros(T, Ns, G, dtype=torch.bfloat16).transpose(1, 2)),
    ("C", lambda: torch.zeros(T, 1, Ns, dtype=torch.bfloat16)),
    ("D", lambda: torch.zeros(Dn, dtype=torch.bfloat16)),
    ("z", lambda: torch.zeros(T - 1, Dn, dtype=torch.bfloat16)),
    ("delta_bias", lambda: torch.zeros(1)),
    ("initial_state", lambda: torch.zeros(N, Dn, Ns, dtype=torch.bfloat16)),
    ("initial_state", lambda: torch.zeros(N, Ns, Dn)),
])
def test_ssm_rejects(name, bad):
    from chunked_gated_delta_kda_amd.scan import check_ssm_fwd_args
    a = _ssm()
    a[name] = bad()
    with pytest.raises(ValueError, match=f"{name}:"):
        check_ssm_fwd_args(**a)


def test_ssm_rejects_outputs():
    from chunked_gated_delta_kda_amd.scan import check_ssm_decode_args, check_ssm_fwd_args
    import chunked_gated_delta_kda_amd as kda
    a = _ssm()
    with pytest.raises(ValueError, match="out"):
        check_ssm_fwd_args(**a, out=torch.empty(T, Dn))
    with pytest.raises(ValueError, match="final_state"):
        check_ssm_fwd_args(**a, final_state=torch.empty(N, Dn, Ns + 1))
    with pytest.raises(ValueError, match="device"):
        kda.ssm_fwd(**a)
    del a["cu_seqlens"], a["initial_state"]
    with pytest.raises(ValueError, match="state"):
        check_ssm_decode_args(**a, state=torch.zeros(N, Dn, Ns))
    with pytest.raises(ValueError, match="state_out"):
        check_ssm_decode_args(**a, state_out="new")
    with pytest.raises(ValueError, match="device"):
        kda.ssm_decode(**a)


def ssm_args(**over):
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    a = {n: (i + 1) << 20 for i, n in enumerate(names)}
    a.update(cu_seqlens=None, initial_state=16 << 20, final_state=17 << 20, out=18 << 20, u_stride=Dn, delta_stride=Dn,
             B_stride=G * Ns, C_stride=G * Ns, z_stride=Dn, num_seqs=1, total_tokens=T, channels=Dn, state_size=Ns, groups=G,
             dtype=1, delta_softplus=1)
    a.update(over)
    return native.KdaSsmArgs(**a)


def test_ssm_abi_refusals(lib):
    fwd = lambda ws=P, n=0, **kw: lib.kda_ssm_fwd(ctypes.byref(ssm_args(**kw)), None, ws, n)  # noqa: E731
    assert lib.kda_ssm_fwd(None, None, None, 0) == 1
    for kw in (dict(dtype=3), dict(delta_softplus=2)):
        assert fwd(**kw) == 3, kw
    for kw in (dict(num_seqs=0), dict(num_seqs=2), dict(total_tokens=-1), dict(channels=0), dict(state_size=0),
               dict(state_size=257), dict(groups=5), dict(groups=0), dict(u_stride=Dn - 1), dict(B_stride=G * Ns - 1),
               dict(z_stride=0), dict(total_tokens=(1 << 27) + 1), dict(C_stride=(1 << 27) + 1)):
        assert fwd(**kw) == 2, kw
    for kw in (dict(u=None), dict(delta=None), dict(A=None), dict(B=None), dict(C=None), dict(out=None)):
        assert fwd(**kw) == 1, kw
    for kw in (dict(out=1 << 20), dict(out=7 << 20), dict(final_state=16 << 20), dict(final_state=3 << 20),
               dict(final_state=18 << 20)):
        assert fwd(**kw) == 7, kw
    long = 1 << 20
    need = lib.kda_ssm_workspace_bytes(1, long, Dn, Ns, G)
    far = {n: (i + 1) << 40 for i, n in enumerate(("u", "delta", "B", "C", "z", "out"))}
    assert need > 0 and fwd(n=need - 1, total_tokens=long, **far) == 4
    assert lib.kda_ssm_workspace_bytes(1, 16, Dn, Ns, G) == 0         # one launch needs none
    assert lib.kda_ssm_workspace_bytes(1, T, Dn, Ns, 5) == 0          # not a valid shape
    assert lib.kda_ssm_workspace_bytes(0, T, Dn, Ns, G) == 0


def test_ssm_decode_abi_refusals(lib):
    dec = lambda **kw: lib.kda_ssm_decode(ctypes.byref(ssm_args(num_seqs=T, **kw)), None)  # noqa: E731
    assert dec(cu_seqlens=P) == 2 and dec(total_tokens=T - 1) == 2
    assert dec(out=None) == 1
    state = T * Dn * Ns * 4
    assert dec(final_state=(16 << 20) + state - 4) == 7
    assert dec(out=2 << 20) == 7


# ---------------------------------------------------------------- paged token attention
def _attn(dt=torch.bfloat16):
    return dict(q=torch.zeros(3, 8, 128, dtype=dt), k_cache=torch.zeros(10, 16, 2, 128, dtype=dt),
                v_cache=torch.zeros(10, 16, 2, 128, dtype=dt), block_table=torch.zeros(3, 4, dtype=torch.int32),
                seq_lens=torch.zeros(3, dtype=torch.int32))


def test_attn_good_arguments():
    from chunked_gated_delta_kda_amd.paged_attention import check_attn_decode_args
    a = _attn()
    assert check_attn_decode_args(**a) == (3, 8, 2, 128, 10, 16, 4)
    joint = torch.zeros(10, 2, 2, 16, 128, dtype=torch.bfloat16)       # keys and values side by side, heads first
    a.update(k_cache=joint[:, 0].transpose(1, 2), v_cache=joint[:, 1].transpose(1, 2))
    assert check_attn_decode_args(**a)[2] == 2
    a["block_table"] = torch.zeros(3, 9, dtype=torch.int32)[:, :4]
    assert check_attn_decode_args(**a)[6] == 4


@pytest.mark.parametrize("name,bad", [
    ("q", lambda: torch.zeros(3, 8, 128)),
    ("q", lambda: torch.zeros(3, 8, 96, dtype=torch.bfloat16)),
    ("q", lambda: torch.zeros(0, 8, 128, dtype=torch.bfloat16)),
    ("q", lambda: torch.zeros(3, 7, 128, dtype=torch.bfloat16)),
    ("q", lambda: torch.zeros(3, 8, 132, dtype=torch.bfloat16)[..., :128]),             # strides not multiples of 8
    ("q", lambda: torch.zeros(3 * 8 * 128 + 1, dtype=torch.bfloat16)[1:].view(3, 8, 128)),  # base not aligned
    ("k_cache", lambda: torch.zeros(10, 16, 2, 128, dtype=torch.float16)),
    ("k_cache", lambda: torch.zeros(10, 16, 2, 64, dtype=torch.bfloat16)),
    ("k_cache", lambda: torch.zeros(0, 16, 2, 128, dtype=torch.bfloat16)),
    ("v_cache", lambda: torch.zeros(10, 8, 2, 128, dtype=torch.bfloat16)),
    ("v_cache", lambda: torch.zeros(10, 16, 128, 2, dtype=torch.bfloat16).transpose(2, 3)),
    ("block_table", lambda: torch.zeros(3, 4, dtype=torch.int64)),
    ("block_table", lambda: torch.zeros(2, 4, dtype=torch.int32)),
    ("block_table", lambda: torch.zeros(4, 3, dtype=torch.int32).t()),
    ("block_table", lambda: torch.zeros(3, 0, dtype=torch.int32)),
    ("seq_lens", lambda: torch.zeros(3, dtype=torch.int64)),
    ("seq_lens", lambda: torch.zeros(4, dtype=torch.int32)),
    ("scale", lambda: float("nan")),
    ("out", lambda: torch.zeros(3, 8, 128)),
    ("lse", lambda: torch.zeros(3, 8, dtype=torch.bfloat16)),
])
def test_attn_rejects(name, bad):
    from chunked_gated_delta_kda_amd.paged_attention import check_attn_decode_args
    a = _attn()
    a[name] = bad()
    with pytest.raises(ValueError, match=f"{name}:"):
        check_attn_decode_args(**a)


def test_attn_needs_device_tensors():
    import chunked_gated_delta_kda_amd as kda
    with pytest.raises(ValueError, match="device"):
        kda.attn_decode(**_attn())


def test_attn_abi_refusals(lib):
    def call(ws=P, n=1 << 40, **over):
        mb = 1 << 20
        a = dict(q=mb, k_cache=16 * mb, v_cache=32 * mb, block_table=48 * mb, seq_lens=49 * mb, out=50 * mb, lse=None,
                 q_stride=1024, q_head_stride=128, k_page_stride=4096, k_token_stride=256, k_head_stride=128,
                 v_page_stride=4096, v_token_stride=256, v_head_stride=128, table_stride=4, num_seqs=3, q_heads=8, kv_heads=2,
                 head_dim=128, num_pages=10, page_size=16, table_width=64, dtype=1, scale=0.1)
        a["table_stride"] = 64
        a.update(over)
        return lib.kda_attn_decode(ctypes.byref(native.KdaAttnArgs(**a)), None, ws, n)

    assert lib.kda_attn_decode(None, None, None, 0) == 1
    for kw in (dict(dtype=0), dict(dtype=3), dict(head_dim=96), dict(scale=float("inf")), dict(k_token_stride=252),
               dict(q_stride=1020), dict(q=(1 << 20) + 8), dict(v_cache=(32 << 20) + 2)):
        assert call(**kw) == 3, kw
    for kw in (dict(num_seqs=0), dict(q_heads=7), dict(kv_heads=0), dict(num_pages=0), dict(page_size=0), dict(table_width=0),
               dict(table_stride=63), dict(k_head_stride=-8), dict(table_width=1 << 27, table_stride=1 << 27),
               dict(num_seqs=1 << 22)):
        assert call(**kw) == 2, kw
    for name in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "out"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(out=1 << 20), dict(out=16 << 20), dict(lse=50 << 20), dict(lse=49 << 20), dict(out=48 << 20)):
        assert call(**kw) == 7, kw
    need = lib.kda_attn_workspace_bytes(3, 8, 2, 128, 64, 16)
    assert need > 0 and call(n=need - 1) == 4
    assert lib.kda_attn_workspace_bytes(3, 8, 2, 128, 1, 16) == 0        # one chunk each: none needed
    assert lib.kda_attn_workspace_bytes(3, 7, 2, 128, 1, 16) == 0


def test_ssm_bwd_rejects():
    from chunked_gated_delta_kda_amd.scan import check_ssm_bwd_args
    import chunked_gated_delta_kda_amd as kda
    a = _ssm()
    dy = torch.zeros(T, 2 * Dn, dtype=torch.bfloat16)[:, :Dn]
    s, stride = check_ssm_bwd_args(**a, dy=dy, d_final_state=torch.zeros(N, Dn, Ns))
    assert (s.T, stride) == (T, 2 * Dn)
    with pytest.raises(ValueError, match="dy"):
        check_ssm_bwd_args(**a, dy=torch.zeros(T, Dn))
    with pytest.raises(ValueError, match="d_final_state"):
        check_ssm_bwd_args(**a, dy=dy, d_final_state=torch.zeros(N, Dn, Ns, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device"):
        kda.ssm_bwd(**a, dy=dy)


def test_ssm_bwd_abi_refusals(lib):
    def bwd(grads=(), ws=P, nbytes=0, **kw):
        names = ("dy", "d_final_state", "du", "ddelta", "dB", "dC", "dz", "dA", "dD", "ddelta_bias", "d_initial_state")
        g = {n: (32 + i) << 20 for i, n in enumerate(names)}
        g["dy_stride"] = Dn
        g.update(grads)
        return lib.kda_ssm_bwd(ctypes.byref(ssm_args(**kw)), ctypes.byref(native.KdaSsmGrads(**g)), None, ws, nbytes)

    assert lib.kda_ssm_bwd(None, None, None, None, 0) == 1
    for g in (dict(dy=None), dict(du=None), dict(ddelta=None), dict(dB=None), dict(dC=None), dict(dz=None), dict(dA=None)):
        assert bwd(g) == 1, g
    assert bwd(dict(dy_stride=Dn - 1)) == 2 and bwd(num_seqs=2) == 2 and bwd(state_size=257) == 2
    assert bwd(dict(dy_stride=(1 << 27) + 1)) == 2      # rows past 32-bit offsets of the kernels' cells
    assert bwd(dtype=7) == 3
    for g in (dict(du=1 << 20), dict(dA=3 << 20), dict(d_initial_state=16 << 20), dict(dB=36 << 20, dC=36 << 20),
              dict(dz=32 << 20), dict(d_initial_state=33 << 20)):
        assert bwd(g) == 7, g
    need = lib.kda_ssm_bwd_workspace_bytes(T, Dn, Ns, G)
    assert need > 0 and bwd(nbytes=need - 1) == 4
    assert bwd(dict(dz=None), z=None, nbytes=need - 1) == 4       # no gate, no gradient of one
    assert lib.kda_ssm_bwd_workspace_bytes(T, Dn, Ns, 5) == 0


# ---------------------------------------------------------------- outputs over parameters and offsets
@pytest.mark.parametrize("name,at,size", [("weight", 100 << 20, C * W * 4), ("bias", 101 << 20, C * 4), ("cu_seqlens", 102 << 20, 8)])
def test_conv_abi_refuses_outputs_over_parameters(lib, name, at, size):
    def grads(**over):
        g = dict(dy=110 << 20, d_final_state=None, dx=111 << 20, dweight=112 << 20, dbias=113 << 20, d_initial_state=None, dy_stride=C)
        g.update(over)
        return lib.kda_conv_bwd(ctypes.byref(conv_args(**{name: at})), ctypes.byref(native.KdaConvGrads(**g)), None, None, 0)

    for end in (at, at + size - 2):                                              # the first and the last of it
        assert lib.kda_conv_fwd(ctypes.byref(conv_args(**{name: at}, out=end)), None) == 7
        assert lib.kda_conv_fwd(ctypes.byref(conv_args(**{name: at}, final_state=end)), None) == 7
        if name != "cu_seqlens":
            for kw in (dict(out=end), dict(final_state=end)):
                assert lib.kda_conv_decode(ctypes.byref(conv_args(**{name: at}, num_seqs=T, **kw)), None) == 7
        for out in ("dx", "dweight", "dbias", "d_initial_state"):
            assert grads(**{out: end}) == 7, out


def test_ssm_abi_refuses_outputs_over_offsets(lib):
    at = 100 << 20
    for end in (at, at + 4):
        for kw in (dict(out=end), dict(final_state=end)):
            assert lib.kda_ssm_fwd(ctypes.byref(ssm_args(cu_seqlens=at, **kw)), None, None, 0) == 7, kw
        names = ("dy", "d_final_state", "du", "ddelta", "dB", "dC", "dz", "dA", "dD", "ddelta_bias", "d_initial_state")
        for out in names[2:]:
            g = {n: (32 + i) << 20 for i, n in enumerate(names)}
            g.update({out: end, "dy_stride": Dn})
            assert lib.kda_ssm_bwd(ctypes.byref(ssm_args(cu_seqlens=at)), ctypes.byref(native.KdaSsmGrads(**g)), None, None, 0) == 7, out


def test_only_the_scan_over_time_limits_strides(lib):
    far = (1 << 27) + 8
    spread = {n: (i + 1) << 45 for i, n in enumerate(("u", "delta", "B", "C", "z", "out"))}
    for name in ("u", "delta", "B", "C", "z"):
        kw = {f"{name}_stride": far, **spread}
        assert lib.kda_ssm_fwd(ctypes.byref(ssm_args(**kw)), None, None, 0) == 2, name
        kw["out"] = kw["u"]             # refused, but for the overlap: the stride has passed
        assert lib.kda_ssm_decode(ctypes.byref(ssm_args(num_seqs=T, **kw)), None) == 7, name


def test_attn_number_of_sequences(lib):
    size = lambda n: lib.kda_attn_workspace_bytes(n, 1, 1, 64, 64, 16)  # noqa: E731
    assert size(1 << 16) > 0 and size((1 << 16) + 1) == 0
    mb = 1 << 20
    a = dict(q=mb << 10, k_cache=mb << 20, v_cache=mb << 21, block_table=mb << 11, seq_lens=mb << 12, out=mb << 13, lse=None,
             q_stride=64, q_head_stride=64, k_page_stride=1024, k_token_stride=64, k_head_stride=64, v_page_stride=1024,
             v_token_stride=64, v_head_stride=64, table_stride=64, num_seqs=1 << 16, q_heads=1, kv_heads=1, head_dim=64,
             num_pages=10, page_size=16, table_width=64, dtype=1, scale=0.1)
    call = lambda: lib.kda_attn_decode(ctypes.byref(native.KdaAttnArgs(**a)), None, P, 0)  # noqa: E731
    assert call() == 4                      # the workspace is too small: the number has passed
    a["num_seqs"] += 1
    assert call() == 2


def test_a_stream_of_another_device_is_refused():
    """Its kernels would run beside what torch's allocator orders on the inputs' device."""
    from types import SimpleNamespace

    from chunked_gated_delta_kda_amd._args import launch_on
    with pytest.raises(ValueError, match="stream:"):
        with launch_on(0, SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)):
            pass
