// ops_api.cpp -- the C ABI of the operators beside the delta rule (include/kda.h): argument
// validation, workspace, launches. No exception crosses the interface.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_launch.hpp"
#include "ops_launch.hpp"

namespace {

using kda::ops::dtype_bytes;

struct Span {
    const char *p;
    size_t n;
};

Span span(const void *p, int64_t bytes) { return {(const char *)p, p && bytes > 0 ? (size_t)bytes : 0}; }

bool meet(Span a, Span b) { return a.n && b.n && a.p < b.p + b.n && b.p < a.p + a.n; }

// bytes that `rows` rows of `len` elements, `stride` apart, lie in
int64_t rows_bytes(int64_t rows, int64_t stride, int64_t len, int64_t es) {
    return rows > 0 ? ((rows - 1) * stride + len) * es : 0;
}

bool dtype_ok(int dt) { return dt == KDA_DTYPE_F32 || dt == KDA_DTYPE_BF16 || dt == KDA_DTYPE_F16; }

// A workspace: the caller's (large enough, aligned to 16 bytes), or one allocated stream-ordered and freed on the stream after the
// call's kernels.
class Workspace {
public:
    Workspace(void *given, size_t bytes, size_t need, hipStream_t st) : st_(st) {
        if (given) {
            rc_ = bytes < need || (need && (uintptr_t)given % 16) ? KDA_ERR_ALLOC : KDA_OK;
            ptr_ = given;
        } else if (need) {
            if (hipMallocAsync(&ptr_, need, st) != hipSuccess) {
                (void)hipGetLastError();
                rc_ = KDA_ERR_ALLOC;
                ptr_ = nullptr;
            } else
                owned_ = true;
        }
    }
    int status() const { return rc_; }
    void *ptr() const { return ptr_; }
    int finish(int rc) {
        if (owned_ && hipFreeAsync(ptr_, st_) != hipSuccess && rc == KDA_OK) rc = KDA_ERR_DEVICE;
        owned_ = false;
        return rc;
    }

private:
    hipStream_t st_;
    void *ptr_ = nullptr;
    bool owned_ = false;
    int rc_ = KDA_OK;
};

int launched(hipError_t e) {
    if (e == hipSuccess) return KDA_OK;
    (void)hipGetLastError();
    return KDA_ERR_LAUNCH;
}

// ---------------------------------------------------------------- short convolution
int check_conv(const kda_conv_args &a, bool grads) {
    if (!dtype_ok(a.dtype) || a.width < 2 || a.width > KDA_CONV_MAX_WIDTH || (a.activation != 0 && a.activation != 1))
        return KDA_ERR_UNSUPPORTED;
    if (a.num_seqs < 1 || a.total_tokens < 0 || a.channels < 1) return KDA_ERR_SHAPE;
    if (a.total_tokens > 1 << 27 || a.channels > 1 << 20 || (int64_t)a.num_seqs * a.channels > (int64_t)1 << 31)
        return KDA_ERR_SHAPE;
    if (a.x_stride < a.channels) return KDA_ERR_SHAPE;
    if (!a.weight || (a.total_tokens > 0 && (!a.x || (!grads && !a.out)))) return KDA_ERR_NULL;
    return KDA_OK;
}

// the convolution's inputs, the initial state last
struct ConvSpans {
    Span in[5];
    int64_t state;      // elements
    explicit ConvSpans(const kda_conv_args &a) {
        const int64_t es = (int64_t)dtype_bytes(a.dtype), C = a.channels;
        state = (int64_t)a.num_seqs * (a.width - 1) * C;
        in[0] = span(a.x, rows_bytes(a.total_tokens, a.x_stride, C, es));
        in[1] = span(a.weight, C * a.width * 4);
        in[2] = span(a.bias, C * 4);
        in[3] = span(a.cu_seqlens, ((int64_t)a.num_seqs + 1) * 4);
        in[4] = span(a.initial_state, state * es);
    }
    bool over(Span out, int count = 5) const {
        for (int i = 0; i < count; ++i)
            if (meet(in[i], out)) return true;
        return false;
    }
};

// ---------------------------------------------------------------- selective scan
bool ssm_sizes_ok(int64_t T, int64_t D, int64_t N, int64_t G) {
    return T >= 0 && T <= 1 << 27 && D >= 1 && D <= 1 << 20 && N >= 1 && N <= KDA_SSM_MAX_STATE && G >= 1 && G <= D && D % G == 0;
}

// far: rows may lie further apart than KDA_SSM_MAX_STRIDE (the token kernel forms 64-bit offsets, those that walk the
// time axis 32-bit ones between a few rows)
int check_ssm(const kda_ssm_args &a, bool grads, bool far = false) {
    if (!dtype_ok(a.dtype) || (a.delta_softplus != 0 && a.delta_softplus != 1)) return KDA_ERR_UNSUPPORTED;
    if (!ssm_sizes_ok(a.total_tokens, a.channels, a.state_size, a.groups) || a.num_seqs < 1 ||
        (int64_t)a.num_seqs * a.channels > (int64_t)1 << 31)
        return KDA_ERR_SHAPE;
    const int64_t bc = (int64_t)a.groups * a.state_size;
    if (a.u_stride < a.channels || a.delta_stride < a.channels || a.B_stride < bc || a.C_stride < bc ||
        (a.z && a.z_stride < a.channels))
        return KDA_ERR_SHAPE;
    for (const int64_t s : {a.u_stride, a.delta_stride, a.B_stride, a.C_stride, a.z ? a.z_stride : 0})
        if (!far && s > KDA_SSM_MAX_STRIDE) return KDA_ERR_SHAPE;
    if (!a.A || (a.total_tokens > 0 && (!a.u || !a.delta || !a.B || !a.C || (!grads && !a.out)))) return KDA_ERR_NULL;
    return KDA_OK;
}

// a scan's inputs, the initial state last
struct SsmSpans {
    Span in[10];
    int64_t state;
    explicit SsmSpans(const kda_ssm_args &a) {
        const int64_t es = (int64_t)dtype_bytes(a.dtype), T = a.total_tokens, D = a.channels, N = a.state_size;
        state = (int64_t)a.num_seqs * D * N * 4;
        in[0] = span(a.u, rows_bytes(T, a.u_stride, D, es));
        in[1] = span(a.delta, rows_bytes(T, a.delta_stride, D, es));
        in[2] = span(a.B, rows_bytes(T, a.B_stride, a.groups * N, es));
        in[3] = span(a.C, rows_bytes(T, a.C_stride, a.groups * N, es));
        in[4] = span(a.z, rows_bytes(T, a.z_stride, D, es));
        in[5] = span(a.A, D * N * 4);
        in[6] = span(a.D, D * 4);
        in[7] = span(a.delta_bias, D * 4);
        in[8] = span(a.cu_seqlens, ((int64_t)a.num_seqs + 1) * 4);
        in[9] = span(a.initial_state, state);
    }
    bool over(Span out, int count = 10) const {
        for (int i = 0; i < count; ++i)
            if (meet(in[i], out)) return true;
        return false;
    }
};

// ---------------------------------------------------------------- paged token attention
// 0, or the status of sizes that the kernels do not take
int check_attn_sizes(int64_t B, int64_t hq, int64_t hkv, int64_t dh, int64_t width, int64_t page) {
    if (dh != 64 && dh != 128 && dh != 256) return KDA_ERR_UNSUPPORTED;
    if (B < 1 || hkv < 1 || hq < hkv || hq % hkv || hq > 65535 || width < 1 || page < 1 || width > (1 << 30) / page) return KDA_ERR_SHAPE;
    // Every block reads all lengths, so that time grows with the square of the sequences: 4.7 ms at 2^14 of one cache head
    // (measured), 0.1 s at 2^16 by that, minutes at 2^22.
    if (B > 1 << 16 || (B + 1) * hkv * ((hq / hkv + 15) / 16) > 1 << 22) return KDA_ERR_SHAPE;
    return KDA_OK;
}

bool by16(const void *p) { return (uintptr_t)p % 16 == 0; }

}  // namespace

extern "C" {

int kda_conv_fwd(const kda_conv_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_conv_args &a = *args;
    if (const int rc = check_conv(a, false)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    const ConvSpans s(a);
    const int64_t es = (int64_t)dtype_bytes(a.dtype);
    const Span out = span(a.out, (int64_t)a.total_tokens * a.channels * es), fin = span(a.final_state, s.state * es);
    if (s.over(out) || s.over(fin) || meet(out, fin)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_conv_fwd(a, kda::device_error_word(), (hipStream_t)stream));
}

int kda_conv_decode(const kda_conv_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_conv_args &a = *args;
    if (const int rc = check_conv(a, false)) return rc;
    if (a.cu_seqlens || a.total_tokens != a.num_seqs) return KDA_ERR_SHAPE;
    const ConvSpans s(a);
    const int64_t es = (int64_t)dtype_bytes(a.dtype);
    const Span out = span(a.out, (int64_t)a.total_tokens * a.channels * es), fin = span(a.final_state, s.state * es);
    const bool in_place = a.initial_state == a.final_state;
    if (s.over(out) || s.over(fin, in_place ? 4 : 5) || meet(out, fin)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_conv_decode(a, (hipStream_t)stream));
}

size_t kda_conv_bwd_workspace_bytes(int32_t total_tokens, int32_t channels, int32_t width) {
    if (total_tokens < 0 || total_tokens > 1 << 27 || channels < 1 || channels > 1 << 20 || width < 2 || width > KDA_CONV_MAX_WIDTH)
        return 0;
    return kda::ops::conv_bwd_workspace(total_tokens, channels, width);
}

int kda_conv_bwd(const kda_conv_args *args, const kda_conv_grads *grads, void *stream, void *workspace,
                 size_t workspace_bytes) {
    if (!args || !grads) return KDA_ERR_NULL;
    kda_conv_args a = *args;
    a.out = a.final_state = nullptr;
    const kda_conv_grads &g = *grads;
    if (const int rc = check_conv(a, true)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    if (g.dy_stride < a.channels) return KDA_ERR_SHAPE;
    if (!g.dweight || (a.total_tokens > 0 && (!g.dy || !g.dx))) return KDA_ERR_NULL;
    const ConvSpans s(a);
    const int64_t es = (int64_t)dtype_bytes(a.dtype), C = a.channels, T = a.total_tokens;
    const Span dy = span(g.dy, rows_bytes(T, g.dy_stride, C, es)), dfin = span(g.d_final_state, s.state * 4);
    const Span out[] = {span(g.dx, T * C * es), span(g.dweight, C * a.width * 4), span(g.dbias, C * 4),
                        span(g.d_initial_state, s.state * 4)};
    for (int o = 0; o < 4; ++o) {
        if (s.over(out[o]) || meet(dy, out[o]) || meet(dfin, out[o])) return KDA_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (meet(out[o], out[q])) return KDA_ERR_ALIAS;
    }
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes, kda::ops::conv_bwd_workspace(T, C, a.width), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_conv_bwd(a, g, (float *)ws.ptr(), kda::device_error_word(), st)));
}

size_t kda_ssm_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t channels, int32_t state_size,
                               int32_t groups) {
    if (num_seqs < 1 || !ssm_sizes_ok(total_tokens, channels, state_size, groups)) return 0;
    return kda::ops::ssm_workspace(total_tokens, channels, state_size, groups, num_seqs);
}

int kda_ssm_fwd(const kda_ssm_args *args, void *stream, void *workspace, size_t workspace_bytes) {
    if (!args) return KDA_ERR_NULL;
    const kda_ssm_args &a = *args;
    if (const int rc = check_ssm(a, false)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    const SsmSpans s(a);
    const Span out = span(a.out, (int64_t)a.total_tokens * a.channels * (int64_t)dtype_bytes(a.dtype));
    const Span fin = span(a.final_state, s.state);
    if (s.over(out) || s.over(fin) || meet(out, fin)) return KDA_ERR_ALIAS;
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes, kda::ops::ssm_workspace(a.total_tokens, a.channels, a.state_size, a.groups, a.num_seqs), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_ssm_fwd(a, (float *)ws.ptr(), kda::device_error_word(), st)));
}

int kda_ssm_decode(const kda_ssm_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_ssm_args &a = *args;
    if (const int rc = check_ssm(a, false, true)) return rc;
    if (a.cu_seqlens || a.total_tokens != a.num_seqs) return KDA_ERR_SHAPE;
    const SsmSpans s(a);
    const Span out = span(a.out, (int64_t)a.total_tokens * a.channels * (int64_t)dtype_bytes(a.dtype));
    const Span fin = span(a.final_state, s.state);
    const bool in_place = a.initial_state == a.final_state;
    if (s.over(out) || s.over(fin, in_place ? 9 : 10) || meet(out, fin)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_ssm_decode(a, (hipStream_t)stream));
}

size_t kda_ssm_bwd_workspace_bytes(int32_t total_tokens, int32_t channels, int32_t state_size, int32_t groups) {
    if (!ssm_sizes_ok(total_tokens, channels, state_size, groups)) return 0;
    return kda::ops::ssm_bwd_workspace(total_tokens, channels, state_size, groups);
}

int kda_ssm_bwd(const kda_ssm_args *args, const kda_ssm_grads *grads, void *stream, void *workspace,
                size_t workspace_bytes) {
    if (!args || !grads) return KDA_ERR_NULL;
    kda_ssm_args a = *args;
    a.out = nullptr, a.final_state = nullptr;
    const kda_ssm_grads &g = *grads;
    if (const int rc = check_ssm(a, true)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    if (g.dy_stride < a.channels || g.dy_stride > KDA_SSM_MAX_STRIDE) return KDA_ERR_SHAPE;
    if (!g.dA || (a.total_tokens > 0 && (!g.dy || !g.du || !g.ddelta || !g.dB || !g.dC || (a.z && !g.dz)))) return KDA_ERR_NULL;
    const SsmSpans s(a);
    const int64_t es = (int64_t)dtype_bytes(a.dtype), T = a.total_tokens, D = a.channels, N = a.state_size;
    const Span dy = span(g.dy, rows_bytes(T, g.dy_stride, D, es)), dfin = span(g.d_final_state, s.state);
    const Span out[] = {span(g.du, T * D * es), span(g.ddelta, T * D * es), span(g.dB, T * a.groups * N * es),
                        span(g.dC, T * a.groups * N * es), span(a.z ? g.dz : nullptr, T * D * es), span(g.dA, D * N * 4),
                        span(g.dD, D * 4), span(g.ddelta_bias, D * 4), span(g.d_initial_state, s.state)};
    constexpr int outs = sizeof(out) / sizeof(out[0]);
    for (int i = 0; i < outs; ++i) {
        if (s.over(out[i]) || meet(dy, out[i]) || meet(dfin, out[i])) return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes, kda::ops::ssm_bwd_workspace(T, D, N, a.groups), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_ssm_bwd(a, g, (float *)ws.ptr(), kda::device_error_word(), st)));
}

size_t kda_attn_workspace_bytes(int32_t num_seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                int32_t table_width, int32_t page_size) {
    if (check_attn_sizes(num_seqs, q_heads, kv_heads, head_dim, table_width, page_size) != KDA_OK) return 0;
    return kda::ops::attn_workspace(num_seqs, q_heads, kv_heads, head_dim, table_width, page_size);
}

int kda_attn_decode(const kda_attn_args *args, void *stream, void *workspace, size_t workspace_bytes) {
    if (!args) return KDA_ERR_NULL;
    const kda_attn_args &a = *args;
    if (a.dtype != KDA_DTYPE_BF16 && a.dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
    if (!std::isfinite(a.scale)) return KDA_ERR_UNSUPPORTED;
    if (const int rc = check_attn_sizes(a.num_seqs, a.q_heads, a.kv_heads, a.head_dim, a.table_width, a.page_size)) return rc;
    if (a.num_pages < 1 || a.table_stride < 0 || (a.num_seqs > 1 && a.table_stride < a.table_width)) return KDA_ERR_SHAPE;
    const int64_t strides[] = {a.q_stride, a.q_head_stride, a.k_page_stride, a.k_token_stride,
                               a.k_head_stride, a.v_page_stride, a.v_token_stride, a.v_head_stride};
    for (const int64_t s : strides)
        if (s < 0) return KDA_ERR_SHAPE;
    for (const int64_t s : strides)
        if (s % 8) return KDA_ERR_UNSUPPORTED;
    if (!a.q || !a.k_cache || !a.v_cache || !a.block_table || !a.seq_lens || !a.out) return KDA_ERR_NULL;
    if (!by16(a.q) || !by16(a.k_cache) || !by16(a.v_cache)) return KDA_ERR_UNSUPPORTED;
    const int64_t es = 2, B = a.num_seqs;
    auto cache = [&](const void *p, int64_t page, int64_t token, int64_t head) {
        return span(p, ((a.num_pages - 1) * page + (a.page_size - 1) * token + (a.kv_heads - 1) * head + a.head_dim) * es);
    };
    const Span in[] = {span(a.q, ((B - 1) * a.q_stride + (a.q_heads - 1) * a.q_head_stride + a.head_dim) * es),
                       cache(a.k_cache, a.k_page_stride, a.k_token_stride, a.k_head_stride),
                       cache(a.v_cache, a.v_page_stride, a.v_token_stride, a.v_head_stride),
                       span(a.block_table, ((B - 1) * a.table_stride + a.table_width) * 4), span(a.seq_lens, B * 4)};
    const Span out = span(a.out, B * a.q_heads * a.head_dim * es), lse = span(a.lse, B * a.q_heads * 4);
    if (meet(out, lse)) return KDA_ERR_ALIAS;
    for (const Span &i : in)
        if (meet(i, out) || meet(i, lse)) return KDA_ERR_ALIAS;
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes,
                 kda::ops::attn_workspace(B, a.q_heads, a.kv_heads, a.head_dim, a.table_width, a.page_size), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_attn_decode(a, (float *)ws.ptr(), kda::device_error_word(), st)));
}

}  // extern "C"
