// ops_api.cpp -- the C ABI of the operators beside the delta rule (include/kda.h): argument
// validation, workspace, launches. No exception crosses the interface.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <utility>

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

// the bytes that a paged cache lies in: rows of `row` elements of `es` bytes
Span cache_span(const void *p, int64_t pages, int64_t page_size, int64_t heads, int64_t page, int64_t token, int64_t head, int64_t row,
                int64_t es) {
    return span(p, ((pages - 1) * page + (page_size - 1) * token + (heads - 1) * head + row) * es);
}

// what both token attentions check of their arguments; strides of the caches are multiples of `unit`
int check_attn(const kda_attn_args &a, int64_t unit) {
    if (a.dtype != KDA_DTYPE_BF16 && a.dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
    if (!std::isfinite(a.scale)) return KDA_ERR_UNSUPPORTED;
    if (const int rc = check_attn_sizes(a.num_seqs, a.q_heads, a.kv_heads, a.head_dim, a.table_width, a.page_size)) return rc;
    if (a.num_pages < 1 || a.table_stride < 0 || (a.num_seqs > 1 && a.table_stride < a.table_width)) return KDA_ERR_SHAPE;
    const int64_t strides[] = {a.q_stride, a.q_head_stride, a.k_page_stride, a.k_token_stride,
                               a.k_head_stride, a.v_page_stride, a.v_token_stride, a.v_head_stride};
    for (const int64_t s : strides)
        if (s < 0) return KDA_ERR_SHAPE;
    for (int i = 0; i < 8; ++i)
        if (strides[i] % (i < 2 ? 8 : unit)) return KDA_ERR_UNSUPPORTED;
    if (!a.q || !a.k_cache || !a.v_cache || !a.block_table || !a.seq_lens || !a.out) return KDA_ERR_NULL;
    if (!by16(a.q) || !by16(a.k_cache) || !by16(a.v_cache)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// whether an output of a token attention lies over an input or the other output
bool attn_over(const kda_attn_args &a, const Span *caches, int count) {
    const int64_t es = 2, B = a.num_seqs;
    const Span in[] = {span(a.q, ((B - 1) * a.q_stride + (a.q_heads - 1) * a.q_head_stride + a.head_dim) * es),
                       span(a.block_table, ((B - 1) * a.table_stride + a.table_width) * 4), span(a.seq_lens, B * 4)};
    const Span out = span(a.out, B * a.q_heads * a.head_dim * es), lse = span(a.lse, B * a.q_heads * 4);
    if (meet(out, lse)) return true;
    for (const Span &i : in)
        if (meet(i, out) || meet(i, lse)) return true;
    for (int i = 0; i < count; ++i)
        if (meet(caches[i], out) || meet(caches[i], lse)) return true;
    return false;
}

size_t attn_need(const kda_attn_args &a) {
    return kda::ops::attn_workspace(a.num_seqs, a.q_heads, a.kv_heads, a.head_dim, a.table_width, a.page_size);
}

// ---------------------------------------------------------------- paged cache
struct Scales {     // of a cache, or its codes
    const uint8_t *p;
    int64_t page, token, head;
};

int check_cache_sizes(int64_t seqs, int64_t tokens, int64_t heads, int64_t dh, int64_t pages, int64_t page, int64_t width, int64_t table_stride) {
    if (dh != 64 && dh != 128 && dh != 256) return KDA_ERR_UNSUPPORTED;
    if (seqs < 1 || tokens < 0 || tokens > 1 << 27 || heads < 1 || heads > 65535 || pages < 1 || page < 1 || width < 1 ||
        width > (1 << 30) / page || table_stride < 0 || (seqs > 1 && table_stride < width))
        return KDA_ERR_SHAPE;
    return KDA_OK;
}

// rows read and written 16 bytes at a time
int check_rows(const Scales &c, int64_t unit) {
    if (c.page < 0 || c.token < 0 || c.head < 0) return KDA_ERR_SHAPE;
    if (c.page % unit || c.token % unit || c.head % unit || !by16(c.p)) return KDA_ERR_UNSUPPORTED;
    return c.p ? KDA_OK : KDA_ERR_NULL;
}

// scales: rows of `sb` bytes, read at once
int check_scales(const Scales &s, int64_t sb) {
    if (s.page < 0 || s.token < 0 || s.head < 0) return KDA_ERR_SHAPE;
    if (s.page % sb || s.token % sb || s.head % sb || (uintptr_t)s.p % sb) return KDA_ERR_UNSUPPORTED;
    return s.p ? KDA_OK : KDA_ERR_NULL;
}

// The rows of a cache, in bytes: its dimensions of more than one entry, by falling stride, and what a dimension's entries (at the end
// a row) span.
struct Layout {
    const char *p;
    int dims = 0;
    int64_t size[3], stride[3], span[4];
    Layout(const Scales &c, int64_t pages, int64_t page_size, int64_t heads, int64_t row, int64_t es) : p((const char *)c.p) {
        const int64_t n[] = {pages, page_size, heads}, s[] = {c.page, c.token, c.head};
        for (int i = 0; i < 3; ++i) {
            if (n[i] == 1) continue;
            int at = dims++;
            for (; at > 0 && stride[at - 1] < s[i] * es; --at) size[at] = size[at - 1], stride[at] = stride[at - 1];
            size[at] = n[i], stride[at] = s[i] * es;
        }
        span[dims] = row * es;
        for (int i = dims - 1; i >= 0; --i) span[i] = span[i + 1] + (size[i] - 1) * stride[i];
    }
    // whether no two of its rows share a byte: each stride steps over what the smaller ones span
    bool apart() const {
        for (int i = 0; i < dims; ++i)
            if (stride[i] < span[i + 1]) return false;
        return true;
    }
    // Whether rows of two layouts with rows apart may share a byte, b's part from dimension `d` on lying `off` bytes behind this one's. Where
    // their parts meet and their strides are the same, the few entries' distances that keep them together decide; where
    // strides differ, they are taken to share.
    bool shares(const Layout &b, int64_t off, int d = 0) const {
        if (off >= span[d] || -off >= b.span[d]) return false;
        if (d == dims) return true;
        if (stride[d] != b.stride[d]) return true;
        const int64_t near = -off / stride[d];
        for (int64_t i = near - 2; i <= near + 2; ++i)      // entry of b less entry of this one
            if (i > -size[d] && i < b.size[d] && shares(b, off + i * stride[d], d + 1)) return true;
        return false;
    }
};

// ---------------------------------------------------------------- linear attention
bool lin_dim(int64_t d) { return d == 64 || d == 128; }

bool lin_sizes_ok(int64_t S, int64_t T, int64_t H) {
    return S >= 1 && T >= 0 && T <= 1 << 27 && H >= 1 && H <= 65535 && S * H <= 1 << 27;
}

// far: rows may lie further apart than KDA_LIN_MAX_STRIDE (a token alone)
int check_lin(const kda_lin_args &a, bool grads, bool far = false) {
    if ((a.dtype != KDA_DTYPE_BF16 && a.dtype != KDA_DTYPE_F16) || !lin_dim(a.key_dim) || !lin_dim(a.value_dim) ||
        (a.g_per_head != 0 && a.g_per_head != 1) || !std::isfinite(a.scale))
        return KDA_ERR_UNSUPPORTED;
    if (!lin_sizes_ok(a.num_seqs, a.total_tokens, a.heads)) return KDA_ERR_SHAPE;
    const int64_t strides[] = {a.q_stride, a.q_head_stride, a.k_stride, a.k_head_stride, a.v_stride, a.v_head_stride};
    for (const int64_t s : strides)
        if (s < 0) return KDA_ERR_SHAPE;
    for (const int64_t s : strides)
        if (s % 8) return KDA_ERR_UNSUPPORTED;
    for (const int64_t s : {a.q_stride, a.k_stride, a.v_stride})
        if (!far && s > KDA_LIN_MAX_STRIDE) return KDA_ERR_SHAPE;
    if (a.total_tokens > 0 && (!a.q || !a.k || !a.v || !a.g || (!grads && !a.out))) return KDA_ERR_NULL;
    if (!by16(a.q) || !by16(a.k) || !by16(a.v) || !by16(a.initial_state) || !by16(a.final_state) || !by16(a.out)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// its inputs, the initial state last
struct LinSpans {
    Span in[6];
    int64_t state;      // bytes
    static Span rows3(const void *p, int64_t T, int64_t stride, int64_t H, int64_t head, int64_t D) {
        return span(T > 0 ? p : nullptr, ((T - 1) * stride + (H - 1) * head + D) * 2);
    }
    explicit LinSpans(const kda_lin_args &a) {
        const int64_t T = a.total_tokens, H = a.heads;
        state = (int64_t)a.num_seqs * H * a.key_dim * a.value_dim * 4;
        in[0] = rows3(a.q, T, a.q_stride, H, a.q_head_stride, a.key_dim);
        in[1] = rows3(a.k, T, a.k_stride, H, a.k_head_stride, a.key_dim);
        in[2] = rows3(a.v, T, a.v_stride, H, a.v_head_stride, a.value_dim);
        in[3] = span(a.g, (a.g_per_head ? H : T * H) * 4);
        in[4] = span(a.cu_seqlens, ((int64_t)a.num_seqs + 1) * 4);
        in[5] = span(a.initial_state, state);
    }
    bool over(Span out, int count = 6) const {
        for (int i = 0; i < count; ++i)
            if (meet(in[i], out)) return true;
        return false;
    }
};

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
    if (const int rc = check_attn(a, 8)) return rc;
    auto cache = [&](const void *p, int64_t page, int64_t token, int64_t head) {
        return cache_span(p, a.num_pages, a.page_size, a.kv_heads, page, token, head, a.head_dim, 2);
    };
    const Span in[] = {cache(a.k_cache, a.k_page_stride, a.k_token_stride, a.k_head_stride),
                       cache(a.v_cache, a.v_page_stride, a.v_token_stride, a.v_head_stride)};
    if (attn_over(a, in, 2)) return KDA_ERR_ALIAS;
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes, attn_need(a), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_attn_decode(a, (float *)ws.ptr(), kda::device_error_word(), st)));
}

size_t kda_attn_fp4_workspace_bytes(int32_t num_seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                                    int32_t page_size) {
    if (check_attn_sizes(num_seqs, q_heads, kv_heads, head_dim, table_width, page_size) != KDA_OK) return 0;
    return kda::ops::attn_fp4_workspace(num_seqs, q_heads, kv_heads, head_dim, table_width, page_size);
}

int kda_attn_decode_fp4(const kda_attn_fp4_args *args, void *stream, void *workspace, size_t workspace_bytes) {
    if (!args) return KDA_ERR_NULL;
    const kda_attn_fp4_args &f = *args;
    const kda_attn_args &a = f.attn;
    if (const int rc = check_attn(a, 16)) return rc;
    for (const int64_t s : {a.k_page_stride, a.k_token_stride, a.v_page_stride, a.v_token_stride, f.k_scale_page_stride,
                            f.k_scale_token_stride, f.v_scale_page_stride, f.v_scale_token_stride})
        if (s > UINT32_MAX) return KDA_ERR_SHAPE;
    const int64_t sb = a.head_dim / KDA_FP4_GROUP;
    const Scales sc[] = {{f.k_scale, f.k_scale_page_stride, f.k_scale_token_stride, f.k_scale_head_stride},
                         {f.v_scale, f.v_scale_page_stride, f.v_scale_token_stride, f.v_scale_head_stride}};
    for (const Scales &s : sc)
        if (const int rc = check_scales(s, sb)) return rc;
    auto cache = [&](const void *p, int64_t page, int64_t token, int64_t head, int64_t row) {
        return cache_span(p, a.num_pages, a.page_size, a.kv_heads, page, token, head, row, 1);
    };
    const Span in[] = {cache(a.k_cache, a.k_page_stride, a.k_token_stride, a.k_head_stride, a.head_dim / 2),
                       cache(a.v_cache, a.v_page_stride, a.v_token_stride, a.v_head_stride, a.head_dim / 2),
                       cache(sc[0].p, sc[0].page, sc[0].token, sc[0].head, sb), cache(sc[1].p, sc[1].page, sc[1].token, sc[1].head, sb)};
    if (attn_over(a, in, 4)) return KDA_ERR_ALIAS;
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes,
                 kda::ops::attn_fp4_workspace(a.num_seqs, a.q_heads, a.kv_heads, a.head_dim, a.table_width, a.page_size), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_attn_decode_fp4(f, (float *)ws.ptr(), kda::device_error_word(), st)));
}

int kda_kv_append(const kda_kv_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_kv_args &a = *args;
    if (a.dtype != KDA_DTYPE_BF16 && a.dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
    if (a.interleaved != 0 && a.interleaved != 1) return KDA_ERR_UNSUPPORTED;
    if (const int rc = check_cache_sizes(a.num_seqs, a.total_tokens, a.kv_heads, a.head_dim, a.num_pages, a.page_size, a.table_width,
                                         a.table_stride)) return rc;
    if (a.rope && (a.rot_dim % 16 || a.rot_dim < 16 || a.rot_dim > a.head_dim)) return KDA_ERR_UNSUPPORTED;
    if (a.q_heads < 0 || a.q_heads > 65535 || (a.q && a.q_heads < 1) || (!a.q && a.q_heads && a.total_tokens > 0) || (a.rope && a.max_positions < 1) ||
        (!a.cu_seqlens && a.total_tokens != a.num_seqs))
        return KDA_ERR_SHAPE;
    const bool four = a.k_scale || a.v_scale;
    const int64_t sb = a.head_dim / KDA_FP4_GROUP, row = four ? a.head_dim / 2 : a.head_dim, unit = four ? 16 : 8;
    const int64_t in_strides[] = {a.k_stride, a.k_head_stride, a.v_stride, a.v_head_stride, a.q ? a.q_stride : 0, a.q ? a.q_head_stride : 0};
    for (const int64_t s : in_strides)
        if (s < 0) return KDA_ERR_SHAPE;
    for (const int64_t s : in_strides)
        if (s % 8) return KDA_ERR_UNSUPPORTED;
    const Scales caches[] = {{(const uint8_t *)a.k_cache, a.k_page_stride, a.k_token_stride, a.k_cache_head_stride},
                             {(const uint8_t *)a.v_cache, a.v_page_stride, a.v_token_stride, a.v_cache_head_stride}};
    const Scales sc[] = {{a.k_scale, a.k_scale_page_stride, a.k_scale_token_stride, a.k_scale_head_stride},
                         {a.v_scale, a.v_scale_page_stride, a.v_scale_token_stride, a.v_scale_head_stride}};
    for (const Scales &c : caches)
        if (const int rc = check_rows(c, unit)) return rc;
    if (four)
        for (const Scales &s : sc)
            if (const int rc = check_scales(s, sb)) return rc;
    if (!a.block_table || !a.seq_lens || (a.total_tokens > 0 && (!a.k || !a.v || (a.q && !a.q_out)))) return KDA_ERR_NULL;
    if (!by16(a.k) || !by16(a.v) || !by16(a.q) || !by16(a.q_out) || !by16(a.rope)) return KDA_ERR_UNSUPPORTED;
    const int64_t ces = four ? 1 : 2;
    const Layout written[] = {{caches[0], a.num_pages, a.page_size, a.kv_heads, row, ces}, {caches[1], a.num_pages, a.page_size, a.kv_heads, row, ces},
                              {sc[0], a.num_pages, a.page_size, a.kv_heads, sb, 1}, {sc[1], a.num_pages, a.page_size, a.kv_heads, sb, 1}};
    const int buffers = four ? 4 : 2;
    for (int i = 0; i < buffers; ++i)
        if (!written[i].apart()) return KDA_ERR_SHAPE;
    const int64_t T = a.total_tokens, es = 2;
    auto rows3 = [&](const void *p, int64_t stride, int64_t head, int64_t heads) {
        return span(T > 0 ? p : nullptr, ((T - 1) * stride + (heads - 1) * head + a.head_dim) * es);
    };
    const Span in[] = {rows3(a.k, a.k_stride, a.k_head_stride, a.kv_heads), rows3(a.v, a.v_stride, a.v_head_stride, a.kv_heads),
                       rows3(a.q, a.q_stride, a.q_head_stride, a.q_heads), span(a.rope, (int64_t)a.max_positions * a.rot_dim * 4),
                       span(a.cu_seqlens, ((int64_t)a.num_seqs + 1) * 4),
                       span(a.block_table, (((int64_t)a.num_seqs - 1) * a.table_stride + a.table_width) * 4), span(a.seq_lens, (int64_t)a.num_seqs * 4)};
    const Span out[] = {span(a.q_out, T * a.q_heads * a.head_dim * es),
                        cache_span(caches[0].p, a.num_pages, a.page_size, a.kv_heads, caches[0].page, caches[0].token, caches[0].head, row, four ? 1 : 2),
                        cache_span(caches[1].p, a.num_pages, a.page_size, a.kv_heads, caches[1].page, caches[1].token, caches[1].head, row, four ? 1 : 2),
                        cache_span(sc[0].p, a.num_pages, a.page_size, a.kv_heads, sc[0].page, sc[0].token, sc[0].head, sb, 1),
                        cache_span(sc[1].p, a.num_pages, a.page_size, a.kv_heads, sc[1].page, sc[1].token, sc[1].head, sb, 1)};
    for (const Span &o : out)
        for (const Span &i : in)
            if (meet(i, o)) return KDA_ERR_ALIAS;
    for (int i = 1; i < 5; ++i)
        if (meet(out[0], out[i])) return KDA_ERR_ALIAS;
    // (caches that are slices of one tensor interleave: their spans may meet, their rows may not)
    for (int i = 0; i < buffers; ++i)
        for (int j = 0; j < i; ++j)
            if (written[j].shares(written[i], written[i].p - written[j].p)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_kv_append(a, kda::device_error_word(), (hipStream_t)stream));
}

int kda_kv_read_fp4(const kda_kv_read_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_kv_read_args &a = *args;
    if (a.dtype != KDA_DTYPE_BF16 && a.dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
    if (const int rc = check_cache_sizes(a.num_seqs, a.total_tokens, a.kv_heads, a.head_dim, a.num_pages, a.page_size, a.table_width,
                                         a.table_stride)) return rc;
    const Scales caches[] = {{(const uint8_t *)a.k_cache, a.k_page_stride, a.k_token_stride, a.k_head_stride},
                             {(const uint8_t *)a.v_cache, a.v_page_stride, a.v_token_stride, a.v_head_stride}};
    const Scales sc[] = {{a.k_scale, a.k_scale_page_stride, a.k_scale_token_stride, a.k_scale_head_stride},
                         {a.v_scale, a.v_scale_page_stride, a.v_scale_token_stride, a.v_scale_head_stride}};
    const int64_t sb = a.head_dim / KDA_FP4_GROUP;
    for (const Scales &c : caches)
        if (const int rc = check_rows(c, 16)) return rc;
    for (const Scales &s : sc)
        if (const int rc = check_scales(s, sb)) return rc;
    if (!a.block_table || !a.cu_seqlens || (a.total_tokens > 0 && (!a.k || !a.v))) return KDA_ERR_NULL;
    if (!by16(a.k) || !by16(a.v)) return KDA_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)a.total_tokens * a.kv_heads * a.head_dim * 2;
    const Span out[] = {span(a.k, rows), span(a.v, rows)};
    const Span in[] = {span(a.block_table, (((int64_t)a.num_seqs - 1) * a.table_stride + a.table_width) * 4),
                       span(a.cu_seqlens, ((int64_t)a.num_seqs + 1) * 4),
                       cache_span(caches[0].p, a.num_pages, a.page_size, a.kv_heads, caches[0].page, caches[0].token, caches[0].head, a.head_dim / 2, 1),
                       cache_span(caches[1].p, a.num_pages, a.page_size, a.kv_heads, caches[1].page, caches[1].token, caches[1].head, a.head_dim / 2, 1),
                       cache_span(sc[0].p, a.num_pages, a.page_size, a.kv_heads, sc[0].page, sc[0].token, sc[0].head, sb, 1),
                       cache_span(sc[1].p, a.num_pages, a.page_size, a.kv_heads, sc[1].page, sc[1].token, sc[1].head, sb, 1)};
    if (meet(out[0], out[1])) return KDA_ERR_ALIAS;
    for (const Span &o : out)
        for (const Span &i : in)
            if (meet(i, o)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_kv_read_fp4(a, kda::device_error_word(), (hipStream_t)stream));
}

size_t kda_lin_workspace_bytes(int32_t total_tokens, int32_t heads, int32_t key_dim, int32_t value_dim) {
    if (!lin_sizes_ok(1, total_tokens, heads) || !lin_dim(key_dim) || !lin_dim(value_dim)) return 0;
    return kda::ops::lin_workspace(total_tokens, heads, key_dim, value_dim);
}

int kda_lin_fwd(const kda_lin_args *args, void *stream, void *workspace, size_t workspace_bytes) {
    if (!args) return KDA_ERR_NULL;
    const kda_lin_args &a = *args;
    if (const int rc = check_lin(a, false)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    const LinSpans s(a);
    const Span out = span(a.out, (int64_t)a.total_tokens * a.heads * a.value_dim * 2), fin = span(a.final_state, s.state);
    if (s.over(out) || s.over(fin) || meet(out, fin)) return KDA_ERR_ALIAS;
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes, kda::ops::lin_workspace(a.total_tokens, a.heads, a.key_dim, a.value_dim), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_lin_fwd(a, (float *)ws.ptr(), kda::device_error_word(), st)));
}

int kda_lin_decode(const kda_lin_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_lin_args &a = *args;
    if (const int rc = check_lin(a, false, true)) return rc;
    if (a.cu_seqlens || a.total_tokens != a.num_seqs) return KDA_ERR_SHAPE;
    const LinSpans s(a);
    const Span out = span(a.out, (int64_t)a.total_tokens * a.heads * a.value_dim * 2), fin = span(a.final_state, s.state);
    const bool in_place = a.initial_state == a.final_state;
    if (s.over(out) || s.over(fin, in_place ? 5 : 6) || meet(out, fin)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_lin_decode(a, (hipStream_t)stream));
}

size_t kda_lin_bwd_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t heads, int32_t key_dim, int32_t value_dim,
                                   int32_t g_per_head, int32_t need_d_initial_state) {
    if (!lin_sizes_ok(num_seqs, total_tokens, heads) || !lin_dim(key_dim) || !lin_dim(value_dim)) return 0;
    return kda::ops::lin_bwd_workspace(total_tokens, heads, num_seqs, key_dim, value_dim, g_per_head != 0, need_d_initial_state == 0);
}

int kda_lin_bwd(const kda_lin_args *args, const kda_lin_grads *grads, void *stream, void *workspace, size_t workspace_bytes) {
    if (!args || !grads) return KDA_ERR_NULL;
    kda_lin_args a = *args;
    a.out = nullptr, a.final_state = nullptr;
    const kda_lin_grads &g = *grads;
    if (const int rc = check_lin(a, true)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    if (g.d_out_stride < 0 || g.d_out_head_stride < 0 || g.d_out_stride > KDA_LIN_MAX_STRIDE) return KDA_ERR_SHAPE;
    if (g.d_out_stride % 8 || g.d_out_head_stride % 8 || !by16(g.d_out) || !by16(g.d_final_state) || !by16(g.dq) || !by16(g.dk) ||
        !by16(g.dv) || !by16(g.d_initial_state))
        return KDA_ERR_UNSUPPORTED;
    const int64_t T = a.total_tokens, H = a.heads;
    if ((a.g_per_head && !g.dg) || (T > 0 && (!g.d_out || !g.dq || !g.dk || !g.dv || !g.dg))) return KDA_ERR_NULL;
    const LinSpans s(a);
    const Span dout = LinSpans::rows3(g.d_out, T, g.d_out_stride, H, g.d_out_head_stride, a.value_dim), dfin = span(g.d_final_state, s.state);
    const Span out[] = {span(g.dq, T * H * a.key_dim * 2), span(g.dk, T * H * a.key_dim * 2), span(g.dv, T * H * a.value_dim * 2),
                        span(g.dg, (a.g_per_head ? H : T * H) * 4), span(g.d_initial_state, s.state)};
    constexpr int outs = sizeof(out) / sizeof(out[0]);
    for (int i = 0; i < outs; ++i) {
        if (s.over(out[i]) || meet(dout, out[i]) || meet(dfin, out[i])) return KDA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes,
                 kda::ops::lin_bwd_workspace(T, H, a.num_seqs, a.key_dim, a.value_dim, a.g_per_head != 0, a.initial_state && !g.d_initial_state), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_lin_bwd(a, g, (float *)ws.ptr(), kda::device_error_word(), st)));
}

}  // extern "C"
