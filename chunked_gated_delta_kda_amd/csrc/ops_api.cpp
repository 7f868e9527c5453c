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

// A workspace: the caller's, or one allocated stream-ordered and freed on the stream after the
// call's kernels.
class Workspace {
public:
    Workspace(void *given, size_t bytes, size_t need, hipStream_t st) : st_(st) {
        if (given) {
            rc_ = bytes < need ? KDA_ERR_ALLOC : KDA_OK;
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

}  // namespace

extern "C" {

int kda_conv_fwd(const kda_conv_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_conv_args &a = *args;
    if (const int rc = check_conv(a, false)) return rc;
    if (!a.cu_seqlens && a.num_seqs != 1) return KDA_ERR_SHAPE;
    const int64_t es = (int64_t)dtype_bytes(a.dtype);
    const Span x = span(a.x, rows_bytes(a.total_tokens, a.x_stride, a.channels, es));
    const Span out = span(a.out, (int64_t)a.total_tokens * a.channels * es);
    const int64_t state = (int64_t)a.num_seqs * (a.width - 1) * a.channels * es;
    const Span si = span(a.initial_state, state), sf = span(a.final_state, state);
    if (meet(x, out) || meet(si, sf) || meet(x, sf) || meet(si, out) || meet(out, sf)) return KDA_ERR_ALIAS;
    return launched(kda::ops::launch_conv_fwd(a, kda::device_error_word(), (hipStream_t)stream));
}

int kda_conv_decode(const kda_conv_args *args, void *stream) {
    if (!args) return KDA_ERR_NULL;
    const kda_conv_args &a = *args;
    if (const int rc = check_conv(a, false)) return rc;
    if (a.cu_seqlens || a.total_tokens != a.num_seqs) return KDA_ERR_SHAPE;
    const int64_t es = (int64_t)dtype_bytes(a.dtype);
    const Span x = span(a.x, rows_bytes(a.total_tokens, a.x_stride, a.channels, es));
    const Span out = span(a.out, (int64_t)a.total_tokens * a.channels * es);
    const int64_t state = (int64_t)a.num_seqs * (a.width - 1) * a.channels * es;
    const Span si = span(a.initial_state, state), sf = span(a.final_state, state);
    if (meet(x, out) || (a.initial_state != a.final_state && meet(si, sf)) || meet(x, sf) || meet(si, out) || meet(out, sf))
        return KDA_ERR_ALIAS;
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
    const int64_t es = (int64_t)dtype_bytes(a.dtype), C = a.channels, T = a.total_tokens;
    const int64_t state = (int64_t)a.num_seqs * (a.width - 1) * C;
    const Span in[] = {span(a.x, rows_bytes(T, a.x_stride, C, es)), span(g.dy, rows_bytes(T, g.dy_stride, C, es)),
                       span(a.weight, C * a.width * 4), span(a.initial_state, state * es), span(g.d_final_state, state * 4)};
    const Span out[] = {span(g.dx, T * C * es), span(g.dweight, C * a.width * 4), span(g.dbias, C * 4),
                        span(g.d_initial_state, state * 4)};
    for (const Span &o : out)
        for (const Span &i : in)
            if (meet(o, i)) return KDA_ERR_ALIAS;
    hipStream_t st = (hipStream_t)stream;
    Workspace ws(workspace, workspace_bytes, kda::ops::conv_bwd_workspace(T, C, a.width), st);
    if (ws.status() != KDA_OK) return ws.status();
    return ws.finish(launched(kda::ops::launch_conv_bwd(a, g, (float *)ws.ptr(), kda::device_error_word(), st)));
}

}  // extern "C"
