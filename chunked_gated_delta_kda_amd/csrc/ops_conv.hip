// ops_conv.hip -- the short causal convolution in front of a recurrence, over a packed batch.
//
// Per channel c, with taps w[c][0..W-1] and the sequence's rows x_s (rows s < 0 are its initial
// state, or zero):
//
//   p_t = b[c] + sum_j w[c][j] x_{t-W+1+j},   y_t = p_t sigmoid(p_t)  (or p_t)
//   backward: e_t = dy_t y'(p_t),   dx_s = sum_j w[c][j] e_{s+W-1-j} (+ the final state's gradient
//   at the last W-1 rows),   dw[c][j] = sum_t e_t x_{t-W+1+j},   db = sum_t e_t
//
// A thread owns VEC neighbouring channels and walks one tile of consecutive packed rows with the
// last W-1 rows in registers, so a row is read once (and W-1 rows again at a tile's start). The
// tile is uniform over the block; the sequences that start or end in it are found from the
// offsets by a search at the tile's start, so no map of the batch is built beforehand.
#include <type_traits>

#include "ops_common.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace {

template <int DT, int VEC> struct Vec {
    using E = typename Elem<DT>::type;
    typedef E type __attribute__((ext_vector_type(VEC)));
};
template <int DT> struct Vec<DT, 1> {
    using E = typename Elem<DT>::type;
    using type = E;
};

template <int DT, int VEC>
__device__ __forceinline__ typename Vec<DT, VEC>::type load_raw(const void *base, int64_t off) {
    return *reinterpret_cast<const typename Vec<DT, VEC>::type *>(reinterpret_cast<const typename Elem<DT>::type *>(base) + off);
}
template <int DT, int VEC>
__device__ __forceinline__ void to_float(const typename Vec<DT, VEC>::type &v, float *out) {
    if constexpr (VEC == 1) out[0] = (float)v;
    else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[i] = (float)v[i];
    }
}
template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const void *base, int64_t off, float *out) {
    to_float<DT, VEC>(load_raw<DT, VEC>(base, off), out);
}

template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void *base, int64_t off, const float *x) {
    using E = typename Elem<DT>::type;
    using V = typename Vec<DT, VEC>::type;
    V v;
    if constexpr (VEC == 1) v = (E)x[0];
    else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = (E)x[i];
    }
    *reinterpret_cast<V *>(reinterpret_cast<E *>(base) + off) = v;
}

// The taps of VEC channels, fp32 [C][W]: contiguous, four at a time where VEC W is a multiple of four (the
// weight is then aligned to 16 bytes).
template <int W, int VEC>
__device__ __forceinline__ void load_taps(const float *w, const float *b, int c, float (&tap)[W][VEC], float (&bias)[VEC]) {
    float flat[VEC * W];
    const float *from = w + (int64_t)c * W;
    if constexpr (VEC > 1 && VEC * W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC * W; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(from + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) flat[i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC * W; ++i) flat[i] = from[i];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        bias[i] = b ? b[c + i] : 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) tap[j][i] = flat[i * W + j];
    }
}

// Row t of a sequence that starts at `start`: of x, or of its initial state (rows before it).
template <int DT, int W, int VEC>
__device__ __forceinline__ void load_row(const kda_conv_args &a, int n, int start, int t, int c, float *out) {
    if (t >= start) load_vec<DT, VEC>(a.x, (int64_t)t * a.x_stride + c, out);
    else if (a.initial_state)
        load_vec<DT, VEC>(a.initial_state, ((int64_t)n * (W - 1) + (t - start + W - 1)) * a.channels + c, out);
    else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[i] = 0.0f;
    }
}

// The final state of sequence n: the W-1 rows in `hist`.
template <int DT, int W, int VEC>
__device__ __forceinline__ void store_final(const kda_conv_args &a, int n, int c, const float (&hist)[W - 1][VEC]) {
    if (!a.final_state) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        store_vec<DT, VEC>(a.final_state, ((int64_t)n * (W - 1) + j) * a.channels + c, hist[j]);
}

template <int DT, int W, int VEC>
__device__ __forceinline__ void empty_final(const kda_conv_args &a, int n, int c) {
    float hist[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<DT, W, VEC>(a, n, 0, j - (W - 1), c, hist[j]);
    store_final<DT, W, VEC>(a, n, c, hist);
}

// Rows in flight ahead of their use, forward and backward. Measured on MI355X (us, forward of 8192 x 4096 bf16 with
// 4 | 8 rows): 26.0 | 27.3; more rows only cost registers (8 rows: 224, two waves a SIMD).
constexpr int AHEAD = 4, BWD_AHEAD = 4;

// Bound by memory: every row is read and written once. 8192 x 4096 bf16, rows of x 16 KiB apart: 134 MB in 26.6 us,
// 5.0 TB/s, where a copy reaches 5.3.
template <int DT, int W, int VEC>
__global__ __launch_bounds__(256) void conv_fwd_kernel(const kda_conv_args a, int32_t *err, int L) {
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    const int tile = blockIdx.x;
    if (tile == 0 && blockIdx.y == 0) check_offsets(off, err, threadIdx.x, blockDim.x);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    const int T = a.total_tokens;
    const int64_t t0l = (int64_t)tile * L;
    if (c >= a.channels || (t0l >= T && tile != 0)) return;
    const int t0 = (int)t0l, t1 = T - t0 < L ? T : t0 + L;

    if (T == 0) {
        for (int i = 0; i < a.num_seqs; ++i) empty_final<DT, W, VEC>(a, i, c);
        return;
    }
    float tap[W][VEC], bias[VEC], hist[W - 1][VEC];
    load_taps<W, VEC>(a.weight, a.bias, c, tap, bias);
    int n = off.find(t0);
    int start = off.at(n), end = off.at(n + 1);
    if (tile == 0)
        for (int i = 0; i < n; ++i) empty_final<DT, W, VEC>(a, i, c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<DT, W, VEC>(a, n, start, t0 - (W - 1) + j, c, hist[j]);
    const bool act = a.activation != 0;
    int t = t0;
    // rows of the tile, AHEAD at a time, the next ones in flight while these are computed (rows past
    // the last are read again from the last)
    typename Vec<DT, VEC>::type next[AHEAD];
    auto fetch = [&](int from) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            next[k] = load_raw<DT, VEC>(a.x, (int64_t)(from + k < t1 ? from + k : t1 - 1) * a.x_stride + c);
    };
    fetch(t);
    while (true) {
        const int stop = end < t1 ? end : t1;
        while (t < stop) {
            const int m = stop - t < AHEAD ? stop - t : AHEAD;
            typename Vec<DT, VEC>::type row[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) row[k] = next[k];
            if (t + m < t1) fetch(t + m);
            auto rows = [&](auto whole) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k)
                    if (whole || k < m) {
                        float x[VEC], y[VEC];
                        to_float<DT, VEC>(row[k], x);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            float p = bias[i];
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) p = __builtin_fmaf(tap[j][i], hist[j][i], p);
                            p = __builtin_fmaf(tap[W - 1][i], x[i], p);
                            y[i] = act ? p * sigmoid_f(p) : p;
#pragma unroll
                            for (int j = 0; j + 1 < W - 1; ++j) hist[j][i] = hist[j + 1][i];
                            hist[W - 2][i] = x[i];
                        }
                        store_vec<DT, VEC>(a.out, (int64_t)(t + k) * a.channels + c, y);
                    }
            };
            if (m == AHEAD) rows(std::true_type{});
            else rows(std::false_type{});
            t += m;
        }
        if (t < end) break;              // the sequence goes on in the next tile
        store_final<DT, W, VEC>(a, n, c, hist);
        for (++n; n < a.num_seqs && off.at(n + 1) <= t; ++n) empty_final<DT, W, VEC>(a, n, c);
        if (t >= t1 || n >= a.num_seqs) break;
        start = t, end = off.at(n + 1);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_row<DT, W, VEC>(a, n, start, t - (W - 1) + j, c, hist[j]);
    }
}

// One row per sequence: the state's rows move up by one and the new row joins them. A thread
// reads all it needs of its channels before it writes, so the state may be updated in place. 256 x 4096 bf16: 17 MB in
// 5.4 us, most of it the latency of a launch and of one round of loads.
template <int DT, int W, int VEC>
__global__ __launch_bounds__(256) void conv_decode_kernel(const kda_conv_args a) {
    const int per = a.channels / VEC;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= (int64_t)a.num_seqs * per) return;
    const int n = (int)(id / per), c = (int)(id - (int64_t)n * per) * VEC;
    float tap[W][VEC], bias[VEC], hist[W - 1][VEC], x[VEC], y[VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<DT, W, VEC>(a, n, 0, j - (W - 1), c, hist[j]);
    load_vec<DT, VEC>(a.x, (int64_t)n * a.x_stride + c, x);
    load_taps<W, VEC>(a.weight, a.bias, c, tap, bias);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float p = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p = __builtin_fmaf(tap[j][i], hist[j][i], p);
        p = __builtin_fmaf(tap[W - 1][i], x[i], p);
        y[i] = a.activation ? p * sigmoid_f(p) : p;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) hist[j][i] = hist[j + 1][i];
        hist[W - 2][i] = x[i];
    }
    store_vec<DT, VEC>(a.out, (int64_t)n * a.channels + c, y);
    store_final<DT, W, VEC>(a, n, c, hist);
}

// ------------------------------------------------------------------------------ backward
// The walk goes forward in time: e_t completes the gradient of row t-(W-1). A tile stores the
// rows that it owns; it walks on for W-1 rows of the next tile for their e, whose weight
// gradients that tile adds. The tiles' sums of dw and db go to the workspace, [tile][W+1][C],
// and conv_dw_kernel adds them in a fixed order.
template <int DT, int W, int VEC>
struct BwdWalk {
    const kda_conv_args &a;
    const kda_conv_grads &g;
    float tap[W][VEC], bias[VEC], hist[W - 1][VEC], e[W][VEC], dw[W][VEC], db[VEC];
    int c, n, start, t0, t1;

    // the gradient of row s: of x, or of the initial state where s lies before the sequence; plain: of a row
    // that this tile owns
    template <bool PLAIN> __device__ __forceinline__ void emit(int s, const float *extra) {
        const bool row = PLAIN || (s >= start && s >= t0 && s < t1);
        const bool init = !PLAIN && s < start && start >= t0 && g.d_initial_state;
        if (!row && !init) return;
        float d[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            d[i] = extra ? extra[i] : 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j) d[i] = __builtin_fmaf(tap[j][i], e[W - 1 - j][i], d[i]);
        }
        if (row) store_vec<DT, VEC>(g.dx, (int64_t)s * a.channels + c, d);
        else store_vec<KDA_DTYPE_F32, VEC>(g.d_initial_state, ((int64_t)n * (W - 1) + (s - start + W - 1)) * a.channels + c, d);
    }
    // e[k] holds e_{t-(W-1)+k} once row t is in: d row t-(W-1) = sum_j w[j] e_{t-j}
    __device__ __forceinline__ void shift() {
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[j][i] = e[j + 1][i];
    }
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[j][i] = 0.0f;
    }
    template <bool PLAIN> __device__ __forceinline__ void step(int t, const float *x, const float *dy, bool mine) {
        shift();
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float p = bias[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) p = __builtin_fmaf(tap[j][i], hist[j][i], p);
            p = __builtin_fmaf(tap[W - 1][i], x[i], p);
            float v = dy[i];
            if (a.activation) {
                const float sg = sigmoid_f(p);
                v *= sg * __builtin_fmaf(p, 1.0f - sg, 1.0f);
            }
            e[W - 1][i] = v;
            if (mine) {         // of the next tile's rows nothing: 0 times an infinite row would be NaN
                db[i] += v;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j][i] = __builtin_fmaf(v, hist[j][i], dw[j][i]);
                dw[W - 1][i] = __builtin_fmaf(v, x[i], dw[W - 1][i]);
            }
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) hist[j][i] = hist[j + 1][i];
            hist[W - 2][i] = x[i];
        }
        emit<PLAIN>(t - (W - 1), nullptr);
    }
    // past the sequence's end: no further e, and the final state's gradient joins its rows
    __device__ __forceinline__ void finish(int end) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            shift();
            float extra[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                e[W - 1][i] = 0.0f;
                extra[i] = 0.0f;
            }
            const int s = end + k - (W - 1);
            if (g.d_final_state && (s < start || s < t1))
                load_vec<KDA_DTYPE_F32, VEC>(g.d_final_state, ((int64_t)n * (W - 1) + k) * a.channels + c, extra);
            emit<false>(s, extra);
        }
    }
};

template <int DT, int VEC, int W>
__device__ __forceinline__ void empty_grad(const kda_conv_args &a, const kda_conv_grads &g, int n, int c) {
    if (!g.d_initial_state) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float v[VEC];
        const int64_t at = ((int64_t)n * (W - 1) + j) * a.channels + c;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.0f;
        if (g.d_final_state) load_vec<KDA_DTYPE_F32, VEC>(g.d_final_state, at, v);
        store_vec<KDA_DTYPE_F32, VEC>(g.d_initial_state, at, v);
    }
}

// Reads x and dy, writes dx; p_t is formed again. 8 x 1024 x 2048 bf16: 101 MB in 27.6 us, 3.7 TB/s; memory and vector
// issue (about 40 operations an element) take about as long as each other. The taps' sums of a tile stay in
// registers and go to the workspace.
template <int DT, int W, int VEC>
__global__ __launch_bounds__(256) void conv_bwd_kernel(const kda_conv_args a, const kda_conv_grads g, float *part,
                                                       int32_t *err, int L) {
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    const int tile = blockIdx.x;
    if (tile == 0 && blockIdx.y == 0) check_offsets(off, err, threadIdx.x, blockDim.x);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    const int T = a.total_tokens;
    const int64_t t0l = (int64_t)tile * L;
    if (c >= a.channels || (t0l >= T && tile != 0)) return;
    BwdWalk<DT, W, VEC> k{a, g};
    k.c = c;
    k.t0 = (int)t0l, k.t1 = T - k.t0 < L ? T : k.t0 + L;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        k.db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) k.dw[j][i] = 0.0f;
    }
    if (T == 0) {
        for (int i = 0; i < a.num_seqs; ++i) empty_grad<DT, VEC, W>(a, g, i, c);
    } else {
        load_taps<W, VEC>(a.weight, a.bias, c, k.tap, k.bias);
        k.n = off.find(k.t0);
        k.start = off.at(k.n);
        int end = off.at(k.n + 1);
        if (tile == 0)
            for (int i = 0; i < k.n; ++i) empty_grad<DT, VEC, W>(a, g, i, c);
        int t = k.t0;
        const int last = T - k.t1 < W - 1 ? T : k.t1 + W - 1;       // rows that this tile reads
        typename Vec<DT, VEC>::type nx[BWD_AHEAD], ndy[BWD_AHEAD];
        auto fetch = [&](int from) {
#pragma unroll
            for (int q = 0; q < BWD_AHEAD; ++q) {
                const int64_t r = from + q < last ? from + q : last - 1;
                nx[q] = load_raw<DT, VEC>(a.x, r * a.x_stride + c);
                ndy[q] = load_raw<DT, VEC>(g.dy, r * g.dy_stride + c);
            }
        };
        fetch(t);
        while (true) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) load_row<DT, W, VEC>(a, k.n, k.start, t - (W - 1) + j, c, k.hist[j]);
            k.begin();
            const int stop = end < last ? end : last;
            while (t < stop) {
                typename Vec<DT, VEC>::type x[BWD_AHEAD], dy[BWD_AHEAD];
#pragma unroll
                for (int q = 0; q < BWD_AHEAD; ++q) x[q] = nx[q], dy[q] = ndy[q];
                const int then = t + BWD_AHEAD < stop ? t + BWD_AHEAD : stop;
                if (then < last) fetch(then);
                auto steps = [&](auto plain) {
#pragma unroll
                    for (int q = 0; q < BWD_AHEAD; ++q)
                        if (plain || t + q < stop) {
                            float xf[VEC], dyf[VEC];
                            to_float<DT, VEC>(x[q], xf);
                            to_float<DT, VEC>(dy[q], dyf);
                            k.template step<decltype(plain)::value>(t + q, xf, dyf, plain || t + q < k.t1);
                        }
                };
                const int lo = k.start > k.t0 ? k.start : k.t0;
                if (t - (W - 1) >= lo && t + BWD_AHEAD <= (stop < k.t1 ? stop : k.t1)) steps(std::true_type{});
                else steps(std::false_type{});
                t = then;
            }
            if (stop < end) break;       // the sequence goes on past this tile's last row
            k.finish(end);
            int n = k.n + 1;
            if (end > k.t1) break;       // what follows belongs to the next tile
            for (; n < a.num_seqs && off.at(n + 1) <= end; ++n) empty_grad<DT, VEC, W>(a, g, n, c);
            if (end >= k.t1 || n >= a.num_seqs) break;
            k.n = n, k.start = end;
            end = off.at(n + 1);
        }
    }
    float *p = part + (int64_t)tile * (W + 1) * a.channels + c;
#pragma unroll
    for (int j = 0; j < W; ++j) store_vec<KDA_DTYPE_F32, VEC>(p, (int64_t)j * a.channels, k.dw[j]);
    store_vec<KDA_DTYPE_F32, VEC>(p, (int64_t)W * a.channels, k.db);
}

// dw[c][j] and db[c] from the tiles' sums: 16 channels' lanes by 16 groups of tiles a block, the
// groups' sums joined in a fixed order. 8 x 1024 x 2048: 4.0 us, latency.
__global__ __launch_bounds__(256) void conv_dw_kernel(const float *part, int tiles, int C, int W, float *dw, float *db) {
    __shared__ float sum[16][17];
    const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int j = blockIdx.y, c = blockIdx.x * 16 + lane;
    float s = 0.0f;
    if (c < C)
        for (int i = grp; i < tiles; i += 16) s += part[((int64_t)i * (W + 1) + j) * C + c];
    sum[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += sum[i][lane];
        if (j < W) dw[(int64_t)c * W + j] = s;
        else if (db) db[c] = s;
    }
}

// ------------------------------------------------------------------------------ launches
bool aligned(const void *p, int64_t bytes) { return ((uintptr_t)p % bytes) == 0; }

// Channels a thread owns: as many as fill 16 bytes where every row starts on that boundary, else
// one (any channel count, stride and alignment).
int conv_vec(const kda_conv_args &a, int full) {
    const int64_t es = (int64_t)dtype_bytes(a.dtype);
    const bool ok = a.channels % full == 0 && a.x_stride % full == 0 && aligned(a.x, full * es) && aligned(a.out, full * es) &&
                    aligned(a.initial_state, full * es) && aligned(a.final_state, full * es) && aligned(a.weight, 16);
    return ok ? full : 1;
}

struct Shape {
    dim3 grid, block;
};

Shape conv_shape(int64_t tiles, int C, int vec) {
    const int lanes = (C + vec - 1) / vec;
    int bx = 64;
    while (bx < lanes && bx < 256) bx *= 2;
    Shape s;
    s.block = dim3(bx, 1);
    s.grid = dim3((unsigned)tiles, (unsigned)((lanes + bx - 1) / bx));
    return s;
}

// Rows per tile: as many tiles as give the card `target` waves, lo to hi rows each. Short tiles read the taps and
// the rows before them (and, backward, behind them) too often, long ones leave the card idle. Measured on MI355X
// (us): forward, 8192 x 4096 bf16, 8 channels a thread, target 1024 | 2048 | 4096 | 8192 waves: 29.5 | 26.0 | 32.2 |
// 33.0; gradients, 8 x 1024 x 2048 bf16, 2 channels a thread, target (of one channel a thread) 4096 | 8192 waves 32.2 |
// 33.8, and with 4 channels a thread 37.6 | 33.6. The forward's count is odd: tiles start at the same time, and with rows of a
// power of two a power of two of them puts all tiles' rows on the same memory channels (forward, 31 | 32 | 33 rows, on
// one card 32.5 | 36.0 | 26.6 us; the gradients do not mind: 64 | 65 rows 33.2 | 37.8).
int conv_tile(int64_t T, int64_t C, int vec, int lo, int hi, int target) {
    const int64_t waves = ceil_div(ceil_div(C, vec), 64);
    int64_t L = T * waves / target;
    L = L < lo ? lo : L > hi ? hi : L;
    return (int)(L / 8 * 8);
}
int fwd_tile(int64_t T, int64_t C, int vec) { return conv_tile(T, C, vec, 8, 64, 2048) + 1; }
int bwd_tile(int64_t T, int64_t C) { return conv_tile(T, C, 1, 32, 128, 4096); }

template <int DT, int W, int VEC> hipError_t fwd_at(const kda_conv_args &a, int32_t *err, hipStream_t st) {
    const int L = fwd_tile(a.total_tokens, a.channels, VEC);
    const int64_t tiles = a.total_tokens ? ceil_div(a.total_tokens, L) : 1;
    const Shape s = conv_shape(tiles, a.channels, VEC);
    conv_fwd_kernel<DT, W, VEC><<<s.grid, s.block, 0, st>>>(a, err, L);
    return hipGetLastError();
}
template <int DT, int W, int VEC> hipError_t decode_at(const kda_conv_args &a, hipStream_t st) {
    const int64_t threads = (int64_t)a.num_seqs * (a.channels / VEC);
    conv_decode_kernel<DT, W, VEC><<<dim3((unsigned)ceil_div(threads, 256)), 256, 0, st>>>(a);
    return hipGetLastError();
}
template <int DT, int W, int VEC>
hipError_t bwd_at(const kda_conv_args &a, const kda_conv_grads &g, float *ws, int32_t *err, hipStream_t st) {
    const int L = bwd_tile(a.total_tokens, a.channels);
    const int64_t tiles = a.total_tokens ? ceil_div(a.total_tokens, L) : 1;
    const Shape s = conv_shape(tiles, a.channels, VEC);
    conv_bwd_kernel<DT, W, VEC><<<s.grid, s.block, 0, st>>>(a, g, ws, err, L);
    if (hipError_t e = hipGetLastError()) return e;
    conv_dw_kernel<<<dim3((unsigned)ceil_div(a.channels, 16), (unsigned)(W + 1)), 256, 0, st>>>(ws, (int)tiles, a.channels, W,
                                                                                                g.dweight, g.dbias);
    return hipGetLastError();
}

template <int DT, int W> hipError_t fwd_w(const kda_conv_args &a, int32_t *err, hipStream_t st) {
    constexpr int FULL = DT == KDA_DTYPE_F32 ? 4 : 8;
    return conv_vec(a, FULL) == FULL ? fwd_at<DT, W, FULL>(a, err, st) : fwd_at<DT, W, 1>(a, err, st);
}
template <int DT, int W> hipError_t decode_w(const kda_conv_args &a, hipStream_t st) {
    constexpr int FULL = 4;
    return conv_vec(a, FULL) == FULL ? decode_at<DT, W, FULL>(a, st) : decode_at<DT, W, 1>(a, st);
}
template <int DT, int W>
hipError_t bwd_w(const kda_conv_args &a, const kda_conv_grads &g, float *ws, int32_t *err, hipStream_t st) {
    constexpr int FULL = 2;
    const bool ok = conv_vec(a, FULL) == FULL && g.dy_stride % FULL == 0 && aligned(g.dy, FULL * dtype_bytes(DT)) &&
                    aligned(g.dx, FULL * dtype_bytes(DT)) && aligned(g.d_final_state, 8) && aligned(g.d_initial_state, 8);
    return ok ? bwd_at<DT, W, FULL>(a, g, ws, err, st) : bwd_at<DT, W, 1>(a, g, ws, err, st);
}

#define KDA_CONV_WIDTHS(CALL)              \
    switch (a.width) {                     \
    case 2: return CALL(2);                \
    case 3: return CALL(3);                \
    case 4: return CALL(4);                \
    case 5: return CALL(5);                \
    case 6: return CALL(6);                \
    case 7: return CALL(7);                \
    case 8: return CALL(8);                \
    default: return hipErrorInvalidValue;  \
    }

template <int DT> hipError_t fwd_dt(const kda_conv_args &a, int32_t *err, hipStream_t st) {
#define CALL(W) fwd_w<DT, W>(a, err, st)
    KDA_CONV_WIDTHS(CALL)
#undef CALL
}
template <int DT> hipError_t decode_dt(const kda_conv_args &a, hipStream_t st) {
#define CALL(W) decode_w<DT, W>(a, st)
    KDA_CONV_WIDTHS(CALL)
#undef CALL
}
template <int DT>
hipError_t bwd_dt(const kda_conv_args &a, const kda_conv_grads &g, float *ws, int32_t *err, hipStream_t st) {
#define CALL(W) bwd_w<DT, W>(a, g, ws, err, st)
    KDA_CONV_WIDTHS(CALL)
#undef CALL
}

}  // namespace

hipError_t launch_conv_fwd(const kda_conv_args &a, int32_t *err, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return fwd_dt<KDA_DTYPE_F32>(a, err, st);
    if (a.dtype == KDA_DTYPE_BF16) return fwd_dt<KDA_DTYPE_BF16>(a, err, st);
    return fwd_dt<KDA_DTYPE_F16>(a, err, st);
}
hipError_t launch_conv_decode(const kda_conv_args &a, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return decode_dt<KDA_DTYPE_F32>(a, st);
    if (a.dtype == KDA_DTYPE_BF16) return decode_dt<KDA_DTYPE_BF16>(a, st);
    return decode_dt<KDA_DTYPE_F16>(a, st);
}
size_t conv_bwd_workspace(int64_t T, int64_t C, int W) {
    const int64_t tiles = T ? ceil_div(T, bwd_tile(T, C)) : 1;
    return (size_t)tiles * (W + 1) * C * sizeof(float);
}
hipError_t launch_conv_bwd(const kda_conv_args &a, const kda_conv_grads &g, float *ws, int32_t *err, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return bwd_dt<KDA_DTYPE_F32>(a, g, ws, err, st);
    if (a.dtype == KDA_DTYPE_BF16) return bwd_dt<KDA_DTYPE_BF16>(a, g, ws, err, st);
    return bwd_dt<KDA_DTYPE_F16>(a, g, ws, err, st);
}

}  // namespace ops
}  // namespace kda
