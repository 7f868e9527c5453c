// ops_lin_bwd.hip -- gradients of the linear attention with a decay for each head (ops_lin.hpp).
//
// With X the state that enters a chunk and Y the gradient of the one that leaves it, three walks give dv and dk (backwards on
// Y), then dq (forwards on X), and on the way u_i = q_i . (part of dq_i from X), w_j = k_j . (part of dk_j from Y).
// A decay's gradient is what passes it, from tokens before t to tokens from t on:
//
//   dg_t = sum_{j < t <= i} W_ij + sum_{i >= t} u_i + sum_{j < t} w_j + e^G <X, Y>,   W_ij = scale e^{G_i - G_j} (q_i . k_j) (do_i . v_j)
//
// over the chunk, the last term what passes all of it. Nothing is subtracted: pairs of a token with itself, which outweigh
// all else where decays are short, never enter, nor does what ends before t or begins behind it, which may be larger by any factor (tokens of
// other sizes, resets). The walk for dk leaves Y at each border of chunks inside a segment for the one for dq, which holds X there: 1 KB for
// a token and head of 128 x 128, written and read once, SLOTS bytes at a time.
//
// 8 x 1024 tokens of 16 heads of 128 x 128 in bf16 (261 MB in and out: 49 us of memory): states both ways 27 us, joins 7, walks for dk and
// dv 112, for dq 90, decays 37; 266 in all. The walks are bound as the forward's is, with three parts where they lead to a
// decay's gradient; the one for dq, a block a CU, waits 66% of its waves' cycles. The states handed on (117 MB each way) take 38 us of them.
#include "ops_lin.hpp"

#include <type_traits>

namespace kda {
namespace ops {
namespace lin {
namespace {

// What both directions add to their states, by blockIdx.z.
template <int DT, int KD, int VD>
__global__ __launch_bounds__(THREADS<VD>, WAVES<VD> / 2) void lin_bwd_state_kernel(const Batch b, const Own x, const Own y) {
    __shared__ OwnLds<DT, KD, VD> lds;
    if (blockIdx.z == 0) own_state<DT, KD, VD, false>(b, x, lds);
    else own_state<DT, KD, VD, true>(b, y, lds);
}

template <int SIZE, int AHEAD>
__global__ __launch_bounds__(JOIN_THREADS) void lin_bwd_join_kernel(const Batch b, float *x, const float *xf, float *y, const float *yf) {
    if (blockIdx.z == 0) join<SIZE, AHEAD>(b, x, xf, false);
    else join<SIZE, AHEAD>(b, y, yf, true);
}

// Walks of one launch, by blockIdx.z: side by side they fill what each leaves of the chip (dv beside dk and then dq 112 + 90 us, dk and
// then dv beside dq 98 + 117). dq's and dk's states lie turned and take a
// wave for every 16 key columns, dv's for every 16 value columns: where these differ, dv's has a launch of its own.
enum { DQ, DK, DV };
template <int DT, int KD, int VD, int W> struct One {
    static constexpr int NT = W == DV ? THREADS<VD> : THREADS<KD>, A_SIMD = W == DV ? WAVES_A_SIMD<DT, VD> : WAVES_A_SIMD<DT, KD>;
    typedef typename std::conditional<W == DV, WalkLds<DT, KD, VD>, WalkLds<DT, VD, KD>>::type Lds;
    static __device__ __forceinline__ void run(const Batch &b, const Walk &a, const Place &p, Lds &lds) {
        if constexpr (W == DV) walk<DT, KD, VD, true, false>(b, a, p, lds);
        else walk<DT, VD, KD, W == DK, true>(b, a, p, lds);
    }
};
// Blocks take the segments of one head after another, from block `first` of all on.
template <int DT, int KD, int VD, int W, int V>
__global__ __launch_bounds__((One<DT, KD, VD, W>::NT), (One<DT, KD, VD, W>::A_SIMD)) void lin_walks_kernel(
    const Batch b, const Walk w, const Walk v, int64_t first, int32_t *err) {
    typedef One<DT, KD, VD, W> A;
    typedef One<DT, KD, VD, V> B;
    static_assert(A::NT == B::NT, "one number of waves for both");
    __shared__ union {
        typename A::Lds a;
        typename B::Lds b;
    } lds;
    const int64_t n = first + blockIdx.x;
    const int h = (int)(n / b.segs), seg = (int)(n - (int64_t)h * b.segs);
    const Place p = {seg, h, 0, seg, b.segs, (int)blockIdx.x};
    if (err && n == 0 && blockIdx.z == 0) check_offsets(b.offsets(), err, threadIdx.x, A::NT);
    if (blockIdx.z == 0) return A::run(b, w, p, lds.a);
    if constexpr (V != W) B::run(b, v, p, lds.b);
}

// ---------------------------------------------------------------- gradients of the decays
struct Decays {
    Role q, k, v, d_out;
    const float *u, *w;         // [T, H]; u with what passes all of a chunk at its last token
    float *dg;                  // [T, H], or partial sums [segs, H]
    float scale;
    int per_head;
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    return x;
}
// 16 rows of a chunk as operands: lane (i, g) has elements 32 s + 8 g .. of row i
template <int DT, int D> struct Sixteen {
    u32x4 r[D / 32];
    __device__ __forceinline__ void load(const Rows &s, const Chunk &c, int first) {
        const Buffer b = s.from(c.first, c.len, D);
        const int row = first + (threadIdx.x & 15);
        const uint32_t at = row < c.len ? row * s.row + (threadIdx.x & 48) : OUTSIDE;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) r[n] = read16(b, at, 64 * n);
    }
    __device__ __forceinline__ void operand(int n, u32x4 (&to)[PLANES<DT>]) const {
        if constexpr (DT == KDA_DTYPE_BF16) to[0] = r[n];
        else {
            typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
            const f16x8 e = __builtin_bit_cast(f16x8, r[n]);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
            split<2>(v, to);
        }
    }
};
template <int DT, int D> __device__ __forceinline__ f32x4 products(const Sixteen<DT, D> &a, const Sixteen<DT, D> &b) {
    constexpr int NP = PLANES<DT>;
    f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        u32x4 x[NP], y[NP];
        a.operand(s, x);
        b.operand(s, y);
        pairs<NP, NP, 4>([&](int m, int k) { c = mma(x[m], y[k], c); });
    }
    return c;
}

// A block takes a segment of one head, four chunks at a time, four waves each: a wave the pairs with 16 of the tokens i. (A
// wave a chunk left two waves a SIMD to wait for their operands: a third more time. Now 37 us for 8192 tokens of 16 heads.)
constexpr int DECAY_WAVES = 16, DECAY_THREADS = 64 * DECAY_WAVES;
struct DecayLds {
    Clock clocks[4];
    float part[DECAY_WAVES];
    float inside[4][C];         // of chunk and token: what passes it within its 16 tokens i
    float rows[4][4][C];        // of chunk, 16 tokens i, token j: W summed over the i
};

template <int DT, int KD, int VD>
__global__ __launch_bounds__(DECAY_THREADS) void lin_decay_kernel(const Batch b, const Decays a) {
    __shared__ DecayLds L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    // its chunk and its tokens i (four waves of a SIMD, which have most pairs at 3, have one of each)
    const int turn = wave >> 2, it = (wave + turn) & 3;
    const int seg = blockIdx.x, h = blockIdx.y;
    const Offsets o = b.offsets();
    const int s0 = seg * b.seg, s1 = s0 + b.seg < b.T ? s0 + b.seg : b.T;
    Chunks<false> chunks(o, s0, s1);
    Clock &clock = L.clocks[turn];
    float all = 0.0f;
    // the wave's chunk of the next four, and what it reads of it first
    const Rows rq(a.q, h), rk(a.k, h), rv(a.v, h), rd(a.d_out, h);
    Chunk own;
    Sixteen<DT, KD> q, k;
    Sixteen<DT, VD> d, v;
    float u, w, decay;
    auto fetch = [&]() {
        Chunks<false> ahead = chunks;
        own = Chunk{0, 0, 0, false, false, false, false};
#pragma unroll 1
        for (int n = 0; n <= turn; ++n) own = ahead.next();
        u = w = decay = 0.0f;
        if (it == 0) {
            const int64_t at = (int64_t)(own.first + lane) * b.H + h;
            if (lane < own.len) u = a.u[at], w = a.w[at];
            decay = b.decay(own.first, own.len, h);
        }
        q.load(rq, own, 16 * it), d.load(rd, own, 16 * it);
        k.load(rk, own, 0), v.load(rv, own, 0);
    };
    fetch();
#pragma unroll 1
    for (;;) {
        int count = 0;
#pragma unroll 1
        while (count < 4 && chunks.next().len) ++count;
        if (!count) break;
        const bool there = it == 0 && lane < own.len;
        const int64_t at = (int64_t)(own.first + lane) * b.H + h;
        if (it == 0) tick<false>(clock, decay, 1.0f, 1.0f);
        lds_barrier();
        // W: rows tokens j, columns tokens i > j. Summed over i from each token on, then over the j before it: nothing is subtracted.
        float inside = 0.0f;        // of token 16 it + i
        const int ti = 16 * it + i;
        const float wi = clock.whole[ti], ri = clock.rest[ti];
#pragma unroll 1
        for (int jt = 0; jt <= it; ++jt) {
            if (16 * it >= own.len) break;
            const f32x4 qk = products(k, q), dv = products(v, d);
            if (jt < it) k.load(rk, own, 16 * jt + 16), v.load(rv, own, 16 * jt + 16);
            const f32x4 wj = *reinterpret_cast<const f32x4 *>(&clock.whole[16 * jt + 4 * g]);
            const f32x4 rj = *reinterpret_cast<const f32x4 *>(&clock.rest[16 * jt + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * jt + 4 * g + r;
                const float x = qk[r] * dv[r] * exp2_f((wi - wj[r]) + (ri - rj[r])) * a.scale;
                const float from = row_suffix(j < ti ? x : 0.0f);
                inside += j < ti ? from : 0.0f;
                if (i == 0) L.rows[turn][it][j] = from;
            }
        }
        inside = swap16_add(inside, inside);
        inside = swap32_add(inside, inside);
        if (g == 0) L.inside[turn][ti] = inside;
        const int len = own.len;
        const float own_u = u, own_w = w;
        fetch();
        lds_barrier();
        if (it == 0) {
            // lane t: what passes within its 16 tokens i, from those behind, u from t on, w before t
            float dg = L.inside[turn][lane], from = own_u, upto = own_w, behind[3];
            float sum = 0.0f;
#pragma unroll
            for (int n = 3; n > 0; --n) {       // to tokens from 16 n on
                if (16 * n < len) sum += g <= n ? L.rows[turn][n][lane] : 0.0f;
                behind[n - 1] = sum;
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const float x = __shfl_down(from, d), y = __shfl_up(upto, d);
                if (lane + d < 64) from += x;
                if (lane >= d) upto += y;
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    const float z = __shfl_up(behind[n], d);
                    if (lane >= d) behind[n] += z;
                }
            }
            // (before t: what the lane before holds; the last tokens have none behind)
            const float y0 = __shfl_up(behind[0], 1), y1 = __shfl_up(behind[1], 1), y2 = __shfl_up(behind[2], 1), before = __shfl_up(upto, 1);
            if (lane && g < 3) dg += g == 0 ? y0 : g == 1 ? y1 : y2;
            dg += from + (lane ? before : 0.0f);
            if (there) {
                if (a.per_head) all += dg;
                else a.dg[at] = dg;
            }
        }
        lds_barrier();        // all of it is read
    }
    if (a.per_head) {
        all = wave_sum(all);
        lds_barrier();
        if (lane == 0) L.part[wave] = all;
        lds_barrier();
        if (wave == 0) {
            all = row_suffix(L.part[i]);
            if (lane == 0) a.dg[(int64_t)seg * b.H + h] = all;
        }
    }
}

// dg [H] from the segments' sums, in their order: a wave a head.
__global__ __launch_bounds__(64) void lin_decay_sum_kernel(const float *part, float *dg, int segs, int H) {
    const int h = blockIdx.x;
    float x = 0.0f;
    for (int s = threadIdx.x; s < segs; s += 64) x += part[(int64_t)s * H + h];
    x = wave_sum(x);
    if (threadIdx.x == 0) dg[h] = x;
}

// ---------------------------------------------------------------- host
// States that the walk for dk hands on take this many bytes at most; larger batches are walked a range of blocks at a time.
constexpr size_t SLOTS = (size_t)1 << 30;
constexpr int LONGEST = 64;      // chunks of a segment: at 128 x 128, SLOTS holds the states of 256 such segments
struct Plan {
    int seg, segs;
    int64_t blocks, most;     // segments and heads; of them in a launch
    size_t state, factor, token, d_init, sums, between;     // elements of the parts of the workspace (d_init: room that callers' sizes count)
};
// 256 blocks of each walk at least. 8192 tokens of 16 heads in all (us, 256 blocks | 352 | 512 | 688): 280 | 354 | 326 | 369, as
// longer segments have fewer states to write, join and read (65536 of 8: 1066 | 1106 | 1002 | 1100).
Plan plan(int64_t T, int64_t H, int64_t S, int64_t size, bool per_head, bool own_d_init) {
    Plan p;
    p.seg = segment(T, H, 256, C);
    if (p.seg > LONGEST * C) p.seg = LONGEST * C;
    p.segs = (int)ceil_div(T > 0 ? T : 1, p.seg);
    p.blocks = (int64_t)p.segs * H;
    const int64_t per = p.seg / C, fit = (int64_t)(SLOTS / (size * sizeof(float))) / per;
    p.most = p.seg == C || fit > p.blocks ? p.blocks : fit;
    p.state = p.segs > 1 ? (size_t)p.segs * H * size : 0;
    p.factor = p.segs > 1 ? (size_t)p.segs * H : 0;
    p.token = (size_t)T * H;
    p.d_init = own_d_init ? (size_t)S * H * size : 0;
    p.sums = per_head ? (size_t)p.segs * H : 0;
    p.between = p.seg > C ? (size_t)(p.most * per * size) : 0;
    return p;
}
inline size_t elements(const Plan &p) { return 2 * p.state + p.d_init + p.between + 2 * p.factor + 2 * p.token + p.sums; }

template <int DT, int KD, int VD> hipError_t backward(const kda_lin_args &a, const kda_lin_grads &r, float *ws, int32_t *err, hipStream_t st) {
    const bool own_d_init = a.initial_state && !r.d_initial_state;
    const Plan p = plan(a.total_tokens, a.heads, a.num_seqs, KD * VD, a.g_per_head, own_d_init);
    const Batch b = {a.cu_seqlens, a.g, a.g_per_head ? 0 : a.heads, a.num_seqs, a.total_tokens, a.heads, p.seg, p.segs, 1};
    const Role q = {a.q, a.q_stride, a.q_head_stride}, k = {a.k, a.k_stride, a.k_head_stride}, v = {a.v, a.v_stride, a.v_head_stride};
    const Role d = {r.d_out, r.d_out_stride, r.d_out_head_stride}, none = {nullptr, 0, 0};
    // 16-byte pieces first
    float *x = ws, *y = x + p.state, *between = y + p.state + p.d_init, *xf = between + p.between, *yf = xf + p.factor, *u = yf + p.factor,
          *w = u + p.token, *sums = w + p.token;
    const dim3 grid((unsigned)p.segs, (unsigned)a.heads);
    hipError_t e;
    if (p.segs > 1) {
        const Own ox = {k, v, a.initial_state, x, xf, 1.0f}, oy = {q, d, r.d_final_state, y, yf, a.scale};
        lin_bwd_state_kernel<DT, KD, VD><<<dim3(grid.x, grid.y, 2), THREADS<VD>, 0, st>>>(b, ox, oy);
        if ((e = hipGetLastError())) return e;
        const dim3 join(KD * VD / JOIN_THREADS, grid.y, 2);
        if (far_ahead(p.segs)) lin_bwd_join_kernel<KD * VD, 32><<<join, JOIN_THREADS, 0, st>>>(b, x, xf, y, yf);
        else lin_bwd_join_kernel<KD * VD, 8><<<join, JOIN_THREADS, 0, st>>>(b, x, xf, y, yf);
        if ((e = hipGetLastError())) return e;
    }
    // dq on X^T, dk on Y^T: their states' rows are value elements
    const Walk wq = {d, v, k, r.dq, x, a.initial_state, nullptr, a.scale, a.scale, 1.0f, q, u, between, y, r.d_final_state};
    const Walk wv = {k, q, d, r.dv, y, r.d_final_state, r.d_initial_state, a.scale, 1.0f, a.scale, none, nullptr, nullptr, nullptr, nullptr};
    const Walk wk = {v, d, q, r.dk, y, r.d_final_state, nullptr, a.scale, 1.0f, a.scale, k, w, between, nullptr, nullptr};
    for (int64_t first = 0; first < p.blocks; first += p.most) {
        const unsigned n = (unsigned)(p.blocks - first < p.most ? p.blocks - first : p.most);
        if constexpr (KD == VD) {
            lin_walks_kernel<DT, KD, VD, DK, DV><<<dim3(n, 1, 2), THREADS<KD>, 0, st>>>(b, wk, wv, first, err);
        } else {
            lin_walks_kernel<DT, KD, VD, DK, DK><<<n, THREADS<KD>, 0, st>>>(b, wk, wk, first, err);
            if ((e = hipGetLastError())) return e;
            lin_walks_kernel<DT, KD, VD, DV, DV><<<n, THREADS<VD>, 0, st>>>(b, wv, wv, first, nullptr);
        }
        if ((e = hipGetLastError())) return e;
        lin_walks_kernel<DT, KD, VD, DQ, DQ><<<n, THREADS<KD>, 0, st>>>(b, wq, wq, first, nullptr);
        if ((e = hipGetLastError())) return e;
    }
    const Decays dec = {q, k, v, d, u, w, a.g_per_head ? sums : r.dg, a.scale, a.g_per_head};
    lin_decay_kernel<DT, KD, VD><<<grid, DECAY_THREADS, 0, st>>>(b, dec);
    if ((e = hipGetLastError())) return e;
    if (a.g_per_head) {
        lin_decay_sum_kernel<<<dim3(grid.y), 64, 0, st>>>(sums, r.dg, p.segs, a.heads);
        if ((e = hipGetLastError())) return e;
    }
    return hipSuccess;
}

template <int DT> hipError_t backward_dt(const kda_lin_args &a, const kda_lin_grads &g, float *ws, int32_t *err, hipStream_t st) {
    if (a.key_dim == 64) return a.value_dim == 64 ? backward<DT, 64, 64>(a, g, ws, err, st) : backward<DT, 64, 128>(a, g, ws, err, st);
    return a.value_dim == 64 ? backward<DT, 128, 64>(a, g, ws, err, st) : backward<DT, 128, 128>(a, g, ws, err, st);
}

}  // namespace
}  // namespace lin

#ifndef KDA_LIN_BWD_F16
size_t lin_bwd_workspace(int64_t T, int64_t H, int64_t S, int64_t KD, int64_t VD, bool per_head, bool own_d_init) {
    return lin::elements(lin::plan(T, H, S, KD * VD, per_head, own_d_init)) * sizeof(float);
}

hipError_t launch_lin_bwd(const kda_lin_args &a, const kda_lin_grads &g, float *ws, int32_t *err, hipStream_t st) {
    return a.dtype == KDA_DTYPE_BF16 ? lin::backward_dt<KDA_DTYPE_BF16>(a, g, ws, err, st) : launch_lin_bwd_f16(a, g, ws, err, st);
}
#else
hipError_t launch_lin_bwd_f16(const kda_lin_args &a, const kda_lin_grads &g, float *ws, int32_t *err, hipStream_t st) {
    return lin::backward_dt<KDA_DTYPE_F16>(a, g, ws, err, st);
}
#endif

}  // namespace ops
}  // namespace kda
