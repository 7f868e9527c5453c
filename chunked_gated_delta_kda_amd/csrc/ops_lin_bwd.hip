// ops_lin_bwd.hip -- gradients of the linear attention with a decay for each head (ops_lin.hpp).
//
// With X the state that enters a chunk and Y the gradient of the one that leaves it, three walks give dq (forwards on X),
// dv and dk (backwards on Y), and on the way u_i = q_i . (part of dq_i from X), w_j = k_j . (part of dk_j from Y).
// A decay's gradient is what passes it, from tokens before t to tokens from t on:
//
//   dg_t = sum_{j < t <= i} W_ij + sum_{i >= t} u_i + sum_{j < t} w_j + c,   W_ij = scale e^{G_i - G_j} (q_i . k_j) (do_i . v_j)
//
// over the chunk, with c what passes all of it: F, what passes its first border (<X, Y> there, formed at a segment's
// border or a sequence's), less the chunk's u; c plus the chunk's w pass the next border. That is the only subtraction, over
// the chunks of a segment: pairs of a token with itself, which outweigh all else where decays are short, never enter,
// and where a chunk leaves less than 2^-24 of a state and c is under 2^-16 of its u's sizes, c is what rounding left of that difference
// and put to 0, so that nothing outlives a reset.
#include "ops_lin.hpp"

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

template <int SIZE>
__global__ __launch_bounds__(JOIN_THREADS) void lin_bwd_join_kernel(const Batch b, float *x, const float *xf, float *y, const float *yf) {
    if (blockIdx.z == 0) join<SIZE>(b, x, xf, false);
    else join<SIZE>(b, y, yf, true);
}

template <int DT, int KD, int VD>
__global__ __launch_bounds__(THREADS<VD>, (WAVES_A_SIMD<DT, VD>)) void lin_dq_kernel(const Batch b, const Walk a, int32_t *err) {
    __shared__ WalkLds<DT, KD, VD> lds;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(b.offsets(), err, threadIdx.x, THREADS<VD>);
    walk<DT, KD, VD, false, true>(b, a, lds);
}
template <int DT, int KD, int VD>
__global__ __launch_bounds__(THREADS<VD>, (WAVES_A_SIMD<DT, VD>)) void lin_dv_kernel(const Batch b, const Walk a) {
    __shared__ WalkLds<DT, KD, VD> lds;
    walk<DT, KD, VD, true, false>(b, a, lds);
}
template <int DT, int KD, int VD>
__global__ __launch_bounds__(THREADS<VD>, (WAVES_A_SIMD<DT, VD>)) void lin_dk_kernel(const Batch b, const Walk a) {
    __shared__ WalkLds<DT, KD, VD> lds;
    walk<DT, KD, VD, true, true>(b, a, lds);
}

// ---------------------------------------------------------------- gradients of the decays
struct Decays {
    Role q, k, v, d_out;
    const float *x, *y;         // joined states and gradients
    const float *init, *d_init; // of sequences, or both NULL
    const float *u, *w;         // [T, H]
    float *dg;                  // [T, H], or partial sums [segs, H]
    float scale;
    int per_head;
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    return x;
}
// operand: 8 elements of a row, as bf16 parts
template <int DT> __device__ __forceinline__ void global_operand(const Role &s, int h, int t, bool there, int at, u32x4 (&to)[PLANES<DT>]) {
    u32x4 r = {0, 0, 0, 0};
    if (there) r = *reinterpret_cast<const u32x4 *>((const uint16_t *)s.p + (int64_t)t * s.row + (int64_t)h * s.head + at);
    if constexpr (DT == KDA_DTYPE_BF16) to[0] = r;
    else {
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        const f16x8 e = __builtin_bit_cast(f16x8, r);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
        split<2>(v, to);
    }
}

// sums over a row's lanes from each lane on: four steps to the right
__device__ __forceinline__ float row_suffix(float x) {
    x += dpp_f<0x101>(x);       // the lane one to the right (0 past the row's end), then two, four, eight
    x += dpp_f<0x102>(x);
    x += dpp_f<0x104>(x);
    x += dpp_f<0x108>(x);
    return x;
}

constexpr int DECAY_THREADS = 256;

// A block takes a segment of one head, four chunks at a time, a wave each.
template <int DT, int KD, int VD>
__global__ __launch_bounds__(DECAY_THREADS) void lin_decay_kernel(const Batch b, const Decays a) {
    constexpr int NP = PLANES<DT>, SIZE = KD * VD;
    __shared__ Clock clocks[4];
    __shared__ float part[4], border[4], sums[4][4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int seg = blockIdx.x, h = blockIdx.y;
    const Offsets o = b.offsets();
    const int s0 = seg * b.seg, s1 = s0 + b.seg < b.T ? s0 + b.seg : b.T;
    Chunks<false> chunks(o, s0, s1);
    Clock &clock = clocks[wave];
    float all = 0.0f, F = 0.0f;
#pragma unroll 1
    for (;;) {
        Chunk own = {0, 0, 0, false, false, false, false};
        int enters = 0, count = 0;
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
            const Chunk c = chunks.next();
            if (!c.len) break;
            ++count;
            if (n == wave) own = c;
            if (!c.enter) continue;
            // what passes the first border of a part: the block together
            enters |= 1 << n;
            const float *x = nullptr, *y = nullptr;
            if (!c.open) x = a.x + ((int64_t)(seg - 1) * b.H + h) * SIZE, y = a.y + ((int64_t)seg * b.H + h) * SIZE;
            else if (a.init) x = a.init + ((int64_t)c.seq * b.H + h) * SIZE, y = a.d_init + ((int64_t)c.seq * b.H + h) * SIZE;
            float sum = 0.0f;
            if (x) {
                for (int e = 4 * threadIdx.x; e < SIZE; e += 4 * DECAY_THREADS) {
                    const f32x4 p = *reinterpret_cast<const f32x4 *>(x + e), q = *reinterpret_cast<const f32x4 *>(y + e);
                    sum += (p[0] * q[0] + p[1] * q[1]) + (p[2] * q[2] + p[3] * q[3]);
                }
            }
            sum = wave_sum(sum);
            __syncthreads();
            if (lane == 0) part[wave] = sum;
            __syncthreads();
            if (threadIdx.x == 0) border[n] = (part[0] + part[1]) + (part[2] + part[3]);
        }
        if (!count) break;
        const bool there = lane < own.len;
        const int64_t at = (int64_t)(own.first + lane) * b.H + h;
        const float u = there ? a.u[at] : 0.0f, w = there ? a.w[at] : 0.0f;
        tick<false>(clock, b.decay(own.first, own.len, h), 1.0f, 1.0f);
        {
            const float su = wave_sum(u), sw = wave_sum(w), size = wave_sum(__builtin_fabsf(u));
            if (lane == 0) sums[wave][0] = su, sums[wave][1] = sw, sums[wave][2] = clock.total, sums[wave][3] = size;
        }
        __syncthreads();
        float mine = 0.0f;      // what passes all of the wave's chunk
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n >= count) break;
            if (enters >> n & 1) F = border[n];
            float c = F - sums[n][0];
            if (sums[n][2] < 0x1p-24f && __builtin_fabsf(c) < 0x1p-16f * sums[n][3]) c = 0.0f;
            if (n == wave) mine = c;
            F = c + sums[n][1];
        }
        // W: rows tokens j, columns tokens i > j. Summed over i from each token on, then over the j before it: nothing is subtracted.
        float inside[4] = {0.0f, 0.0f, 0.0f, 0.0f};      // of token 16 it + i
        float later[4][4];                              // over the tiles of i behind
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
#pragma unroll
            for (int r = 0; r < 4; ++r) later[jt][r] = 0.0f;
#pragma unroll
        for (int it = 3; it >= 0; --it) {
            if (16 * it >= own.len) continue;
            const int ti = 16 * it + i;
            const float wi = clock.whole[ti], ri = clock.rest[ti];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                if (jt > it) continue;
                const int tj = 16 * jt + i;
                f32x4 qk = {0, 0, 0, 0}, dv = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < KD / 32; ++s) {
                    u32x4 x[NP], y[NP];
                    global_operand<DT>(a.k, h, own.first + tj, tj < own.len, 32 * s + 8 * g, x);
                    global_operand<DT>(a.q, h, own.first + ti, ti < own.len, 32 * s + 8 * g, y);
                    pairs<NP, NP, 4>([&](int m, int k) { qk = mma(x[m], y[k], qk); });
                }
#pragma unroll
                for (int s = 0; s < VD / 32; ++s) {
                    u32x4 x[NP], y[NP];
                    global_operand<DT>(a.v, h, own.first + tj, tj < own.len, 32 * s + 8 * g, x);
                    global_operand<DT>(a.d_out, h, own.first + ti, ti < own.len, 32 * s + 8 * g, y);
                    pairs<NP, NP, 4>([&](int m, int k) { dv = mma(x[m], y[k], dv); });
                }
                const f32x4 wj = *reinterpret_cast<const f32x4 *>(&clock.whole[16 * jt + 4 * g]);
                const f32x4 rj = *reinterpret_cast<const f32x4 *>(&clock.rest[16 * jt + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * jt + 4 * g + r;
                    const float x = qk[r] * dv[r] * exp2_f((wi - wj[r]) + (ri - rj[r])) * a.scale;
                    const float from = row_suffix(j < ti ? x : 0.0f) + later[jt][r];
                    inside[it] += j < ti ? from : 0.0f;
                    later[jt][r] = __shfl(from, lane & 48);     // of the tile's first token
                }
            }
        }
        // lane t: the tokens' own sums, u from t on, w before t
        float dg = 0.0f;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            float x = swap16_add(inside[it], inside[it]);
            x = swap32_add(x, x);
            if (g == it) dg = x;
        }
        float from = u, upto = w;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const float x = __shfl_down(from, d), y = __shfl_up(upto, d);
            if (lane + d < 64) from += x;
            if (lane >= d) upto += y;
        }
        const float before = __shfl_up(upto, 1);
        dg += from + (lane ? before : 0.0f) + mine;
        if (there) {
            if (a.per_head) all += dg;
            else a.dg[at] = dg;
        }
        __syncthreads();        // border and sums are read
    }
    if (a.per_head) {
        all = wave_sum(all);
        __syncthreads();
        if (lane == 0) part[wave] = all;
        __syncthreads();
        if (threadIdx.x == 0) a.dg[(int64_t)seg * b.H + h] = (part[0] + part[1]) + (part[2] + part[3]);
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
struct Plan {
    int seg, segs;
    size_t state, factor, token, d_init, sums;     // elements of the parts of the workspace
};
Plan plan(int64_t T, int64_t H, int64_t S, int64_t size, bool per_head, bool own_d_init) {
    Plan p;
    p.seg = segment(T, H, 512, C);
    p.segs = (int)ceil_div(T > 0 ? T : 1, p.seg);
    p.state = p.segs > 1 ? (size_t)p.segs * H * size : 0;
    p.factor = p.segs > 1 ? (size_t)p.segs * H : 0;
    p.token = (size_t)T * H;
    p.d_init = own_d_init ? (size_t)S * H * size : 0;
    p.sums = per_head ? (size_t)p.segs * H : 0;
    return p;
}
inline size_t elements(const Plan &p) { return 2 * p.state + p.d_init + 2 * p.factor + 2 * p.token + p.sums; }

template <int DT, int KD, int VD> hipError_t backward(const kda_lin_args &a, const kda_lin_grads &r, float *ws, int32_t *err, hipStream_t st) {
    const bool own_d_init = a.initial_state && !r.d_initial_state;
    const Plan p = plan(a.total_tokens, a.heads, a.num_seqs, KD * VD, a.g_per_head, own_d_init);
    const Batch b = {a.cu_seqlens, a.g, a.g_per_head ? 0 : a.heads, a.num_seqs, a.total_tokens, a.heads, p.seg, p.segs};
    const Role q = {a.q, a.q_stride, a.q_head_stride}, k = {a.k, a.k_stride, a.k_head_stride}, v = {a.v, a.v_stride, a.v_head_stride};
    const Role d = {r.d_out, r.d_out_stride, r.d_out_head_stride}, none = {nullptr, 0, 0};
    // 16-byte pieces first
    float *x = ws, *y = x + p.state, *di = y + p.state, *xf = di + p.d_init, *yf = xf + p.factor, *u = yf + p.factor, *w = u + p.token,
          *sums = w + p.token;
    float *d_init = own_d_init ? di : r.d_initial_state;
    const dim3 grid((unsigned)p.segs, (unsigned)a.heads);
    hipError_t e;
    if (p.segs > 1) {
        const Own ox = {k, v, a.initial_state, x, xf, 1.0f}, oy = {q, d, r.d_final_state, y, yf, a.scale};
        lin_bwd_state_kernel<DT, KD, VD><<<dim3(grid.x, grid.y, 2), THREADS<VD>, 0, st>>>(b, ox, oy);
        if ((e = hipGetLastError())) return e;
        lin_bwd_join_kernel<KD * VD><<<dim3(KD * VD / JOIN_THREADS, grid.y, 2), JOIN_THREADS, 0, st>>>(b, x, xf, y, yf);
        if ((e = hipGetLastError())) return e;
    }
    // dq on X^T, dk on Y^T: their states' rows are value elements
    const Walk wq = {d, v, k, r.dq, x, a.initial_state, nullptr, a.scale, a.scale, 1.0f, q, u};
    const Walk wv = {k, q, d, r.dv, y, r.d_final_state, d_init, a.scale, 1.0f, a.scale, none, nullptr};
    const Walk wk = {v, d, q, r.dk, y, r.d_final_state, nullptr, a.scale, 1.0f, a.scale, k, w};
    lin_dq_kernel<DT, VD, KD><<<grid, THREADS<KD>, 0, st>>>(b, wq, err);
    if ((e = hipGetLastError())) return e;
    lin_dv_kernel<DT, KD, VD><<<grid, THREADS<VD>, 0, st>>>(b, wv);
    if ((e = hipGetLastError())) return e;
    lin_dk_kernel<DT, VD, KD><<<grid, THREADS<KD>, 0, st>>>(b, wk);
    if ((e = hipGetLastError())) return e;
    const Decays dec = {q, k, v, d, x, y, a.initial_state, d_init, u, w, a.g_per_head ? sums : r.dg, a.scale, a.g_per_head};
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
