// ops_lin.hip -- linear attention with a decay for each head: prompts (a pass for what segments of the time axis add to
// their states, a join, the walk over the chunks; ops_lin.hpp) and single tokens.
#include "ops_lin.hpp"

namespace kda {
namespace ops {
namespace lin {
namespace {

template <int DT, int KD, int VD>
__global__ __launch_bounds__(THREADS<VD>, WAVES<VD> / 2) void lin_state_kernel(const Batch b, const Own a) {
    __shared__ OwnLds<DT, KD, VD> lds;
    own_state<DT, KD, VD, false>(b, a, lds);
}

template <int SIZE, int AHEAD>
__global__ __launch_bounds__(JOIN_THREADS) void lin_join_kernel(const Batch b, float *state, const float *factor) {
    join<SIZE, AHEAD>(b, state, factor, false);
}

template <int DT, int KD, int VD>
__global__ __launch_bounds__(THREADS<VD>, (WAVES_A_SIMD<DT, VD>)) void lin_walk_kernel(const Batch b, const Walk a, int32_t *err) {
    __shared__ WalkLds<DT, KD, VD> lds;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(b.offsets(), err, threadIdx.x, THREADS<VD>);
    const int seg = (int)blockIdx.x / b.turns;
    const Place place = {seg, (int)blockIdx.y, (int)blockIdx.x - seg * b.turns, (int)blockIdx.x, (int)gridDim.x, 0};
    if (__syncthreads_or(walk<DT, KD, VD, false, false>(b, a, place, lds))) {      // a value was not finite
        // (other strides as far as the compiler knows: rows' places that it keeps for this walk through the first cost that 5%)
        Walk again = a;
        asm volatile("" : "+s"(again.q.row), "+s"(again.k.row), "+s"(again.v.row));
        walk<DT, KD, VD, false, false, true>(b, again, place, lds);
    }
}

// One token of each sequence: S <- e^g S + k v^T, out = scale S^T q. The state is read and written once; a block takes one
// head of one sequence, a thread 4 value columns of every GROUPS-th row. Bound by memory: 256 sequences of 32 heads of 128 x
// 128 move 1.08 GB in 207 us, 5.2 TB/s (a copy reaches 5.4).
constexpr int DECODE_THREADS = 256;
template <int DT, int KD, int VD>
__global__ __launch_bounds__(DECODE_THREADS) void lin_decode_kernel(const kda_lin_args a) {
    using E = typename Elem<DT>::type;
    constexpr int COLS = VD / 4, GROUPS = DECODE_THREADS / COLS, ROWS = KD / GROUPS;
    __shared__ float q[KD], k[KD];
    __shared__ f32x4 part[GROUPS][COLS];
    const int n = blockIdx.x, h = blockIdx.y, x = threadIdx.x % COLS, grp = threadIdx.x / COLS;
    const int64_t at = ((int64_t)n * a.heads + h) * (KD * VD);
    f32x4 S[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        S[r] = f32x4{0, 0, 0, 0};
        if (a.initial_state) S[r] = *reinterpret_cast<const f32x4 *>(a.initial_state + at + (r * GROUPS + grp) * VD + 4 * x);
    }
    if (threadIdx.x < KD) q[threadIdx.x] = (float)((const E *)a.q)[n * a.q_stride + h * a.q_head_stride + threadIdx.x] * a.scale;
    else if (threadIdx.x < 2 * KD) k[threadIdx.x - KD] = (float)((const E *)a.k)[n * a.k_stride + h * a.k_head_stride + threadIdx.x - KD];
    typedef E E4 __attribute__((ext_vector_type(4)));
    const E4 ve = *reinterpret_cast<const E4 *>((const E *)a.v + n * a.v_stride + h * a.v_head_stride + 4 * x);
    f32x4 v, o = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)ve[e];
    const float decay = exp2_f((float)log2_decay(a.g[a.g_per_head ? h : (int64_t)n * a.heads + h]));
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = r * GROUPS + grp;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[r][e] = __builtin_fmaf(decay, S[r][e], k[row] * v[e]);
            o[e] = __builtin_fmaf(q[row], S[r][e], o[e]);
        }
        if (a.final_state) *reinterpret_cast<f32x4 *>(a.final_state + at + row * VD + 4 * x) = S[r];
    }
    part[grp][x] = o;
    __syncthreads();
    if (threadIdx.x < COLS) {
#pragma unroll
        for (int p = 1; p < GROUPS; ++p) o += part[p][x];
        E4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = (E)o[i];
        *reinterpret_cast<E4 *>((E *)a.out + ((int64_t)n * a.heads + h) * VD + 4 * x) = e;
    }
}

struct Plan {
    int seg, segs;
};
// A block a segment and head, as many as run at once: 8192 tokens of 32 heads in bf16 (two blocks a CU) 131 us with 512, 135 with
// 256, 150 with 1024; 9442 ragged ones of 5 in fp16 (one a CU) 48 us with 256, 59 with 512.
// Few chunks are walked one after another, which takes one launch for three (us a call, 2 | 64 heads: 128 tokens 15.2 | 15.4 for 21.0 | 21.6,
// 256 tokens 20.8 | 22.5 for 21.3 | 31.4, 512 tokens, which stay with three, 37.0 | 39.2 for 21.4 | 49.7).
constexpr int MOST = 512, FEW = 4;
Plan plan(int64_t T, int64_t H, int64_t chunks, int64_t blocks) {
    Plan p;
    p.seg = chunks <= FEW ? FEW * C : segment(T, H, blocks, C);
    p.segs = (int)ceil_div(T > 0 ? T : 1, p.seg);
    return p;
}

template <int DT, int KD, int VD> hipError_t forward(const kda_lin_args &a, float *ws, int32_t *err, hipStream_t st) {
    static_assert(RUN<DT, KD, VD> <= MOST, "the workspace holds the states of as many segments");
    const int64_t chunks = ceil_div(a.total_tokens, C) + a.num_seqs - 1;      // at most
    const Plan p = plan(a.total_tokens, a.heads, chunks, RUN<DT, KD, VD>);
    const Batch b = {a.cu_seqlens, a.g, a.g_per_head ? 0 : a.heads, a.num_seqs, a.total_tokens, a.heads, p.seg, p.segs, turns(a.num_seqs, p.segs)};
    const Role q = {a.q, a.q_stride, a.q_head_stride}, k = {a.k, a.k_stride, a.k_head_stride}, v = {a.v, a.v_stride, a.v_head_stride};
    const dim3 grid((unsigned)p.segs, (unsigned)a.heads);
    if (p.segs > 1) {
        float *factor = ws + (size_t)p.segs * a.heads * (KD * VD);
        const Own own = {k, v, a.initial_state, ws, factor, 1.0f};
        lin_state_kernel<DT, KD, VD><<<grid, THREADS<VD>, 0, st>>>(b, own);
        if (hipError_t e = hipGetLastError()) return e;
        const dim3 join(KD * VD / JOIN_THREADS, (unsigned)a.heads);
        if (far_ahead(p.segs)) lin_join_kernel<KD * VD, 32><<<join, JOIN_THREADS, 0, st>>>(b, ws, factor);
        else lin_join_kernel<KD * VD, 8><<<join, JOIN_THREADS, 0, st>>>(b, ws, factor);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const Walk w = {q, k, v, a.out, ws, a.initial_state, a.final_state, a.scale, a.scale, 1.0f, {nullptr, 0, 0}, nullptr, nullptr, nullptr, nullptr};
    lin_walk_kernel<DT, KD, VD><<<dim3(grid.x * b.turns, grid.y), THREADS<VD>, 0, st>>>(b, w, err);
    return hipGetLastError();
}

template <int DT, int KD, int VD> hipError_t decode(const kda_lin_args &a, hipStream_t st) {
    lin_decode_kernel<DT, KD, VD><<<dim3((unsigned)a.num_seqs, (unsigned)a.heads), DECODE_THREADS, 0, st>>>(a);
    return hipGetLastError();
}

template <int DT> hipError_t forward_dt(const kda_lin_args &a, float *ws, int32_t *err, hipStream_t st) {
    if (a.key_dim == 64) return a.value_dim == 64 ? forward<DT, 64, 64>(a, ws, err, st) : forward<DT, 64, 128>(a, ws, err, st);
    return a.value_dim == 64 ? forward<DT, 128, 64>(a, ws, err, st) : forward<DT, 128, 128>(a, ws, err, st);
}
template <int DT> hipError_t decode_dt(const kda_lin_args &a, hipStream_t st) {
    if (a.key_dim == 64) return a.value_dim == 64 ? decode<DT, 64, 64>(a, st) : decode<DT, 64, 128>(a, st);
    return a.value_dim == 64 ? decode<DT, 128, 64>(a, st) : decode<DT, 128, 128>(a, st);
}

}  // namespace
}  // namespace lin

size_t lin_workspace(int64_t T, int64_t H, int64_t KD, int64_t VD) {
    const lin::Plan p = lin::plan(T, H, lin::FEW + 1, lin::MOST);      // (fewer blocks, few chunks: fewer segments)
    return p.segs > 1 ? (size_t)p.segs * H * (KD * VD + 1) * sizeof(float) : 0;
}

hipError_t launch_lin_fwd(const kda_lin_args &a, float *ws, int32_t *err, hipStream_t st) {
    return a.dtype == KDA_DTYPE_BF16 ? lin::forward_dt<KDA_DTYPE_BF16>(a, ws, err, st) : lin::forward_dt<KDA_DTYPE_F16>(a, ws, err, st);
}

hipError_t launch_lin_decode(const kda_lin_args &a, hipStream_t st) {
    return a.dtype == KDA_DTYPE_BF16 ? lin::decode_dt<KDA_DTYPE_BF16>(a, st) : lin::decode_dt<KDA_DTYPE_F16>(a, st);
}

}  // namespace ops
}  // namespace kda
