// ops_attn.hpp -- what the attentions of one new token over a paged cache share: probabilities split in two,
// the layout of all sequences' tokens in chunks, the join of chunks (ops_attn.hip, ops_attn_fp4.hip).
#pragma once

#include "ops_common.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace attn {
namespace {

constexpr int WAVES = 4;
constexpr int TILE = 32;                  // tokens of a wave at a time
constexpr int ROUND = WAVES * TILE;       // tokens of a block at a time
constexpr float NEG_INF = -__builtin_inff();

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// UP: what probabilities (0 to 1) are multiplied by before they are split. fp16 ends at 2^-24 below, and with a
// largest score 10 above the rest (one token that draws the attention) the many small probabilities beside it would
// lose their digits there, at 17 above it themselves; times 2^15 they fill fp16's range up to its top. The
// factor, a power of two, leaves with the wave's results.
template <int DT> struct Ops;
template <> struct Ops<KDA_DTYPE_BF16> {
    typedef __bf16 x8 __attribute__((ext_vector_type(8)));
    typedef __bf16 x2 __attribute__((ext_vector_type(2)));
    using E = __bf16;
    static constexpr float UP = 1.0f;
    static constexpr uint32_t EXPONENT = 0x7f80;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
};
template <> struct Ops<KDA_DTYPE_F16> {
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
    typedef _Float16 x2 __attribute__((ext_vector_type(2)));
    using E = _Float16;
    static constexpr float UP = 32768.0f;
    static constexpr uint32_t EXPONENT = 0x7c00;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    }
};

// Two probabilities to a rounded pair and the pair of what rounding left. RAISED: a rounded part is at least
// the type's smallest normal number where the probability is not zero (what is left may then be negative).
template <int DT, bool RAISED> __device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    using x2 = typename Ops<DT>::x2;
    using E = typename Ops<DT>::E;
    x2 h = {(E)a, (E)b};
    if constexpr (RAISED && DT == KDA_DTYPE_F16) {      // in bf16 they share fp32's range
        constexpr float LEAST = 0x1p-14f;
        h = {(E)(a > 0.0f ? __builtin_fmaxf(a, LEAST) : a), (E)(b > 0.0f ? __builtin_fmaxf(b, LEAST) : b)};
    }
    const x2 l = {(E)(a - (float)h[0]), (E)(b - (float)h[1])};
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, l);
}

// Pairs of values with infinities and NaN put to zero: their exponent is all ones.
template <int DT> __device__ __forceinline__ u32x4 finite_of(u32x4 x) {
    constexpr uint32_t LO = Ops<DT>::EXPONENT, HI = LO << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] &= ((x[i] & LO) == LO ? 0u : 0xffffu) | ((x[i] & HI) == HI ? 0u : 0xffff0000u);
    return x;
}

// maximum and sum over a lane's column (its four 16-lane rows)
__device__ __forceinline__ float column_max(float x) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float x) {
    x = swap16_add(x, x);
    return swap32_add(x, x);
}

// What a sequence holds: its length, at most what its row of the table can address.
__device__ __forceinline__ int seq_len(const kda_attn_args &a, int s) {
    const int64_t most = (int64_t)a.table_width * a.page_size;
    const int n = a.seq_lens[s];
    return n < 0 ? 0 : n > most ? (int)most : n;
}

__device__ __forceinline__ int64_t wave_sum64(int64_t x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    return x;
}

struct Work {
    int seq, slot;        // slot: where the chunk's partial result lies
    bool whole;           // the sequence's only chunk
    int begin, end;       // its tokens
};

// Tokens of a chunk: all tokens over `spread` chunks, whole tiles, at least min_chunk.
__device__ __forceinline__ int chunk_len(int64_t total, int spread, int min_chunk) {
    const int64_t c = (total + spread - 1) / spread;
    const int64_t r = (c + TILE - 1) / TILE * TILE;
    return r < min_chunk ? min_chunk : (int)(r < (1 << 30) ? r : 1 << 30);
}
// A sequence's full chunks; what is left (or all of a sequence without any) is one chunk more.
__device__ __forceinline__ int full_of(int len, int chunk) { return len / chunk; }
__device__ __forceinline__ bool rest_of(int len, int chunk) { return len % chunk != 0 || len == 0; }

// The chunk of index `slot`, found by every wave for itself; false past the last. Indexes count the full
// chunks of all sequences in order, then the rests: blocks start in that order, the short ones last.
__device__ __forceinline__ bool find_work(const kda_attn_args &a, int slot, int spread, int min_chunk, Work &w) {
    const int lane = threadIdx.x & 63;
    int64_t total = 0;
    for (int s = lane; s < a.num_seqs; s += 64) total += seq_len(a, s);
    const int chunk = chunk_len(wave_sum64(total), spread, min_chunk);
    w.slot = slot;
    int before = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass)
        for (int s0 = 0; s0 < a.num_seqs; s0 += 64) {
            const int s = s0 + lane;
            const int len = s < a.num_seqs ? seq_len(a, s) : 0;
            const int full = full_of(len, chunk);
            const int mine = s >= a.num_seqs ? 0 : pass == 0 ? full : rest_of(len, chunk);
            int upto = mine;      // inclusive sum over lanes
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(upto, d);
                if (lane >= d) upto += v;
            }
            const int all = __shfl(upto, 63);
            if (slot < before + all) {
                const uint64_t at = __ballot(before + upto > slot);
                const int l = __builtin_ctzll(at);
                const int n = __shfl(len, l), f = __shfl(full, l);
                const int part = pass == 0 ? slot - (before + __shfl(upto, l) - f) : f;
                w.seq = s0 + l;
                w.whole = f + (rest_of(n, chunk) ? 1 : 0) == 1;
                w.begin = part * chunk;
                w.end = pass == 0 ? w.begin + chunk : n;
                return true;
            }
            before += all;
        }
    return false;
}

// Blocks that all tokens are spread over: 768 run at once at head dimension 128, three to each of 256 CUs (166 registers allow
// three waves a SIMD). Measured on MI355X (us, 512 | 768 | 1024 | 1536): 1 x 65536 tokens, 32 heads over 8, 58.9 | 61.3 |
// 61.8 | 65.8; 64 skewed sequences fp16, 32 heads over 4, 92.5 | 90.2 | 87.6 | 88.7: fewer blocks suit one long sequence (fewer
// chunks to join), more of them skewed ones, and what lies between loses 4% and 3% to the best of each.
constexpr int SPREAD = 768, MAX_SPREAD = 1024, MAX_PARTS = MAX_SPREAD + 1;

// Joins the chunks of one (sequence, head), in their order, where there are several: threads take four
// elements each, groups of threads every GROUPS-th chunk. 1 x 65536 tokens, 32 heads: 97 chunks in 6.8 us, two rounds
// of loads' latency.
template <int DT, int DH>
__global__ __launch_bounds__(256) void attn_join_kernel(const kda_attn_args a, const float *acc, const float *ml, int spread,
                                                        int min_chunk) {
    using E = typename Ops<DT>::E;
    constexpr int LANES = DH / 4, GROUPS = 256 / LANES;
    __shared__ float weight[MAX_PARTS];
    __shared__ f32x4 part[256];
    const int s = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63;
    int64_t total = 0;
    for (int q = lane; q < a.num_seqs; q += 64) total += seq_len(a, q);
    const int chunk = chunk_len(wave_sum64(total), spread, min_chunk);
    const int len = seq_len(a, s), full = full_of(len, chunk), parts = full + (rest_of(len, chunk) ? 1 : 0);
    if (parts == 1) return;
    // where its full chunks begin, and its rest: after everyone's full chunks and the rests before it
    int64_t first = 0, rest = 0;
    for (int q = lane; q < a.num_seqs; q += 64) {
        const int n = seq_len(a, q), f = full_of(n, chunk);
        first += q < s ? f : 0;
        rest += f + (q < s && rest_of(n, chunk) ? 1 : 0);
    }
    first = wave_sum64(first), rest = wave_sum64(rest);
    const int64_t step = (int64_t)a.q_heads * 2;
    auto stat_of = [&](int p) { return ml + (p < full ? first + p : rest) * step + 2 * h; };
    float M = NEG_INF, L = 0.0f;
    for (int p = lane; p < parts; p += 64) M = __builtin_fmaxf(M, stat_of(p)[0]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) M = __builtin_fmaxf(M, __shfl_xor(M, d));
    const float ref = M == NEG_INF ? 0.0f : M;
    for (int p = lane; p < parts; p += 64) {       // every wave the whole sum, the first one the weights
        const float *st = stat_of(p);
        const float w = exp2_f(st[0] - ref);
        if (threadIdx.x < 64) weight[p] = w;
        L += st[1] * w;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) L += __shfl_xor(L, d);
    __syncthreads();
    const int grp = threadIdx.x / LANES, x = threadIdx.x % LANES;
    const f32x4 *from = reinterpret_cast<const f32x4 *>(acc) + (int64_t)h * LANES + x;
    const int64_t row = (int64_t)a.q_heads * LANES;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll 8
    for (int p = grp; p < parts; p += GROUPS) o += from[(p < full ? first + p : rest) * row] * weight[p];
    part[threadIdx.x] = o;
    __syncthreads();
    if (threadIdx.x < LANES) {
#pragma unroll
        for (int q = 1; q < GROUPS; ++q) o += part[q * LANES + x];
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        E *to = reinterpret_cast<E *>(a.out) + ((int64_t)s * a.q_heads + h) * DH + 4 * x;
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = (E)(o[e] * inv);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)s * a.q_heads + h] = L == 0.0f ? NEG_INF : (ref + __builtin_log2f(L)) * LN2_F;
}

// The host's part of the plan: how many chunks all tokens are spread over, how many there can be,
// and whether any sequence can have more than one.
struct Plan {
    int spread, slots, min_chunk, tiles_h;
    bool join;
};
// run: blocks that run at once where that is more than SPREAD, or 0. Chunks of rests come on top of those that tokens are spread over, one
// a sequence, so that they are taken off, but for three quarters of `run` that are always there.
inline Plan plan(int64_t B, int64_t hq, int64_t hkv, int64_t width, int64_t page, int64_t run = 0) {
    Plan p;
    p.tiles_h = (int)ceil_div(hq / hkv, 16);
    const int64_t per = hkv * p.tiles_h;
    p.min_chunk = 2 * ROUND;
    const int64_t most = width * page;
    int64_t spread = ceil_div(SPREAD, per);
    if (run / per - B > spread) spread = run / per - B;
    p.spread = (int)spread;
    p.join = most > p.min_chunk;
    // sum of ceil(len / chunk) <= spread + B, and no sequence has more than its table allows
    const int64_t by_len = B * ceil_div(most > 0 ? most : 1, p.min_chunk);
    p.slots = (int)(spread + B < by_len ? spread + B : by_len);
    return p;
}

}  // namespace
}  // namespace attn
}  // namespace ops
}  // namespace kda
