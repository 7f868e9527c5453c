// ops_attn.hip -- attention of one new token per sequence over a paged key-value cache, split
// over the cache's length and joined.
//
//   out[h] = sum_t softmax_t(scale q[h].k_t) v_t over the len cached tokens of the sequence, in
//   one pass with the running maximum and sum; lse[h] = log sum_t e^{scale q[h].k_t}
//
// Bound by the bytes of the cache, each read once for every 16 query heads that share a cache head (8 x 4096
// tokens of 128 bf16: 64 heads over 1 take 22.0 us, as long as over 4). A wave takes 32 tokens of one
// key-value head at a time, for up to 16 query heads that share it:
//  * S^T = K Q^T (v_mfma_f32_16x16x32: rows tokens, columns heads). A lane holds the scores of one
//    head for 8 tokens, so maxima and sums are lane-local but for two exchanges between the
//    wave's four 16-lane rows.
//  * O^T = V^T P^T. P leaves S^T in the very lanes its operand wants (the 32 tokens of the
//    contraction are relabelled: slot 8 g + i is token 4 g + i for i < 4, 16 + 4 g + i - 4 else), split
//    into a rounded part and the rest, two products, so that P does not lose what the output
//    keeps: 2^-16 of a probability in bf16; 2^-22 in fp16, or 2^-40 of the wave's largest one. V's operand holds 8 tokens of one element: a lane loads DV neighbouring elements
//    of 8 tokens (whole rows of the cache per instruction) and pairs the tokens' halves up with
//    byte permutes. Neither K nor V passes through LDS.
//  * The result has a head's elements in its own lanes, so rescaling needs no exchange.
// Blocks take chunks of one sequence's tokens. Every block works the chunk length out from all
// lengths (on the device: the host does not know them), so that skewed batches spread evenly and a
// captured launch stays right when lengths change. Chunks' partial results go to the workspace;
// attn_join_kernel joins them in their order. A sequence of one chunk is written at once.
#include <type_traits>

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

// Row offsets (elements, from the caches' bases) of 32 tokens, and which of them are there.
struct Rows {
    int64_t k[TILE], v[TILE];
};

// 1 x 65536 tokens, 32 heads over 8, bf16: 268 MB in 44 to 54 us, 5.0 to 6.1 TB/s; 64 skewed sequences, 32 heads over 4, fp16: 364
// MB in 80 us, 4.5 TB/s; 256 x 1024 tokens, 32 heads over 8, bf16: 1.07 GB in 210 us, 5.1 TB/s. Every wave finds its chunk
// from all lengths, which shows from about a thousand sequences on: 1024 x 16 tokens, 32 heads over 8, 195 us for 67 MB.
template <int DT, int DH>
__global__ __launch_bounds__(64 * WAVES) void attn_chunk_kernel(const kda_attn_args a, float *acc_out, float *ml_out,
                                                                int32_t *err, int spread, int min_chunk, int tiles_h) {
    using O = Ops<DT>;
    using E = typename O::E;
    constexpr int KD = DH / 32;      // 32-element steps of a score
    constexpr int DV = DH / 16;      // elements of a lane in O^T's operand rows
    __shared__ Rows rows[WAVES][2];
    __shared__ float join[WAVES][16 * (DH + 4)];
    __shared__ float stat[WAVES][16][2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int per = a.kv_heads * tiles_h;
    const int slot = blockIdx.x / per, rest = blockIdx.x - slot * per;
    const int kvh = rest / tiles_h, ht = rest - kvh * tiles_h;
    Work w;
    if (!find_work(a, slot, spread, min_chunk, w)) return;
    const int seq = __builtin_amdgcn_readfirstlane(w.seq);
    const int begin = __builtin_amdgcn_readfirstlane(w.begin), end = __builtin_amdgcn_readfirstlane(w.end);
    if (err && w.begin == 0 && rest == 0 && threadIdx.x == 0) {
        const int n = a.seq_lens[seq];
        if (n < 0 || n > (int64_t)a.table_width * a.page_size) atomicOr(err, KDA_DEVERR_PAGES);
    }
    const int group = a.q_heads / a.kv_heads;
    const int heads = group - ht * 16 < 16 ? group - ht * 16 : 16;      // of this block
    const int head0 = kvh * group + ht * 16;
    u32x4 q[KD];
#pragma unroll
    for (int k = 0; k < KD; ++k) {
        q[k] = u32x4{0, 0, 0, 0};
        if (i < heads)
            q[k] = *reinterpret_cast<const u32x4 *>((const E *)a.q + seq * a.q_stride + (int64_t)(head0 + i) * a.q_head_stride +
                                                    32 * k + 8 * g);
    }
    const float scale = a.scale * LOG2E_F;
    f32x4 acc[DV];
    float m, l;
    const int32_t *table = a.block_table + (int64_t)seq * a.table_stride;
    const E *kc = (const E *)a.k_cache + (int64_t)kvh * a.k_head_stride;
    const E *vc = (const E *)a.v_cache + (int64_t)kvh * a.v_head_stride;
    Rows *const R = rows[wave];
    bool bad = false;

    u32x4 kr[2][KD];
    uint32_t vr[8][DV / 2];
    // Page numbers are fetched two tiles ahead, a tile's rows are placed one tile ahead; its keys are
    // loaded once the scores before them have used theirs, its values likewise: the registers that a
    // tile leaves carry the loads of the next.
    auto page_of = [&](int t0) {
        const int t = t0 + (lane & 31), tc = t < end ? t : end - 1;
        return table[tc / a.page_size];
    };
    // every lane one token (the upper half of the wave repeats the lower): its page, checked
    auto place = [&](int t0, int page, int turn) {
        const int t = t0 + (lane & 31), tc = t < end ? t : end - 1;
        const int at = tc - tc / a.page_size * a.page_size;
        bool there = t < end;
        if (page < 0 || page >= a.num_pages) bad = true, there = false, page = 0;
        if (lane < 32) R[turn].k[lane] = (int64_t)page * a.k_page_stride + (int64_t)at * a.k_token_stride;
        else R[turn].v[lane - 32] = (int64_t)page * a.v_page_stride + (int64_t)at * a.v_token_stride;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        return (uint32_t)__ballot(there);
    };
    auto load_k = [&](int turn) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const E *row = kc + R[turn].k[16 * h + i] + 8 * g;
#pragma unroll
            for (int k = 0; k < KD; ++k) kr[h][k] = *reinterpret_cast<const u32x4 *>(row + 32 * k);
        }
    };
    auto load_v = [&](int turn) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int tok = (s < 4 ? 0 : 12) + 4 * g + s;
            const E *row = vc + R[turn].v[tok] + DV * i;
            if constexpr (DV == 4) {
                const uint2 x = *reinterpret_cast<const uint2 *>(row);
                vr[s][0] = x.x, vr[s][1] = x.y;
            } else {
#pragma unroll
                for (int c = 0; c < DV / 8; ++c) {
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(row + 8 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) vr[s][4 * c + e] = x[e];
                }
            }
        }
    };
    // One pass over the wave's tokens. An infinite value times a rest that is zero or negative would make NaN of
    // an infinite result. Nothing is spent on that in the first pass; where it ends with a NaN, a second one
    // keeps values that are not finite out of the product with the rest (that with the rounded part gives
    // what they give), and lets no rounded part be zero that stands for a positive probability.
    auto walk = [&](auto careful) {
        constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
        for (int d = 0; d < DV; ++d) acc[d] = f32x4{0, 0, 0, 0};
        m = NEG_INF, l = 0.0f;
        int t0 = begin + wave * TILE, turn = 0, ahead = 0;
        uint32_t seen = 0;
        if (t0 < end) {
            seen = place(t0, page_of(t0), 0);
            load_k(0);
            load_v(0);
            if (t0 + ROUND < end) ahead = page_of(t0 + ROUND);
        }
        for (; t0 < end; t0 += ROUND, turn ^= 1) {
            const bool more = t0 + ROUND < end;
            uint32_t then = 0;
            if (more) {
                then = place(t0 + ROUND, ahead, turn ^ 1);
                if (t0 + 2 * ROUND < end) ahead = page_of(t0 + 2 * ROUND);
            }
            f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int k = 0; k < KD; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) st[h] = O::mma(kr[h][k], q[k], st[h]);
            if (more) load_k(turn ^ 1);
            // this lane's tokens: 4 g + j and 16 + 4 g + j
            float sc[8], top = NEG_INF;
            const uint32_t mine = (seen >> (4 * g)) & 0xf000f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const bool on = (mine >> ((s < 4 ? 0 : 12) + s)) & 1;
                sc[s] = on ? st[s >> 2][s & 3] * scale : NEG_INF;
                top = __builtin_fmaxf(top, sc[s]);
            }
            const float mn = __builtin_fmaxf(m, column_max(top));
            if (__any(mn > m)) {
                const float f = mn > m ? exp2_f(m - mn) : 1.0f;      // m may be -inf: 0
                l *= f;
#pragma unroll
                for (int d = 0; d < DV; ++d) acc[d] *= f;
                m = mn;
            }
            const float ref = m == NEG_INF ? 0.0f : m;
            float p[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                p[s] = exp2_f(sc[s] - ref);
                l += p[s];
            }
            u32x4 hi, lo;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t x, y;
                split_pair<DT, CAREFUL>(p[2 * s] * O::UP, p[2 * s + 1] * O::UP, x, y);
                hi[s] = x, lo[s] = y;
            }
            if (seen != 0xffffffffu) {          // rows that are not there may hold anything: 0 x NaN
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const bool on = (mine >> ((s < 4 ? 0 : 12) + s)) & 1;
#pragma unroll
                    for (int e = 0; e < DV / 2; ++e) vr[s][e] = on ? vr[s][e] : 0u;
                }
            }
#pragma unroll
            for (int e = 0; e < DV / 2; ++e) {
                u32x4 even, odd;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    even[s] = __builtin_amdgcn_perm(vr[2 * s + 1][e], vr[2 * s][e], 0x05040100);
                    odd[s] = __builtin_amdgcn_perm(vr[2 * s + 1][e], vr[2 * s][e], 0x07060302);
                }
                acc[2 * e] = O::mma(even, hi, acc[2 * e]);
                acc[2 * e + 1] = O::mma(odd, hi, acc[2 * e + 1]);
                if constexpr (CAREFUL) even = finite_of<DT>(even), odd = finite_of<DT>(odd);
                acc[2 * e] = O::mma(even, lo, acc[2 * e]);
                acc[2 * e + 1] = O::mma(odd, lo, acc[2 * e + 1]);
            }
            if (more) load_v(turn ^ 1);
            seen = then;
        }
    };
    walk(std::false_type{});
    bool nan = false;
#pragma unroll
    for (int d = 0; d < DV; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) nan |= acc[d][j] != acc[d][j];
    if (__any(nan)) walk(std::true_type{});
    if (err && __any(bad) && lane == 0) atomicOr(err, KDA_DEVERR_PAGES);
    l = column_sum(l);

    // the waves' results, against the block's largest maximum
    if (g == 0) stat[wave][i][0] = m, stat[wave][i][1] = l;
    __syncthreads();
    float M = NEG_INF, L = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) M = __builtin_fmaxf(M, stat[v][i][0]);
    const float ref = M == NEG_INF ? 0.0f : M;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) L += stat[v][i][1] * exp2_f(stat[v][i][0] - ref);
    const float f = exp2_f(m - ref) * (1.0f / O::UP);
    // O^T: element DV (4 g + j) + d of head i
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < DV; ++d) join[wave][i * (DH + 4) + DV * (4 * g + j) + d] = acc[d][j] * f;
    __syncthreads();
    const bool whole = w.whole;
    for (int x = threadIdx.x; x < heads * DH; x += 64 * WAVES) {
        const int h = x / DH, d = x - h * DH;
        float o = 0.0f;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) o += join[v][h * (DH + 4) + d];
        if (whole) {
            float hm = NEG_INF, hl = 0.0f;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) hm = __builtin_fmaxf(hm, stat[v][h][0]);
            const float hr = hm == NEG_INF ? 0.0f : hm;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) hl += stat[v][h][1] * exp2_f(stat[v][h][0] - hr);
            reinterpret_cast<E *>(a.out)[((int64_t)seq * a.q_heads + head0 + h) * DH + d] = (E)(hl == 0.0f ? 0.0f : o / hl);
        } else acc_out[((int64_t)w.slot * a.q_heads + head0 + h) * DH + d] = o;
    }
    if (threadIdx.x < heads) {      // wave 0: lane i is head i
        if (whole) {
            if (a.lse) a.lse[(int64_t)seq * a.q_heads + head0 + i] = L == 0.0f ? NEG_INF : (ref + __builtin_log2f(L)) * LN2_F;
        } else {
            float *ml = ml_out + ((int64_t)w.slot * a.q_heads + head0 + i) * 2;
            ml[0] = M, ml[1] = L;
        }
    }
}

// Blocks that all tokens are spread over: 768 run at once at head dimension 128, three to each of 256 CUs (166 registers allow
// three waves a SIMD). Measured on MI355X (us, 512 | 768 | 1024 | 1536): 1 x 65536 tokens, 32 heads over 8, 58.9 | 61.3 |
// 61.8 | 65.8; 64 skewed sequences fp16, 32 heads over 4, 92.5 | 90.2 | 87.6 | 88.7: fewer blocks suit one long sequence (fewer
// chunks to join), more of them skewed ones, and what lies between loses 4% and 3% to the best of each.
constexpr int SPREAD = 768, MAX_PARTS = SPREAD + 1;

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
Plan plan(int64_t B, int64_t hq, int64_t hkv, int64_t width, int64_t page) {
    Plan p;
    p.tiles_h = (int)ceil_div(hq / hkv, 16);
    const int64_t per = hkv * p.tiles_h;
    p.min_chunk = 2 * ROUND;
    const int64_t most = width * page;
    const int64_t spread = ceil_div(SPREAD, per);
    p.spread = (int)spread;
    p.join = most > p.min_chunk;
    // sum of ceil(len / chunk) <= spread + B, and no sequence has more than its table allows
    const int64_t by_len = B * ceil_div(most > 0 ? most : 1, p.min_chunk);
    p.slots = (int)(spread + B < by_len ? spread + B : by_len);
    return p;
}

template <int DT, int DH>
hipError_t run(const kda_attn_args &a, const Plan &p, float *acc, float *ml, int32_t *err, hipStream_t st) {
    const int64_t blocks = (int64_t)p.slots * a.kv_heads * p.tiles_h;
    attn_chunk_kernel<DT, DH><<<dim3((unsigned)blocks), 64 * WAVES, 0, st>>>(a, acc, ml, err, p.spread, p.min_chunk, p.tiles_h);
    if (hipError_t e = hipGetLastError()) return e;
    if (p.join) attn_join_kernel<DT, DH><<<dim3((unsigned)a.num_seqs, (unsigned)a.q_heads), 256, 0, st>>>(a, acc, ml, p.spread, p.min_chunk);
    return hipGetLastError();
}

template <int DT> hipError_t run_dt(const kda_attn_args &a, const Plan &p, float *acc, float *ml, int32_t *err, hipStream_t st) {
    if (a.head_dim == 64) return run<DT, 64>(a, p, acc, ml, err, st);
    if (a.head_dim == 128) return run<DT, 128>(a, p, acc, ml, err, st);
    return run<DT, 256>(a, p, acc, ml, err, st);
}

}  // namespace
}  // namespace attn

size_t attn_workspace(int64_t B, int64_t hq, int64_t hkv, int64_t dh, int64_t width, int64_t page) {
    const attn::Plan p = attn::plan(B, hq, hkv, width, page);
    return p.join ? (size_t)p.slots * hq * (dh + 2) * sizeof(float) : 0;
}

hipError_t launch_attn_decode(const kda_attn_args &a, float *ws, int32_t *err, hipStream_t st) {
    const attn::Plan p = attn::plan(a.num_seqs, a.q_heads, a.kv_heads, a.table_width, a.page_size);
    float *ml = ws ? ws + (size_t)p.slots * a.q_heads * a.head_dim : nullptr;
    if (a.dtype == KDA_DTYPE_BF16) return attn::run_dt<KDA_DTYPE_BF16>(a, p, ws, ml, err, st);
    return attn::run_dt<KDA_DTYPE_F16>(a, p, ws, ml, err, st);
}

}  // namespace ops
}  // namespace kda
