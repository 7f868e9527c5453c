// ops_attn_fp4.hip -- attention of one new token per sequence over a paged key-value cache of 4 bits an element:
// e2m1 codes with one power of two (e8m0) for every 32 elements of a row.
//
//   out[h] = sum_t softmax_t(scale q[h].k_t) v_t,   lse[h] = log sum_t e^{scale q[h].k_t}
//
// A quarter of the bytes of the 16-bit cache (68 for 256 a row of 128) under the same products, so that what a tile
// costs the vector units decides as much as memory does. The layout of the work is ops_attn.hip's: chunks of all
// sequences' tokens, a wave takes 32 tokens of one cache head for up to 16 query heads, S^T = K Q^T, then
// O^T = V^T P^T with P where the first product left it. What the 4 bits change:
//  * v_cvt_scalef32_pk makes two 16-bit values of a byte of codes and applies their scale on the way: exact, as a code
//    has two significant bits and the scale is a power of two. No zero points, no multiplications, and the products run
//    in the type of q.
//  * The contraction of S^T is relabelled: lane group g holds the g-th quarter of a key row, so that a lane loads its
//    part of a key at once (16 bytes of a row of 128) and needs one scale for it (two in rows of 256).
//  * Scales of 32 keys and 32 values come with one load, a lane each, and go through LDS to the lanes that need
//    them; the conversion reads the exponent's bits of its scale operand only, so a scale is one rotation of its word.
// Measured: 1 x 65536 tokens, 32 heads over 8 of 128 (71 MB) 22.9 us, 3.1 TB/s, and the join 7.9 (16 bits: 46-54); 64 skewed
// sequences, 32 heads over 4, fp16 (97 MB) 30.4, 3.2 TB/s; 64 x 4096 tokens (285 MB) 52, 5.5 TB/s. What is short of
// memory's rate is the time in which a block begins and ends: its first pages, keys and values wait for one another.
#include <type_traits>

#include "ops_attn.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace attn {
namespace {

// Two values of byte J of w times 2^(exponent bits of scale).
template <int DT, int J> __device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t scale) {
    const float s = __uint_as_float(scale);
    if constexpr (DT == KDA_DTYPE_BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, J));
    else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, J));
}

template <int BYTES> struct Word;
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };

// w rotated so that its byte b lies at the exponent of a float (bits 23 to 30).
__device__ __forceinline__ uint32_t at_exponent(uint32_t w, uint32_t b) { return __builtin_amdgcn_alignbit(w, w, 8 * b + 9); }

template <int DT, int DH>
__global__ __launch_bounds__(64 * WAVES, (DH == 256 ? 2 : 4)) void attn_fp4_chunk_kernel(const kda_attn_fp4_args f, float *acc_out, float *ml_out,
                                                                    int32_t *err, int spread, int min_chunk, int tiles_h) {
    using O = Ops<DT>;
    using E = typename O::E;
    constexpr int KW = DH / 32;      // words of codes in a lane's part of a key, each a step of 32 of the score's contraction
    constexpr int DV = DH / 16;      // elements of a lane in O^T's operand rows
    constexpr int VW = DV / 8 ? DV / 8 : 1;
    constexpr int ROW = DH / 2;      // bytes of a row
    constexpr int NV = TILE * ROW / 1024;      // 16-byte loads of a lane for a tile of values
    constexpr int SB = DH / 32;      // bytes of a row's scales
    constexpr int SW = SB / 4 ? SB / 4 : 1;
    // What a wave keeps while it walks its tokens, and q; at the end, the waves' results.
    struct Own {
        u32x4 values[TILE * ROW / 16];          // the tile of values
        uint32_t scales[2][SW][TILE];           // of its keys and values
        int64_t places[2][2 * TILE];            // of 32 keys' rows and 32 values', bytes from the caches' bases
    };
    struct Walking {
        u32x4 q[KW][64];
        Own own[WAVES];
    };
    union Lds {
        Walking walking;
        float join[WAVES][16 * (DH + 4)];
    };
    __shared__ Lds lds;
    __shared__ float stat[WAVES][16][2];
    const kda_attn_args &a = f.attn;
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
    // q's operands, kept in LDS: the registers are worth more. A negative scale turns q's signs over, so that the largest
    // product is that of the largest score.
    for (int k = wave; k < KW; k += WAVES) {
        u32x4 q = {0, 0, 0, 0};
        if (i < heads)
            q = *reinterpret_cast<const u32x4 *>((const E *)a.q + seq * a.q_stride + (int64_t)(head0 + i) * a.q_head_stride +
                                                 DH / 4 * g + 8 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] ^= a.scale < 0.0f ? 0x80008000u : 0u;
        lds.walking.q[k][lane] = q;
    }
    __syncthreads();
    const float scale = __builtin_fabsf(a.scale) * LOG2E_F;
    f32x4 acc[DV];
    const int32_t *table = a.block_table + (int64_t)seq * a.table_stride;
    const uint8_t *kc = (const uint8_t *)a.k_cache + (int64_t)kvh * a.k_head_stride;
    const uint8_t *vc = (const uint8_t *)a.v_cache + (int64_t)kvh * a.v_head_stride;
    // this lane's side: the lower half of the wave keys, the upper one values
    const bool keys = lane < 32;
    const uint8_t *sc_base = keys ? f.k_scale + (int64_t)kvh * f.k_scale_head_stride : f.v_scale + (int64_t)kvh * f.v_scale_head_stride;
    const uint32_t to_page = (uint32_t)(keys ? a.k_page_stride : a.v_page_stride);
    const uint32_t to_token = (uint32_t)(keys ? a.k_token_stride : a.v_token_stride);
    const uint32_t sc_page = (uint32_t)(keys ? f.k_scale_page_stride : f.v_scale_page_stride);
    const uint32_t sc_token = (uint32_t)(keys ? f.k_scale_token_stride : f.v_scale_token_stride);
    auto &R = lds.walking.own[wave].places;
    auto &S = lds.walking.own[wave].scales;
    uint8_t *const tile = reinterpret_cast<uint8_t *>(lds.walking.own[wave].values);
    bool bad = false;

    uint32_t kr[2][KW], sr[SW];
    u32x4 vq[NV];
    // Every lane one token of a tile (the upper half of the wave repeats the lower): its page's place in the table and its own in
    // the page, moved on by a round a time without a division.
    struct Spot {
        int page, at;
    };
    const int whole_pages = ROUND / a.page_size, rest_of_round = ROUND - whole_pages * a.page_size;
    auto next_of = [&](Spot s) {
        s.page += whole_pages, s.at += rest_of_round;
        if (s.at >= a.page_size) s.at -= a.page_size, ++s.page;
        return s;
    };
    const int most = (end - 1) / a.page_size;       // the last page in use: those behind it are not read
    auto page_of = [&](Spot s) { return table[s.page < most ? s.page : most]; };
    // Its page, checked, its row and its scales. Rows that are not there stand for finite numbers (scales of 1), which
    // probabilities of 0 take away.
    auto place = [&](int t0, Spot s, int page, int turn) {
        bool there = t0 + (lane & 31) < end;
        if (page < 0 || page >= a.num_pages) bad = true, there = false, page = 0;
        R[turn][lane] = (int64_t)((uint64_t)(uint32_t)page * to_page + (uint64_t)(uint32_t)s.at * to_token);
        const uint8_t *from = sc_base + ((uint64_t)(uint32_t)page * sc_page + (uint64_t)(uint32_t)s.at * sc_token);
        const auto x = *reinterpret_cast<const typename Word<SB>::type *>(from);
        if constexpr (SB == 8) sr[0] = there ? x[0] : 0x7f7f7f7fu, sr[1] = there ? x[1] : 0x7f7f7f7fu;
        else sr[0] = there ? x : 0x7f7f7f7fu;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        return (uint32_t)__ballot(there);
    };
    auto load_k = [&](int turn) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *row = kc + (R[turn][16 * h + i] + DH / 8 * g);
            if constexpr (KW == 2) {
                const uint2 x = *reinterpret_cast<const uint2 *>(row);
                kr[h][0] = x.x, kr[h][1] = x.y;
            } else {
#pragma unroll
                for (int c = 0; c < KW / 4; ++c) {
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(row + 16 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) kr[h][4 * c + e] = x[e];
                }
            }
        }
    };
    // Values are loaded as whole lines (16 bytes a lane, 1 KiB at a time: loads of 4 bytes a lane for 4 tokens each wait in L1 for lines
    // that the load before them asked for) and handed over through LDS, rows in the order in which lanes want them: row
    // 4 s + g is token 4 g + s for s < 4, 16 + 4 g + s - 4 else.
    auto load_v = [&](int turn) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int x = 16 * (64 * n + lane), row = x / ROW, s = row >> 2, tok = 4 * (row & 3) + (s < 4 ? 0 : 12) + s;
            vq[n] = *reinterpret_cast<const u32x4 *>(vc + (R[turn][TILE + tok] + x % ROW));
        }
    };

#pragma unroll
    for (int d = 0; d < DV; ++d) acc[d] = f32x4{0, 0, 0, 0};
    float m = NEG_INF, l = 0.0f;        // the largest product of q and k, before the scale
    int t0 = begin + wave * TILE, turn = 0, ahead = 0;
    uint32_t seen = 0;
    Spot spot;
    spot.page = (t0 + (lane & 31)) / a.page_size, spot.at = t0 + (lane & 31) - spot.page * a.page_size;
    if (t0 < end) {
        seen = place(t0, spot, page_of(spot), 0);
        load_k(0);
        load_v(0);
        spot = next_of(spot);
        if (t0 + ROUND < end) ahead = page_of(spot);
    }
    for (; t0 < end; t0 += ROUND, turn ^= 1) {
        const bool more = t0 + ROUND < end;
        // this tile's scales, to the lanes that need them
#pragma unroll
        for (int c = 0; c < SW; ++c) S[lane >> 5][c][lane & 31] = sr[c];
#pragma unroll
        for (int n = 0; n < NV; ++n) *reinterpret_cast<u32x4 *>(tile + 16 * (64 * n + lane)) = vq[n];
        uint32_t then = 0;
        if (more) {
            then = place(t0 + ROUND, spot, ahead, turn ^ 1);
            load_v(turn ^ 1);
            spot = next_of(spot);
            if (t0 + 2 * ROUND < end) ahead = page_of(spot);
        } else {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t ks[DH == 256 ? 2 : 1];
            if constexpr (DH == 256) {
                const uint32_t word = S[0][g >> 1][16 * h + i];
                ks[0] = at_exponent(word, 2 * (g & 1)), ks[1] = at_exponent(word, 2 * (g & 1) + 1);
            } else
                ks[0] = at_exponent(S[0][0][16 * h + i], DH == 128 ? g : g >> 1);
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const uint32_t x = kr[h][k], s = ks[DH == 256 ? k / 4 : 0];
                const u32x4 row = {pair_of<DT, 0>(x, s), pair_of<DT, 1>(x, s), pair_of<DT, 2>(x, s), pair_of<DT, 3>(x, s)};
                st[h] = O::mma(row, lds.walking.q[k][lane], st[h]);
            }
        }
        if (more) load_k(turn ^ 1);
        // this lane's tokens: 4 g + j and 16 + 4 g + j
        const bool all = seen == 0xffffffffu;
        const uint32_t mine = (seen >> (4 * g)) & 0xf000f;
        if (!all) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (!((mine >> ((s < 4 ? 0 : 12) + s)) & 1)) st[s >> 2][s & 3] = NEG_INF;
        }
        float top = NEG_INF;
#pragma unroll
        for (int s = 0; s < 8; ++s) top = __builtin_fmaxf(top, st[s >> 2][s & 3]);
        const float mn = __builtin_fmaxf(m, column_max(top));
        if (__any(mn > m)) {
            const float r = m == NEG_INF ? 0.0f : mn > m ? exp2_f((m - mn) * scale) : 1.0f;
            l *= r;
#pragma unroll
            for (int d = 0; d < DV; ++d) acc[d] *= r;
            m = mn;
        }
        const float ref = m == NEG_INF ? 0.0f : -m * scale;
        float p[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) p[s] = exp2_f(__builtin_fmaf(st[s >> 2][s & 3], scale, ref));
        if (!all) {         // (-infinity times a scale of 0 is NaN)
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (!((mine >> ((s < 4 ? 0 : 12) + s)) & 1)) p[s] = 0.0f;
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) l += p[s];
        u32x4 hi, lo;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t x, y;
            split_pair<DT, false>(p[2 * s] * O::UP, p[2 * s + 1] * O::UP, x, y);
            hi[s] = x, lo[s] = y;
        }
        // scales of this lane's elements in its eight tokens
        uint32_t vs[8];
        {
            const int grp = DV * i / 32;
            const u32x4 x = *reinterpret_cast<const u32x4 *>(&S[1][grp >> 2][4 * g]);
            const u32x4 y = *reinterpret_cast<const u32x4 *>(&S[1][grp >> 2][16 + 4 * g]);
#pragma unroll
            for (int s = 0; s < 4; ++s) vs[s] = at_exponent(x[s], grp & 3), vs[4 + s] = at_exponent(y[s], grp & 3);
        }
        uint32_t vr[8][VW];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const auto x = *reinterpret_cast<const typename Word<DV / 2>::type *>(tile + (4 * s + g) * ROW + DV / 2 * i);
            if constexpr (DV == 16) vr[s][0] = x[0], vr[s][1] = x[1];
            else vr[s][0] = x;
        }
        auto product = [&](auto word, auto pr, int e) {      // elements 2 e and 2 e + 1
            uint32_t x[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) x[s] = pair_of<DT, decltype(pr)::value>(vr[s][decltype(word)::value], vs[s]);
            u32x4 even, odd;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                even[s] = __builtin_amdgcn_perm(x[2 * s + 1], x[2 * s], 0x05040100);
                odd[s] = __builtin_amdgcn_perm(x[2 * s + 1], x[2 * s], 0x07060302);
            }
            acc[2 * e] = O::mma(even, hi, acc[2 * e]);
            acc[2 * e + 1] = O::mma(odd, hi, acc[2 * e + 1]);
            acc[2 * e] = O::mma(even, lo, acc[2 * e]);
            acc[2 * e + 1] = O::mma(odd, lo, acc[2 * e + 1]);
        };
        using std::integral_constant;
        product(integral_constant<int, 0>{}, integral_constant<int, 0>{}, 0);
        product(integral_constant<int, 0>{}, integral_constant<int, 1>{}, 1);
        if constexpr (DV >= 8) {
            product(integral_constant<int, 0>{}, integral_constant<int, 2>{}, 2);
            product(integral_constant<int, 0>{}, integral_constant<int, 3>{}, 3);
        }
        if constexpr (DV >= 16) {
            product(integral_constant<int, 1>{}, integral_constant<int, 0>{}, 4);
            product(integral_constant<int, 1>{}, integral_constant<int, 1>{}, 5);
            product(integral_constant<int, 1>{}, integral_constant<int, 2>{}, 6);
            product(integral_constant<int, 1>{}, integral_constant<int, 3>{}, 7);
        }
        seen = then;
    }
    if (err && __any(bad) && lane == 0) atomicOr(err, KDA_DEVERR_PAGES);
    l = column_sum(l);
    m = m == NEG_INF ? NEG_INF : m * scale;      // as a score, base 2

    // the waves' results, against the block's largest maximum
    if (g == 0) stat[wave][i][0] = m, stat[wave][i][1] = l;
    __syncthreads();
    float M = NEG_INF, L = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) M = __builtin_fmaxf(M, stat[v][i][0]);
    const float ref = M == NEG_INF ? 0.0f : M;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) L += stat[v][i][1] * exp2_f(stat[v][i][0] - ref);
    const float r = exp2_f(m - ref) * (1.0f / O::UP);
    // O^T: element DV (4 g + j) + d of head i
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < DV; ++d) lds.join[wave][i * (DH + 4) + DV * (4 * g + j) + d] = acc[d][j] * r;
    __syncthreads();
    const bool whole = w.whole;
    for (int x = threadIdx.x; x < heads * DH; x += 64 * WAVES) {
        const int h = x / DH, d = x - h * DH;
        float o = 0.0f;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) o += lds.join[v][h * (DH + 4) + d];
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

// Blocks that run at once at head dimension 128: four to each of 256 CUs. Tokens are spread over as many.
constexpr int RUN = 1024;
static_assert(RUN <= MAX_SPREAD, "the join holds a weight for each chunk of a sequence");

template <int DT, int DH>
hipError_t run_fp4(const kda_attn_fp4_args &f, const Plan &p, float *acc, float *ml, int32_t *err, hipStream_t st) {
    const kda_attn_args &a = f.attn;
    const int64_t blocks = (int64_t)p.slots * a.kv_heads * p.tiles_h;
    attn_fp4_chunk_kernel<DT, DH><<<dim3((unsigned)blocks), 64 * WAVES, 0, st>>>(f, acc, ml, err, p.spread, p.min_chunk, p.tiles_h);
    if (hipError_t e = hipGetLastError()) return e;
    if (p.join) attn_join_kernel<DT, DH><<<dim3((unsigned)a.num_seqs, (unsigned)a.q_heads), 256, 0, st>>>(a, acc, ml, p.spread, p.min_chunk);
    return hipGetLastError();
}

template <int DT> hipError_t run_fp4_dt(const kda_attn_fp4_args &f, const Plan &p, float *acc, float *ml, int32_t *err, hipStream_t st) {
    if (f.attn.head_dim == 64) return run_fp4<DT, 64>(f, p, acc, ml, err, st);
    if (f.attn.head_dim == 128) return run_fp4<DT, 128>(f, p, acc, ml, err, st);
    return run_fp4<DT, 256>(f, p, acc, ml, err, st);
}

}  // namespace
}  // namespace attn

size_t attn_fp4_workspace(int64_t B, int64_t hq, int64_t hkv, int64_t dh, int64_t width, int64_t page) {
    const attn::Plan p = attn::plan(B, hq, hkv, width, page, attn::RUN);
    return p.join ? (size_t)p.slots * hq * (dh + 2) * sizeof(float) : 0;
}

hipError_t launch_attn_decode_fp4(const kda_attn_fp4_args &f, float *ws, int32_t *err, hipStream_t st) {
    const kda_attn_args &a = f.attn;
    const attn::Plan p = attn::plan(a.num_seqs, a.q_heads, a.kv_heads, a.table_width, a.page_size, attn::RUN);
    float *ml = ws ? ws + (size_t)p.slots * a.q_heads * a.head_dim : nullptr;
    if (a.dtype == KDA_DTYPE_BF16) return attn::run_fp4_dt<KDA_DTYPE_BF16>(f, p, ws, ml, err, st);
    return attn::run_fp4_dt<KDA_DTYPE_F16>(f, p, ws, ml, err, st);
}

}  // namespace ops
}  // namespace kda
