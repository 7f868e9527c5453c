// ops_kv.hip -- new keys and values into a paged cache, with the position rotation on the way (kv_append), into a
// cache of the activations' type or one of 4 bits, and the read-back of the latter (kv_read_fp4).
//
//   pair (x, y) at position p:  (x c - y s, y c + x s),  c, s = the row p of the table of cosines and sines
//   4 bits: e = floor(log2 max|x|) - 2 over 32 elements, one more where max|x| > 1.75 2^{e + 2} (then the largest
//   value lies over 3.5 and up to 7 steps of 2^e, and is off by at most the half step that values between 4 and 6 are);
//   codes = x 2^-e rounded to e2m1, to even halfway, at most 6
//
// Bound by memory: each row is read and written once. A thread has 8 neighbouring elements of one head (16 bytes) and
// goes from head to head of its token with the same 8 cosines and sines in registers; the elements that they are
// paired with come through the cache, which the neighbouring lanes fill. Measured at heads of 128: 8192 ragged tokens of 32 + 4 + 4
// heads in fp16 (170 MB) 37 us, 4.5 TB/s; 8192 of 32 + 8 + 8 into 4 bits (176 MB) 45 us, 3.9 TB/s: 59% of its waves' cycles are
// waits, with five waves a SIMD (96 registers) and look-ups that wait for each other (sequence, length, page, angles); vector
// instructions of all kinds take 22 us, the rotation of keys in 64 bits under 1 of them; 256 tokens 4.5 us, latency.
#include <type_traits>

#include "ops_common.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace kv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int THREADS = 256;

// Packed new rows: offsets clamped to [0, T]; rows before the first sequence or behind the last one belong to none.
struct Batch {
    const int32_t *cu;      // NULL: row n is sequence n
    int N, T;
    __device__ __forceinline__ int at(int i) const {
        const int c = cu[i];
        return c < 0 ? 0 : c > T ? T : c;
    }
    // the sequence of row t and the rows left from t on (t included); 0 left: none
    __device__ __forceinline__ void find(int t, int &seq, int &left, int &past) const {
        if (!cu) {
            seq = t, left = 1, past = 0;
            return;
        }
        int lo = 0, hi = N;      // at(lo) <= t < at(hi), where offsets are in order
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (at(mid) <= t) lo = mid;
            else hi = mid;
        }
        seq = lo;
        past = t - at(lo);
        left = past < 0 ? 0 : at(lo + 1) - t;
        if (left < 0) left = 0;
    }
};

// Raises KDA_DEVERR_CU_SEQLENS unless 0 = c_0 <= ... <= c_N <= T (rows behind c_N are padding).
__device__ __forceinline__ void check_batch(const Batch &b, int32_t *err) {
    if (!b.cu || !err) return;
    bool bad = false;
    for (int i = threadIdx.x; i <= b.N; i += THREADS) {
        const int c = b.cu[i];
        bad |= i == 0 ? c != 0 : c < b.cu[i - 1];
        bad |= c > b.T;
    }
    if (bad) atomicOr(err, KDA_DEVERR_CU_SEQLENS);
}

template <int DT> __device__ __forceinline__ void store8(void *p, int64_t at, const float (&x)[8]) {
    using E = typename Elem<DT>::type;
    typedef E E8 __attribute__((ext_vector_type(8)));
    E8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (E)x[i];
    *reinterpret_cast<E8 *>((E *)p + at) = r;
}

template <int DT> using Row8 = typename Elem<DT>::type __attribute__((ext_vector_type(8)));
__device__ __forceinline__ u32x4 raw8(const void *p, int64_t at) { return *reinterpret_cast<const u32x4 *>((const uint16_t *)p + at); }

// How 8 elements of a head are rotated: x_i c_i + y_i s_i with y the elements they are paired with, half a rotation away or
// their neighbours, and the sign of either in s.
struct Turn {
    bool on;
    int other;          // where the paired elements lie (their own place: neighbours)
    float c[8], s[8];
};

__device__ __forceinline__ void turn_of(const kda_kv_args &a, int e, Turn &r) {
    const int d = 8 * e, half = a.rot_dim / 2;
    r.on = a.rope && d < a.rot_dim;
    r.other = !r.on || a.interleaved ? d : d < half ? d + half : d - half;
}

__device__ __forceinline__ void angles_of(const kda_kv_args &a, int pos, int d, Turn &r) {
    const int half = a.rot_dim / 2;
    const float *row = a.rope + (int64_t)pos * a.rot_dim;
    if (a.interleaved) {
        const f32x4 c = *reinterpret_cast<const f32x4 *>(row + d / 2), s = *reinterpret_cast<const f32x4 *>(row + half + d / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) r.c[i] = c[i / 2], r.s[i] = i & 1 ? s[i / 2] : -s[i / 2];
    } else {
        const int at = d < half ? d : d - half;
        const float sign = d < half ? -1.0f : 1.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const f32x4 c = *reinterpret_cast<const f32x4 *>(row + at + 4 * n), s = *reinterpret_cast<const f32x4 *>(row + half + at + 4 * n);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.c[4 * n + i] = c[i], r.s[4 * n + i] = sign * s[i];
        }
    }
}

// F double: rounded once from 64 bits (the products of a 16-bit and a 32-bit number are exact there), so that which side of
// a border of the 4-bit codes a value falls on does not hang on the order of roundings.
template <int DT, class F> __device__ __forceinline__ void rotated(bool on, bool neighbours, const Turn &r, u32x4 own, u32x4 other, float (&x)[8]) {
    const Row8<DT> u = __builtin_bit_cast(Row8<DT>, own);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)u[i];
    if (!on) return;
    if (neighbours) {
#pragma unroll
        for (int i = 0; i < 4; ++i) other[i] = own[i] << 16 | own[i] >> 16;
    }
    const Row8<DT> v = __builtin_bit_cast(Row8<DT>, other);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(F) == 8) x[i] = (float)__builtin_fma((F)x[i], (F)r.c[i], (F)(float)v[i] * (F)r.s[i]);
        else x[i] = __builtin_fmaf(x[i], r.c[i], (float)v[i] * r.s[i]);
    }
}

// What DPP hands on within four neighbouring lanes: the maximum over their 32 elements.
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
    uint32_t y = __builtin_amdgcn_update_dpp(0, x, 0xb1, 0xf, 0xf, true);      // lanes 1 0 3 2
    x = x > y ? x : y;
    y = __builtin_amdgcn_update_dpp(0, x, 0x4e, 0xf, 0xf, true);               // lanes 2 3 0 1
    return x > y ? x : y;
}

// 8 values of this lane (32 of the four lanes it belongs to) to codes; returns the biased exponent of the scale.
// Infinities and NaN: 255, the scale that stands for NaN. MOST keeps 6 2^e in the type that reads it back.
template <int DT> __device__ __forceinline__ uint32_t to_fp4(const float (&x)[8], uint32_t &code) {
    constexpr uint32_t MOST = DT == KDA_DTYPE_BF16 ? 252 : 140;
    uint32_t top = 0;      // magnitudes compare as their bits do; those of infinities and NaN lie above all others
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
        top = top > b ? top : b;
    }
    top = group_max(top);
    uint32_t e = (top + 0x1fffffu) >> 23;       // 0x600000 of the mantissa is 1.75
    e = e < 3 ? 1 : e - 2;
    e = e > MOST ? MOST : e;
    e = top >= 0x7f800000u ? 255 : e;
    const float s = __uint_as_float(e << 23);
    code = 0;
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[0], x[1], s, 0);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[2], x[3], s, 1);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[4], x[5], s, 2);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[6], x[7], s, 3);
    return e;
}

// A block takes one new token; its threads 8 elements of a head each, head after head: queries, keys, values. The rows
// of AHEAD heads are asked for before the token's place is looked up: the look-ups (sequence, length, page, angles) wait
// for one another, and the rows with them otherwise: 8192 tokens of 32 + 8 + 8 heads of 128 into 4 bits 49 us for 67. What is left of
// a token with more rows than that is asked for in turn. 2 | 3 | 4 ahead for 8192 tokens (us in 16, in 4 bits): 32 + 8 + 8 heads of 128 47, 50 |
// 46, 46 | 75, 69; 64 + 8 + 8 69, 75 | 73, 73 | 119, 108; 32 + 8 + 8 of 256 82, 88 | 86, 86 | 139, 117; 16 + 2 + 2 of 256 40, 45 | 38, 41 |
// 68, 63 (spills). Registers are held to what 6 waves a SIMD leave each, 5 for 4 bits (37 us for 39 with 8192 ragged tokens, 45 for
// 48): fewer spill.
constexpr int AHEAD = 3;
template <int DT, int DH, bool FOUR>
__global__ __launch_bounds__(THREADS, (FOUR ? 5 : 6)) void kv_append_kernel(const kda_kv_args a, int32_t *err) {
    constexpr int LANES = DH / 8, HEADS = THREADS / LANES;      // of a head; heads at a time
    const Batch batch = {a.cu_seqlens, a.num_seqs, a.total_tokens};
    if (blockIdx.x == 0) check_batch(batch, err);
    const int t = blockIdx.x;
    if (t >= a.total_tokens) return;
    const int e = threadIdx.x % LANES, d = 8 * e, slots = a.q_heads + 2 * a.kv_heads;
    Turn turn;
    turn_of(a, e, turn);
    const bool neighbours = a.interleaved;
    u32x4 own[AHEAD], other[AHEAD];
    auto load = [&](int h0) {
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) {
            const int h = h0 + n * HEADS;
            if (h >= slots) continue;
            const void *p = a.v;
            int64_t row = t * a.v_stride + (h - a.q_heads - a.kv_heads) * a.v_head_stride;
            int paired = d;
            if (h < a.q_heads) p = a.q, row = t * a.q_stride + h * a.q_head_stride, paired = turn.other;
            else if (h < a.q_heads + a.kv_heads) p = a.k, row = t * a.k_stride + (h - a.q_heads) * a.k_head_stride, paired = turn.other;
            own[n] = raw8(p, row + d);
            if (!neighbours) other[n] = raw8(p, row + paired);
        }
    };
    const int first = threadIdx.x / LANES;
    load(first);
    int seq, left, past;
    batch.find(t, seq, left, past);
    if (!left) return;
    const int len = a.seq_lens[seq];
    if (len == 0) return;       // an empty slot
    const int64_t pos = (int64_t)len - left;
    int page = -1;
    const bool inside = len > 0 && pos >= 0 && pos < (int64_t)a.table_width * a.page_size && (!a.rope || pos < a.max_positions);
    if (inside) {
        page = a.block_table[(int64_t)seq * a.table_stride + pos / a.page_size];
        if (turn.on) angles_of(a, (int)pos, d, turn);
    }
    if (page < 0 || page >= a.num_pages) {
        if (err && threadIdx.x == 0) atomicOr(err, KDA_DEVERR_PAGES);
        return;
    }
    const int at = (int)(pos % a.page_size);
    for (int h0 = first; h0 < slots; h0 += AHEAD * HEADS) {
        if (h0 != first) load(h0);
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) {
            const int h = h0 + n * HEADS;
            if (h >= slots) continue;
            float x[8];
            if (h < a.q_heads) {
                rotated<DT, float>(turn.on, neighbours, turn, own[n], other[n], x);
                store8<DT>(a.q_out, ((int64_t)t * a.q_heads + h) * DH + d, x);
                continue;
            }
            const bool key = h < a.q_heads + a.kv_heads;
            const int c = h - a.q_heads - (key ? 0 : a.kv_heads);
            rotated<DT, std::conditional_t<FOUR, double, float>>(key && turn.on, neighbours, turn, own[n], other[n], x);
            void *cache = key ? a.k_cache : a.v_cache;
            const int64_t row = key ? page * a.k_page_stride + at * a.k_token_stride + c * a.k_cache_head_stride
                                    : page * a.v_page_stride + at * a.v_token_stride + c * a.v_cache_head_stride;
            if constexpr (!FOUR) store8<DT>(cache, row + d, x);
            else {
                uint32_t code;
                const uint32_t s = to_fp4<DT>(x, code);
                *reinterpret_cast<uint32_t *>((uint8_t *)cache + row + d / 2) = code;
                uint8_t *scale = key ? a.k_scale + page * a.k_scale_page_stride + at * a.k_scale_token_stride + c * a.k_scale_head_stride
                                     : a.v_scale + page * a.v_scale_page_stride + at * a.v_scale_token_stride + c * a.v_scale_head_stride;
                if (e % 4 == 0) scale[e / 4] = (uint8_t)s;
            }
        }
    }
}

// Eight values of codes w times the scale s.
template <int DT> __device__ __forceinline__ u32x4 values_of(uint32_t w, uint32_t scale) {
    const float s = __uint_as_float(scale << 23);
    if constexpr (DT == KDA_DTYPE_BF16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3))};
}

// A block takes TOKENS rows of the packed result, their look-ups (sequence, page, codes) side by side (9216 tokens of 8
// heads of 128, 43 MB: 15.6 us, 19 with one at a time).
constexpr int TOKENS = 4;
template <int DT, int DH>
__global__ __launch_bounds__(THREADS) void kv_read_fp4_kernel(const kda_kv_read_args a, int32_t *err) {
    constexpr int LANES = DH / 8, HEADS = THREADS / LANES;
    using E = typename Elem<DT>::type;
    const Batch batch = {a.cu_seqlens, a.num_seqs, a.total_tokens};
    if (blockIdx.x == 0) check_batch(batch, err);
    const int e = threadIdx.x % LANES, t0 = blockIdx.x * TOKENS;
    int left[TOKENS], place[TOKENS], page[TOKENS];
    bool there[TOKENS], bad = false;
#pragma unroll
    for (int n = 0; n < TOKENS; ++n) {
        int seq = 0, past = 0;
        left[n] = 0, page[n] = -1;
        if (t0 + n < a.total_tokens) batch.find(t0 + n, seq, left[n], past);
        if (left[n] && past < (int64_t)a.table_width * a.page_size) page[n] = a.block_table[(int64_t)seq * a.table_stride + past / a.page_size];
        place[n] = past % a.page_size;
    }
#pragma unroll
    for (int n = 0; n < TOKENS; ++n) {
        there[n] = page[n] >= 0 && page[n] < a.num_pages;
        bad |= left[n] && !there[n];
    }
    if (bad && err && threadIdx.x == 0) atomicOr(err, KDA_DEVERR_PAGES);
    for (int h = threadIdx.x / LANES; h < 2 * a.kv_heads; h += HEADS) {
        const bool key = h < a.kv_heads;
        const int64_t c = key ? h : h - a.kv_heads;
        const uint8_t *cache = key ? (const uint8_t *)a.k_cache + c * a.k_head_stride : (const uint8_t *)a.v_cache + c * a.v_head_stride;
        const uint8_t *scale = key ? a.k_scale + c * a.k_scale_head_stride : a.v_scale + c * a.v_scale_head_stride;
        const int64_t to_page = key ? a.k_page_stride : a.v_page_stride, to_token = key ? a.k_token_stride : a.v_token_stride;
        const int64_t sc_page = key ? a.k_scale_page_stride : a.v_scale_page_stride, sc_token = key ? a.k_scale_token_stride : a.v_scale_token_stride;
        uint32_t w[TOKENS], s[TOKENS];
#pragma unroll
        for (int n = 0; n < TOKENS; ++n) {
            w[n] = s[n] = 0;
            if (there[n]) {
                w[n] = *reinterpret_cast<const uint32_t *>(cache + page[n] * to_page + place[n] * to_token + 4 * e);
                s[n] = scale[page[n] * sc_page + place[n] * sc_token + e / 4];
            }
        }
        E *to = (E *)(key ? a.k : a.v) + ((int64_t)t0 * a.kv_heads + c) * DH + 8 * e;
#pragma unroll
        for (int n = 0; n < TOKENS; ++n)
            if (left[n]) *reinterpret_cast<u32x4 *>(to + (int64_t)n * a.kv_heads * DH) = values_of<DT>(w[n], s[n]);
    }
}

template <int DT, int DH> hipError_t append(const kda_kv_args &a, int32_t *err, hipStream_t st) {
    const dim3 grid(a.total_tokens > 0 ? (unsigned)a.total_tokens : 1);      // without rows: the check of the offsets
    if (a.k_scale) kv_append_kernel<DT, DH, true><<<grid, THREADS, 0, st>>>(a, err);
    else kv_append_kernel<DT, DH, false><<<grid, THREADS, 0, st>>>(a, err);
    return hipGetLastError();
}
template <int DT> hipError_t append_dt(const kda_kv_args &a, int32_t *err, hipStream_t st) {
    if (a.head_dim == 64) return append<DT, 64>(a, err, st);
    if (a.head_dim == 128) return append<DT, 128>(a, err, st);
    return append<DT, 256>(a, err, st);
}
template <int DT, int DH> hipError_t read(const kda_kv_read_args &a, int32_t *err, hipStream_t st) {
    const int64_t blocks = ceil_div(a.total_tokens, TOKENS);
    kv_read_fp4_kernel<DT, DH><<<dim3(blocks > 0 ? (unsigned)blocks : 1), THREADS, 0, st>>>(a, err);
    return hipGetLastError();
}
template <int DT> hipError_t read_dt(const kda_kv_read_args &a, int32_t *err, hipStream_t st) {
    if (a.head_dim == 64) return read<DT, 64>(a, err, st);
    if (a.head_dim == 128) return read<DT, 128>(a, err, st);
    return read<DT, 256>(a, err, st);
}

}  // namespace
}  // namespace kv

hipError_t launch_kv_append(const kda_kv_args &a, int32_t *err, hipStream_t st) {
    return a.dtype == KDA_DTYPE_BF16 ? kv::append_dt<KDA_DTYPE_BF16>(a, err, st) : kv::append_dt<KDA_DTYPE_F16>(a, err, st);
}

hipError_t launch_kv_read_fp4(const kda_kv_read_args &a, int32_t *err, hipStream_t st) {
    return a.dtype == KDA_DTYPE_BF16 ? kv::read_dt<KDA_DTYPE_BF16>(a, err, st) : kv::read_dt<KDA_DTYPE_F16>(a, err, st);
}

}  // namespace ops
}  // namespace kda
