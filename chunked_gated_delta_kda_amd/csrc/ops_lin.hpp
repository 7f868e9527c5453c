// ops_lin.hpp -- linear attention with a decay for each head: what its forward (ops_lin.hip) and its gradients
// (ops_lin_bwd.hip) share.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// The time axis is cut into segments of whole chunks of 64 tokens. A chunk that S enters gives, with G_i the sum of g
// from its first token to i and G its sum over the chunk,
//
//   o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S <- e^G S + sum_j e^{G - G_j} k_j v_j^T
//
// and its gradients are three more linear attentions with the roles exchanged, two of them from the end:
//   dq: (q, k, v) = (do, v, k) on S^T;   dv: (k, q, do), backwards;   dk: (v, do, q), backwards
// so that one walk over the chunks of a segment (`Walk`) serves them all. What enters a segment comes from a pass over the
// segments before it (states of their own tokens alone) and a join of those.
//
// Matrix products run on bf16 matrix instructions: fp16 inputs go in as two bf16 numbers each (11 = 8 + 3 bits, and
// bf16's exponents hold fp16's), and what is computed in fp32 as two (2^-17 of it is lost; where it ends in a 16-bit output) or three
// (2^-25; where it ends in fp32: states and gradients of decays). States themselves stay in fp32 registers.
//
// 8192 tokens of 32 heads of 128 x 128 in bf16 (268 MB in and out: 51 us of memory): states of segments 39 us, join 15,
// walk 81. In the walk matrix instructions (79 a wave and chunk, 16 cycles each) take 17 us, vector ones (377, for splits, decays
// and conversions) 20, LDS 21: no unit is full. They meet where the two waves and two blocks of a SIMD allow; the phases of a
// chunk, between barriers, keep them from meeting more often. Without its loads it takes 82% of the time, without the update 74%.
#pragma once

#include "ops_common.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace lin {
namespace {

constexpr int C = 64;              // tokens of a chunk
// A block has a wave for every 16 value columns, which holds those columns of the state.
template <int VD> constexpr int WAVES = VD / 16;
template <int VD> constexpr int THREADS = 64 * WAVES<VD>;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// bf16 numbers that one element of an input is
template <int DT> constexpr int PLANES = DT == KDA_DTYPE_BF16 ? 1 : 2;

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Nothing is moved over this place: without such places reads are taken so far ahead that their registers spill.
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

// Two fp32 numbers rounded to bf16, in one word.
__device__ __forceinline__ uint32_t pack(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
}

// 8 fp32 numbers as N bf16 numbers each: each the rounding of what those before it leave.
template <int N> __device__ __forceinline__ void split(const float (&x)[8], u32x4 (&to)[N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t w = pack(a, b);
            to[n][i] = w;
            if (n + 1 < N) a -= __uint_as_float(w << 16), b -= __uint_as_float(w & 0xffff0000u);
        }
    }
}

// A product of numbers in A and in B parts: the pairs whose first parts' places add up to less than MOST (a pair at
// MOST is 2^-8 MOST of the result).
template <int A, int B, int MOST, class F> __device__ __forceinline__ void pairs(F f) {
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (a + b < MOST) f(a, b);
}

// Memory through buffer descriptors: a base that is the same for the block, 32-bit offsets, and reads past `bytes` that give
// zeros, writes that are dropped, so that short chunks need no branches.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t OUTSIDE = 0xffffffffu;
__device__ __forceinline__ const char *same(const void *p) {     // told to be the same in all lanes: kept in scalar registers
    const uint64_t x = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (const char *)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ Buffer buffer(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)same(p), 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00027000);
}
__device__ __forceinline__ u32x4 read16(Buffer b, uint32_t at, uint32_t more = 0) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, __builtin_amdgcn_readfirstlane((int)more), 0));
}

// One chunk of rows in LDS. LDS serves 256 bytes at once; 16-byte reads of 64 lanes go in groups of lanes 0-3, 12-15, 20-27
// and the like, which are units of 8 rows in one lane group g and of the other 8 in its neighbour (row_operand): 16 bytes
// between rows and 64 more between every four keep them from meeting in a bank at 128 columns.
template <int NP, int D> struct Tile {
    static constexpr int ROW = D + 8, FOUR = 4 * ROW + (D == 128 ? 32 : 0);      // elements of a row, of four
    uint16_t x[NP][C / 4 * FOUR];
    static __device__ __forceinline__ int at(int row) { return (row >> 2) * FOUR + (row & 3) * ROW; }
    __device__ __forceinline__ void put(int plane, int row, int unit, u32x4 e) {
        *reinterpret_cast<u32x4 *>(&x[plane][at(row) + 8 * unit]) = e;
    }
};

// An input in one of the three roles: rows [T, H, D], contiguous elements.
struct Role {
    const void *p;
    int64_t row, head;       // strides, elements
};
// One head of it.
struct Rows {
    const char *p;
    uint32_t row;            // bytes
    __device__ __forceinline__ Rows(const Role &r, int h) : p(same((const char *)r.p + 2 * h * r.head)), row(2 * (uint32_t)r.row) {}
    // from row `first` on, the last of `len` rows of D elements included
    __device__ __forceinline__ Buffer from(int first, int len, int D) const {
        return buffer(p + (uint64_t)(uint32_t)first * row, len ? (len - 1) * row + 2 * D : 0);
    }
};

// Rows of a chunk on their way from memory to LDS, 8 elements of a row a time. NT: threads of the block. Offsets from
// a chunk's first row fit 32 bits (strides are at most KDA_LIN_MAX_STRIDE).
template <int DT, int D, int NT> struct Stage {
    static constexpr int N = C * D / 8 / NT, ROWS = NT / (D / 8);     // rows of a piece
    u32x4 r[N];
    __device__ __forceinline__ void load(const Rows &s, int first, int len) {
        const Buffer b = s.from(first, len, D);
        const uint32_t row = threadIdx.x / (D / 8), at = row * s.row + 16 * (threadIdx.x % (D / 8));
#pragma unroll
        for (int n = 0; n < N; ++n)      // (rows that lie over each other, strides of 0, are cut off as well)
            r[n] = read16(b, (int)row + ROWS * n < len ? at : OUTSIDE, ROWS * n * s.row);
    }
    // whether this lane has an infinity or a NaN
    __device__ __forceinline__ bool not_finite() const {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        constexpr unsigned short INF = DT == KDA_DTYPE_BF16 ? 0x7f80 : 0x7c00;
        u16x2 top = {0, 0};
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, r[n][i] & 0x7fff7fffu));
        return top[0] >= INF || top[1] >= INF;
    }
    __device__ __forceinline__ void store(Tile<PLANES<DT>, D> &t) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int row = threadIdx.x / (D / 8) + ROWS * n, q = threadIdx.x % (D / 8);
            if constexpr (DT == KDA_DTYPE_BF16) t.put(0, row, q, r[n]);
            else {
                typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
                const f16x8 e = __builtin_bit_cast(f16x8, r[n]);
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
                u32x4 part[2];
                split<2>(v, part);
                t.put(0, row, q, part[0]);
                t.put(1, row, q, part[1]);
            }
        }
    }
};

// Operands of v_mfma_f32_16x16x32: a lane (i = lane & 15, g = lane >> 4) holds 8 numbers of row (or column) i, places 8 g .. of the
// contraction, which may be labelled at will as long as both operands agree. A result holds rows 4 g + r of column i; two
// results of 16 rows each are an operand as they are, if their rows are labelled so:
//  * tokens of two tiles of pairs: slot 8 g + s is token 4 g + s for s < 4, 16 + 4 g + s - 4 else (value_operand reads
//    values in that order);
//  * key elements of two tiles of a state: lane group g's rows 4 g .. + 3 of tiles 2 s and 2 s + 1 are the halves of unit
//    s + K / 32 g of a key row, which row_operand reads at once.
template <int KD> __device__ __forceinline__ int key_element(int t, int g) { return 8 * ((t >> 1) + KD / 32 * g) + 4 * (t & 1); }

// of row 16 t + i, units s + D / 32 g
template <int NP, int D> __device__ __forceinline__ u32x4 row_operand(const Tile<NP, D> &m, int plane, int t, int s) {
    const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    return *reinterpret_cast<const u32x4 *>(&m.x[plane][m.at(i) + 4 * t * m.FOUR + 8 * (s + D / 32 * g)]);
}

// A transposing read hands the 16 lanes of a row of 16 columns (each lane's address: 4 columns of row lane / 4) a column of 4
// rows each; two of them make an operand of rows 32 s .. of the tile.
template <int NP, int D> __device__ __forceinline__ u32x4 turned(const uint16_t *p) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * Tile<NP, D>::FOUR));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return u32x4{x[0], x[1], y[0], y[1]};
}
// of the key element that tile t has in row i, rows 32 s ..
template <int NP, int D> __device__ __forceinline__ u32x4 key_operand(const Tile<NP, D> &m, int plane, int t, int s) {
    const int i = threadIdx.x & 15, row = 4 * ((threadIdx.x & 63) >> 4) + (i >> 2);
    return turned<NP, D>(&m.x[plane][m.at(row) + 8 * s * m.FOUR + key_element<D>(t, i & 3)]);
}
// of value element 16 t + i, rows 32 s ..
template <int NP, int D> __device__ __forceinline__ u32x4 value_operand(const Tile<NP, D> &m, int plane, int t, int s) {
    const int i = threadIdx.x & 15, row = 4 * ((threadIdx.x & 63) >> 4) + (i >> 2);
    return turned<NP, D>(&m.x[plane][m.at(row) + 8 * s * m.FOUR + 16 * t + 4 * (i & 3)]);
}
// What a chunk's tokens are multiplied by. Sums of decays are formed in 64 bits; G_i is kept as a whole number and
// a rest of at most 1/2 (base 2), so that differences lose nothing where the sums are large.
struct __attribute__((aligned(16))) Clock {
    float whole[C], rest[C];
    float in[C];       // of the state that enters, at a token
    float up[C];       // of a token, in the state that leaves
    float total;       // of the state that enters, in the one that leaves
};

// log2 of a decay; e^g under 2^-4096 is 0 all the same, and -infinity (a reset) makes no NaN of differences
__device__ __forceinline__ double log2_decay(float g) {
    const double x = (double)g * 1.4426950408889634;
    return x < -4096.0 ? -4096.0 : x;
}

// what lane - D of the 16-lane row holds, 0 before the row
template <int D> __device__ __forceinline__ double row_shr(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)b, 0x110 + D, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(b >> 32), 0x110 + D, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// by one wave, lane t for token t: its log decay, 0 past the chunk's end. Returns the sum of the chunk's, base 2. (The caller
// loads g a chunk ahead: what it does with it before it calls would wait for the load.)
template <bool REV> __device__ __forceinline__ double tick(Clock &c, float g, float in_scale, float up_scale) {
    const int lane = threadIdx.x & 63;
    double x = log2_decay(g);
    x += row_shr<1>(x);
    x += row_shr<2>(x);
    x += row_shr<4>(x);
    x += row_shr<8>(x);
    const double a = lane_of(x, 15), b = a + lane_of(x, 31), d = b + lane_of(x, 47);
    x += lane < 16 ? 0.0 : lane < 32 ? a : lane < 48 ? b : d;
    const double total = lane_of(x, 63);
    const double whole = __builtin_rint(x);
    const float from = exp2_f((float)x), to = exp2_f((float)(total - x));
    c.whole[lane] = (float)whole;
    c.rest[lane] = (float)(x - whole);
    c.in[lane] = in_scale * (REV ? to : from);
    c.up[lane] = up_scale * (REV ? from : to);
    if (lane == 0) c.total = exp2_f((float)total);
    return total;
}

// The chunks of a segment [s0, s1) in order, forwards or backwards: a part is what it holds of one sequence, and chunks
// start from a part's first token in both directions. Parts need nothing of each other: forwards, `turns` blocks may share a segment's,
// each those of every turns-th sequence.
struct Chunk {
    int first, len;      // len 0: none
    int seq;
    bool enter, leave;   // the first, the last of its part
    bool open, close;    // (with enter) the sequence begins here, (with leave) it ends here
};

template <bool REV> struct Chunks {
    Offsets o;
    int s0, s1, at, seq, begin, end, p0, p1;     // the sequence; the part [p0, p1); at: the next chunk's first token (REV: the end of the rest)
    int turns, mine;
    bool fresh;
    __device__ __forceinline__ Chunks(const Offsets &off, int a, int b, int every = 1, int own = 0)
        : o(off), s0(a), s1(b), at(REV ? b : a), seq(-1), begin(0), end(0), p0(0), p1(0), turns(every), mine(own), fresh(true) {}
    // the sequence of token t, next to the last one where that is so
    __device__ __forceinline__ int find(int t) const {
        if (seq >= 0) {
            const int n = REV ? seq - 1 : seq + 1;
            if (n >= 0 && n < o.N && o.at(n) <= t && t < o.at(n + 1)) return n;
        }
        return o.find(t);
    }
    // the part of the next sequence of this block that has tokens in the segment
    __device__ __forceinline__ bool take() {
        auto own_from = [&](int n) { return n + (mine + turns - n % turns) % turns; };
        int n = seq < 0 ? own_from(o.find(s0)) : seq + turns;
#pragma unroll 1
        for (;;) {
            n = __builtin_amdgcn_readfirstlane(n);
            if (n >= o.N) return false;
            begin = __builtin_amdgcn_readfirstlane(o.at(n)), end = __builtin_amdgcn_readfirstlane(o.at(n + 1));
            if (begin >= s1) return false;
            if (end > begin) break;
            const int s = o.find(begin);        // an empty one: on to the one that has its place
            n = s > n ? own_from(s) : n + turns;
        }
        seq = n;
        p0 = begin < s0 ? s0 : begin;
        p1 = end > s1 ? s1 : end <= p0 ? p0 + 1 : end;      // (clamped as below)
        at = p0;
        return true;
    }
    __device__ __forceinline__ Chunk next() {
        Chunk c = {0, 0, 0, false, false, false, false};
        if (REV ? at <= s0 : at >= s1) return c;
        if (fresh && turns > 1) {
            if (!take()) return c;
        } else if (fresh) {
            const int t = REV ? at - 1 : at;
            seq = __builtin_amdgcn_readfirstlane(find(t));
            begin = __builtin_amdgcn_readfirstlane(o.at(seq)), end = __builtin_amdgcn_readfirstlane(o.at(seq + 1));
            const int b = begin, e = end;
            p0 = __builtin_amdgcn_readfirstlane(REV ? (b < s0 ? s0 : b > t ? t : b) : t);            // (clamped where offsets are out of order)
            p1 = __builtin_amdgcn_readfirstlane(REV ? t + 1 : (e > s1 ? s1 : e <= t ? t + 1 : e));
        }
        c.seq = seq;
        c.enter = fresh;
        if constexpr (REV) {
            c.first = p0 + (at - 1 - p0) / C * C;
            c.len = at - c.first;
            at = c.first;
            c.leave = at <= p0;
        } else {
            c.first = at;
            c.len = p1 - at < C ? p1 - at : C;
            at += c.len;
            c.leave = at >= p1;
        }
        // (scalars: told to be the same in all lanes)
        at = __builtin_amdgcn_readfirstlane(at);
        c.first = __builtin_amdgcn_readfirstlane(c.first), c.len = __builtin_amdgcn_readfirstlane(c.len);
        // (only the part at the segment's edge continues what lies beyond, whatever the offsets say)
        const bool begins = begin >= p0 || p0 != s0, ends = end <= p1 || p1 != s1;
        c.open = REV ? ends : begins;
        c.close = REV ? begins : ends;
        fresh = c.leave;
        return c;
    }
};

// up_j v_j of the wave's column, tokens 32 s ..; v's operands as the second product wants them
template <int NP> __device__ __forceinline__ void weighted(const u32x4 (&v)[NP][2], const Clock &clock, int s, float (&x)[8]) {
    const int g = (threadIdx.x & 63) >> 4;
    const f32x4 a = *reinterpret_cast<const f32x4 *>(&clock.up[32 * s + 4 * g]);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(&clock.up[32 * s + 16 + 4 * g]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float e = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const uint32_t word = v[p][s][i / 2];
            const float f = __uint_as_float(i & 1 ? word & 0xffff0000u : word << 16);
            e = p ? e + f : f;
        }
        x[i] = e * (i < 4 ? a[i & 3] : b[i & 3]);
    }
}
// S += sum_j k_j w_j^T for those pairs of parts p of k and n of w that take(p, n) names, w's tokens 32 s ..
template <int NP, int KD, int N, class F>
__device__ __forceinline__ void add_products(f32x4 (&S)[KD / 16], const Tile<NP, KD> &k, const u32x4 (&w)[N], int s, F take) {
#pragma unroll
    for (int kt = 0; kt < KD / 16; kt += 2) {
        u32x4 row[2][NP];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int p = 0; p < NP; ++p) row[t][p] = key_operand(k, p, kt + t, s);
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (take(p, n)) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) S[kt + t] = mma(row[t][p], w[n], S[kt + t]);
                }
        hold();
    }
}
// S <- total S + sum_j k_j (up_j v_j)^T over a chunk, for the wave's columns, up_j v_j in N parts
template <int NP, int KD, int N>
__device__ __forceinline__ void update(f32x4 (&S)[KD / 16], const Tile<NP, KD> &k, const u32x4 (&v)[NP][2], const Clock &clock) {
    const float total = clock.total;
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt) S[kt] *= total;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        float x[8];
        weighted<NP>(v, clock, s, x);
        u32x4 w[N];
        split<N>(x, w);
        add_products<NP, KD>(S, k, w, s, [](int p, int n) { return p + n < N; });
    }
}
// the third part of those sums, where two have been taken (a pass of its own, for a few chunks: its registers are not held
// through the first)
template <int NP, int KD>
__device__ __forceinline__ void refine(f32x4 (&S)[KD / 16], const Tile<NP, KD> &k, const u32x4 (&v)[NP][2], const Clock &clock) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        float x[8];
        weighted<NP>(v, clock, s, x);
        u32x4 w[3];
        split<3>(x, w);
        add_products<NP, KD>(S, k, w, s, [](int p, int n) { return p + n == 2; });
    }
}

template <int NP, int VD> __device__ __forceinline__ void value_operands(const Tile<NP, VD> &v, int wave, u32x4 (&to)[NP][2]) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int s = 0; s < 2; ++s) to[p][s] = value_operand(v, p, wave, s);
}

// A state of KD x VD between memory and the wave's columns. TURNED: memory holds it as [VD][KD]. p NULL: zeros.
template <int KD, int VD, bool TURNED> __device__ __forceinline__ void load_state(f32x4 (&S)[KD / 16], const float *p, int wave) {
    const uint32_t i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if (!p) {
#pragma unroll
        for (int kt = 0; kt < KD / 16; ++kt) S[kt] = f32x4{0, 0, 0, 0};
        return;
    }
    const Buffer b = buffer(p, 4 * KD * VD);
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt) {
        const uint32_t k = key_element<KD>(kt & 1, g);
        if constexpr (TURNED) S[kt] = __builtin_bit_cast(f32x4, read16(b, 4 * ((16 * wave + i) * KD + k), 32 * (kt >> 1)));
        else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[kt][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, 4 * (k * VD + 16 * wave + i), 4 * VD * (8 * (kt >> 1) + r), 0));
        }
    }
}
template <int KD, int VD> __device__ __forceinline__ void store_state(const f32x4 (&S)[KD / 16], float *p, int wave) {
    const uint32_t i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const Buffer b = buffer(p, 4 * KD * VD);
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[kt][r]), b, 4 * (key_element<KD>(kt & 1, g) * VD + 16 * wave + i),
                                                  4 * VD * (8 * (kt >> 1) + r), 0);
}
// The same as lanes hold it, 16 bytes of each after the other's.
template <int KD, int VD> __device__ __forceinline__ void store_lanes(const f32x4 (&S)[KD / 16], float *p, int wave) {
    const Buffer b = buffer(p, 4 * KD * VD);
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[kt]), b, 4 * KD * 16 * wave + 16 * (threadIdx.x & 63), 1024 * kt, 0);
}
// One of either form (lanes, or [VD][KD]). p NULL: zeros.
template <int KD, int VD> __device__ __forceinline__ void load_either(f32x4 (&S)[KD / 16], const float *p, int wave, bool lanes) {
    const uint32_t i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const uint32_t at = lanes ? 16 * (threadIdx.x & 63) : 4 * (i * KD + key_element<KD>(0, g)), step = lanes ? 1024 : 16;
    const Buffer b = buffer(p, p ? 4 * KD * VD : 0);
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt) S[kt] = __builtin_bit_cast(f32x4, read16(b, 4 * KD * 16 * wave + at, kt * step));
}

// The batch and its segments.
struct Batch {
    const int32_t *cu;
    const float *g;         // decays [T, H] or [H]
    int64_t g_row;          // 0 where they are [H]
    int N, T, H, seg, segs; // seg: tokens of a segment (a multiple of C); segs of them
    int turns;              // blocks that share the parts of a segment in the walks
    __device__ __forceinline__ Offsets offsets() const { return Offsets{cu, N, T}; }
    // lane t's, of token first + t; 0 from len on
    __device__ __forceinline__ float decay(int first, int len, int h) const {
        const uint32_t lane = threadIdx.x & 63, row = 4 * (uint32_t)g_row;
        const Buffer b = buffer(g + (uint64_t)(uint32_t)first * (uint32_t)g_row + h, len ? (len - 1) * row + 4 : 0);
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (int)((int)lane < len ? lane * row : OUTSIDE), 0, 0));
    }
};

// ---------------------------------------------------------------- segments' own states
// Forwards: what the last sequence of segment blockIdx.x, if it goes on behind it, adds to the state there (from its
// initial state where it begins in the segment); factor: what is left of the state before the segment, or -1 where the sequence begins in it.
// Backwards the same from the other end. Bound by memory and its latency: k and v are read at 3.3 TB/s (8192 tokens of 32 heads,
// 134 MB in 40 us), a chunk ahead, in registers.
struct Own {
    Role k, v;
    const float *init;      // [N, H, KD, VD] or NULL
    float *state;           // [segs, H, KD, VD]
    float *factor;          // [segs, H]
    float up;
};

template <int DT, int KD, int VD> struct OwnLds {
    Tile<PLANES<DT>, KD> k;
    Tile<PLANES<DT>, VD> v;
    Clock clock[2];
};

template <int DT, int KD, int VD, bool REV> __device__ __forceinline__ void own_state(const Batch &b, const Own &a, OwnLds<DT, KD, VD> &L) {
    constexpr int NP = PLANES<DT>, NT = THREADS<VD>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), seg = blockIdx.x, h = blockIdx.y;
    const Offsets o = b.offsets();
    const int s0 = seg * b.seg, s1 = s0 + b.seg < b.T ? s0 + b.seg : b.T;
    float *factor = a.factor + (int64_t)seg * b.H + h;
    // the part that goes on past the segment
    int p0 = s0, p1 = s1;
    bool open, on;
    const int edge = REV ? s0 : s1 - 1, seq = __builtin_amdgcn_readfirstlane(o.find(edge));
    const int sb = __builtin_amdgcn_readfirstlane(o.at(seq)), se = __builtin_amdgcn_readfirstlane(o.at(seq + 1));
    if constexpr (REV) on = sb < s0, open = se <= s1, p1 = se < s1 ? (se <= s0 ? s0 + 1 : se) : s1;
    else on = se > s1, open = sb >= s0, p0 = sb > s0 ? (sb >= s1 ? s1 - 1 : sb) : s0;
    if (!on) {
        if (threadIdx.x == 0) *factor = -1.0f;
        return;
    }
    f32x4 S[KD / 16];
    load_state<KD, VD, false>(S, open && a.init ? a.init + ((int64_t)seq * b.H + h) * (KD * VD) : nullptr, wave);
    double sum = 0.0;
    float g = 0.0f;
    Stage<DT, KD, NT> sk;
    Stage<DT, VD, NT> sv;
    const Rows rk(a.k, h), rv(a.v, h);
    const int count = (p1 - p0 + C - 1) / C;
    auto load = [&](int n) {
        const int first = p0 + C * (REV ? count - 1 - n : n), len = p1 - first < C ? p1 - first : C;
        if (wave == 0) g = b.decay(first, len, h);
        sk.load(rk, first, len);
        sv.load(rv, first, len);
    };
    load(0);
    if (wave == 0) sum += tick<REV>(L.clock[0], g, 1.0f, a.up);
#pragma unroll 1
    for (int n = 0; n < count; ++n) {
        lds_barrier();
        sk.store(L.k);
        sv.store(L.v);
        lds_barrier();
        if (n + 1 < count) load(n + 1);
        u32x4 v[NP][2];
        value_operands(L.v, wave, v);
        update<NP, KD, 3>(S, L.k, v, L.clock[n & 1]);
        if (wave == 0 && n + 1 < count) sum += tick<REV>(L.clock[(n + 1) & 1], g, 1.0f, a.up);
    }
    store_state<KD, VD>(S, a.state + ((int64_t)seg * b.H + h) * (KD * VD), wave);
    if (threadIdx.x == 0) *factor = open ? -1.0f : exp2_f((float)sum);
}

// ---------------------------------------------------------------- join
// state[s] <- what leaves segment s (backwards: what it hands to the one before), in the order of the segments. Each step waits
// for the one before, so that AHEAD segments' states are asked for at once.
constexpr int JOIN_THREADS = 256;
template <int SIZE, int AHEAD> __device__ __forceinline__ void join(const Batch &b, float *state, const float *factor, bool rev) {
    const int h = blockIdx.y, x = blockIdx.x * JOIN_THREADS + threadIdx.x;
    float c = 0.0f;
    const int64_t step = (int64_t)b.H * SIZE;
    float *p = state + (int64_t)h * SIZE + x;
    for (int n0 = 0; n0 < b.segs - 1; n0 += AHEAD) {
        float u[AHEAD], f[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int n = n0 + i, s = rev ? b.segs - 1 - n : n;
            if (n < b.segs - 1) f[i] = factor[(int64_t)s * b.H + h], u[i] = p[s * step];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int n = n0 + i, s = rev ? b.segs - 1 - n : n;
            if (n < b.segs - 1) {
                if (f[i] >= 0.0f) c = __builtin_fmaf(f[i], c, u[i]), p[s * step] = c;
                else c = u[i];
            }
        }
    }
}
// Few segments: 8 ahead (2 x 16 segments of 16 heads 6.7 us for 8.3), more: 32 (64 of 8 heads 14 us for 20).
inline bool far_ahead(int segs) { return segs > 16; }

// ---------------------------------------------------------------- the walk
// A block takes a segment of one head, a wave 16 value columns: its part of the state (KD x 16) stays in registers, where a lane
// has 4 neighbouring key elements of a column, which is what the products with the state and into it want (no state
// passes through LDS, no wave needs another's). A chunk's rows come through LDS, the next chunk's are on their way in
// registers meanwhile. The pairs' weights, which all waves need, are made by 8 of them once, as operands.
//
// The gradients of decays need what passes all of a chunk, e^G <X, Y> with X the state that enters it and Y the gradient of the one that
// leaves: the walk for dk, from the end, leaves Y where the one for dq, which holds X, reads it.
struct Walk {
    Role q, k, v;
    void *out;              // [T, H, VD], contiguous
    const float *carry;     // joined states [segs, H, KD, VD]
    const float *init;      // [N, H, KD, VD] or NULL: what enters a sequence
    float *fin;             // what leaves it, or NULL (not with DOT, whose states lie turned in memory)
    float pair_scale, in_scale, up_scale;
    Role e;                 // DOT: rows that the part of the result from the state that enters is multiplied with; states are [VD][KD]
    float *dot;             // DOT: [T, H]; forwards with what passes all of a chunk at its last token
    float *between;         // DOT: states [blocks of the launch, seg / C], as lanes hold them, that enter chunks from the ones behind them, which
                            // the walk from the end writes and the one forwards reads
    const float *end, *last; // DOT forwards: the states that enter segments from behind [segs, H, KD, VD], and sequences [N, H, KD, VD] or NULL
};
// Which walk of a launch a block does: its segment and head, its turn among the blocks that share the segment, its place
// among the blocks of the head and their number, its place in the launch.
struct Place {
    int seg, h, turn, at, of, block;
};

// The pairs' weights go in as two parts.
constexpr int PARTS = 2;
template <int DT, int KD, int VD> struct WalkLds {
    Tile<PLANES<DT>, KD> q, k;
    Tile<PLANES<DT>, VD> v;
    u32x4 pair[4][2][PARTS][64];      // operands of the pairs' weights: 16 columns (tokens i), 32 tokens j, part, lane
    Clock clock[2];
    float dots[WAVES<VD>][C], passing[WAVES<VD>];
    int from[VD];       // PICKED: the first token of the chunk whose value in a column is not finite, C for none
};

// Puts values that are not finite to 0 in LDS, and notes where each column has its first. A thread takes a column.
template <int NP, int VD> __device__ __forceinline__ void take_out(Tile<NP, VD> &v, int (&from)[VD]) {
    if (threadIdx.x < VD) {
        int first = C;
#pragma unroll 1
        for (int t = C - 1; t >= 0; --t) {
            const int at = v.at(t) + threadIdx.x;
            if ((v.x[0][at] & 0x7f80) != 0x7f80) continue;      // (as bf16: the first part of an fp16 value is infinite or NaN where that is)
            first = t;
#pragma unroll
            for (int p = 0; p < NP; ++p) v.x[p][at] = 0;
        }
        from[threadIdx.x] = first;
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

// Returns whether this wave has met a value that is not finite (not with DOT or REV). Such a value makes NaN of its column in tokens of its chunk
// before it, whose weights for it are 0: a walk that is PICKED takes them out and puts NaN where they reach.
template <int DT, int KD, int VD, bool REV, bool DOT, bool PICKED = false>
__device__ __forceinline__ bool walk(const Batch &b, const Walk &a, const Place &place, WalkLds<DT, KD, VD> &L) {
    constexpr int NP = PLANES<DT>, NT = THREADS<VD>, NW = WAVES<VD>, IN = DOT ? 3 : 2;      // IN: parts of the state in its product with q
    using E = typename Elem<DT>::type;
    typedef E E4 __attribute__((ext_vector_type(4)));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int seg = place.seg, h = place.h;
    const Offsets o = b.offsets();
    const int s0 = seg * b.seg, s1 = s0 + b.seg < b.T ? s0 + b.seg : b.T;
    constexpr int SIZE = KD * VD;
    // empty sequences, spread over the segments: what enters them leaves them
    if (a.fin && (b.cu || !b.T)) {
        for (int64_t n0 = (int64_t)place.at * 64; n0 < b.N; n0 += (int64_t)place.of * 64) {
            const int n = (int)n0 + lane;
            uint64_t none = __ballot(n < b.N && o.at(n) >= o.at(n + 1));
            while (none) {
                const int at = (int)n0 + __builtin_ctzll(none);
                none &= none - 1;
                for (int x = threadIdx.x; x < SIZE; x += NT) {
                    const int64_t to = ((int64_t)at * b.H + h) * SIZE + x;
                    a.fin[to] = a.init ? a.init[to] : 0.0f;
                }
            }
        }
    }
    const Rows rq(a.q, h), rk(a.k, h), rv(a.v, h), re(a.e, h);
    float *const dots = DOT ? a.dot + h : nullptr;
    Chunks<REV> chunks(o, s0, s1, b.turns, place.turn);
    Stage<DT, KD, NT> sq, sk;
    Stage<DT, VD, NT> sv;
    float decay = 0.0f;
    auto load = [&](const Chunk &c) {
        if (wave == 0) decay = b.decay(c.first, c.len, h);
        sq.load(rq, c.first, c.len);
        sk.load(rk, c.first, c.len);
        sv.load(rv, c.first, c.len);
    };
    auto put_dots = [&](int first, int len) {
        if ((int)threadIdx.x < len) {
            float sum = L.dots[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < NW; ++w) sum += L.dots[w][threadIdx.x];
            if (!REV && (int)threadIdx.x == len - 1) {
                float pass = L.passing[0];
#pragma unroll
                for (int w = 1; w < NW; ++w) pass += L.passing[w];
                sum += pass;
            }
            (dots + (uint64_t)(uint32_t)first * (uint32_t)b.H)[threadIdx.x * (uint32_t)b.H] = sum;
        }
    };
    // (only the last chunk of a part may be short: no two others begin in the same 64 tokens of the segment)
    auto between = [&](const Chunk &c) { return a.between + ((int64_t)place.block * (b.seg / C) + (c.first - s0) / C) * SIZE; };
    Chunk c = chunks.next();
    int before_first = 0, before_len = 0, turn = 0;
    bool met = false;
    load(c);
    if (wave == 0) tick<REV>(L.clock[0], decay, a.in_scale, a.up_scale);
#pragma unroll 1
    while (c.len) {      // a part
        f32x4 S[KD / 16];
        load_state<KD, VD, DOT>(S, c.open ? (a.init ? a.init + ((int64_t)c.seq * b.H + h) * SIZE : nullptr)
                                          : a.carry + ((int64_t)(REV ? seg + 1 : seg - 1) * b.H + h) * SIZE, wave);
        bool leave;
#pragma unroll 1
        do {
        const Chunk then = chunks.next();
        const Clock &clock = L.clock[turn];
        f32x4 Y[DOT && !REV ? KD / 16 : 1];
        if constexpr (DOT && !REV)
            load_either<KD, VD>(Y, !c.leave ? between(c) : !c.close ? a.end + ((int64_t)(seg + 1) * b.H + h) * SIZE
                                          : a.last ? a.last + ((int64_t)c.seq * b.H + h) * SIZE : nullptr, wave, !c.leave);
        lds_barrier();
        if constexpr (DOT) put_dots(before_first, before_len);
        sq.store(L.q);
        sk.store(L.k);
        sv.store(L.v);
        if constexpr (!REV && !DOT && !PICKED) met |= __any(sv.not_finite());
        lds_barrier();
        if constexpr (PICKED) {
            take_out(L.v, L.from);
            lds_barrier();
        }
        if constexpr (DOT && !REV) {
            const float total = clock.total;
            float pass = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KD / 16; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) pass = __builtin_fmaf(total * S[kt][r], Y[kt][r], pass);
            pass = swap16_add(pass, pass);
            pass = row_suffix(swap32_add(pass, pass));
            if (lane == 0) L.passing[wave] = pass;
            hold();
        }
        load(then);
        if constexpr (DOT && REV)       // (after the loads, which would wait for it)
            if (!c.enter) store_lanes<KD, VD>(S, between(c), wave);
        // weights of the pairs: columns 16 tokens i, rows 32 tokens j, an operand a wave (two of four waves' each)
#pragma unroll 1
        for (int f = wave; f < 8; f += NW) {
            const int it = f >> 1, s = f & 1;
            if (REV ? 2 * s + 1 < it : 2 * s > it) continue;      // no pairs there
            f32x4 st[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int n = 0; n < KD / 32; ++n) {
                u32x4 qq[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) qq[p] = row_operand(L.q, p, it, n);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    u32x4 kk[NP];
#pragma unroll
                    for (int p = 0; p < NP; ++p) kk[p] = row_operand(L.k, p, 2 * s + t, n);
                    pairs<NP, NP, 4>([&](int x, int y) { st[t] = mma(kk[x], qq[y], st[t]); });
                }
            }
            const int ti = 16 * it + i;
            const float wi = clock.whole[ti], ri = clock.rest[ti];
            float x[8];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int j0 = 32 * s + 16 * t + 4 * g;
                const f32x4 wj = *reinterpret_cast<const f32x4 *>(&clock.whole[j0]);
                const f32x4 rj = *reinterpret_cast<const f32x4 *>(&clock.rest[j0]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float y = REV ? (wj[r] - wi) + (rj[r] - ri) : (wi - wj[r]) + (ri - rj[r]);
                    x[4 * t + r] = (REV ? j0 + r >= ti : j0 + r <= ti) ? st[t][r] * exp2_f(y) * a.pair_scale : 0.0f;
                }
            }
            u32x4 part[PARTS];
            split<PARTS>(x, part);
#pragma unroll
            for (int n = 0; n < PARTS; ++n) L.pair[it][s][n][lane] = part[n];
        }
        lds_barrier();
        // from the state that enters: columns are tokens, rows value elements of the wave
        f32x4 acc[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) acc[it] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KD / 32; ++s) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = S[2 * s][r], x[4 + r] = S[2 * s + 1][r];
            u32x4 part[IN];
            split<IN>(x, part);
#pragma unroll
            for (int it = 0; it < 4; it += 2) {     // (products into one result wait for each other: two in turn)
                u32x4 qq[2][NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) qq[0][p] = row_operand(L.q, p, it, s), qq[1][p] = row_operand(L.q, p, it + 1, s);
                pairs<IN, NP, IN>([&](int x, int y) {
                    acc[it] = mma(part[x], qq[0][y], acc[it]);
                    acc[it + 1] = mma(part[x], qq[1][y], acc[it + 1]);
                });
                if constexpr (DOT) hold();
            }
            hold();
        }
        Buffer e = buffer(nullptr, 0);
        if constexpr (DOT) e = re.from(c.first, c.len, VD);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            acc[it] *= clock.in[16 * it + i];
            if constexpr (DOT) {
                float sum = 0.0f;
                const E4 x = __builtin_bit_cast(E4, __builtin_amdgcn_raw_buffer_load_b64(e, (16 * it + i) * re.row + 2 * (16 * wave + 4 * g), 0, 0));
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(acc[it][r], (float)x[r], sum);
                sum = swap16_add(sum, sum);
                sum = swap32_add(sum, sum);
                if (g == 0) L.dots[wave][16 * it + i] = sum;
            }
        }
        hold();
        // from the chunk's own tokens
        u32x4 v[NP][2];
        value_operands(L.v, wave, v);
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (REV ? 2 * s + 1 < it : 2 * s > it) continue;
                u32x4 part[PARTS];
#pragma unroll
                for (int n = 0; n < PARTS; ++n) part[n] = L.pair[it][s][n][lane];
                pairs<NP, PARTS, 2>([&](int x, int y) { acc[it] = mma(v[x][s], part[y], acc[it]); });
            }
        if constexpr (PICKED) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int from = L.from[16 * wave + 4 * g + r];
#pragma unroll
                for (int it = 0; it < 4; ++it)
                    if (16 * it + i >= from) acc[it][r] = __builtin_nanf("");
            }
            if (L.from[16 * wave + i] < C) {
#pragma unroll
                for (int kt = 0; kt < KD / 16; ++kt) S[kt] = f32x4{} + __builtin_nanf("");
            }
        }
        const uint32_t out_row = 2 * (uint32_t)(b.H * VD);
        const Buffer out = buffer((char *)a.out + ((int64_t)c.first * b.H + h) * (2 * VD), (c.len - 1) * out_row + 2 * VD);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            E4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = (E)acc[it][r];
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), out, (16 * it + i) * out_row + 2 * (16 * wave + 4 * g), 0, 0);
        }
        hold();
        leave = c.leave;
        // exact where the state ends in fp32: a final state (that of the part), gradients of decays
        if (!leave || (c.close && a.fin)) {
            update<NP, KD, DOT ? 3 : 2>(S, L.k, v, clock);
            if constexpr (!DOT)
                if (c.close && a.fin) refine<NP, KD>(S, L.k, v, clock);
        }
        if constexpr (!DOT)
            if (leave && c.close && a.fin) store_state<KD, VD>(S, a.fin + ((int64_t)c.seq * b.H + h) * SIZE, wave);
        if (wave == 0) tick<REV>(L.clock[turn ^ 1], decay, a.in_scale, a.up_scale);
        before_first = c.first, before_len = c.len;
        turn ^= 1;
        c = then;
        } while (!leave);
    }
    if constexpr (DOT) {
        lds_barrier();
        put_dots(before_first, before_len);
    }
    return met;
}

// The second argument of launch bounds, waves a SIMD: two blocks on a CU where LDS holds them.
template <int DT, int VD> constexpr int WAVES_A_SIMD = (PLANES<DT> == 1 ? 2 : 1) * WAVES<VD> / 4;

// Blocks that run at once on 256 CUs: two a CU where LDS holds them.
template <int DT, int KD, int VD> constexpr int RUN = 256 * (2 * sizeof(WalkLds<DT, KD, VD>) <= 160 * 1024 ? 2 : 1);

// Tokens of a segment: short enough for `blocks` blocks (segments x heads) where the batch has the chunks for it.
inline int segment(int64_t T, int64_t H, int64_t blocks, int64_t least) {
    const int64_t want = ceil_div(T * H, blocks);
    const int64_t len = ceil_div(want < T ? want : T, C) * C;
    return (int)(len < least ? least : len);
}

// Blocks that share the parts of a segment in the forward's walk: more than one where segments hold many. Of 32 heads, 64 single
// tokens (us, with states) 68 for 401, 64 beside a prompt of 4096 223 for 507; 16 heads, 512 sequences of 16 tokens, which fill the card
// without, 270 for 266 (110 for 89 without states). 4 blocks leave 294 of the 507, 16 the same 223.
inline int turns(int64_t S, int64_t segs) {
    const int64_t most = 8, parts = ceil_div(S, segs);
    return (int)(parts < 2 ? 1 : parts < most ? parts : most);
}

}  // namespace
}  // namespace lin
}  // namespace ops
}  // namespace kda
