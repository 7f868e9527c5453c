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
#pragma once

#include "ops_common.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace lin {
namespace {

constexpr int C = 64;              // tokens of a chunk
constexpr int PAD = 8;             // elements behind a row in LDS: rows 4 banks apart

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

// 8 fp32 numbers as N bf16 numbers each: each the rounding of what those before it leave.
template <int N> __device__ __forceinline__ void split(const float (&x)[8], u32x4 (&to)[N]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        bf16x8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (__bf16)r[i];
        to[n] = __builtin_bit_cast(u32x4, h);
        if (n + 1 < N) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] -= (float)h[i];
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

// One chunk of rows in LDS.
template <int NP, int D> struct Tile {
    uint16_t x[NP][C][D + PAD];
};

// An input in one of the three roles: rows [T, H, D], contiguous elements.
struct Role {
    const void *p;
    int64_t row, head;       // strides, elements
};

// Rows of a chunk on their way from memory to LDS, 8 elements of a row a time. NT: threads of the block. Offsets from
// a chunk's first row fit 32 bits (strides are at most KDA_LIN_MAX_STRIDE).
template <int DT, int D, int NT> struct Stage {
    static constexpr int N = C * D / 8 / NT, ROWS = NT / (D / 8);     // rows of a piece
    u32x4 r[N];
    __device__ __forceinline__ void load(const Role &s, int h, int first, int len) {
        const char *p = (const char *)s.p + 2 * ((int64_t)first * s.row + (int64_t)h * s.head);
        const uint32_t row = threadIdx.x / (D / 8), at = 2 * (row * (uint32_t)s.row + 8 * (threadIdx.x % (D / 8)));
#pragma unroll
        for (int n = 0; n < N; ++n) {
            r[n] = u32x4{0, 0, 0, 0};
            if ((int)row + ROWS * n < len) r[n] = *reinterpret_cast<const u32x4 *>(p + 2 * ROWS * n * s.row + at);
        }
    }
    __device__ __forceinline__ void store(Tile<PLANES<DT>, D> &t) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int row = threadIdx.x / (D / 8) + ROWS * n, col = 8 * (threadIdx.x % (D / 8));
            if constexpr (DT == KDA_DTYPE_BF16) *reinterpret_cast<u32x4 *>(&t.x[0][row][col]) = r[n];
            else {
                typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
                const f16x8 e = __builtin_bit_cast(f16x8, r[n]);
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
                u32x4 part[2];
                split<2>(v, part);
                *reinterpret_cast<u32x4 *>(&t.x[0][row][col]) = part[0];
                *reinterpret_cast<u32x4 *>(&t.x[1][row][col]) = part[1];
            }
        }
    }
};

// Operands of v_mfma_f32_16x16x32: a lane (i = lane & 15, g = lane >> 4) holds 8 numbers of row (or column) i. Their places in
// the contraction are relabelled alike in both operands: slot 8 g + s is place 4 g + s for s < 4, 16 + 4 g + s - 4 else,
// where a result (rows 4 g + r of column i) of two 16-row tiles leaves its numbers, so that results are operands as
// they are.
// of row 16 t + i, elements 32 s ..
template <int NP, int D> __device__ __forceinline__ u32x4 row_operand(const Tile<NP, D> &m, int plane, int t, int s) {
    const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const uint16_t *p = &m.x[plane][16 * t + i][32 * s + 4 * g];
    const u32x2 a = *reinterpret_cast<const u32x2 *>(p), b = *reinterpret_cast<const u32x2 *>(p + 16);
    return u32x4{a[0], a[1], b[0], b[1]};
}
// of element 16 t + i, rows 32 s ..: a transposing read hands the 16 lanes of a row of 16 columns a column of 4 rows each
template <int NP, int D> __device__ __forceinline__ u32x4 column_operand(const Tile<NP, D> &m, int plane, int t, int s) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const uint16_t *p = &m.x[plane][32 * s + 4 * g + (i >> 2)][16 * t + 4 * (i & 3)];
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * (D + PAD)));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return u32x4{x[0], x[1], y[0], y[1]};
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

// by one wave, lane t for token t: x, log2 of the token's decay, 0 past the chunk's end. Returns the chunk's sum.
template <bool REV> __device__ __forceinline__ double tick(Clock &c, double x, float in_scale, float up_scale) {
    const int lane = threadIdx.x & 63;
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
// start from a part's first token in both directions.
struct Chunk {
    int first, len;      // len 0: none
    int seq;
    bool enter, leave;   // the first, the last of its part
    bool open, close;    // (with enter) the sequence begins here, (with leave) it ends here
};

template <bool REV> struct Chunks {
    Offsets o;
    int s0, s1, at, seq, p0, p1;     // the part [p0, p1); at: the next chunk's first token (REV: the end of the rest)
    bool fresh;
    __device__ __forceinline__ Chunks(const Offsets &off, int a, int b) : o(off), s0(a), s1(b), at(REV ? b : a), seq(-1), p0(0), p1(0), fresh(true) {}
    // the sequence of token t, next to the last one where that is so
    __device__ __forceinline__ int find(int t) const {
        if (seq >= 0) {
            const int n = REV ? seq - 1 : seq + 1;
            if (n >= 0 && n < o.N && o.at(n) <= t && t < o.at(n + 1)) return n;
        }
        return o.find(t);
    }
    __device__ __forceinline__ Chunk next() {
        Chunk c = {0, 0, 0, false, false, false, false};
        if (REV ? at <= s0 : at >= s1) return c;
        if (fresh) {
            const int t = REV ? at - 1 : at;
            seq = find(t);
            const int b = o.at(seq), e = o.at(seq + 1);
            p0 = REV ? (b < s0 ? s0 : b > t ? t : b) : t;            // (clamped where offsets are out of order)
            p1 = REV ? t + 1 : (e > s1 ? s1 : e <= t ? t + 1 : e);
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
        // (only the part at the segment's edge continues what lies beyond, whatever the offsets say)
        const bool begins = o.at(seq) >= p0 || p0 != s0, ends = o.at(seq + 1) <= p1 || p1 != s1;
        c.open = REV ? ends : begins;
        c.close = REV ? begins : ends;
        fresh = c.leave;
        return c;
    }
};

// S <- total S + sum_j k_j (up_j v_j)^T over a chunk, for the wave's columns. v's operands as the second product wants them.
template <int NP, int KD>
__device__ __forceinline__ void update(f32x4 (&S)[KD / 16], const Tile<NP, KD> &k, const u32x4 (&v)[NP][2], const Clock &clock) {
    const int g = (threadIdx.x & 63) >> 4;
    const float total = clock.total;
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt) S[kt] *= total;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(&clock.up[32 * s + 4 * g]);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(&clock.up[32 * s + 16 + 4 * g]);
        float x[8];
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
        u32x4 w[3];
        split<3>(x, w);
#pragma unroll
        for (int kt = 0; kt < KD / 16; ++kt) {
            u32x4 row[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) row[p] = column_operand(k, p, kt, s);
            pairs<NP, 3, 3>([&](int p, int n) { S[kt] = mma(row[p], w[n], S[kt]); });
        }
    }
}

template <int NP, int VD> __device__ __forceinline__ void value_operands(const Tile<NP, VD> &v, int wave, u32x4 (&to)[NP][2]) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int s = 0; s < 2; ++s) to[p][s] = column_operand(v, p, wave, s);
}

// A state [KD][VD] between memory (element (a, b) at a sk + b sv) and the wave's columns. p NULL: zeros.
template <int KD> __device__ __forceinline__ void load_state(f32x4 (&S)[KD / 16], const float *p, int sk, int sv, int wave) {
    const uint32_t at = 4 * ((threadIdx.x & 63) >> 4) * sk + (16 * wave + (threadIdx.x & 15)) * sv;
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[kt][r] = p ? (p + (16 * kt + r) * sk)[at] : 0.0f;
}
template <int KD> __device__ __forceinline__ void store_state(const f32x4 (&S)[KD / 16], float *p, int sk, int sv, int wave) {
    const uint32_t at = 4 * ((threadIdx.x & 63) >> 4) * sk + (16 * wave + (threadIdx.x & 15)) * sv;
#pragma unroll
    for (int kt = 0; kt < KD / 16; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) (p + (16 * kt + r) * sk)[at] = S[kt][r];
}

// The batch and its segments.
struct Batch {
    const int32_t *cu;
    const float *g;         // decays [T, H] or [H]
    int64_t g_row;          // 0 where they are [H]
    int N, T, H, seg, segs; // seg: tokens of a segment (a multiple of C); segs of them
    __device__ __forceinline__ Offsets offsets() const { return Offsets{cu, N, T}; }
    __device__ __forceinline__ float decay(int t, int h) const { return g[(int64_t)t * g_row + h]; }
};

// ---------------------------------------------------------------- segments' own states
// Forwards: what the last sequence of segment blockIdx.x, if it goes on behind it, adds to the state there (from its
// initial state where it begins in the segment); factor: what is left of the state before the segment, or -1 where the sequence begins in it.
// Backwards the same from the other end.
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
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, seg = blockIdx.x, h = blockIdx.y;
    const Offsets o = b.offsets();
    const int s0 = seg * b.seg, s1 = s0 + b.seg < b.T ? s0 + b.seg : b.T;
    float *factor = a.factor + (int64_t)seg * b.H + h;
    // the part that goes on past the segment
    int p0 = s0, p1 = s1;
    bool open, on;
    const int edge = REV ? s0 : s1 - 1, seq = o.find(edge), sb = o.at(seq), se = o.at(seq + 1);
    if constexpr (REV) on = sb < s0, open = se <= s1, p1 = se < s1 ? (se <= s0 ? s0 + 1 : se) : s1;
    else on = se > s1, open = sb >= s0, p0 = sb > s0 ? (sb >= s1 ? s1 - 1 : sb) : s0;
    if (!on) {
        if (threadIdx.x == 0) *factor = -1.0f;
        return;
    }
    f32x4 S[KD / 16];
    load_state<KD>(S, open && a.init ? a.init + ((int64_t)seq * b.H + h) * (KD * VD) : nullptr, VD, 1, wave);
    double sum = 0.0, g = 0.0;
    Stage<DT, KD, NT> sk;
    Stage<DT, VD, NT> sv;
    const int count = (p1 - p0 + C - 1) / C;
    auto load = [&](int n) {
        const int first = p0 + C * (REV ? count - 1 - n : n), len = p1 - first < C ? p1 - first : C;
        if (wave == 0) g = lane < len ? log2_decay(b.decay(first + lane, h)) : 0.0;
        sk.load(a.k, h, first, len);
        sv.load(a.v, h, first, len);
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
        update<NP, KD>(S, L.k, v, L.clock[n & 1]);
        if (wave == 0 && n + 1 < count) sum += tick<REV>(L.clock[(n + 1) & 1], g, 1.0f, a.up);
    }
    store_state<KD>(S, a.state + ((int64_t)seg * b.H + h) * (KD * VD), VD, 1, wave);
    if (threadIdx.x == 0) *factor = open ? -1.0f : exp2_f((float)sum);
}

// ---------------------------------------------------------------- join
// state[s] <- what leaves segment s (backwards: what it hands to the one before), in the order of the segments.
constexpr int JOIN_THREADS = 256;
template <int SIZE> __device__ __forceinline__ void join(const Batch &b, float *state, const float *factor, bool rev) {
    const int h = blockIdx.y, x = blockIdx.x * JOIN_THREADS + threadIdx.x;
    float c = 0.0f;
    const int64_t step = (int64_t)b.H * SIZE;
    float *p = state + (int64_t)h * SIZE + x;
    constexpr int AHEAD = 8;
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

// ---------------------------------------------------------------- the walk
struct Walk {
    Role q, k, v;
    void *out;              // [T, H, VD], contiguous
    const float *carry;     // joined states [segs, H, KD, VD]
    const float *init;      // [N, H, KD, VD] or NULL: what enters a sequence
    float *fin;             // what leaves it, or NULL
    int sk, sv;             // strides of a state's elements in carry, init and fin
    float pair_scale, in_scale, up_scale;
    Role e;                 // DOT: rows that the part of the result from the state that enters is multiplied with
    float *dot;             // DOT: [T, H]
};

// The pairs' weights go in as two parts.
constexpr int PARTS = 2;
template <int DT, int KD, int VD> struct WalkLds {
    Tile<PLANES<DT>, KD> q, k;
    Tile<PLANES<DT>, VD> v;
    u32x4 pair[4][2][PARTS][64];      // operands of the pairs' weights: 16 columns (tokens i), 32 tokens j, part, lane
    Clock clock[2];
    float dots[WAVES<VD>][C];
};

template <int DT, int KD, int VD, bool REV, bool DOT>
__device__ __forceinline__ void walk(const Batch &b, const Walk &a, WalkLds<DT, KD, VD> &L) {
    constexpr int NP = PLANES<DT>, NT = THREADS<VD>, NW = WAVES<VD>, IN = DOT ? 3 : 2;      // IN: parts of the state in its product with q
    using E = typename Elem<DT>::type;
    typedef E E4 __attribute__((ext_vector_type(4)));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int seg = blockIdx.x, h = blockIdx.y;
    const Offsets o = b.offsets();
    const int s0 = seg * b.seg, s1 = s0 + b.seg < b.T ? s0 + b.seg : b.T;
    constexpr int SIZE = KD * VD;
    // empty sequences, spread over the segments: what enters them leaves them
    if (a.fin && b.cu) {
        for (int n0 = seg * 64; n0 < b.N; n0 += b.segs * 64) {
            const int n = n0 + lane;
            uint64_t none = __ballot(n < b.N && o.at(n) >= o.at(n + 1));
            while (none) {
                const int at = n0 + __builtin_ctzll(none);
                none &= none - 1;
                for (int x = threadIdx.x; x < SIZE; x += NT) {
                    const int64_t to = ((int64_t)at * b.H + h) * SIZE + x;
                    a.fin[to] = a.init ? a.init[to] : 0.0f;
                }
            }
        }
    }
    Chunks<REV> chunks(o, s0, s1);
    Stage<DT, KD, NT> sq, sk;
    Stage<DT, VD, NT> sv;
    double decay = 0.0;
    auto load = [&](const Chunk &c) {
        if (wave == 0) decay = lane < c.len ? log2_decay(b.decay(c.first + lane, h)) : 0.0;
        sq.load(a.q, h, c.first, c.len);
        sk.load(a.k, h, c.first, c.len);
        sv.load(a.v, h, c.first, c.len);
    };
    auto put_dots = [&](int first, int len) {
        if ((int)threadIdx.x < len) {
            float sum = L.dots[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < NW; ++w) sum += L.dots[w][threadIdx.x];
            a.dot[(int64_t)(first + threadIdx.x) * b.H + h] = sum;
        }
    };
    f32x4 S[KD / 16];
    Chunk c = chunks.next();
    int before_first = 0, before_len = 0, turn = 0;
    if (c.len) {
        load(c);
        if (wave == 0) tick<REV>(L.clock[0], decay, a.in_scale, a.up_scale);
    }
#pragma unroll 1
    while (c.len) {
        const Chunk then = chunks.next();
        const Clock &clock = L.clock[turn];
        lds_barrier();
        if constexpr (DOT) put_dots(before_first, before_len);
        sq.store(L.q);
        sk.store(L.k);
        sv.store(L.v);
        lds_barrier();
        if (then.len) load(then);
        if (c.enter) {
            const float *from = c.open ? (a.init ? a.init + ((int64_t)c.seq * b.H + h) * SIZE : nullptr)
                                       : a.carry + ((int64_t)(REV ? seg + 1 : seg - 1) * b.H + h) * SIZE;
            load_state<KD>(S, from, a.sk, a.sv, wave);
        }
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
            for (int it = 0; it < 4; ++it) {
                u32x4 qq[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) qq[p] = row_operand(L.q, p, it, s);
                pairs<IN, NP, IN>([&](int x, int y) { acc[it] = mma(part[x], qq[y], acc[it]); });
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            acc[it] *= clock.in[16 * it + i];
            if constexpr (DOT) {
                float sum = 0.0f;
                if (16 * it + i < c.len) {
                    const char *e = (const char *)a.e.p + 2 * ((int64_t)c.first * a.e.row + (int64_t)h * a.e.head);
                    const E4 x = *reinterpret_cast<const E4 *>(e + 2 * ((16 * it + i) * (uint32_t)a.e.row + 16 * wave + 4 * g));
#pragma unroll
                    for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(acc[it][r], (float)x[r], sum);
                }
                sum = swap16_add(sum, sum);
                sum = swap32_add(sum, sum);
                if (g == 0) L.dots[wave][16 * it + i] = sum;
            }
        }
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
        {
            char *out = (char *)a.out + 2 * (((int64_t)c.first * b.H + h) * VD);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                if (16 * it + i >= c.len) continue;
                E4 e;
#pragma unroll
                for (int r = 0; r < 4; ++r) e[r] = (E)acc[it][r];
                *reinterpret_cast<E4 *>(out + 2 * ((16 * it + i) * (uint32_t)(b.H * VD) + 16 * wave + 4 * g)) = e;
            }
        }
        if (!c.leave || (c.close && a.fin)) update<NP, KD>(S, L.k, v, clock);
        if (c.leave && c.close && a.fin) store_state<KD>(S, a.fin + ((int64_t)c.seq * b.H + h) * SIZE, a.sk, a.sv, wave);
        if (wave == 0 && then.len) tick<REV>(L.clock[turn ^ 1], decay, a.in_scale, a.up_scale);
        before_first = c.first, before_len = c.len;
        turn ^= 1;
        c = then;
    }
    if constexpr (DOT) {
        lds_barrier();
        put_dots(before_first, before_len);
    }
}

// The second argument of launch bounds, waves a SIMD: two blocks on a CU where LDS holds them.
template <int DT, int VD> constexpr int WAVES_A_SIMD = (PLANES<DT> == 1 ? 2 : 1) * WAVES<VD> / 4;

// Tokens of a segment: short enough for `blocks` blocks (segments x heads) where the batch has the chunks for it.
inline int segment(int64_t T, int64_t H, int64_t blocks, int64_t least) {
    const int64_t want = ceil_div(T * H, blocks);
    const int64_t len = ceil_div(want, C) * C;
    return (int)(len < least ? least : len);
}

}  // namespace
}  // namespace lin
}  // namespace ops
}  // namespace kda
