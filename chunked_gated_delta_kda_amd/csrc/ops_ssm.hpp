// ops_ssm.hpp -- what the kernels of the selective state space scan share.
//
// Per channel c (of group g = c / (D/G)) and state n, in fp32:
//
//   s_t = softplus(delta_t[c] + bias[c])   (or without softplus)
//   h_t[n] = e^{s_t A[c][n]} h_{t-1}[n] + s_t u_t[c] B_t[g][n]
//   out_t  = (sum_n C_t[g][n] h_t[n] + Dskip[c] u_t[c]) * silu(z_t[c])
//
// A wave owns 16 CB channels of one group and all their states, as M times the four 16 x 16
// blocks (states x channels) of a v_mfma_f32_16x16x1_4b_f32 result: lane l = 16 g + i, register
// 4 b + j of product m holds channel 16 (b % CB) + i and state 16 (b / CB + m 4/CB) + 4 g + j. So
// 4 CB-channel blocks serve state sizes up to 16 (CB = 4), 32 (2), 64 (1), and M products up
// to 64 M. The recurrence's outer product s u (x) B is that instruction's own: with a h as its
// addend it forms h in 41 cycles, where 16 multiplications would take 64 (measured; fp32 MFMA and
// vector instructions share the issue here, so nothing hides behind it).
// The "natural" lane order is that of the instruction's channel operand: lane l carries channel
// 16 (g % CB) + i of the wave, so activations are loaded, and outputs stored, one element a
// lane, at any stride and alignment; step sizes and C rows reach the other order through a
// few KiB of LDS that only this wave touches.
#pragma once

#include <type_traits>

#include "ops_common.hpp"
#include "ops_launch.hpp"

namespace kda {
namespace ops {
namespace ssm {

constexpr int WAVES = 4;      // independent waves of a block

// One element of a row, from the row's address and the lane's own offset in bytes.
template <int DT> __device__ __forceinline__ typename Elem<DT>::type at(const char *row, uint32_t bytes) {
    return *reinterpret_cast<const typename Elem<DT>::type *>(row + bytes);
}
// A row's address that all lanes share, held in scalar registers (and known to be global memory): an
// access to it plus a lane's 32-bit offset then needs no address arithmetic of the lanes.
#define KDA_GLOBAL __attribute__((address_space(1)))
template <class P> __device__ __forceinline__ KDA_GLOBAL P *uniform(P *row) {
    KDA_GLOBAL P *g = (KDA_GLOBAL P *)row;
    asm("" : "+s"(g));
    return g;
}
template <int DT> __device__ __forceinline__ typename Elem<DT>::type at(KDA_GLOBAL const char *row, uint32_t bytes) {
    return *(KDA_GLOBAL const typename Elem<DT>::type *)(row + bytes);
}
// K rows of an array from row t on, those past `last` (0 .. K - 1) row `last` again: one 64-bit product an array
// and a few scalar operations a row. Strides of KDA_SSM_MAX_STRIDE = 2^27 elements keep 8 rows of fp32 under 2^32 bytes.
struct RowsOf {
    const char *first;
    uint32_t step;
    __device__ __forceinline__ RowsOf(const char *p, int64_t stride, int t, uint32_t es) : step((uint32_t)stride * es) {
        first = p + (uint64_t)(uint32_t)t * step;
    }
    __device__ __forceinline__ KDA_GLOBAL const char *at(int k, int last) const {
        return uniform(first + (uint32_t)(k < last ? k : last) * step);
    }
};
static_assert(7ull * KDA_SSM_MAX_STRIDE * 4 < (1ull << 32), "eight rows within 32 bits");

template <class E> __device__ __forceinline__ void put(KDA_GLOBAL char *row, uint32_t bytes, E v) { *(KDA_GLOBAL E *)(row + bytes) = v; }

// The step of delta + bias. Both forms are computed and one is taken: a branch here would keep the
// compiler from interleaving the tokens of a stage.
__device__ __forceinline__ float step_of(float d, bool softplus) {
    const float s = softplus_f(d);
    return softplus ? s : d;
}

template <int DT> __device__ __forceinline__ float load1(const void *p, int64_t off) {
    return (float)reinterpret_cast<const typename Elem<DT>::type *>(p)[off];
}

// One wave's place: its channels, its tile of tokens, its lane's part of both orders.
template <int CB, int M>
struct Place {
    static constexpr int NB = 4 / CB;       // 16-state blocks of one product
    static constexpr int CHANNELS = 16 * CB;
    int lane, i, g;
    int group;         // of B and C
    int ch;            // natural channel; past the group's last one, that one again: everything about
                       // such a channel is a copy, and what its lane stores is the same value
    bool mine;         // natural channel exists and this is the one lane that stores it
    int base, last;    // first channel of the wave, last channel of the group
    int N;
    __device__ __forceinline__ Place(const kda_ssm_args &a, int block) {
        lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
        N = a.state_size;
        const int per = a.channels / a.groups;
        const int blocks = (per + CHANNELS - 1) / CHANNELS;
        group = block / blocks;
        base = group * per + (block - group * blocks) * CHANNELS;
        last = group * per + per - 1;
        const int want = base + 16 * (g % CB) + i;
        ch = want < last ? want : last;
        mine = want <= last && g < CB;
    }
    // state held by register 4 b + j of product m; channel of block b
    __device__ __forceinline__ int state(int m, int b, int j) const { return 16 * (b / CB + m * NB) + 4 * g + j; }
    __device__ __forceinline__ int channel(int b) const { return base + 16 * (b % CB) + i; }
    __device__ __forceinline__ int copied(int b) const { return channel(b) <= last ? channel(b) : last; }
    // state of this lane's element of the instruction's B-row operand of product m
    __device__ __forceinline__ int nat_state(int m) const { return 16 * (g / CB + m * NB) + i; }
};

template <int CB, int M>
__device__ __forceinline__ void load_decay(const kda_ssm_args &a, const Place<CB, M> &p, f32x16 (&A2)[M]) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = p.state(m, b, j);
                A2[m][4 * b + j] = n < p.N ? a.A[(int64_t)p.copied(b) * p.N + n] * LOG2E_F : 0.0f;
            }
}

// State [seq][channel][state] of fp32 memory to registers; zeros where `s` is NULL or the state lies past the last.
template <int CB, int M>
__device__ __forceinline__ void load_state(const float *s, int64_t seq, const kda_ssm_args &a, const Place<CB, M> &p,
                                           f32x16 (&h)[M]) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const float *row = s ? s + (seq * a.channels + p.copied(b)) * p.N : nullptr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = p.state(m, b, j);
                h[m][4 * b + j] = row && n < p.N ? row[n] : 0.0f;
            }
        }
}
template <int CB, int M>
__device__ __forceinline__ void store_state(float *s, int64_t seq, const kda_ssm_args &a, const Place<CB, M> &p,
                                            const f32x16 (&h)[M]) {
    if (!s) return;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int c = p.channel(b);
            if (c > p.last) continue;
            float *row = s + (seq * a.channels + c) * p.N;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (p.state(m, b, j) < p.N) row[p.state(m, b, j)] = h[m][4 * b + j];
        }
}
// The state of an empty sequence passes through.
template <int CB, int M>
__device__ __forceinline__ void pass_state(float *to, const float *from, int64_t seq, const kda_ssm_args &a,
                                           const Place<CB, M> &p) {
    if (!to) return;
    f32x16 h[M];
    load_state<CB, M>(from, seq, a, p, h);
    store_state<CB, M>(to, seq, a, p, h);
}

// A tile's states in the workspace, registers by lanes: [tile][block][16 M][64].
template <int M> __device__ __forceinline__ float *tile_state(float *ws, int64_t tile, int blocks, int block) {
    return ws + (tile * blocks + block) * (1024 * M);
}

// Sums over a channel's four lane groups, from block order (r[cb]: channel 16 cb + i) to the
// natural order.
template <int CB> __device__ __forceinline__ float to_natural(const float (&r)[CB]) {
    if constexpr (CB == 4) return swap16_add(swap32_add(r[0], r[2]), swap32_add(r[1], r[3]));
    else if constexpr (CB == 2) {
        const float s = swap16_add(r[0], r[1]);
        return swap32_add(s, s);
    } else {
        const float s = swap16_add(r[0], r[0]);
        return swap32_add(s, s);
    }
}

// a wave's own LDS traffic stays in program order; the compiler must keep it so too
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The step sizes of CB channels of one staged token, and its C rows.
template <int CB> __device__ __forceinline__ void read_steps(const float *row, int i, float (&s)[CB]) {
    if constexpr (CB == 4) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(row + 4 * i);
#pragma unroll
        for (int b = 0; b < 4; ++b) s[b] = v[b];
    } else {
#pragma unroll
        for (int b = 0; b < CB; ++b) s[b] = row[CB * i + b];
    }
}

// The states that the tiles start from: the tiles' maps h -> e^{A S} h + E (E alone where `alone` says so) one
// after another, from h = 0, for one register (r) of one block's lanes: what enters a tile takes its E's place.
// back: from the last tile to the first. The four waves of the calling block take a quarter of the tiles each:
// their quarters' maps first, then the states, so that the chain of loads is half as long as the tiles. Loads
// of AHEAD tiles are in flight together.
struct JoinLds {
    float P[4][64], E[4][64];
    int cut[4];
};
template <int CB, int M>
__device__ __forceinline__ void join_tiles(const kda_ssm_args &a, JoinLds &lds, float *states, const float *sums, const int32_t *alone,
                                           int alone_step, int tiles, int blocks, int block, int r, bool back) {
    constexpr int AHEAD = 8;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place<CB, M> p(a, block);
    const int c = p.copied((r % 16) / 4), n = p.state(r / 16, (r % 16) / 4, r % 4);
    const float A2 = n < p.N ? a.A[(int64_t)c * p.N + n] * LOG2E_F : 0.0f;
    const int64_t step = (int64_t)blocks * 1024 * M;
    float *at = states + (int64_t)block * (1024 * M) + r * 64 + p.lane;
    const int quarter = (tiles + 3) / 4, lo = w * quarter, hi = lo + quarter < tiles ? lo + quarter : tiles;
    float P = 1.0f, h = 0.0f;
    bool cut = false;
    auto walk = [&](auto write) {
        for (int k0 = lo; k0 < hi; k0 += AHEAD) {
            float E[AHEAD], S[AHEAD];
            int al[AHEAD];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const int f = k0 + q < hi ? k0 + q : hi - 1, k = back ? tiles - 1 - f : f;
                E[q] = at[k * step];
                S[q] = sums[(int64_t)k * a.channels + c];
                al[q] = alone[k * alone_step];
            }
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                if (k0 + q < hi) {
                    const int k = back ? tiles - 1 - (k0 + q) : k0 + q;
                    if (write) at[k * step] = h;
                    const float d = exp2_f(A2 * S[q]);
                    if (!write) P *= d, cut = cut || al[q];
                    h = al[q] ? E[q] : __builtin_fmaf(d, h, E[q]);
                }
            }
        }
    };
    walk(std::false_type{});
    lds.P[w][p.lane] = P, lds.E[w][p.lane] = h;
    if (p.lane == 0) lds.cut[w] = cut;
    __syncthreads();
    h = 0.0f;
    for (int v = 0; v < w; ++v) h = lds.cut[v] ? lds.E[v][p.lane] : __builtin_fmaf(lds.P[v][p.lane], h, lds.E[v][p.lane]);
    walk(std::true_type{});
}

// Host side: the form of a state size, and the tiles of a batch.
struct Form {
    int cb, m;
};
inline Form form_of(int N) { return N <= 16 ? Form{4, 1} : N <= 32 ? Form{2, 1} : N <= 64 ? Form{1, 1} : N <= 128 ? Form{1, 2} : Form{1, 4}; }
int tile_len(int64_t T, int64_t blocks);
inline int64_t blocks_of(const Form &f, int64_t D, int64_t G) { return G * ceil_div(D / G, 16 * f.cb); }

}  // namespace ssm
}  // namespace ops
}  // namespace kda
