// ops_ssm_bwd.hip -- gradients of the selective state space scan. With dy' = dy silu(z), a_t = e^{s_t A}
// and dh_t the gradient of h_t (of h_last: the final state's):
//
//   dh_t = C_t dy'_t + a_{t+1} dh_{t+1},  dC_t = sum_c dy' h,  dB_t = sum_c dh s u,  du = s sum_n dh B + Dskip dy'
//   ds = sum_n dh A a h_{t-1} + u sum_n dh B,  ddelta = ds sigmoid(delta + bias),  dA = sum_t s dh a h_{t-1}
//
// Tiles of the time axis as in the forward, and the same layout of states (ops_ssm.hpp):
//   1. ssm_bwd_tile_kernel: each tile from a zero state, for both directions at once: its end state,
//      the gradient G that it sends to the state before it (sum_t P_t C_t dy'_t, P_t the product of
//      the decays so far: one exponential serves both), the local states before every KR-th token
//   2. ssm_bwd_join_kernel: states forward and gradients backward over the tiles
//   3. ssm_bwd_kernel: each tile from its end, KR tokens at a time: their decayed states again from the
//      stored state (completed by e^{A S} times the tile's first state), kept in registers, then the
//      gradients. Decays are formed again on the way back: the registers that would keep them cost
//      more than the exponential.
//   4. ssm_bwd_rows_kernel, ssm_bwd_params_kernel: the sums over channel blocks (dB, dC) and over
//      tiles (dA, dD, dbias), in a fixed order.
// A cell is KR tokens of the tiles' grid, a group what one sequence has of a cell: the kernels go from group to
// group, the cell's other tokens masked (no step, nothing in, nothing out; what they would store goes to a
// place that nobody reads), so that the code of the tokens knows no borders.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ops_ssm.hpp"

namespace kda {
namespace ops {
namespace ssm {
namespace {

template <int M> constexpr int KR_OF = 4 / M;   // tokens of a cell, whose decayed states are held: 64 registers

// Where the workspace keeps what, in floats.
struct Layout {
    int64_t units, subs;                    // (tile, block) pairs; stored states of a tile
    int64_t end_state, grad, local, sums, first_sums, dA, drow, rows, flags, none, total;
    // NP: states of a wave, 16 to a state block
    Layout(int64_t T, int64_t D, int64_t NP, int64_t tiles, int64_t blocks, int L, int M) {
        const int KR = 4 / M;
        units = tiles * blocks, subs = L / KR;
        const int64_t state = units * 1024 * M;
        end_state = 0;
        grad = end_state + state;
        local = grad + state;
        sums = local + state * subs;                 // [tile][sub][D]: step sums before each stored state
        first_sums = sums + tiles * subs * D;        // [tile][D]: of the whole tile
        dA = first_sums + tiles * D;
        drow = dA + state;                           // [tile][2][D]: dD, dbias
        rows = drow + 2 * tiles * D;                 // [block][T][2][NP]: dB, dC, NP the padded state size
        flags = rows + blocks * T * 2 * NP;          // [tile][2]
        none = flags + 2 * tiles + (-(flags + 2 * tiles) & 3);   // [2 NP or D]: where masked tokens store
        total = none + std::max(2 * NP, D);
    }
};

template <int DT, int M> struct RawBwd {
    using E = typename Elem<DT>::type;
    static constexpr int KB = KR_OF<M>;
    E delta[KB], u[KB], z[KB], dy[KB], B[KB][M], C[KB][M];
    template <int CB>
    __device__ __forceinline__ void load(const kda_ssm_args &a, const kda_ssm_grads &d, const Place<CB, M> &p, int t, int stop) {
        const uint32_t ch = (uint32_t)p.ch * sizeof(E);
        const int64_t g0 = (int64_t)p.group * p.N * sizeof(E);
        t = t < stop ? t : stop - 1;            // rows past the end: the last one again
        const int last = stop - 1 - t;
        const RowsOf dr((const char *)a.delta, a.delta_stride, t, sizeof(E)), ur((const char *)a.u, a.u_stride, t, sizeof(E));
        const RowsOf yr((const char *)d.dy, d.dy_stride, t, sizeof(E)), zr((const char *)a.z, a.z_stride, t, sizeof(E));
        const RowsOf Br((const char *)a.B + g0, a.B_stride, t, sizeof(E)), Cr((const char *)a.C + g0, a.C_stride, t, sizeof(E));
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            delta[k] = at<DT>(dr.at(k, last), ch);
            u[k] = at<DT>(ur.at(k, last), ch);
            dy[k] = at<DT>(yr.at(k, last), ch);
            if (a.z) z[k] = at<DT>(zr.at(k, last), ch);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int n = p.nat_state(m);
                const uint32_t st = (uint32_t)(n < p.N ? n : p.N - 1) * sizeof(E);
                B[k][m] = at<DT>(Br.at(k, last), st);
                C[k][m] = at<DT>(Cr.at(k, last), st);
            }
        }
    }
};

// Staged tokens of a wave in LDS: per channel (natural lane l at CB i + g % CB) and per state.
template <int CB, int M> struct StageTile {
    static constexpr int CH = 16 * CB, NS = 64 / CB * M, KB = KR_OF<M>;
    float s[KB][CH], x[KB][CH], dy[KB][CH];       // step, step times input, dy'
    float B[KB][NS], C[KB][NS];
};
template <int CB, int M> struct StageBwd : StageTile<CB, M> {     // and what the gradients need on top
    static constexpr int CH = 16 * CB, KB = KR_OF<M>;
    float u[KB][CH], sig[KB][CH], dz[KB][CH];     // input, sigmoid(delta + bias), dy silu'(z)
};

// Tokens lo to hi - 1 of a cell are staged, the others masked.
template <int DT, int CB, int M, class Stage>
__device__ __forceinline__ void stage(Stage &S, const RawBwd<DT, M> &raw, const kda_ssm_args &a, const Place<CB, M> &p,
                                      float bias, int lo, int hi, float &steps) {
    const int at = CB * p.i + p.g % CB;
#pragma unroll
    for (int k = 0; k < KR_OF<M>; ++k) {
        const bool on = k >= lo && k < hi;
        const float d = (float)raw.delta[k] + bias, u = (float)raw.u[k], dy = (float)raw.dy[k];
        const float z = (float)raw.z[k], sz = sigmoid_f(z);
        const float g = dy * (a.z ? z * sz : 1.0f);
        float s = step_of(d, a.delta_softplus);
        s = on ? s : 0.0f;
        steps += s;
        S.s[k][at] = s, S.x[k][at] = on ? s * u : 0.0f, S.dy[k][at] = on ? g : 0.0f;
        if constexpr (std::is_same_v<Stage, StageBwd<CB, M>>) {
            const float sd = sigmoid_f(d), sig = a.delta_softplus ? sd : 1.0f;
            S.u[k][at] = on ? u : 0.0f, S.sig[k][at] = on ? sig : 0.0f;
            S.dz[k][at] = dy * (sz * __builtin_fmaf(z, 1.0f - sz, 1.0f));
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const bool is = on && p.nat_state(m) < p.N;
            S.B[k][p.nat_state(m)] = is ? (float)raw.B[k][m] : 0.0f;
            S.C[k][p.nat_state(m)] = is ? (float)raw.C[k][m] : 0.0f;
        }
    }
    wave_fence();
}

template <int CB, int M>
__device__ __forceinline__ void operands(const float *row, const Place<CB, M> &p, float (&v)[M]) {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = row[p.nat_state(m)];
}

// x += f * state `s`[seq]
template <int CB, int M>
__device__ __forceinline__ void add_state(f32x16 (&x)[M], const f32x16 (&f)[M], const float *s, int64_t seq, const kda_ssm_args &a,
                                          const Place<CB, M> &p) {
    if (!s) return;
    f32x16 v[M];
    load_state<CB, M>(s, seq, a, p, v);
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[m][r] = __builtin_fmaf(f[m][r], v[m][r], x[m][r]);
}

// 8 x 1024 x 2048 x 16 bf16 with a gate: 111 us, 64% of the busy cycles issue vector instructions; 268 MB of states go out.
// Two waves a SIMD: with registers for four it spills (710 us for all kernels against 400), for three nothing changes. At
// two only the form of more than 128 states spills (about 300 registers).
template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_tile_kernel(const kda_ssm_args a, const kda_ssm_grads d, float *ws,
                                                                     const Layout lay, int32_t *err, int L, int tiles, int blocks) {
    constexpr int KR = KR_OF<M>;
    __shared__ __align__(16) StageTile<CB, M> stages[WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * WAVES + wave;
    if (unit >= (int64_t)tiles * blocks) return;
    const int tile = (int)(unit / blocks), block = (int)(unit - (int64_t)tile * blocks);
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    if (unit == 0) check_offsets(off, err, threadIdx.x & 63, 64);
    const Place<CB, M> p(a, block);
    const int T = a.total_tokens, t0 = tile * L, t1 = T - t0 < L ? T : t0 + L;
    int n = off.find(t0), start = off.at(n), end = off.at(n + 1);
    bool first = true, reset = start == t0;
    f32x16 A2[M], h[M], P[M], G[M], zero[M];
    load_decay<CB, M>(a, p, A2);
    load_state<CB, M>(reset ? a.initial_state : nullptr, n, a, p, h);
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) P[m][r] = 1.0f, G[m][r] = 0.0f, zero[m][r] = 0.0f;
    const float bias = a.delta_bias ? a.delta_bias[p.ch] : 0.0f;
    const int nat = CB * p.i + p.g % CB;
    float sum = 0.0f;
    StageTile<CB, M> &S = stages[wave];
    float *const grad = ws + lay.grad + unit * (1024 * M);
    auto store_grad = [&] {
#pragma unroll
        for (int r = 0; r < 16 * M; ++r) grad[r * 64 + p.lane] = G[r / 16][r % 16];
    };
    RawBwd<DT, M> raw{};
    raw.template load<CB>(a, d, p, t0, t1);
    int gs = t0;                                    // the group's first token
    while (gs < t1) {
        const int tb = t0 + (gs - t0) / KR * KR, cell_end = tb + KR < t1 ? tb + KR : t1, ge = end < cell_end ? end : cell_end;
        if (gs == tb) {                             // the state before the cell, and the steps so far
            const int64_t sub = (tb - t0) / KR;
            float *to = ws + lay.local + (unit * lay.subs + sub) * (1024 * M);
#pragma unroll
            for (int r = 0; r < 16 * M; r += 4)
                *reinterpret_cast<f32x4 *>(to + r * 64 + 4 * p.lane) =
                    f32x4{h[r / 16][r % 16], h[r / 16][r % 16 + 1], h[r / 16][r % 16 + 2], h[r / 16][r % 16 + 3]};
            if (p.mine) ws[lay.sums + ((int64_t)tile * lay.subs + sub) * a.channels + p.ch] = sum;
        }
        stage<DT, CB, M>(S, raw, a, p, bias, gs - tb, ge - tb, sum);
        if (ge == cell_end && ge < t1) raw.template load<CB>(a, d, p, ge, t1);
#pragma unroll
        for (int k = 0; k < KR; ++k) {
            float sc[CB], B[M], C[M];
            read_steps<CB>(S.s[k], p.i, sc);
            operands<CB, M>(S.B[k], p, B);
            operands<CB, M>(S.C[k], p, C);
            const float x = S.x[k][nat], dy = S.dy[k][nat];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                f32x16 e;
#pragma unroll
                for (int r = 0; r < 16; ++r) e[r] = exp2_f(A2[m][r] * sc[(r / 4) % CB]);
#pragma unroll
                for (int r = 0; r < 16; ++r) h[m][r] *= e[r];
                h[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(B[m], x, h[m], 0, 0, 0);
                const f32x16 w = __builtin_amdgcn_mfma_f32_16x16x1f32(C[m], dy, zero[m], 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    P[m][r] *= e[r];
                    G[m][r] = __builtin_fmaf(P[m][r], w[r], G[m][r]);
                }
            }
        }
        wave_fence();
        gs = ge;
        if (gs == end) {                            // the sequence ends: with the first one G is complete
            if (first) {
                add_state<CB, M>(G, P, d.d_final_state, n, a, p);
                store_grad();
            }
            first = false;
            if (gs < t1) {
                reset = true;
                for (++n; n < a.num_seqs - 1 && off.at(n + 1) <= gs; ++n) {}
                end = off.at(n + 1);
                load_state<CB, M>(a.initial_state, n, a, p, h);
            }
        }
    }
    if (first) store_grad();
    float *to = ws + lay.end_state + unit * (1024 * M);
#pragma unroll
    for (int r = 0; r < 16 * M; ++r) to[r * 64 + p.lane] = h[r / 16][r % 16];
    if (p.mine) ws[lay.first_sums + (int64_t)tile * a.channels + p.ch] = sum;
    if (block == 0 && p.lane == 0) {
        int32_t *f = reinterpret_cast<int32_t *>(ws + lay.flags) + 2 * tile;
        f[0] = reset;                       // a sequence starts in the tile: its end state stands alone
        f[1] = !first;                      // one ends in it: nothing of what lies behind reaches back
    }
}

// blockIdx.y 0: the state before every tile, in its end state's place; 1: the gradient that comes to
// every tile's end from the tiles behind it, in G's place.
template <int CB, int M>
__global__ __launch_bounds__(256) void ssm_bwd_join_kernel(const kda_ssm_args a, float *ws, const Layout lay, int tiles, int blocks) {
    __shared__ JoinLds lds;
    const bool back = blockIdx.y == 1;
    join_tiles<CB, M>(a, lds, ws + (back ? lay.grad : lay.end_state), ws + lay.first_sums,
                      reinterpret_cast<const int32_t *>(ws + lay.flags) + (back ? 1 : 0), 2, tiles, blocks, blockIdx.x / (16 * M),
                      blockIdx.x % (16 * M), back);
}

// Sums of four values over the 16 lanes of a row: in lane i that of v[i % 4]. Four lanes have the same sum, and all
// of them store it: it has to be the same to the last bit, so the quads' sums are added as (0 + 2) + (1 + 3) in each
// (halves first; quarters first would add other pairs in lanes 4 apart).
__device__ __forceinline__ float row_sum4(float v0, float v1, float v2, float v3, bool odd, bool upper) {
    const float a = (odd ? v1 : v0) + dpp_f<0xb1>(odd ? v0 : v1);       // quad_perm [1,0,3,2]
    const float b = (odd ? v3 : v2) + dpp_f<0xb1>(odd ? v2 : v3);
    float c = (upper ? b : a) + dpp_f<0x4e>(upper ? a : b);             // quad_perm [2,3,0,1]
    c += dpp_f<0x128>(c);                                               // row_ror:8
    c += dpp_f<0x124>(c);                                               // row_ror:4
    return c;
}

// 8 x 1024 x 2048 x 16 bf16 with a gate: 264 us, 76% of the busy cycles issue vector instructions (379 a token of a
// wave), two waves a SIMD at 256 registers, 21 to 23 of them spilled (88 to 96 bytes a lane). States of 17 to 64 do not
// spill; of 65 to 128 they spill 113 registers, of more 530 to 560, and there the time is the spills': all kernels of 8 x
// 1024 x 2048 with 16 | 32 | 64 | 128 | 256 states take 0.39 | 0.73 | 1.6 | 5.6 | 54 ms.
template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_kernel(const kda_ssm_args a, const kda_ssm_grads d, float *ws,
                                                                const Layout lay, int L, int tiles, int blocks) {
    using E = typename Elem<DT>::type;
    constexpr int KR = KR_OF<M>, NB = 4 / CB, NP = 16 * NB * M;
    __shared__ __align__(16) StageBwd<CB, M> stages[WAVES];
    __shared__ __align__(16) float entry[WAVES][1024 * M];       // the state before the tile
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * WAVES + wave;
    if (unit >= (int64_t)tiles * blocks) return;
    const int tile = (int)(unit / blocks), block = (int)(unit - (int64_t)tile * blocks);
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    const Place<CB, M> p(a, block);
    const int T = a.total_tokens, t0 = tile * L, t1 = T - t0 < L ? T : t0 + L;
    if (T == 0) {
        for (int q = 0; q < a.num_seqs; ++q) pass_state<CB, M>(d.d_initial_state, d.d_final_state, q, a, p);
        return;
    }
    int n = off.find(t1 - 1), start = off.at(n), end = off.at(n + 1);
    if (end == t1)          // empty sequences at the tile's end are this tile's
        for (int q = n + 1; q < a.num_seqs && off.at(q + 1) <= t1; ++q)
            pass_state<CB, M>(d.d_initial_state, d.d_final_state, q, a, p);
    f32x16 A2[M], g[M], dA[M];
    load_decay<CB, M>(a, p, A2);
    {
        const float *fg = ws + lay.grad + unit * (1024 * M), *fh = ws + lay.end_state + unit * (1024 * M);
#pragma unroll
        for (int r = 0; r < 16 * M; ++r) {
            g[r / 16][r % 16] = fg[r * 64 + p.lane];
            entry[wave][r / 4 * 256 + 4 * p.lane + r % 4] = fh[r * 64 + p.lane];
            dA[r / 16][r % 16] = 0.0f;
        }
    }
    const float bias = a.delta_bias ? a.delta_bias[p.ch] : 0.0f, skip = a.D ? a.D[p.ch] : 0.0f;
    const bool odd = p.i & 1, upper = p.i & 2;
    float real[CB];         // copies of a channel do not count in sums over channels
#pragma unroll
    for (int b = 0; b < CB; ++b) real[b] = p.channel(b) <= p.last ? 1.0f : 0.0f;
    const uint32_t ch = (uint32_t)p.ch * sizeof(E), srow = (uint32_t)(4 * p.g + (p.i & 3)) * 4;
    float dD = 0.0f, dbias = 0.0f;
    StageBwd<CB, M> &S = stages[wave];
    const int nat = CB * p.i + p.g % CB;
    char *const none = (char *)(ws + lay.none);
    RawBwd<DT, M> raw{};
    f32x16 local[M];            // the stored state before the next cell, and the steps up to it
    float lsum[CB];
    auto fetch = [&](int tb) {
        const int64_t sub = (tb - t0) / KR;
        const float *from = ws + lay.local + (unit * lay.subs + sub) * (1024 * M);
#pragma unroll
        for (int r = 0; r < 16 * M; r += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(from + r * 64 + 4 * p.lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) local[r / 16][r % 16 + j] = v[j];
        }
        const float *sums = ws + lay.sums + ((int64_t)tile * lay.subs + sub) * a.channels;
#pragma unroll
        for (int b = 0; b < CB; ++b) lsum[b] = sums[p.copied(b)];
    };
    int ge = t1;                                    // the token after the group
    {
        const int tb = t0 + (t1 - 1 - t0) / KR * KR;
        raw.template load<CB>(a, d, p, tb, t1);
        fetch(tb);
    }
    while (ge > t0) {
        const int tb = t0 + (ge - 1 - t0) / KR * KR, gs = start > tb ? start : tb;
        const bool opens = gs == start;             // the group starts its sequence
        float steps = 0.0f;
        stage<DT, CB, M>(S, raw, a, p, bias, gs - tb, ge - tb, steps);
        f32x16 h[M], ah[KR][M];
        if (opens) load_state<CB, M>(a.initial_state, n, a, p, h);
        else {
#pragma unroll
            for (int m = 0; m < M; ++m) h[m] = local[m];
            if (start < t0) {
#pragma unroll
                for (int r = 0; r < 16 * M; r += 4) {
                    const f32x4 f = *reinterpret_cast<const f32x4 *>(&entry[wave][r / 4 * 256 + 4 * p.lane]);
                    const int m = r / 16, q = r % 16;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[m][q + j] = __builtin_fmaf(exp2_f(A2[m][q + j] * lsum[(q / 4) % CB]), f[j], h[m][q + j]);
                }
            }
        }
        if (ge == end) load_state<CB, M>(d.d_final_state, n, a, p, g);
        // forward over the cell: decayed states; y for dz, dC
        float *const rows = ws + lay.rows + ((int64_t)block * T + tb) * (2 * NP);
#pragma unroll
        for (int k = 0; k < KR; ++k) {
            const bool on = tb + k >= gs && tb + k < ge;
            KDA_GLOBAL char *const row = uniform(on ? (char *)(rows + k * 2 * NP) : none);
            float sc[CB], dyc[CB], B[M], r[CB];
            read_steps<CB>(S.s[k], p.i, sc);
            read_steps<CB>(S.dy[k], p.i, dyc);
            operands<CB, M>(S.B[k], p, B);
            const float x = S.x[k][nat];
#pragma unroll
            for (int b = 0; b < CB; ++b) r[b] = 0.0f, dyc[b] *= real[b];
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int q = 0; q < 16; ++q) ah[k][m][q] = exp2_f(A2[m][q] * sc[(q / 4) % CB]) * h[m][q];
                h[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(B[m], x, ah[k][m], 0, 0, 0);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const f32x4 c4 = *reinterpret_cast<const f32x4 *>(&S.C[k][p.state(m, nb * CB, 0)]);
                    float dC[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dC[j] = 0.0f;
#pragma unroll
                        for (int b = 0; b < CB; ++b) {
                            const float hv = h[m][4 * (nb * CB + b) + j];
                            r[b] = __builtin_fmaf(c4[j], hv, r[b]);
                            dC[j] = __builtin_fmaf(dyc[b], hv, dC[j]);
                        }
                    }
                    put(row + (NP + 16 * (nb + m * NB)) * 4, srow, row_sum4(dC[0], dC[1], dC[2], dC[3], odd, upper));
                }
            }
            if (a.z) {
                const float y = __builtin_fmaf(skip, S.u[k][nat], to_natural<CB>(r));
                put(uniform(on ? (char *)d.dz + (int64_t)(tb + k) * a.channels * sizeof(E) : none), ch, (E)(S.dz[k][nat] * y));
            }
        }
        // and back; what the next cell needs is fetched half way, when registers have come free
#pragma unroll
        for (int k = KR - 1; k >= 0; --k) {
            const bool on = tb + k >= gs && tb + k < ge;
            if (k == (KR - 1) / 2) {
                __builtin_amdgcn_sched_barrier(0);
                if (gs == tb && tb > t0) {
                    fetch(tb - KR);
                    raw.template load<CB>(a, d, p, tb - KR, t1);
                }
            }
            KDA_GLOBAL char *const row = uniform(on ? (char *)(rows + k * 2 * NP) : none);
            float sc[CB], xc[CB], C[M], r1[CB], r2[CB];
            read_steps<CB>(S.s[k], p.i, sc);
            read_steps<CB>(S.x[k], p.i, xc);
            operands<CB, M>(S.C[k], p, C);
            const float dy = S.dy[k][nat];
#pragma unroll
            for (int b = 0; b < CB; ++b) r1[b] = 0.0f, r2[b] = 0.0f, xc[b] *= real[b];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                g[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(C[m], dy, g[m], 0, 0, 0);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const f32x4 b4 = *reinterpret_cast<const f32x4 *>(&S.B[k][p.state(m, nb * CB, 0)]);
                    float dB[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dB[j] = 0.0f;
#pragma unroll
                        for (int b = 0; b < CB; ++b) {
                            const int q = 4 * (nb * CB + b) + j;
                            const float dh = g[m][q];
                            r1[b] = __builtin_fmaf(b4[j], dh, r1[b]);
                            dB[j] = __builtin_fmaf(xc[b], dh, dB[j]);
                            const float v = dh * ah[k][m][q];
                            r2[b] = __builtin_fmaf(A2[m][q], v, r2[b]);
                            dA[m][q] = __builtin_fmaf(sc[b], v, dA[m][q]);
                            g[m][q] = dh * exp2_f(A2[m][q] * sc[b]);
                        }
                    }
                    put(row + 16 * (nb + m * NB) * 4, srow, row_sum4(dB[0], dB[1], dB[2], dB[3], odd, upper));
                }
            }
            const float into = to_natural<CB>(r1), dec = to_natural<CB>(r2) * LN2_F;
            const float u = S.u[k][nat], s = S.s[k][nat];
            const float ddelta = __builtin_fmaf(u, into, dec) * S.sig[k][nat];
            const int64_t o = (int64_t)(tb + k) * a.channels * sizeof(E);
            put(uniform(on ? (char *)d.du + o : none), ch, (E)__builtin_fmaf(s, into, skip * dy));
            put(uniform(on ? (char *)d.ddelta + o : none), ch, (E)ddelta);
            dD = __builtin_fmaf(dy, u, dD);
            dbias += on ? ddelta : 0.0f;
        }
        wave_fence();
        ge = gs;
        if (opens) {        // what is left belongs to the initial state
            store_state<CB, M>(d.d_initial_state, n, a, p, g);
            if (gs > t0 || gs == 0) {
                for (--n; n >= 0 && off.at(n) >= gs; --n) pass_state<CB, M>(d.d_initial_state, d.d_final_state, n, a, p);
                n = n < 0 ? 0 : n;
                start = off.at(n), end = gs;
            }
        }
    }
    float *to = ws + lay.dA + unit * (1024 * M);
#pragma unroll
    for (int r = 0; r < 16 * M; ++r) to[r * 64 + p.lane] = dA[r / 16][r % 16];
    if (p.mine) {
        float *row = ws + lay.drow + (int64_t)tile * 2 * a.channels + p.ch;
        row[0] = dD, row[a.channels] = dbias;
    }
}

// dB and dC of every (token, group, state): the sums over the group's channel blocks. 8192 tokens, 32 blocks: 34 MB in
// 7.5 us.
template <int DT>
__global__ __launch_bounds__(256) void ssm_bwd_rows_kernel(const kda_ssm_args a, const kda_ssm_grads d, const float *rows, int per_group,
                                                           int NP) {
    using E = typename Elem<DT>::type;
    const int N = a.state_size, G = a.groups;
    const int64_t line = (int64_t)a.total_tokens * 2 * NP;           // of one block
    // id: (token, which, state)
    for (int grp = blockIdx.y; grp < G; grp += gridDim.y)
        for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < line; id += (int64_t)gridDim.x * 256) {
            const int64_t t = id / (2 * NP);
            const int r = (int)(id - t * 2 * NP), n = r < NP ? r : r - NP;
            if (n >= N) continue;
            const float *from = rows + (int64_t)grp * per_group * line + id;
            float s = 0.0f;
#pragma unroll 8
            for (int b = 0; b < per_group; ++b) s += from[b * line];
            E *to = reinterpret_cast<E *>(r < NP ? d.dB : d.dC);
            to[(t * G + grp) * N + n] = (E)s;
        }
}

// dA (blockIdx.y 0 .. 16 M - 1: a register of every block's lanes), dD and dbias (the last): sums over tiles. Without
// tiles (no tokens) the offsets are checked here.
template <int CB, int M>
__global__ __launch_bounds__(256) void ssm_bwd_params_kernel(const kda_ssm_args a, const kda_ssm_grads d, const float *ws,
                                                             const Layout lay, int32_t *err, int tiles, int blocks) {
    const int r = blockIdx.y;
    if (tiles == 0 && r == 0 && blockIdx.x == 0) check_offsets(Offsets{a.cu_seqlens, a.num_seqs, a.total_tokens}, err, threadIdx.x, 256);
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (r < 16 * M) {
        const int block = (int)(id >> 6);
        if (block >= blocks) return;
        const Place<CB, M> p(a, block);
        const int c = p.channel((r % 16) / 4), n = p.state(r / 16, (r % 16) / 4, r % 4);
        const float *from = ws + lay.dA + (int64_t)block * (1024 * M) + r * 64 + p.lane;
        const int64_t step = (int64_t)blocks * 1024 * M;
        float s = 0.0f;
#pragma unroll 8
        for (int k = 0; k < tiles; ++k) s += from[k * step];
        if (c <= p.last && n < p.N) d.dA[(int64_t)c * p.N + n] = s;
    } else {
        if (id >= 2 * (int64_t)a.channels) return;
        const float *from = ws + lay.drow + id;
        float s = 0.0f;
#pragma unroll 8
        for (int k = 0; k < tiles; ++k) s += from[(int64_t)k * 2 * a.channels];
        if (id < a.channels) {
            if (d.dD) d.dD[id] = s;
        } else if (d.ddelta_bias) d.ddelta_bias[id - a.channels] = s;
    }
}

// Tokens of a tile: as many tiles as give the card 2048 waves (two to a SIMD), of 4 tokens or more. 8 x 1024 x 2048 x
// 16 with 2048 | 4096 waves: 401 | 426 us. Few channels: sqrt(0.06 T), a wave's time for a token against the join's for a tile (as
// in the forward); with 0 | 0.03 | 0.06 | 0.12 T under the root 65536 x 64 x 16 326 | 303 | 251 | 267, 32768 x 128 x 16 217 | 218 |
// 219 | 194, 16384 x 48 x 64 199 | 199 | 180 | 199, 4096 x 40 x 16 75 | 75 | 75 | 81. At least 16 | 8 | 4 tokens: 60 x 1876 x 74 168 |
// 125 | 124, 24 x 4096 x 16 55 | 44 | 40, 500 x 128 x 64 58 | 49 | 50.
int bwd_tile_len(int64_t T, int64_t blocks) {
    int64_t L = std::max<int64_t>(T * blocks / 2048, (int64_t)std::sqrt(0.06 * (double)T));
    L = L < 4 ? 4 : L > T ? T : L;
    return (int)((L + 3) / 4 * 4);
}

template <int DT, int CB, int M>
hipError_t bwd_form(const kda_ssm_args &a, const kda_ssm_grads &d, float *ws, int32_t *err, hipStream_t st) {
    const int64_t T = a.total_tokens, blocks = blocks_of(Form{CB, M}, a.channels, a.groups);
    const int L = bwd_tile_len(T, blocks);
    const int64_t tiles = T ? ceil_div(T, L) : 1;
    const Layout lay(T, a.channels, 64 / CB * M, tiles, blocks, L, M);
    const dim3 grid((unsigned)ceil_div(lay.units, WAVES));
    if (T) {
        ssm_bwd_tile_kernel<DT, CB, M><<<grid, 64 * WAVES, 0, st>>>(a, d, ws, lay, err, L, (int)tiles, (int)blocks);
        if (hipError_t e = hipGetLastError()) return e;
    }
    // One tile has no neighbours to join; more than one there are for less than 2048 blocks only, so that the
    // threads of a launch stay under 2^32 whatever the number of groups.
    if (tiles > 1) {
        ssm_bwd_join_kernel<CB, M><<<dim3((unsigned)(blocks * 16 * M), 2), 256, 0, st>>>(a, ws, lay, (int)tiles, (int)blocks);
        if (hipError_t e = hipGetLastError()) return e;
    }
    ssm_bwd_kernel<DT, CB, M><<<grid, 64 * WAVES, 0, st>>>(a, d, ws, lay, L, (int)tiles, (int)blocks);
    if (hipError_t e = hipGetLastError()) return e;
    if (T) {
        const int64_t line = T * 2 * (64 / CB * M);
        ssm_bwd_rows_kernel<DT><<<dim3((unsigned)std::min<int64_t>(1 << 20, ceil_div(line, 256)), (unsigned)std::min(65535, a.groups)), 256, 0, st>>>(
            a, d, ws + lay.rows, (int)(blocks / a.groups), 64 / CB * M);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const int64_t wide = std::max<int64_t>(blocks * 64, 2 * (int64_t)a.channels);
    ssm_bwd_params_kernel<CB, M><<<dim3((unsigned)ceil_div(wide, 256), 16 * M + 1), 256, 0, st>>>(a, d, ws, lay, err,
                                                                                                  T ? (int)tiles : 0, (int)blocks);
    return hipGetLastError();
}

template <int DT> hipError_t bwd_dt(const kda_ssm_args &a, const kda_ssm_grads &d, float *ws, int32_t *err, hipStream_t st) {
    const Form f = form_of(a.state_size);
    if (f.cb == 4) return bwd_form<DT, 4, 1>(a, d, ws, err, st);
    if (f.cb == 2) return bwd_form<DT, 2, 1>(a, d, ws, err, st);
    if (f.m == 1) return bwd_form<DT, 1, 1>(a, d, ws, err, st);
    if (f.m == 2) return bwd_form<DT, 1, 2>(a, d, ws, err, st);
    return bwd_form<DT, 1, 4>(a, d, ws, err, st);
}

}  // namespace
}  // namespace ssm

size_t ssm_bwd_workspace(int64_t T, int64_t D, int64_t N, int64_t G) {
    using namespace ssm;
    const Form f = form_of((int)N);
    const int64_t blocks = blocks_of(f, D, G);
    const int L = bwd_tile_len(T, blocks);
    return (size_t)Layout(T, D, 64 / f.cb * f.m, T ? ceil_div(T, L) : 1, blocks, L, f.m).total * sizeof(float);
}

hipError_t launch_ssm_bwd(const kda_ssm_args &a, const kda_ssm_grads &d, float *ws, int32_t *err, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return ssm::bwd_dt<KDA_DTYPE_F32>(a, d, ws, err, st);
    if (a.dtype == KDA_DTYPE_BF16) return ssm::bwd_dt<KDA_DTYPE_BF16>(a, d, ws, err, st);
    return ssm::bwd_dt<KDA_DTYPE_F16>(a, d, ws, err, st);
}

}  // namespace ops
}  // namespace kda
