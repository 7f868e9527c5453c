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
//   3. ssm_bwd_kernel: each tile from its end, KR tokens at a time: their decays and decayed states
//      again from the stored state (completed by e^{A S} times the tile's first state), kept in
//      registers, then the gradients
//   4. ssm_bwd_rows_kernel, ssm_bwd_params_kernel: the sums over channel blocks (dB, dC) and over
//      tiles (dA, dD, dbias), in a fixed order.
#include <algorithm>

#include "ops_ssm.hpp"

namespace kda {
namespace ops {
namespace ssm {
namespace {

constexpr int KB = 4;                       // tokens staged at a time
template <int M> constexpr int KR_OF = 4 / M;   // tokens whose decays and states are held: 128 registers

// Where the workspace keeps what, in floats.
struct Layout {
    int64_t units, subs;                    // (tile, block) pairs; stored states of a tile
    int64_t end_state, grad, local, sums, first_sums, dA, drow, rows, flags, total;
    Layout(int64_t T, int64_t D, int64_t N, int64_t tiles, int64_t blocks, int L, int M) {
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
        rows = drow + 2 * tiles * D;                 // [block][T][2][N]: dB, dC
        flags = rows + blocks * T * 2 * N;           // [tile][2]
        total = flags + 2 * tiles;
    }
};

template <int DT, int M> struct RawBwd {
    using E = typename Elem<DT>::type;
    E delta[KB], u[KB], z[KB], dy[KB], B[KB][M], C[KB][M];
    template <int CB>
    __device__ __forceinline__ void load(const kda_ssm_args &a, const kda_ssm_grads &d, const Place<CB, M> &p, int t, int stop) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int64_t r = t + k < stop ? t + k : stop - 1;
            delta[k] = reinterpret_cast<const E *>(a.delta)[r * a.delta_stride + p.ch];
            u[k] = reinterpret_cast<const E *>(a.u)[r * a.u_stride + p.ch];
            dy[k] = reinterpret_cast<const E *>(d.dy)[r * d.dy_stride + p.ch];
            if (a.z) z[k] = reinterpret_cast<const E *>(a.z)[r * a.z_stride + p.ch];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int n = p.nat_state(m);
                const int64_t at = (int64_t)p.group * p.N + n;
                B[k][m] = n < p.N ? reinterpret_cast<const E *>(a.B)[r * a.B_stride + at] : (E)0.0f;
                C[k][m] = n < p.N ? reinterpret_cast<const E *>(a.C)[r * a.C_stride + at] : (E)0.0f;
            }
        }
    }
};

// Staged tokens of a wave in LDS: per channel (natural lane l at CB i + g % CB) and per state.
template <int CB, int M> struct StageBwd {
    static constexpr int CH = 16 * CB, NS = 64 / CB * M;
    float s[KB][CH], x[KB][CH], dy[KB][CH];       // step, step times input, dy'
    float u[KB][CH], sig[KB][CH], dz[KB][CH];     // input, sigmoid(delta + bias), dy silu'(z)
    float B[KB][NS], C[KB][NS];
};

template <int DT, int CB, int M>
__device__ __forceinline__ void stage(StageBwd<CB, M> &S, const RawBwd<DT, M> &raw, const kda_ssm_args &a, const Place<CB, M> &p,
                                      float bias, int count, float (&step)[KB]) {
    const int at = CB * p.i + p.g % CB;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
        const bool on = k < count, in = on && !p.dup;
        const float d = (float)raw.delta[k] + bias, u = (float)raw.u[k], dy = (float)raw.dy[k];
        float s = d, sig = 1.0f, g = dy, dz = 0.0f;
        if (a.delta_softplus) s = softplus_f(d), sig = sigmoid_f(d);
        if (a.z) {
            const float z = (float)raw.z[k], sz = sigmoid_f(z);
            g = dy * z * sz;
            dz = dy * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f);
        }
        // past the tile's end no step, nothing in, nothing out; a channel past the group's last, which
        // repeats it, adds nothing to the sums over channels
        s = on ? s : 0.0f;
        step[k] = s;
        S.s[k][at] = s, S.x[k][at] = in ? s * u : 0.0f, S.dy[k][at] = in ? g : 0.0f;
        S.u[k][at] = u, S.sig[k][at] = sig, S.dz[k][at] = dz;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            S.B[k][p.nat_state(m)] = on ? (float)raw.B[k][m] : 0.0f;
            S.C[k][p.nat_state(m)] = on ? (float)raw.C[k][m] : 0.0f;
        }
    }
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

template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_tile_kernel(const kda_ssm_args a, const kda_ssm_grads d, float *ws,
                                                                     const Layout lay, int32_t *err, int L, int tiles, int blocks) {
    constexpr int KR = KR_OF<M>;
    __shared__ __align__(16) StageBwd<CB, M> stages[WAVES];
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
    float sum = 0.0f;
    StageBwd<CB, M> &S = stages[wave];
    RawBwd<DT, M> raw;
    raw.template load<CB>(a, d, p, t0, t1);
    for (int t = t0; t < t1; t += KB) {
        float step[KB];
        stage<DT, CB, M>(S, raw, a, p, bias, t1 - t, step);
        wave_fence();
        if (t + KB < t1) raw.template load<CB>(a, d, p, t + KB, t1);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            if (t + k == end && t + k < t1) {           // the next sequence starts with this token
                if (first) add_state<CB, M>(G, P, d.d_final_state, n, a, p);
                first = false, reset = true;
                for (++n; n < a.num_seqs - 1 && off.at(n + 1) <= t + k; ++n) {}
                end = off.at(n + 1);
                load_state<CB, M>(a.initial_state, n, a, p, h);
            }
            if (k % KR == 0) {                          // the state before this token, and the steps so far
                const int64_t sub = (t - t0 + k) / KR;
                float *to = ws + lay.local + (unit * lay.subs + sub) * (1024 * M);
#pragma unroll
                for (int r = 0; r < 16 * M; ++r) to[r * 64 + p.lane] = h[r / 16][r % 16];
                if (p.mine) ws[lay.sums + ((int64_t)tile * lay.subs + sub) * a.channels + p.ch] = sum;
            }
            sum += step[k];
            float sc[CB], B[M], C[M];
            read_steps<CB>(S.s[k], p.i, sc);
            operands<CB, M>(S.B[k], p, B);
            operands<CB, M>(S.C[k], p, C);
            const int nat = CB * p.i + p.g % CB;
            const float x = S.x[k][nat], dy = S.dy[k][nat];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                f32x16 e;
#pragma unroll
                for (int r = 0; r < 16; ++r) e[r] = exp2_f(A2[m][r] * sc[(r / 4) % CB]);
#pragma unroll
                for (int r = 0; r < 16; ++r) h[m][r] *= e[r];
                h[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(B[m], x, h[m], 0, 0, 0);
                if (first) {
                    const f32x16 w = __builtin_amdgcn_mfma_f32_16x16x1f32(C[m], dy, zero[m], 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        P[m][r] *= e[r];
                        G[m][r] = __builtin_fmaf(P[m][r], w[r], G[m][r]);
                    }
                }
            }
        }
        wave_fence();
    }
    const bool ends = end == t1;            // the last token's sequence
    if (first && ends) add_state<CB, M>(G, P, d.d_final_state, n, a, p);
    float *to = ws + lay.end_state + unit * (1024 * M), *tg = ws + lay.grad + unit * (1024 * M);
#pragma unroll
    for (int r = 0; r < 16 * M; ++r) {
        to[r * 64 + p.lane] = h[r / 16][r % 16];
        tg[r * 64 + p.lane] = G[r / 16][r % 16];
    }
    if (p.mine) ws[lay.first_sums + (int64_t)tile * a.channels + p.ch] = sum;
    if (block == 0 && p.lane == 0) {
        int32_t *f = reinterpret_cast<int32_t *>(ws + lay.flags) + 2 * tile;
        f[0] = reset;                       // a sequence starts in the tile: its end state stands alone
        f[1] = !first || ends;              // one ends in it: nothing of what lies behind reaches back
    }
}

// blockIdx.y 0: the state before every tile, in its end state's place; 1: the gradient that comes to
// every tile's end from the tiles behind it, in G's place.
template <int CB, int M>
__global__ __launch_bounds__(256) void ssm_bwd_join_kernel(const kda_ssm_args a, float *ws, const Layout lay, int tiles, int blocks) {
    constexpr int AHEAD = 8;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int unit = blockIdx.x * 4 + wave;
    if (unit >= blocks * 16 * M) return;
    const int block = unit / (16 * M), r = unit - block * (16 * M);
    const Place<CB, M> p(a, block);
    const int m = r / 16, b = (r % 16) / 4, j = r % 4;
    const int c = p.channel(b), n = p.state(m, b, j);
    const int cc = c <= p.last ? c : p.last;
    const float A2 = c <= p.last && n < p.N ? a.A[(int64_t)c * p.N + n] * LOG2E_F : 0.0f;
    const bool back = blockIdx.y == 1;
    const int64_t step = (int64_t)blocks * 1024 * M;
    float *at = ws + (back ? lay.grad : lay.end_state) + (int64_t)block * (1024 * M) + r * 64 + p.lane;
    const float *sums = ws + lay.first_sums;
    const int32_t *flags = reinterpret_cast<const int32_t *>(ws + lay.flags) + (back ? 1 : 0);
    float h = 0.0f;
    for (int k0 = 0; k0 < tiles; k0 += AHEAD) {
        float E[AHEAD], S[AHEAD];
        int alone[AHEAD];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const int f = k0 + q < tiles ? k0 + q : tiles - 1, k = back ? tiles - 1 - f : f;
            E[q] = at[k * step];
            S[q] = sums[(int64_t)k * a.channels + cc];
            alone[q] = flags[2 * k];
        }
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            if (k0 + q < tiles) {
                const int k = back ? tiles - 1 - (k0 + q) : k0 + q;
                at[k * step] = h;
                h = alone[q] ? E[q] : __builtin_fmaf(exp2_f(A2 * S[q]), h, E[q]);
            }
        }
    }
}

template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_kernel(const kda_ssm_args a, const kda_ssm_grads d, float *ws,
                                                                const Layout lay, int L, int tiles, int blocks) {
    using E = typename Elem<DT>::type;
    constexpr int KR = KR_OF<M>, NB = 4 / CB;
    __shared__ __align__(16) StageBwd<CB, M> stages[WAVES];
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
    f32x16 A2[M], g[M], dA[M], first[M];
    load_decay<CB, M>(a, p, A2);
    {
        const float *fg = ws + lay.grad + unit * (1024 * M), *fh = ws + lay.end_state + unit * (1024 * M);
#pragma unroll
        for (int r = 0; r < 16 * M; ++r) {
            g[r / 16][r % 16] = fg[r * 64 + p.lane];
            first[r / 16][r % 16] = fh[r * 64 + p.lane];
            dA[r / 16][r % 16] = 0.0f;
        }
    }
    const float bias = a.delta_bias ? a.delta_bias[p.ch] : 0.0f, skip = a.D ? a.D[p.ch] : 0.0f;
    float dD = 0.0f, dbias = 0.0f;
    StageBwd<CB, M> &S = stages[wave];
    const int nat = CB * p.i + p.g % CB;
    RawBwd<DT, M> raw;
    int t = t0 + (t1 - t0 - 1) / KB * KB;
    raw.template load<CB>(a, d, p, t, t1);
    for (; t >= t0; t -= KB) {
        float step[KB];
        const int count = t1 - t < KB ? t1 - t : KB;
        stage<DT, CB, M>(S, raw, a, p, bias, count, step);
        wave_fence();
        if (t > t0) raw.template load<CB>(a, d, p, t - KB, t1);
#pragma unroll 1
        for (int ks = KB - KR; ks >= 0; ks -= KR) {
            const int tb = t + ks;
            if (tb >= t1) continue;
            // the state before token tb
            const bool mixed = start > tb || end < (tb + KR < t1 ? tb + KR : t1);   // sequences meet among these tokens
            int fn = n, fstart = start, fend = end;
            if (start > tb) fn = off.find(tb), fstart = off.at(fn), fend = off.at(fn + 1);
            f32x16 h[M], e[KR][M], ah[KR][M];
            if (fstart == tb) load_state<CB, M>(a.initial_state, fn, a, p, h);
            else {
                const int64_t sub = (tb - t0) / KR;
                const float *from = ws + lay.local + (unit * lay.subs + sub) * (1024 * M);
#pragma unroll
                for (int r = 0; r < 16 * M; ++r) h[r / 16][r % 16] = from[r * 64 + p.lane];
                if (fstart < t0) {
                    const float *sums = ws + lay.sums + ((int64_t)tile * lay.subs + sub) * a.channels;
                    float sc[CB];
#pragma unroll
                    for (int b = 0; b < CB; ++b) sc[b] = sums[p.channel(b) <= p.last ? p.channel(b) : p.last];
#pragma unroll
                    for (int m = 0; m < M; ++m)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            h[m][r] = __builtin_fmaf(exp2_f(A2[m][r] * sc[(r / 4) % CB]), first[m][r], h[m][r]);
                }
            }
            // forward over these tokens: decays, decayed states; y for dz, dC
#pragma unroll
            for (int k = 0; k < KR; ++k) {
                const int kk = ks + k;
                if (mixed && k > 0 && tb + k == fend && tb + k < t1) {
                    for (++fn; fn < a.num_seqs - 1 && off.at(fn + 1) <= tb + k; ++fn) {}
                    fend = off.at(fn + 1);
                    load_state<CB, M>(a.initial_state, fn, a, p, h);
                }
                float sc[CB], dyc[CB], B[M], r[CB];
                read_steps<CB>(S.s[kk], p.i, sc);
                read_steps<CB>(S.dy[kk], p.i, dyc);
                operands<CB, M>(S.B[kk], p, B);
                const float x = S.x[kk][nat];
#pragma unroll
                for (int b = 0; b < CB; ++b) r[b] = 0.0f;
                float *rows = ws + lay.rows + (((int64_t)block * T + tb + k) * 2 + 1) * p.N;
#pragma unroll
                for (int m = 0; m < M; ++m) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) e[k][m][q] = exp2_f(A2[m][q] * sc[(q / 4) % CB]);
#pragma unroll
                    for (int q = 0; q < 16; ++q) ah[k][m][q] = e[k][m][q] * h[m][q];
                    h[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(B[m], x, ah[k][m], 0, 0, 0);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const f32x4 c4 = *reinterpret_cast<const f32x4 *>(&S.C[kk][p.state(m, nb * CB, 0)]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float dC = 0.0f;
#pragma unroll
                            for (int b = 0; b < CB; ++b) {
                                const float hv = h[m][4 * (nb * CB + b) + j];
                                r[b] = __builtin_fmaf(c4[j], hv, r[b]);
                                dC = __builtin_fmaf(dyc[b], hv, dC);
                            }
                            dC = row_sum(dC);
                            const int st = p.state(m, nb * CB, j);
                            if (p.i == j && st < p.N && tb + k < t1) rows[st] = dC;
                        }
                    }
                }
                if (a.z && tb + k < t1) {
                    const float y = __builtin_fmaf(skip, S.u[kk][nat], to_natural<CB>(r));
                    if (p.mine) reinterpret_cast<E *>(d.dz)[(int64_t)(tb + k) * a.channels + p.ch] = (E)(S.dz[kk][nat] * y);
                }
            }
            // and back
#pragma unroll
            for (int k = KR - 1; k >= 0; --k) {
                const int kk = ks + k, tk = tb + k;
                if (tk >= t1) continue;
                if (tk + 1 == end) load_state<CB, M>(d.d_final_state, n, a, p, g);
                float sc[CB], xc[CB], C[M], r1[CB], r2[CB];
                read_steps<CB>(S.s[kk], p.i, sc);
                read_steps<CB>(S.x[kk], p.i, xc);
                operands<CB, M>(S.C[kk], p, C);
                const float dy = S.dy[kk][nat];
#pragma unroll
                for (int b = 0; b < CB; ++b) r1[b] = 0.0f, r2[b] = 0.0f;
                float *rows = ws + lay.rows + ((int64_t)block * T + tk) * 2 * p.N;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    g[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(C[m], dy, g[m], 0, 0, 0);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const f32x4 b4 = *reinterpret_cast<const f32x4 *>(&S.B[kk][p.state(m, nb * CB, 0)]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float dB = 0.0f;
#pragma unroll
                            for (int b = 0; b < CB; ++b) {
                                const int q = 4 * (nb * CB + b) + j;
                                const float dh = g[m][q];
                                r1[b] = __builtin_fmaf(b4[j], dh, r1[b]);
                                dB = __builtin_fmaf(xc[b], dh, dB);
                                const float v = dh * ah[k][m][q];
                                r2[b] = __builtin_fmaf(A2[m][q], v, r2[b]);
                                dA[m][q] = __builtin_fmaf(sc[b], v, dA[m][q]);
                                g[m][q] = dh * e[k][m][q];
                            }
                            dB = row_sum(dB);
                            const int st = p.state(m, nb * CB, j);
                            if (p.i == j && st < p.N) rows[st] = dB;
                        }
                    }
                }
                const float into = to_natural<CB>(r1), dec = to_natural<CB>(r2) * LN2_F;
                const float u = S.u[kk][nat], s = S.s[kk][nat];
                const float ddelta = __builtin_fmaf(u, into, dec) * S.sig[kk][nat];
                if (p.mine) {
                    const int64_t o = (int64_t)tk * a.channels + p.ch;
                    reinterpret_cast<E *>(d.du)[o] = (E)__builtin_fmaf(s, into, skip * dy);
                    reinterpret_cast<E *>(d.ddelta)[o] = (E)ddelta;
                }
                dD = __builtin_fmaf(dy, u, dD);
                dbias += ddelta;
                if (tk == start) {      // a sequence's first token: what is left belongs to its initial state
                    store_state<CB, M>(d.d_initial_state, n, a, p, g);
                    if (tk > t0 || tk == 0) {
                        for (--n; n >= 0 && off.at(n) >= tk; --n)
                            pass_state<CB, M>(d.d_initial_state, d.d_final_state, n, a, p);
                        n = n < 0 ? 0 : n;
                        start = off.at(n), end = tk;
                    }
                }
            }
        }
        wave_fence();
    }
    float *to = ws + lay.dA + unit * (1024 * M);
#pragma unroll
    for (int r = 0; r < 16 * M; ++r) to[r * 64 + p.lane] = dA[r / 16][r % 16];
    if (p.mine) {
        float *row = ws + lay.drow + (int64_t)tile * 2 * a.channels + p.ch;
        row[0] = dD, row[a.channels] = dbias;
    }
}

// dB and dC of every (token, group, state): the sums over the group's channel blocks.
template <int DT>
__global__ __launch_bounds__(256) void ssm_bwd_rows_kernel(const kda_ssm_args a, const kda_ssm_grads d, const float *rows, int per_group) {
    using E = typename Elem<DT>::type;
    const int N = a.state_size, G = a.groups;
    const int64_t line = (int64_t)a.total_tokens * 2 * N;            // of one block
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;      // (token, which, state)
    const int grp = blockIdx.y;
    if (id >= line) return;
    const float *from = rows + (int64_t)grp * per_group * line + id;
    float s = 0.0f;
#pragma unroll 8
    for (int b = 0; b < per_group; ++b) s += from[b * line];
    const int64_t t = id / (2 * N);
    const int r = (int)(id - t * 2 * N);
    E *to = reinterpret_cast<E *>(r < N ? d.dB : d.dC);
    to[(t * G + grp) * N + (r < N ? r : r - N)] = (E)s;
}

// dA (blockIdx.y 0 .. 16 M - 1: a register of every block's lanes), dD and dbias (the last): sums over tiles.
template <int CB, int M>
__global__ __launch_bounds__(256) void ssm_bwd_params_kernel(const kda_ssm_args a, const kda_ssm_grads d, const float *ws,
                                                             const Layout lay, int tiles, int blocks) {
    const int r = blockIdx.y;
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

// Tokens of a tile: as many tiles as give the card 2048 waves (two to a SIMD), of 16 tokens or more.
int bwd_tile_len(int64_t T, int64_t blocks) {
    int64_t L = T * blocks / 2048;
    L = L < 16 ? 16 : L > T ? T : L;
    return (int)((L + KB - 1) / KB * KB);
}

template <int DT, int CB, int M>
hipError_t bwd_form(const kda_ssm_args &a, const kda_ssm_grads &d, float *ws, int32_t *err, hipStream_t st) {
    const int64_t T = a.total_tokens, blocks = blocks_of(Form{CB, M}, a.channels, a.groups);
    const int L = bwd_tile_len(T, blocks);
    const int64_t tiles = T ? ceil_div(T, L) : 1;
    const Layout lay(T, a.channels, a.state_size, tiles, blocks, L, M);
    const dim3 grid((unsigned)ceil_div(lay.units, WAVES));
    if (T) {
        ssm_bwd_tile_kernel<DT, CB, M><<<grid, 64 * WAVES, 0, st>>>(a, d, ws, lay, err, L, (int)tiles, (int)blocks);
        if (hipError_t e = hipGetLastError()) return e;
        ssm_bwd_join_kernel<CB, M><<<dim3((unsigned)ceil_div(blocks * 16 * M, 4), 2), 256, 0, st>>>(a, ws, lay, (int)tiles, (int)blocks);
        if (hipError_t e = hipGetLastError()) return e;
    }
    ssm_bwd_kernel<DT, CB, M><<<grid, 64 * WAVES, 0, st>>>(a, d, ws, lay, L, (int)tiles, (int)blocks);
    if (hipError_t e = hipGetLastError()) return e;
    if (T) {
        const int64_t line = T * 2 * a.state_size;
        ssm_bwd_rows_kernel<DT><<<dim3((unsigned)ceil_div(line, 256), (unsigned)a.groups), 256, 0, st>>>(
            a, d, ws + lay.rows, (int)(blocks / a.groups));
        if (hipError_t e = hipGetLastError()) return e;
    }
    const int64_t wide = std::max<int64_t>(blocks * 64, 2 * (int64_t)a.channels);
    ssm_bwd_params_kernel<CB, M><<<dim3((unsigned)ceil_div(wide, 256), 16 * M + 1), 256, 0, st>>>(a, d, ws, lay, T ? (int)tiles : 0,
                                                                                                  (int)blocks);
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
    return (size_t)Layout(T, D, N, T ? ceil_div(T, L) : 1, blocks, L, f.m).total * sizeof(float);
}

hipError_t launch_ssm_bwd(const kda_ssm_args &a, const kda_ssm_grads &d, float *ws, int32_t *err, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return ssm::bwd_dt<KDA_DTYPE_F32>(a, d, ws, err, st);
    if (a.dtype == KDA_DTYPE_BF16) return ssm::bwd_dt<KDA_DTYPE_BF16>(a, d, ws, err, st);
    return ssm::bwd_dt<KDA_DTYPE_F16>(a, d, ws, err, st);
}

}  // namespace ops
}  // namespace kda
