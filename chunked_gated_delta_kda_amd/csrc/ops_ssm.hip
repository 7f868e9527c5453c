// ops_ssm.hip -- the selective state space scan: prompts (over a packed batch) and one token of
// each sequence. The mathematics and the register layout are in ops_ssm.hpp.
//
// Prompts. The time axis is cut into tiles of consecutive packed tokens, whatever sequences start
// or end in them, so that few channels still fill the card:
//   1. ssm_tile_kernel: each tile from a zero state: its end state E and the sum S of its
//      step sizes, so that the tile maps a state h to e^{A S} h + E (to E alone where a sequence
//      starts in it);
//   2. ssm_join_kernel: those maps one after another per (channel, state): the state each tile
//      starts from, in E's place;
//   3. ssm_scan_kernel: the scan itself, from that state.
// One tile needs the last step only. Bound by vector issue: a (token, channel, state) costs two
// multiplications, an exponential and the product with C, and steps 1 and 3 both pay the first
// three.
#include "ops_ssm.hpp"

namespace kda {
namespace ops {
namespace ssm {
namespace {

// K tokens' activations of a wave, one element a lane, in flight while the tokens before are
// computed.
template <int DT, int CB, int M, bool OUT> struct Raw {
    using E = typename Elem<DT>::type;
    E delta[K], u[K], z[K], B[K][M], C[K][M];
    __device__ __forceinline__ void load(const kda_ssm_args &a, const Place<CB, M> &p, int t, int stop) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t r = t + k < stop ? t + k : stop - 1;   // past the end: the last row again
            delta[k] = reinterpret_cast<const E *>(a.delta)[r * a.delta_stride + p.ch];
            u[k] = reinterpret_cast<const E *>(a.u)[r * a.u_stride + p.ch];
            if (OUT && a.z) z[k] = reinterpret_cast<const E *>(a.z)[r * a.z_stride + p.ch];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int n = p.nat_state(m);
                const int64_t at = (int64_t)p.group * p.N + n;
                B[k][m] = n < p.N ? reinterpret_cast<const E *>(a.B)[r * a.B_stride + at] : (E)0.0f;
                if (OUT) C[k][m] = n < p.N ? reinterpret_cast<const E *>(a.C)[r * a.C_stride + at] : (E)0.0f;
            }
        }
    }
};

// h <- e^{s A} h + (s u) (x) B for one token
template <int CB, int M>
__device__ __forceinline__ void advance(f32x16 (&h)[M], const f32x16 (&A2)[M], const float (&s)[CB], float x, const float *B) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) h[m][4 * b + j] *= exp2_f(A2[m][4 * b + j] * s[b % CB]);
        h[m] = __builtin_amdgcn_mfma_f32_16x16x1f32(B[m], x, h[m], 0, 0, 0);
    }
}

template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES) void ssm_tile_kernel(const kda_ssm_args a, float *ws, float *sums, int32_t *resets,
                                                              int32_t *err, int L, int tiles, int blocks) {
    __shared__ __align__(16) float lds[WAVES][K * 16 * CB];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * WAVES + wave;
    if (unit >= (int64_t)tiles * blocks) return;
    const int tile = (int)(unit / blocks), block = (int)(unit - (int64_t)tile * blocks);
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    if (unit == 0) check_offsets(off, err, threadIdx.x & 63, 64);
    const Place<CB, M> p(a, block);
    const int T = a.total_tokens, t0 = tile * L, t1 = T - t0 < L ? T : t0 + L;
    // the sequence of the tile's last token: where it starts in the tile, what came before it is
    // of no account; where it ends with the tile, nobody asks for the end state
    const int n = off.find(t1 - 1), start = off.at(n);
    const bool reset = start >= t0;
    if (block == 0 && p.lane == 0) resets[tile] = reset;
    if (off.at(n + 1) == t1) return;
    f32x16 A2[M], h[M];
    load_decay<CB, M>(a, p, A2);
    load_state<CB, M>(reset ? a.initial_state : nullptr, n, a, p, h);
    const float bias = a.delta_bias ? a.delta_bias[p.ch] : 0.0f;
    float sum = 0.0f;
    float *steps = lds[wave];
    int t = reset ? start : t0;
    Raw<DT, CB, M, false> raw;
    raw.load(a, p, t, t1);
    while (t < t1) {
        float s[K], x[K], B[K][M];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float d = (float)raw.delta[k] + bias;
            s[k] = a.delta_softplus ? softplus_f(d) : d;
            x[k] = s[k] * (float)raw.u[k];
            const bool step = t + k < t1;
            if (step) sum += s[k];
            else s[k] = 0.0f, x[k] = 0.0f;      // no step: e^0 h + 0 (B too: what is repeated may be infinite)
            steps[k * 16 * CB + CB * p.i + p.g % CB] = s[k];
#pragma unroll
            for (int m = 0; m < M; ++m) B[k][m] = step ? (float)raw.B[k][m] : 0.0f;
        }
        wave_fence();
        t += K;
        if (t < t1) raw.load(a, p, t, t1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float sc[CB];
            read_steps<CB>(steps + k * 16 * CB, p.i, sc);
            advance<CB, M>(h, A2, sc, x[k], B[k]);
        }
        wave_fence();
    }
    float *to = tile_state<M>(ws, tile, blocks, block);
#pragma unroll
    for (int r = 0; r < 16 * M; ++r) to[r * 64 + p.lane] = h[r / 16][r % 16];
    if (p.mine) sums[(int64_t)tile * a.channels + p.ch] = sum;
}

// The state every tile starts from: h <- e^{A S} h + E per (channel, state), tile after tile; loads
// of AHEAD tiles are in flight together.
template <int CB, int M>
__global__ __launch_bounds__(256) void ssm_join_kernel(const kda_ssm_args a, float *ws, const float *sums,
                                                       const int32_t *resets, int tiles, int blocks) {
    constexpr int AHEAD = 8;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int unit = blockIdx.x * 4 + wave;                 // (block, register)
    if (unit >= blocks * 16 * M) return;
    const int block = unit / (16 * M), r = unit - block * (16 * M);
    const Place<CB, M> p(a, block);
    const int m = r / 16, b = (r % 16) / 4, j = r % 4;
    const int c = p.channel(b), n = p.state(m, b, j);
    const bool in = c <= p.last && n < p.N;
    const int cc = c <= p.last ? c : p.last;
    const float A2 = in ? a.A[(int64_t)c * p.N + n] * LOG2E_F : 0.0f;
    const int64_t step = (int64_t)blocks * 1024 * M;
    float *at = tile_state<M>(ws, 0, blocks, block) + r * 64 + p.lane;
    float h = 0.0f;
    for (int k0 = 0; k0 < tiles; k0 += AHEAD) {
        float E[AHEAD], S[AHEAD];
        int reset[AHEAD];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const int k = k0 + q < tiles ? k0 + q : tiles - 1;
            E[q] = at[k * step];
            S[q] = sums[(int64_t)k * a.channels + cc];
            reset[q] = resets[k];
        }
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            if (k0 + q < tiles) {
                at[(k0 + q) * step] = h;
                h = reset[q] ? E[q] : __builtin_fmaf(exp2_f(A2 * S[q]), h, E[q]);
            }
        }
    }
}

template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES) void ssm_scan_kernel(const kda_ssm_args a, const float *ws, int32_t *err, int L,
                                                              int tiles, int blocks) {
    using E = typename Elem<DT>::type;
    constexpr int NS = 64 / CB * M;            // states of a staged C row
    __shared__ __align__(16) float lds[WAVES][K * (16 * CB + NS)];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * WAVES + wave;
    if (unit >= (int64_t)tiles * blocks) return;
    const int tile = (int)(unit / blocks), block = (int)(unit - (int64_t)tile * blocks);
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    if (tiles == 1 && unit == 0) check_offsets(off, err, threadIdx.x & 63, 64);
    const Place<CB, M> p(a, block);
    const int T = a.total_tokens, t0 = tile * L, t1 = T - t0 < L ? T : t0 + L;
    if (T == 0) {
        for (int q = 0; q < a.num_seqs; ++q) pass_state<CB, M>(a.final_state, a.initial_state, q, a, p);
        return;
    }
    int n = off.find(t0), start = off.at(n), end = off.at(n + 1);
    if (tile == 0)
        for (int q = 0; q < n; ++q) pass_state<CB, M>(a.final_state, a.initial_state, q, a, p);
    f32x16 A2[M], h[M];
    load_decay<CB, M>(a, p, A2);
    if (start < t0) {
        const float *from = tile_state<M>(const_cast<float *>(ws), tile, blocks, block);
#pragma unroll
        for (int r = 0; r < 16 * M; ++r) h[r / 16][r % 16] = from[r * 64 + p.lane];
    } else load_state<CB, M>(a.initial_state, n, a, p, h);
    const float bias = a.delta_bias ? a.delta_bias[p.ch] : 0.0f, skip = a.D ? a.D[p.ch] : 0.0f;
    float *steps = lds[wave], *rows = lds[wave] + K * 16 * CB;
    int t = t0;
    Raw<DT, CB, M, true> raw;
    raw.load(a, p, t, t1);
    while (true) {
        // one sequence's tokens of this tile, or what of them fits a stage
        const int stop = end < t1 ? end : t1;
        float s[K], x[K], u[K], z[K], B[K][M], y[K];
        const int count = stop - t < K ? stop - t : K;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float d = (float)raw.delta[k] + bias;
            s[k] = a.delta_softplus ? softplus_f(d) : d;
            u[k] = (float)raw.u[k];
            x[k] = s[k] * u[k];
            if (k >= count) s[k] = 0.0f, x[k] = 0.0f;
            z[k] = a.z ? (float)raw.z[k] : 0.0f;
            steps[k * 16 * CB + CB * p.i + p.g % CB] = s[k];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                B[k][m] = k < count ? (float)raw.B[k][m] : 0.0f;   // the next sequence's rows stay out of this state
                rows[k * NS + p.nat_state(m)] = (float)raw.C[k][m];
            }
        }
        wave_fence();
        const int from = t;
        t += count;
        if (t < t1) raw.load(a, p, t, t1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float sc[CB], r[CB];
            read_steps<CB>(steps + k * 16 * CB, p.i, sc);
            advance<CB, M>(h, A2, sc, x[k], B[k]);
#pragma unroll
            for (int b = 0; b < CB; ++b) r[b] = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int nb = 0; nb < 4 / CB; ++nb) {
                    const f32x4 c4 = *reinterpret_cast<const f32x4 *>(rows + k * NS + p.state(m, nb * CB, 0));
#pragma unroll
                    for (int b = 0; b < CB; ++b)
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[b] = __builtin_fmaf(c4[j], h[m][4 * (nb * CB + b) + j], r[b]);
                }
            y[k] = to_natural<CB>(r);
        }
        wave_fence();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float v = __builtin_fmaf(skip, u[k], y[k]);
            if (a.z) v *= z[k] * sigmoid_f(z[k]);
            if (k < count && p.mine) reinterpret_cast<E *>(a.out)[(int64_t)(from + k) * a.channels + p.ch] = (E)v;
        }
        if (t < end) {
            if (t < t1) continue;
            break;
        }
        store_state<CB, M>(a.final_state, n, a, p, h);
        for (++n; n < a.num_seqs && off.at(n + 1) <= t; ++n) pass_state<CB, M>(a.final_state, a.initial_state, n, a, p);
        if (t >= t1 || n >= a.num_seqs) break;
        end = off.at(n + 1);
        load_state<CB, M>(a.initial_state, n, a, p, h);
    }
}

// One token of each sequence: four states a lane, NL lanes a channel. Every state is read and
// written once, by one lane, so it may be updated in place.
template <int DT, int NL, bool ALIGNED>
__global__ __launch_bounds__(256) void ssm_decode_kernel(const kda_ssm_args a) {
    using E = typename Elem<DT>::type;
    const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / NL;     // (row, channel)
    const int n0 = (threadIdx.x % NL) * 4, N = a.state_size;
    const int64_t total = (int64_t)a.num_seqs * a.channels;
    const int64_t at = id < total ? id : total - 1;
    const int64_t row = at / a.channels;
    const int c = (int)(at - row * a.channels);
    const int64_t bc = (int64_t)(c / (a.channels / a.groups)) * N;
    float h[4], A[4], Bv[4], Cv[4];
    if constexpr (ALIGNED) {
        f32x4 v = {0, 0, 0, 0}, w = {0, 0, 0, 0};
        if (n0 < N) {
            if (a.initial_state) v = *reinterpret_cast<const f32x4 *>(a.initial_state + at * N + n0);
            w = *reinterpret_cast<const f32x4 *>(a.A + (int64_t)c * N + n0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = v[j], A[j] = w[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool in = n0 + j < N;
        if constexpr (!ALIGNED) {
            h[j] = in && a.initial_state ? a.initial_state[at * N + n0 + j] : 0.0f;
            A[j] = in ? a.A[(int64_t)c * N + n0 + j] : 0.0f;
        }
        Bv[j] = in ? load1<DT>(a.B, row * a.B_stride + bc + n0 + j) : 0.0f;
        Cv[j] = in ? load1<DT>(a.C, row * a.C_stride + bc + n0 + j) : 0.0f;
    }
    const float u = load1<DT>(a.u, row * a.u_stride + c);
    float s = load1<DT>(a.delta, row * a.delta_stride + c) + (a.delta_bias ? a.delta_bias[c] : 0.0f);
    if (a.delta_softplus) s = softplus_f(s);
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = __builtin_fmaf(exp2_f(s * (A[j] * LOG2E_F)), h[j], s * u * Bv[j]);
        y = __builtin_fmaf(Cv[j], h[j], y);
    }
#pragma unroll
    for (int q = 1; q < NL; q *= 2) y += __shfl_xor(y, q);
    if (id >= total) return;
    if (a.final_state) {
        if constexpr (ALIGNED) {
            if (n0 < N) *reinterpret_cast<f32x4 *>(a.final_state + at * N + n0) = f32x4{h[0], h[1], h[2], h[3]};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + j < N) a.final_state[at * N + n0 + j] = h[j];
        }
    }
    if (n0 == 0) {
        y = __builtin_fmaf(a.D ? a.D[c] : 0.0f, u, y);
        if (a.z) {
            const float z = load1<DT>(a.z, row * a.z_stride + c);
            y *= z * sigmoid_f(z);
        }
        reinterpret_cast<E *>(a.out)[row * a.channels + c] = (E)y;
    }
}

// ------------------------------------------------------------------------------ launches
template <int DT, int CB, int M>
hipError_t fwd_form(const kda_ssm_args &a, float *ws, int32_t *err, hipStream_t st) {
    const Form f{CB, M};
    const int64_t T = a.total_tokens, blocks = blocks_of(f, a.channels, a.groups);
    const int L = tile_len(T, blocks);
    const int64_t tiles = T ? ceil_div(T, L) : 1, units = tiles * blocks;
    const dim3 grid((unsigned)ceil_div(units, WAVES));
    if (tiles > 1) {
        float *sums = ws + units * 1024 * M;
        int32_t *resets = (int32_t *)(sums + tiles * a.channels);
        ssm_tile_kernel<DT, CB, M><<<grid, 64 * WAVES, 0, st>>>(a, ws, sums, resets, err, L, (int)tiles, (int)blocks);
        if (hipError_t e = hipGetLastError()) return e;
        ssm_join_kernel<CB, M><<<dim3((unsigned)ceil_div(blocks * 16 * M, 4)), 256, 0, st>>>(a, ws, sums, resets, (int)tiles,
                                                                                             (int)blocks);
        if (hipError_t e = hipGetLastError()) return e;
    }
    ssm_scan_kernel<DT, CB, M><<<grid, 64 * WAVES, 0, st>>>(a, ws, err, L, (int)tiles, (int)blocks);
    return hipGetLastError();
}

template <int DT> hipError_t fwd_dt(const kda_ssm_args &a, float *ws, int32_t *err, hipStream_t st) {
    const Form f = form_of(a.state_size);
    if (f.cb == 4) return fwd_form<DT, 4, 1>(a, ws, err, st);
    if (f.cb == 2) return fwd_form<DT, 2, 1>(a, ws, err, st);
    if (f.m == 1) return fwd_form<DT, 1, 1>(a, ws, err, st);
    if (f.m == 2) return fwd_form<DT, 1, 2>(a, ws, err, st);
    return fwd_form<DT, 1, 4>(a, ws, err, st);
}

template <int DT, int NL> hipError_t decode_nl(const kda_ssm_args &a, hipStream_t st) {
    const int64_t threads = (int64_t)a.num_seqs * a.channels * NL;
    const dim3 grid((unsigned)ceil_div(threads, 256));
    const bool aligned = a.state_size % 4 == 0 && ((uintptr_t)a.initial_state | (uintptr_t)a.final_state | (uintptr_t)a.A) % 16 == 0;
    if (aligned) ssm_decode_kernel<DT, NL, true><<<grid, 256, 0, st>>>(a);
    else ssm_decode_kernel<DT, NL, false><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}
template <int DT> hipError_t decode_dt(const kda_ssm_args &a, hipStream_t st) {
    const int lanes = (a.state_size + 3) / 4;
    if (lanes <= 1) return decode_nl<DT, 1>(a, st);
    if (lanes <= 2) return decode_nl<DT, 2>(a, st);
    if (lanes <= 4) return decode_nl<DT, 4>(a, st);
    if (lanes <= 8) return decode_nl<DT, 8>(a, st);
    if (lanes <= 16) return decode_nl<DT, 16>(a, st);
    if (lanes <= 32) return decode_nl<DT, 32>(a, st);
    return decode_nl<DT, 64>(a, st);
}

}  // namespace

// Tokens of a tile: as many tiles as give the card about 4096 waves, of 16 tokens or more.
int tile_len(int64_t T, int64_t blocks) {
    int64_t L = T * blocks / 4096;
    L = L < 16 ? 16 : L > T ? T : L;
    return (int)((L + K - 1) / K * K);
}

}  // namespace ssm

size_t ssm_workspace(int64_t T, int64_t D, int64_t N, int64_t G) {
    using namespace ssm;
    const Form f = form_of((int)N);
    const int64_t blocks = blocks_of(f, D, G), tiles = T ? ceil_div(T, tile_len(T, blocks)) : 1;
    return tiles > 1 ? (size_t)(tiles * blocks * 1024 * f.m + tiles * D + tiles) * 4 : 0;
}

hipError_t launch_ssm_fwd(const kda_ssm_args &a, float *ws, int32_t *err, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return ssm::fwd_dt<KDA_DTYPE_F32>(a, ws, err, st);
    if (a.dtype == KDA_DTYPE_BF16) return ssm::fwd_dt<KDA_DTYPE_BF16>(a, ws, err, st);
    return ssm::fwd_dt<KDA_DTYPE_F16>(a, ws, err, st);
}
hipError_t launch_ssm_decode(const kda_ssm_args &a, hipStream_t st) {
    if (a.dtype == KDA_DTYPE_F32) return ssm::decode_dt<KDA_DTYPE_F32>(a, st);
    if (a.dtype == KDA_DTYPE_BF16) return ssm::decode_dt<KDA_DTYPE_BF16>(a, st);
    return ssm::decode_dt<KDA_DTYPE_F16>(a, st);
}

}  // namespace ops
}  // namespace kda
