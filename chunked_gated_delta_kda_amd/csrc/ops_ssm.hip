// ops_ssm.hip -- the selective state space scan: prompts (over a packed batch) and one token of
// each sequence. The mathematics and the register layout are in ops_ssm.hpp.
//
// Prompts go one of two ways (by_blocks): in one launch, a block of waves per 16 channels walking the
// tokens (ssm_scan_kernel), or by waves. Then the time axis is cut into tiles of consecutive packed
// tokens, whatever sequences start or end in them, so that few channels still fill the card:
//   1. ssm_tile_kernel: each tile from a zero state: its end state E and the sum S of its
//      step sizes, so that the tile maps a state h to e^{A S} h + E (to E alone where a sequence
//      starts in it);
//   2. ssm_join_kernel: those maps one after another per (channel, state): the state each tile
//      starts from, in E's place;
//   3. ssm_wide_kernel: the scan itself, from that state.
// Bound by vector issue: a (token, channel, state) costs two multiplications, an exponential and the
// product with C, and steps 1 and 3 both pay the first three. Measured on MI355X, 65536 x 1024 x 16 bf16 with a
// gate: tiles 189 us (93% of the issue that their instructions cost), join 18, scan 272; staging the activations
// (softplus, gate, borders) is about a third of both.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "kda_launch.hpp"
#include "ops_ssm.hpp"

namespace kda {
namespace ops {
namespace ssm {
namespace {

constexpr int K_TILE = 8, K_SCAN = 4;   // tokens a wave stages at a time

// K tokens' activations of a wave, one element a lane, in flight while the tokens before are
// computed.
template <int DT, int K, int M, bool OUT> struct Raw {
    using E = typename Elem<DT>::type;
    E delta[K], u[K], z[K], B[K][M], C[K][M];
    template <int CB>
    __device__ __forceinline__ void load(const kda_ssm_args &a, const Place<CB, M> &p, int t, int stop) {
        const uint32_t ch = (uint32_t)p.ch * sizeof(E);
        const int64_t g0 = (int64_t)p.group * p.N * sizeof(E);
        t = t < stop ? t : stop - 1;            // rows past the end: the last one again
        const int last = stop - 1 - t;
        const RowsOf dr((const char *)a.delta, a.delta_stride, t, sizeof(E)), ur((const char *)a.u, a.u_stride, t, sizeof(E));
        const RowsOf zr((const char *)a.z, a.z_stride, t, sizeof(E));
        const RowsOf Br((const char *)a.B + g0, a.B_stride, t, sizeof(E)), Cr((const char *)a.C + g0, a.C_stride, t, sizeof(E));
        static_assert(K <= 8, "rows of RowsOf");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            delta[k] = at<DT>(dr.at(k, last), ch);
            u[k] = at<DT>(ur.at(k, last), ch);
            if (OUT && a.z) z[k] = at<DT>(zr.at(k, last), ch);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int n = p.nat_state(m);
                const uint32_t st = (uint32_t)(n < p.N ? n : p.N - 1) * sizeof(E);
                B[k][m] = at<DT>(Br.at(k, last), st);
                if (OUT) C[k][m] = at<DT>(Cr.at(k, last), st);
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
    constexpr int K = K_TILE;
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
    Raw<DT, K, M, false> raw;
    raw.load(a, p, t, t1);
    while (t < t1) {
        float x[K], B[K][M];
        const int count = t1 - t;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float d = (float)raw.delta[k] + bias;
            float s = step_of(d, a.delta_softplus);
            x[k] = s * (float)raw.u[k];
            const bool step = k < count;
            s = step ? s : 0.0f, x[k] = step ? x[k] : 0.0f;    // no step: e^0 h + 0 (B too: what is repeated may be infinite)
            sum += s;
            steps[k * 16 * CB + CB * p.i + p.g % CB] = s;
#pragma unroll
            for (int m = 0; m < M; ++m) B[k][m] = step && p.nat_state(m) < p.N ? (float)raw.B[k][m] : 0.0f;
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

template <int CB, int M>
__global__ __launch_bounds__(256) void ssm_join_kernel(const kda_ssm_args a, float *ws, const float *sums, const int32_t *resets,
                                                       int tiles, int blocks) {
    __shared__ JoinLds lds;
    join_tiles<CB, M>(a, lds, ws, sums, resets, 1, tiles, blocks, blockIdx.x / (16 * M), blockIdx.x % (16 * M), false);
}

// The scan where by_blocks takes the other one not (state sizes over 32, many sequences, few channels of many
// tokens): a wave by itself, all states of its channels in its registers, from the joined states of its tile. Four
// waves a SIMD cost the form of up to 16 states 1 (fp32, fp16) or 5 (bf16) spilled registers.
template <int DT, int CB, int M>
__global__ __launch_bounds__(64 * WAVES, M == 1 ? 4 : 1) void ssm_wide_kernel(const kda_ssm_args a, const float *ws, int32_t *err, int L,
                                                              int tiles, int blocks) {
    using E = typename Elem<DT>::type;
    constexpr int K = K_SCAN;
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
    const uint32_t ch = (uint32_t)p.ch * sizeof(E);
    int t = t0;
    Raw<DT, K, M, true> raw{};
    raw.load(a, p, t, t1);
    // `count` tokens of one sequence
    auto stage = [&](int count, auto whole) {
        float x[K], u[K], z[K], B[K][M], y[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool on = whole || k < count;     // the next sequence's rows stay out of this state
            const float d = (float)raw.delta[k] + bias;
            const float s = step_of(d, a.delta_softplus);
            u[k] = (float)raw.u[k];
            x[k] = on ? s * u[k] : 0.0f;
            z[k] = a.z ? (float)raw.z[k] : 0.0f;
            steps[k * 16 * CB + CB * p.i + p.g % CB] = on ? s : 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const bool in = p.nat_state(m) < p.N;
                B[k][m] = on && in ? (float)raw.B[k][m] : 0.0f;
                rows[k * NS + p.nat_state(m)] = in ? (float)raw.C[k][m] : 0.0f;
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
        char *out = (char *)a.out + (int64_t)from * a.channels * sizeof(E);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float gated = z[k] * sigmoid_f(z[k]);
            const float v = __builtin_fmaf(skip, u[k], y[k]) * (a.z ? gated : 1.0f);
            if (whole || k < count) put(uniform(out + (int64_t)k * a.channels * sizeof(E)), ch, (E)v);
        }
    };
    while (true) {
        const int stop = end < t1 ? end : t1;
        while (stop - t >= K) stage(K, std::true_type{});     // lanes of one channel store the same
        if (t < stop) {
            stage(stop - t < K ? stop - t : K, std::false_type{});
            if (t < stop) continue;
        }
        if (t < end) break;             // the sequence goes on in the next tile
        store_state<CB, M>(a.final_state, n, a, p, h);
        for (++n; n < a.num_seqs && off.at(n + 1) <= t; ++n) pass_state<CB, M>(a.final_state, a.initial_state, n, a, p);
        if (t >= t1 || n >= a.num_seqs) break;
        end = off.at(n + 1);
        load_state<CB, M>(a.initial_state, n, a, p, h);
    }
}

// The scan in one launch, for state sizes up to 32 where the channels alone fill the card or the batch is
// short (by_blocks): a block of W = 8 waves owns 16 channels and walks all tokens in steps of up to W KT of
// one sequence, each wave KT of them. The exponential of a (token, channel, state) is formed once and
// one pass over the inputs is enough. Per step:
//   1. a wave forms its tokens' decays and inputs, kept in registers, and runs them from a zero
//      state: E; with P = e^{A sum s} that is the wave's map h -> P h + E;
//   2. the block's first threads, one per (channel, state), run the state through the W maps in LDS,
//      leaving each wave's input state there, while every wave stages its tokens of the next step;
//   3. a wave runs its tokens again from its input state, for y.
// NB: 16-state blocks. The four blocks of a product are TP = 4/NB tokens by NB blocks of states; product
// q holds tokens TP q + b / NB, states 16 (b % NB) + 4 g + j, channel i.
// 8192 x 4096 x 16 bf16 with a gate: 235 us with rows one after another, 270 where u and z are halves of rows of 16
// KiB; 70% of the busy cycles issue vector instructions, the rest are the two barriers of a step.
template <int NB> struct Scan {
    static constexpr int W = 8, Q = 4, KT = 4 * Q / NB, TP = 4 / NB;   // waves, tokens of a wave, of a product, products
    static constexpr int NS = 16 * NB, PAIRS = 256 * NB, SROW = KT + 4, STEP = W * KT;
};
template <int NB> struct ScanLds {
    using S = Scan<NB>;
    float E[S::W][S::PAIRS], P[S::W][S::PAIRS], h[S::W][S::PAIRS];
    float steps[S::W][16 * S::SROW], C[S::W][2][S::KT * S::NS];
};

// From one value per token of a product (sums over j) to the lane that carries the token: TP q + g / NB.
template <int TP> __device__ __forceinline__ float token_lane(const float (&r)[TP]) {
    if constexpr (TP == 4) return swap16_add(swap32_add(r[0], r[2]), swap32_add(r[1], r[3]));
    else {
        const float s = swap32_add(r[0], r[TP - 1]);
        return swap16_add(s, s);
    }
}

// A step: its first token, how many, and the sequence they belong to.
struct Step {
    int t, count, n, end;
    template <int STEP> __device__ __forceinline__ void size(int T) {
        const int stop = end < T ? end : T;
        count = stop - t < STEP ? stop - t : STEP;
    }
    // the step after this one
    template <int STEP> __device__ __forceinline__ Step next(const Offsets &off, int T) const {
        Step s{t + count, 0, n, end};
        if (s.t == s.end && s.t < T) {
            for (++s.n; s.n < off.N - 1 && off.at(s.n + 1) <= s.t; ++s.n) {}
            s.end = off.at(s.n + 1);
        }
        s.template size<STEP>(T);
        return s;
    }
};

template <int DT, int NB>
__global__ __launch_bounds__(64 * Scan<NB>::W) void ssm_scan_kernel(const kda_ssm_args a, int32_t *err, int blocks, int xcds) {
    using E = typename Elem<DT>::type;
    using Z = Scan<NB>;
    constexpr int KT = Z::KT, TP = Z::TP, Q = Z::Q, NS = Z::NS, SROW = Z::SROW, W = Z::W, STEP = Z::STEP;
    constexpr uint32_t es = sizeof(E);
    extern __shared__ __align__(16) char lds_raw[];
    ScanLds<NB> &lds = *reinterpret_cast<ScanLds<NB> *>(lds_raw);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    // Blocks go to the XCDs in turn: neighbouring channels (of one memory line) to one XCD.
    const int id = blockIdx.x, block = xcds > 1 ? (id % xcds) * (blocks / xcds) + id / xcds : id;
    const Offsets off{a.cu_seqlens, a.num_seqs, a.total_tokens};
    if (id == 0) check_offsets(off, err, threadIdx.x, 64 * W);
    const int N = a.state_size, per = a.channels / a.groups, pb = (per + 15) / 16;
    const int group = block / pb, base = group * per + (block - group * pb) * 16, last = group * per + per - 1;
    const int c = base + i, cc = c <= last ? c : last;
    const int T = a.total_tokens;

    // The block's state, one (channel, state) a thread: pair 4 lane + j of state block b, as E and P lie.
    const int op = threadIdx.x & 255, ob = threadIdx.x >> 8;
    const int oc = base + ((op >> 2) & 15), on = 16 * ob + 4 * (op >> 6) + (op & 3);
    const bool owner = threadIdx.x < Z::PAIRS, holds = owner && oc <= last && on < N;
    const int64_t own_at = (int64_t)oc * N + on, own_step = (int64_t)a.channels * N;
    auto first_state = [&](int seq) { return holds && a.initial_state ? a.initial_state[seq * own_step + own_at] : 0.0f; };
    auto last_state = [&](int seq, float h) {
        if (holds && a.final_state) a.final_state[seq * own_step + own_at] = h;
    };
    if (T == 0) {
        for (int q = 0; q < a.num_seqs; ++q) last_state(q, first_state(q));
        return;
    }
    Step cur{0, 0, off.find(0), 0};
    cur.end = off.at(cur.n + 1);
    cur.size<STEP>(T);
    float state = first_state(cur.n);
    for (int q = 0; q < cur.n; ++q) last_state(q, first_state(q));

    float A2[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = 16 * b + 4 * g + j;
            A2[b][j] = c <= last && n < N ? a.A[(int64_t)c * N + n] * LOG2E_F : 0.0f;
        }
    const float bias = a.delta_bias ? a.delta_bias[cc] : 0.0f, skip = a.D ? a.D[cc] : 0.0f;
    // A lane's place in a product's rows: its token of the product, its channel and its state.
    const int nat_st = 16 * (g % NB) + i, tl = g / NB;
    const bool state_in = nat_st < N;
    const uint32_t ch = (uint32_t)cc * es, st = (uint32_t)(state_in ? nat_st : N - 1) * es;
    const uint32_t od = (uint32_t)(tl * a.delta_stride) * es + ch, ou = (uint32_t)(tl * a.u_stride) * es + ch;
    const uint32_t oz = (uint32_t)(tl * a.z_stride) * es + ch, oo = (uint32_t)(tl * a.channels) * es + ch;
    const uint32_t oB = (uint32_t)(tl * a.B_stride) * es + st, oC = (uint32_t)(tl * a.C_stride) * es + st;
    const char *const u0 = (const char *)a.u, *const d0 = (const char *)a.delta, *const z0 = (const char *)a.z;
    const char *const B0 = (const char *)a.B + (int64_t)group * N * es, *const C0 = (const char *)a.C + (int64_t)group * N * es;
    const bool has_z = a.z != nullptr;
    E rdelta[Q], ru[Q], rz[Q] = {}, rB[Q], rC[Q];
    auto load = [&](const Step &s) {
        const int t = s.t + w * KT;
        if (t + KT <= T) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int64_t r = (int64_t)(t + TP * q) * es;
                rdelta[q] = at<DT>(d0 + r * a.delta_stride, od);
                ru[q] = at<DT>(u0 + r * a.u_stride, ou);
                if (has_z) rz[q] = at<DT>(z0 + r * a.z_stride, oz);
                rB[q] = at<DT>(B0 + r * a.B_stride, oB);
                rC[q] = at<DT>(C0 + r * a.C_stride, oC);
            }
        } else {
#pragma unroll
            for (int q = 0; q < Q; ++q) {     // rows past the batch's end: its last one again
                const int tq = t + TP * q + tl;
                const int64_t r = (int64_t)(tq < T ? tq : T - 1) * es;
                rdelta[q] = at<DT>(d0 + r * a.delta_stride, ch);
                ru[q] = at<DT>(u0 + r * a.u_stride, ch);
                if (has_z) rz[q] = at<DT>(z0 + r * a.z_stride, ch);
                rB[q] = at<DT>(B0 + r * a.B_stride, st);
                rC[q] = at<DT>(C0 + r * a.C_stride, st);
            }
        }
    };
    float u[Q], gate[Q], x[Q], Bq[Q];
    auto stage = [&](const Step &sp, int turn) {
        const int left = sp.count - w * KT;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = TP * q + tl;
            const bool is = k < left;         // past the step's end: no step, nothing in (B too: what lies there may be infinite)
            const float d = (float)rdelta[q] + bias;
            float s = step_of(d, a.delta_softplus);
            s = is ? s : 0.0f;
            u[q] = is ? (float)ru[q] : 0.0f;
            x[q] = s * u[q];
            const float gated = (float)rz[q] * sigmoid_f((float)rz[q]);
            gate[q] = has_z ? gated : 1.0f;
            Bq[q] = is && state_in ? (float)rB[q] : 0.0f;
            lds.steps[w][i * SROW + k] = s;
            lds.C[w][turn][k * NS + nat_st] = state_in ? (float)rC[q] : 0.0f;
        }
        wave_fence();
    };
    load(cur);
    stage(cur, 0);
    Step nxt = cur.next<STEP>(off, T);
    if (nxt.t < T) load(nxt);
    for (int turn = 0;; turn ^= 1) {
        float step[KT], e[KT][NB][4], in_[KT][NB][4], sum = 0.0f;
#pragma unroll
        for (int k = 0; k < KT; k += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(&lds.steps[w][i * SROW + k]);
#pragma unroll
            for (int b = 0; b < 4; ++b) step[k + b] = v[b];
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            f32x16 zero;
#pragma unroll
            for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
            const f32x16 v = __builtin_amdgcn_mfma_f32_16x16x1f32(Bq[q], x[q], zero, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int k = TP * q + (r / 4) / NB, b = (r / 4) % NB, j = r % 4;
                in_[k][b][j] = v[r];
                e[k][b][j] = exp2_f(A2[b][j] * step[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < KT; ++k) sum += step[k];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            f32x4 ve, vp;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ve[j] = in_[0][b][j];
#pragma unroll
                for (int k = 1; k < KT; ++k) ve[j] = __builtin_fmaf(e[k][b][j], ve[j], in_[k][b][j]);
                vp[j] = exp2_f(A2[b][j] * sum);
            }
            *reinterpret_cast<f32x4 *>(&lds.E[w][256 * b + 4 * lane]) = ve;
            *reinterpret_cast<f32x4 *>(&lds.P[w][256 * b + 4 * lane]) = vp;
        }
        float uc[Q], gc[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) uc[q] = u[q], gc[q] = gate[q];
        lds_barrier();
        const bool more = nxt.t < T;
        if (owner) {
#pragma unroll
            for (int v0 = 0; v0 < W; v0 += 4) {
                float me[4], mp[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) me[v] = lds.E[v0 + v][threadIdx.x], mp[v] = lds.P[v0 + v][threadIdx.x];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    lds.h[v0 + v][threadIdx.x] = state;
                    state = __builtin_fmaf(mp[v], state, me[v]);
                }
            }
        }
        if (cur.t + cur.count == cur.end) {      // the sequence's last token; empty ones may follow, and the next one begins
            last_state(cur.n, state);
            for (int q = cur.n + 1; q < a.num_seqs && off.at(q + 1) <= cur.end; ++q) last_state(q, first_state(q));
            if (more) state = first_state(nxt.n);
        }
        Step after = nxt;
        if (more) {
            stage(nxt, turn ^ 1);
            after = nxt.next<STEP>(off, T);
            if (after.t < T) load(after);
        }
        lds_barrier();
        float own[NB][4], y[Q];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(&lds.h[w][256 * b + 4 * lane]);
#pragma unroll
            for (int j = 0; j < 4; ++j) own[b][j] = v[j];
        }
        const float *Cr = lds.C[w][turn];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float r[TP];
#pragma unroll
            for (int b0 = 0; b0 < TP; ++b0) {
                const int k = TP * q + b0;
                r[b0] = 0.0f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const f32x4 c4 = *reinterpret_cast<const f32x4 *>(Cr + k * NS + 16 * b + 4 * g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        own[b][j] = __builtin_fmaf(e[k][b][j], own[b][j], in_[k][b][j]);
                        r[b0] = __builtin_fmaf(c4[j], own[b][j], r[b0]);
                    }
                }
            }
            y[q] = token_lane<TP>(r);
        }
        const int left = c <= last ? cur.count - w * KT : 0;
        char *out = (char *)a.out + (int64_t)(cur.t + w * KT) * a.channels * es;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const float v = __builtin_fmaf(skip, uc[q], y[q]) * gc[q];
            if (TP * q + tl < left) put(uniform(out + (int64_t)(TP * q) * a.channels * es), oo, (E)v);
        }
        if (!more) break;
        cur = nxt, nxt = after;
    }
}

// One token of each sequence: four states a lane, NL lanes a channel, ROWS sequences a thread, whose loads
// are in flight together and share the channel's A. Every state is read and written once, by one lane,
// so it may be updated in place. ALIGNED: four states, and four elements of a B or C row, in one access.
// Measured on MI355X, 256 x 4096 x 16 bf16 with 1 | 2 | 4 | 8 rows: 41.6 | 31.1 | 32.0 | 33.9 us (4.6 TB/s at 2).
constexpr int ROWS = 2;
template <int DT, int NL, bool ALIGNED>
__global__ __launch_bounds__(256) void ssm_decode_kernel(const kda_ssm_args a) {
    using E = typename Elem<DT>::type;
    typedef E E4 __attribute__((ext_vector_type(4)));
    const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / NL;     // channel
    const int n0 = (threadIdx.x % NL) * 4, N = a.state_size;
    const int c = (int)(id < a.channels ? id : a.channels - 1);
    const int64_t bc = (int64_t)(c / (a.channels / a.groups)) * N;
    float A2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] = n0 + j < N ? a.A[(int64_t)c * N + n0 + j] * LOG2E_F : 0.0f;
    const float bias = a.delta_bias ? a.delta_bias[c] : 0.0f, skip = a.D ? a.D[c] : 0.0f;
    for (int64_t r0 = (int64_t)blockIdx.y * ROWS; r0 < a.num_seqs; r0 += (int64_t)gridDim.y * ROWS) {
        float h[ROWS][4], Bv[ROWS][4], Cv[ROWS][4], u[ROWS], s[ROWS], z[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t row = r0 + k < a.num_seqs ? r0 + k : a.num_seqs - 1;
            const int64_t at = (row * a.channels + c) * N + n0;
            if constexpr (ALIGNED) {
                f32x4 v = {0, 0, 0, 0};
                E4 b = {0, 0, 0, 0}, q = {0, 0, 0, 0};
                if (n0 < N) {
                    if (a.initial_state) v = *reinterpret_cast<const f32x4 *>(a.initial_state + at);
                    b = *reinterpret_cast<const E4 *>((const E *)a.B + row * a.B_stride + bc + n0);
                    q = *reinterpret_cast<const E4 *>((const E *)a.C + row * a.C_stride + bc + n0);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) h[k][j] = v[j], Bv[k][j] = (float)b[j], Cv[k][j] = (float)q[j];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = n0 + j < N;
                    h[k][j] = in && a.initial_state ? a.initial_state[at + j] : 0.0f;
                    Bv[k][j] = in ? load1<DT>(a.B, row * a.B_stride + bc + n0 + j) : 0.0f;
                    Cv[k][j] = in ? load1<DT>(a.C, row * a.C_stride + bc + n0 + j) : 0.0f;
                }
            }
            u[k] = load1<DT>(a.u, row * a.u_stride + c);
            s[k] = load1<DT>(a.delta, row * a.delta_stride + c);
            z[k] = a.z ? load1<DT>(a.z, row * a.z_stride + c) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t row = r0 + k;
            if (row >= a.num_seqs) break;
            float st = s[k] + bias;
            if (a.delta_softplus) st = softplus_f(st);
            const float x = st * u[k];
            float y = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[k][j] = __builtin_fmaf(exp2_f(st * A2[j]), h[k][j], x * Bv[k][j]);
                y = __builtin_fmaf(Cv[k][j], h[k][j], y);
            }
#pragma unroll
            for (int q = 1; q < NL; q *= 2) y += __shfl_xor(y, q);
            if (id >= a.channels) continue;
            const int64_t at = (row * a.channels + c) * N + n0;
            if (a.final_state) {
                if constexpr (ALIGNED) {
                    if (n0 < N) *reinterpret_cast<f32x4 *>(a.final_state + at) = f32x4{h[k][0], h[k][1], h[k][2], h[k][3]};
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n0 + j < N) a.final_state[at + j] = h[k][j];
                }
            }
            if (n0 == 0) {
                y = __builtin_fmaf(skip, u[k], y);
                if (a.z) y *= z[k] * sigmoid_f(z[k]);
                reinterpret_cast<E *>(a.out)[row * a.channels + c] = (E)y;
            }
        }
    }
}

// ------------------------------------------------------------------------------ launches
// Whether the scan by blocks takes a batch. Its blocks of 16 channels run one to a CU, ceil(blocks / 256) rounds of
// 28 to 33 ns a token (inputs in the caches, or not); a step of it is one sequence's, so every sequence wastes half a
// step of 128 tokens. The scan by waves costs 29 ns a token and 256 blocks' channels, spread over the card at any
// count, and 40 us for its three launches and joined states. A second block of states costs 1.65 and 1.8 times that.
// Measured on MI355X (us, blocks | waves; bf16, gate, tokens x channels x states, inputs in the caches where they
// fit): 2048 x 4096 x 16 59 | 90, 4096 x 4096 x 16 113 | 144, 8192 x 4096 x 16 232 | 262 (not in the caches: 271 | 271),
// 12288 x 4096 x 16 398 | 361, 16384 x 4096 x 16 528 | 470, 2048 x 8192 x 16 109 | 143, 4096 x 5120 x 16 217 | 170, 8192 x
// 4096 x 32 432 | 464, 2048 x 2048 x 16 52 | 65, 4096 x 1024 x 16 101 | 70, 1024 x 1024 x 16 27 | 30, 1024 x 256 x 16 27 |
// 27, 2048 x 256 x 16 51 | 31, 512 x 256 x 16 15.5 | 25; 8192 tokens in 32 sequences x 4096 x 16 265 | 255, in 100 439 | 232.
bool by_blocks(int64_t T, int64_t S, int64_t D, int64_t N, int64_t G) {
    if (N > 32) return false;
    const bool two = N > 16;
    const double blocks = (double)(G * ceil_div(D / G, 16));
    const double by_block = std::ceil(blocks / 256.0) * ((double)T + (two ? 32.0 : 64.0) * (double)S) * 0.0325 * (two ? 1.65 : 1.0);
    return by_block <= blocks / 256.0 * (double)T * 0.029 * (two ? 1.8 : 1.0) + 40.0;
}

template <int DT, int CB, int M>
hipError_t tile_states(const kda_ssm_args &a, float *ws, int32_t *err, int L, int64_t tiles, int64_t blocks, hipStream_t st) {
    const int64_t units = tiles * blocks;
    float *sums = ws + units * 1024 * M;
    int32_t *resets = (int32_t *)(sums + tiles * a.channels);
    ssm_tile_kernel<DT, CB, M><<<dim3((unsigned)ceil_div(units, WAVES)), 64 * WAVES, 0, st>>>(a, ws, sums, resets, err, L, (int)tiles,
                                                                                             (int)blocks);
    if (hipError_t e = hipGetLastError()) return e;
    ssm_join_kernel<CB, M><<<dim3((unsigned)(blocks * 16 * M)), 256, 0, st>>>(a, ws, sums, resets, (int)tiles, (int)blocks);
    return hipGetLastError();
}

template <int DT, int NB> hipError_t fwd_block(const kda_ssm_args &a, int32_t *err, hipStream_t st) {
    const int64_t blocks = a.groups * ceil_div(a.channels / a.groups, 16);
    static std::atomic<uint64_t> done;
    constexpr int bytes = (int)sizeof(ScanLds<NB>);
    if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void *>(ssm_scan_kernel<DT, NB>), bytes, done)) return e;
    ssm_scan_kernel<DT, NB><<<dim3((unsigned)blocks), 64 * Scan<NB>::W, bytes, st>>>(a, err, (int)blocks, blocks % 8 == 0 ? 8 : 1);
    return hipGetLastError();
}

template <int DT, int CB, int M>
hipError_t fwd_wide(const kda_ssm_args &a, float *ws, int32_t *err, hipStream_t st) {
    const int64_t T = a.total_tokens, blocks = blocks_of(Form{CB, M}, a.channels, a.groups);
    const int L = tile_len(T, blocks);
    const int64_t tiles = T ? ceil_div(T, L) : 1;
    if (tiles > 1)
        if (hipError_t e = tile_states<DT, CB, M>(a, ws, err, L, tiles, blocks, st)) return e;
    ssm_wide_kernel<DT, CB, M><<<dim3((unsigned)ceil_div(tiles * blocks, WAVES)), 64 * WAVES, 0, st>>>(a, ws, err, L, (int)tiles,
                                                                                                      (int)blocks);
    return hipGetLastError();
}

template <int DT> hipError_t fwd_dt(const kda_ssm_args &a, float *ws, int32_t *err, hipStream_t st) {
    const Form f = form_of(a.state_size);
    if (by_blocks(a.total_tokens, a.num_seqs, a.channels, a.state_size, a.groups))
        return f.cb == 4 ? fwd_block<DT, 1>(a, err, st) : fwd_block<DT, 2>(a, err, st);
    if (f.cb == 4) return fwd_wide<DT, 4, 1>(a, ws, err, st);
    if (f.cb == 2) return fwd_wide<DT, 2, 1>(a, ws, err, st);
    if (f.m == 1) return fwd_wide<DT, 1, 1>(a, ws, err, st);
    if (f.m == 2) return fwd_wide<DT, 1, 2>(a, ws, err, st);
    return fwd_wide<DT, 1, 4>(a, ws, err, st);
}

template <int DT, int NL> hipError_t decode_nl(const kda_ssm_args &a, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div((int64_t)a.channels * NL, 256), (unsigned)std::min<int64_t>(65535, ceil_div(a.num_seqs, ROWS)));
    const int64_t es = (int64_t)dtype_bytes(DT);
    const bool aligned = a.state_size % 4 == 0 && ((uintptr_t)a.initial_state | (uintptr_t)a.final_state) % 16 == 0 &&
                         a.B_stride % 4 == 0 && a.C_stride % 4 == 0 && ((uintptr_t)a.B | (uintptr_t)a.C) % (4 * es) == 0;
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

// Tokens of a tile: as many tiles as give the card about 4096 waves (four to a SIMD), of 8 tokens or more; and where
// the channels are few, sqrt(0.12 T): a wave takes 0.25 us a token in each of its two kernels, the join 0.06 us a tile.
// Measured on MI355X (us, with 0 | 0.06 | 0.12 | 0.25 T under the root; bf16): 23739 x 9 x 16 106 | 68 | 68 | 75, 65536 x 64 x 16
// 259 | 106 | 107 | 117, 32768 x 128 x 16 157 | 98 | 79 | 89, 8192 x 64 x 16 48 | 45 | 45 | 51, 65536 x 48 x 64 181 | 163 | 178 | 171. At
// least 16 | 8 tokens: 128 x 64 x 64 26 | 21, 500 x 128 x 128 36 | 32, 300 x 1000 x 128 in 3 sequences 64 | 67.
int tile_len(int64_t T, int64_t blocks) {
    int64_t L = std::max<int64_t>(T * blocks / 4096, (int64_t)std::sqrt(0.12 * (double)T));
    L = L < 8 ? 8 : L > T ? T : L;
    return (int)((L + 7) / 8 * 8);
}

}  // namespace ssm

size_t ssm_workspace(int64_t T, int64_t D, int64_t N, int64_t G, int64_t S) {
    using namespace ssm;
    const Form f = form_of((int)N);
    const int64_t blocks = blocks_of(f, D, G);
    const int64_t tiles = T ? ceil_div(T, tile_len(T, blocks)) : 1;
    if (tiles <= 1 || by_blocks(T, S, D, N, G)) return 0;
    return (size_t)(tiles * blocks * 1024 * f.m + tiles * D + tiles) * 4;
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
