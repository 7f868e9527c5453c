// ops_common.hpp -- device building blocks shared by the operators beside the delta rule:
// the short convolution (ops_conv.hip), the selective scan (ops_ssm.hip, ops_ssm_bwd.hip)
// and the paged token attention (ops_attn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace ops {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float LOG2E_F = 1.4426950408889634f;
constexpr float LN2_F = 0.6931471805599453f;

// Element types of activations. Arithmetic is fp32 throughout; a store rounds once, to
// nearest even.
template <int DT> struct Elem;
template <> struct Elem<KDA_DTYPE_F32> { using type = float; };
template <> struct Elem<KDA_DTYPE_BF16> { using type = __bf16; };
template <> struct Elem<KDA_DTYPE_F16> { using type = _Float16; };

// Row lookups over packed offsets. Offsets are clamped to [0, T] on reading, with c_0 = 0 and
// c_N = T whatever the array holds, so every index formed from them is in bounds even where
// the array is malformed (check_offsets raises the error bit for that).
struct Offsets {
    const int32_t *cu;   // NULL: one sequence
    int N, T;
    __device__ __forceinline__ int at(int i) const {
        if (i <= 0) return 0;
        if (i >= N) return T;
        const int c = cu[i];
        return c < 0 ? 0 : c > T ? T : c;
    }
    // the sequence n of row t (0 <= t < T): at(n) <= t < at(n + 1)
    __device__ __forceinline__ int find(int t) const {
        int lo = 0, hi = N;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (at(mid) <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

// Raises KDA_DEVERR_CU_SEQLENS unless 0 = c_0 <= ... <= c_N = T. Called by the threads of one
// block of a launch.
__device__ __forceinline__ void check_offsets(const Offsets &o, int32_t *err, int tid, int nthreads) {
    if (!o.cu || !err) return;
    bool bad = false;
    for (int i = tid; i <= o.N; i += nthreads) {
        const int c = o.cu[i];
        bad |= i == 0 ? c != 0 : c < o.cu[i - 1];
        bad |= i == o.N && c != o.T;
    }
    if (bad) atomicOr(err, KDA_DEVERR_CU_SEQLENS);
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_f(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + e^-x): 0 and 1 at the ends (e^-x overflows to infinity, whose reciprocal is 0).
__device__ __forceinline__ float sigmoid_f(float x) { return rcp_f(1.0f + exp2_f(-x * LOG2E_F)); }

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), with log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, and
// atanh(s) / s = 1 + q p(q), q = s^2 <= 1/9: p is the polynomial of degree 3 whose largest relative error in the
// result is smallest (found by linear programming): 5.5e-9 with these coefficients, as good as the odd series to s^13
// and two operations shorter. Unlike log(1 + e) the form keeps its relative precision where e is small (step
// sizes near 1e-3 come from there).
__device__ __forceinline__ float softplus_f(float x) {
    const float e = exp2_f(-__builtin_fabsf(x) * LOG2E_F);
    const float s = e * rcp_f(2.0f + e);
    const float q = s * s;
    float p = __builtin_fmaf(q, 0.14005993f, 0.14000903f);
    p = __builtin_fmaf(p, q, 0.20010763f);
    p = __builtin_fmaf(p, q, 0.33333209f);
    p = __builtin_fmaf(p, q, 1.0f);
    return __builtin_fmaf(2.0f * s, p, __builtin_fmaxf(x, 0.0f));
}

// Sums across the four 16-lane rows of a wave. v_permlane32_swap exchanges the upper half of
// its first operand with the lower half of its second, v_permlane16_swap the odd rows of its
// first with the even rows of its second; adding the two results leaves in each lane a sum
// over a pair of rows, of the first value in one half and of the second in the other.
__device__ __forceinline__ float swap32_add(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_add(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// What another lane of the row holds, by a DPP control word.
template <int CTRL> __device__ __forceinline__ float dpp_f(float x) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// Barrier of a block over its LDS traffic alone: unlike __syncthreads it does not wait for global
// loads in flight, so what is loaded ahead stays in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_waitcnt(0xc07f);     // lgkmcnt(0), the others open
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace ops
}  // namespace kda
