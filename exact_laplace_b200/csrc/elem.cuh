// elem.cuh -- storage types of the sequence operators and the type they
// compute in (16-bit and fp32 rows in fp32, fp64 rows in fp64).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace lx {

template <typename T> struct AccOf { using A = float; };
template <> struct AccOf<double> { using A = double; };

template <typename A, typename T> __device__ __forceinline__ A to_acc(T v) { return (A)v; }
template <> __device__ __forceinline__ float to_acc<float, __half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_acc<float, __nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// one rounding to the nearest
template <typename T, typename A> __device__ __forceinline__ T from_acc(A v) { return (T)v; }
template <> __device__ __forceinline__ __half from_acc<__half, float>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_acc<__nv_bfloat16, float>(float v) { return __float2bfloat16_rn(v); }

// elements of T in one 16-byte access
template <typename T> struct VecOf { static constexpr int N = 16 / (int)sizeof(T); };

// N elements of T, moved in accesses of at most 16 bytes
template <typename T, int N> struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack { T v[N]; };

// The kernels of one call follow one another by programmatic launches (launch in seqop.h):
// a kernel is placed on the SMs while the last blocks of the one before still run.
// Its first statement waits for that kernel's end and its writes; then the next one
// may be placed.  (Without such a launch before or after, both do nothing.)
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// e^(lam d): lam is a log decay; -inf (no memory) acts as a decay that no d >= 1
// survives, without the NaN of -inf * 0.  fp32: what the product lam d rounds off
// (2^-24 of it, so 1e-6 of the result at lam d = 16) is put back.
__device__ __forceinline__ float clamp_lam(float lam) { return lam < -1e25f ? -1e25f : lam; }
__device__ __forceinline__ double clamp_lam(double lam) { return lam < -1e25 ? -1e25 : lam; }
__device__ __forceinline__ float decay(float lam, float d) {
    const float x = lam * d, e = expf(x);
    return fmaf(e, fmaf(lam, d, -x), e);
}
__device__ __forceinline__ double decay(double lam, double d) { return exp(lam * d); }

}  // namespace lx
