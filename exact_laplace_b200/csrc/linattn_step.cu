// linattn_step.cu -- decayed linear attention for one token per row, against a
// cache of states updated in place:
//     S <- e^lam S + k v^T,      o = scale S^T q.
//
// Bound by memory: a state of dk dv values is read and written once (8 dk dv
// bytes in fp32), against 3 + 2 (q-heads per state) flops a value.  A block
// holds a [dk, TC] piece of one state in registers: all of its loads are in
// flight before the first is used, and the state is not read again for the
// outputs.  TC = 64 columns of fp32 (16 lanes x 16 bytes) where there are enough
// blocks to fill the GPU, 32 where there are few, so that one token's states
// spread over more SMs.
//
// 4096 states of 128 x 128 (543 MB in all): 101 us, 5.4 TB/s, five blocks of 256
// threads on an SM (48 registers; without that limit four: 107 us; two: 154).
// TC = 128: 111 us, and 62 against 35 us for 64 x 64, whose blocks were half idle;
// TC = 32: 142 us.  One row of 16 states: 3.5 us, launch and latency.  fp64 states,
// two blocks on an SM: 4096 of 128 x 128 in 311 us, 3.5 TB/s.
// With slots every block looks through all of them for its own: nothing beside the
// states of a few hundred rows, but 186 against 138 us for 8192 rows of 2 states of
// 64 x 64.
#include <algorithm>

#include "devcache.h"
#include "elem.cuh"
#include "seqop.h"

namespace lx {

constexpr int STEP_NT = 256;
constexpr int STEP_GB = 4;  // q-heads whose partial sums are joined at a time
constexpr int STEP_DK = 128;

// LANES lanes across the columns, STEP_NT / LANES row groups
template <typename T, int LANES>
__global__ void __launch_bounds__(STEP_NT, sizeof(T) == 8 ? 2 : 5) k_step(const __grid_constant__ LinStep P) {
    using A = typename AccOf<T>::A;
    constexpr int VN = 16 / (int)sizeof(A), TC = LANES * VN, RG = STEP_NT / LANES, RPT = STEP_DK / RG;
    constexpr int NW = STEP_NT / 32;
    __shared__ A ks[STEP_DK], qs[STEP_GB][STEP_DK], vs[TC];
    __shared__ __align__(16) A red[STEP_GB][NW][TC];
    __shared__ int next;
    const int tid = threadIdx.x, h = blockIdx.y, c0 = blockIdx.z * TC;
    const int lane = tid % LANES, rg = tid / LANES, col = c0 + lane * VN;
    const bool in = col < P.dv;  // dv is a multiple of 8: a thread's columns are all in or all out
    int64_t row = blockIdx.x;
    int64_t slot = row;
    if (P.slot) slot = P.slot[row];
    const int G = P.hq / P.hkv;
    if (slot < 0 || slot >= P.slots) {  // no state: a row of zeros
        for (int g = 0; g < G; ++g)
            for (int c = c0 + tid; c < min(P.dv, c0 + TC); c += STEP_NT)
                static_cast<T*>(P.o)[row * P.o_ts + (int64_t)(h * G + g) * P.o_hs + c] = from_acc<T, A>((A)0);
        return;
    }
    A* st = static_cast<A*>(P.states) + ((slot * P.hkv + h) * P.dk) * (int64_t)P.dv + col;
    Pack<A, VN> S[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int i = r * RG + rg;
#pragma unroll
        for (int c = 0; c < VN; ++c) S[r].v[c] = 0;
        if (in && i < P.dk) S[r] = *reinterpret_cast<const Pack<A, VN>*>(st + (int64_t)i * P.dv);
    }
    const auto load_q = [&](int g0, int gn) {
        for (int i = tid; i < gn * STEP_DK; i += STEP_NT) {
            const int g = i / STEP_DK, c = i % STEP_DK;
            qs[g][c] = c < P.dk ? to_acc<A, T>(static_cast<const T*>(
                                      P.q.p)[row * P.q.ts + (int64_t)(h * G + g0 + g) * P.q.hs + c])
                                : (A)0;
        }
    };
    const auto load_kv = [&]() {
        for (int i = tid; i < STEP_DK; i += STEP_NT)
            ks[i] = i < P.dk ? to_acc<A, T>(static_cast<const T*>(P.k.p)[row * P.k.ts + (int64_t)h * P.k.hs + i]) : (A)0;
        for (int i = tid; i < TC; i += STEP_NT)
            vs[i] = c0 + i < P.dv ? to_acc<A, T>(static_cast<const T*>(P.v.p)[row * P.v.ts + (int64_t)h * P.v.hs + c0 + i])
                                  : (A)0;
    };
    // all loads of the row before the first barrier
    load_kv();
    load_q(0, min(STEP_GB, G));
    if (tid == 0) next = INT32_MAX;
    // Rows that name one slot are applied in row order: the first one's block
    // takes them all, the others leave.
    bool more = false;
    if (P.slot) {
        int earlier = 0, later = 0;
        for (int64_t m = tid; m < P.rows; m += STEP_NT) {
            const int same = P.slot[m] == (int32_t)slot;
            if (m < row) earlier |= same;
            if (m > row) later |= same;
        }
        if (__syncthreads_or(earlier)) return;
        more = __syncthreads_or(later);
    }
    // e^lam as a sum of two values: rounded once to fp32, its error would add
    // up over the tokens that a slow decay remembers
    const double g2 = decay((double)clamp_lam(static_cast<const A*>(P.lam)[h]), 1.0);
    const A ghi = (A)g2, glo = (A)(g2 - (double)ghi);
    const A scale = (A)P.scale;
    while (true) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const A kk = ks[r * RG + rg];
#pragma unroll
            for (int c = 0; c < VN; ++c)
                S[r].v[c] = dfma(ghi, S[r].v[c], dfma(glo, S[r].v[c], kk * vs[lane * VN + c]));
        }
        for (int g0 = 0; g0 < G; g0 += STEP_GB) {
            const int gn = min(STEP_GB, G - g0);
            if (g0 > 0) {
                load_q(g0, gn);
                __syncthreads();
            }
            for (int g = 0; g < gn; ++g) {
                A p[VN];
#pragma unroll
                for (int c = 0; c < VN; ++c) p[c] = 0;
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    const A qq = qs[g][r * RG + rg];
#pragma unroll
                    for (int c = 0; c < VN; ++c) p[c] = dfma(qq, S[r].v[c], p[c]);
                }
                if constexpr (LANES < 32) {  // the row groups inside the warp
#pragma unroll
                    for (int s = LANES; s < 32; s <<= 1)
#pragma unroll
                        for (int c = 0; c < VN; ++c) p[c] += __shfl_xor_sync(FULL, p[c], s);
                }
                if (tid % 32 < LANES) {
#pragma unroll
                    for (int c = 0; c < VN; ++c) red[g][tid / 32][lane * VN + c] = p[c];
                }
            }
            __syncthreads();
            for (int i = tid; i < gn * TC; i += STEP_NT) {
                const int g = i / TC, c = i % TC;
                A s = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w) s += red[g][w][c];
                if (c0 + c < P.dv)
                    static_cast<T*>(P.o)[row * P.o_ts + (int64_t)(h * G + g0 + g) * P.o_hs + c0 + c] =
                        from_acc<T, A>(s * scale);
            }
        }
        if (!more) break;
        int mine = INT32_MAX;
        for (int64_t m = row + 1 + tid; m < P.rows; m += STEP_NT)
            if (P.slot[m] == (int32_t)slot) { mine = (int)m; break; }
        if (!__syncthreads_or(mine != INT32_MAX)) break;
        if (mine != INT32_MAX) atomicMin(&next, mine);
        __syncthreads();
        row = next;
        __syncthreads();
        if (tid == 0) next = INT32_MAX;
        load_kv();
        load_q(0, min(STEP_GB, G));
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int i = r * RG + rg;
        if (in && i < P.dk) *reinterpret_cast<Pack<A, VN>*>(st + (int64_t)i * P.dv) = S[r];
    }
}

template <typename T>
static cudaError_t step_launch(const LinStep& P, cudaStream_t st) {
    using A = typename AccOf<T>::A;
    constexpr int VN = 16 / (int)sizeof(A);
    int dev = 0, sms = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const auto grid = [&](int lanes) {
        return dim3((unsigned)P.rows, (unsigned)P.hkv, (unsigned)((P.dv + lanes * VN - 1) / (lanes * VN)));
    };
    const dim3 g = grid(16);
    if ((int64_t)g.x * g.y * g.z >= 2 * sms) k_step<T, 16><<<g, STEP_NT, 0, st>>>(P);
    else k_step<T, 8><<<grid(8), STEP_NT, 0, st>>>(P);
    return cudaGetLastError();
}

cudaError_t step_run(laplex_dtype dt, const LinStep& P, cudaStream_t st) {
    if (P.rows == 0) return cudaSuccess;
    switch (dt) {
        case LAPLEX_F32: return step_launch<float>(P, st);
        case LAPLEX_F64: return step_launch<double>(P, st);
        case LAPLEX_F16: return step_launch<__half>(P, st);
        case LAPLEX_BF16: return step_launch<__nv_bfloat16>(P, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lx
