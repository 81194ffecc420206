// linattn_tc.cu -- decayed linear attention of 16-bit rows on the 5th-generation
// tensor cores.
//
// The recurrence S_t = e^lam S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, taken
// over chunks of 128 tokens, is four matrix products a chunk (rows t, s of the
// chunk, n of them valid; S the state before it):
//     P  = Q K^T                                  [128, 128]
//     O1 = (P .* scale e^{lam (t - s)} [s <= t]) V   [128, dv]
//     O2 = Q S,     o_t = O1_t + scale e^{lam (t + 1)} O2_t
//     U  = (K .* e^{lam (n - 1 - s)})^T V,  S <- e^{lam n} S + U   [dk, dv]
// and the reversed products (the gradients dk and dv) are the same with the
// mask s >= t, e^{lam (n - 1 - t)} before O2 and e^{lam s} inside U.
//
// A block of two warpgroups walks one segment of one head.  TMA boxes bring Q,
// K, V into swizzled tiles (K and V two stages ahead); one thread issues the
// products; all accumulators lie in tensor memory.  A thread owns a row: half of
// the columns of P (weighted, rounded once to the rows' type, and put back into
// tensor memory as the A operand of O1), of O1 and O2 (combined and stored), and
// of the state, which stays in fp32 registers and reaches shared memory rounded
// to the rows' type, for O2 alone.  K's weights are applied as a sum of two
// 16-bit values (hi in place, lo beside it), so that U, and the states that
// leave the call, carry 2^-17, not 2^-9.
//
// fp16: weights, states and weighted K are scaled by powers of two (per row, per
// state, per chunk) to 2^14..2^15 before they are rounded, so that nothing
// overflows and small ones do not sink below the type's normal range.
//
// Causality: a masked weight is 0, and 0 times a NaN or Inf of a later row of V
// would be NaN.  Each chunk's V is scanned (a few integer operations per 16
// bytes, while P runs); non-finite values are replaced by 0 and their products
// added by hand to the rows that they do reach.
//
// Bound by memory at full grids: a chunk of dk = dv = 128 moves 128 KB (2.8 us
// of an SM's share of the measured bandwidth) against 2560 cycles of tensor work.
#include <algorithm>
#include <atomic>

#include "devcache.h"
#include "elem.cuh"
#include "seqop.h"
#include "tc5.cuh"

namespace lx {

constexpr int TC_NT = 256;
constexpr int TC_C = 128;  // tokens per chunk
constexpr uint32_t TILE_BYTES = TC_C * 128;

struct TcRole {
    int mq, mk, mv;  // maps of the operands
    int nq, nk, dk, dv, reverse, transposed, in_by_slot, out_by_slot, skip_last;
    float sq, sk;
    const void* k;   // rows of k and v (for what a NaN or Inf reaches)
    int64_t k_ts, k_hs;
    const void* v;
    int64_t v_ts, v_hs;
    void* o;
    int64_t o_ts, o_hs;
    const float* state_in;
    float* state_out;
};

struct alignas(64) TcArgs {
    CUtensorMap map[4];
    LinSeqs S;
    int H, nroles;
    const float* lam;
    uint32_t* status;
    TcRole role[3];
};

// shared memory behind the tiles
struct TcShared {
    uint64_t kv_full[2], q_full, p_done, o2_done, o_done, u_done;
    uint32_t tmem;
    uint32_t bad[2][4];  // rows of V with a NaN or Inf, by parity of the load
    float wk[TC_C];      // weights of K's rows
    float rmax[2][TC_C]; // fp16: largest weight of a row, by half
    float red[2][8];     // fp16: block maxima
};

template <int DK, int DV, bool OUT> struct TcSize {
    static constexpr uint32_t KBY = DK / 64 * TILE_BYTES, VBY = DV / 64 * TILE_BYTES;
    static constexpr uint32_t SBY = DK * 128 * (DV / 64);
    static constexpr uint32_t K = 0, V = 2 * KBY, LO = V + 2 * VBY, S = LO + KBY, Q = S + (OUT ? SBY : 0);
    static constexpr uint32_t TILES = Q + (OUT ? KBY : 0);
    static constexpr uint32_t BYTES = TILES + sizeof(TcShared);
    // tensor memory columns: P (whose first half then holds the rounded weights), O1, O2, U
    static constexpr uint32_t P = 0, O1 = 128, O2 = 128 + DV, U = !OUT ? 0 : DV == 64 ? 64 : 128 + 2 * DV;
    static constexpr uint32_t COLS = !OUT ? DV : DV == 64 ? 256 : 512;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// two values to 16 bits, the first in the low half
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// the power of two that brings a largest magnitude m to [2^14, 2^15) (1 for 0, Inf and NaN)
__device__ __forceinline__ float scale_to_fp16(float m) {
    if (!(m > 0.0f) || m > 3.0e38f) return 1.0f;
    const int e = (int)(__float_as_uint(m) >> 23) - 127;
    return __uint_as_float((uint32_t)(127 + 14 - max(e, -100)) << 23);
}

template <typename T, int DK, int DV, bool OUT>
__global__ void __launch_bounds__(TC_NT, 1) k_lin_tc(const __grid_constant__ TcArgs A) {
    using Z = TcSize<DK, DV, OUT>;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    constexpr int HV = DV / 2;  // state and output columns of a thread
    extern __shared__ __align__(1024) unsigned char sm[];
    TcShared& sh = *reinterpret_cast<TcShared*>(sm + Z::TILES);
    const TcRole& R = A.role[blockIdx.x % A.nroles];
    const int slot = blockIdx.x / A.nroles, h = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    int seq, len;
    int64_t t0;
    if (!A.S.find(slot, &seq, &t0, &len)) return;
    const bool rev = R.reverse;
    if (!OUT && R.skip_last && (rev ? t0 == A.S.at(seq) : t0 + len == A.S.at(seq + 1))) return;

    if (smem_u32(sm) & 1023u) {  // the swizzle goes by address bits: the tiles must start on 1024 bytes
        if (tid == 0) set_status(A.status, ST_TIMEOUT);
        return;
    }
    if (tid == 0) {
        mbar_init(&sh.kv_full[0], 1);
        mbar_init(&sh.kv_full[1], 1);
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.p_done, 1);
        mbar_init(&sh.o2_done, 1);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.u_done, 1);
        fence_proxy_async();
    }
    __syncwarp();
    if (warp == 0) tmem_alloc(&sh.tmem, Z::COLS);
    if (tid < 8) sh.bad[tid >> 2][tid & 3] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh.tmem;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t smb = smem_u32(sm);

    const int nch = (len + TC_C - 1) / TC_C;
    const int nq = R.nq, nk = R.nk, G = max(nq, nk);
    const int n_kv = nch * nk, n_q = OUT ? nch * nq : 0;
    const auto chunk_at = [&](int c, int* n) -> int64_t {
        if (!rev) {
            *n = min(TC_C, len - c * TC_C);
            return t0 + (int64_t)c * TC_C;
        }
        const int end = len - c * TC_C, a = max(end - TC_C, 0);
        *n = end - a;
        return t0 + a;
    };
    const auto load_kv = [&](int i) {
        if (i >= n_kv) return;
        int n;
        const int64_t a = chunk_at(i / nk, &n);
        const int head = h * nk + i % nk;
        uint64_t* bar = &sh.kv_full[i & 1];
        mbar_expect_tx(bar, Z::KBY + Z::VBY);
        for (int b = 0; b < DK / 64; ++b)
            tma_load3(sm + Z::K + (i & 1) * Z::KBY + b * TILE_BYTES, &A.map[R.mk], b * 64, head, (int)a, bar);
        for (int b = 0; b < DV / 64; ++b)
            tma_load3(sm + Z::V + (i & 1) * Z::VBY + b * TILE_BYTES, &A.map[R.mv], b * 64, head, (int)a, bar);
    };
    const auto load_q = [&](int i) {
        if (i >= n_q) return;
        int n;
        const int64_t a = chunk_at(i / nq, &n);
        mbar_expect_tx(&sh.q_full, Z::KBY);
        for (int b = 0; b < DK / 64; ++b)
            tma_load3(sm + Z::Q + b * TILE_BYTES, &A.map[R.mq], b * 64, h * nq + i % nq, (int)a, &sh.q_full);
    };
    if (tid == 0) {
        load_kv(0);
        if (OUT) load_q(0);
        load_kv(1);
    }

    const float l2 = clamp_lam(A.lam[h]) * 1.44269504088896341f;
    float pw[8];  // e^{lam j}, in the order of a row's columns
#pragma unroll
    for (int j = 0; j < 8; ++j) pw[j] = ex2(l2 * (float)(rev ? j : 7 - j));
    const float ssk = R.sq * R.sk;
    // reversed: K carries e^{lam s}, and U the e^lam that leads out of the chunk,
    // so that the largest of K's weights is 1 (fp16: a fast decay would sink all)
    const float u_out = rev ? exp2f(l2) : 1.0f;

    float S[HV];  // the state: row `row` of dk, columns wg * HV ...
#pragma unroll
    for (int c = 0; c < HV; ++c) S[c] = 0.0f;
    const int64_t by_slot = (int64_t)slot * A.H + h, by_seq = (int64_t)seq * A.H + h;
    const int64_t ri = R.transposed ? 1 : R.dv, ci = R.transposed ? R.dk : 1;
    bool has_state = R.state_in != nullptr;
    if (has_state && row < R.dk) {
        const float* p = R.state_in + (R.in_by_slot ? by_slot : by_seq) * R.dk * R.dv + row * ri;
#pragma unroll
        for (int c = 0; c < HV; ++c)
            if (wg * HV + c < R.dv) S[c] = p[(wg * HV + c) * ci];
    }
    float s_inv = 1.0f;  // the rounded state is the state / s_inv
    // the state, rounded, into shared memory as the B operand of O2 (by all threads)
    const auto store_state = [&]() {
        float up = 1.0f;
        if constexpr (!BF) {
            float m = 0.0f;
#pragma unroll
            for (int c = 0; c < HV; ++c) m = fmaxf(m, fabsf(S[c]));
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, s));
            if (lane == 0) sh.red[1][warp] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 8; ++w) m = fmaxf(m, sh.red[1][w]);
            up = scale_to_fp16(m);
            s_inv = 1.0f / up;
        }
        if (row < DK) {
#pragma unroll
            for (int u = 0; u < HV / 8; ++u) {
                uint4 w;
                uint32_t* q = &w.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = pack2<T>(S[u * 8 + 2 * e] * up, S[u * 8 + 2 * e + 1] * up);
                const int col = wg * HV + u * 8;
                *reinterpret_cast<uint4*>(sm + Z::S + (col >> 6) * (DK * 128) + tile_at(row, (col & 63) >> 3)) = w;
            }
        }
        fence_proxy_async();
    };
    if (OUT && has_state) store_state();

    bool ok = true;
    int wk_n = -1;       // tokens that the weights of K were made for
    float k_inv = 1.0f;  // fp16: the weighted K is K / k_inv
    float oacc[!BF && OUT ? HV : 1];
    bool stop = false;
    uint32_t item = 0, u_count = 0;
    for (int c = 0; c < nch && !stop; ++c) {
        int n;
        const int64_t a = chunk_at(c, &n);
        const float wq = R.sq * exp2f(l2 * (float)(rev ? n - 1 - row : row + 1));
        const float whole = exp2f(l2 * (float)n);
        for (int i = 0; i < G; ++i, ++item) {
            const int kv = c * nk + (nk > 1 ? i : 0), qi = c * nq + (nq > 1 ? i : 0);
            const bool new_kv = i == 0 || nk > 1, new_q = i == 0 || nq > 1;
            const bool last = i == G - 1;
            const bool conv = nk > 1 || last;        // K is needed no more: weigh it
            const bool emit = nq > 1 || last;        // O1 is whole
            unsigned char* Ks = sm + Z::K + (kv & 1) * Z::KBY;
            unsigned char* Vs = sm + Z::V + (kv & 1) * Z::VBY;
            const uint32_t Ka = smb + Z::K + (kv & 1) * Z::KBY, Va = smb + Z::V + (kv & 1) * Z::VBY;
            if (new_kv) ok &= mbar_wait(&sh.kv_full[kv & 1], (uint32_t)(kv >> 1) & 1);
            if (OUT && new_q) ok &= mbar_wait(&sh.q_full, (uint32_t)qi & 1);
            tc_fence_before();
            if (__syncthreads_or(!ok)) {
                stop = true;
                break;
            }
            if (OUT && tid == 0) {
                tc_fence_after();
                constexpr uint32_t id = mma_desc(BF, false, false, 128, 128);
#pragma unroll
                for (int s = 0; s < DK / 16; ++s) {
                    const uint32_t off = (s >> 2) * TILE_BYTES + (s & 3) * 32;
                    mma_ss(tm + Z::P, tile_desc(smb + Z::Q + off, 16, 1024), tile_desc(Ka + off, 16, 1024), id, s > 0);
                }
                mma_commit(&sh.p_done);
                if (new_q) {
                    if (has_state) {
                        constexpr uint32_t id2 = mma_desc(BF, false, true, 128, DV);
#pragma unroll
                        for (int s = 0; s < DK / 16; ++s) {
                            const uint32_t off = (s >> 2) * TILE_BYTES + (s & 3) * 32;
                            mma_ss(tm + Z::O2, tile_desc(smb + Z::Q + off, 16, 1024),
                                   tile_desc(smb + Z::S + s * 2048, DK * 128, 1024), id2, s > 0);
                        }
                    }
                    mma_commit(&sh.o2_done);
                }
            }
            if (wk_n != n) {  // (the last chunk's are read no more: all threads have passed the barrier above)
                wk_n = n;
                if (tid < TC_C) sh.wk[tid] = tid < n ? R.sk * exp2f(l2 * (float)(rev ? tid : n - 1 - tid)) : 0.0f;
            }
            if (new_kv) {
                // V: rows past the chunk's tokens become 0, and so do NaN and Inf
                if (tid < 4) sh.bad[(kv + 1) & 1][tid] = 0;
                constexpr uint32_t ONE = BF ? 0x00800080u : 0x04000400u;
#pragma unroll
                for (int x = 0; x < DV / 64 * 4; ++x) {
                    const int u = x * TC_NT + tid, r = (u >> 3) & 127, b = u >> 10;
                    uint4* p = reinterpret_cast<uint4*>(Vs + b * TILE_BYTES + tile_at(r, u & 7));
                    if (r >= n) {
                        *p = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 w = *p;
                    const uint32_t any = ((w.x & 0x7fff7fffu) + ONE) | ((w.y & 0x7fff7fffu) + ONE) |
                                         ((w.z & 0x7fff7fffu) + ONE) | ((w.w & 0x7fff7fffu) + ONE);
                    if (OUT && (any & 0x80008000u)) {
                        atomicOr(&sh.bad[kv & 1][r >> 5], 1u << (r & 31));
                        uint32_t* q = &w.x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t t = (q[e] & 0x7fff7fffu) + ONE;
                            q[e] &= (t & 0x8000u ? 0u : 0xffffu) | (t & 0x80000000u ? 0u : 0xffff0000u);
                        }
                        *p = w;
                    }
                }
                if constexpr (!BF) {
                    uint32_t m = 0;
#pragma unroll
                    for (int x = 0; x < DK / 64 * 4; ++x) {
                        const int u = x * TC_NT + tid, r = (u >> 3) & 127, b = u >> 10;
                        if (r >= n) continue;
                        const uint4 w = *reinterpret_cast<const uint4*>(Ks + b * TILE_BYTES + tile_at(r, u & 7));
                        m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                                 __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
                    }
                    m = max(m & 0xffffu, m >> 16);
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(FULL, m, s));
                    if (lane == 0) sh.red[0][warp] = __half2float(__ushort_as_half((unsigned short)m));
                }
            }
            uint32_t pk[32];       // the weights, rounded, two a word
            float pf[BF ? 1 : 64];  // fp16: before they are rounded
            float p_inv = 1.0f;
            if constexpr (OUT) {
                ok &= mbar_wait(&sh.p_done, item & 1);
                tc_fence_after();
                const int tw = (warp & 3) * 32;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t r[32];
                    const int base = wg * 64 + half * 32;
                    tmem_ld32(tm + lanes + Z::P + base, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int s0 = base + b * 8;
                        float w[8];
                        const bool none = rev ? s0 + 7 < tw || s0 >= n : s0 > tw + 31;
                        const bool all = rev ? s0 >= tw + 31 && s0 + 8 <= n : s0 + 7 <= tw;
                        if (none) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = 0.0f;
                        } else if (all) {
                            const float f = ssk * ex2(l2 * (float)(rev ? s0 - row : row - s0 - 7));
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = __uint_as_float(r[b * 8 + j]) * (f * pw[j]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int s = s0 + j, d = rev ? s - row : row - s;
                                w[j] = d >= 0 && s < n ? __uint_as_float(r[b * 8 + j]) * (ssk * ex2(l2 * (float)d)) : 0.0f;
                            }
                        }
                        if constexpr (BF) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) pk[half * 16 + b * 4 + j] = pack2<T>(w[2 * j], w[2 * j + 1]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) pf[half * 32 + b * 8 + j] = w[j];
                        }
                    }
                }
                if constexpr (!BF) {
                    float m = 0.0f;
#pragma unroll
                    for (int j = 0; j < 64; ++j) m = fmaxf(m, fabsf(pf[j]));
                    sh.rmax[wg][row] = m;
                }
                tc_fence_before();
            }
            __syncthreads();  // all of P is read (its columns take the rounded weights), block maxima are there
            if constexpr (OUT) {
                if constexpr (!BF) {
                    const float up = scale_to_fp16(fmaxf(sh.rmax[0][row], sh.rmax[1][row]));
                    p_inv = 1.0f / up;
#pragma unroll
                    for (int j = 0; j < 32; ++j) pk[j] = pack2<T>(pf[2 * j] * up, pf[2 * j + 1] * up);
                }
                tc_fence_after();
                tmem_st32(tm + lanes + Z::P + wg * 32, pk);
                tmem_wait_st();
            }
            if (conv) {
                float k_up = 1.0f;
                if constexpr (!BF) {
                    float m = 0.0f;
#pragma unroll
                    for (int w = 0; w < 8; ++w) m = fmaxf(m, sh.red[0][w]);
                    k_up = scale_to_fp16(m * fabsf(R.sk));
                    k_inv = 1.0f / k_up;
                }
#pragma unroll
                for (int x = 0; x < DK / 64 * 4; ++x) {
                    const int u = x * TC_NT + tid, r = (u >> 3) & 127, b = u >> 10;
                    const uint32_t at = b * TILE_BYTES + tile_at(r, u & 7);
                    uint4 w = *reinterpret_cast<const uint4*>(Ks + at), hi, lo;
                    const float f = sh.wk[r] * k_up;
                    const uint32_t* q = &w.x;
                    uint32_t *qh = &hi.x, *ql = &lo.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 v = unpack2<T>(q[e]);
                        v.x *= f;
                        v.y *= f;
                        qh[e] = pack2<T>(v.x, v.y);
                        const float2 g = unpack2<T>(qh[e]);
                        float2 d = make_float2(v.x - g.x, v.y - g.y);
                        d.x = d.x == d.x ? d.x : 0.0f;  // Inf - Inf: the upper part says it
                        d.y = d.y == d.y ? d.y : 0.0f;
                        ql[e] = pack2<T>(d.x, d.y);
                    }
                    if (r >= n) hi = lo = make_uint4(0, 0, 0, 0);  // not 0 * NaN
                    *reinterpret_cast<uint4*>(Ks + at) = hi;
                    *reinterpret_cast<uint4*>(sm + Z::LO + at) = lo;
                }
            }
            fence_proxy_async();  // V, K and its lower part are read by the products
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                if constexpr (OUT) {
                    constexpr uint32_t id = mma_desc(BF, false, true, 128, DV);
                    const bool more = BF && nk > 1 && i > 0;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_ts(tm + Z::O1, tm + Z::P + s * 8, tile_desc(Va + s * 2048, TILE_BYTES, 1024), id, more || s > 0);
                    mma_commit(&sh.o_done);
                }
                if (conv) {
                    // dk = 64: M stays 128, the second half repeats the first (leading offset 0) and is not read
                    constexpr uint32_t id = mma_desc(BF, true, true, 128, DV), lead = DK == 64 ? 0 : TILE_BYTES;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_ss(tm + Z::U, tile_desc(Ka + s * 2048, lead, 1024), tile_desc(Va + s * 2048, TILE_BYTES, 1024),
                               id, s > 0);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_ss(tm + Z::U, tile_desc(smb + Z::LO + s * 2048, lead, 1024),
                               tile_desc(Va + s * 2048, TILE_BYTES, 1024), id, true);
                    mma_commit(&sh.u_done);
                }
            }
            const bool patch = OUT && (sh.bad[kv & 1][0] | sh.bad[kv & 1][1] | sh.bad[kv & 1][2] | sh.bad[kv & 1][3]);
            if constexpr (OUT) {
                ok &= mbar_wait(&sh.o_done, item & 1);
                if (new_q) ok &= mbar_wait(&sh.o2_done, (uint32_t)qi & 1);
                tc_fence_after();
                if (emit && tid == 0) load_q(qi + 1);  // P and O2 have read Q
                T* out = static_cast<T*>(R.o) + (a + row) * R.o_ts + (int64_t)(h * nq + (nq > 1 ? i : 0)) * R.o_hs;
#pragma unroll
                for (int cb = 0; cb < HV; cb += 32) {
                    if (BF && !emit && !patch) continue;  // the sum goes on in tensor memory
                    uint32_t r1[32];
                    __syncwarp();
                    tmem_ld32(tm + lanes + Z::O1 + wg * HV + cb, r1);
                    tmem_wait_ld();
                    if constexpr (!BF) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float v = __uint_as_float(r1[j]) * p_inv;
                            oacc[cb + j] = nk > 1 && i > 0 ? oacc[cb + j] + v : v;
                            r1[j] = __float_as_uint(oacc[cb + j]);
                        }
                    }
                    if (patch) {
                        // + weight (t, s) v_s where v_s is not finite and s reaches t; weights as O1 took them
#pragma unroll 1
                        for (int s = 0; s < n; ++s) {
                            if (!(sh.bad[kv & 1][s >> 5] >> (s & 31) & 1)) continue;
                            __syncwarp();
                            const uint32_t w2 = tmem_ld1(tm + lanes + Z::P + (s >> 1));
                            tmem_wait_ld();
                            const float2 wp = unpack2<T>(w2);
                            const float w = (s & 1 ? wp.y : wp.x) * p_inv;
                            if (rev ? s < row : s > row) continue;
                            const T* vr = static_cast<const T*>(R.v) + (a + s) * R.v_ts +
                                          (int64_t)(h * nk + (nk > 1 ? i : 0)) * R.v_hs + wg * HV + cb;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                if (wg * HV + cb + j >= R.dv) break;
                                const float v = to_acc<float, T>(vr[j]);
                                if (!(fabsf(v) <= 3.0e38f)) r1[j] = __float_as_uint(__uint_as_float(r1[j]) + w * v);
                            }
                        }
                        if constexpr (!BF) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) oacc[cb + j] = __uint_as_float(r1[j]);
                        } else if (!emit) {
                            __syncwarp();
                            tmem_st32(tm + lanes + Z::O1 + wg * HV + cb, r1);
                            tmem_wait_st();
                        }
                    }
                    if (emit) {
                        uint32_t r2[32];
                        if (has_state) {
                            __syncwarp();
                            tmem_ld32(tm + lanes + Z::O2 + wg * HV + cb, r2);
                            tmem_wait_ld();
                        }
                        if (row < n) {
                            const float w2 = wq * s_inv;
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                if (wg * HV + cb + u * 8 >= R.dv) break;
                                uint4 w;
                                uint32_t* q = &w.x;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int j = u * 8 + 2 * e;
                                    float x = __uint_as_float(r1[j]), y = __uint_as_float(r1[j + 1]);
                                    if (has_state) {
                                        x = fmaf(w2, __uint_as_float(r2[j]), x);
                                        y = fmaf(w2, __uint_as_float(r2[j + 1]), y);
                                    }
                                    q[e] = pack2<T>(x, y);
                                }
                                *reinterpret_cast<uint4*>(out + wg * HV + cb + u * 8) = w;
                            }
                        }
                    }
                }
            }
            if (conv) {
                ok &= mbar_wait(&sh.u_done, u_count & 1);
                ++u_count;
                tc_fence_after();
                if (tid == 0) load_kv(kv + 2);  // O1 and U have read K and V
                const float d = nk > 1 && i > 0 ? 1.0f : whole, us = BF ? u_out : u_out * k_inv;
#pragma unroll
                for (int cb = 0; cb < HV; cb += 32) {
                    uint32_t r[32];
                    __syncwarp();
                    tmem_ld32(tm + lanes + Z::U + wg * HV + cb, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        S[cb + j] = fmaf(d, S[cb + j], us * __uint_as_float(r[j]));
                    }
                }
                if (patch && row < R.dk) {
#pragma unroll 1
                    for (int s = 0; s < n; ++s) {
                        if (!(sh.bad[kv & 1][s >> 5] >> (s & 31) & 1)) continue;
                        const int64_t head = h * nk + (nk > 1 ? i : 0);
                        const float kw = u_out * sh.wk[s] * to_acc<float, T>(static_cast<const T*>(R.k)[(a + s) * R.k_ts + head * R.k_hs + row]);
                        const T* vr = static_cast<const T*>(R.v) + (a + s) * R.v_ts + head * R.v_hs + wg * HV;
#pragma unroll
                        for (int j = 0; j < HV; ++j) {
                            if (wg * HV + j >= R.dv) break;
                            const float v = to_acc<float, T>(vr[j]);
                            if (!(fabsf(v) <= 3.0e38f)) S[j] = fmaf(kw, v, S[j]);
                        }
                    }
                }
                if (last) {
                    has_state = true;
                    if (OUT && c + 1 < nch) store_state();
                }
            }
        }
    }
    if (!ok || stop) {
        // a copy or a product did not come: report it, and let the copies in flight land
        if (tid == 0) {
            set_status(A.status, ST_TIMEOUT);
            mbar_wait(&sh.kv_full[0], 0);
            mbar_wait(&sh.kv_full[1], 0);
            mbar_wait(&sh.q_full, 0);
        }
    } else if (R.state_out && row < R.dk) {
        float* p = R.state_out + (R.out_by_slot ? by_slot : by_seq) * R.dk * R.dv + row * ri;
#pragma unroll
        for (int c = 0; c < HV; ++c)
            if (wg * HV + c < R.dv) p[(wg * HV + c) * ci] = S[c];
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free(tm, Z::COLS);
    }
}

// ---------------------------------------------------------------- host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_fn() {
    static std::atomic<void*> cache{nullptr};
    void* f = cache.load(std::memory_order_relaxed);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        cache.store(f, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// boxes of [128 tokens][one head][64 values]; values past dim and tokens past T read as 0
static cudaError_t encode(CUtensorMap* m, laplex_dtype dt, const LinRows& x, int dim, int heads, int64_t T) {
    EncodeTiled f = encode_fn();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)x.hs * 2, (cuuint64_t)x.ts * 2};
    const cuuint32_t box[3] = {64, 1, TC_C}, es[3] = {1, 1, 1};
    const CUresult r = f(m, dt == LAPLEX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(x.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tokens per segment (a multiple of 128).  A block takes an SM, so a launch of
// `roles` products runs ceil(blocks / 148) rounds of one segment each; a cut
// adds the state pass (about half of a product's time, over all but each
// sequence's last segment) and two launches.  Sequences of one known length take
// the cheapest number of cuts by that count.  Lengths that only the device knows:
// pieces for two rounds where the heads do not fill the GPU, else only sequences
// four times longer than the mean are cut.
int tc_segment(int64_t T, int N, int H, int roles, bool equal) {
    const int64_t whole = std::min<int64_t>(std::max<int64_t>(T, 1) + 1, INT32_MAX);
    if (N == 0 || T == 0) return (int)whole;
    constexpr int64_t SMS = 148;
    const auto up = [](int64_t x) { return (x + TC_C - 1) / TC_C * TC_C; };
    const int64_t heads = (int64_t)N * H;
    int64_t seg;
    if (equal) {
        const int64_t L = T / N;
        double best = 0;
        seg = whole;
        for (int64_t m = 1; m <= 512 && (m == 1 || L / m >= 2 * TC_C); ++m) {
            const int64_t s = up((L + m - 1) / m), pieces = (L + s - 1) / s;
            const double rounds = (double)((heads * pieces * roles + SMS - 1) / SMS);
            const double state = (double)((heads * (pieces - 1) + SMS - 1) / SMS) * (roles > 1 ? 2 : 1);
            const double cost = rounds * s + (m > 1 ? 0.5 * state * s + 400.0 : 0.0);
            if (m == 1 || cost < best) {
                best = cost;
                seg = m == 1 ? whole : s;
            }
        }
        return (int)seg;
    }
    if (heads < SMS) seg = std::max<int64_t>(512, up(T * H / (2 * SMS)));
    else seg = std::max<int64_t>(2048, up(4 * T / N));
    return (int)(seg >= T ? whole : seg);
}

template <typename T, int DK, int DV, bool OUT>
static cudaError_t tc_launch(const TcArgs& A, cudaStream_t st) {
    constexpr auto kern = k_lin_tc<T, DK, DV, OUT>;
    constexpr size_t smem = TcSize<DK, DV, OUT>::BYTES;
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e == cudaSuccess) e = blocks_per_sm<kern>(dev, TC_NT, smem, &per);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(A.S.slots * A.nroles), (unsigned)A.H);
    if (grid.x == 0) return cudaSuccess;
    kern<<<grid, TC_NT, smem, st>>>(A);
    return cudaGetLastError();
}

template <typename T, bool OUT>
static cudaError_t tc_dims(const TcArgs& A, int dk, int dv, cudaStream_t st) {
    if (dk <= 64) return dv <= 64 ? tc_launch<T, 64, 64, OUT>(A, st) : tc_launch<T, 64, 128, OUT>(A, st);
    return dv <= 64 ? tc_launch<T, 128, 64, OUT>(A, st) : tc_launch<T, 128, 128, OUT>(A, st);
}

cudaError_t tc_run(laplex_dtype dt, const LinRole* roles, int count, const LinSeqs& S, int H, const void* lam,
                   bool state_only, uint32_t* status, cudaStream_t st) {
    // roles of one padded shape share a launch (they read the same rows at about the same time)
    const auto pad = [](int d) { return d <= 64 ? 64 : 128; };
    bool done[3] = {false, false, false};
    for (int i = 0; i < count; ++i) {
        if (done[i]) continue;
        TcArgs A = {};
        A.S = S;
        A.H = H;
        A.lam = static_cast<const float*>(lam);
        A.status = status;
        struct { LinRows x; int dim, heads; } key[4];
        int maps = 0;
        for (int j = i; j < count; ++j) {
            const LinRole& L = roles[j];
            if (done[j] || pad(L.dk) != pad(roles[i].dk) || pad(L.dv) != pad(roles[i].dv)) continue;
            done[j] = true;
            TcRole& R = A.role[A.nroles++];
            const auto map_of = [&](const LinRows& x, int dim, int heads, int* m) -> cudaError_t {
                for (*m = 0; *m < maps; ++*m)
                    if (key[*m].x.p == x.p && key[*m].x.ts == x.ts && key[*m].x.hs == x.hs && key[*m].dim == dim &&
                        key[*m].heads == heads)
                        return cudaSuccess;
                if (maps == 4) return cudaErrorInvalidValue;
                key[maps++] = {x, dim, heads};
                return S.T > 0 ? encode(&A.map[*m], dt, x, dim, heads, S.T) : cudaSuccess;
            };
            cudaError_t e = state_only ? cudaSuccess : map_of(L.q, L.dk, H * L.nq, &R.mq);
            if (e == cudaSuccess) e = map_of(L.k, L.dk, H * L.nk, &R.mk);
            if (e == cudaSuccess) e = map_of(L.v, L.dv, H * L.nk, &R.mv);
            if (e != cudaSuccess) return e;
            R.nq = L.nq;
            R.nk = L.nk;
            R.dk = L.dk;
            R.dv = L.dv;
            R.reverse = L.reverse;
            R.transposed = L.transposed;
            R.in_by_slot = L.in_by_slot;
            R.out_by_slot = L.out_by_slot;
            R.skip_last = L.skip_last;
            R.sq = (float)L.sq;
            R.sk = (float)L.sk;
            R.k = L.k.p;
            R.k_ts = L.k.ts;
            R.k_hs = L.k.hs;
            R.v = L.v.p;
            R.v_ts = L.v.ts;
            R.v_hs = L.v.hs;
            R.o = L.o;
            R.o_ts = L.o_ts;
            R.o_hs = L.o_hs;
            R.state_in = static_cast<const float*>(L.state_in);
            R.state_out = static_cast<float*>(L.state_out);
        }
        const int dk = roles[i].dk, dv = roles[i].dv;
        cudaError_t e;
        if (dt == LAPLEX_BF16)
            e = state_only ? tc_dims<__nv_bfloat16, false>(A, dk, dv, st) : tc_dims<__nv_bfloat16, true>(A, dk, dv, st);
        else
            e = state_only ? tc_dims<__half, false>(A, dk, dv, st) : tc_dims<__half, true>(A, dk, dv, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace lx
