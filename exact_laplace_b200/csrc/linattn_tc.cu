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
// A block walks one segment of one head.  TMA boxes bring Q, K, V into swizzled
// tiles (K and V two chunks ahead); all accumulators lie in tensor memory.  Three
// kinds of warps work at the same time and meet at mbarriers:
//   issue (one warp):  the copies and the products, from one thread;
//   state (8 warps):   V's scan, K's weights, the state.  The state is U's
//                      accumulator in tensor memory (fp32): once a chunk each
//                      thread reads half a row of it, writes it, rounded to the
//                      rows' type, to shared memory (for O2 alone) and scales it
//                      by the next chunk's e^{lam n}, on which the next U adds.
//                      K is weighed as a sum of two 16-bit values (hi in place,
//                      lo beside it), so that U carries 2^-17, not 2^-9;
//   rows (8 warps):    P's weights, rounded once to the rows' type and put back
//                      into tensor memory as the A operand of O1, and the outputs.
// One group of 8 warps that did all of this in turn took 8.9 us a chunk of
// dk = dv = 128 (issue slots 21 % busy, the rest latencies of the chain).  The
// tiles leave hardly any L1: a spilled register is a trip to L2, so nothing is
// kept in registers from chunk to chunk, and the loops over columns are not unrolled.
//
// States that leave the call, and those at the starts of segments, come from a
// second kernel, the state pass: U alone, over chunks of 64 tokens, each chunk's
// added to the state in fp32 registers.  (Sums in tensor memory are cut off, not
// rounded, at each product: 3e-8 of the sum each, always downwards, 1e-5 over the
// 300 products that a slow decay remembers.)  There K's weights come from fp32
// products, for bf16 in three parts, where the state is a result.
//
// fp16: weights, states and weighted K are scaled by powers of two (per row, per
// state, per chunk) to 2^14..2^15 before they are rounded, so that nothing
// overflows and small ones do not sink below the type's normal range.
//
// Causality: a masked weight is 0, and 0 times a NaN or Inf of a later row of V
// is NaN in O1.  A warp that finds an output not finite although its O2 is takes
// that output from the definition (repair).  The state may keep the NaN: V's
// token is in it.  (A scan of V before its use cost a read of the tile from
// shared memory, whose bandwidth the products need.)
//
// Bounds of a chunk of dk = dv = 128: 128 KB of device memory (2.8 us of an SM's
// share of the measured bandwidth), 2560 cycles of tensor work, by count about 5000
// cycles of shared memory (operands of the products 2300, copies 770, K's parts 770,
// the state 256, outputs, tables).  A chunk takes about 8000, and nothing is
// saturated (32768 tokens, 16 heads: DRAM 46 %, tensor pipe 32 %, issue 40 %, the
// warps' shared accesses 23 %; fp16, four q-heads: 21, 21, 37 and 10 %): what bounds
// it is the chain P, weights, O1, outputs of one item after another, with one buffer
// of each.
//
// Rounding to 16 bits: P's weights and the state that O2 reads, once each, because a
// product of the tensor cores takes 16-bit operands (a second part of each would cost
// half as many products again and 32 KB that the tiles do not leave at 128 x 128).
// Independent roundings add in the mean square, so an output is off by about sqrt(2)
// times its own rounding: rms 2.3e-3 in bf16 and 2.9e-4 in fp16, against 1.65e-3 and
// 2.1e-4 of an output rounded once.  Rows given in fp32 take linattn_rec.cu, which
// rounds neither.
#include <algorithm>
#include <atomic>

#include "devcache.h"
#include "elem.cuh"
#include "seqop.h"
#include "tc5.cuh"

namespace lx {

constexpr int TC_GROUP = 256;  // threads of the state warps, and of the rows warps
constexpr int TC_C = 128;  // tokens per chunk
constexpr int WORK_REGS = 104, ISSUE_REGS = 64;  // a thread's registers in the products kernel

struct TcRole {
    int mq, mk, mv;  // maps of the operands
    int nq, nk, dk, dv, reverse, transposed, in_by_slot, out_by_slot, skip_last;
    int exact;       // state pass: the state is a result, not only rounded for O2
    float sq, sk;
    const void* q;   // rows of q, k and v (for repair)
    int64_t q_ts, q_hs;
    const void* k;
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
    uint32_t polls;    // bound of each wait
    int force_expiry;  // test hook: every block's first copy of K and V is never issued
    TcRole role[3];
};

// shared memory behind the tiles
struct TcShared {
    uint64_t kv_full[2], q_full;             // copies
    // A waiter names a phase by its parity, so no barrier may run two phases ahead of one of
    // its waiters.  (p_done is waited for by the rows warps at every item; k_free says the same
    // to the state warps where they weigh K; v_ready, k_ready and u_done run one load ahead: two of each.)
    uint64_t p_done, k_free, o2_done, o_done, u_done[2];  // products
    uint64_t v_ready[2], k_ready[2], s_ready;          // from the state warps
    uint64_t p_ready, o_read;                          // from the rows warps
    uint64_t k_max, s_max, p_max[4];                   // fp16: maxima exchanged among the state warps, in a pair of rows warps
    uint64_t drain;      // after a wait that ran out
    int kv_phase[2], q_phase;  // the last phase of kv_full and q_full whose copies were issued, or -1
    uint32_t tmem;
    uint32_t dead;       // a wait ran out
    alignas(16) float grow[16];  // e^{lam j}, 16 columns of P towards the row's end
    float wt[TC_C + 32]; // P's weights scale e^{lam |x|} at 32 + x (reversed: 127 + x), x = row - column; 0 up to 31 past the diagonal
    union {                // K's weights g1 e^{lam d}, d >= 0
        float dec[TC_C];   // in fp32 (exact)
        uint2 dec2[TC_C];  // as sums of two 16-bit values, each twice
    };
    float s_inv[2];      // fp16: what the rounded state is to be multiplied by, by chunk
    uint8_t rexp[2][2][TC_C];  // fp16: the exponent of a row's largest weight, by item and half
    float red[3][8];     // fp16: maxima of the state warps: of K, by load, and of the state
};

// Products: chunks of 128 tokens.  The state pass takes 64, with two blocks on an SM: it only
// streams K and V, and one block with two stages of 128 left the copies' latency (about 3500
// cycles under load) in the open.
template <int DK, int DV, bool OUT> struct TcSize {
    static constexpr int CH = OUT ? 128 : 64, STAGES = 2, BLOCKS = OUT ? 1 : 2;
    static constexpr uint32_t TB = CH * 128;  // bytes of a tile of 64 columns
    static constexpr uint32_t KBY = DK / 64 * TB, VBY = DV / 64 * TB;
    // LO: K's second part.  S: the rounded state; in the state pass K's third part, or a second buffer
    // of the second.
    static constexpr uint32_t SBY = OUT ? DK * 128 * (DV / 64) : KBY;
    static constexpr uint32_t K = 0, V = STAGES * KBY, LO = V + STAGES * VBY, S = LO + KBY, Q = S + SBY;
    static constexpr uint32_t TILES = Q + (OUT ? KBY : 0);
    static constexpr uint32_t BYTES = TILES + sizeof(TcShared);
    // tensor memory columns: P, O1, O2, U.  The rounded weights of P's columns 0-63
    // take columns 0-31, those of 64-127 columns 64-95: each warp writes over what it alone read.
    // The state pass: U and, behind it, the state.
    static constexpr uint32_t P = 0, O1 = 128, O2 = 256, U = OUT ? 384 : 0;
    static constexpr uint32_t COLS = OUT ? 512 : 2 * DV;
    // the issuing warp brings three idle ones: registers are moved between groups of four warps
    static constexpr int NT = OUT ? 2 * TC_GROUP + 128 : TC_GROUP + 32;
};

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

// the power of two that brings a largest magnitude m to [2^14, 2^15) (2^100 for less
// than 2^-86; 1 for Inf and NaN)
__device__ __forceinline__ float scale_of_exponent(int e) {
    return __uint_as_float((uint32_t)(127 + 14 - max(e - 127, -86)) << 23);
}
__device__ __forceinline__ float scale_to_fp16(float m) {
    return m <= 3.0e38f ? scale_of_exponent((int)(__float_as_uint(m) >> 23)) : 1.0f;
}

// (a, b) * (c, d)
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 r;
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 c, a, b;\n"
        " mov.b64 {%0, %1}, c;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ float2 sub2(float2 x, float2 y) { return fma2(y, make_float2(-1.0f, -1.0f), x); }
__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// 16-bit pairs: a b + c, a b, a b - c, each rounded once
template <typename T> struct Pair;
#define LX_PAIR(T, S)                                                                                      \
    template <> struct Pair<T> {                                                                           \
        static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {               \
            uint32_t r;                                                                                    \
            asm("fma.rn." S " %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));                         \
            return r;                                                                                      \
        }                                                                                                  \
        static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {                           \
            uint32_t r;                                                                                    \
            asm("mul.rn." S " %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));                                     \
            return r;                                                                                      \
        }                                                                                                  \
        static __device__ __forceinline__ uint32_t fms(uint32_t a, uint32_t b, uint32_t c) {               \
            uint32_t r;                                                                                    \
            asm("{\n .reg .b32 n;\n neg." S " n, %3;\n fma.rn." S " %0, %1, %2, n;\n}\n"                    \
                : "=r"(r)                                                                                  \
                : "r"(a), "r"(b), "r"(c));                                                                 \
            return r;                                                                                      \
        }                                                                                                  \
    };
LX_PAIR(__nv_bfloat16, "bf16x2")
LX_PAIR(__half, "f16x2")
#undef LX_PAIR

// 32 bytes at a 32-byte boundary
__device__ __forceinline__ void st32(void* p, const uint32_t* a, const uint32_t* b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]),
                 "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
                 : "memory");
}
__device__ __forceinline__ void ld32(const float* p, uint32_t* r) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}

// What every warp of a block knows.
template <typename T, int DK, int DV, bool OUT>
struct TcBlock {
    static constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    using Z = TcSize<DK, DV, OUT>;
    static constexpr int CH = Z::CH, NS = Z::STAGES;
    static constexpr uint32_t TB = Z::TB;
    static constexpr int HV = DV / 2;  // columns of a thread of the state and of the outputs

    const TcArgs& A;
    const TcRole& R;
    unsigned char* sm;
    TcShared& sh;
    uint32_t smb, tm;
    int slot, h, seq, len, nch, nq, nk, G;
    int64_t t0;
    bool rev, exact;  // exact (state pass): K's weights from fp32, in three parts for bf16
    float l2, g1, up1;  // K's largest weight (e^lam sk reversed, sk forward), times up1, a power of two (fp16)

    __device__ __forceinline__ int64_t chunk_at(int c, int* n) const {
        if (!rev) {
            *n = min(CH, len - c * CH);
            return t0 + (int64_t)c * CH;
        }
        const int end = len - c * CH, a = max(end - CH, 0);
        *n = end - a;
        return t0 + a;
    }
    // bounded; false once any wait of the block has run out
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
        if (mbar_test(bar, parity & 1)) return true;
        for (uint32_t it = 0; it < A.polls; ++it) {
            if (mbar_sleep(bar, parity & 1)) return true;
            if ((it & 15) == 15 && *(volatile uint32_t*)&sh.dead) return false;
        }
        *(volatile uint32_t*)&sh.dead = 1;
        return false;
    }
    // one arrival per warp, after its lanes' accesses
    __device__ __forceinline__ void arrive(uint64_t* bar) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    }

    // a barrier of the warps that arrive there; bounded, unlike bar.sync, since a warp whose wait ran out does not come
    __device__ __forceinline__ bool meet(uint64_t* bar, uint32_t parity) const {
        arrive(bar);
        return wait(bar, parity);
    }

    // ---- copies and products: by one warp, all lanes of which walk through them together (the
    // operands of a product are uniform registers), and one of which acts
    __device__ __forceinline__ void load_kv(int i) const {
        if (i >= nch * nk) return;
        int n;
        const int64_t a = chunk_at(i / nk, &n);
        const int head = h * nk + i % nk;
        uint64_t* bar = &sh.kv_full[i % NS];
        if (elect()) {
            sh.kv_phase[i % NS] = i / NS;
            mbar_expect_tx(bar, Z::KBY + Z::VBY);
            for (int b = 0; b < DK / 64; ++b)
                tma_load3(sm + Z::K + (i % NS) * Z::KBY + b * TB, &A.map[R.mk], b * 64, head, (int)a, bar);
            for (int b = 0; b < DV / 64; ++b)
                tma_load3(sm + Z::V + (i % NS) * Z::VBY + b * TB, &A.map[R.mv], b * 64, head, (int)a, bar);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void load_q(int i) const {
        if (i >= nch * nq) return;
        int n;
        const int64_t a = chunk_at(i / nq, &n);
        if (elect()) {
            sh.q_phase = i;
            mbar_expect_tx(&sh.q_full, Z::KBY);
            for (int b = 0; b < DK / 64; ++b)
                tma_load3(sm + Z::Q + b * TB, &A.map[R.mq], b * 64, h * nq + i % nq, (int)a, &sh.q_full);
        }
        __syncwarp();
    }
    // where the second (1) and third (2) part of K go for the us-th U
    __device__ __forceinline__ uint32_t part(int x, int us) const {
        if (OUT || (BF && exact)) return x == 1 ? Z::LO : Z::S;
        return us & 1 ? Z::S : Z::LO;
    }
    __device__ __forceinline__ void commit(uint64_t* bar) const {
        if (elect()) mma_commit(bar);
        __syncwarp();
    }
    __device__ __forceinline__ void issue() const {
        if (!A.force_expiry) load_kv(0);
        if (OUT) load_q(0);
        for (int i = 1; i < NS; ++i) load_kv(i);
        bool has_state = R.state_in != nullptr;
        int item = 0, us = 0, refill = -1;
        for (int c = 0; c < nch; ++c) {
            for (int i = 0; i < G; ++i, ++item) {
                const int kv = c * nk + (nk > 1 ? i : 0), qi = c * nq + (nq > 1 ? i : 0);
                const bool new_kv = i == 0 || nk > 1, new_q = i == 0 || nq > 1, last = i == G - 1;
                const bool conv = nk > 1 || last, emit = nq > 1 || last;
                const uint32_t Ka = smb + Z::K + (kv % NS) * Z::KBY, Va = smb + Z::V + (kv % NS) * Z::VBY;
                if (new_kv && !wait(&sh.kv_full[kv % NS], kv / NS)) return;
                if constexpr (OUT) {
                    if (new_q && !wait(&sh.q_full, qi)) return;
                    if (item > 0 && !wait(&sh.o_done, item - 1)) return;  // O1 has read the weights in P's place
                    tc_fence_after();
                    constexpr uint32_t id = mma_desc(BF, false, false, 128, 128);
                    const uint64_t dq = tile_desc(smb + Z::Q, 16, 1024), dk = tile_desc(Ka, 16, 1024);
                    if (elect()) {
#pragma unroll
                        for (int s = 0; s < DK / 16; ++s) {
                            const uint32_t off = ((s >> 2) * TB + (s & 3) * 32) >> 4;
                            mma_ss(tm + Z::P, dq + off, dk + off, id, s > 0);
                        }
                        mma_commit(&sh.p_done);
                        if (conv) mma_commit(&sh.k_free);
                    }
                    __syncwarp();
                }
                if (refill >= 0) {  // the last products have read their K and V
                    if (!wait(&sh.u_done[(us - 1) & 1], (us - 1) >> 1)) return;
                    load_kv(refill);
                    refill = -1;
                }
                if constexpr (OUT) {
                    if (item > 0 && !wait(&sh.o_read, item - 1)) return;
                    if (new_q) {
                        if (has_state) {
                            if (i == 0 && !wait(&sh.s_ready, R.state_in ? c : c - 1)) return;
                            tc_fence_after();
                            constexpr uint32_t id = mma_desc(BF, false, true, 128, DV);
                            const uint64_t dq = tile_desc(smb + Z::Q, 16, 1024), ds = tile_desc(smb + Z::S, DK * 128, 1024);
                            if (elect()) {
#pragma unroll
                                for (int s = 0; s < DK / 16; ++s)
                                    mma_ss(tm + Z::O2, dq + (((s >> 2) * TB + (s & 3) * 32) >> 4),
                                           ds + s * (2048 >> 4), id, s > 0);
                            }
                            __syncwarp();
                        }
                        commit(&sh.o2_done);
                    }
                    if (emit && new_q) {  // P and O2 have read Q
                        if (!wait(&sh.o2_done, qi)) return;
                        load_q(qi + 1);
                    }
                    if (!wait(&sh.p_ready, item)) return;
                    if (emit && !new_q) load_q(qi + 1);  // (O2 was before the last P)
                    if (new_kv && !wait(&sh.v_ready[kv & 1], kv >> 1)) return;
                    tc_fence_after();
                    constexpr uint32_t id = mma_desc(BF, false, true, 128, DV);
                    const bool more = nk > 1 && i > 0;
                    const uint64_t dv = tile_desc(Va, TB, 1024);
                    if (elect()) {
#pragma unroll
                        for (int s = 0; s < 8; ++s)
                            mma_ts(tm + Z::O1, tm + Z::P + (s >> 2) * 64 + (s & 3) * 8, dv + s * (2048 >> 4), id, more || s > 0);
                        mma_commit(&sh.o_done);
                    }
                    __syncwarp();
                }
                if (conv) {
                    if (!wait(&sh.k_ready[us & 1], us >> 1)) return;  // and the state is scaled
                    tc_fence_after();
                    // dk = 64: M stays 128, the second half repeats the first (leading offset 0) and is not read
                    constexpr uint32_t id = mma_desc(BF, true, true, 128, DV), lead = DK == 64 ? 0 : TB;
                    const uint64_t dv = tile_desc(Va, TB, 1024), d0 = tile_desc(Ka, lead, 1024),
                                   d1 = tile_desc(smb + part(1, us), lead, 1024), d2 = tile_desc(smb + part(2, us), lead, 1024);
                    // products: onto the scaled state.  State pass: each chunk's by itself, small parts first
                    const bool add = OUT && (us > 0 || R.state_in);
                    const uint32_t U = tm + Z::U;
                    if (elect()) {
                        if (!OUT && BF && exact) {
#pragma unroll
                            for (int s = 0; s < CH / 16; ++s) mma_ss(U, d2 + s * (2048 >> 4), dv + s * (2048 >> 4), id, s > 0);
                        }
                        const bool third = !OUT && BF && exact;
#pragma unroll
                        for (int s = 0; s < CH / 16; ++s)
                            mma_ss(U, d1 + s * (2048 >> 4), dv + s * (2048 >> 4), id, add || third || s > 0);
#pragma unroll
                        for (int s = 0; s < CH / 16; ++s) mma_ss(U, d0 + s * (2048 >> 4), dv + s * (2048 >> 4), id, true);
                        mma_commit(&sh.u_done[us & 1]);
                    }
                    __syncwarp();
                    ++us;
                    refill = kv + NS;
                }
            }
            has_state = true;
        }
    }

    // ---- K's weights, the state
    // V of load kv: rows past the chunk's n tokens become 0 (theirs are of other sequences).  fp16: the largest |k|.
    // (Thread tid has unit tid % 8 of the rows tid / 8 + 32 y of each tile: one offset, 4096 bytes apart.)
    __device__ __forceinline__ float scan(int kv, int n, int tid) const {
        const int r0 = tid >> 3;
        if (n < CH) {
            unsigned char* Vs = sm + Z::V + (kv % NS) * Z::VBY + tile_at(tid >> 3, tid & 7);
            for (int b = 0; b < DV / 64; ++b)
                for (int y = 0; y < CH / 32; ++y)
                    if (r0 + 32 * y >= n) *reinterpret_cast<uint4*>(Vs + b * TB + y * 4096) = make_uint4(0, 0, 0, 0);
        }
        float km = 0.0f;
        if constexpr (!BF) {
            const unsigned char* Ks = sm + Z::K + (kv % NS) * Z::KBY + tile_at(tid >> 3, tid & 7);
            uint32_t m = 0;
#pragma unroll
            for (int x = 0; x < DK / 64 * (CH / 32); ++x) {
                if (r0 + 32 * (x % (CH / 32)) >= n) continue;
                const uint4 w = *reinterpret_cast<const uint4*>(Ks + (x / (CH / 32)) * TB + (x % (CH / 32)) * 4096);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                         __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
            }
            m = max(m & 0xffffu, m >> 16);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(FULL, m, s));
            km = __half2float(__ushort_as_half((unsigned short)m));  // of the warp
        }
        fence_proxy_async();
        if (OUT) arrive(&sh.v_ready[kv & 1]);
        return km;
    }

    // K of load kv, times g1 e^{lam d} (and k_up, fp16), as a sum of 16-bit parts
    // (us: the number of the U that takes it)
    __device__ __forceinline__ void weigh(int kv, int n, float k_up, int tid, int us) const {
        const uint32_t at0 = tile_at(tid >> 3, tid & 7);
        unsigned char* Ks = sm + Z::K + (kv % NS) * Z::KBY + at0;
        unsigned char* Ls = sm + part(1, us) + at0;
        const int r0 = tid >> 3, d0 = rev ? r0 : n - 1 - r0, dd = rev ? 32 : -32;
        using H = Pair<T>;
#pragma unroll 2
        for (int x = 0; x < DK / 64 * (CH / 32); ++x) {
            const uint32_t at = (x / (CH / 32)) * TB + (x % (CH / 32)) * 4096;
            const uint4 w = *reinterpret_cast<const uint4*>(Ks + at);
            const int d = (d0 + (x % (CH / 32)) * dd) & 127;
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
            uint32_t a0[4], a1[4];
            if (!OUT && !BF && exact) {  // (bf16: weigh3)
                // from an fp32 product, what the first part rounds off is the second (and weights below fp16's
                // smallest still count)
                const float f = sh.dec[d] * k_up;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 v = mul2(unpack2<T>(q[e]), make_float2(f, f));
                    a0[e] = pack2<T>(v.x, v.y);
                    v = sub2(v, unpack2<T>(a0[e]));
                    a1[e] = pack2<T>(v.x, v.y);
                }
            } else {
                // k (f1 + f2): the first part rn(k f1); k f1 less it is exact, and with k f2 gives the second
                const uint2 f = sh.dec2[d];
                const uint32_t up = BF ? 0u : pack2<T>(k_up, k_up);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t k = BF ? q[e] : H::mul(q[e], up);  // (exact)
                    a0[e] = H::mul(k, f.x);
                    a1[e] = H::fma(k, f.y, H::fms(k, f.x, a0[e]));
                }
            }
            if (n < CH && r0 + 32 * (x % (CH / 32)) >= n) {  // not 0 * NaN
#pragma unroll
                for (int e = 0; e < 4; ++e) a0[e] = a1[e] = 0;
            }
            *reinterpret_cast<uint4*>(Ks + at) = make_uint4(a0[0], a0[1], a0[2], a0[3]);
            *reinterpret_cast<uint4*>(Ls + at) = make_uint4(a1[0], a1[1], a1[2], a1[3]);
        }
        fence_proxy_async();
    }

    // The same in three parts of bf16, what one rounds off going to the next: 2^-24.  The second and third have one
    // buffer, which the U before (the prev-th, or -1) reads: they wait in registers until it is done.
    // (All of this behind that U: 156 us for the states of 65536 tokens, 16 heads of 128 x 128, 126 with this.)
    __device__ __forceinline__ bool weigh3(int kv, int n, int tid, int prev) const {
        constexpr int X = DK / 64 * (CH / 32);
        const uint32_t at0 = tile_at(tid >> 3, tid & 7);
        unsigned char* Ks = sm + Z::K + (kv % NS) * Z::KBY + at0;
        const int r0 = tid >> 3, d0 = rev ? r0 : n - 1 - r0, dd = rev ? 32 : -32;
        uint32_t a1[X][4], a2[X][4];
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const uint32_t at = (x / (CH / 32)) * TB + (x % (CH / 32)) * 4096;
            const uint4 w = *reinterpret_cast<const uint4*>(Ks + at);
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
            const float f = sh.dec[(d0 + (x % (CH / 32)) * dd) & 127];
            const bool in = r0 + 32 * (x % (CH / 32)) < n;  // not 0 * NaN
            uint32_t a0[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 v = mul2(unpack2<T>(in ? q[e] : 0u), make_float2(f, f));
                a0[e] = pack2<T>(v.x, v.y);
                v = sub2(v, unpack2<T>(a0[e]));
                a1[x][e] = pack2<T>(v.x, v.y);
                v = sub2(v, unpack2<T>(a1[x][e]));
                a2[x][e] = pack2<T>(v.x, v.y);
            }
            *reinterpret_cast<uint4*>(Ks + at) = make_uint4(a0[0], a0[1], a0[2], a0[3]);
        }
        if (prev >= 0 && !wait(&sh.u_done[prev & 1], prev >> 1)) return false;
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const uint32_t at = (x / (CH / 32)) * TB + (x % (CH / 32)) * 4096;
            *reinterpret_cast<uint4*>(sm + Z::LO + at0 + at) = make_uint4(a1[x][0], a1[x][1], a1[x][2], a1[x][3]);
            *reinterpret_cast<uint4*>(sm + Z::S + at0 + at) = make_uint4(a2[x][0], a2[x][1], a2[x][2], a2[x][3]);
        }
        fence_proxy_async();
        return true;
    }

    // The state, in tensor memory in units of 1 / up: rounded into shared memory as the B operand of O2 (which: its number);
    // scaled for the next U.
    __device__ __forceinline__ bool pass(int tid, float up, bool round, int which, float factor) const {
        const int warp = tid >> 5, lane = tid & 31, wg = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t St = tm + ((uint32_t)((warp & 3) * 32) << 16) + Z::U + wg * HV;
        float s_up = 1.0f / up;
        if (!BF && round) {
            float m = 0.0f;
#pragma unroll 1
            for (int cb = 0; cb < HV; cb += 32) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(St + cb, r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float v = fabsf(__uint_as_float(r[j]));
                    m = v <= 3.0e38f ? fmaxf(m, v) : m;  // (NaN and Inf stay what they are at any scale)
                }
            }
            if (row >= R.dk) m = 0.0f;  // (dk < 128: rows that repeat others or hold nothing)
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, s));
            if (lane == 0) sh.red[2][warp] = m;
            if (!meet(&sh.s_max, which)) return false;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = fmaxf(m, sh.red[2][w]);
            s_up = scale_to_fp16(m);
            if (tid == 0) sh.s_inv[which & 1] = 1.0f / (s_up * up);
        }
#pragma unroll 1
        for (int cb = 0; cb < HV; cb += 32) {
            uint32_t r[32];
            __syncwarp();
            tmem_ld32(St + cb, r);
            tmem_wait_ld();
            if (round && row < DK) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint4 w;
                    uint32_t* q = &w.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = __uint_as_float(r[u * 8 + 2 * e]), y = __uint_as_float(r[u * 8 + 2 * e + 1]);
                        q[e] = BF ? pack2<T>(x, y) : pack2<T>(x * s_up, y * s_up);
                    }
                    const int at = wg * HV + cb + u * 8;
                    *reinterpret_cast<uint4*>(sm + Z::S + (at >> 6) * (DK * 128) + tile_at(row, (at & 63) >> 3)) = w;
                }
            }
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 x = mul2(pair(r[j], r[j + 1]), make_float2(factor, factor));
                r[j] = __float_as_uint(x.x);
                r[j + 1] = __float_as_uint(x.y);
            }
            __syncwarp();
            tmem_st32(St + cb, r);
        }
        if (round) {
            fence_proxy_async();
            arrive(&sh.s_ready);
        }
        tmem_wait_st();
        tc_fence_before();
        return true;
    }

    // fp16: the power of two for the K of load kv, from the warps' maxima; 0 after a wait that ran out.  (A buffer's
    // second use is behind the U of its first, for which all warps have read it.)
    __device__ __forceinline__ float k_scale(float km, int tid, int kv) const {
        if constexpr (BF) return 1.0f;
        float* red = sh.red[kv & 1];
        if ((tid & 31) == 0) red[tid >> 5] = km;
        if (!meet(&sh.k_max, kv)) return 0.0f;
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
        return fminf(scale_to_fp16(m), 32768.0f);
    }

    // 32 columns from `col` of a state's row in memory (in: where the row starts, or NULL for zeros)
    __device__ __forceinline__ void read_row(const float* in, int64_t ci, bool has, int col, uint32_t (&r)[32]) const {
        if (ci == 1) {  // (a row is dv values, a multiple of 8)
            const bool whole = (reinterpret_cast<uintptr_t>(in) & 31) == 0;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[j + e] = 0;
                if (has && col + j < R.dv) {
                    if (whole) ld32(in + col + j, r + j);
                    else {
                        const uint4 x = *reinterpret_cast<const uint4*>(in + col + j), y = *reinterpret_cast<const uint4*>(in + col + j + 4);
                        r[j] = x.x, r[j + 1] = x.y, r[j + 2] = x.z, r[j + 3] = x.w;
                        r[j + 4] = y.x, r[j + 5] = y.y, r[j + 6] = y.z, r[j + 7] = y.w;
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = has && col + j < R.dv ? __float_as_uint(in[(col + j) * ci]) : 0u;
        }
    }
    __device__ __forceinline__ void write_row(float* out, int64_t ci, int col, const uint32_t (&r)[32]) const {
        if (ci == 1) {
            const bool whole = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                float* p = out + col + j;
                if (col + j >= R.dv) break;
                if (whole) st32(p, r + j, r + j + 4);
                else {
                    *reinterpret_cast<uint4*>(p) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
                    *reinterpret_cast<uint4*>(p + 4) = make_uint4(r[j + 4], r[j + 5], r[j + 6], r[j + 7]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (col + j < R.dv) out[(col + j) * ci] = __uint_as_float(r[j]);
        }
    }

    // The state pass: thread = row `row` of dk, columns wg * HV .. of the state, which lies in tensor
    // memory but is summed in registers.  A chunk is weighed while the one before is multiplied.
    __device__ __forceinline__ void sum_states(int tid) const {
        const int warp = tid >> 5, lane = tid & 31, wg = warp >> 2, row = (warp & 3) * 32 + lane;
        const int64_t at = ((R.out_by_slot ? (int64_t)slot : (int64_t)seq) * A.H + h) * R.dk * R.dv;
        const int64_t from = ((R.in_by_slot ? (int64_t)slot : (int64_t)seq) * A.H + h) * R.dk * R.dv;
        const int64_t ri = R.transposed ? 1 : R.dv, ci = R.transposed ? R.dk : 1;
        const uint32_t Ut = tm + ((uint32_t)((warp & 3) * 32) << 16) + Z::U + wg * HV, St = Ut + DV;
        const float whole = exp2f(l2 * (float)len);
#pragma unroll 1
        for (int b = 0; b < HV; b += 32) {
            uint32_t r[32];
            read_row(R.state_in ? R.state_in + from + row * ri : nullptr, ci, R.state_in && row < R.dk, wg * HV + b, r);
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * whole);
            __syncwarp();
            tmem_st32(St + b, r);
        }
        tmem_wait_st();
        float unit = 0.0f;  // of the last chunk's U
        const auto add = [&](int us) -> bool {
            if (!wait(&sh.u_done[us & 1], us >> 1)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < HV; b += 16) {
                uint32_t r[16], s[16];
                __syncwarp();
                tmem_ld16(Ut + b, r);
                tmem_ld16(St + b, s);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 x = fma2(make_float2(unit, unit), pair(r[j], r[j + 1]), pair(s[j], s[j + 1]));
                    s[j] = __float_as_uint(x.x);
                    s[j + 1] = __float_as_uint(x.y);
                }
                __syncwarp();
                tmem_st16(St + b, s);
            }
            tmem_wait_st();
            tc_fence_before();
            return true;
        };
        const int n_kv = nch * nk;
        for (int kv = 0; kv < n_kv; ++kv) {
            int n;
            const int64_t a = chunk_at(kv / nk, &n);
            if (!wait(&sh.kv_full[kv % NS], kv / NS)) return;
            const float k_up = k_scale(scan(kv, n, tid), tid, kv);
            if (k_up == 0.0f) return;
            if (BF && exact) {
                if (!weigh3(kv, n, tid, kv - 1)) return;
            } else {
                weigh(kv, n, k_up, tid, kv);
            }
            if (kv > 0 && !add(kv - 1)) return;
            arrive(&sh.k_ready[kv & 1]);
            unit = exp2f(l2 * (float)(rev ? a - t0 : t0 + len - a - n)) / (k_up * up1);
        }
        if (n_kv > 0 && !add(n_kv - 1)) return;
#pragma unroll 1
        for (int b = 0; b < HV; b += 32) {
            uint32_t r[32];
            __syncwarp();
            tmem_ld32(St + b, r);
            tmem_wait_ld();
            if (row < R.dk) write_row(R.state_out + at + row * ri, ci, wg * HV + b, r);
        }
    }

    // The state warps of the products.
    __device__ __forceinline__ void states(int tid) const {
        const int warp = tid >> 5, lane = tid & 31, wg = warp >> 2, row = (warp & 3) * 32 + lane;
        if (nch == 0) return;
        int n;
        chunk_at(0, &n);
        if (R.state_in) {
            const int64_t ri = R.transposed ? 1 : R.dv, ci = R.transposed ? R.dk : 1;
            const float* in = R.state_in + ((R.in_by_slot ? (int64_t)slot : (int64_t)seq) * A.H + h) * R.dk * R.dv + row * ri;
            const uint32_t St = tm + ((uint32_t)((warp & 3) * 32) << 16) + Z::U + wg * HV;
#pragma unroll 1
            for (int cb = 0; cb < HV; cb += 32) {
                uint32_t r[32];
                read_row(in, ci, row < R.dk, wg * HV + cb, r);
                __syncwarp();
                tmem_st32(St + cb, r);
            }
            tmem_wait_st();
        }
        if (!wait(&sh.kv_full[0], 0)) return;
        float k_up = k_scale(scan(0, n, tid), tid, 0);
        if (k_up == 0.0f) return;
        if (R.state_in && !pass(tid, 1.0f, true, 0, exp2f(l2 * (float)n) * (k_up * up1))) return;
        const int n_kv = nch * nk;
        for (int kv = 0; kv < n_kv; ++kv) {  // (a chunk's q-heads share one load)
            const int c = kv / nk, c2 = (kv + 1) / nk;
            chunk_at(c, &n);
            if (!wait(&sh.k_free, kv)) return;  // P has read K
            weigh(kv, n, k_up, tid, kv);
            arrive(&sh.k_ready[kv & 1]);
            const float up = k_up * up1;
            if (kv + 1 == n_kv) {
                wait(&sh.u_done[kv & 1], kv >> 1);  // (before the tensor memory goes)
                return;
            }
            // the next load's scan, while U runs
            int n2;
            chunk_at(c2, &n2);
            if (!wait(&sh.kv_full[(kv + 1) % NS], (kv + 1) / NS)) return;
            k_up = k_scale(scan(kv + 1, n2, tid), tid, kv + 1);
            if (k_up == 0.0f) return;
            const float factor = (c2 != c ? exp2f(l2 * (float)n2) : 1.0f) * (BF ? 1.0f : k_up * up1 / up);
            if (!wait(&sh.u_done[kv & 1], kv >> 1)) return;
            tc_fence_after();
            if ((!BF || c2 != c) && !pass(tid, up, c2 != c, R.state_in ? c2 : c2 - 1, factor)) return;
        }
    }

    // ---- P's weights and the outputs
    // 16 columns base .. of row `row` of P, weighted; tw: the warp's first row
    __device__ __forceinline__ void weights(uint32_t (&r)[16], int base, int row, int tw, int n) const {
        if (rev ? base + 15 < tw || base >= n : base > tw + 31) {
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = 0;
            return;
        }
        const float* w = sh.wt + (rev ? TC_C - 1 : 32) + row - base;
        if (rev ? base > tw + 31 : base + 15 < tw) {
            // nothing masked: e^{lam (row - edge)} e^{lam (edge - s)}, edge the nearest column; both at most 1
            const float f = rev ? w[0] : w[-15];
            const float4* g = reinterpret_cast<const float4*>(sh.grow);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = g[j];
                const float2 a = mul2(pair(r[4 * j], r[4 * j + 1]), mul2(make_float2(f, f), make_float2(x.x, x.y)));
                const float2 b = mul2(pair(r[4 * j + 2], r[4 * j + 3]), mul2(make_float2(f, f), make_float2(x.z, x.w)));
                r[4 * j] = __float_as_uint(a.x);
                r[4 * j + 1] = __float_as_uint(a.y);
                r[4 * j + 2] = __float_as_uint(b.x);
                r[4 * j + 3] = __float_as_uint(b.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float f = w[-j], p = __uint_as_float(r[j]) * f;
                r[j] = f != 0.0f ? __float_as_uint(p) : 0u;  // not 0 * NaN
            }
        }
        if (n < CH) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (base + j >= n) r[j] = 0;
        }
    }

    // Outputs whose O1 is not finite while their O2 is: a NaN or Inf of V that their row
    // may not see, times a weight of 0.  They come from the definition, over the rows s that
    // reach them; 8 columns at a time.  (In the chunk of the first such token: afterwards it is
    // in the state.)
    __device__ __forceinline__ void repair(uint32_t O1, uint32_t O2, T* out, int64_t a, int n, int row, int wg, int head,
                                           bool has_state, float w2) const {
        const T* qr = static_cast<const T*>(R.q) + (a + row) * R.q_ts + (int64_t)(h * nq + head) * R.q_hs;
#pragma unroll 1
        for (int cb = 0; cb < HV && wg * HV + cb < R.dv; cb += 8) {
            float sum[8];
            uint32_t want = 0;
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                __syncwarp();
                const float x = __uint_as_float(tmem_ld1(O1 + cb + j));
                const float y = has_state ? __uint_as_float(tmem_ld1(O2 + cb + j)) : 0.0f;
                tmem_wait_ld();
                if (row < n && !(fabsf(x) <= 3.3e38f) && fabsf(w2 * y) <= 3.3e38f) want |= 1u << j;
            }
            if (!__any_sync(FULL, want != 0)) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
            if (want) {
#pragma unroll 1
                for (int g = 0; g < nk; ++g)
#pragma unroll 1
                    for (int s = rev ? row : 0; rev ? s < n : s <= row; ++s) {
                        const T* kr = static_cast<const T*>(R.k) + (a + s) * R.k_ts + (int64_t)(h * nk + g) * R.k_hs;
                        const T* vr = static_cast<const T*>(R.v) + (a + s) * R.v_ts + (int64_t)(h * nk + g) * R.v_hs + wg * HV + cb;
                        float dot = 0.0f;
#pragma unroll 1
                        for (int e = 0; e < R.dk; ++e) dot = fmaf(to_acc<float, T>(qr[e]), to_acc<float, T>(kr[e]), dot);
                        dot *= R.sq * R.sk * exp2f(l2 * (float)(rev ? s - row : row - s));
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum[j] = fmaf(dot, to_acc<float, T>(vr[j]), sum[j]);
                    }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                __syncwarp();
                const float y = has_state ? __uint_as_float(tmem_ld1(O2 + cb + j)) : 0.0f;
                tmem_wait_ld();
                if (want >> j & 1) out[cb + j] = from_acc<T, float>(fmaf(w2, y, sum[j]));
            }
        }
    }

    __device__ __forceinline__ void rows(int tid) const {
        const int warp = tid >> 5, lane = tid & 31, wg = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int tw = (warp & 3) * 32;
        const uint32_t Pc = tm + lanes + Z::P + wg * 64;  // this warp's columns of P, and of the rounded weights
        const uint32_t O1 = tm + lanes + Z::O1 + wg * HV, O2 = tm + lanes + Z::O2 + wg * HV;
        // outputs in whole 32-byte sectors where they start on one
        const bool wide = ((reinterpret_cast<uintptr_t>(R.o) | (uintptr_t)(R.o_ts * 2) | (uintptr_t)(R.o_hs * 2)) & 31) == 0;
        int wq_n = -1;
        float wq = 0.0f;
        float up = 1.0f;  // fp16: the scale of this row's weights and of O1
        int item = 0;
        for (int c = 0; c < nch; ++c) {
            int n;
            const int64_t a = chunk_at(c, &n);
            const bool has_state = c > 0 || R.state_in;
            if (n != wq_n) {
                wq_n = n;
                wq = R.sq * exp2f(l2 * (float)(rev ? n - 1 - row : row + 1));
            }
            for (int i = 0; i < G; ++i, ++item) {
                const int qi = c * nq + (nq > 1 ? i : 0);
                const bool emit = nq > 1 || i == G - 1;
                if (!wait(&sh.p_done, item)) return;
                tc_fence_after();
                // 16 columns at a time, the next ones on their way
                const float before = up;
                uint32_t r[2][16], pk[8];
                float m = 0.0f;
                __syncwarp();
                tmem_ld16(Pc, r[0]);
                tmem_wait_ld();
#pragma unroll 1
                for (int x = 0; x < 64; x += 32) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        __syncwarp();
                        if (y == 0 || x == 0) tmem_ld16(Pc + x + y * 16 + 16, r[y ^ 1]);
                        weights(r[y], wg * 64 + x + y * 16, row, tw, n);
                        __syncwarp();
                        if constexpr (BF) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                pk[j] = pack2<T>(__uint_as_float(r[y][2 * j]), __uint_as_float(r[y][2 * j + 1]));
                            tmem_st8(Pc + (x + y * 16) / 2, pk);  // over columns that have been read
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float v = fabsf(__uint_as_float(r[y][j]));
                                m = v <= 3.0e38f ? fmaxf(m, v) : m;  // (NaN and Inf stay what they are at any scale)
                            }
                            tmem_st16(Pc + x + y * 16, r[y]);
                        }
                        tmem_wait_ld();
                    }
                }
                if constexpr (!BF) {
                    const int e = (int)(__float_as_uint(m) >> 23);  // (m is finite)
                    uint8_t(*const rexp)[TC_C] = sh.rexp[item & 1];
                    rexp[wg][row] = (uint8_t)e;
                    if (!meet(&sh.p_max[warp & 3], item)) return;
                    const float fresh = scale_of_exponent(max(e, (int)rexp[wg ^ 1][row]));
                    // heads that sum into one O1 share a scale that only falls
                    const bool sum = nk > 1 && i > 0;
                    up = sum ? fminf(before, fresh) : fresh;
                    tmem_wait_st();
#pragma unroll 1
                    for (int x = 0; x < 64; x += 16) {
                        __syncwarp();
                        tmem_ld16(Pc + x, r[0]);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            pk[j] = pack2<T>(__uint_as_float(r[0][2 * j]) * up, __uint_as_float(r[0][2 * j + 1]) * up);
                        tmem_st8(Pc + x / 2, pk);
                    }
                    if (sum) {
                        const float f = up / before;
#pragma unroll 1
                        for (int cb = 0; cb < HV; cb += 16) {
                            __syncwarp();
                            tmem_ld16(O1 + cb, r[0]);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) r[0][j] = __float_as_uint(__uint_as_float(r[0][j]) * f);
                            tmem_st16(O1 + cb, r[0]);
                        }
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(&sh.p_ready);
                if (!wait(&sh.o_done, item)) return;
                if (emit && !wait(&sh.o2_done, qi)) return;
                tc_fence_after();
                const float w1 = BF ? 1.0f : 1.0f / up;
                const float w2 = BF ? wq : wq * (has_state ? sh.s_inv[(R.state_in ? c : c - 1) & 1] : 1.0f);
                T* out = static_cast<T*>(R.o) + (a + row) * R.o_ts + (int64_t)(h * nq + (nq > 1 ? i : 0)) * R.o_hs + wg * HV;
                if (emit) {
                    uint32_t q[2][16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) q[0][j] = q[1][j] = 0;  // (without a state)
                    __syncwarp();
                    tmem_ld16(O1, r[0]);
                    if (has_state) tmem_ld16(O2, q[0]);
                    tmem_wait_ld();
                    const bool in = row < n;
                    const int cols = R.dv - wg * HV;
                    uint32_t odd = 0;  // the sum of the outputs times 0: NaN if one is not finite
#pragma unroll 1
                    for (int cb = 0; cb < HV; cb += 32) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            __syncwarp();
                            if (y == 0 || cb + 32 < HV) {
                                tmem_ld16(O1 + cb + y * 16 + 16, r[y ^ 1]);
                                if (has_state) tmem_ld16(O2 + cb + y * 16 + 16, q[y ^ 1]);
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                float2 p = pair(r[y][2 * j], r[y][2 * j + 1]);
                                if constexpr (!BF) p = mul2(p, make_float2(w1, w1));
                                p = fma2(make_float2(w2, w2), pair(q[y][2 * j], q[y][2 * j + 1]), p);
                                pk[j] = pack2<T>(p.x, p.y);
                                odd = Pair<T>::fma(pk[j], 0u, odd);
                            }
                            const int at = cb + y * 16;
                            if (in && wide && at + 16 <= cols) {
                                st32(out + at, pk, pk + 4);
                            } else if (in) {
                                if (at < cols) *reinterpret_cast<uint4*>(out + at) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                                if (at + 8 < cols) *reinterpret_cast<uint4*>(out + at + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                            }
                            __syncwarp();
                            tmem_wait_ld();
                        }
                    }
                    if (__any_sync(FULL, in && (odd & 0x7fff7fffu) != 0))
                        repair(O1, O2, out, a, n, row, wg, nq > 1 ? i : 0, has_state, w2);
                }
                tc_fence_before();
                arrive(&sh.o_read);
            }
        }
    }
};

// block: its segment and role
template <typename T, int DK, int DV, bool OUT>
__device__ __forceinline__ void lin_block(const TcArgs& A, int block, unsigned char* sm) {
    after_previous();
    using Z = TcSize<DK, DV, OUT>;
    TcShared& sh = *reinterpret_cast<TcShared*>(sm + Z::TILES);
    const TcRole& R = A.role[block % A.nroles];
    const int slot = block / A.nroles, h = blockIdx.y, tid = threadIdx.x;
    int seq, len;
    int64_t t0;
    if (!A.S.find(slot, &seq, &t0, &len)) return;
    const bool rev = R.reverse;
    if (!OUT && R.skip_last && (rev ? t0 == A.S.at(seq) : t0 + len == A.S.at(seq + 1))) return;
    if (smem_u32(sm) & 1023u) {  // the swizzle goes by address bits: the tiles must start on 1024 bytes
        if (tid == 0) set_status(A.status, ST_TIMEOUT);
        return;
    }
    constexpr int ISSUE = (OUT ? 2 : 1) * TC_GROUP / 32;  // the issuing warp
    if (tid == 0) {
        for (uint64_t* b : {&sh.kv_full[0], &sh.kv_full[1], &sh.q_full, &sh.p_done, &sh.k_free, &sh.o2_done, &sh.o_done, &sh.u_done[0], &sh.u_done[1], &sh.drain})
            mbar_init(b, 1);
        for (uint64_t* b : {&sh.v_ready[0], &sh.v_ready[1], &sh.k_ready[0], &sh.k_ready[1], &sh.s_ready, &sh.p_ready, &sh.o_read, &sh.k_max, &sh.s_max})
            mbar_init(b, TC_GROUP / 32);
        for (uint64_t& b : sh.p_max) mbar_init(&b, 2);
        sh.kv_phase[0] = sh.kv_phase[1] = sh.q_phase = -1;
        sh.dead = 0;
        fence_proxy_async();
    }
    __syncwarp();
    if (tid / 32 == ISSUE) tmem_alloc(&sh.tmem, Z::COLS);
    const float l2 = clamp_lam(A.lam[h]) * 1.44269504088896341f;
    const bool exact = !OUT && R.exact;
    // K's weights are g1 e^{lam d}, d >= 0.  fp16: a fast decay (reversed) or a small scale
    // would sink all of them, so a power of two goes from g1 into the state's unit.
    float g1 = R.sk * (rev ? exp2f(l2) : 1.0f), up1 = 1.0f;
    if (std::is_same<T, __half>::value) {
        const float most = g1 * exp2f(fmaxf(l2, 0.0f) * (float)(TC_C - 1));  // (a positive lam: they grow)
        const int e = (int)(__float_as_uint(most) >> 23 & 255) - 127;
        up1 = __uint_as_float((uint32_t)(127 - min(max(e, -40), 40)) << 23);
        g1 *= up1;
    }
    if (tid < TC_C) {
        const float e = exp2f(l2 * (float)tid), d = g1 * e;
        if (tid < 16) sh.grow[rev ? tid : 15 - tid] = e;
        sh.wt[rev ? TC_C - 1 - tid : 32 + tid] = R.sq * R.sk * e;
        if (tid < 32) sh.wt[rev ? TC_C + tid : tid] = 0.0f;
        if (exact) sh.dec[tid] = d;
        else {
            const uint32_t hi = pack2<T>(d, d);
            const float left = d - unpack2<T>(hi).x;
            sh.dec2[tid] = make_uint2(hi, pack2<T>(left, left));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int nch = (len + Z::CH - 1) / Z::CH;
    const TcBlock<T, DK, DV, OUT> B{A,   R,   sm,  sh,   smem_u32(sm), sh.tmem, slot, h,   seq, len, nch,
                                    R.nq, R.nk, max(R.nq, R.nk), t0, rev, exact, l2, g1, up1};
    if constexpr (OUT) {
        // registers: 640 threads x 96 = 512 x 104 + 128 x 64
        if (tid < TC_GROUP) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(WORK_REGS));
            B.states(tid);
        } else if (tid < 2 * TC_GROUP) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(WORK_REGS));
            B.rows(tid - TC_GROUP);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ISSUE_REGS));
            if (tid < 2 * TC_GROUP + 32) B.issue();
        }
    } else {
        if (tid < TC_GROUP) B.sum_states(tid);
        else if (tid / 32 == ISSUE) B.issue();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sh.dead) {
        // a copy or a product did not come: report it, and let what is in flight end (within a bound): the products,
        // the last copies issued to each buffer (those before them have been waited for), stores to tensor memory
        if (tid / 32 == ISSUE) B.commit(&sh.drain);
        if (tid == 0) {
            set_status(A.status, ST_TIMEOUT);
            for (int s = 0; s < 2; ++s)
                if (sh.kv_phase[s] >= 0) mbar_wait(&sh.kv_full[s], sh.kv_phase[s] & 1);
            if (sh.q_phase >= 0) mbar_wait(&sh.q_full, sh.q_phase & 1);
            mbar_wait(&sh.drain, 0);
        }
        __syncwarp();
        tmem_wait_st();
        tc_fence_before();
        __syncthreads();
    }
    if (tid / 32 == ISSUE) {
        tc_fence_after();
        tmem_free(sh.tmem, Z::COLS);
    }
}

template <typename T, int DK, int DV, bool OUT>
__global__ void __launch_bounds__(TcSize<DK, DV, OUT>::NT,
                                  TcSize<DK, DV, OUT>::BLOCKS) k_lin_tc(const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) unsigned char sm[];
    lin_block<T, DK, DV, OUT>(A, blockIdx.x, sm);
}

// Two launches in one, side by side: products, and products of another shape (OUT2) or a state pass.
template <typename T, int DK, int DV, int DK2, int DV2, bool OUT2>
__global__ void __launch_bounds__(TcSize<DK, DV, true>::NT, 1) k_lin_pair(const __grid_constant__ TcArgs A,
                                                                         const __grid_constant__ TcArgs B, int first) {
    extern __shared__ __align__(1024) unsigned char sm[];
    if ((int)blockIdx.x < first) lin_block<T, DK, DV, true>(A, blockIdx.x, sm);
    else lin_block<T, DK2, DV2, OUT2>(B, blockIdx.x - first, sm);
}

// ---------------------------------------------------------------- host side

static thread_local uint32_t g_tc_polls = MBAR_POLLS;
static thread_local int g_tc_force_expiry = 0;

void set_linattn_wait(uint32_t polls, int force_expiry) {
    g_tc_polls = polls ? polls : MBAR_POLLS;
    g_tc_force_expiry = force_expiry;
}

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

// boxes of [tokens][one head][64 values]; values past dim and tokens past T read as 0
static cudaError_t encode(CUtensorMap* m, laplex_dtype dt, const LinRows& x, int dim, int heads, int64_t T, int tokens) {
    EncodeTiled f = encode_fn();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)x.hs * 2, (cuuint64_t)x.ts * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)tokens}, es[3] = {1, 1, 1};
    const CUresult r = f(m, dt == LAPLEX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(x.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tokens per segment (a multiple of 128).  A block of the products takes an SM, so a launch of
// `roles` products runs ceil(blocks / 148) rounds of one segment each; a round costs its tokens
// (28 a microsecond) and about 160 tokens' time to start and end.  A cut adds the state pass (0.35
// of a product's time a token, two blocks on an SM, over all but each sequence's last segment),
// per direction, and the join of the states.  Sequences of one known length take the cheapest
// number of cuts by that count.  Lengths that only the device knows: pieces of a third (with three
// roles a quarter) of an SM's share of all tokens, so that the longest sequence does not decide
// (24 ragged sequences, 16384 tokens, 8 heads of 4 q-heads: 259 us against 490 us with cuts of 2816).
// Known lengths, bf16, heads of 128 x 128, us; the rule's choice in brackets:
//     1 x 65536 tokens, 16 heads: whole 1863, 16384 815, 7424 397, [3712 362], 1920 458
//     1 x 4096, 8 heads:          whole 129, 1024 68, 512 48, [256 47]
//     4 x 8192, 16 heads:         whole 247, 4096 240, [2048 214], 1024 241
//     8 x 8192, 16 heads:         [whole 256], 4096 396, 2048 450
//     10 x 4096, 16 heads:        whole 261, 2048 283, [1024 292]: 15 % off, the worst of 20
//     gradients, 1 x 65536:       whole 1987, 14592 1263, [7296 928], 3712 1103
//     gradients, 4 x 8192:        whole 551, 4096 530, [2816 475], 2048 604
//     gradients, 16 x 4096:       [whole 865], 2048 1055, 1024 1058
int tc_segment(int64_t T, int N, int H, int roles, bool equal) {
    const int64_t whole = std::min<int64_t>(std::max<int64_t>(T, 1) + 1, INT32_MAX);
    if (N == 0 || T == 0) return (int)whole;
    constexpr int64_t SMS = 148, ENDS = 160;
    const auto up = [](int64_t x) { return (x + TC_C - 1) / TC_C * TC_C; };
    const int64_t heads = (int64_t)N * H;
    int64_t seg;
    if (equal) {
        const int64_t L = T / N;
        const int dirs = roles > 1 ? 2 : 1;
        double best = 0;
        seg = whole;
        for (int64_t m = 1; m <= 512 && (m == 1 || L / m >= 2 * TC_C); ++m) {
            const int64_t s = up((L + m - 1) / m), pieces = (L + s - 1) / s;
            double cost = (double)((heads * pieces * roles + SMS - 1) / SMS) * (s + ENDS);
            if (m > 1) {
                cost += 0.35 * (double)((heads * (pieces - 1) * dirs + 2 * SMS - 1) / (2 * SMS)) * 2 * (s + ENDS);
                cost += dirs * (300.0 + 0.7 * heads * pieces);
            }
            if (m == 1 || cost < best) {
                best = cost;
                seg = m == 1 ? whole : s;
            }
        }
        return (int)seg;
    }
    seg = std::max<int64_t>(T * H * roles <= SMS * 256 ? 256 : 512, up(T * H * roles / ((roles > 1 ? 4 : 3) * SMS)));
    return (int)(seg >= T ? whole : seg);
}

// the warps' shares of registers have to fit into what a block of products is launched with
template <auto kern> static cudaError_t registers_suffice(int threads) {
    static std::atomic<int> regs{0};
    int r = regs.load(std::memory_order_relaxed);
    if (r == 0) {
        cudaFuncAttributes at;
        const cudaError_t e = cudaFuncGetAttributes(&at, kern);
        if (e != cudaSuccess) return e;
        regs.store(r = at.numRegs, std::memory_order_relaxed);
    }
    return r * threads < 2 * TC_GROUP * WORK_REGS + 128 * ISSUE_REGS ? cudaErrorInvalidConfiguration : cudaSuccess;
}

template <typename T, int DK, int DV, bool OUT>
static cudaError_t tc_launch(const TcArgs& A, bool next, cudaStream_t st) {
    constexpr auto kern = k_lin_tc<T, DK, DV, OUT>;
    using Z = TcSize<DK, DV, OUT>;
    constexpr size_t smem = Z::BYTES;
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e == cudaSuccess) e = blocks_per_sm<kern>(dev, Z::NT, smem, &per);
    if (e == cudaSuccess && OUT) e = registers_suffice<kern>(Z::NT);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(A.S.slots * A.nroles), (unsigned)A.H);
    if (grid.x == 0) return cudaSuccess;
    return launch(next, kern, grid, Z::NT, smem, st, A);
}

template <typename T, int DK, int DV, int DK2, int DV2, bool OUT2>
static cudaError_t pair_launch(const TcArgs& A, const TcArgs& B, bool next, cudaStream_t st) {
    constexpr auto kern = k_lin_pair<T, DK, DV, DK2, DV2, OUT2>;
    using Z = TcSize<DK, DV, true>;
    constexpr size_t smem = std::max(Z::BYTES, TcSize<DK2, DV2, OUT2>::BYTES);
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e == cudaSuccess) e = blocks_per_sm<kern>(dev, Z::NT, smem, &per);
    if (e == cudaSuccess) e = registers_suffice<kern>(Z::NT);
    if (e != cudaSuccess) return e;
    const int first = A.S.slots * A.nroles;
    const dim3 grid((unsigned)(first + B.S.slots * B.nroles), (unsigned)A.H);
    if (grid.x == 0) return cudaSuccess;
    return launch(next, kern, grid, Z::NT, smem, st, A, B, first);
}

static_assert(TcSize<128, 128, true>::BYTES <= 232448 && TcSize<128, 128, false>::BYTES <= 232448 / 2 - 1024,
              "shared memory of a block");

template <typename T, bool OUT>
static cudaError_t tc_dims(const TcArgs& A, int dk, int dv, bool next, cudaStream_t st) {
    if (dk <= 64) return dv <= 64 ? tc_launch<T, 64, 64, OUT>(A, next, st) : tc_launch<T, 64, 128, OUT>(A, next, st);
    return dv <= 64 ? tc_launch<T, 128, 64, OUT>(A, next, st) : tc_launch<T, 128, 128, OUT>(A, next, st);
}

static int tc_pad(int d) { return d <= 64 ? 64 : 128; }

// The arguments of one launch: those of the roles not yet done that have the first one's padded shape
// (they read the same rows at about the same time).
static cudaError_t tc_args(laplex_dtype dt, const LinRole* roles, int count, bool* done, const LinSeqs& S, int H,
                           const void* lam, bool state_only, uint32_t* status, TcArgs* args) {
    TcArgs& A = *args;
    A = {};
    A.S = S;
    A.H = H;
    A.lam = static_cast<const float*>(lam);
    A.status = status;
    A.polls = g_tc_polls;
    A.force_expiry = g_tc_force_expiry;
    struct { LinRows x; int dim, heads; } key[4];
    int maps = 0, dk = 0, dv = 0;
    for (int j = 0; j < count; ++j) {
        const LinRole& L = roles[j];
        if (done[j] || (A.nroles && (tc_pad(L.dk) != dk || tc_pad(L.dv) != dv))) continue;
        done[j] = true;
        dk = tc_pad(L.dk);
        dv = tc_pad(L.dv);
        TcRole& R = A.role[A.nroles++];
        const auto map_of = [&](const LinRows& x, int dim, int heads, int* m) -> cudaError_t {
            for (*m = 0; *m < maps; ++*m)
                if (key[*m].x.p == x.p && key[*m].x.ts == x.ts && key[*m].x.hs == x.hs && key[*m].dim == dim &&
                    key[*m].heads == heads)
                    return cudaSuccess;
            if (maps == 4) return cudaErrorInvalidValue;
            key[maps++] = {x, dim, heads};
            return S.T > 0 ? encode(&A.map[*m], dt, x, dim, heads, S.T, state_only ? 64 : TC_C) : cudaSuccess;
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
        R.exact = state_only && !L.skip_last;
        R.sq = (float)L.sq;
        R.sk = (float)L.sk;
        R.q = L.q.p;
        R.q_ts = L.q.ts;
        R.q_hs = L.q.hs;
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
    return cudaSuccess;
}

template <typename T>
static cudaError_t tc_both(const TcArgs& A, const TcArgs& B, bool out2, bool next, cudaStream_t st) {
    const int dk = tc_pad(A.role[0].dk), dv = tc_pad(A.role[0].dv);
    if (out2)  // of two shapes: one is the other transposed
        return dk < dv ? pair_launch<T, 64, 128, 128, 64, true>(A, B, next, st) : pair_launch<T, 64, 128, 128, 64, true>(B, A, next, st);
    if (dk <= 64) return dv <= 64 ? pair_launch<T, 64, 64, 64, 64, false>(A, B, next, st) : pair_launch<T, 64, 128, 64, 128, false>(A, B, next, st);
    return dv <= 64 ? pair_launch<T, 128, 64, 128, 64, false>(A, B, next, st) : pair_launch<T, 128, 128, 128, 128, false>(A, B, next, st);
}

// The products of roles[0 .. count), and the states of `last` if there is one.  Two launches that fit on the GPU
// together go as one where they are of the same shape (a state pass) or of transposed ones.  (200 tokens of 8 heads
// of 64 x 64 with their last state: 10.5 us against 19 in turn; the gradients of 1500 tokens of 4 heads of 64 x 96: 17
// against 30.  More blocks than SMs: the state pass does better by itself, two blocks on an SM.)
cudaError_t tc_run(laplex_dtype dt, const LinRole* roles, int count, const LinRole* last, const LinSeqs& S, int H,
                   const void* lam, uint32_t* status, bool next, cudaStream_t st) {
    TcArgs A[3];
    int n = 0;
    bool done[3] = {false, false, false}, state[3] = {false, false, false};
    for (int i = 0; i < count; ++i) {
        if (done[i]) continue;
        const cudaError_t e = tc_args(dt, roles, count, done, S, H, lam, false, status, &A[n++]);
        if (e != cudaSuccess) return e;
    }
    if (last) {
        bool one = false;
        state[n] = true;
        const cudaError_t e = tc_args(dt, last, 1, &one, S, H, lam, true, status, &A[n++]);
        if (e != cudaSuccess) return e;
    }
    int dev = 0, sms = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    int at = 0;
    while (e == cudaSuccess && at < n) {
        const TcArgs& X = A[at];
        const int dk = tc_pad(X.role[0].dk), dv = tc_pad(X.role[0].dv);
        // (a state that is replaced in place is read by the products first)
        if (!state[at] && at + 1 < n && (int64_t)S.slots * H * (X.nroles + A[at + 1].nroles) <= sms &&
            (!state[at + 1] || (tc_pad(A[at + 1].role[0].dk) == dk && tc_pad(A[at + 1].role[0].dv) == dv &&
                                A[at + 1].role[0].state_out != X.role[0].state_in))) {
            e = dt == LAPLEX_BF16 ? tc_both<__nv_bfloat16>(X, A[at + 1], !state[at + 1], next, st)
                                  : tc_both<__half>(X, A[at + 1], !state[at + 1], next, st);
            at += 2;
            next = true;
            continue;
        }
        if (dt == LAPLEX_BF16)
            e = state[at] ? tc_dims<__nv_bfloat16, false>(X, dk, dv, next, st) : tc_dims<__nv_bfloat16, true>(X, dk, dv, next, st);
        else
            e = state[at] ? tc_dims<__half, false>(X, dk, dv, next, st) : tc_dims<__half, true>(X, dk, dv, next, st);
        ++at;
        next = true;
    }
    return e;
}

cudaError_t tc_states(laplex_dtype dt, const LinRole* roles, int count, const LinSeqs& S, int H, const void* lam,
                      uint32_t* status, cudaStream_t st) {
    bool done[3] = {false, false, false};
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < count && e == cudaSuccess; ++i) {
        if (done[i]) continue;
        TcArgs A;
        e = tc_args(dt, roles, count, done, S, H, lam, true, status, &A);
        if (e != cudaSuccess) return e;
        const int dk = tc_pad(A.role[0].dk), dv = tc_pad(A.role[0].dv);
        e = dt == LAPLEX_BF16 ? tc_dims<__nv_bfloat16, false>(A, dk, dv, i > 0, st) : tc_dims<__half, false>(A, dk, dv, i > 0, st);
    }
    return e;
}

}  // namespace lx
