// seqop.h -- internal host-side interface of the sequence operators (decayed
// linear attention, embedding lookup) between their C ABI (capi_seq.cu) and
// the kernel files.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "laplex.h"

namespace lx {

// One operand of a product: rows of `dim` elements at ptr + token * ts + head * hs.
struct LinRows {
    const void* p;
    int64_t ts, hs;  // elements
};

// The packed sequences and their cut into segments.  Sequence n owns the tokens
// [cu(n), cu(n + 1)); a segment is a run of at most `seg` of its tokens, and
// segment j of sequence n has the slot floor(cu(n) / seg) + n + j: slots are
// distinct, and there are floor(T / seg) + N of them, whatever the lengths,
// which only the device knows.
struct LinSeqs {
    const int32_t* cu;  // [N + 1] on the device; NULL: N sequences of T / N tokens
    int64_t T;
    int N;
    int seg;
    int slots;
#ifdef __CUDACC__
    // bounds clamped to [0, T], so that no cu sends an access out of the tensors
    __device__ __forceinline__ int64_t at(int n) const {
        if (!cu) return (int64_t)n * (T / N);
        const int64_t c = cu[n];
        return c < 0 ? 0 : (c > T ? T : c);
    }
    __device__ __forceinline__ int first_slot(int n) const { return (int)(at(n) / seg) + n; }
    // Segment `slot`: its sequence, first token and length; false for a slot
    // that no sequence uses.  An empty sequence has one segment of length 0.
    __device__ __forceinline__ bool find(int slot, int* seq, int64_t* t0, int* len) const {
        int lo = 0, hi = N - 1;  // the last sequence whose first slot is <= slot
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first_slot(mid) <= slot) lo = mid; else hi = mid - 1;
        }
        const int64_t a = at(lo), b = at(lo + 1);
        const int64_t j = (int64_t)slot - first_slot(lo);
        const int64_t left = b - a - j * seg;
        *seq = lo;
        *t0 = a + j * seg;
        *len = (int)(left < 0 ? 0 : (left > seg ? seg : left));
        return j >= 0 && (left > 0 || j == 0);
    }
#endif
};

// One directed product of the family o_t = sq sum_{s <= t} e^{lam (t - s)} <q_t, k_s> v_s
// (reverse: s >= t), with the states X_t = sum e^{lam (t - s)} sk k_s v_s^T.
// The forward product and the three gradients are this product with the
// operands exchanged:
//     o : (q,  k, v)            dq : (do, v, k)
//     dv: (k, q, do) reversed   dk : (v, do, q) reversed
// A group of nq q-heads reads one state; the k and v of nk heads sum into it
// (one of nq, nk is 1).
struct LinRole {
    LinRows q, k, v;
    void* o;
    int64_t o_ts, o_hs;
    int nq, nk;
    int dk, dv;       // dims of q, k and of v, o
    int reverse;
    int transposed;   // the states in memory are [dv, dk] (seen from this role)
    double sq, sk;
    const void* state_in;  // per segment (by slot) or per sequence, or NULL (zero)
    int in_by_slot;
    void* state_out;       // per segment or per sequence, or NULL
    int out_by_slot;
    int skip_last;         // state pass: the segment at the direction's end is not needed
    void* w_out;           // the states' derivatives in lam (state pass), by slot, or NULL
};

struct LinCarry {
    LinSeqs S;
    int H, reverse;
    int64_t len;              // dk * dv
    const void* lam;
    const void* init;         // per sequence, or NULL
    void* states;             // by slot: in, each segment's own state; out, the state before it
    void* w;                  // the same of the derivatives, or NULL
    void* last;               // per sequence: the state behind the last segment, or NULL
};

// (next: the call has launched a kernel before)
// ---- recurrent kernels (every type; linattn_rec.cu)
int rec_segment(int64_t T, int N, int H, int dv, bool equal);
cudaError_t rec_run(laplex_dtype dt, const LinRole& R, const LinSeqs& S, int H, const void* lam, bool state_only,
                    bool next, cudaStream_t st);
cudaError_t carry_run(laplex_dtype dt, const LinCarry* C, int count, cudaStream_t st);  // up to two directions
// dlam[h] = sum over the sequences of scale <do_t, W_t^T q_t> (+ <dstate, W_last>)
size_t dlam_ws_bytes(laplex_dtype dt, int64_t T, int N, int Hkv, int dk, int dv, bool equal);
cudaError_t dlam_run(laplex_dtype dt, LinRole fwd, LinRows dout, LinSeqs S, int H, const void* lam,
                     const void* state, const void* dstate, void* dlam, void* ws, size_t ws_bytes, cudaStream_t st);

// ---- 16-bit rows on the tensor cores (linattn_tc.cu): up to three products at a time and, with
// them, the states behind the last tokens (`last`, or NULL); states of segments, two directions at a time
int tc_segment(int64_t T, int N, int H, int roles, bool equal);
cudaError_t tc_run(laplex_dtype dt, const LinRole* roles, int count, const LinRole* last, const LinSeqs& S, int H,
                   const void* lam, uint32_t* status, bool next, cudaStream_t st);
cudaError_t tc_states(laplex_dtype dt, const LinRole* roles, int count, const LinSeqs& S, int H, const void* lam,
                      uint32_t* status, cudaStream_t st);

// bound of each wait inside the calling thread's later products and state passes (0: the default, 2^20
// polls), and a test switch under which a block's first copy is never issued
void set_linattn_wait(uint32_t polls, int force_expiry);

// ---- single tokens (linattn_step.cu)
struct LinStep {
    LinRows q, k, v;
    void* o;
    int64_t o_ts, o_hs;
    int64_t rows, slots;
    int hq, hkv, dk, dv;
    const int32_t* slot;  // [rows] or NULL (row n uses state n)
    const void* lam;
    double scale;
    void* states;
};
cudaError_t step_run(laplex_dtype dt, const LinStep& A, cudaStream_t st);

// ---- embedding (embed.cu)
struct EmbedArgs {
    const void* tokens;
    int tok64;
    int64_t n, rows, dim;
    const void* src;   // lookup: the table; gradient: g
    int64_t src_ld;
    void* dst;         // lookup: the rows; gradient: the table's gradient
    int64_t dst_ld;
    double scale;
    int accumulate;
};
cudaError_t embed_run(laplex_dtype dt, const EmbedArgs& A, cudaStream_t st);
size_t embed_bwd_ws_bytes(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt);
cudaError_t embed_bwd_run(laplex_dtype dt, laplex_dtype out_dt, const EmbedArgs& A, void* ws, size_t ws_bytes,
                          uint32_t* status, cudaStream_t st);

// stable order of 32-bit keys in [0, top] (sort.cu): skeys ascending, perm[r]
// the index of the r-th
size_t sort_keys_ws_bytes(int64_t n);
cudaError_t sort_keys_run(const uint32_t* keys, int64_t n, uint32_t top, uint32_t* skeys, int32_t* perm, void* ws,
                          size_t ws_bytes, uint32_t* status, cudaStream_t st);

// A launch; `next`: behind another kernel of the same call, on whose end it waits by itself (after_previous).
template <typename... P, typename... A>
cudaError_t launch(bool next, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = next ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

inline size_t elem_bytes(laplex_dtype dt) { return dt == LAPLEX_F64 ? 8 : dt == LAPLEX_F32 ? 4 : 2; }
inline size_t acc_bytes(laplex_dtype dt) { return dt == LAPLEX_F64 ? 8 : 4; }

}  // namespace lx
