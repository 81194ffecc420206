// linattn_rec.cu -- decayed linear attention as a recurrence over tokens, for
// every type (16-bit and fp32 rows computed in fp32, fp64 rows in fp64).
//
// The anchors of a causal sequence are a_t = -lam t, so the printed recurrence
// L_{i+1} = x_{i+1} + exp(a_i - a_{i+1}) L_i (summary §2.2) runs over the tokens
// in order; x_t is the outer product k_t v_t^T, and the output reads the running
// sum through q_t:
//     S_t = e^lam S_{t-1} + k_t v_t^T,      o_t = scale S_t^T q_t.
// A block holds 64 columns of one head's state in registers (8 row groups x 4
// columns per thread) and walks a segment of the sequence.  Tokens are taken in
// blocks of n: the state is scaled by e^{lam n} once, and inside the block v_tau
// carries e^{lam (n - 1 - tau)} and the output its inverse, so that a token costs
// two multiply-adds per state element and the rounding of e^lam enters once per n
// tokens (a product of 2000 rounded e^lam would be off by 6e-5).  n is at most
// 16 / |lam|: neither factor leaves [e^-16, e^16], so fp32 loses nothing to its
// range, and decay() gives both to 2^-23.  (At most 4 / |lam| made blocks of one
// token where lam = -4: 195 against 91 us for 6000 tokens of 6 heads.)
//
// Rows of the type that it computes in come by asynchronous copies, a block of
// tokens ahead; 16-bit rows (only in the decay's derivative: their products run in
// linattn_tc.cu) are converted on their way in.  fp32 multiply-adds go two at a time (a pair of
// the state's rows): half the instructions to issue.
//
// Bound by those multiply-adds (4 dk dv flops a token and head) and the latencies
// around them: 32768 tokens, 16 heads of 128 x 128 take 942 us for the outputs, 477
// for the states alone, 36 Tflop/s of the 72 that 128 fp32 units an SM give.  (6000
// tokens, 6 heads of 72 x 104: 72 and 37 us; with one multiply-add an instruction and
// outputs reduced token by token 119 and 54.)
// Long sequences are cut into segments (see LinSeqs): a first pass sums each
// segment's own state, carry_run joins them, and the product starts each segment
// from its state.
#include <algorithm>
#include <type_traits>

#include "devcache.h"
#include "elem.cuh"
#include "seqop.h"

namespace lx {

constexpr int REC_NT = 128;
constexpr int REC_COLS = 64;  // state columns of a block
constexpr int REC_OUT = 80;   // pitch of a row of outputs: four rows' stores in distinct banks
constexpr int REC_MAX = 32;   // most rows (tokens times heads of a group) in one stage

struct RecArgs {
    LinRole R;
    LinSeqs S;
    int H;
    const void* lam;
    LinRows dout;        // derivative: the output's cotangent
    const void* w_in;    // derivative: by slot, or NULL (zero)
    const void* dstate;  // derivative: the last state's cotangent, or NULL
    double* part;        // derivative: one sum per block
    int rows;            // rows of k, v, q in one of the two stages: 24, or 32 for more than 24 heads
};

// Rows (token tau of the block, head g) of X into dst[row][PITCH], from column c0; a warp to a row.  `first`: row
// `warp` of the block in memory, at this lane's first column, where ONE; it moves on by the block's nb tokens.
// (From the token's index, the addresses were 15 of a token's 75 instructions in the state pass.)
template <typename T, typename A, int PITCH, bool ONE>
__device__ __forceinline__ void rec_load(A* dst, const LinRows& X, const T*& first, int heads, int h, int64_t t0, int len,
                                         int base, int n, int nb, bool rev, int dim, int c0) {
    constexpr int VN = VecOf<T>::N;
    const int per = min(PITCH, dim - c0) / VN;  // (dims are multiples of 8)
    const int lane = threadIdx.x & 31;
    const auto move = [&](int row, const T* src) {
        for (int c = lane; c < per; c += 32, src += 32 * VN) {
            if constexpr (sizeof(T) == sizeof(A)) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(dst + row * PITCH + c * VN)),
                             "l"(src)
                             : "memory");
            } else {
                const Pack<T, VN> v = *reinterpret_cast<const Pack<T, VN>*>(src);
#pragma unroll
                for (int e = 0; e < VN; ++e) dst[row * PITCH + c * VN + e] = to_acc<A, T>(v.v[e]);
            }
        }
    };
    if constexpr (ONE) {
        const int64_t ts = rev ? -X.ts : X.ts;
        const T* src = first;
        for (int row = threadIdx.x >> 5; row < n; row += REC_NT / 32, src += REC_NT / 32 * ts) move(row, src);
        first += nb * ts;
    } else {
        for (int row = threadIdx.x >> 5; row < n * heads; row += REC_NT / 32) {
            const int tau = heads == 1 ? row : row / heads, g = row - tau * heads;
            const int64_t t = t0 + (rev ? len - 1 - base - tau : base + tau);
            move(row, static_cast<const T*>(X.p) + t * X.ts + (int64_t)(h * heads + g) * X.hs + c0 + lane * VN);
        }
    }
}

// Two values that one multiply-add instruction takes together (fp32; fp64 in two).
template <typename A> struct Two;
template <> struct Two<float> {
    unsigned long long v;
    static __device__ __forceinline__ Two of(float x, float y) {
        Two r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
        return r;
    }
    __device__ __forceinline__ float at(int i) const {
        float x, y;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
        return i ? y : x;
    }
    static __device__ __forceinline__ Two fma(Two a, Two b, Two c) {
        Two r;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
        return r;
    }
    static __device__ __forceinline__ Two mul(Two a, Two b) {
        Two r;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
        return r;
    }
    static __device__ __forceinline__ Two add(Two a, Two b) {
        Two r;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
        return r;
    }
};
template <> struct Two<double> {
    double x, y;
    static __device__ __forceinline__ Two of(double x, double y) { return {x, y}; }
    __device__ __forceinline__ double at(int i) const { return i ? y : x; }
    static __device__ __forceinline__ Two fma(Two a, Two b, Two c) { return {dfma(a.x, b.x, c.x), dfma(a.y, b.y, c.y)}; }
    static __device__ __forceinline__ Two mul(Two a, Two b) { return {a.x * b.x, a.y * b.y}; }
    static __device__ __forceinline__ Two add(Two a, Two b) { return {a.x + b.x, a.y + b.y}; }
};

// A thread's part of a state: rows 32 m + 4 rg + (0..3), in pairs, of 4 columns.
template <typename A, int RPT>
__device__ __forceinline__ void rec_state_io(Two<A> (&S)[RPT / 2][4], const LinRole& R, A* mem, int64_t at, int rg, int col,
                                             bool store) {
    const int64_t ri = R.transposed ? 1 : R.dv, ci = R.transposed ? R.dk : 1;
    A* p = mem + at * R.dk * R.dv;
#pragma unroll
    for (int r = 0; r < RPT; r += 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = (r / 4) * 32 + rg * 4 + (r % 4), j = col + c;
            if (i < R.dk && j < R.dv) {  // (dk is even)
                A* a = p + i * ri + j * ci;
                if (store) {
                    a[0] = S[r / 2][c].at(0);
                    a[ri] = S[r / 2][c].at(1);
                } else {
                    S[r / 2][c] = Two<A>::of(a[0], a[ri]);
                }
            }
        }
}

// The sums over the 8 row groups (lane bits 0-2) of p[row][column], U rows of 4 columns, times each row's wq, into os.
// Every step halves what a lane keeps.
template <typename A, int U>
__device__ __forceinline__ void rec_reduce(const A (&p)[U][4], const A* wq, A* os, int lane) {
    const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
    if constexpr (U == 4) {
        A x[2][4], y[4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                x[u][c] = (b0 ? p[2 + u][c] : p[u][c]) + __shfl_xor_sync(FULL, b0 ? p[u][c] : p[2 + u][c], 1);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = (b1 ? x[1][c] : x[0][c]) + __shfl_xor_sync(FULL, b1 ? x[0][c] : x[1][c], 2);
        const A z0 = (b2 ? y[2] : y[0]) + __shfl_xor_sync(FULL, b2 ? y[0] : y[2], 4);
        const A z1 = (b2 ? y[3] : y[1]) + __shfl_xor_sync(FULL, b2 ? y[1] : y[3], 4);
        const int u = (b0 ? 2 : 0) + (b1 ? 1 : 0);
        Pack<A, 2> o;
        o.v[0] = z0 * wq[u];
        o.v[1] = z1 * wq[u];
        *reinterpret_cast<Pack<A, 2>*>(os + u * REC_OUT + (b2 ? 2 : 0)) = o;
    } else {
        A u0 = b0 ? p[0][2] : p[0][0], u1 = b0 ? p[0][3] : p[0][1];
        u0 += __shfl_xor_sync(FULL, b0 ? p[0][0] : p[0][2], 1);
        u1 += __shfl_xor_sync(FULL, b0 ? p[0][1] : p[0][3], 1);
        A w = b1 ? u1 : u0;
        w += __shfl_xor_sync(FULL, b1 ? u0 : u1, 2);
        w += __shfl_xor_sync(FULL, w, 4);
        if (!b2) os[(b0 ? 2 : 0) + (b1 ? 1 : 0)] = w * wq[0];
    }
}

// READ 0: states only; 1: outputs; 2: the decay's derivative.  DER: also run the
// states' derivative in lam, W_t = e^lam (W_{t-1} + S_{t-1}).  ONE: one q-head and one
// k-head to a state.
template <typename T, int RPT, int READ, bool DER, bool ONE>
__global__ void __launch_bounds__(REC_NT) k_rec(const __grid_constant__ RecArgs P) {
    using A = typename AccOf<T>::A;
    after_previous();
    constexpr int DKP = RPT * 8;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    constexpr int STAGE = DKP * (READ ? 2 : 1) + REC_COLS * (READ == 2 ? 2 : 1);  // values of a row in all operands
    const int cap = P.rows;
    A* const stages = reinterpret_cast<A*>(smem_raw);
    A* const os = stages + 2 * cap * STAGE;  // outputs of a block
    __shared__ A down[REC_MAX + 1];  // e^{lam j}
    __shared__ A wks[REC_MAX], wqs[REC_MAX];  // a block's weights, by token: sk e^{lam (n - 1 - j)}; by row of q: sq e^{-lam (n - 1 - j)}
    const LinRole& R = P.R;
    const int nq = ONE ? 1 : R.nq, nk = ONE ? 1 : R.nk;
    const int slot = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * REC_COLS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rg = lane & 7, cl = warp * 16 + (lane >> 3) * 4, col = c0 + cl;
    int seq, len;
    int64_t t0;
    const bool used = P.S.find(slot, &seq, &t0, &len);
    if (READ == 2 && !used && threadIdx.x == 0)
        P.part[((int64_t)slot * P.H + h) * gridDim.z + blockIdx.z] = 0.0;
    if (!used) return;
    if (READ == 0 && R.skip_last && (R.reverse ? t0 == P.S.at(seq) : t0 + len == P.S.at(seq + 1))) return;
    const A lam = clamp_lam(static_cast<const A*>(P.lam)[h]);
    const int heads = nq > nk ? nq : nk;
    int nb = cap / heads;
    const A al = lam < 0 ? -lam : lam;
    if (al * nb > (A)16) nb = max(1, (int)((A)16 / al));
    if (threadIdx.x <= nb) down[threadIdx.x] = decay(lam, (A)threadIdx.x);
    if (R.dk < DKP || R.dv - c0 < REC_COLS)  // columns past dk, dv stay 0
        for (int i = threadIdx.x; i < 2 * cap * STAGE; i += REC_NT) stages[i] = 0;
    __syncthreads();
    const bool rev = R.reverse;
    const auto first = [&](const LinRows& X, int c) {
        const int64_t t = t0 + (rev ? len - 1 - warp : warp);
        return static_cast<const T*>(X.p) + t * X.ts + (int64_t)h * X.hs + c + lane * VecOf<T>::N;
    };
    const T *kp = nullptr, *vp = nullptr, *qp = nullptr, *dp = nullptr;
    if constexpr (ONE) {
        kp = first(R.k, 0);
        vp = first(R.v, c0);
        if (READ != 0) qp = first(R.q, 0);
    }
    const auto load = [&](int base, int s) {
        if (base < len) {
            const int n = min(nb, len - base);
            A* ks = stages + s * cap * STAGE;
            A *vs = ks + cap * DKP, *qs = vs + cap * REC_COLS, *ds = qs + cap * DKP;
            rec_load<T, A, DKP, ONE>(ks, R.k, kp, nk, h, t0, len, base, n, nb, rev, R.dk, 0);
            rec_load<T, A, REC_COLS, ONE>(vs, R.v, vp, nk, h, t0, len, base, n, nb, rev, R.dv, c0);
            if constexpr (READ != 0) rec_load<T, A, DKP, ONE>(qs, R.q, qp, nq, h, t0, len, base, n, nb, rev, R.dk, 0);
            if constexpr (READ == 2) rec_load<T, A, REC_COLS, ONE>(ds, P.dout, dp, nq, h, t0, len, base, n, nb, rev, R.dv, c0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(0, 0);

    using V = Two<A>;
    V S[RPT / 2][4], W[DER ? RPT / 2 : 1][4];
#pragma unroll
    for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            S[r][c] = V::of(0, 0);
            if constexpr (DER) W[r][c] = V::of(0, 0);
        }
    const int64_t by_slot = (int64_t)slot * P.H + h, by_seq = (int64_t)seq * P.H + h;
    if (R.state_in)
        rec_state_io<A, RPT>(S, R, (A*)const_cast<void*>(R.state_in), R.in_by_slot ? by_slot : by_seq, rg, col, false);
    if constexpr (DER)
        if (P.w_in) rec_state_io<A, RPT>(W, R, (A*)const_cast<void*>(P.w_in), by_slot, rg, col, false);
    A dsum = 0;
    int stage = 0, weights_n = 0;
    for (int base = 0; base < len; base += nb, stage ^= 1) {
        const int n = min(nb, len - base);
        load(base + nb, stage ^ 1);
        if (n != weights_n) {
            weights_n = n;
            for (int j = threadIdx.x; j < n * heads; j += REC_NT) {
                if (j < n) wks[j] = (A)R.sk * decay(lam, (A)(n - 1 - j));
                if (j < n * nq) wqs[j] = (A)R.sq * decay(lam, -(A)(n - 1 - j / nq));
            }
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const A* ks = stages + stage * cap * STAGE;
        const A *vs = ks + cap * DKP, *qs = vs + cap * REC_COLS, *ds = qs + cap * DKP;
        const V pre = V::of(down[rev ? n - 1 : n], down[rev ? n - 1 : n]);
#pragma unroll
        for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                S[r][c] = V::mul(S[r][c], pre);
                if constexpr (DER) W[r][c] = V::mul(W[r][c], pre);
            }
        const bool some = c0 + warp * 16 < R.dv;  // (a warp past dv has no column)
        // row r of k and v, of token tau
        const auto update = [&](int r, int tau) {
            const Pack<A, 4> x = *reinterpret_cast<const Pack<A, 4>*>(vs + r * REC_COLS + cl);
            const A wk = wks[tau];
            V vv[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) vv[c] = V::of(x.v[c] * wk, x.v[c] * wk);
#pragma unroll
            for (int m = 0; m < RPT / 4; ++m) {
                const Pack<V, 2> kk = *reinterpret_cast<const Pack<V, 2>*>(ks + r * DKP + m * 32 + rg * 4);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) S[m * 2 + j][c] = V::fma(kk.v[j], vv[c], S[m * 2 + j][c]);
            }
        };
        // row r of q: this thread's part of S^T q (READ 2: of W^T q)
        const auto read = [&](int r, A (&p)[4]) {
            V a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) a[c] = V::of(0, 0);
#pragma unroll
            for (int m = 0; m < RPT / 4; ++m) {
                const Pack<V, 2> qq = *reinterpret_cast<const Pack<V, 2>*>(qs + r * DKP + m * 32 + rg * 4);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if constexpr (READ == 2) a[c] = V::fma(qq.v[j], W[m * 2 + j][c], a[c]);
                        else a[c] = V::fma(qq.v[j], S[m * 2 + j][c], a[c]);
                    }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) p[c] = a[c].at(0) + a[c].at(1);
        };
        const auto advance = [&](int tau) {  // token tau's k and v into the state
            if constexpr (DER) {
#pragma unroll
                for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) W[r][c] = V::add(W[r][c], S[r][c]);
            }
            for (int g = 0; g < nk; ++g) update(tau * nk + g, tau);
        };
        if (some) {
            if constexpr (READ == 1) {
                // rows four at a time: their sums over the row groups take 14 exchanges and one store, not 16 and four
                const int rows = n * nq;
                int r = 0, tau = 0, g = 0;
                const auto batch = [&](auto U) {
                    A p[U.value][4];
#pragma unroll
                    for (int u = 0; u < U.value; ++u) {
                        if (ONE) update(r + u, r + u);
                        else {
                            if (g == 0) advance(tau);
                            if (++g == nq) {
                                g = 0;
                                ++tau;
                            }
                        }
                        read(r + u, p[u]);
                    }
                    rec_reduce<A, U.value>(p, wqs + r, os + r * REC_OUT + cl, lane);
                };
                for (; r + 4 <= rows; r += 4) batch(std::integral_constant<int, 4>());
                for (; r < rows; ++r) batch(std::integral_constant<int, 1>());
            } else {
                constexpr int U = !DER ? 4 : sizeof(A) == 8 ? 1 : 2;
#pragma unroll U
                for (int tau = 0; tau < n; ++tau) {
                    advance(tau);
                    if constexpr (READ == 2) {
                        for (int g = 0; g < nq; ++g) {
                            const int row = tau * nq + g;
                            A p[4], x = 0;
                            read(row, p);
                            const Pack<A, 4> d = *reinterpret_cast<const Pack<A, 4>*>(ds + row * REC_COLS + cl);
#pragma unroll
                            for (int c = 0; c < 4; ++c) x = dfma(d.v[c], p[c], x);
                            dsum = dfma(wqs[row], x, dsum);
                        }
                    }
                }
            }
        }
        if (rev) {
            const V post = V::of(down[1], down[1]);
#pragma unroll
            for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[r][c] = V::mul(S[r][c], post);
        }
        if constexpr (READ == 1) {
            __syncthreads();
            constexpr int Q = REC_COLS / 4;  // (dv is a multiple of 8)
            const int cols = min(REC_COLS, R.dv - c0);
            for (int i = threadIdx.x; i < n * nq * Q; i += REC_NT) {
                const int row = i / Q, c = i % Q * 4;
                if (c >= cols) continue;
                const int tau = row / nq, g = row - tau * nq;
                const int64_t t = t0 + (rev ? len - 1 - base - tau : base + tau);
                *reinterpret_cast<Pack<A, 4>*>(static_cast<A*>(R.o) + t * R.o_ts + (int64_t)(h * nq + g) * R.o_hs + c0 + c) =
                    *reinterpret_cast<const Pack<A, 4>*>(os + row * REC_OUT + c);
            }
        }
        __syncthreads();  // this stage, and the outputs, have been read
    }
    if (R.state_out)
        rec_state_io<A, RPT>(S, R, (A*)R.state_out, R.out_by_slot ? by_slot : by_seq, rg, col, true);
    if constexpr (DER && READ == 0) rec_state_io<A, RPT>(W, R, (A*)R.w_out, by_slot, rg, col, true);
    if constexpr (READ == 2) {
        // the last segment of a sequence: <dstate, W_last>
        const bool last = t0 + len >= P.S.at(seq + 1);
        if (P.dstate && last) {
            V D[RPT / 2][4], sum = V::of(0, 0);
#pragma unroll
            for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) D[r][c] = V::of(0, 0);
            rec_state_io<A, RPT>(D, R, (A*)const_cast<void*>(P.dstate), by_seq, rg, col, false);
#pragma unroll
            for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) sum = V::fma(D[r][c], W[r][c], sum);
            dsum += sum.at(0) + sum.at(1);
        }
        double* red = reinterpret_cast<double*>(smem_raw);
        __syncthreads();
        red[threadIdx.x] = (double)dsum;
        __syncthreads();
        for (int s = REC_NT / 2; s > 0; s >>= 1) {  // a fixed order: the result does not vary from run to run
            if ((int)threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
            __syncthreads();
        }
        if (threadIdx.x == 0) P.part[by_slot * gridDim.z + blockIdx.z] = red[0];
    }
}

// dlam[h]: the blocks' sums of head h, in a fixed order
template <typename A>
__global__ void __launch_bounds__(256) k_dlam_join(const double* __restrict__ part, int64_t slots, int H, int cb,
                                                   A* __restrict__ dlam) {
    __shared__ double red[256];
    after_previous();
    const int h = blockIdx.x;
    double s = 0;
    for (int64_t i = threadIdx.x; i < slots * cb; i += 256) s += part[(i / cb * H + h) * cb + i % cb];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int w = 128; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) dlam[h] = (A)red[0];
}

// States before each segment from the segments' own: per element a serial walk
// over the segments of a sequence.
//     X_in(j + 1) = e^{lam len_j} X_in(j) + X_j            (reverse: towards smaller j)
//     W_in(j + 1) = e^{lam len_j} (W_in(j) + len_j X_in(j)) + W_j
// Each segment's state is read and written once; a thread walks 16 bytes, the
// loads of the next four segments in flight while it writes these.  Both
// directions of a backward call share a launch.  (One value a thread and four
// loads at a time: 86 us for 37 segments x 16 heads of 128 x 128, which move 78 MB,
// now 7.  Eight segments at a time hold so many registers that the many short
// sequences of a ragged batch wait for a place: 29 us against 17 for 24 sequences x
// 8 heads; two: 14 us there, but 16 against 13 us for the long backward pass.)
struct CarryArgs {
    LinCarry dir[2];
    int count;
};

template <typename A, bool DER>
__global__ void __launch_bounds__(128) k_carry(const __grid_constant__ CarryArgs args) {
    after_previous();
    const LinCarry& C = args.dir[args.count > 1 && blockIdx.x >= gridDim.x / 2];
    const unsigned bx = args.count > 1 ? blockIdx.x % (gridDim.x / 2) : blockIdx.x;
    constexpr int VN = 16 / (int)sizeof(A), U = DER ? 2 : 4;
    using V = Pack<A, VN>;
    const int seq = blockIdx.y, h = blockIdx.z;
    const int64_t e = ((int64_t)bx * 128 + threadIdx.x) * VN;
    if (e >= C.len) return;
    const A lam = clamp_lam(static_cast<const A*>(C.lam)[h]);
    const int64_t total = C.S.at(seq + 1) - C.S.at(seq);
    int count = total <= 0 ? 1 : (int)((total + C.S.seg - 1) / C.S.seg);
    const int s0 = C.S.first_slot(seq);
    count = min(count, C.S.slots - s0);  // (bounds that do not ascend)
    const int64_t by_seq = ((int64_t)seq * C.H + h) * C.len + e;
    V x, w;
#pragma unroll
    for (int k = 0; k < VN; ++k) x.v[k] = w.v[k] = 0;
    if (C.init) x = *reinterpret_cast<const V*>(static_cast<const A*>(C.init) + by_seq);
    const int64_t tail = total - (int64_t)(count - 1) * C.S.seg;
    const A full = decay(lam, (A)C.S.seg), part = decay(lam, (A)tail);
    const int64_t step = (C.reverse ? -1 : 1) * (int64_t)C.H * C.len;
    const int64_t at0 = ((int64_t)(s0 + (C.reverse ? count - 1 : 0)) * C.H + h) * C.len + e;
    A* st = static_cast<A*>(C.states) + at0;
    A* wt = DER ? static_cast<A*>(C.w) + at0 : nullptr;
    V own[2][U], wown[2][DER ? U : 1];
    const auto load = [&](int b, int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < count) {
                own[b][u] = *reinterpret_cast<const V*>(st + (i0 + u) * step);
                if constexpr (DER) wown[b][u] = *reinterpret_cast<const V*>(wt + (i0 + u) * step);
            }
    };
    const auto walk = [&](int b, int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i < count) {
                const bool end = C.reverse ? i == 0 : i == count - 1;  // the sequence's last segment
                const A d = end ? part : full;
                *reinterpret_cast<V*>(st + i * step) = x;
                if constexpr (DER) {
                    const A n = (A)(end ? tail : (int64_t)C.S.seg);
                    *reinterpret_cast<V*>(wt + i * step) = w;
#pragma unroll
                    for (int k = 0; k < VN; ++k) w.v[k] = dfma(d, dfma(n, x.v[k], w.v[k]), wown[b][u].v[k]);
                }
#pragma unroll
                for (int k = 0; k < VN; ++k) x.v[k] = dfma(d, x.v[k], own[b][u].v[k]);
            }
        }
    };
    load(0, 0);
    for (int i0 = 0; i0 < count; i0 += 2 * U) {
        load(1, i0 + U);
        walk(0, i0);
        load(0, i0 + 2 * U);
        walk(1, i0 + U);
    }
    if (C.last) *reinterpret_cast<V*>(static_cast<A*>(C.last) + by_seq) = x;
}

// ---------------------------------------------------------------- host side

// Tokens per segment.  Enough blocks for two rounds of the resident ones (148
// SMs x 4), but not under 128 tokens, below which the extra pass over k and v and
// the states' traffic cost as much as they spread (6000 tokens, 6 heads of 72 x 104:
// 121 us with 128, 120 with 64, 127 with 192; 560 heads of 128 tokens of 64 x 64:
// 55 us whole, 104 cut at 64) -- or 64 where 128 leaves SMs without a block (256
// tokens, 6 heads: 33 against 52 us).  Sequences of one known length that fill the
// GPU by themselves are not cut.
int rec_segment(int64_t T, int N, int H, int dv, bool equal) {
    const int64_t cb = (dv + REC_COLS - 1) / REC_COLS;
    const int64_t whole = std::max<int64_t>(T, 1) + 1;
    if (equal && (int64_t)N * H * cb >= 592) return (int)std::min<int64_t>(whole, INT32_MAX);
    int64_t seg = (T * H * cb / 1184 + 63) / 64 * 64;
    seg = std::max<int64_t>(seg, T * H * cb < 128 * 148 ? 64 : 128);
    return (int)std::min<int64_t>(seg >= T ? whole : seg, INT32_MAX);
}

template <typename T, int RPT, int READ, bool DER, bool ONE>
static cudaError_t rec_launch(const RecArgs& P, bool next, cudaStream_t st) {
    using A = typename AccOf<T>::A;
    constexpr auto kern = k_rec<T, RPT, READ, DER, ONE>;
    constexpr size_t row = sizeof(A) * (2 * (RPT * 8 * (READ ? 2 : 1) + REC_COLS * (READ == 2 ? 2 : 1)) + (READ == 1 ? REC_OUT : 0));
    constexpr size_t most = row * REC_MAX;
    const size_t smem = row * P.rows;
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e == cudaSuccess) e = blocks_per_sm<kern>(dev, REC_NT, most, &per);  // (raises the limit)
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)P.S.slots, (unsigned)P.H, (unsigned)((P.R.dv + REC_COLS - 1) / REC_COLS));
    if (grid.x == 0) return cudaSuccess;
    return launch(next, kern, grid, REC_NT, smem, st, P);
}

template <typename T, int READ, bool DER, bool ONE = false>
static cudaError_t rec_dim(RecArgs P, bool next, cudaStream_t st) {
    P.rows = std::max(P.R.nq, P.R.nk) > 24 ? 32 : 24;  // (16: 1479 us against 1426 for 32768 tokens of 16 heads of 128 x 128)
    return P.R.dk <= 64   ? rec_launch<T, 8, READ, DER, ONE>(P, next, st)
           : P.R.dk <= 96 ? rec_launch<T, 12, READ, DER, ONE>(P, next, st)
                          : rec_launch<T, 16, READ, DER, ONE>(P, next, st);
}

template <typename F>
static cudaError_t with_type(laplex_dtype dt, F f) {
    switch (dt) {
        case LAPLEX_F32: return f(float());
        case LAPLEX_F64: return f(double());
        case LAPLEX_F16: return f(__half());
        case LAPLEX_BF16: return f(__nv_bfloat16());
    }
    return cudaErrorInvalidValue;
}

cudaError_t rec_run(laplex_dtype dt, const LinRole& R, const LinSeqs& S, int H, const void* lam, bool state_only,
                    bool next, cudaStream_t st) {
    RecArgs P = {};
    P.R = R;
    P.S = S;
    P.H = H;
    P.lam = lam;
    const auto go = [&](auto t) {
        using T = decltype(t);
        if (R.nq == 1 && R.nk == 1) return state_only ? rec_dim<T, 0, false, true>(P, next, st) : rec_dim<T, 1, false, true>(P, next, st);
        return state_only ? rec_dim<T, 0, false>(P, next, st) : rec_dim<T, 1, false>(P, next, st);
    };
    return dt == LAPLEX_F64 ? go(double()) : go(float());
}

cudaError_t carry_run(laplex_dtype dt, const LinCarry* C, int count, cudaStream_t st) {
    if (count == 0 || C->S.N == 0 || C->H == 0) return cudaSuccess;
    // sequences ride in grid.y (at most 65535): the C boundary checks their number
    const int64_t per = 128 * (16 / (int64_t)acc_bytes(dt));  // dk dv is a multiple of 64
    const dim3 grid((unsigned)((C->len + per - 1) / per * count), (unsigned)C->S.N, (unsigned)C->H);
    CarryArgs args = {};
    args.count = count;
    for (int i = 0; i < count; ++i) args.dir[i] = C[i];
    if (dt == LAPLEX_F64) {
        return C->w ? launch(true, k_carry<double, true>, grid, 128, 0, st, args)
                    : launch(true, k_carry<double, false>, grid, 128, 0, st, args);
    }
    return C->w ? launch(true, k_carry<float, true>, grid, 128, 0, st, args)
                : launch(true, k_carry<float, false>, grid, 128, 0, st, args);
}

static LinSeqs dlam_seqs(int64_t T, int N, const int32_t* cu, int Hkv, int dv) {
    LinSeqs S;
    S.cu = cu;
    S.T = T;
    S.N = N;
    S.seg = rec_segment(T, N, Hkv, dv, cu == nullptr);
    S.slots = (int)(T / S.seg) + N;
    return S;
}

size_t dlam_ws_bytes(laplex_dtype dt, int64_t T, int N, int Hkv, int dk, int dv, bool equal) {
    const int seg = rec_segment(T, N, Hkv, dv, equal);
    const int64_t slots = T / seg + N;
    const int64_t cb = (dv + REC_COLS - 1) / REC_COLS;
    const size_t part = (size_t)((slots * Hkv * cb * 8 + 255) / 256 * 256);
    if (seg > T) return part;
    return part + 2 * (size_t)((slots * Hkv * dk * dv * (int64_t)acc_bytes(dt) + 255) / 256 * 256);
}

cudaError_t dlam_run(laplex_dtype dt, LinRole fwd, LinRows dout, LinSeqs S0, int H, const void* lam,
                     const void* state, const void* dstate, void* dlam, void* ws, size_t ws_bytes, cudaStream_t st) {
    const LinSeqs S = dlam_seqs(S0.T, S0.N, S0.cu, H, fwd.dv);
    const int cb = (fwd.dv + REC_COLS - 1) / REC_COLS;
    const size_t need = dlam_ws_bytes(dt, S.T, S.N, H, fwd.dk, fwd.dv, S.cu == nullptr);
    if (ws_bytes < need) return cudaErrorInvalidValue;
    char* base = static_cast<char*>(ws);
    RecArgs P = {};
    P.S = S;
    P.H = H;
    P.lam = lam;
    P.part = reinterpret_cast<double*>(base);
    base += ((size_t)S.slots * H * cb * 8 + 255) / 256 * 256;
    P.R = fwd;
    P.R.state_in = state;
    P.R.in_by_slot = 0;
    P.R.state_out = nullptr;
    cudaError_t e = cudaSuccess;
    if (S.seg <= S.T) {
        const size_t sb = ((size_t)S.slots * H * fwd.dk * fwd.dv * acc_bytes(dt) + 255) / 256 * 256;
        RecArgs Q = P;
        Q.R.state_in = nullptr;
        Q.R.state_out = base;
        Q.R.out_by_slot = 1;
        Q.R.w_out = base + sb;
        e = with_type(dt, [&](auto t) { return rec_dim<decltype(t), 0, true>(Q, false, st); });
        if (e != cudaSuccess) return e;
        LinCarry C = {};
        C.S = S;
        C.H = H;
        C.len = (int64_t)fwd.dk * fwd.dv;
        C.lam = lam;
        C.init = state;
        C.states = base;
        C.w = base + sb;
        if ((e = carry_run(dt, &C, 1, st)) != cudaSuccess) return e;
        P.R.state_in = base;
        P.R.in_by_slot = 1;
        P.w_in = base + sb;
    }
    P.dout = dout;
    P.dstate = dstate;
    e = with_type(dt, [&](auto t) { return rec_dim<decltype(t), 2, true>(P, S.seg <= S.T, st); });
    if (e != cudaSuccess) return e;
    const bool next = S.slots > 0;  // (without a sequence no kernel ran)
    return dt == LAPLEX_F64 ? launch(next, k_dlam_join<double>, H, 256, 0, st, P.part, (int64_t)S.slots, H, cb, (double*)dlam)
                            : launch(next, k_dlam_join<float>, H, 256, 0, st, P.part, (int64_t)S.slots, H, cb, (float*)dlam);
}

}  // namespace lx
