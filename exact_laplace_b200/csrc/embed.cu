// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
// In the limit of small temperature the kernel exp(-|a_i - b_j| / t) becomes the
// routing [a_i == b_j] (summary §2.1): the lookup is K x with the tokens as a
// and the rows' numbers as b, the gradient is K^T g.
//     out_i = scale table[token_i]
//     dtable_r = scale sum over {i: token_i = r}, i ascending, of g_i
// A token outside [0, rows) has a row of zeros and no gradient.
//
// Lookup: bound by memory, each row read and written once; a warp moves pieces
// of 32 lanes x 16 bytes x 4, all four loads in flight.
//
// Gradient: the tokens are sorted with their positions, which turns the gradient
// into sums over runs.  Adding rows into the table with atomics would need fp32
// atomics on every value, a pass of rounding for 16-bit tables, and would change
// from run to run.
//   k_token_sort (up to 65536 tokens): one cluster of up to 8 blocks keeps the
//     tokens in its shared memory through the stable digit passes and scatters
//     through distributed shared memory; one launch in place of seven to ten.  The
//     other SMs zero a part of the table meanwhile.  More tokens take the digit passes
//     of sort.cu.
//   k_embed_sum: a warp takes R consecutive sorted positions and 32 lanes x 16
//     bytes of columns, reads the rows of g (16 to 32 in flight), sums in fp32 in
//     position order, and writes the rows whose run lies inside its R positions.
//     A run that crosses a boundary by up to 16 positions belongs to the warp before
//     it; a longer one leaves one partial sum per side.  Blocks that
//     zero the other rows without a token, by a bitmap of the tokens that occur, lie
//     between them, so that reads and writes overlap (write-only traffic ran at
//     3.8 TB/s).
//   k_embed_join: the partial sums of the long runs, which k_embed_sum lists, in a
//     fixed order: a warp to 32 lanes x 16 bytes of a run, eight where it has many parts.
#include <algorithm>

#include "devcache.h"
#include "elem.cuh"
#include "seqop.h"

namespace lx {

constexpr int EMB_NT = 256;
constexpr int EMB_U = 4;  // 16-byte pieces of a row per lane

template <typename T, int VN>
__global__ void __launch_bounds__(EMB_NT) k_embed(const __grid_constant__ EmbedArgs P) {
    using A = typename AccOf<T>::A;
    using V = Pack<T, VN>;
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * (EMB_NT / 32) + (threadIdx.x >> 5);
    if (i >= P.n) return;
    const int64_t tok = P.tok64 ? static_cast<const int64_t*>(P.tokens)[i] : (int64_t)static_cast<const int32_t*>(P.tokens)[i];
    const bool known = tok >= 0 && tok < P.rows;
    const A scale = (A)P.scale;
    T* dst = static_cast<T*>(P.dst) + i * P.dst_ld;
    const T* src = static_cast<const T*>(P.src) + (known ? tok : 0) * P.src_ld;
    for (int64_t c0 = (int64_t)blockIdx.y * (32 * VN * EMB_U); c0 < P.dim; c0 += (int64_t)gridDim.y * (32 * VN * EMB_U)) {
        V v[EMB_U];
#pragma unroll
        for (int u = 0; u < EMB_U; ++u) {
            const int64_t c = c0 + (u * 32 + lane) * VN;
#pragma unroll
            for (int e = 0; e < VN; ++e) v[u].v[e] = from_acc<T, A>((A)0);
            if (known && c < P.dim) v[u] = *reinterpret_cast<const V*>(src + c);
        }
#pragma unroll
        for (int u = 0; u < EMB_U; ++u) {
            const int64_t c = c0 + (u * 32 + lane) * VN;
            if (known)
#pragma unroll
                for (int e = 0; e < VN; ++e) v[u].v[e] = from_acc<T, A>(to_acc<A, T>(v[u].v[e]) * scale);
            if (c < P.dim) *reinterpret_cast<V*>(dst + c) = v[u];
        }
    }
}

static bool vec_ok(const EmbedArgs& A, int VN, size_t src_es, size_t dst_es, int dst_vb) {
    return A.dim % VN == 0 && (A.src_ld * src_es) % 16 == 0 && (A.dst_ld * dst_es) % dst_vb == 0;
}

template <typename T>
static cudaError_t embed_launch(const EmbedArgs& A, cudaStream_t st) {
    constexpr int VN = VecOf<T>::N;
    const bool vec = vec_ok(A, VN, sizeof(T), sizeof(T), 16);
    const int64_t piece = 32 * EMB_U * (vec ? VN : 1);
    const dim3 grid((unsigned)((A.n + EMB_NT / 32 - 1) / (EMB_NT / 32)),
                    (unsigned)std::min<int64_t>((A.dim + piece - 1) / piece, 65535));
    if (vec) k_embed<T, VN><<<grid, EMB_NT, 0, st>>>(A);
    else k_embed<T, 1><<<grid, EMB_NT, 0, st>>>(A);
    return cudaGetLastError();
}

cudaError_t embed_run(laplex_dtype dt, const EmbedArgs& A, cudaStream_t st) {
    if (A.n == 0 || A.dim == 0) return cudaSuccess;
    switch (dt) {
        case LAPLEX_F32: return embed_launch<float>(A, st);
        case LAPLEX_F64: return embed_launch<double>(A, st);
        case LAPLEX_F16: return embed_launch<__half>(A, st);
        case LAPLEX_BF16: return embed_launch<__nv_bfloat16>(A, st);
    }
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------- gradient

// sort keys of the tokens (one outside [0, rows): rows, which sorts last), and
// the bitmap of the rows that occur
__device__ __forceinline__ int64_t token_at(const void* tokens, int tok64, int64_t i) {
    return tok64 ? static_cast<const int64_t*>(tokens)[i] : (int64_t)static_cast<const int32_t*>(tokens)[i];
}

__global__ void __launch_bounds__(256) k_embed_keys(const void* tokens, int tok64, int64_t n, int64_t rows,
                                                    uint32_t* __restrict__ keys, uint32_t* __restrict__ seen,
                                                    uint32_t* __restrict__ counts) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < 2) counts[i] = 0;
    if (i >= n) return;
    const int64_t tok = token_at(tokens, tok64, i);
    const bool known = tok >= 0 && tok < rows;
    keys[i] = known ? (uint32_t)tok : (uint32_t)rows;
    if (known && seen) atomicOr(seen + (tok >> 5), 1u << (tok & 31));  // an or: the order does not matter
}

// ---- up to TS_MAX tokens: one cluster
constexpr int TS_NT = 512, TS_NW = TS_NT / 32, TS_CAP = 8192, TS_MAX = 8 * TS_CAP, TS_BINS = 1024;

struct TokenSort {
    const void* tokens;
    int tok64;
    int n, shift;      // a block holds 1 << shift tokens
    int64_t rows;
    int passes, bits;  // digits of `bits` bits
    uint32_t* skeys;
    int32_t* perm;
    uint32_t* seen;    // or NULL
    int64_t words;     // of seen
    uint32_t* counts;  // two, set to 0 for k_embed_sum
    int blocks;        // of the sort; the others zero rows of the table
    unsigned char* zero;
    int64_t zero_rows, zero_bytes, zero_ld;  // bytes of a row, and from row to row: multiples of 16
};

struct TokenSortShared {
    uint2 pair[2][TS_CAP];         // key, position
    uint32_t cnt[TS_NW][TS_BINS];  // per warp: counts, then the earlier warps' counts and the smaller digits'
    uint32_t hist[TS_BINS];        // this block's counts, read by the whole cluster
    uint32_t hist2[TS_BINS];       // where a digit starts in this block's order
    uint32_t delta[TS_BINS];       // from a place in this block's order to the one in the cluster's
    uint32_t wsum[2][TS_NW];
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_remote(uint32_t a, uint2 v) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}

// Stable LSD passes.  Block b holds the positions b << shift .. of the current
// order, each warp a contiguous part; a key's place is the count of smaller digits
// in the cluster, of its digit in earlier blocks, in earlier warps of its block,
// and before it in its warp.
__global__ void __launch_bounds__(TS_NT) k_token_sort(const __grid_constant__ TokenSort P) {
    extern __shared__ __align__(16) unsigned char raw[];
    TokenSortShared& sh = *reinterpret_cast<TokenSortShared*>(raw);
    after_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int me = blockIdx.x, blocks = P.blocks;  // the first cluster
    if (me >= blocks) {
        const int64_t w = (int64_t)(me - blocks) * TS_NW + warp, all = (int64_t)(gridDim.x - blocks) * TS_NW;
        for (int64_t r = w; r < P.zero_rows; r += all)
            for (int64_t c = lane * 16; c < P.zero_bytes; c += 512)
                *reinterpret_cast<uint4*>(P.zero + r * P.zero_ld + c) = make_uint4(0, 0, 0, 0);
        return;
    }
    const int lo = me << P.shift, count = max(0, min(1 << P.shift, P.n - lo));
    const int bins = 1 << P.bits;
    if (P.seen)
        for (int64_t i = (int64_t)me * TS_NT + tid; i < P.words; i += (int64_t)blocks * TS_NT) P.seen[i] = 0;
    if (me == 0 && tid < 2) P.counts[tid] = 0;
    cluster_sync();  // the bitmap is clear (and every block of the cluster runs)
    for (int i = tid; i < count; i += TS_NT) {
        const int64_t tok = token_at(P.tokens, P.tok64, lo + i);
        const bool known = tok >= 0 && tok < P.rows;
        sh.pair[0][i] = make_uint2(known ? (uint32_t)tok : (uint32_t)P.rows, (uint32_t)(lo + i));
    }
    const int per = ((1 << P.shift) / TS_NW + 31) / 32 * 32;  // positions of a warp
    const int w0 = warp * per, w1 = min(count, w0 + per);
    for (int pass = 0; pass < P.passes; ++pass) {
        const uint2* pair = sh.pair[pass & 1];
        const int down = P.bits * pass;
        for (int i = lane; i < bins; i += 32) sh.cnt[warp][i] = 0;
        __syncthreads();
        // ranks in the warp; the pairs move to registers
        uint32_t rank[TS_CAP / TS_NT];
        uint2 v[TS_CAP / TS_NT];
#pragma unroll
        for (int r = 0; r < TS_CAP / TS_NT; ++r) {
            const int i = w0 + r * 32 + lane;
            if (w0 + r * 32 >= w1) break;
            const bool in = i < w1;
            v[r] = in ? pair[i] : make_uint2(0, 0);
            const uint32_t d = in ? v[r].x >> down & (bins - 1) : TS_BINS;
            // the lanes with this digit, a ballot per bit (a warp match takes a step per distinct digit)
            uint32_t same = __ballot_sync(FULL, in);
            for (int k = 0; k < P.bits; ++k) {
                const bool bit = d >> k & 1;
                const uint32_t m = __ballot_sync(FULL, bit);
                same &= bit ? m : ~m;
            }
            const uint32_t before = in ? sh.cnt[warp][d] : 0;
            rank[r] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (in && lane == 31 - __clz(same)) sh.cnt[warp][d] = rank[r] + 1;
            __syncwarp();
        }
        __syncthreads();
        for (int d = tid; d < bins; d += TS_NT) {
            uint32_t s = 0;
#pragma unroll
            for (int w = 0; w < TS_NW; ++w) {
                const uint32_t c = sh.cnt[w][d];
                sh.cnt[w][d] = s;
                s += c;
            }
            sh.hist[d] = s;
        }
        cluster_sync();
        // exclusive sums over the digits (a warp takes bins / 16 consecutive ones) of the cluster's
        // and of this block's counts; the first plus the earlier blocks' is where a digit goes
        const int span = max(1, bins / TS_NW);
        uint32_t sum = 0, own = 0;
        for (int x = 0; x < span; x += 32) {
            const int d = warp * span + x + lane;
            const bool in = x + lane < span && d < bins;
            uint32_t mine = 0, all = 0, here = 0;
            if (in) {
                uint32_t c[8];
#pragma unroll
                for (int b = 0; b < 8; ++b) c[b] = b < blocks ? ld_remote(remote(&sh.hist[d], b)) : 0;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    if (b < me) mine += c[b];
                    if (b == me) here = c[b];
                    all += c[b];
                }
            }
            uint32_t sa = all, so = here;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t p = __shfl_up_sync(FULL, sa, o), q = __shfl_up_sync(FULL, so, o);
                if (lane >= o) {
                    sa += p;
                    so += q;
                }
            }
            if (in) {
                sh.delta[d] = (sum + sa - all + mine) - (own + so - here);
                sh.hist2[d] = own + so - here;
            }
            sum += __shfl_sync(FULL, sa, 31);
            own += __shfl_sync(FULL, so, 31);
        }
        if (lane == 0) {
            sh.wsum[0][warp] = sum;
            sh.wsum[1][warp] = own;
        }
        __syncthreads();
        uint32_t lead = 0, mylead = 0;
        for (int w = 0; w < warp; ++w) {
            lead += sh.wsum[0][w];
            mylead += sh.wsum[1][w];
        }
        for (int x = lane; x < span; x += 32)
            if (warp * span + x < bins) {
                sh.delta[warp * span + x] += lead - mylead;
                sh.hist2[warp * span + x] += mylead;
            }
        __syncthreads();
        // into this block's order first: scattered writes of single pairs to other blocks, and of
        // single words to device memory, take a cycle each (38 us for 65536 tokens, 19 a pass)
        uint2* order = sh.pair[pass & 1];
#pragma unroll
        for (int r = 0; r < TS_CAP / TS_NT; ++r) {
            if (w0 + r * 32 + lane >= w1) break;
            const uint32_t d = v[r].x >> down & (bins - 1);
            order[sh.hist2[d] + sh.cnt[warp][d] + rank[r]] = v[r];
        }
        __syncthreads();
        const bool last = pass == P.passes - 1;
        for (int i = tid; i < count; i += TS_NT) {
            const uint2 x = order[i];
            const uint32_t at = i + sh.delta[x.x >> down & (bins - 1)];
            if (last) {
                P.skeys[at] = x.x;
                P.perm[at] = (int32_t)x.y;
                // once per run and block (equal keys lie together): atomics on the word of a frequent
                // token, one per occurrence, took a third of the kernel
                if (P.seen && x.x != (uint32_t)P.rows && (i == 0 || order[i - 1].x != x.x))
                    atomicOr(P.seen + (x.x >> 5), 1u << (x.x & 31));
            } else
                st_remote(remote(&sh.pair[~pass & 1][at & ((1u << P.shift) - 1)], at >> P.shift), x);
        }
        cluster_sync();  // the keys have arrived (and no block leaves while its memory is read)
    }
}

// Rows of the table that the sort's launch zeroes on the SMs beside its cluster: as many as its time (9 us for
// 4000 tokens, 31 for 65536, in the two digits of 1024 to 2^20 rows) lets write at 3.5 TB/s.  (The sort alone,
// in one, two and three digits: 7.4, 10.2, 12.5 us for 4000 tokens, 17, 29, 39 for 65536.  The line is for two:
// a table of one digit is mostly zeroed as a whole, one of three leaves a fifth of the time unused.)  Rows with
// a token are written again by the sums; the others are left to k_embed_sum's blocks.  (All of them there: 197 us
// for 65536 tokens and 131072 rows of 2048 bf16 values, 26.5 for 4000 and 8192 of 520 fp32; so 189 and 24.5.)
static int64_t zeroed_early(const EmbedArgs& A, int64_t es) {
    const int64_t bytes = A.dim * es;
    if (A.accumulate || bytes % 16 != 0 || (A.rows > 1 && A.dst_ld * es % 16 != 0)) return 0;
    const double budget = (8.0 + 0.00035 * (double)A.n) * 3.5e6;
    const int64_t rows = (int64_t)(budget / (double)bytes) / 32 * 32;
    return rows >= A.rows ? A.rows : rows;
}

static cudaError_t token_sort(const EmbedArgs& A, uint32_t* skeys, int32_t* perm, uint32_t* seen, uint32_t* counts,
                              int64_t zero_rows, int64_t es, cudaStream_t st) {
    TokenSort P;
    P.tokens = A.tokens;
    P.tok64 = A.tok64;
    P.n = (int)A.n;
    P.rows = A.rows;
    P.skeys = skeys;
    P.perm = perm;
    P.seen = seen;
    P.words = (A.rows + 31) / 32;
    P.counts = counts;
    P.zero = static_cast<unsigned char*>(A.dst);
    P.zero_rows = zero_rows;
    P.zero_bytes = A.dim * es;
    P.zero_ld = A.dst_ld * es;
    int bits = 1;
    while (bits < 31 && (A.rows >> bits) != 0) ++bits;
    P.passes = (bits + 9) / 10;  // as few as 1024 digits allow
    P.bits = (bits + P.passes - 1) / P.passes;
    P.shift = 10;  // from 1024 tokens a block: fewer leave most of its warps idle
    while (((int64_t)8 << P.shift) < A.n) ++P.shift;
    const unsigned blocks = (unsigned)((A.n + (1 << P.shift) - 1) >> P.shift);
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e == cudaSuccess) e = blocks_per_sm<&k_token_sort>(dev, TS_NT, sizeof(TokenSortShared), &per);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    P.blocks = (int)blocks;
    const unsigned more = zero_rows ? std::max(1, (sms - (int)blocks) / (int)blocks) : 0;  // clusters
    cfg.gridDim = dim3(blocks * (1 + more));
    cfg.blockDim = dim3(TS_NT);
    cfg.dynamicSmemBytes = sizeof(TokenSortShared);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_token_sort, P);
}

struct EmbedSum {
    EmbedArgs A;
    const uint32_t* keys;   // sorted
    const int32_t* perm;
    const uint32_t* seen;
    void* part;             // [tiles][2][dim]: sums of the runs that enter / leave a tile
    int64_t tiles;
    int R;                  // sorted positions per tile
    int32_t* list;          // [2][tiles]: tiles in which a long run begins; those of many parts
    uint32_t* counts;       // of both
    int64_t sum_blocks, zero_blocks;  // blocks of the sums, and those that zero the rows without a token
    int64_t zero_from;                // from this row on (a multiple of 8)
};

template <typename T, typename W, int VN>
__device__ __forceinline__ void embed_write(const EmbedArgs& A, int64_t row, int64_t c, const typename AccOf<T>::A* s) {
    using Ac = typename AccOf<T>::A;
    using AW = typename AccOf<W>::A;
    W* p = static_cast<W*>(A.dst) + row * A.dst_ld + c;
    Pack<W, VN> o;
    if (A.accumulate) o = *reinterpret_cast<const Pack<W, VN>*>(p);
#pragma unroll
    for (int e = 0; e < VN; ++e) {
        Ac v = s[e] * (Ac)A.scale;
        if (A.accumulate) v += (Ac)to_acc<AW, W>(o.v[e]);
        o.v[e] = from_acc<W, AW>((AW)v);
    }
    *reinterpret_cast<Pack<W, VN>*>(p) = o;
}

// Whether the run across position p (a tile's start) is long, that is, reaches more than SUM_H
// positions past p: its parts are joined later.  A short one belongs to the tile before p, and
// *end is where it ends (p: no run crosses).
constexpr int SUM_H = 16;
__device__ __forceinline__ bool border(const uint32_t* keys, int64_t p, int64_t n, int lane, int64_t* end) {
    *end = min(p, n);
    if (p <= 0 || p >= n) return false;
    const uint32_t k = keys[p - 1];
    const bool same = lane <= SUM_H && p + lane < n && keys[p + lane] == k;
    const int run = __ffs(~__ballot_sync(FULL, same)) - 1;  // (lane 31 never has it)
    *end = p + run;
    return run > SUM_H;
}

constexpr int SUM_NT = 128;
constexpr int MANY = 16;  // parts of a run that one warp joins

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// VN > 1: rows come through a ring in shared memory by asynchronous copies, 16 in flight
// while 16 are summed (a lane reads only what it copied).  Loads into registers, eight
// at a time, left the latency of each round in the open (1.5 TB/s).
template <typename T, typename W, int VN>
__global__ void __launch_bounds__(SUM_NT) k_embed_sum(const __grid_constant__ EmbedSum P) {
    using A = typename AccOf<T>::A;
    constexpr bool RING = VN > 1;
    constexpr int NW = SUM_NT / 32;
    extern __shared__ __align__(16) unsigned char raw[];
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const EmbedArgs& E = P.A;
    // the zeroing blocks lie evenly between the others: block b is the (b zero / all)-th of them
    const int64_t all = P.sum_blocks + P.zero_blocks, b = blockIdx.x;
    const int64_t z = b * P.zero_blocks / all, z1 = (b + 1) * P.zero_blocks / all;
    if (z1 > z) {
        // a warp takes 8 rows at a time
        Pack<W, VN> o;
#pragma unroll
        for (int e = 0; e < VN; ++e) o.v[e] = from_acc<W, typename AccOf<W>::A>(0);
        for (int64_t r = P.zero_from + (z * NW + warp) * 8; r < E.rows; r += P.zero_blocks * NW * 8) {
            const uint32_t word = P.seen[r >> 5] >> (r & 31);
            for (int k = 0; k < 8 && r + k < E.rows; ++k) {
                if (word >> k & 1) continue;
                W* p = static_cast<W*>(E.dst) + (r + k) * E.dst_ld;
                for (int64_t c = lane * VN; c < E.dim; c += 32 * VN) *reinterpret_cast<Pack<W, VN>*>(p + c) = o;
            }
        }
        return;
    }
    const int64_t cols = (E.dim + 32 * VN - 1) / (32 * VN);
    const int64_t w = (b - z) * NW + warp;
    const int64_t tile = w / cols;
    if (tile >= P.tiles) return;
    const int64_t c = ((w - tile * cols) * 32 + lane) * VN;
    int64_t p0 = tile * P.R, p1 = p0 + P.R, e0, e1;
    bool entered = border(P.keys, p0, E.n, lane, &e0);  // the run began in an earlier tile
    const bool leaves = border(P.keys, p1, E.n, lane, &e1);
    if (!entered) p0 = e0;
    p1 = leaves ? p1 : e1;
    if (p0 >= p1) return;
    // A key or position outside its range counts as no token: a sort whose wait ran out (ST_TIMEOUT) leaves
    // what was in the workspace before.
    const uint32_t none = (uint32_t)E.rows;
    const bool in = c < E.dim;
    A s[VN];
#pragma unroll
    for (int e = 0; e < VN; ++e) s[e] = 0;
    uint32_t cur = min(P.keys[p0], none);
    A* part = static_cast<A*>(P.part) + tile * 2 * E.dim + c;
    Pack<T, VN>* ring = reinterpret_cast<Pack<T, VN>*>(raw) + warp * 2 * SUM_H * 32 + lane;
    const T* src = static_cast<const T*>(E.src) + c;
    const int halves = (int)((p1 - p0 + SUM_H - 1) / SUM_H);
    // a lane's key and row of the half being copied
    uint32_t key_of[2] = {none, none};
    int32_t row_of[2] = {0, 0};
    const auto fetch = [&](int h, uint32_t& k, int32_t& i) {
        const int64_t p = p0 + (int64_t)h * SUM_H + lane;
        const bool has = lane < SUM_H && h < halves && p < p1;
        k = has ? P.keys[p] : none;
        i = has ? P.perm[p] : 0;
    };
    const auto start = [&](int h, uint32_t k, int32_t i) {
        if constexpr (RING) {
#pragma unroll 4
            for (int u = 0; u < SUM_H; ++u) {
                const uint32_t key = __shfl_sync(FULL, k, u);
                const int64_t row = __shfl_sync(FULL, i, u);
                if (in && key != none) copy16(ring + ((h & 1) * SUM_H + u) * 32, src + row * E.src_ld);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    // (where the values are used first, not where they are loaded: 179 us against 193 for 65536 Zipf tokens, 2048 columns)
    const auto limit = [&](uint32_t& k, int32_t i) { k = (uint32_t)i < (uint32_t)E.n ? min(k, none) : none; };
    fetch(0, key_of[0], row_of[0]);
    limit(key_of[0], row_of[0]);
    start(0, key_of[0], row_of[0]);
    fetch(1, key_of[1], row_of[1]);
    for (int h = 0; h < halves; ++h) {
        const uint32_t mykey = key_of[0];
        const int32_t myrow = row_of[0];
        limit(key_of[1], row_of[1]);
        start(h + 1, key_of[1], row_of[1]);
        key_of[0] = key_of[1];
        row_of[0] = row_of[1];
        fetch(h + 2, key_of[1], row_of[1]);
        if constexpr (RING) asm volatile("cp.async.wait_group 1;" ::: "memory");
        const int m = (int)min((int64_t)SUM_H, p1 - p0 - (int64_t)h * SUM_H);
#pragma unroll 2
        for (int u = 0; u < m; ++u) {
            const uint32_t key = __shfl_sync(FULL, mykey, u);
            const int64_t row = __shfl_sync(FULL, myrow, u);
            if (key != cur) {
                if (in && cur != none) {
                    if (entered) {
#pragma unroll
                        for (int e = 0; e < VN; ++e) part[e] = s[e];
                    } else embed_write<T, W, VN>(E, cur, c, s);
                }
#pragma unroll
                for (int e = 0; e < VN; ++e) s[e] = 0;
                cur = key;
                entered = false;
            }
            if (in && cur != none) {
                Pack<T, VN> v;
                if constexpr (RING) v = ring[((h & 1) * SUM_H + u) * 32];
                else v = *reinterpret_cast<const Pack<T, VN>*>(src + row * E.src_ld);
#pragma unroll
                for (int e = 0; e < VN; ++e) s[e] += to_acc<A, T>(v.v[e]);
            }
        }
    }
    if (!in || cur == none) return;
    if (entered) {
#pragma unroll
        for (int e = 0; e < VN; ++e) part[e] = s[e];
    } else if (leaves) {
#pragma unroll
        for (int e = 0; e < VN; ++e) part[E.dim + e] = s[e];
        if (c == 0) {  // for the join, in any order: each run has its own row
            const int64_t far = p1 + (int64_t)(MANY - 1) * P.R + SUM_H;
            const int many = far < E.n && P.keys[far] == cur;
            P.list[many * P.tiles + atomicAdd(P.counts + many, 1u)] = (int32_t)tile;
        }
    } else embed_write<T, W, VN>(E, cur, c, s);
}

// The long runs: part 0 is the one of the end of the tile where the run begins, part
// i > 0 the one of the start of the i-th tile after it.  Runs of up to MANY parts take
// a warp for each 32 VN columns; longer ones a block, whose warps sum an eighth of
// the parts each, in order, and are joined in order.  (Found by a search over all
// tiles' borders, a block to a run: 210 us for the gradient of 65536 Zipf tokens, 2048
// columns, 170 such runs; so 197.)
template <typename T, typename W, int VN>
__global__ void __launch_bounds__(EMB_NT) k_embed_join(const __grid_constant__ EmbedSum P) {
    using A = typename AccOf<T>::A;
    constexpr int NW = EMB_NT / 32;
    __shared__ __align__(16) A red[NW][32 * VN];
    after_previous();
    const EmbedArgs& E = P.A;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t pieces = (E.dim + 32 * VN - 1) / (32 * VN);
    const int64_t few = P.counts[0] * pieces, many = P.counts[1] * pieces;
    // the run that begins in `tile`: its key and parts (by a whole warp).  (k_embed_sum lists a tile only by a key
    // of a row; keys that do not ascend give other parts, but no tile past the last.)
    const auto find = [&](int64_t tile, uint32_t* key) -> int64_t {
        const uint32_t k = P.keys[(tile + 1) * P.R - 1];
        *key = k;
        const auto enters = [&](int64_t t) {  // (long at its start; ascending keys: true up to the last such tile)
            const int64_t p = t * P.R + SUM_H;
            return p < E.n && P.keys[p] == k;
        };
        int64_t end = tile + 1;  // all tiles between are entered
        for (;;) {
            const int n = __popc(__ballot_sync(FULL, enters(end + lane * 32)));
            if (n == 0) break;
            end += (n - 1) * 32 + 1;
            if (n < 32) {
                end += __popc(__ballot_sync(FULL, enters(end + lane)));
                break;
            }
        }
        return end - tile;
    };
    const auto sum = [&](int64_t tile, int64_t a0, int64_t a1, int64_t c, A(&s)[VN]) {
        const A* part = static_cast<const A*>(P.part) + tile * 2 * E.dim + c;
#pragma unroll
        for (int e = 0; e < VN; ++e) s[e] = 0;
#pragma unroll 8
        for (int64_t i = a0; i < a1; ++i) {
            const Pack<A, VN> v = *reinterpret_cast<const Pack<A, VN>*>(part + (i == 0 ? E.dim : i * 2 * E.dim));
#pragma unroll
            for (int e = 0; e < VN; ++e) s[e] += v.v[e];
        }
    };
    for (int64_t x = blockIdx.x; x < many; x += gridDim.x) {
        const int64_t tile = P.list[P.tiles + x / pieces], cb = x % pieces * 32 * VN, c = cb + lane * VN;
        uint32_t key;
        const int64_t parts = find(tile, &key);
        A s[VN];
        if (c < E.dim) {
            sum(tile, parts * warp / NW, parts * (warp + 1) / NW, c, s);
#pragma unroll
            for (int e = 0; e < VN; ++e) red[warp][lane * VN + e] = s[e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * VN; i += EMB_NT) {
            if (cb + i >= E.dim) break;
            A t = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) t += red[w][i];
            embed_write<T, W, 1>(E, key, cb + i, &t);
        }
        __syncthreads();
    }
    // (from the last block on: the first ones have the long runs)
    for (int64_t x = (int64_t)(gridDim.x - 1 - blockIdx.x) * NW + warp; x < few; x += (int64_t)gridDim.x * NW) {
        const int64_t tile = P.list[x / pieces], c = x % pieces * 32 * VN + lane * VN;
        uint32_t key;
        const int64_t parts = find(tile, &key);
        if (c >= E.dim) continue;
        A s[VN];
        sum(tile, 0, parts, c, s);
#pragma unroll
        for (int e = 0; e < VN; ++e) embed_write<T, W, 1>(E, key, c + e, &s[e]);
    }
}

// Positions per tile: enough warps to fill the GPU (148 SMs x 64), between 16 and
// 256 (the partial sums of a tile are two rows of fp32, against R rows read).
// Twice the warps: 193 us against 183 for 65536 tokens of 2048 columns, 132 against
// 118 of 1024; a quarter: 205 and 122.
static int embed_tile(int64_t n, int64_t dim, int es) {
    const int64_t cols = std::max<int64_t>(1, (dim * es + 511) / 512);
    int64_t R = 16;
    while (R < 256 && n * cols / R > 148 * 64) R *= 2;
    return (int)R;
}

struct EmbedWs {
    size_t keys, skeys, perm, seen, part, list, sort;
    size_t all() const { return keys + skeys + perm + seen + part + list + sort; }
};
static EmbedWs embed_ws(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt) {
    EmbedWs W;
    const int64_t tiles = (n + embed_tile(n, dim, (int)elem_bytes(dt)) - 1) / embed_tile(n, dim, (int)elem_bytes(dt));
    W.keys = Carve::need((size_t)n, 4);
    W.skeys = Carve::need((size_t)n, 4);
    W.perm = Carve::need((size_t)n, 4);
    W.seen = Carve::need((size_t)((rows + 31) / 32), 4);
    W.part = Carve::need((size_t)(tiles * 2 * dim), acc_bytes(dt));
    W.list = Carve::need((size_t)(2 * tiles + 2), 4);
    W.sort = n <= TS_MAX ? 0 : sort_keys_ws_bytes(n);
    return W;
}

size_t embed_bwd_ws_bytes(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt) {
    return embed_ws(n, rows, dim, dt).all();
}

template <typename T, typename W>
static cudaError_t embed_sum_launch(EmbedSum S, int sms, bool sorted, cudaStream_t st) {
    constexpr int VN = VecOf<T>::N;
    const bool vec = vec_ok(S.A, VN, sizeof(T), sizeof(W), std::min<int>(16, VN * sizeof(W)));
    const int64_t cols = (S.A.dim + 32 * (vec ? VN : 1) - 1) / (32 * (vec ? VN : 1));
    constexpr int NW = SUM_NT / 32;
    S.sum_blocks = (S.tiles * cols + NW - 1) / NW;
    S.zero_blocks = S.A.accumulate ? 0 : std::min<int64_t>((S.A.rows - S.zero_from + 8 * NW - 1) / (8 * NW), 16 * (int64_t)sms);
    const int64_t grid = S.sum_blocks + S.zero_blocks;
    if (grid > 0) {
        constexpr size_t ring = (size_t)NW * 2 * SUM_H * 32 * 16;
        int dev = 0, per = 0, n = 0;
        cudaError_t e = current_device_sms(&dev, &n);
        if (e == cudaSuccess) e = blocks_per_sm<&k_embed_sum<T, W, VN>>(dev, SUM_NT, ring, &per);
        if (e != cudaSuccess) return e;
        e = vec ? launch(sorted, k_embed_sum<T, W, VN>, (unsigned)grid, SUM_NT, ring, st, S)
                : launch(sorted, k_embed_sum<T, W, 1>, (unsigned)grid, SUM_NT, 0, st, S);
        if (e != cudaSuccess) return e;
    }
    if (S.tiles > 1) {
        constexpr int JN = 16 / (int)sizeof(typename AccOf<T>::A);
        const bool jvec = S.A.dim % JN == 0;
        const int64_t jcols = (S.A.dim + 32 * (jvec ? JN : 1) - 1) / (32 * (jvec ? JN : 1));
        const unsigned jg = (unsigned)std::min<int64_t>((S.tiles * jcols + EMB_NT / 32 - 1) / (EMB_NT / 32), 4 * (int64_t)sms);
        return jvec ? launch(true, k_embed_join<T, W, JN>, jg, EMB_NT, 0, st, S)
                    : launch(true, k_embed_join<T, W, 1>, jg, EMB_NT, 0, st, S);
    }
    return cudaSuccess;
}

cudaError_t embed_bwd_run(laplex_dtype dt, laplex_dtype out_dt, const EmbedArgs& A, void* ws, size_t ws_bytes,
                          uint32_t* status, cudaStream_t st) {
    if (A.dim == 0 || (A.rows == 0)) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const EmbedWs Z = embed_ws(A.n, A.rows, A.dim, dt);
    if (ws_bytes < Z.all()) return cudaErrorInvalidValue;
    char* p = static_cast<char*>(ws);
    uint32_t* keys = (uint32_t*)p;
    uint32_t* skeys = (uint32_t*)(p += Z.keys);
    int32_t* perm = (int32_t*)(p += Z.skeys);
    uint32_t* seen = (uint32_t*)(p += Z.perm);
    void* part = p += Z.seen;
    int32_t* list = (int32_t*)(p += Z.part);
    void* sort = p += Z.list;
    const int R = embed_tile(A.n, A.dim, (int)elem_bytes(dt));
    const int64_t tiles = (A.n + R - 1) / R;
    uint32_t* counts = (uint32_t*)list + 2 * tiles;
    const bool sorted = A.n > 0 && A.n <= TS_MAX;  // by a kernel of this call
    const int64_t es = out_dt == LAPLEX_F64 ? 8 : out_dt == LAPLEX_F32 ? 4 : 2;
    const int64_t early = sorted ? zeroed_early(A, es) : 0;
    uint32_t* bits = A.accumulate || early == A.rows ? nullptr : seen;
    if (sorted) {
        e = token_sort(A, skeys, perm, bits, counts, early, es, st);
        if (e != cudaSuccess) return e;
    } else {
        if (bits) e = cudaMemsetAsync(seen, 0, (size_t)((A.rows + 31) / 32) * 4, st);
        if (e == cudaSuccess && A.n > 0) {
            k_embed_keys<<<(unsigned)((A.n + 255) / 256), 256, 0, st>>>(A.tokens, A.tok64, A.n, A.rows, keys, bits, counts);
            e = cudaGetLastError();
            if (e == cudaSuccess)
                e = sort_keys_run(keys, A.n, (uint32_t)A.rows, skeys, perm, sort, Z.sort, status, st);
        }
        if (e != cudaSuccess) return e;
    }
    EmbedSum S;
    S.A = A;
    S.keys = skeys;
    S.perm = perm;
    S.seen = seen;
    S.part = part;
    S.R = R;
    S.tiles = tiles;
    S.list = list;
    S.counts = counts;
    S.sum_blocks = S.zero_blocks = 0;
    S.zero_from = early;
    const bool f32 = out_dt == LAPLEX_F32;
    switch (dt) {
        case LAPLEX_F32: return embed_sum_launch<float, float>(S, sms, sorted, st);
        case LAPLEX_F64: return embed_sum_launch<double, double>(S, sms, sorted, st);
        case LAPLEX_F16: return f32 ? embed_sum_launch<__half, float>(S, sms, sorted, st) : embed_sum_launch<__half, __half>(S, sms, sorted, st);
        case LAPLEX_BF16:
            return f32 ? embed_sum_launch<__nv_bfloat16, float>(S, sms, sorted, st)
                       : embed_sum_launch<__nv_bfloat16, __nv_bfloat16>(S, sms, sorted, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lx
