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
// Gradient: the tokens are sorted with their positions (sort.cu), which turns
// the gradient into sums over runs.  Adding rows into the table with atomics
// would need fp32 atomics on every value, a pass of rounding for 16-bit tables,
// and would change from run to run.  k_embed_sum gives each warp R consecutive
// sorted positions and 32 lanes x 16 bytes of columns: it reads the rows of g
// (the next rows' loads in flight), sums in fp32 in position order, and writes
// the rows whose run lies inside its R positions.  A run that crosses a boundary
// leaves one partial sum per side, joined in order by k_embed_join.  Rows
// without a token are zeroed by further blocks of the same launch, from a bitmap
// of the tokens that occur, so that each row of the table is written once.
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
__global__ void __launch_bounds__(256) k_embed_keys(const void* tokens, int tok64, int64_t n, int64_t rows,
                                                    uint32_t* __restrict__ keys, uint32_t* __restrict__ seen) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t tok = tok64 ? static_cast<const int64_t*>(tokens)[i] : (int64_t)static_cast<const int32_t*>(tokens)[i];
    const bool known = tok >= 0 && tok < rows;
    keys[i] = known ? (uint32_t)tok : (uint32_t)rows;
    if (known && seen) atomicOr(seen + (tok >> 5), 1u << (tok & 31));  // an or: the order does not matter
}

struct EmbedSum {
    EmbedArgs A;
    const uint32_t* keys;   // sorted
    const int32_t* perm;
    const uint32_t* seen;
    void* part;             // [tiles][2][dim]: sums of the runs that enter / leave a tile
    int64_t tiles;
    int R;                  // sorted positions per tile
    int64_t sum_blocks;     // blocks of the sums; the rest zero the rows without a token
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

template <typename T, typename W, int VN>
__global__ void __launch_bounds__(EMB_NT) k_embed_sum(const __grid_constant__ EmbedSum P) {
    using A = typename AccOf<T>::A;
    constexpr int U = 8;  // rows in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const EmbedArgs& E = P.A;
    if ((int64_t)blockIdx.x >= P.sum_blocks) {
        // zero rows: a warp per row
        const int64_t zb = (int64_t)gridDim.x - P.sum_blocks;
        for (int64_t r = ((int64_t)blockIdx.x - P.sum_blocks) * (EMB_NT / 32) + warp; r < E.rows; r += zb * (EMB_NT / 32)) {
            if (P.seen[r >> 5] >> (r & 31) & 1) continue;
            W* p = static_cast<W*>(E.dst) + r * E.dst_ld;
            Pack<W, VN> z;
#pragma unroll
            for (int e = 0; e < VN; ++e) z.v[e] = from_acc<W, typename AccOf<W>::A>(0);
            for (int64_t c = lane * VN; c < E.dim; c += 32 * VN) *reinterpret_cast<Pack<W, VN>*>(p + c) = z;
        }
        return;
    }
    const int64_t cols = (E.dim + 32 * VN - 1) / (32 * VN);
    const int64_t w = (int64_t)blockIdx.x * (EMB_NT / 32) + warp;
    const int64_t tile = w / cols;
    if (tile >= P.tiles) return;
    const int64_t c = ((w - tile * cols) * 32 + lane) * VN;
    const int64_t p0 = tile * P.R, p1 = min(p0 + P.R, E.n);
    const uint32_t none = (uint32_t)E.rows;
    const bool in = c < E.dim;
    const uint32_t before = p0 > 0 ? P.keys[p0 - 1] : 0xffffffffu;
    const uint32_t after = p1 < E.n ? P.keys[p1] : 0xffffffffu;
    A s[VN];
#pragma unroll
    for (int e = 0; e < VN; ++e) s[e] = 0;
    uint32_t cur = P.keys[p0];
    bool entered = cur == before;  // the run began in an earlier tile
    A* part = static_cast<A*>(P.part) + tile * 2 * E.dim + c;
    for (int64_t p = p0; p < p1; p += U) {
        Pack<T, VN> v[U];
        uint32_t key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            key[u] = p + u < p1 ? P.keys[p + u] : none;
            if (in && key[u] != none) {
                const int64_t i = P.perm[p + u];
                v[u] = *reinterpret_cast<const Pack<T, VN>*>(static_cast<const T*>(E.src) + i * E.src_ld + c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p + u >= p1) break;
            if (key[u] != cur) {
                if (in && cur != none) {
                    if (entered) {
#pragma unroll
                        for (int e = 0; e < VN; ++e) part[e] = s[e];
                    } else embed_write<T, W, VN>(E, cur, c, s);
                }
#pragma unroll
                for (int e = 0; e < VN; ++e) s[e] = 0;
                cur = key[u];
                entered = false;
            }
            if (in && cur != none)
#pragma unroll
                for (int e = 0; e < VN; ++e) s[e] += to_acc<A, T>(v[u].v[e]);
        }
    }
    if (!in || cur == none) return;
    if (entered) {
#pragma unroll
        for (int e = 0; e < VN; ++e) part[e] = s[e];
    } else if (cur == after) {
#pragma unroll
        for (int e = 0; e < VN; ++e) part[E.dim + e] = s[e];
    } else embed_write<T, W, VN>(E, cur, c, s);
}

// The runs that cross tile boundaries: the tile a run leaves joins its parts in order.
template <typename T, typename W>
__global__ void __launch_bounds__(EMB_NT) k_embed_join(const __grid_constant__ EmbedSum P) {
    using A = typename AccOf<T>::A;
    const EmbedArgs& E = P.A;
    const int64_t tile = blockIdx.x, p0 = tile * P.R, p1 = p0 + P.R;
    if (p1 >= E.n) return;
    const uint32_t key = P.keys[p1 - 1];
    if (key == (uint32_t)E.rows || P.keys[p1] != key) return;
    if (P.keys[p0] == key && p0 > 0 && P.keys[p0 - 1] == key) return;  // it began earlier
    // tiles that the run enters: as long as their first key is this one
    int64_t lo = tile + 1, hi = P.tiles;  // the first tile past the run (keys ascend)
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (P.keys[mid * P.R] == key) lo = mid + 1; else hi = mid;
    }
    const A* part = static_cast<const A*>(P.part);
    for (int64_t c = (int64_t)blockIdx.y * EMB_NT + threadIdx.x; c < E.dim; c += (int64_t)gridDim.y * EMB_NT) {
        A s = part[(tile * 2 + 1) * E.dim + c];
#pragma unroll 8
        for (int64_t t = tile + 1; t < lo; ++t) s += part[t * 2 * E.dim + c];
        embed_write<T, W, 1>(E, key, c, &s);
    }
}

// Positions per tile: enough warps to fill the GPU (148 SMs x 64), between 16
// and 256 (the partial sums of a tile are two rows of fp32, against R rows read).
static int embed_tile(int64_t n, int64_t dim, int es) {
    const int64_t cols = std::max<int64_t>(1, (dim * es + 511) / 512);
    int64_t R = 16;
    while (R < 256 && n * cols / R > 2 * 148 * 64) R *= 2;
    return (int)R;
}

struct EmbedWs {
    size_t keys, skeys, perm, seen, part, sort;
};
static EmbedWs embed_ws(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt) {
    EmbedWs W;
    const int64_t tiles = (n + embed_tile(n, dim, (int)elem_bytes(dt)) - 1) / embed_tile(n, dim, (int)elem_bytes(dt));
    W.keys = Carve::need((size_t)n, 4);
    W.skeys = Carve::need((size_t)n, 4);
    W.perm = Carve::need((size_t)n, 4);
    W.seen = Carve::need((size_t)((rows + 31) / 32), 4);
    W.part = Carve::need((size_t)(tiles * 2 * dim), acc_bytes(dt));
    W.sort = sort_keys_ws_bytes(n);
    return W;
}

size_t embed_bwd_ws_bytes(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt) {
    const EmbedWs W = embed_ws(n, rows, dim, dt);
    return W.keys + W.skeys + W.perm + W.seen + W.part + W.sort;
}

template <typename T, typename W>
static cudaError_t embed_sum_launch(EmbedSum S, int sms, cudaStream_t st) {
    constexpr int VN = VecOf<T>::N;
    const bool vec = vec_ok(S.A, VN, sizeof(T), sizeof(W), std::min<int>(16, VN * sizeof(W)));
    const int64_t cols = (S.A.dim + 32 * (vec ? VN : 1) - 1) / (32 * (vec ? VN : 1));
    S.sum_blocks = (S.tiles * cols + EMB_NT / 32 - 1) / (EMB_NT / 32);
    const int64_t zero = S.A.accumulate ? 0 : std::min<int64_t>((S.A.rows + EMB_NT / 32 - 1) / (EMB_NT / 32), 8 * (int64_t)sms);
    const int64_t grid = S.sum_blocks + zero;
    if (grid > 0) {
        if (vec) k_embed_sum<T, W, VN><<<(unsigned)grid, EMB_NT, 0, st>>>(S);
        else k_embed_sum<T, W, 1><<<(unsigned)grid, EMB_NT, 0, st>>>(S);
    }
    if (S.tiles > 1) {
        const dim3 jg((unsigned)(S.tiles - 1), (unsigned)std::min<int64_t>((S.A.dim + EMB_NT - 1) / EMB_NT, 65535));
        k_embed_join<T, W><<<jg, EMB_NT, 0, st>>>(S);
    }
    return cudaGetLastError();
}

cudaError_t embed_bwd_run(laplex_dtype dt, laplex_dtype out_dt, const EmbedArgs& A, void* ws, size_t ws_bytes,
                          uint32_t* status, cudaStream_t st) {
    if (A.dim == 0 || (A.rows == 0)) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = current_device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    const EmbedWs Z = embed_ws(A.n, A.rows, A.dim, dt);
    if (ws_bytes < Z.keys + Z.skeys + Z.perm + Z.seen + Z.part + Z.sort) return cudaErrorInvalidValue;
    char* p = static_cast<char*>(ws);
    uint32_t* keys = (uint32_t*)p;
    uint32_t* skeys = (uint32_t*)(p += Z.keys);
    int32_t* perm = (int32_t*)(p += Z.skeys);
    uint32_t* seen = (uint32_t*)(p += Z.perm);
    void* part = p += Z.seen;
    void* sort = p += Z.part;
    if (!A.accumulate) {
        e = cudaMemsetAsync(seen, 0, (size_t)((A.rows + 31) / 32) * 4, st);
        if (e != cudaSuccess) return e;
    }
    if (A.n > 0) {
        k_embed_keys<<<(unsigned)((A.n + 255) / 256), 256, 0, st>>>(A.tokens, A.tok64, A.n, A.rows, keys,
                                                                   A.accumulate ? nullptr : seen);
        e = cudaGetLastError();
        if (e == cudaSuccess)
            e = sort_keys_run(keys, A.n, (uint32_t)A.rows, skeys, perm, sort, Z.sort, status, st);
        if (e != cudaSuccess) return e;
    }
    EmbedSum S;
    S.A = A;
    S.keys = skeys;
    S.perm = perm;
    S.seen = seen;
    S.part = part;
    S.R = embed_tile(A.n, A.dim, (int)elem_bytes(dt));
    S.tiles = (A.n + S.R - 1) / S.R;
    S.sum_blocks = 0;
    const bool f32 = out_dt == LAPLEX_F32;
    switch (dt) {
        case LAPLEX_F32: return embed_sum_launch<float, float>(S, sms, st);
        case LAPLEX_F64: return embed_sum_launch<double, double>(S, sms, st);
        case LAPLEX_F16: return f32 ? embed_sum_launch<__half, float>(S, sms, st) : embed_sum_launch<__half, __half>(S, sms, st);
        case LAPLEX_BF16:
            return f32 ? embed_sum_launch<__nv_bfloat16, float>(S, sms, st)
                       : embed_sum_launch<__nv_bfloat16, __nv_bfloat16>(S, sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lx
