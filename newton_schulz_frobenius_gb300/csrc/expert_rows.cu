// Rows of a block that is split over experts: slots sorted by expert, tokens
// copied to their experts' rows and the experts' results brought back with
// weights, and the gradients of both.  Slot t k + j is token t's j-th choice.
//
//   sort       row_of[slot], slot_of[row]: slots in the order of their experts,
//              equal experts in slot order; those without an expert behind bounds[E]
//   dispatch   xs[row_of[t, j]] = x[t]
//   combine    y[t] = residual[t] + sum_j w[t, j] ys[row_of[t, j]]
//              (without weights: the gradient of dispatch)
//   backward   dys[row_of[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[row_of[t, j]]>
//
// All are bound by HBM; the sort by latency.
#include "host.h"
#include "epilogue.cuh"
#include "tc_ptx.cuh"

namespace muon {

namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int64_t MAX_SLOTS = 1 << 24;
constexpr int64_t MAX_HIDDEN = 1 << 20;

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
//
// A stable counting sort in one launch of one cluster.  Every warp takes a run
// of consecutive slots and counts them by expert in its own row of a table;
// columns are summed over the CTA's warps and, through distributed shared
// memory, over the cluster's CTAs before it, experts are summed in order, and a
// second walk over the same slots hands out the places.  Within 32 slots equal
// experts find each other by a match, so nothing depends on scheduling.
constexpr int SORT_T = 1024;
constexpr int SORT_WARPS = SORT_T / 32;
constexpr int SORT_CLUSTER = 16;
constexpr int SORT_AHEAD = 8;       // loads of a warp in flight

struct SortArgs {
    const void* experts;
    int index64;
    int slots, experts_n;
    int per_warp;               // slots of a warp, a multiple of 32
    int* row_of;
    int* slot_of;
    int* bounds;
};

__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, uint32_t rank) {
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Expert of a slot: experts_n for none, -1 beyond the run's last slot.
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t i, int64_t last) {
    if (i >= last) return -1;
    if (a.index64) {
        const int64_t e = static_cast<const int64_t*>(a.experts)[i];
        return e >= 0 && e < a.experts_n ? (int)e : a.experts_n;
    }
    const int e = static_cast<const int*>(a.experts)[i];
    return e >= 0 && e < a.experts_n ? e : a.experts_n;
}

__global__ void __launch_bounds__(SORT_T, 1) expert_sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ uint32_t sort_smem[];
    const int E = a.experts_n, bins = E + 1;
    uint32_t* table = sort_smem;                        // [SORT_WARPS][bins]
    uint32_t* total = table + SORT_WARPS * bins;        // [bins] of this CTA, read by the others
    __shared__ uint32_t sums[SORT_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_ctarank(), C = (int)gridDim.x;
    for (int i = threadIdx.x; i < SORT_WARPS * bins; i += SORT_T) table[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    const int64_t first = ((int64_t)rank * SORT_WARPS + warp) * a.per_warp;
    const int64_t last = min(first + a.per_warp, (int64_t)a.slots);
    uint32_t* mine = table + warp * bins;
    int e[SORT_AHEAD];
    for (int64_t i = first; i < last; i += 32 * SORT_AHEAD) {
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r) e[r] = expert_of(a, i + 32 * r + lane, last);
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r) {
            const uint32_t same = __match_any_sync(0xffffffffu, e[r]);
            if (e[r] >= 0 && lane == __ffs((int)same) - 1) mine[e[r]] += (uint32_t)__popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // per expert: the warps' counts become the places before each warp's first
    for (int b = threadIdx.x; b < bins; b += SORT_T) {
        uint32_t n = 0;
#pragma unroll 8
        for (int w = 0; w < SORT_WARPS; ++w) {
            const uint32_t c = table[w * bins + b];
            table[w * bins + b] = n;
            n += c;
        }
        total[b] = n;
    }
    tc::cluster_sync();
    // all CTAs' counts of expert threadIdx.x, and those of the CTAs before this one
    uint32_t all = 0, before = 0, rest = 0;
    if ((int)threadIdx.x < E) {
        for (int c = 0; c < C; ++c) {
            const uint32_t n = ld_cluster(total + threadIdx.x, (uint32_t)c);
            if (c < rank) before += n;
            all += n;
        }
    }
    if (threadIdx.x == 0)
        for (int c = 0; c < rank; ++c) rest += ld_cluster(total + E, (uint32_t)c);
    __syncwarp();
    tc::cluster_sync();                 // the others have read this CTA's counts
    uint32_t upto = all;                // inclusive sum over experts
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += n;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = sums[lane];
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += n;
        }
        sums[lane] = s;
    }
    __syncthreads();
    upto += warp ? sums[warp - 1] : 0;
    if ((int)threadIdx.x < E) {
        total[threadIdx.x] = upto - all + before;
        if (rank == 0) a.bounds[threadIdx.x + 1] = (int)upto;
    }
    if (threadIdx.x == 0) {
        total[E] = sums[SORT_WARPS - 1] + rest;
        if (rank == 0) a.bounds[0] = 0;
    }
    __syncthreads();
    for (int64_t i = first; i < last; i += 32 * SORT_AHEAD) {
        if (a.per_warp > 32 * SORT_AHEAD) {     // else the first walk's are still here
#pragma unroll
            for (int r = 0; r < SORT_AHEAD; ++r) e[r] = expert_of(a, i + 32 * r + lane, last);
        }
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r) {
            const uint32_t same = __match_any_sync(0xffffffffu, e[r]);
            const uint32_t at = e[r] >= 0 ? mine[e[r]] : 0;
            __syncwarp();
            if (e[r] >= 0) {
                if (lane == __ffs((int)same) - 1) mine[e[r]] = at + (uint32_t)__popc(same);
                const int row = (int)(total[e[r]] + at + (uint32_t)__popc(same & ((1u << lane) - 1)));
                a.row_of[i + 32 * r + lane] = row;
                a.slot_of[row] = (int)(i + 32 * r + lane);
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

struct RowArgs {
    const void* x;              // dispatch: x; combine: ys; backward: ys
    const void* y;              // combine: residual or null; backward: dy
    int64_t ldx, ldy;           // pitches of the token-side matrices (elements)
    void* out;
    const int* row_of;
    const int* bounds;
    const float* weights;
    float* dweights;
    int64_t tokens;
    int k, hidden, experts_n;
    int dtype;
    int pieces;                 // 16-byte pieces of a row
    int group;                  // backward: warps that share a row
};

constexpr int RT = 256;

// Rows of live slots: those before the last expert's end.
__device__ __forceinline__ int live_rows(const RowArgs& a) {
    const int64_t rows = a.tokens * a.k;
    return (int)min((int64_t)max(a.bounds[a.experts_n], 0), rows);
}

// Piece c (16 bytes) of a row that starts at element e.
template <int ES, bool VEC>
__device__ __forceinline__ uint4 load_piece(const void* p, int64_t e, int c, int hidden) {
    constexpr int V = 16 / ES;
    if (VEC) return reinterpret_cast<const uint4*>(static_cast<const char*>(p) + e * ES)[c];
    uint32_t w[4] = {0, 0, 0, 0};
    const int n = min(V, hidden - c * V);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= n) break;
        if (ES == 4) w[i % 4] = static_cast<const uint32_t*>(p)[e + c * V + i];
        else w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[e + c * V + i] << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int ES, bool VEC>
__device__ __forceinline__ void store_piece(void* p, int64_t e, int c, int hidden, const uint4& q) {
    constexpr int V = 16 / ES;
    if (VEC) {
        reinterpret_cast<uint4*>(static_cast<char*>(p) + e * ES)[c] = q;
        return;
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const int n = min(V, hidden - c * V);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= n) break;
        if (ES == 4) static_cast<uint32_t*>(p)[e + c * V + i] = w[i % 4];
        else static_cast<uint16_t*>(p)[e + c * V + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

template <int ES>
__device__ __forceinline__ void to_floats(const uint4& q, float (&v)[16 / ES], bool f16) {
    if constexpr (ES == 2) {
        unpack8_h(q, v, f16);
    } else {
        v[0] = __uint_as_float(q.x);
        v[1] = __uint_as_float(q.y);
        v[2] = __uint_as_float(q.z);
        v[3] = __uint_as_float(q.w);
    }
}

template <int ES>
__device__ __forceinline__ uint4 from_floats(const float (&v)[16 / ES], bool f16) {
    if constexpr (ES == 2) return pack8_h(v, f16);
    else return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// A warp takes one token and a run of its pieces, reads them once and writes
// them to the token's k rows.
template <int ES, bool VEC>
__global__ void __launch_bounds__(RT) dispatch_kernel(const __grid_constant__ RowArgs a) {
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, live = live_rows(a);
    const int runs = (a.pieces + 32 * U - 1) / (32 * U);
    const int64_t rows = a.tokens * a.k, items = a.tokens * runs;
    for (int64_t i = (int64_t)blockIdx.x * (RT / 32) + (threadIdx.x >> 5); i < items; i += (int64_t)gridDim.x * (RT / 32)) {
        const int64_t t = i / runs;
        const int c0 = (int)(i - t * runs) * 32 * U + lane;
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < a.pieces) q[u] = load_piece<ES, VEC>(a.x, t * a.ldx, c0 + 32 * u, a.hidden);
        for (int j = 0; j < a.k; ++j) {
            const int64_t r = a.row_of[t * a.k + j];
            if (r < 0 || r >= rows) continue;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < a.pieces)
                    store_piece<ES, VEC>(a.out, r * a.hidden, c0 + 32 * u, a.hidden,
                                         r < live ? q[u] : make_uint4(0, 0, 0, 0));
        }
    }
}

// A warp takes one token and a run of its pieces and sums the token's k rows
// there in fp32, in the order of the choices; one rounding.
template <int ES, bool VEC>
__global__ void __launch_bounds__(RT) combine_kernel(const __grid_constant__ RowArgs a) {
    constexpr int V = 16 / ES;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, live = live_rows(a);
    const bool f16 = a.dtype == MUON_F16;
    const int runs = (a.pieces + 31) / 32;
    const int64_t items = a.tokens * runs;
    for (int64_t i = (int64_t)blockIdx.x * (RT / 32) + (threadIdx.x >> 5); i < items; i += (int64_t)gridDim.x * (RT / 32)) {
        const int64_t t = i / runs;
        const int c = (int)(i - t * runs) * 32 + lane;
        if (c >= a.pieces) continue;
        float acc[V], v[V];
#pragma unroll
        for (int n = 0; n < V; ++n) acc[n] = 0.f;
        if (a.y) to_floats<ES>(load_piece<ES, VEC>(a.y, t * a.ldy, c, a.hidden), acc, f16);
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int r = a.row_of[t * a.k + j];
            if (r < 0 || r >= live) continue;
            const float w = a.weights ? a.weights[t * a.k + j] : 1.f;
            to_floats<ES>(load_piece<ES, VEC>(a.x, (int64_t)r * a.hidden, c, a.hidden), v, f16);
#pragma unroll
            for (int n = 0; n < V; ++n) acc[n] = fmaf(w, v[n], acc[n]);
        }
        store_piece<ES, VEC>(a.out, t * a.hidden, c, a.hidden, from_floats<ES>(acc, f16));
    }
}

// `group` warps share a slot's row: they read it beside its token's dy (which
// the slots of a token, neighbours in a CTA, take from L1), write w dy, and sum
// the products in a fixed order.
template <int ES, bool VEC>
__global__ void __launch_bounds__(RT) combine_backward_kernel(const __grid_constant__ RowArgs a) {
    constexpr int V = 16 / ES, U = 2;
    __shared__ float part[RT / 32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, live = live_rows(a);
    const bool f16 = a.dtype == MUON_F16;
    const int G = a.group, per = RT / 32 / G, place = warp % G;
    const int64_t rows = a.tokens * a.k;
    for (int64_t s0 = (int64_t)blockIdx.x * per; s0 < rows; s0 += (int64_t)gridDim.x * per) {
        const int64_t s = s0 + warp / G;
        float dot = 0.f;
        const int64_t r = s < rows ? a.row_of[s] : -1;
        if (r >= 0 && r < rows) {
            const bool on = r < live;
            const int64_t t = s / a.k;
            const float w = on ? a.weights[s] : 0.f;
            for (int c0 = place * 32 + lane; c0 < a.pieces; c0 += 32 * G * U) {
                uint4 qd[U], qy[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + 32 * G * u;
                    if (!on || c >= a.pieces) continue;
                    qd[u] = load_piece<ES, VEC>(a.y, t * a.ldy, c, a.hidden);
                    qy[u] = load_piece<ES, VEC>(a.x, r * a.hidden, c, a.hidden);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + 32 * G * u;
                    if (c >= a.pieces) continue;
                    float d[V], y[V];
#pragma unroll
                    for (int n = 0; n < V; ++n) d[n] = 0.f;
                    if (on) {
                        to_floats<ES>(qd[u], d, f16);
                        to_floats<ES>(qy[u], y, f16);
#pragma unroll
                        for (int n = 0; n < V; ++n) {
                            dot = fmaf(d[n], y[n], dot);
                            d[n] *= w;
                        }
                    }
                    store_piece<ES, VEC>(a.out, r * a.hidden, c, a.hidden, from_floats<ES>(d, f16));
                }
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (G > 1) {
            __syncthreads();
            if (lane == 0) part[warp] = dot;
            __syncthreads();
            dot = 0.f;
            for (int g = 0; g < G; ++g) dot += part[warp / G * G + g];
        }
        if (s < rows && place == 0 && lane == 0) a.dweights[s] = dot;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int rows_check(int64_t tokens, int64_t k, int64_t hidden, int dtype, int64_t experts_n) {
    if (!valid_dtype(dtype)) return fail(MUON_EDTYPE, "dtype %d", dtype);
    if (k < 1 || k > MAX_EXPERTS) return fail(MUON_EINVAL, "k outside [1, %d]", MAX_EXPERTS);
    if (tokens < 0 || tokens > MAX_SLOTS / k) return fail(MUON_EINVAL, "tokens k outside [0, 2^24]");
    if (hidden < 1 || hidden > MAX_HIDDEN) return fail(MUON_EINVAL, "hidden outside [1, 2^20]");
    if (experts_n < 1 || experts_n > MAX_EXPERTS) return fail(MUON_EINVAL, "experts outside [1, %d]", MAX_EXPERTS);
    return MUON_OK;
}

int pointer_check(int dtype, std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & (esize(dtype) - 1)) return fail(MUON_EINVAL, "pointer not aligned to its element");
    return MUON_OK;
}

RowArgs row_args(int64_t tokens, int64_t k, int64_t hidden, int dtype, const int* row_of, const int* bounds,
                 int64_t experts_n) {
    RowArgs a;
    std::memset(&a, 0, sizeof a);
    a.tokens = tokens; a.k = (int)k; a.hidden = (int)hidden; a.dtype = dtype;
    a.row_of = row_of; a.bounds = bounds; a.experts_n = (int)experts_n;
    a.pieces = (int)((hidden * (int64_t)esize(dtype) + 15) / 16);
    return a;
}

template <typename K>
int launch_rows(K kernel, const RowArgs& a, int64_t ctas, int sms, cudaStream_t s, const char* what) {
    note_launch_begin(KC_OTHER, s);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)sms * 8))),
                                     dim3(RT), 0, s, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, what);
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" int muon_expert_sort(const void* experts, int index_dtype, int64_t slots, int64_t num_experts, int* row_of,
                                int* slot_of, int* bounds, void* stream) try {
    if (index_dtype != MUON_I32 && index_dtype != MUON_I64) return fail(MUON_EDTYPE, "index dtype %d", index_dtype);
    if (slots < 0 || slots > MAX_SLOTS) return fail(MUON_EINVAL, "slots outside [0, 2^24]");
    if (num_experts < 1 || num_experts > MAX_EXPERTS) return fail(MUON_EINVAL, "experts outside [1, %d]", MAX_EXPERTS);
    if (!bounds || (slots > 0 && (!experts || !row_of || !slot_of))) return fail(MUON_EINVAL, "NULL argument");
    int r = pointer_check(MUON_F32, {row_of, slot_of, bounds, experts});
    if (r) return r;
    if (index_dtype == MUON_I64 && (reinterpret_cast<uintptr_t>(experts) & 7))
        return fail(MUON_EINVAL, "pointer not aligned to its element");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int C = 1;                              // CTAs: four slots per thread until the cluster is full
    while (C < SORT_CLUSTER && (int64_t)C * SORT_T * 4 < slots) C *= 2;
    SortArgs a;
    a.experts = experts;
    a.index64 = index_dtype == MUON_I64;
    a.slots = (int)slots;
    a.experts_n = (int)num_experts;
    a.per_warp = (int)((slots + (int64_t)C * SORT_T - 1) / ((int64_t)C * SORT_T)) * 32;
    a.row_of = row_of; a.slot_of = slot_of; a.bounds = bounds;
    static OncePer<int, int> attr;          // by device
    int set = 0;
    const size_t most = (size_t)(SORT_WARPS + 1) * (MAX_EXPERTS + 1) * 4;
    cudaError_t e = attr.get(dc.device, &set, [&](int&) {
        cudaError_t r = cudaFuncSetAttribute(expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(expert_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
    });
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(SORT_T);
    cfg.dynamicSmemBytes = (size_t)(SORT_WARPS + 1) * (size_t)(num_experts + 1) * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    note_launch_begin(KC_OTHER, s);
    e = cudaLaunchKernelEx(&cfg, expert_sort_kernel, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "expert sort launch");
} MUON_CATCH_ALL

extern "C" int muon_expert_dispatch(const void* x, int64_t ldx, int64_t tokens, int64_t k, int64_t hidden, int dtype,
                                    const int* row_of, const int* bounds, int64_t num_experts, void* xs,
                                    void* stream) try {
    int r = rows_check(tokens, k, hidden, dtype, num_experts);
    if (r) return r;
    if (ldx < hidden) return fail(MUON_EINVAL, "pitch below the row's length");
    if (tokens == 0) return MUON_OK;
    if (!x || !row_of || !bounds || !xs) return fail(MUON_EINVAL, "NULL argument");
    if ((r = pointer_check(dtype, {x, xs})) || (r = pointer_check(MUON_F32, {row_of, bounds}))) return r;
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    RowArgs a = row_args(tokens, k, hidden, dtype, row_of, bounds, num_experts);
    a.x = x; a.ldx = ldx; a.out = xs;
    const int es = (int)esize(dtype);
    const bool vec = aligned16(x) && aligned16(xs) && (ldx * es) % 16 == 0 && (hidden * es) % 16 == 0;
    const int64_t ctas = (tokens * ((a.pieces + 127) / 128) + 7) / 8;
    auto kern = es == 2 ? (vec ? dispatch_kernel<2, true> : dispatch_kernel<2, false>)
                        : (vec ? dispatch_kernel<4, true> : dispatch_kernel<4, false>);
    return launch_rows(kern, a, ctas, dc.sms, s, "expert dispatch launch");
} MUON_CATCH_ALL

extern "C" int muon_expert_combine(const void* ys, int64_t tokens, int64_t k, int64_t hidden, int dtype,
                                   const int* row_of, const int* bounds, int64_t num_experts, const float* weights,
                                   const void* residual, int64_t ld_residual, void* y, void* stream) try {
    int r = rows_check(tokens, k, hidden, dtype, num_experts);
    if (r) return r;
    if (residual && ld_residual < hidden) return fail(MUON_EINVAL, "pitch below the row's length");
    if (tokens == 0) return MUON_OK;
    if (!ys || !row_of || !bounds || !y) return fail(MUON_EINVAL, "NULL argument");
    if ((r = pointer_check(dtype, {ys, residual, y})) || (r = pointer_check(MUON_F32, {row_of, bounds, weights}))) return r;
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    RowArgs a = row_args(tokens, k, hidden, dtype, row_of, bounds, num_experts);
    a.x = ys; a.y = residual; a.ldy = ld_residual; a.out = y; a.weights = weights;
    const int es = (int)esize(dtype);
    const bool vec = aligned16(ys) && aligned16(y) && aligned16(residual) && (hidden * es) % 16 == 0 &&
                     (!residual || (ld_residual * es) % 16 == 0);
    const int64_t ctas = (tokens * ((a.pieces + 31) / 32) + 7) / 8;
    auto kern = es == 2 ? (vec ? combine_kernel<2, true> : combine_kernel<2, false>)
                        : (vec ? combine_kernel<4, true> : combine_kernel<4, false>);
    return launch_rows(kern, a, ctas, dc.sms, s, "expert combine launch");
} MUON_CATCH_ALL

extern "C" int muon_expert_combine_backward(const void* dy, int64_t ld_dy, const void* ys, int64_t tokens, int64_t k,
                                            int64_t hidden, int dtype, const int* row_of, const int* bounds,
                                            int64_t num_experts, const float* weights, void* dys, float* dweights,
                                            void* stream) try {
    int r = rows_check(tokens, k, hidden, dtype, num_experts);
    if (r) return r;
    if (ld_dy < hidden) return fail(MUON_EINVAL, "pitch below the row's length");
    if (tokens == 0) return MUON_OK;
    if (!dy || !ys || !row_of || !bounds || !weights || !dys || !dweights) return fail(MUON_EINVAL, "NULL argument");
    if ((r = pointer_check(dtype, {dy, ys, dys})) || (r = pointer_check(MUON_F32, {row_of, bounds, weights, dweights})))
        return r;
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    RowArgs a = row_args(tokens, k, hidden, dtype, row_of, bounds, num_experts);
    a.x = ys; a.y = dy; a.ldy = ld_dy; a.out = dys; a.weights = weights; a.dweights = dweights;
    const int es = (int)esize(dtype);
    const bool vec = aligned16(dy) && aligned16(ys) && aligned16(dys) && (hidden * es) % 16 == 0 && (ld_dy * es) % 16 == 0;
    const int64_t slots = tokens * k;
    a.group = 1;                            // more warps to a row while rows are too few to fill the device
    while (a.group < RT / 32 && slots * a.group < (int64_t)dc.sms * 16 && a.group * 64 < a.pieces) a.group *= 2;
    const int per = RT / 32 / a.group;
    auto kern = es == 2 ? (vec ? combine_backward_kernel<2, true> : combine_backward_kernel<2, false>)
                        : (vec ? combine_backward_kernel<4, true> : combine_backward_kernel<4, false>);
    return launch_rows(kern, a, (slots + per - 1) / per, dc.sms, s, "expert combine backward launch");
} MUON_CATCH_ALL
