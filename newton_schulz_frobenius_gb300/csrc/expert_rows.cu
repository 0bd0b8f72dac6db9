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
// Rows that start on 16 bytes are bound by HBM, others by instructions (Words below),
// the sort by latency.
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
// A stable counting sort, up to 131072 slots in one launch of one cluster.  Every
// warp takes a run of consecutive slots and counts them by expert in its own row of
// a table; columns are summed over the CTA's warps and, through distributed shared
// memory, over the cluster's CTAs before it, experts are summed in order, and a
// second walk over the same slots hands out the places.  Within 32 slots equal
// experts find each other by votes, so nothing depends on scheduling.  Bound by
// latency: 4.5 us for 16384 slots and 64 experts, 7.7 for 65536, 12.0 for 131072
// (back to back in a graph).  More slots are sorted by the whole device in three
// launches: the CTAs' counts (left in slot_of, which is not written until the last),
// the places, and slot_of from them; 2^20 slots 26 us, 2^22 78 (one cluster, bound by
// its SMs' instructions and scattered stores: 95 and 342; at 131072 three launches take
// 12.3).  Each by itself, of 2^20 and 2^22 slots: counts 8 and 23 us, places 18 and 47,
// slot_of 7 and 20: the walks issue a vote per bit of the expert for 32 slots, one CTA
// to an SM, and slot_of is 4-byte stores a row apart, so that the floors of their bytes
// (2 and 7 us) are out of reach in this form.
constexpr int SORT_T = 1024;
constexpr int SORT_WARPS = SORT_T / 32;
constexpr int SORT_CLUSTER = 16;
constexpr int SORT_AHEAD = 8;       // loads of a warp in flight
enum SortStep : int { SORTED = 0, COUNTS = 1, PLACES = 2 };        // all in one cluster; the first two of three launches

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
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Lanes with the same expert, by a vote on each of its bits (the instruction that
// matches values takes its time for each different one: 65536 slots to 64 experts
// 10.8 us with it).
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
    uint32_t same = 0xffffffffu;
#pragma unroll 4
    for (int b = 0; b < bits; ++b) {
        const bool set = (e >> b) & 1;
        const uint32_t m = __ballot_sync(0xffffffffu, set);
        same &= set ? m : ~m;
    }
    return same;
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

template <int STEP>
__global__ void __launch_bounds__(SORT_T, 1) expert_sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ uint32_t sort_smem[];
    const int E = a.experts_n, bins = E + 1;
    uint32_t* table = sort_smem;                        // [SORT_WARPS][bins]
    uint32_t* total = table + SORT_WARPS * bins;        // [bins] of this CTA, read by the others
    __shared__ uint32_t sums[SORT_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x, C = (int)gridDim.x;          // (in one cluster: the CTA's rank there)
    for (int i = threadIdx.x; i < SORT_WARPS * bins; i += SORT_T) table[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    const int64_t first = ((int64_t)rank * SORT_WARPS + warp) * a.per_warp;
    const int64_t last = min(first + a.per_warp, (int64_t)a.slots);
    uint32_t* mine = table + warp * bins;
    const int bits = 33 - __clz(E);         // of 0 .. E, and one that -1 alone has set
    int e[SORT_AHEAD];
    uint32_t same[SORT_AHEAD];
    auto read = [&](int64_t i) {
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r) e[r] = expert_of(a, i + 32 * r + lane, last);
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r)
            if (i + 32 * r < last) same[r] = same_expert(e[r], bits);
    };
    for (int64_t i = first; i < last; i += 32 * SORT_AHEAD) {
        read(i);
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r) {
            if (i + 32 * r >= last) break;
            if (e[r] >= 0 && lane == __ffs((int)same[r]) - 1) mine[e[r]] += (uint32_t)__popc(same[r]);
            __syncwarp();
        }
        if (STEP == SORTED) break;          // a warp of a cluster has no more slots than one step takes
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
        if (STEP == COUNTS) a.slot_of[rank * bins + b] = (int)n;
        else total[b] = n;
    }
    if (STEP == COUNTS) return;
    if (STEP == SORTED) tc::cluster_sync();
    // all CTAs' counts of expert threadIdx.x, and those of the CTAs before this one
    uint32_t all = 0, before = 0, rest = 0, none = 0;
    auto counts = [&](int bin, uint32_t& upto_here, uint32_t& of_all) {
        for (int c0 = 0; c0 < (STEP == SORTED ? 1 : C); c0 += SORT_CLUSTER) {
            uint32_t n[SORT_CLUSTER];       // all on their way before the first is used
#pragma unroll
            for (int c = 0; c < SORT_CLUSTER; ++c)
                n[c] = c0 + c >= C ? 0
                       : STEP == SORTED ? ld_cluster(total + bin, (uint32_t)c) : (uint32_t)a.slot_of[(c0 + c) * bins + bin];
#pragma unroll
            for (int c = 0; c < SORT_CLUSTER; ++c) {
                if (c0 + c < rank) upto_here += n[c];
                of_all += n[c];
            }
        }
    };
    if ((int)threadIdx.x < E) counts(threadIdx.x, before, all);
    if (threadIdx.x == SORT_T - 1) counts(E, rest, none);
    __syncwarp();
    if (STEP == SORTED) tc::cluster_sync();             // the others have read this CTA's counts
    else __syncthreads();
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
    if (threadIdx.x == SORT_T - 1) total[E] = sums[SORT_WARPS - 1] + rest;
    if (threadIdx.x == 0 && rank == 0) a.bounds[0] = 0;
    __syncthreads();
    for (int64_t i = first; i < last; i += 32 * SORT_AHEAD) {
        // (else the first walk's are still here)
        if (STEP == PLACES && a.per_warp > 32 * SORT_AHEAD) read(i);
#pragma unroll
        for (int r = 0; r < SORT_AHEAD; ++r) {
            if (i + 32 * r >= last) break;
            const uint32_t at = e[r] >= 0 ? mine[e[r]] : 0;
            __syncwarp();
            if (e[r] >= 0) {
                if (lane == __ffs((int)same[r]) - 1) mine[e[r]] = at + (uint32_t)__popc(same[r]);
                const int row = (int)(total[e[r]] + at + (uint32_t)__popc(same[r] & ((1u << lane) - 1)));
                a.row_of[i + 32 * r + lane] = row;
                if (STEP == SORTED) a.slot_of[row] = (int)(i + 32 * r + lane);
            }
            __syncwarp();
        }
        if (STEP == SORTED) break;
    }
}

// slot_of, after the launches of COUNTS and PLACES: every row has one slot.
__global__ void __launch_bounds__(256) expert_invert_kernel(const int* row_of, int* slot_of, int slots) {
    pdl_wait();
    pdl_trigger();
    for (int i = blockIdx.x * 1024 + threadIdx.x, n = 0; n < 4 && i < slots; i += 256, ++n) slot_of[row_of[i]] = i;
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
    int slots;                  // of a row: 16-byte pieces, or 4-byte words that it can touch
    int span;                   // dispatch, combine: slots of a warp; rings: chunks of a unit
    int parts, units;           // rings: units of a token, of the call
    int group;                  // backward: warps that share a token's rows, a power of two
};

constexpr int RT = 256;
constexpr int J = 4;                // slots of a token that a warp of the backward pass works at once

// Rows of live slots: those before the last expert's end.
__device__ __forceinline__ int live_rows(const RowArgs& a) {
    const int64_t rows = a.tokens * a.k;
    return (int)min((int64_t)max(a.bounds[a.experts_n], 0), rows);
}

// Rows that start on 16 bytes are read and written as pieces of 16 bytes, others as
// the aligned 4-byte words that their elements fall into, 32 neighbours per warp
// and access: as few wavefronts, four times the instructions, but none to shift
// 16 bytes into place (16384 tokens, 4 rows of 1001 bf16 each: combine 59 us, 73
// with aligned 16-byte loads shifted through the neighbour lane).
//
// Word i of a row of 16-bit elements holds columns 2 i - odd and 2 i - odd + 1, odd = 1 if
// the row starts in the middle of a word.  Words whose columns are all the row's
// go 128 at a time per warp, four to a lane, without a question about the ends;
// a first or last column that shares its word with another row is an edge and worked
// by itself.  Instructions bound these rows: 30000 x 77 bf16 with 3 choices, 13 us
// dispatched (floor 3), 16384 x 1001 with 4, 39 (24).
template <int ES>
struct Words {
    static constexpr int E = 4 / ES, U = 4;     // elements of a word, words of a lane at once (32 apart)
    char* row;                  // the first element
    int odd, end, hidden;       // whole words: [odd, end)
    bool inside;                // words around its ends are in the matrix too
    __device__ __forceinline__ Words(const void* base, int64_t n, int64_t e, int h) : hidden(h) {
        row = static_cast<char*>(const_cast<void*>(base)) + e * ES;
        odd = ES == 2 ? (int)(reinterpret_cast<uintptr_t>(row) & 2) / 2 : 0;
        end = (h + odd) / E;
        inside = (e > 0 || !odd) && (e + h < n || end * E == h + odd);
    }
    __device__ __forceinline__ uint32_t* words() const { return reinterpret_cast<uint32_t*>(row - odd * ES); }
    // Which of words i, i + 32 .. are whole ones of a row of parity `as`, a bit each.
    static __device__ __forceinline__ uint32_t whole(int i, int as, int hidden) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if ((uint32_t)(i + 32 * u - as) < (uint32_t)((hidden + as) / E - as)) m |= 1u << u;
        return m;
    }
    // The columns of words i, i + 32 .. of a row of parity `as`; 0 for those not in `m`.
    __device__ __forceinline__ void load(uint32_t (&q)[U], int i, int as, uint32_t m) const {
        if (ES == 4 || odd == as) {
            const uint32_t* p = words() + i;
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = m >> u & 1 ? p[32 * u] : 0;
        } else if (inside) {                    // each from two words
            const uint32_t* p = words() + i - as;
            uint32_t next[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                q[u] = m >> u & 1 ? p[32 * u] : 0;
                next[u] = m >> u & 1 ? p[32 * u + 1] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = __funnelshift_r(q[u], next[u], 16);
        } else {                                // at one of the matrix' two ends
            const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + 2 * i - as;
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = m >> u & 1 ? p[64 * u] | (uint32_t)p[64 * u + 1] << 16 : 0;
        }
    }
    __device__ __forceinline__ void store(int i, const uint32_t (&v)[U], uint32_t m) const {
        uint32_t* p = words() + i;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (m >> u & 1) __stcs(p + 32 * u, v[u]);
    }
    // The edges' columns, lanes 0 and 1: -1 if this lane has none.
    __device__ __forceinline__ int edge(int lane) const {
        if (ES == 4) return -1;
        if (lane == 0) return odd ? 0 : -1;
        return lane == 1 && end * E != hidden + odd ? hidden - 1 : -1;
    }
    __device__ __forceinline__ uint16_t& at(int column) const { return reinterpret_cast<uint16_t*>(row)[column]; }
};

__device__ __forceinline__ float half_float(uint16_t q, bool f16) {
    return f16 ? __half2float(__ushort_as_half(q)) : __bfloat162float(__ushort_as_bfloat16(q));
}
__device__ __forceinline__ uint16_t half_of(float v, bool f16) {
    return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int ES>
__device__ __forceinline__ void word_floats(uint32_t q, float (&v)[4 / ES], bool f16) {
    if constexpr (ES == 4) {
        v[0] = __uint_as_float(q);
    } else {
        const float2 f = f16 ? __half22float2(*reinterpret_cast<const __half2*>(&q))
                             : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q));
        v[0] = f.x;
        v[1] = f.y;
    }
}

template <int ES>
__device__ __forceinline__ uint32_t word_of(const float (&v)[4 / ES], bool f16) {
    if constexpr (ES == 4) {
        return __float_as_uint(v[0]);
    } else if (f16) {
        const __half2 h = __floats2half2_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

__device__ __forceinline__ uint4 no_piece() { return make_uint4(0, 0, 0, 0); }

// Piece c of a row on 16 bytes that starts at element e.
template <int ES>
__device__ __forceinline__ const uint4* piece(const void* p, int64_t e, int c) {
    return reinterpret_cast<const uint4*>(static_cast<const char*>(p) + e * ES) + c;
}
template <int ES>
__device__ __forceinline__ void put_piece(void* p, int64_t e, int c, const uint4& q) {
    // (rows leave the caches to what is read again)
    __stcs(reinterpret_cast<uint4*>(static_cast<char*>(p) + e * ES) + c, q);
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

// Indices (and weights) of 32 choices of a token from j0 on, a lane each, so that
// nothing waits for one at a time.
__device__ __forceinline__ int rows_of(const RowArgs& a, int64_t t, int j0, int64_t rows) {
    const int j = j0 + (threadIdx.x & 31);
    const int r = j < a.k ? a.row_of[t * a.k + j] : -1;
    return r < rows ? r : -1;
}

// A warp takes one token and some runs of its slots, reads them once and writes
// them to the token's k rows.  Bound by HBM: 16384 tokens of 2048 bf16 to eight rows
// each (604 MB) 93 us, 6.5 TB/s.
template <int ES, bool VEC>
__global__ void __launch_bounds__(RT) dispatch_kernel(const __grid_constant__ RowArgs a) {
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, live = live_rows(a);
    const int64_t t = (int64_t)blockIdx.x * (RT / 32) + (threadIdx.x >> 5), rows = a.tokens * a.k;
    if (t >= a.tokens) return;
    const int begin = blockIdx.y * a.span, end = min(a.slots, begin + a.span);
    for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int some = min(32, a.k - j0), mine = rows_of(a, t, j0, rows);
        for (int c = begin + lane; c - lane < end; c += 32 * U) {
            if constexpr (VEC) {
                uint4 q[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + 32 * u < a.slots) q[u] = *piece<ES>(a.x, t * a.ldx, c + 32 * u);
#pragma unroll 4
                for (int j = 0; j < some; ++j) {
                    const int64_t r = __shfl_sync(0xffffffffu, mine, j);
                    if (r < 0) continue;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (c + 32 * u < a.slots) put_piece<ES>(a.out, r * a.hidden, c + 32 * u, r < live ? q[u] : no_piece());
                }
            } else {
                const Words<ES> in(a.x, (a.tokens - 1) * a.ldx + a.hidden, t * a.ldx, a.hidden);
                // for rows of either parity
                const uint32_t m[2] = {Words<ES>::whole(c, 0, a.hidden), ES == 2 ? Words<ES>::whole(c, 1, a.hidden) : 0};
                uint32_t q[2][U];
                const uint32_t zeros[U] = {0, 0, 0, 0};
                in.load(q[0], c, 0, m[0]);
                if (ES == 2) in.load(q[1], c, 1, m[1]);
#pragma unroll 2
                for (int j = 0; j < some; ++j) {
                    const int64_t r = __shfl_sync(0xffffffffu, mine, j);
                    if (r < 0) continue;
                    const Words<ES> out(a.out, rows * a.hidden, r * a.hidden, a.hidden);
                    const bool odd = ES == 2 && out.odd;
                    if (r >= live) out.store(c, zeros, odd ? m[1] : m[0]);
                    else if (odd) out.store(c, q[1], m[1]);
                    else out.store(c, q[0], m[0]);
                    const int edge = c == lane && begin == 0 ? out.edge(lane) : -1;
                    if (edge >= 0) out.at(edge) = r < live ? in.at(edge) : (uint16_t)0;
                }
            }
        }
    }
}

// A warp takes one token and some runs of its slots and sums the token's k rows
// there in fp32, in the order of the choices; one rounding.  Bound by latency, so
// by warps: 8192 tokens, 8 rows of 2048 bf16 each onto a residual (336 MB): 60-63 us
// at eight CTAs per SM, 69 at six, 71 at three with twice the loads in flight per warp
// (such calls go by rings now, see below; few tokens, short rows and many choices here).
// Eight CTAs leave 32 registers: 12 to 36 bytes per thread are spilled there.
template <int ES, bool VEC>
__global__ void __launch_bounds__(RT, VEC || ES == 4 ? 8 : 5) combine_kernel(const __grid_constant__ RowArgs a) {
    constexpr int V = VEC ? 16 / ES : 4 / ES, U = VEC ? 1 : 4;      // elements of a slot, slots of a lane
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, live = live_rows(a);
    const bool f16 = a.dtype == MUON_F16;
    const int64_t t = (int64_t)blockIdx.x * (RT / 32) + (threadIdx.x >> 5), rows = a.tokens * a.k;
    if (t >= a.tokens) return;
    const Words<ES> out(a.out, a.tokens * a.hidden, t * a.hidden, a.hidden);
    const int begin = blockIdx.y * a.span, end = min(a.slots, begin + a.span);
    const int first = rows_of(a, t, 0, live);
    const float first_weight = a.weights && lane < a.k ? a.weights[t * a.k + lane] : 1.f;
    for (int c = begin + lane; c - lane < end; c += 32 * U) {
        float acc[U][V], v[V];
        const uint32_t m = VEC ? 0 : Words<ES>::whole(c, out.odd, a.hidden);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[u][k] = 0.f;
        if (a.y) {
            if constexpr (VEC) {
                if (c < a.slots) to_floats<ES>(*piece<ES>(a.y, t * a.ldy, c), acc[0], f16);
            } else {
                const Words<ES> add(a.y, (a.tokens - 1) * a.ldy + a.hidden, t * a.ldy, a.hidden);
                uint32_t q[U];
                add.load(q, c, out.odd, m);
#pragma unroll
                for (int u = 0; u < U; ++u) word_floats<ES>(q[u], acc[u], f16);
            }
        }
        for (int j0 = 0; j0 < a.k; j0 += 32) {
            int mine = first;
            float weight = first_weight;
            if (j0) {
                mine = rows_of(a, t, j0, live);
                weight = a.weights && j0 + lane < a.k ? a.weights[t * a.k + j0 + lane] : 1.f;
            }
            const int some = min(32, a.k - j0);
#pragma unroll(VEC ? 4 : 2)
            for (int j = 0; j < some; ++j) {
                const int r = __shfl_sync(0xffffffffu, mine, j);
                const float w = __shfl_sync(0xffffffffu, weight, j);
                if (r < 0) continue;
                if constexpr (VEC) {
                    if (c >= a.slots) continue;
                    to_floats<ES>(*piece<ES>(a.x, (int64_t)r * a.hidden, c), v, f16);
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[0][k] = fmaf(w, v[k], acc[0][k]);
                } else {
                    const Words<ES> in(a.x, rows * a.hidden, (int64_t)r * a.hidden, a.hidden);
                    uint32_t q[U];
                    in.load(q, c, out.odd, m);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        word_floats<ES>(q[u], v, f16);
#pragma unroll
                        for (int k = 0; k < V; ++k) acc[u][k] = fmaf(w, v[k], acc[u][k]);
                    }
                }
            }
        }
        if constexpr (VEC) {
            if (c < a.slots) put_piece<ES>(a.out, t * a.hidden, c, from_floats<ES>(acc[0], f16));
        } else {
            uint32_t q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = word_of<ES>(acc[u], f16);
            out.store(c, q, m);
        }
    }
    if constexpr (!VEC) {
        const int edge = begin == 0 ? out.edge(lane) : -1;
        if (edge < 0) return;
        float sum = a.y ? half_float(static_cast<const uint16_t*>(a.y)[t * a.ldy + edge], f16) : 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int r = a.row_of[t * a.k + j];
            if (r < 0 || r >= live) continue;
            sum = fmaf(a.weights ? a.weights[t * a.k + j] : 1.f,
                       half_float(static_cast<const uint16_t*>(a.x)[(int64_t)r * a.hidden + edge], f16), sum);
        }
        out.at(edge) = half_of(sum, f16);
    }
}

// `group` warps share J slots of a token: they read its dy once and the slots'
// rows beside it, write w dy, and sum the products in a fixed order.  Bound by HBM:
// 8192 tokens, 8 rows of 2048 bf16 each (570 MB) 98 us, 5.8 TB/s.
template <int ES, bool VEC>
__global__ void __launch_bounds__(RT, 4) combine_backward_kernel(const __grid_constant__ RowArgs a) {
    constexpr int V = VEC ? 16 / ES : 4 / ES, U = VEC ? 1 : 4;
    __shared__ float part[RT / 32][J];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, live = live_rows(a);
    const bool f16 = a.dtype == MUON_F16;
    const int G = a.group, place = warp & (G - 1);
    const int64_t rows = a.tokens * a.k, n = rows * a.hidden;
    const int64_t t = (int64_t)blockIdx.x * (RT / 32 / G) + warp / G, s = t * a.k + blockIdx.y * J;    // the first slot
    const int some = t < a.tokens ? min(J, a.k - (int)blockIdx.y * J) : 0;
    int r[J];
    float w[J], dot[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        r[j] = j < some ? a.row_of[s + j] : -1;
        if (r[j] >= rows) r[j] = -1;
        w[j] = r[j] >= 0 && r[j] < live ? a.weights[s + j] : 0.f;
        dot[j] = 0.f;
    }
    for (int c = place * 32 * U + lane; some > 0 && c - lane < a.slots; c += 32 * U * G) {
        if constexpr (VEC) {
            uint4 qd, qy[J];
            if (c >= a.slots) break;
            qd = *piece<ES>(a.y, t * a.ldy, c);
#pragma unroll
            for (int j = 0; j < J; ++j)
                qy[j] = r[j] >= 0 && r[j] < live ? *piece<ES>(a.x, (int64_t)r[j] * a.hidden, c) : no_piece();
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (r[j] < 0) continue;
                float d[V], y[V];
                to_floats<ES>(qd, d, f16);
                to_floats<ES>(qy[j], y, f16);
                const bool on = r[j] < live;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (on) dot[j] = fmaf(d[k], y[k], dot[j]);
                    d[k] *= w[j];
                }
                put_piece<ES>(a.out, (int64_t)r[j] * a.hidden, c, on ? from_floats<ES>(d, f16) : no_piece());
            }
        } else {
            const Words<ES> dy(a.y, (a.tokens - 1) * a.ldy + a.hidden, t * a.ldy, a.hidden);
            const bool ends = c == lane;    // (the first step works the edges)
            // for rows of either parity
            const uint32_t m[2] = {Words<ES>::whole(c, 0, a.hidden), ES == 2 ? Words<ES>::whole(c, 1, a.hidden) : 0};
            uint32_t qd[2][U];
            dy.load(qd[0], c, 0, m[0]);
            if (ES == 2) dy.load(qd[1], c, 1, m[1]);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (r[j] < 0) continue;
                const bool on = r[j] < live;
                const int64_t e = (int64_t)r[j] * a.hidden;
                const Words<ES> in(a.x, n, e, a.hidden), out(a.out, n, e, a.hidden);
                const bool odd = ES == 2 && out.odd;
                const uint32_t mine = odd ? m[1] : m[0];
                uint32_t q[U] = {0, 0, 0, 0};
                if (on) {
                    in.load(q, c, out.odd, mine);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float d[V], y[V];
                        word_floats<ES>(odd ? qd[1][u] : qd[0][u], d, f16);
                        word_floats<ES>(q[u], y, f16);
#pragma unroll
                        for (int k = 0; k < V; ++k) {
                            dot[j] = fmaf(d[k], y[k], dot[j]);
                            d[k] *= w[j];
                        }
                        q[u] = word_of<ES>(d, f16);
                    }
                }
                out.store(c, q, mine);
                const int edge = ends ? out.edge(lane) : -1;
                if (edge >= 0) {
                    const float d = on ? half_float(dy.at(edge), f16) : 0.f;
                    if (on) dot[j] = fmaf(d, half_float(in.at(edge), f16), dot[j]);
                    out.at(edge) = on ? half_of(d * w[j], f16) : (uint16_t)0;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
    }
    if (G > 1) {
        __syncthreads();
        if (lane < J) part[warp][lane] = lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            dot[j] = 0.f;
            for (int g = 0; g < G; ++g) dot[j] += part[warp / G * G + g][j];
        }
    }
    if (place == 0 && lane < some) a.dweights[s + lane] = lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
}

// Copies of rows on their way to a warp's shared memory, RING_D slots of 128 pieces
// (2 KB of one row): reads of a row stand together in DRAM, none waits for the sum of the one
// before, none holds registers.  A warp takes units u, u + total ..: a token and some
// chunks of its row; a unit's items are, chunk by chunk, the token's own row (if `own`)
// and its k rows.  Each lane reads only what it copied itself, so it waits for nothing
// but its own copies.  (8192 tokens, 8 rows of 2048 bf16 each onto a residual: slots of
// 512 bytes 59-67 us, of 1 KB 57-61, of 2 KB 55-56.  combine_backward, which writes
// beside its reads, was slower this way: 107 us against 97.)
constexpr int RING_D = 4, RING_W = 4, RING_CTAS = 3;       // slots, pieces of a lane in one, CTAs per SM
constexpr int RING_SMEM = RT / 32 * RING_D * RING_W * 32 * 16;

template <int ES>
struct Ring {
    uint4* buf;                             // this lane's pieces: slot, then 32 apart
    int64_t rows;                           // rows from here on are not read
    int u, t, c, end, j, slot;              // the next copy: unit, token, chunk, item, its slot
    int idx, next;                          // rows of that unit, of the one after, a lane each
    int own;

    static __device__ __forceinline__ int total() { return (int)gridDim.x * (RT / 32); }
    static __device__ __forceinline__ int first() { return (int)blockIdx.x + (int)(threadIdx.x >> 5) * (int)gridDim.x; }
    // Chunks [c, end) of token t.
    static __device__ __forceinline__ void place(const RowArgs& a, int u, int& t, int& c, int& end) {
        t = (int)((uint32_t)u / (uint32_t)a.parts);
        c = (u - t * a.parts) * a.span;
        end = min(c + a.span, (a.slots + 32 * RING_W - 1) / (32 * RING_W));
    }
    static __device__ __forceinline__ int token_rows(const RowArgs& a, int u, int64_t rows) {
        return u < a.units ? rows_of(a, (uint32_t)u / (uint32_t)a.parts, 0, rows) : -1;
    }
    __device__ __forceinline__ void start(const RowArgs& a, uint4* smem, int64_t limit) {
        buf = smem + (threadIdx.x >> 5) * (RING_D * RING_W * 32) + (threadIdx.x & 31);
        rows = limit;
        own = a.y != nullptr;
        j = slot = 0;
        u = first();
        place(a, u, t, c, end);
        idx = token_rows(a, u, rows);
        next = token_rows(a, u + total(), rows);
#pragma unroll
        for (int i = 0; i < RING_D - 1; ++i) issue(a);
    }
    __device__ __forceinline__ void issue(const RowArgs& a) {
        if (u < a.units) {
            const bool mine = own && j == 0;
            const int r = __shfl_sync(0xffffffffu, idx, j - own);
            if (mine || r >= 0) {
                const uint4* p = mine ? piece<ES>(a.y, t * a.ldy, 0) : piece<ES>(a.x, (int64_t)r * a.hidden, 0);
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(buf + slot * (RING_W * 32));
#pragma unroll
                for (int i = 0; i < RING_W; ++i) {
                    const int at = (c * RING_W + i) * 32 + (threadIdx.x & 31);
                    if (at < a.slots)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512), "l"(p + at) : "memory");
                }
            }
            if (++j == a.k + own) {
                j = 0;
                if (++c == end) {
                    u += total();
                    place(a, u, t, c, end);
                    idx = next;
                    next = token_rows(a, u + total(), rows);
                }
            }
            if (++slot == RING_D) slot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Makes the copy after those in flight and waits for the oldest of them.
    __device__ __forceinline__ void turn(const RowArgs& a) {
        issue(a);
        asm volatile("cp.async.wait_group %0;" ::"n"(RING_D - 1) : "memory");
    }
};

// combine_kernel for rows on 16 bytes that are not few, the same sums.  Bound by HBM:
// 16384 tokens, 8 rows of 2048 bf16 each onto a residual (671 MB) 107 us, 6.3 TB/s
// (combine_kernel 121); 8192 tokens 56 (61); 4096 tokens, 2 rows of 4096, 24.6 (29.9).
template <int ES>
__global__ void __launch_bounds__(RT, RING_CTAS) combine_ring_kernel(const __grid_constant__ RowArgs a) {
    constexpr int V = 16 / ES;
    extern __shared__ uint4 ring_smem[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, live = live_rows(a);
    const bool f16 = a.dtype == MUON_F16;
    Ring<ES> ring;
    int u = Ring<ES>::first(), slot = 0;
    auto weights = [&](int of) {
        return a.weights && of < a.units && lane < a.k ? a.weights[(int64_t)((uint32_t)of / (uint32_t)a.parts) * a.k + lane] : 1.f;
    };
    int next = Ring<ES>::token_rows(a, u, live);
    float next_weight = weights(u);
    ring.start(a, ring_smem, live);
    for (; u < a.units; u += Ring<ES>::total()) {
        const int mine = next;
        const float weight = next_weight;
        next = Ring<ES>::token_rows(a, u + Ring<ES>::total(), live);
        next_weight = weights(u + Ring<ES>::total());
        int t, c, end;
        Ring<ES>::place(a, u, t, c, end);
        for (; c < end; ++c) {
            float acc[RING_W][V];
#pragma unroll
            for (int i = 0; i < RING_W; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) acc[i][k] = 0.f;
            for (int j = -ring.own; j < a.k; ++j) {
                ring.turn(a);
                const uint4* from = ring.buf + slot * (RING_W * 32);
                if (++slot == RING_D) slot = 0;
                if (j < 0) {
#pragma unroll
                    for (int i = 0; i < RING_W; ++i) to_floats<ES>(from[32 * i], acc[i], f16);
                    continue;
                }
                const float w = __shfl_sync(0xffffffffu, weight, j);
                if (__shfl_sync(0xffffffffu, mine, j) < 0) continue;
#pragma unroll
                for (int i = 0; i < RING_W; ++i) {
                    float v[V];
                    to_floats<ES>(from[32 * i], v, f16);
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[i][k] = fmaf(w, v[k], acc[i][k]);
                }
            }
#pragma unroll
            for (int i = 0; i < RING_W; ++i) {
                const int at = (c * RING_W + i) * 32 + lane;
                if (at < a.slots) put_piece<ES>(a.out, (int64_t)t * a.hidden, at, from_floats<ES>(acc[i], f16));
            }
        }
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
    return a;
}

// Slots of a row: its pieces, or its words, one more where it may start inside one.
int slots_of(const RowArgs& a, bool vec) {
    const int es = (int)esize(a.dtype);
    return vec ? (int)((int64_t)a.hidden * es / 16) : es == 4 ? a.hidden : a.hidden / 2 + 1;
}

template <typename K>
int launch_rows(K kernel, const RowArgs& a, int64_t x, int64_t y, cudaStream_t s, const char* what) {
    note_launch_begin(KC_OTHER, s);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)x, (unsigned)y), dim3(RT), 0, s, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, what);
}

// A token's row in steps of a warp: one warp takes them all once the tokens fill the device.
template <typename K>
int launch_token_rows(K kernel, RowArgs& a, int step, int sms, cudaStream_t s, const char* what) {
    const int steps = (a.slots + step - 1) / step;
    const int each = (int)std::max<int64_t>(1, std::min<int64_t>(steps, a.tokens * steps / ((int64_t)sms * 64)));
    a.span = each * step;
    return launch_rows(kernel, a, (a.tokens + RT / 32 - 1) / (RT / 32), (steps + each - 1) / each, s, what);
}

template <int STEP>
int launch_sort(const SortArgs& a, int C, const DevCtx& dc, cudaStream_t s) {
    static OncePer<int, int> attr;          // by device
    int set = 0;
    cudaError_t e = attr.get(dc.device, &set, [&](int&) {
        cudaError_t r = cudaFuncSetAttribute(expert_sort_kernel<STEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (SORT_WARPS + 1) * (MAX_EXPERTS + 1) * 4);
        if (r == cudaSuccess && STEP == SORTED)
            r = cudaFuncSetAttribute(expert_sort_kernel<STEP>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
    });
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(SORT_T);
    cfg.dynamicSmemBytes = (size_t)(SORT_WARPS + 1) * (size_t)(a.experts_n + 1) * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    if (STEP == SORTED) {
        cudaLaunchAttribute& c = at[cfg.numAttrs++];
        c.id = cudaLaunchAttributeClusterDimension;
        c.val.clusterDim.x = (unsigned)C;
        c.val.clusterDim.y = c.val.clusterDim.z = 1;
    }
    note_launch_begin(KC_OTHER, s);
    e = cudaLaunchKernelEx(&cfg, expert_sort_kernel<STEP>, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "expert sort launch");
}

// Whether combine goes by rings, and the units then: whole tokens, or chunks of
// them while that leaves warps without any.  Rows whose chunks are half empty gain
// nothing (16384 x 512 bf16, 8 choices: 34 us against 33; x 1032 43 both ways), few
// units neither (64 tokens of 2048: 5.2 against 3.5; 256: 5.5 against 5.9).
bool set_ring(RowArgs& a, int sms) {
    const int chunks = (a.slots + 32 * RING_W - 1) / (32 * RING_W);
    if (a.k > 32 || a.slots <= chunks * 16 * RING_W || a.tokens * chunks < 4 * (int64_t)sms) return false;
    const int64_t warps = (int64_t)sms * RING_CTAS * (RT / 32);
    a.span = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, a.tokens * chunks / (warps * 2)));
    a.parts = (chunks + a.span - 1) / a.span;
    a.units = (int)(a.tokens * a.parts);
    return true;
}

template <typename K>
int launch_ring(K kernel, const RowArgs& a, const DevCtx& dc, cudaStream_t s, const char* what) {
    static OncePer<std::pair<int, int>, int> attr;          // by device and element's size
    int set = 0;
    cudaError_t e = attr.get({dc.device, (int)esize(a.dtype)}, &set, [&](int&) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_SMEM);
    });
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    const int64_t ctas = std::min<int64_t>((int64_t)dc.sms * RING_CTAS, (a.units + RT / 32 - 1) / (RT / 32));
    note_launch_begin(KC_OTHER, s);
    e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(RT), RING_SMEM, s, a);
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
    SortArgs a;
    a.experts = experts;
    a.index64 = index_dtype == MUON_I64;
    a.slots = (int)slots;
    a.experts_n = (int)num_experts;
    a.row_of = row_of; a.slot_of = slot_of; a.bounds = bounds;
    if (slots > (int64_t)SORT_CLUSTER * SORT_T * SORT_AHEAD) {
        // more than a cluster's warps keep in registers; 128 slots or more to a warp
        // (262144 slots, 64 experts: 14.9 us, with 64 17.6, with 256 18.5), counts that slot_of has room for
        int64_t C = std::min<int64_t>(dc.sms, std::min<int64_t>(slots / (128 * SORT_WARPS), slots / (num_experts + 1)));
        a.per_warp = (int)((slots + C * SORT_T - 1) / (C * SORT_T)) * 32;
        C = (slots + (int64_t)a.per_warp * SORT_WARPS - 1) / ((int64_t)a.per_warp * SORT_WARPS);
        if ((r = launch_sort<COUNTS>(a, (int)C, dc, s)) || (r = launch_sort<PLACES>(a, (int)C, dc, s))) return r;
        note_launch_begin(KC_OTHER, s);
        const cudaError_t e = launch_pdl(expert_invert_kernel, dim3((unsigned)((slots + 1023) / 1024)), dim3(256), 0, s,
                                         (const int*)row_of, slot_of, (int)slots);
        note_launch_end(KC_OTHER, 0.0, s);
        return e == cudaSuccess ? MUON_OK : cuda_fail(e, "expert sort launch");
    }
    int C = 1;                              // CTAs: a slot per thread until the cluster is full
    while (C < SORT_CLUSTER && (int64_t)C * SORT_T < slots) C *= 2;
    a.per_warp = (int)((slots + (int64_t)C * SORT_T - 1) / ((int64_t)C * SORT_T)) * 32;
    return launch_sort<SORTED>(a, C, dc, s);
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
    a.slots = slots_of(a, vec);
    auto kern = es == 2 ? (vec ? dispatch_kernel<2, true> : dispatch_kernel<2, false>)
                        : (vec ? dispatch_kernel<4, true> : dispatch_kernel<4, false>);
    return launch_token_rows(kern, a, 128, dc.sms, s, "expert dispatch launch");
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
    a.slots = slots_of(a, vec);
    if (vec && set_ring(a, dc.sms))
        return launch_ring(es == 2 ? combine_ring_kernel<2> : combine_ring_kernel<4>, a, dc, s, "expert combine launch");
    auto kern = es == 2 ? (vec ? combine_kernel<2, true> : combine_kernel<2, false>)
                        : (vec ? combine_kernel<4, true> : combine_kernel<4, false>);
    return launch_token_rows(kern, a, vec ? 32 : 128, dc.sms, s, "expert combine launch");
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
    a.slots = slots_of(a, vec);
    const int64_t items = tokens * ((k + 3) / 4);
    a.group = 1;                            // more warps to a token while tokens are too few to fill the device
    while (a.group < RT / 32 && items * a.group < (int64_t)dc.sms * 16 && a.group * (vec ? 32 : 128) < a.slots) a.group *= 2;
    const int per = RT / 32 / a.group;
    auto kern = es == 2 ? (vec ? combine_backward_kernel<2, true> : combine_backward_kernel<2, false>)
                        : (vec ? combine_backward_kernel<4, true> : combine_backward_kernel<4, false>);
    return launch_rows(kern, a, (tokens + per - 1) / per, (k + 3) / 4, s, "expert combine backward launch");
} MUON_CATCH_ALL
