// Products of a block that is split over experts.  Rows are sorted by expert
// (expert e has the rows [bounds[e], bounds[e + 1]), known on the device alone), and
// every expert has matrices of its own:
//
//   gated block   G = X Wg_e^T, U = X Wu_e^T, H = act(G) U over expert e's rows
//     backward    dG = dH U act'(G), dU = dH act(G)
//                 dX = dG Wg_e + dU Wu_e, dWg_e = dG^T X, dWu_e = dU^T X
//   linear        Y = X W_e^T;  dX = dY W_e, dW_e = dY^T X
//
// One persistent launch of 2-SM tcgen05 pairs covers all experts (M = 256, N up to
// 256, fp32 accumulation in TMEM, two accumulators so that a tile's epilogue runs
// under the next tile's products), fed by TMA through a ring of three stages per CTA of
// two k-blocks each (64 KB).  Every warp finds its tiles from the bounds, so no host copy of them is
// needed and a captured call follows new ones.
//
// Results over sorted rows (family a: forward, dX) are computed transposed: 256
// rows of the weights are the M side and an expert's rows the N side, whose extent
// follows the expert (32, or in steps of 64).  An expert's rows are cut into
// ceil(rows / 256) tiles of nearly equal extent, so that ragged or small experts
// cost little more than their rows.  The epilogue turns 32 x 32 chunks
// around in shared memory.  In the gated forward pass each CTA's M side
// is 64 rows of Wg and the same 64 of Wu: gate and value of a result are in two
// warps, which exchange half of their rows through shared memory.  (Sixteen rows of
// each in turn would put them in one warp, but eight copies of 2 KB per stage and
// CTA hold the copy engine up: 16384 rows, 8 x 4096 x 14336 3468 us.)
//
// Where an expert ends inside a tile, rows of the next one are multiplied along
// and not stored (their results are columns of their own, whatever they hold).
// In the weights' gradients (family b) the rows are the contraction, so there an
// expert's last k-block must not hold rows of the next one: a launch before
// copies these blocks, zeros behind their rows, and the products read the copies.
// (Zeroed in shared memory instead, between the copy's arrival and the products, a
// tile waited about 1 us for its last stage: dW of 64 ragged experts of 512 rows on
// average, 2048 x 1024, 146 us against 114 of even ones; now 132 against 118.)
//
// What bounds it: with long contractions the rate at which L2 delivers operands, 64
// bytes per cycle and SM, which a 256 x 256 tile takes in full, and the power cap: 8
// experts of 4096 x 14336, 16384 rows, even: gated forward 1.97-2.3 ms (1.67-1.95
// PFLOP/s, by the card's temperature), linear forward 1.06-1.2, linear backward 2.25-2.4;
// uneven experts, whose last tiles are smaller, 2.37-2.48, 1.1-1.3 and 2.28-2.5.  With short ones (64 experts of
// 512 rows, 2048 x 1024) a tile's epilogue beside its 8 to 32 k-blocks, 60-70 % of the
// product's floor; with few rows HBM (16 rows through 8 experts of 2048 x 8192: 73 us where six
// of them have any, 77 seven, 87 eight, 5.5-6.2 TB/s), and in the weights' gradients of few rows HBM's rate of writes alone.  An
// epilogue of sixteen warps (of 96 registers), plain instead of tile stores, and the weights'
// tiles prefetched into L2 ahead of the ring (gated forward of those uneven experts 2.1-2.2 ->
// 2.55 ms) were built and were slower.
#include "epilogue.cuh"
#include "glu_parts.cuh"

#include <climits>

namespace muon {

namespace {

using namespace tc;

constexpr int GM = 128;                     // rows of a CTA's half of the M side
constexpr int GK = 64;                      // k-block: 128 bytes
constexpr int NEPI = 8;
constexpr int GT = 64 + 32 * NEPI;          // producer, issuer, epilogue
// k-blocks of a stage.  A stage costs its waits and its copies' issue whatever it
// holds: gated forward 16384 rows, 8 x 4096 x 14336: two 1972 us, one 2097 (short
// contractions, as of 64 experts of 512 rows, gain 1 % with one); three 2360, too
// coarse a ring.
constexpr int SUB = 2;
constexpr int STAGES = 6 / SUB;
constexpr int OP_BYTES = GM * GK * 2;       // one operand's k-block of a stage (A, or this CTA's half of B)
constexpr int OUT_BYTES = 32 * 32 * 2;      // output chunk of a warp: 32 x 32, 64-byte swizzled rows
constexpr int NBARS = 2 * STAGES + 5;
constexpr int EXP_SMEM = STAGES * SUB * 2 * OP_BYTES + NEPI * 2 * OUT_BYTES + NBARS * 8 + 16 + 1024;
static_assert(EXP_SMEM <= 232448, "shared memory per CTA");
constexpr int GROUP = 16;                   // row tiles that share their weights' tiles in L2
constexpr int ROW_TILE = 256;
// The accumulators truncate: a sum of n terms of one sign comes out short by
// 6.4e-9 n of its value, so contractions are cut into parts of at most MAX_BLOCKS
// k-blocks (65536 terms), whose fp32 sums are added in round-to-nearest.
constexpr int MAX_BLOCKS = 1024;
constexpr size_t PART_BYTES = (size_t)GM * 256 * 4;     // a CTA's running sums

// wait_bounded(), which reads the clock as soon as a wait does not succeed at once:
// some hundred nanoseconds that a stage of a full ring then comes late (linear
// forward 16384 x 14336 x 4096 in eight ragged experts: 1217 -> 1120 us with one
// k-block per stage).  Here the clock starts after the waits of a normal pass.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_bounded(bar, parity, abort_flag, status);
}

// The address of a barrier of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t bar_of(uint32_t bar, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(bar), "r"(rank));
    return r;
}

// A tile load to this CTA's shared memory that reports to a barrier (bar_of) of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 128 columns from c of 64 rows from r of matrix z, as two blocks of 64 columns:
// one copy from a map by blocks of columns, or two.
__device__ __forceinline__ void load_columns(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, int r, int z,
                                             bool whole) {
    if (whole) {
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(r), "r"(c / 64), "r"(z)
            : "memory");
    } else {
        tma_load_pair(dst, map, bar, c, r, z);
        tma_load_pair(dst + OP_BYTES / 2, map, bar, c + 64, r, z);
    }
}

enum Mode : int { FWD_GLU = 0, FWD_LINEAR = 1, BACKWARD = 2 };

// Division of numbers below 2^31 by a number known beforehand: the product with
// 2^32 / d, rounded up, is at most one too high.
struct Div {
    uint32_t d, m;
    __host__ __device__ __forceinline__ void set(int by) {
        d = (uint32_t)(by < 1 ? 1 : by);
        m = 0xffffffffu / d + 1;                // (0 for 1)
    }
    __device__ __forceinline__ int of(int n) const {
        uint32_t q = d == 1 ? (uint32_t)n : __umulhi((uint32_t)n, m);
        if (q * d > (uint32_t)n) --q;
        return (int)q;
    }
};

struct ExpArgs {
    int dtype, act;
    int save;                   // gated forward: G and U leave too
    int tma_out;                // outputs' rows start on 16 bytes
    int whole_a, whole_a2, whole_b2;        // MN-major operands' maps are by blocks of 64 columns
    int rows, experts;
    const int* bounds;
    // family a: results over the sorted rows (forward, dX)
    int a_on, cols_a, tiles_w;  // columns of the result, tiles of them
    int seg_blocks, segs;       // k-blocks of one segment (one A and B map each), segments
    // family b: the weights' gradients
    int nb;                     // results per expert: 0, 1 or 2
    int rows_b, cols_b, tiles_mb, tiles_nb;
    int tails_by_row;           // tail_block()
    Div group_a, group_b, rest_b, matrix_b;     // tiles of a group of either family, rows of b's last group, tiles of a result of b
    GluOut out[3];              // H, G, U; Y; or dX, dW, dWu
    float* part;                // running sums of contractions in several parts
    int* status;
    int stall;                  // test hook: k + 1 = CTA 0 leaves the k-th stage that it comes to unfilled; 0 = off
};

// Extents of family a's tiles: 32, or multiples of 64 rows, half of them per CTA in
// one box, so that each copy brings the tile's rows alone.
constexpr int BOXES = 5;
__host__ __device__ constexpr int box_rows(int i) { return i == 0 ? 16 : 32 * i; }

struct ExpMaps {
    CUtensorMap a[2];           // family a: weights by segment (gated forward: Wg, Wu)
    CUtensorMap b[2][BOXES];    // rows by segment, in boxes of box_rows()
    CUtensorMap a2[2], b2;      // family b: dG, dU (dY) read MN-major; X
    CUtensorMap a2_tail[2], b2_tail;        // the experts' last k-blocks of them
    CUtensorMap out[3];
};

// [first, last) of `rows` rows that are expert e's, whatever the bounds hold.
__device__ __forceinline__ void expert_rows(const int* bounds, int rows, int e, int& first, int& last) {
    const int lo = e == 0 ? 0 : bounds[e];
    first = min(max(lo, 0), rows);
    last = min(max(bounds[e + 1], first), rows);
}

// The block of the scratch that holds an expert's last k-block: its own, or, where rows
// are fewer than experts, its first row's, so that no more blocks than rows are
// kept (256 experts of 7168 x 2048, 64 rows: 92 MB, by experts 369).
__device__ __forceinline__ int tail_block(bool by_row, int e, int first) { return by_row ? first : e; }

struct Tile {
    int family, which;          // 0: a, 1: b; output index
    int e;
    int first, last;            // the expert's rows
    int r0, n;                  // family a: the tile's first row, and its extent
    int tm, tn;                 // family a: tn = weights' tile; b: row and column tile
    int blocks;                 // k-blocks of its contraction (0: the result is zero)
};

// The tiles of one cluster, in order.  Family a's go round-robin, the clusters
// left with one fewer then take `extra` of family b's, and the rest of family b
// goes round-robin starting with those: with a's tiles the longer ones, every
// cluster ends within a tile of the others.
//
// Every warp walks them, so a step between tiles is on everybody's way: nothing is
// divided but by numbers known before, of an expert's once per expert (128 rows through
// 8 experts of 4096 x 14336, whose gradients' tiles are a k-block each: backward 844 ->
// 812 us).
template <bool B>                           // with a family b
struct Walk {
    int c, P, j;
    int nb, mine, light, extra;
    // family a: current expert, id of its first tile, its rows and tiles, tiles along its rows, their extent
    int e, base, first, last, here, along, per, ready;
    Div rest;                               // rows of tiles of its last group
    int end;                                // of the experts' rows; "expert" g.experts has those behind, results zero

    __device__ __forceinline__ void tiles_of(const ExpArgs& g) {
        if (e < g.experts) {
            expert_rows(g.bounds, g.rows, e, first, last);
        } else {
            first = end;
            last = g.rows;
        }
        along = (last - first + ROW_TILE - 1) / ROW_TILE;
        here = along * g.tiles_w;
    }
    // Called by whole warps.
    __device__ __forceinline__ void init(const ExpArgs& g, int cluster, int clusters) {
        c = cluster;
        P = clusters;
        j = 0;
        int na = 0;
        const int lane = threadIdx.x & 31;
        end = 0;
        if (g.a_on) {
            for (int k = lane; k < g.experts; k += 32) {
                int lo, hi;
                expert_rows(g.bounds, g.rows, k, lo, hi);
                na += (hi - lo + ROW_TILE - 1) / ROW_TILE * g.tiles_w;
                end = max(end, hi);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                na += __shfl_xor_sync(0xffffffffu, na, d);
                end = max(end, __shfl_xor_sync(0xffffffffu, end, d));
            }
            na += (g.rows - end + ROW_TILE - 1) / ROW_TILE * g.tiles_w;
        }
        const int r = na % P;
        mine = na / P + (c < r ? 1 : 0);
        light = r ? P - r : 0;
        nb = B ? g.experts * g.nb * g.tiles_mb * g.tiles_nb : 0;
        // a tile's time in k-blocks; one of few costs what its results take to leave
        const int ca = max(8, g.segs * g.seg_blocks);
        const int cb = max(8, (g.rows / g.experts + GK - 1) / GK);
        extra = light ? min(nb / light, (ca + cb / 2) / cb) : 0;
        e = 0;
        base = 0;
        ready = -1;
        tiles_of(g);
    }
    // The next tile; t holds the one before.
    __device__ __forceinline__ bool next(const ExpArgs& g, Tile& t) {
        if (j < mine) {
            int l = c + j * P;
            ++j;
            while (l >= base + here && e < g.experts) {
                base += here;
                ++e;
                tiles_of(g);
            }
            l -= base;
            if (l < 0 || l >= here) {       // bounds that fall over and over, more tiles than 2^31: nothing
                t = Tile{};
                return true;
            }
            if (ready != e) {               // (not for the experts passed by)
                ready = e;
                per = extent((last - first + along - 1) / along);
                rest.set(along % GROUP);
            }
            t.family = 0;
            t.which = 0;
            t.e = e;
            t.first = first;
            t.last = last;
            t.blocks = e == g.experts ? 0 : g.segs * g.seg_blocks;
            place(l, along, g.group_a, rest, t);
            t.r0 = first + t.tm * per;
            t.n = min(per, extent(last - t.r0));
            return true;
        }
        if (!B) return false;
        const int k = j - mine;
        ++j;
        int id;
        const int lead = light * extra;
        if (light && c >= P - light) id = k < extra ? (c - (P - light)) + k * light : lead + (c - (P - light)) + (k - extra) * P;
        else id = lead + (light ? light + c : c) + k * P;
        if (id >= nb) return false;
        const int matrix = g.matrix_b.of(id), expert = matrix >> (g.nb - 1);        // one or two of an expert
        if (t.family == 0 || t.e != expert) {
            expert_rows(g.bounds, g.rows, expert, t.first, t.last);
            t.blocks = (t.last - t.first + GK - 1) / GK;
        }
        t.family = 1;
        t.e = expert;
        t.which = matrix & (g.nb - 1);
        place(id - matrix * (int)g.matrix_b.d, g.tiles_mb, g.group_b, g.rest_b, t);
        return true;
    }
    static __device__ __forceinline__ int extent(int rows) { return rows <= 32 ? 32 : (rows + 63) & ~63; }
    // Tile l of tiles in groups of GROUP rows (the last one may have fewer, `rest`), down a group's columns.
    static __device__ __forceinline__ void place(int l, int tiles_m, const Div& group, const Div& rest, Tile& t) {
        const int grp = group.of(l), from = grp * GROUP;
        l -= grp * (int)group.d;
        if (tiles_m - from >= GROUP) {
            t.tm = from + l % GROUP;
            t.tn = l / GROUP;
        } else {
            t.tn = rest.of(l);
            t.tm = from + l - t.tn * (int)rest.d;
        }
    }
};

// Where a chunk of results goes: 32 rows from r0 of `rows`, 32 columns from c0 of
// `cols`, of matrix z (z_rows rows each).
struct Place {
    int rows, cols, r0, c0, z, z_rows;
};

// Whether a chunk of `n` rows leaves as a tile: a tile store ends with the matrix, an
// expert's last rows leave row by row.
__device__ __forceinline__ bool as_tile(const Place& p, int n) { return p.r0 + n <= p.rows || p.rows == p.z_rows; }

// The warp's next output buffer, once the store that last used it has read it.
__device__ __forceinline__ uint8_t* out_buffer(uint8_t* stage, int groups, bool tile) {
    if (groups >= 2 || !tile) {
        if ((threadIdx.x & 31) == 0) {
            if (tile) bulk_wait_read1();
            else bulk_wait_read0();
        }
        __syncwarp();
    }
    return stage + (groups & 1) * OUT_BYTES;
}

__device__ __forceinline__ uint32_t pack2_h(float lo, float hi, bool f16) {
    if (f16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Offset of 16-byte piece k of row r in a chunk: 64-byte swizzle, piece k at k ^ ((r / 2) % 4).
__device__ __forceinline__ int piece_at(int r, int k) { return r * 64 + ((k ^ ((r >> 1) & 3)) << 4); }

// A chunk of a matrix whose rows start on 16 bytes that does not leave as a tile: rows up to
// p.rows, eight of them per step.
__device__ __forceinline__ void store_rows(const GluOut& o, const Place& p, const uint8_t* buf) {
    const int lane = threadIdx.x & 31, n = min(32, p.rows - p.r0), k = lane & 3;
    uint16_t* out = static_cast<uint16_t*>(o.p) + ((int64_t)p.z * p.z_rows + p.r0) * o.ld + p.c0;
    for (int i = lane >> 2; i < n; i += 8)
        if (p.c0 + 8 * k < p.cols)
            *reinterpret_cast<uint4*>(out + (int64_t)i * o.ld + 8 * k) = *reinterpret_cast<const uint4*>(buf + piece_at(i, k));
}

// N rows of a chunk of other matrices, a column per lane: a row's 32 columns per store
// (by way of shared memory 16 experts of 1001 x 2731, 16384 rows, took 305 us, so 249).
template <int N>
__device__ __forceinline__ void store_columns(const GluOut& o, const Place& p, const float (&v)[32], bool f16) {
    const int lane = threadIdx.x & 31, n = p.rows - p.r0;
    uint16_t* out = static_cast<uint16_t*>(o.p) + ((int64_t)p.z * p.z_rows + p.r0) * o.ld + p.c0 + lane;
    if (p.c0 + lane >= p.cols) return;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const uint32_t q = pack2_h(v[k], v[k + 1], f16);
        if (k < n) out[(int64_t)k * o.ld] = (uint16_t)q;
        if (k + 1 < n) out[(int64_t)(k + 1) * o.ld] = (uint16_t)(q >> 16);
    }
}

// One warp's 32 rows x 64 columns of family b, a row per lane, in two steps of 32
// columns: both into the warp's two buffers as 128-byte rows (swizzled: piece k of row
// r at k ^ (r % 8)), then one store (32 columns per store: backward of the case above
// 812 us instead of 783).  A cluster's tiles of family b come after those of a.
__device__ __forceinline__ void put_half(const float (&v)[32], int step, bool f16, uint8_t* stage) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(stage + lane * 128 + (((step * 4 + k) ^ (lane & 7)) << 4)) = pack8_h(v + 8 * k, f16);
}

template <bool TILES>
__device__ __forceinline__ void store_wide(const CUtensorMap* map, const GluOut& o, const Place& p,
                                           uint8_t* stage, int& groups) {
    const int lane = threadIdx.x & 31;
    if (TILES) {                            // (a tile store ends with the expert's matrix)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, smem_u32(stage), p.c0, p.r0, p.z);
            bulk_commit();
        }
        groups = 2;                         // both buffers are taken
        return;
    }
    __syncwarp();
    const int n = min(32, p.rows - p.r0);
    uint16_t* out = static_cast<uint16_t*>(o.p) + ((int64_t)p.z * p.z_rows + p.r0) * o.ld + p.c0;
#pragma unroll
    for (int c = lane; c < 64; c += 32) {
        if (p.c0 + c >= p.cols) break;
#pragma unroll 8
        for (int i = 0; i < n; ++i)
            out[(int64_t)i * o.ld + c] = *reinterpret_cast<const uint16_t*>(stage + i * 128 + (((c >> 3) ^ (i & 7)) << 4) + (c & 7) * 2);
    }
    __syncwarp();
}

// Rows k and k + 1 (even k) of a warp's chunk, a column per lane.  (Neighbours that exchanged
// a value of each pair and stored two columns took longer, for the instructions: 65536
// rows, 256 experts of 1024 x 512: linear forward 168 us, 119 so; gated 275, 200.)
__device__ __forceinline__ void put_rows(uint8_t* buf, int k, float lo, float hi, bool f16) {
    const int lane = threadIdx.x & 31;
    const uint32_t q = pack2_h(lo, hi, f16);
    uint16_t* at = reinterpret_cast<uint16_t*>(buf + k * 64 + (((lane >> 3) ^ ((k >> 1) & 3)) << 4) + (lane & 7) * 2);
    at[0] = (uint16_t)q;
    at[32] = (uint16_t)(q >> 16);
}

// One warp's 32 x 32 chunk, a column per lane.
template <bool TILES>
__device__ __forceinline__ void store_turned(const ExpArgs& g, const CUtensorMap* map, const GluOut& o, const Place& p,
                                             const float (&v)[32], uint8_t* stage, int& groups) {
    const int lane = threadIdx.x & 31;
    const bool tile = as_tile(p, 32), f16 = g.dtype == MUON_F16;
    if (!TILES) {
        store_columns<32>(o, p, v, f16);
        __syncwarp();
        return;
    }
    uint8_t* buf = out_buffer(stage, groups, tile);
#pragma unroll
    for (int k = 0; k < 32; k += 2) put_rows(buf, k, v[k], v[k + 1], f16);
    if (tile) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (tile) {
        if (lane == 0) {
            tma_store_3d(map, smem_u32(buf), p.c0, p.r0, p.z);
            bulk_commit();
        }
        ++groups;
        return;
    }
    store_rows(o, p, buf);
    __syncwarp();
}

// The two warps that hold G and U of the same columns.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
// Whether both of them say so.
__device__ __forceinline__ bool pair_all(int id, bool v) {
    int all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.and.pred q, %2, 64, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"((uint32_t)v), "r"(id) : "memory");
    return all != 0;
}

// One copy of the loop per activation: chosen per element, the code of the other two
// stands between the elements of the one, and an epilogue of 32 chunks spends
// its time fetching it (64 experts, 512 rows each, 2048 x 1024: 383 us per call, 316
// with one copy each).
template <int ACT>
__device__ __forceinline__ void times_act(const float (&gate)[16], float (&v)[32]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        if constexpr (ACT == ACT_GELU) {
            v[k] *= activate<false>(gate[k], ACT, nullptr);
            continue;
        }
        // g sigmoid(z), as activate() has it but for the quotient: two ulp instead of half
        // of one, far below the results' rounding, for a third of the instructions (286 us
        // -> 207 in the case above).  With e^-|z| the divisor is between 1 and 2: the fast
        // quotient by more than 2^126 is 0, which e^-z reaches at z = -87, where bf16 still
        // holds the result.
        const float x = gate[k];
        const float z = ACT == ACT_SILU ? x : 1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.0f);
        const float t = __expf(-fabsf(z));
        v[k] *= __fdividef(z < 0.f ? x * t : x, 1.0f + t);
    }
}

// A pair's 32 x 32 chunk of the gated block, a column per lane, G in one warp and U
// in the other.  Each stores its own matrix where it is kept; then they exchange half
// of their rows through their second buffers and write the results of 16 rows each.
template <bool TILES>
__device__ __forceinline__ void store_gated(const ExpArgs& g, const CUtensorMap* maps, const Place& p, bool is_up, int id,
                                            float (&v)[32], uint8_t* stage, uint8_t* others, int& groups) {
    const int lane = threadIdx.x & 31;
    const bool f16 = g.dtype == MUON_F16;
    if (g.save) {
        int own = 0;                        // (the first buffer, whatever was stored before)
        const int w = is_up ? 2 : 1;
        if (groups > 0) {
            if (lane == 0) bulk_wait_read0();
            __syncwarp();
        }
        store_turned<TILES>(g, &maps[w], g.out[w], p, v, stage, own);
        groups += own;
    } else if (groups > 0) {
        if (lane == 0) bulk_wait_read0();
        __syncwarp();
    }
    // rows 0 .. 15 are the G warp's, rows 16 .. 31 the U warp's
    float4* send = reinterpret_cast<float4*>(stage + OUT_BYTES);
    const float4* got = reinterpret_cast<const float4*>(others + OUT_BYTES);
#pragma unroll
    for (int k = 0; k < 16; k += 4)
        send[k * 8 + lane] = is_up ? make_float4(v[k], v[k + 1], v[k + 2], v[k + 3])
                                   : make_float4(v[16 + k], v[17 + k], v[18 + k], v[19 + k]);
    pair_sync(id);
    float gate[16];
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
        const float4 q = got[k * 8 + lane];
        const float o[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gate[k + i] = is_up ? o[i] : v[k + i];
            v[k + i] = is_up ? v[16 + k + i] : o[i];
        }
    }
    pair_sync(id);                          // the other has read this warp's
    if (g.act == ACT_GELU) times_act<ACT_GELU>(gate, v);
    else if (g.act == ACT_GELU_TANH) times_act<ACT_GELU_TANH>(gate, v);
    else times_act<ACT_SILU>(gate, v);
    Place mine = p;
    mine.r0 += is_up ? 16 : 0;
    if (mine.r0 >= p.rows) return;
    if (!TILES) {
        store_columns<16>(g.out[0], mine, v, f16);
        __syncwarp();
        return;
    }
    const bool tile = as_tile(mine, 16);
    uint8_t* buf = stage + OUT_BYTES;
#pragma unroll
    for (int k = 0; k < 16; k += 2) put_rows(buf, k, v[k], v[k + 1], f16);
    if (tile) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (tile) {
        if (lane == 0) {
            tma_store_3d(&maps[0], smem_u32(buf), p.c0, mine.r0, 0);
            bulk_commit();
        }
        ++groups;
        return;
    }
    mine.rows = min(p.rows, mine.r0 + 16);
    store_rows(g.out[0], mine, buf);
    __syncwarp();
}

// TILES: the outputs' rows start on 16 bytes, so that chunks can leave by tile stores (a
// form of its own: the code of the other between costs the gated forward pass 2 %).
template <int MODE, bool TILES>
__global__ void __launch_bounds__(GT, 1)
expert_kernel(const __grid_constant__ ExpMaps maps, const __grid_constant__ ExpArgs g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * SUB * OP_BYTES;
    uint8_t* sOut = sB + STAGES * SUB * OP_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + NEPI * 2 * OUT_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, accf0 = empty0 + 8 * STAGES;
    const uint32_t acce0 = accf0 + 16, drain_bar = acce0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 2);                    // the even CTA's: both CTAs' copies
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf0 + 8 * i, 1);
            mbar_init(acce0 + 8 * i, 2 * NEPI);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc2(smem_u32(tmem_slot), 512);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    Walk<MODE == BACKWARD> w;
    w.init(g, (int)cluster_idx(), (int)cluster_count());
    Tile t = {};
    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            uint32_t flight = 0, phases = 0;            // per stage: copies were issued, and their phase
            const uint32_t full_pair = bar_of(full0, 0), a0 = smem_u32(sA), b0 = smem_u32(sB);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int until_stall = blockIdx.x == 0 ? g.stall : 0;
            // waits for a stage to be free and says how many bytes the pair's copies bring;
            // false where this CTA brings none
            auto open = [&](uint32_t bytes) {
                ok = wait_for(empty0 + 8 * stage, phase ^ 1u, abort_flag, g.status);
                if (!ok) return false;
                if (until_stall && --until_stall == 0) return false;
                if (rank == 0) mbar_expect_tx(full0 + 8 * stage, 2 * bytes);
                else arrive_relaxed(full_pair + 8 * stage);
                flight |= 1u << stage;
                phases = (phases & ~(1u << stage)) | (phase << stage);
                return true;
            };
            auto close = [&] {
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            while (ok && w.next(g, t)) {
                if (MODE == BACKWARD && t.family) {
                    const bool ragged = (t.last - t.first) % GK != 0;
                    const int m0 = t.tm * 2 * GM + rank * GM, n0 = t.tn * 2 * GM + rank * GM;
                    const CUtensorMap *ma = &maps.a2[t.which], *mb = &maps.b2;
                    int k0 = t.first;
                    for (int left = t.blocks; left > 0; left -= SUB) {
                        if (!open((uint32_t)(min(left, SUB) * 2 * OP_BYTES))) {
                            if (!ok) break;
                            close();
                            continue;
                        }
                        const uint32_t bar = full_pair + 8 * stage, at = (uint32_t)(stage * SUB * OP_BYTES);
#pragma unroll
                        for (int i = 0; i < SUB; ++i) {
                            if (i >= left) break;
                            if (ragged && left - i == 1) {
                                // a last k-block of fewer rows stands padded with zeros in the scratch
                                ma = &maps.a2_tail[t.which];
                                mb = &maps.b2_tail;
                                k0 = tail_block(g.tails_by_row, t.e, t.first) * GK;
                            }
                            load_columns(a0 + at + i * OP_BYTES, ma, bar, m0, k0, 0, g.whole_a2);
                            load_columns(b0 + at + i * OP_BYTES, mb, bar, n0, k0, 0, g.whole_b2);
                            k0 += GK;
                        }
                        close();
                    }
                    continue;
                }
                const int hn = t.n / 2, r0 = t.r0 + rank * hn;      // this CTA's rows of the tile
                const int c0 = MODE == FWD_GLU ? t.tn * GM + rank * (GM / 2) : t.tn * 2 * GM + rank * GM;
                const uint32_t bytes = OP_BYTES + hn * GK * 2;
                const CUtensorMap *ma = &maps.a[0], *mb = &maps.b[0][hn / 32];
                int k0 = 0;
                for (int left = t.blocks; left > 0; left -= SUB) {
                    if (!open(min(left, SUB) * bytes)) {
                        if (!ok) break;
                        close();
                        continue;
                    }
                    const uint32_t bar = full_pair + 8 * stage, at = (uint32_t)(stage * SUB * OP_BYTES);
#pragma unroll
                    for (int i = 0; i < SUB; ++i) {
                        if (i >= left) break;
                        const uint32_t a = a0 + at + i * OP_BYTES, b = b0 + at + i * OP_BYTES;
                        if (MODE == FWD_GLU) {
                            tma_load_pair(a, &maps.a[0], bar, k0, c0, t.e);
                            tma_load_pair(a + OP_BYTES / 2, &maps.a[1], bar, k0, c0, t.e);
                        } else if (MODE == FWD_LINEAR) {
                            tma_load_pair(a, &maps.a[0], bar, k0, c0, t.e);
                        } else {
                            load_columns(a, ma, bar, c0, k0, t.e, g.whole_a);
                        }
                        tma_load_pair(b, mb, bar, k0, r0, 0);
                        k0 += GK;
                        if (MODE == BACKWARD && k0 >= g.seg_blocks * GK) {      // from dG Wg to dU Wu
                            k0 = 0;
                            ma = &maps.a[1];
                            mb = &maps.b[1][hn / 32];
                        }
                    }
                    close();
                }
            }
            // copies still in flight (after an abort nobody consumes them): the even CTA
            // sees those of both in the stages that it has opened (see the end for others)
            for (int s = 0; s < STAGES; ++s)
                if (rank == 0 && ((flight >> s) & 1)) wait_drain(full0 + 8 * s, (phases >> s) & 1);
        }
        __syncwarp();
    } else if (warp == 1 && rank == 1) {
        // (the even CTA issues the pair's products)
    } else if (warp == 1) {
        // ---------------- MMA issuer (even CTA) ----------------
        if (lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, aphase = 0;
            bool ok = true;
            constexpr bool A_MN = MODE == BACKWARD;     // the weights (dX) or rows (dW) as stored are MN-major there
            const uint64_t ad0 = A_MN ? sdesc(smem_u32(sA), GK * 128, 1024) : sdesc(smem_u32(sA), 16, 1024);
            while (ok && w.next(g, t)) {
                const bool b_mn = MODE == BACKWARD && t.family;
                const uint32_t idesc =
                    idesc_f16kind(2 * GM, t.family ? 256 : t.n, b_mn, g.dtype == MUON_F16) | (A_MN ? (1u << 15) : 0u);
                const uint64_t bd0 = b_mn ? sdesc(smem_u32(sB), GK * 128, 1024) : sdesc(smem_u32(sB), 16, 1024);
                const int b_step = b_mn ? 2048 / 16 : 2;
                for (int from = 0; ok && from < t.blocks; from += MAX_BLOCKS) {
                    const int upto = min(from + MAX_BLOCKS, t.blocks);
                    if (!wait_for(acce0 + 8 * acc, aphase ^ 1u, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(acc * 256);
                    for (int k1 = from; k1 < upto; k1 += SUB) {
                        if (!wait_for(full0 + 8 * stage, phase, abort_flag, g.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < SUB; ++i) {
                            if (k1 + i >= upto) break;
                            // (addresses count in 16 bytes in a descriptor's lowest bits)
                            const uint64_t at = (uint64_t)((stage * SUB + i) * (OP_BYTES / 16));
#pragma unroll
                            for (int kk = 0; kk < GK / 16; ++kk)
                                tc_mma2_bf16(d, ad0 + at + kk * (A_MN ? 2048 / 16 : 2), bd0 + at + kk * b_step, idesc,
                                             (k1 + i > from || kk > 0) ? 1u : 0u);
                        }
                        tc_commit2(empty0 + 8 * stage, (uint16_t)0x3);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    tc_commit2(accf0 + 8 * acc, (uint16_t)0x3);
                    acc ^= 1;
                    if (acc == 0) aphase ^= 1u;
                }
            }
            if (!ok) {
                tc_commit2(drain_bar, (uint16_t)0x1);
                wait_drain(drain_bar, 0);
            }
        }
        __syncwarp();
    } else {
        // ---------------- epilogue (warps 2..9) ----------------
        const int q = warp & 3, half = (warp - 2) / 4;
        uint8_t* stage = sOut + (warp - 2) * 2 * OUT_BYTES;
        // gated forward: quarters 0, 1 hold G and quarters 2, 3 U of the same columns
        const int pair = 1 + half * 2 + (q & 1);
        uint8_t* others = sOut + (((warp - 2) & ~3) + ((warp - 2 + 2) & 3)) * 2 * OUT_BYTES;
        int groups = 0, acc = 0;
        uint32_t aphase = 0;
        bool ok = true;
        while (ok && w.next(g, t)) {
            Place p;
            int o = 0, chunks;              // output, 32-column chunks of the accumulator
            if (MODE == BACKWARD && t.family) {
                p = Place{g.rows_b, g.cols_b, t.tm * 2 * GM + rank * GM + q * 32, t.tn * 2 * GM, t.e, g.rows_b};
                o = 1 + t.which;
                chunks = min(8, (p.cols - p.c0 + 31) / 32);
                if (p.r0 >= p.rows) chunks = 0;
            } else {
                const int c0 = MODE == FWD_GLU ? t.tn * GM + rank * (GM / 2) + (q & 1) * 32 : t.tn * 2 * GM + rank * GM + q * 32;
                p = Place{t.last, g.cols_a, t.r0, c0, 0, g.rows};
                chunks = c0 < p.cols ? t.n / 32 : 0;
            }
            // chunk ch: rows 32 ch.. (family a) or columns 32 ch.. (family b, which takes them by twos)
            const int by = MODE == BACKWARD && t.family ? 2 : 1, first = half * by, step = 2 * by;
            auto chunk = [&](int ch, float(&v)[32]) {
                Place c = p;
                if (MODE == BACKWARD && t.family) {
                    c.c0 += 32 * (ch & ~1);
                    if ((ch & 1) == 0 && groups > 0) {
                        if (lane == 0) bulk_wait_read0();
                        __syncwarp();
                    }
                    put_half(v, ch & 1, g.dtype == MUON_F16, stage);
                    if ((ch & 1) || ch + 1 == chunks) store_wide<TILES>(&maps.out[o], g.out[o], c, stage, groups);
                } else {
                    c.r0 += 32 * ch;
                    if (MODE == FWD_GLU) store_gated<TILES>(g, maps.out, c, q >= 2, pair, v, stage, others, groups);
                    else store_turned<TILES>(g, &maps.out[0], g.out[0], c, v, stage, groups);
                }
            };
            if (t.blocks == 0) {
                // nothing to sum (an expert without rows, rows behind the last expert)
                float v[32];
#pragma unroll 1
                for (int c0 = first; c0 < chunks; c0 += step)
#pragma unroll 1
                    for (int ch = c0; ch < min(c0 + by, chunks); ++ch) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0.f;
                        chunk(ch, v);
                    }
                continue;
            }
            for (int from = 0; from < t.blocks; from += MAX_BLOCKS) {
                const bool got = wait_for(accf0 + 8 * acc, aphase, abort_flag, g.status);
                // a pair goes on together, whichever of its warps saw the wait give up
                ok = MODE == FWD_GLU ? pair_all(pair, got) : __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
                const bool more = from + MAX_BLOCKS < t.blocks;
                // this thread's running sums: its lane of the accumulator, 256 columns
                float* part = g.part + ((size_t)blockIdx.x * GM + q * 32 + lane) * 256;
                auto release = [&] {        // the accumulator has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 1) mbar_arrive_remote(acce0 + 8 * acc, 0);
                        else mbar_arrive(acce0 + 8 * acc);
                    }
                };
                if (first >= chunks) release();
                int ch = first;
#pragma unroll 1
                while (ch < chunks) {
                    float v[32];
                    tmem_ld32(lanes + (uint32_t)(ch * 32), v);
                    const int next = by == 2 && (ch & 1) == 0 ? ch + 1 : ch + step - by + 1;
                    if (next >= chunks) release();
                    float* at = part + ch * 32;
                    if (from) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(at + k);
                            v[k] += f.x;
                            v[k + 1] += f.y;
                            v[k + 2] += f.z;
                            v[k + 3] += f.w;
                        }
                    }
                    if (more) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(at + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    } else {
                        chunk(ch, v);
                    }
                    ch = next;
                }
                acc ^= 1;
                if (acc == 0) aphase ^= 1u;
            }
        }
        if (groups > 0 && lane == 0) bulk_wait0();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // After an abort the odd CTA may have copies in flight that the even one does not know
    // of, also where its producer had come to its end: it waits out the limit on a
    // barrier that nothing completes.  (Without one its epilogue has seen every product done.)
    if (rank == 1 && warp == 0) {
        if (lane == 0 && *abort_flag) wait_drain(full0, 0);
        __syncwarp();
    }
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

// Up to three dense matrices of 16-bit elements whose rows start anywhere, copied to
// pitches of whole 16-byte pieces (zeros behind the columns).  A warp takes a row,
// 128 pieces at a time: every lane loads four aligned vectors and shifts them into
// place with its neighbours'.  Bound by HBM: the weights and rows of 20 experts of
// 1001 x 2731 (285 MB read and written) 43 us.  Matrices of experts without rows are
// left out: no product reads them.
struct PadRows {
    const void* src[3];
    void* dst[3];
    int64_t rows[3];
    int cols[3];
    Div each[3];                // rows of an expert's matrix; 0: the rows are not the experts'
    const int* bounds;
    int all;                    // sorted rows
};

__global__ void __launch_bounds__(256) pad_rows_kernel(const __grid_constant__ PadRows a) {
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const int o = blockIdx.y, lane = threadIdx.x & 31, cols = a.cols[o], pieces = (cols + 7) / 8;
    const int64_t rows = a.rows[o], n = rows * cols, step = (int64_t)gridDim.x * 8;
    for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += step) {
        if (a.each[o].d) {
            int first, last;
            expert_rows(a.bounds, a.all, a.each[o].of((int)row), first, last);
            if (first == last) continue;
        }
        const uint16_t* at = static_cast<const uint16_t*>(a.src[o]) + row * cols;
        const int off = (int)(reinterpret_cast<uintptr_t>(at) & 15) / 2;
        const int64_t e = row * cols - off;         // element of slot 0
        at -= off;
        // slot i: columns 8 i - off .., as far as it has any of the row's
        auto slot = [&](int i) {
            if (8 * i - off >= cols) return make_uint4(0, 0, 0, 0);
            if (e + 8 * i >= 0 && e + 8 * i + 8 <= n) return *reinterpret_cast<const uint4*>(at + 8 * i);
            uint32_t w[4] = {0, 0, 0, 0};           // at the matrix' two ends
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (8 * i + k >= off && 8 * i + k < off + cols) w[k / 2] |= (uint32_t)at[8 * i + k] << (16 * (k & 1));
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        uint4* dst = static_cast<uint4*>(a.dst[o]) + row * pieces;
        for (int i0 = 0; i0 < pieces; i0 += 32 * U) {
            uint4 q[U + 1];
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = slot(i0 + 32 * u + lane);
            q[U] = slot(i0 + 32 * U);               // (the same for all lanes)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + 32 * u + lane;
                uint32_t w[8] = {q[u].x, q[u].y, q[u].z, q[u].w, 0, 0, 0, 0};
                const uint32_t next[4] = {q[u + 1].x, q[u + 1].y, q[u + 1].z, q[u + 1].w};
                if (off) {                          // the lane behind has the next slot, of the last lane the next set's first
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t first = __shfl_sync(0xffffffffu, next[k], 0), other = __shfl_down_sync(0xffffffffu, w[k], 1);
                        w[k + 4] = lane == 31 ? first : other;
                    }
                }
                const bool by4 = off & 4, by2 = off & 2;
#pragma unroll
                for (int k = 0; k < 6; ++k) w[k] = by4 ? w[k + 2] : w[k];
#pragma unroll
                for (int k = 0; k < 5; ++k) w[k] = by2 ? w[k + 1] : w[k];
                const int left = cols - 8 * i;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[k] = __funnelshift_r(w[k], w[k + 1], (off & 1) * 16);
                    if (left < 8) w[k] = 2 * k + 1 < left ? w[k] : 2 * k < left ? w[k] & 0xFFFFu : 0u;
                }
                if (i < pieces) dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// The experts' last k-blocks of up to three matrices (rows on 16 bytes, pitch ld):
// an expert's tail_block() of dst holds the rows of its last, partial k-block, zeros
// behind them; experts without one are left out (nothing reads theirs).
struct TailArgs {
    const void* src[3];
    void* dst[3];
    int64_t ld[3];              // of both
    int rows, by_row;
    const int* bounds;
};

__global__ void __launch_bounds__(256) tails_kernel(const __grid_constant__ TailArgs a) {
    pdl_wait();
    pdl_trigger();
    const int m = blockIdx.z, e = blockIdx.x;
    int first, last;
    expert_rows(a.bounds, a.rows, e, first, last);
    const int left = (last - first) % GK;
    if (left == 0) return;
    const int pieces = (int)(a.ld[m] / 8);
    const uint4* src = static_cast<const uint4*>(a.src[m]) + (int64_t)(last - left) * pieces;
    uint4* dst = static_cast<uint4*>(a.dst[m]) + (int64_t)tail_block(a.by_row, e, first) * GK * pieces;
    const int n = GK * pieces, live = left * pieces;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < n; i += gridDim.y * 256)
        dst[i] = i < live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int MAX_EXPERTS = 1024;
constexpr int64_t MAX_SIDE = 1 << 20;
constexpr int64_t MAX_ROWS = 1 << 24;

int blocks_of(int64_t k) { return (int)((k + GK - 1) / GK); }

// The launch's bounds on tiles, and its family a (cols, contraction, columns of a
// tile) and b where they are asked for.
int set_tiles(ExpArgs& g, int64_t cols_a, int tile_cols, int64_t k, int segs, int nb, int64_t rows_b, int64_t cols_b,
              int64_t* most) {
    g.cols_a = (int)cols_a;
    g.tiles_w = (int)((cols_a + tile_cols - 1) / tile_cols);
    g.seg_blocks = blocks_of(k);
    g.segs = segs;
    g.nb = nb;
    g.rows_b = (int)rows_b;
    g.cols_b = (int)cols_b;
    g.tiles_mb = (int)((rows_b + 2 * GM - 1) / (2 * GM));
    g.tiles_nb = (int)((cols_b + 2 * GM - 1) / (2 * GM));
    g.group_a.set(GROUP * g.tiles_w);
    g.group_b.set(GROUP * g.tiles_nb);
    g.rest_b.set(g.tiles_mb % GROUP);
    *most = (g.a_on ? ((int64_t)g.rows / ROW_TILE + g.experts + 1) * g.tiles_w : 0) +
            (int64_t)g.experts * nb * g.tiles_mb * g.tiles_nb;
    // (their results alone, 128 KB a tile, are more than the device holds)
    if (*most > 1 << 30) return fail(MUON_ENOMEM, "products of more than 2^30 tiles");
    g.matrix_b.set(g.tiles_mb * g.tiles_nb);
    return MUON_OK;
}

// Whether a contraction of this launch can take more than one part.
bool in_parts(const ExpArgs& g) {
    return (g.a_on && g.segs * g.seg_blocks > MAX_BLOCKS) || (g.nb && blocks_of(g.rows) > MAX_BLOCKS);
}

// Points the operands that need it at padded copies from `at` on and makes these;
// `rows` are all experts', `weights` num_experts matrices each.
int pad_rows(std::initializer_list<Operand*> rows, std::initializer_list<Operand*> weights, const ExpArgs& g, char* at,
             int sms, cudaStream_t s) {
    PadRows p;
    std::memset(&p, 0, sizeof p);
    p.bounds = g.bounds;
    p.all = g.rows;
    int n = 0;
    int64_t most = 0;
    auto pad = [&](Operand* o, bool by_expert) {
        const size_t bytes = padded_bytes(*o);
        if (!bytes) return;
        p.src[n] = o->p; p.dst[n] = at; p.rows[n] = o->rows; p.cols[n] = (int)o->cols;
        if (by_expert) p.each[n].set((int)(o->rows / g.experts));
        most = std::max(most, o->rows);
        o->p = at;
        o->ld = pad8(o->cols);
        at += bytes;
        ++n;
    };
    for (Operand* o : rows) pad(o, false);
    for (Operand* o : weights) pad(o, true);
    if (n == 0) return MUON_OK;
    note_launch_begin(KC_OTHER, s);
    const cudaError_t e = launch_pdl(pad_rows_kernel, dim3((unsigned)std::min<int64_t>((most + 7) / 8, (int64_t)sms * 16), (unsigned)n),
                                     dim3(256), 0, s, p);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "expert operands launch");
}

// A matrix read MN-major: by blocks of 64 columns, where its columns are whole ones
// (128 of them are one copy then: half the instructions of the producer, whose time
// per stage the ring feels), else as it is.
bool map_columns(CUtensorMap* m, const Operand& o, int dtype, int* whole, int64_t batch = 1) {
    *whole = o.cols % 64 == 0;
    if (!*whole) return map_in(m, o, dtype, 64, GK, batch);
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)o.rows, (cuuint64_t)(o.cols / 64), (cuuint64_t)batch};
    cuuint64_t strides[3] = {(cuuint64_t)o.ld * 2, 128, (cuuint64_t)(o.rows * o.ld) * 2};
    cuuint32_t box[4] = {64, GK, 2, 1}, elem[4] = {1, 1, 1, 1};
    return fn(m, dtype == MUON_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(o.p), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Family b's results, in boxes of 64 columns and 32 rows.
bool map_wide(CUtensorMap* m, const GluOut& o, int dtype, int64_t rows, int64_t cols, int64_t batch) {
    return map_in(m, Operand{o.p, rows, cols, o.ld}, dtype, 64, 32, batch);
}

// Rows and bytes of the experts' last k-blocks of a matrix of pitch ld: one block for
// each expert that can have rows.
int64_t tail_rows(const ExpArgs& g) { return (int64_t)std::min(g.experts, g.rows) * GK; }
size_t tail_bytes(const ExpArgs& g, int64_t ld) { return g.nb ? align_up((size_t)tail_rows(g) * ld * 2, 256) : 0; }

// Copies them for the matrices of family b to `at`, one after the other, and maps
// both: which of ops is family b's B operand, the others are its A operands.
int set_family_b(ExpMaps& maps, ExpArgs& g, const Operand* const* ops, int n, char* at, int sms, cudaStream_t s) {
    TailArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = g.rows;
    a.by_row = g.tails_by_row = g.rows < g.experts;
    a.bounds = g.bounds;
    int64_t widest = 1;
    for (int i = 0; i < n; ++i) {
        const Operand& o = *ops[i];
        CUtensorMap* whole = i < n - 1 ? &maps.a2[i] : &maps.b2;
        CUtensorMap* tail = i < n - 1 ? &maps.a2_tail[i] : &maps.b2_tail;
        const Operand t{at, tail_rows(g), o.cols, o.ld};
        int* by_blocks = i < n - 1 ? &g.whole_a2 : &g.whole_b2;         // (the A operands have one shape)
        if (!map_columns(whole, o, g.dtype, by_blocks) || !map_columns(tail, t, g.dtype, by_blocks))
            return fail(MUON_ECUDA, "tensor map creation failed");
        a.src[i] = o.p; a.dst[i] = at; a.ld[i] = o.ld;
        widest = std::max(widest, o.ld);
        at += tail_bytes(g, o.ld);
    }
    // a few pieces per thread, fewer CTAs per expert where experts fill the device
    const int64_t y = std::max<int64_t>(1, std::min<int64_t>((widest * GK / 8 + 511) / 512, (int64_t)sms * 16 / (g.experts * n)));
    note_launch_begin(KC_OTHER, s);
    const cudaError_t e = launch_pdl(tails_kernel, dim3((unsigned)g.experts, (unsigned)y, (unsigned)n), dim3(256), 0, s, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "expert tails launch");
}

// Rows as family a's N side, in the boxes that experts of no more than all rows take.
bool map_rows(CUtensorMap (&m)[BOXES], const Operand& o, int dtype) {
    for (int i = 0; i < BOXES && (i == 0 || 2 * box_rows(i - 1) < o.rows); ++i)
        if (!map_in(&m[i], o, dtype, GK, (uint32_t)box_rows(i))) return false;
    return true;
}

template <int MODE>
cudaError_t clusters_at_once(int device, int* n) {
    static OncePer<int, int> fits;          // by device: pairs resident at once, of either form
    return fits.get(device, n, [&](int& v) {
        v = INT_MAX;
        for (auto kernel : {expert_kernel<MODE, false>, expert_kernel<MODE, true>}) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, EXP_SMEM);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2);
            cfg.blockDim = dim3(GT);
            cfg.dynamicSmemBytes = EXP_SMEM;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 2;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int one = 0;
            e = cudaOccupancyMaxActiveClusters(&one, kernel, &cfg);
            if (e != cudaSuccess || one < 1) return e == cudaSuccess ? cudaErrorInvalidConfiguration : e;
            v = std::min(v, one);
        }
        return cudaSuccess;
    });
}

template <int MODE>
int launch_expert(const ExpMaps& maps, ExpArgs& g, int64_t most, double work, const DevCtx& dc, cudaStream_t s) {
    int n = 0;
    cudaError_t e = clusters_at_once<MODE>(dc.device, &n);
    if (e != cudaSuccess) return cuda_fail(e, "expert products set-up");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(n, most)));
    cfg.blockDim = dim3(GT);
    cfg.dynamicSmemBytes = EXP_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    g.stall = take_stall(STALL_EXPERT);
    note_launch_begin(KC_GLU, s);
    e = cudaLaunchKernelEx(&cfg, g.tma_out ? expert_kernel<MODE, true> : expert_kernel<MODE, false>, maps, g);
    note_launch_end(KC_GLU, work, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "expert products launch");
}

int exp_check(int64_t rows, int64_t experts, int64_t in, int64_t out, int dtype, std::initializer_list<const void*> ps,
              const int* bounds) {
    if (!is_half(dtype)) return fail(MUON_EDTYPE, "dtype %d: MUON_BF16 or MUON_F16", dtype);
    if (rows < 0 || rows > MAX_ROWS) return fail(MUON_EINVAL, "rows outside [0, 2^24]");
    if (experts < 1 || experts > MAX_EXPERTS) return fail(MUON_EINVAL, "experts outside [1, %d]", MAX_EXPERTS);
    if (in < 1 || in > MAX_SIDE || out < 1 || out > MAX_SIDE) return fail(MUON_EINVAL, "a side outside [1, 2^20]");
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 1) return fail(MUON_EINVAL, "pointer not aligned to its element");
    if (reinterpret_cast<uintptr_t>(bounds) & 3) return fail(MUON_EINVAL, "pointer not aligned to its element");
    return MUON_OK;
}

// The call's scratch: enough and on 256 bytes, or what it has to be.
int scratch_check(void* scratch, int64_t* have, size_t need) {
    if (need == 0) return MUON_OK;
    if (!have) return fail(MUON_EINVAL, "NULL argument");
    if (!scratch && *have == 0) {           // asked, no mistake
        *have = (int64_t)need;
        return MUON_ENOMEM;
    }
    if (!scratch || *have < (int64_t)need) {
        *have = (int64_t)need;
        return fail(MUON_ENOMEM, "the call needs %zu bytes of scratch", need);
    }
    if (reinterpret_cast<uintptr_t>(scratch) & 255) return fail(MUON_EINVAL, "scratch must start on 256 bytes");
    return MUON_OK;
}

ExpArgs exp_args(int64_t rows, int64_t experts, const int* bounds, int dtype, int act, int* status) {
    ExpArgs g;
    std::memset(&g, 0, sizeof g);
    g.rows = (int)rows; g.experts = (int)experts; g.bounds = bounds;
    g.dtype = dtype; g.act = act; g.status = status;
    return g;
}

// The weights' gradients of a call without rows.
int zero_weights(void* p, size_t bytes, cudaStream_t s) {
    if (p) MUON_CUDA(cudaMemsetAsync(p, 0, bytes, s));
    return MUON_OK;
}

// Bytes of the running sums, where a contraction takes several parts.
template <int MODE>
int part_bytes(const ExpArgs& g, int64_t most, const DevCtx& dc, size_t* bytes) {
    *bytes = 0;
    if (!in_parts(g)) return MUON_OK;
    int n = 0;
    const cudaError_t e = clusters_at_once<MODE>(dc.device, &n);
    if (e != cudaSuccess) return cuda_fail(e, "expert products set-up");
    *bytes = 2 * (size_t)std::min<int64_t>(n, most) * PART_BYTES;
    return MUON_OK;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" int muon_expert_glu_forward(const void* x, const void* w_gate, const void* w_up, const int* bounds, void* h,
                                       void* gate, void* up, int64_t rows, int64_t num_experts, int64_t hidden,
                                       int64_t ffn, int dtype, int act, void* scratch, int64_t* scratch_bytes,
                                       void* stream) try {
    int r = exp_check(rows, num_experts, hidden, ffn, dtype, {x, w_gate, w_up, h, gate, up}, bounds);
    if (r) return r;
    if (act < ACT_SILU || act > ACT_GELU_TANH) return fail(MUON_EINVAL, "activation %d", act);
    if ((gate == nullptr) != (up == nullptr)) return fail(MUON_EINVAL, "gate and up: both or neither");
    if (rows == 0) return MUON_OK;
    if (!x || !w_gate || !w_up || !bounds || !h) return fail(MUON_EINVAL, "NULL argument");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Operand X{x, rows, hidden, hidden}, G{w_gate, num_experts * ffn, hidden, hidden}, U{w_up, num_experts * ffn, hidden, hidden};
    ExpArgs g = exp_args(rows, num_experts, bounds, dtype, act, dc.status);
    g.a_on = 1;
    g.save = gate != nullptr;
    int64_t most = 0;
    if ((r = set_tiles(g, ffn, GM, hidden, 1, 0, 0, 0, &most))) return r;
    size_t part = 0;
    if ((r = part_bytes<FWD_GLU>(g, most, dc, &part))) return r;
    const size_t pads = padded_bytes(X) + padded_bytes(G) + padded_bytes(U);
    if ((r = scratch_check(scratch, scratch_bytes, part + pads))) return r;
    g.part = static_cast<float*>(scratch);
    if ((r = pad_rows({&X}, {&G, &U}, g, static_cast<char*>(scratch) + part, dc.sms, s))) return r;
    G.rows = U.rows = ffn;
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{h, ffn}; g.out[1] = GluOut{gate, ffn}; g.out[2] = GluOut{up, ffn};
    g.tma_out = tma_ok(h, ffn) && tma_ok(gate, ffn) && tma_ok(up, ffn);
    bool ok = map_in(&maps.a[0], G, dtype, GK, GM / 2, num_experts) && map_in(&maps.a[1], U, dtype, GK, GM / 2, num_experts) &&
              map_rows(maps.b[0], X, dtype);
    for (int i = 0; ok && g.tma_out && i < (g.save ? 3 : 1); ++i) ok = map_out(&maps.out[i], g.out[i], dtype, rows, ffn, 1, i ? 32 : 16);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    return launch_expert<FWD_GLU>(maps, g, most, 4.0 * (double)rows * hidden * ffn, dc, s);
} MUON_CATCH_ALL

extern "C" int muon_expert_glu_backward(const void* x, const void* w_gate, const void* w_up, const void* gate,
                                        const void* up, const void* dh, const int* bounds, void* dx, void* dw_gate,
                                        void* dw_up, int64_t rows, int64_t num_experts, int64_t hidden, int64_t ffn,
                                        int dtype, int act, void* scratch, int64_t* scratch_bytes, void* stream) try {
    int r = exp_check(rows, num_experts, hidden, ffn, dtype, {x, w_gate, w_up, gate, up, dh, dx, dw_gate, dw_up}, bounds);
    if (r) return r;
    if (act < ACT_SILU || act > ACT_GELU_TANH) return fail(MUON_EINVAL, "activation %d", act);
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return fail(MUON_EINVAL, "dw_gate and dw_up: both or neither");
    if (!dx && !dw_gate) return MUON_OK;
    if (rows > 0 && (!x || !w_gate || !w_up || !gate || !up || !dh || !bounds)) return fail(MUON_EINVAL, "NULL argument");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ExpArgs g = exp_args(rows, num_experts, bounds, dtype, act, dc.status);
    g.a_on = dx != nullptr;
    int64_t most = 0;
    if ((r = set_tiles(g, hidden, 2 * GM, ffn, 2, dw_gate ? 2 : 0, ffn, hidden, &most))) return r;
    if (rows == 0) {
        const size_t bytes = (size_t)(num_experts * ffn * hidden) * 2;
        if ((r = zero_weights(dw_gate, bytes, s)) || (r = zero_weights(dw_up, bytes, s))) return r;
        return MUON_OK;
    }
    // (operands of products that are not asked for have no rows to pad)
    Operand X{x, dw_gate ? rows : 0, hidden, hidden}, G{w_gate, dx ? num_experts * ffn : 0, hidden, hidden}, U = G;
    U.p = w_up;
    const int64_t ldw = pad8(ffn);
    const size_t half = align_up((size_t)rows * ldw * 2, 256);
    size_t part = 0;
    if ((r = part_bytes<BACKWARD>(g, most, dc, &part))) return r;
    const size_t pads = padded_bytes(X) + padded_bytes(G) + padded_bytes(U);
    const size_t tails = 2 * tail_bytes(g, ldw) + tail_bytes(g, pad8(hidden));
    if ((r = scratch_check(scratch, scratch_bytes, part + 2 * half + pads + tails))) return r;
    char* at = static_cast<char*>(scratch);
    g.part = reinterpret_cast<float*>(at);
    GluGradArgs ga;
    ga.dh = dh; ga.gate = gate; ga.up = up;
    ga.dg = at + part; ga.du = at + part + half;
    ga.rows = rows; ga.ffn = (int)ffn; ga.pieces = (int)(ldw / 8);
    ga.dtype = dtype; ga.act = act;
    ga.vec = tma_ok(dh, ffn) && tma_ok(gate, ffn) && tma_ok(up, ffn);
    if ((r = pad_rows({&X}, {&G, &U}, g, at + part + 2 * half, dc.sms, s))) return r;
    if ((r = glu_prepare(nullptr, nullptr, &ga, dc.sms, s))) return r;
    G.rows = U.rows = ffn;
    const Operand DG{ga.dg, rows, ffn, ldw}, DU{ga.du, rows, ffn, ldw};
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{dx, hidden}; g.out[1] = GluOut{dw_gate, hidden}; g.out[2] = GluOut{dw_up, hidden};
    g.tma_out = tma_ok(dx, hidden) && tma_ok(dw_gate, hidden) && tma_ok(dw_up, hidden);
    bool ok = true;
    if (dx)
        ok = map_columns(&maps.a[0], G, dtype, &g.whole_a, num_experts) && map_columns(&maps.a[1], U, dtype, &g.whole_a, num_experts) &&
             map_rows(maps.b[0], DG, dtype) && map_rows(maps.b[1], DU, dtype);
    if (ok && g.tma_out && dx) ok = map_out(&maps.out[0], g.out[0], dtype, rows, hidden);
    if (ok && g.tma_out && dw_gate)
        ok = map_wide(&maps.out[1], g.out[1], dtype, ffn, hidden, num_experts) &&
             map_wide(&maps.out[2], g.out[2], dtype, ffn, hidden, num_experts);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    const Operand* const contracted[3] = {&DG, &DU, &X};
    if (dw_gate && (r = set_family_b(maps, g, contracted, 3, at + part + 2 * half + pads, dc.sms, s))) return r;
    return launch_expert<BACKWARD>(maps, g, most, ((dx ? 4.0 : 0.0) + (dw_gate ? 4.0 : 0.0)) * (double)rows * hidden * ffn, dc, s);
} MUON_CATCH_ALL

extern "C" int muon_expert_linear_forward(const void* x, const void* w, const int* bounds, void* y, int64_t rows,
                                          int64_t num_experts, int64_t in, int64_t out, int dtype, void* scratch,
                                          int64_t* scratch_bytes, void* stream) try {
    int r = exp_check(rows, num_experts, in, out, dtype, {x, w, y}, bounds);
    if (r) return r;
    if (rows == 0) return MUON_OK;
    if (!x || !w || !bounds || !y) return fail(MUON_EINVAL, "NULL argument");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Operand X{x, rows, in, in}, W{w, num_experts * out, in, in};
    ExpArgs g = exp_args(rows, num_experts, bounds, dtype, 0, dc.status);
    g.a_on = 1;
    int64_t most = 0;
    if ((r = set_tiles(g, out, 2 * GM, in, 1, 0, 0, 0, &most))) return r;
    size_t part = 0;
    if ((r = part_bytes<FWD_LINEAR>(g, most, dc, &part))) return r;
    const size_t pads = padded_bytes(X) + padded_bytes(W);
    if ((r = scratch_check(scratch, scratch_bytes, part + pads))) return r;
    g.part = static_cast<float*>(scratch);
    if ((r = pad_rows({&X}, {&W}, g, static_cast<char*>(scratch) + part, dc.sms, s))) return r;
    W.rows = out;
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{y, out};
    g.tma_out = tma_ok(y, out);
    bool ok = map_in(&maps.a[0], W, dtype, GK, GM, num_experts) && map_rows(maps.b[0], X, dtype);
    if (ok && g.tma_out) ok = map_out(&maps.out[0], g.out[0], dtype, rows, out);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    return launch_expert<FWD_LINEAR>(maps, g, most, 2.0 * (double)rows * in * out, dc, s);
} MUON_CATCH_ALL

extern "C" int muon_expert_linear_backward(const void* x, const void* w, const void* dy, const int* bounds, void* dx,
                                           void* dw, int64_t rows, int64_t num_experts, int64_t in, int64_t out,
                                           int dtype, void* scratch, int64_t* scratch_bytes, void* stream) try {
    int r = exp_check(rows, num_experts, in, out, dtype, {x, w, dy, dx, dw}, bounds);
    if (r) return r;
    if (!dx && !dw) return MUON_OK;
    if (rows > 0 && (!x || !w || !dy || !bounds)) return fail(MUON_EINVAL, "NULL argument");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ExpArgs g = exp_args(rows, num_experts, bounds, dtype, 0, dc.status);
    g.a_on = dx != nullptr;
    int64_t most = 0;
    if ((r = set_tiles(g, in, 2 * GM, out, 1, dw ? 1 : 0, out, in, &most))) return r;
    if (rows == 0) return zero_weights(dw, (size_t)(num_experts * in * out) * 2, s);
    Operand X{x, dw ? rows : 0, in, in}, W{w, dx ? num_experts * out : 0, in, in}, D{dy, rows, out, out};
    size_t part = 0;
    if ((r = part_bytes<BACKWARD>(g, most, dc, &part))) return r;
    const size_t pads = padded_bytes(X) + padded_bytes(W) + padded_bytes(D);
    const size_t tails = tail_bytes(g, pad8(out)) + tail_bytes(g, pad8(in));
    if ((r = scratch_check(scratch, scratch_bytes, part + pads + tails))) return r;
    g.part = static_cast<float*>(scratch);
    if ((r = pad_rows({&X, &D}, {&W}, g, static_cast<char*>(scratch) + part, dc.sms, s))) return r;
    W.rows = out;
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{dx, in}; g.out[1] = GluOut{dw, in};
    g.tma_out = tma_ok(dx, in) && tma_ok(dw, in);
    bool ok = !dx || (map_columns(&maps.a[0], W, dtype, &g.whole_a, num_experts) && map_rows(maps.b[0], D, dtype));
    if (ok && g.tma_out && dx) ok = map_out(&maps.out[0], g.out[0], dtype, rows, in);
    if (ok && g.tma_out && dw) ok = map_wide(&maps.out[1], g.out[1], dtype, out, in, num_experts);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    const Operand* const contracted[2] = {&D, &X};
    if (dw && (r = set_family_b(maps, g, contracted, 2, static_cast<char*>(scratch) + part + pads, dc.sms, s))) return r;
    return launch_expert<BACKWARD>(maps, g, most, ((dx ? 2.0 : 0.0) + (dw ? 2.0 : 0.0)) * (double)rows * in * out, dc, s);
} MUON_CATCH_ALL
