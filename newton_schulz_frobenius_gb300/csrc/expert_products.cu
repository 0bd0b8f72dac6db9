// Products of a block that is split over experts.  Rows are sorted by expert
// (expert e has the rows [bounds[e], bounds[e + 1]), known on the device alone), and
// every expert has matrices of its own:
//
//   gated block   G = X Wg_e^T, U = X Wu_e^T, H = act(G) U over expert e's rows
//     backward    dG = dH U act'(G), dU = dH act(G)
//                 dX = dG Wg_e + dU Wu_e, dWg_e = dG^T X, dWu_e = dU^T X
//   linear        Y = X W_e^T;  dX = dY W_e, dW_e = dY^T X
//
// One persistent launch of 2-SM tcgen05 pairs covers all experts: M = 256,
// N = 256, fp32 accumulation in TMEM, two accumulators so that a tile's epilogue
// runs under the next tile's products, fed by TMA through a ring of six 32 KB
// stages per CTA.  A tile never spans two experts; where one ends inside a tile
//   - rows of the next expert are multiplied along and not stored (their results
//     are rows of their own, so whatever they hold stays theirs),
//   - in dW, where rows are the contraction, the last k-block's rows of the next
//     expert are zeroed in shared memory before the tensor core reads them.
// Every warp finds its tiles from the bounds, so no host copy of them is needed
// and a captured call follows new ones.
#include "epilogue.cuh"
#include "glu_parts.cuh"

namespace muon {

namespace {

using namespace tc;

constexpr int GM = 128;                     // rows of a CTA's half-tile
constexpr int GK = 64;                      // k-block: 128 bytes
constexpr int NEPI = 8;
constexpr int GT = 64 + 32 * NEPI;
constexpr int STAGES = 6;
constexpr int OP_BYTES = GM * GK * 2;       // one operand tile of a stage (A, or this CTA's half of B)
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int OUT_BYTES = 32 * 32 * 2;      // one output chunk of a warp: 32 x 32, 64-byte swizzled rows
constexpr int NBARS = 2 * STAGES + 6;
constexpr int EXP_SMEM = STAGES * STAGE_BYTES + NEPI * 2 * OUT_BYTES + NBARS * 8 + 16 + 1024;
static_assert(EXP_SMEM <= 232448, "shared memory per CTA");
constexpr int GROUP = 16;                   // row pairs of tiles that share their B tiles in L2
// The accumulators truncate: a sum of n terms of one sign comes out short by
// 6.4e-9 n of its value, so contractions are cut into parts of at most MAX_BLOCKS
// k-blocks (65536 terms), whose fp32 sums are added in round-to-nearest.
constexpr int MAX_BLOCKS = 1024;
constexpr size_t PART_BYTES = (size_t)GM * 256 * 4;     // a CTA's running sums

enum Mode : int { FWD_GLU = 0, FWD_LINEAR = 1, BACKWARD = 2 };

struct ExpArgs {
    int dtype, act;
    int save;                   // gated forward: G and U leave too
    int tma_out;                // outputs leave through tile stores
    int rows, experts;
    const int* bounds;
    // family a: results over the sorted rows (forward, dX)
    int a_on, cols_a, tiles_n;  // columns of the result, column tiles
    int seg_blocks, segs;       // k-blocks of one segment (one A and B map each), segments
    // family b: the weights' gradients
    int nb;                     // results per expert: 0, 1 or 2
    int rows_b, cols_b, tiles_mb, tiles_nb;
    GluOut out[3];              // H, G, U; Y; or dX, dW, dWu
    float* part;                // running sums of contractions in several parts
    int* status;
};

struct ExpMaps {
    CUtensorMap a[2], b[2];     // family a: operands by segment (gated forward: b = Wg, Wu)
    CUtensorMap a2[2], b2;      // family b: dG, dU (dY) read MN-major; X
    CUtensorMap out[3];
};

// [first, last) rows of expert e, within the matrix whatever the bounds hold.
// Expert `experts` has the rows behind the last one's, whose results are zero.
__device__ __forceinline__ void expert_rows(const ExpArgs& g, int e, int& first, int& last) {
    const int lo = e == 0 ? 0 : g.bounds[e];
    first = min(max(lo, 0), g.rows);
    last = e == g.experts ? g.rows : min(max(g.bounds[e + 1], first), g.rows);
}

struct Tile {
    int family, which;          // 0: a, 1: b; output index
    int e;
    int first, last;            // the expert's rows
    int tm, tn;
    int blocks;                 // k-blocks of its contraction (0: the result is zero)
};

// The tiles of one cluster, in order.  Family a's go round-robin, the clusters
// left with one fewer then take `extra` of family b's, and the rest of family b
// goes round-robin starting with those: with a's tiles the longer ones, every
// cluster ends within a tile of the others.
struct Walk {
    int c, P, j;
    int na, nb, mine, light, extra;
    int e, base, first, last, here;         // family a: current expert, id of its first tile, its rows and tiles

    __device__ __forceinline__ void tiles_of(const ExpArgs& g) {
        expert_rows(g, e, first, last);
        here = (last - first + 2 * GM - 1) / (2 * GM) * g.tiles_n;
    }
    // Called by whole warps.
    __device__ __forceinline__ void init(const ExpArgs& g, int cluster, int clusters) {
        c = cluster;
        P = clusters;
        j = 0;
        na = 0;
        const int lane = threadIdx.x & 31;
        if (g.a_on) {
            for (int k = lane; k <= g.experts; k += 32) {
                int lo, hi;
                expert_rows(g, k, lo, hi);
                na += (hi - lo + 2 * GM - 1) / (2 * GM) * g.tiles_n;
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) na += __shfl_xor_sync(0xffffffffu, na, d);
        }
        nb = g.experts * g.nb * g.tiles_mb * g.tiles_nb;
        const int r = na % P;
        mine = na / P + (c < r ? 1 : 0);
        light = r ? P - r : 0;
        // a tile's time in k-blocks; one of few costs what its results take to leave
        const int ca = max(8, g.segs * g.seg_blocks);
        const int cb = max(8, (g.rows / g.experts + GK - 1) / GK);
        extra = light ? min(nb / light, (ca + cb / 2) / cb) : 0;
        e = 0;
        base = 0;
        tiles_of(g);
    }
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
            t.family = 0;
            t.which = 0;
            t.e = e;
            t.first = first;
            t.last = last;
            t.blocks = e == g.experts ? 0 : g.segs * g.seg_blocks;
            place(l, here / g.tiles_n, g.tiles_n, t);
            return true;
        }
        const int k = j - mine;
        ++j;
        int id;
        const int lead = light * extra;
        if (light && c >= P - light) id = k < extra ? (c - (P - light)) + k * light : lead + (c - (P - light)) + (k - extra) * P;
        else id = lead + (light ? light + c : c) + k * P;
        if (id >= nb) return false;
        const int tiles = g.tiles_mb * g.tiles_nb;
        t.family = 1;
        t.e = id / (g.nb * tiles);
        id -= t.e * g.nb * tiles;
        t.which = id / tiles;
        expert_rows(g, t.e, t.first, t.last);
        t.blocks = (t.last - t.first + GK - 1) / GK;
        place(id - t.which * tiles, g.tiles_mb, g.tiles_nb, t);
        return true;
    }
    __device__ __forceinline__ void place(int l, int tiles_m, int tiles_n, Tile& t) {
        const int per = GROUP * tiles_n, grp = l / per, from = grp * GROUP, size = min(GROUP, tiles_m - from);
        l -= grp * per;
        t.tm = from + l % size;
        t.tn = l / size;
    }
};

// One warp's 32 x 32 chunk (rows r0 + lane of `rows`, columns c0 .. of `cols`) of
// matrix z of an output of z_rows rows each.
__device__ __forceinline__ void store_chunk(const ExpArgs& g, const CUtensorMap* map, const GluOut& o, int rows, int cols,
                                            int r0, int c0, int z, int z_rows, const float (&v)[32], uint8_t* stage,
                                            int& groups) {
    const int lane = threadIdx.x & 31;
    // a tile store ends with the matrix: an expert's last rows leave row by row
    const bool tile = g.tma_out && (r0 + 32 <= rows || rows == z_rows);
    if (groups >= 2 || !tile) {             // the store that last used this buffer has read it
        if (lane == 0) {
            if (tile) bulk_wait_read1();
            else bulk_wait_read0();
        }
        __syncwarp();
    }
    uint8_t* buf = stage + (groups & 1) * OUT_BYTES;
    // 64-byte swizzle: 16-byte piece k of row r at k ^ ((r / 2) % 4)
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(buf + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
            pack8_h(v + 8 * k, g.dtype == MUON_F16);
    if (tile) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, smem_u32(buf), c0, r0, z);
            bulk_commit();
        }
        ++groups;
        return;
    }
    __syncwarp();
    const int n = min(32, rows - r0);
    uint16_t* p = static_cast<uint16_t*>(o.p) + ((int64_t)z * z_rows + r0) * o.ld + c0;
    if (g.tma_out) {                        // rows start on 16 bytes: eight of them per step
        const int k = lane & 3;
        for (int i = lane >> 2; i < n; i += 8)
            if (c0 + 8 * k < cols)
                *reinterpret_cast<uint4*>(p + (int64_t)i * o.ld + 8 * k) =
                    *reinterpret_cast<const uint4*>(buf + i * 64 + ((k ^ ((i >> 1) & 3)) << 4));
    } else if (c0 + lane < cols) {          // a row's 32 columns per store
#pragma unroll 8
        for (int i = 0; i < n; ++i)
            p[(int64_t)i * o.ld + lane] = *reinterpret_cast<const uint16_t*>(
                buf + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
    }
    __syncwarp();
}

template <int MODE>
__global__ void __launch_bounds__(GT, 1)
expert_kernel(const __grid_constant__ ExpMaps maps, const __grid_constant__ ExpArgs g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * OP_BYTES;
    uint8_t* sOut = sB + STAGES * OP_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + NEPI * 2 * OUT_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, accf0 = empty0 + 8 * STAGES;
    const uint32_t acce0 = accf0 + 16, drain_bar = acce0 + 16, tail_bar = drain_bar + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, rank == 0 ? 2 : 1);    // own copies (even CTA: and the odd one's relay)
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf0 + 8 * i, 1);
            mbar_init(acce0 + 8 * i, 2 * NEPI);
        }
        mbar_init(drain_bar, 1);
        mbar_init(tail_bar, 1);
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

    Walk w;
    w.init(g, (int)cluster_idx(), (int)cluster_count());
    Tile t;
    if (warp == 0) {
        // ---------------- TMA producer ----------------
        uint32_t flight = 0, phases = 0;            // per stage: a copy was issued, and its phase
        int stage = 0;
        uint32_t phase = 0, tail_phase = 0;
        bool ok = true, tail_flight = false;
        while (ok && w.next(g, t)) {
            const int m0 = t.tm * 2 * GM + rank * GM;
            for (int kb = 0; kb < t.blocks; ++kb) {
                const uint32_t fb = full0 + 8 * stage;
                const uint32_t a = smem_u32(sA + stage * OP_BYTES), b = smem_u32(sB + stage * OP_BYTES);
                // rows of this k-block that are the expert's, where rows are the contraction
                const int left = t.family ? t.last - t.first - kb * GK : GK;
                if (lane == 0) {
                    ok = wait_bounded(empty0 + 8 * stage, phase ^ 1u, abort_flag, g.status);
                    if (ok) {
                        const uint32_t bar = left < GK ? tail_bar : fb;
                        mbar_expect_tx(bar, STAGE_BYTES);
                        if (MODE == FWD_GLU) {
                            tma_load_3d(a, &maps.a[0], bar, kb * GK, t.first + m0, 0);
                            tma_load_3d(b, &maps.b[rank], bar, kb * GK, t.tn * GM, t.e);    // 128 rows of Wg or of Wu
                        } else if (MODE == FWD_LINEAR) {
                            tma_load_3d(a, &maps.a[0], bar, kb * GK, t.first + m0, 0);
                            tma_load_3d(b, &maps.b[0], bar, kb * GK, t.tn * 2 * GM + rank * GM, t.e);
                        } else {
                            const int n0 = t.tn * 2 * GM + rank * GM;
                            if (t.family == 0) {
                                const int seg = kb >= g.seg_blocks ? 1 : 0, k0 = (kb - seg * g.seg_blocks) * GK;
                                tma_load_3d(a, &maps.a[seg], bar, k0, t.first + m0, 0);
                                tma_load_3d(b, &maps.b[seg], bar, n0, k0, t.e);
                                tma_load_3d(b + OP_BYTES / 2, &maps.b[seg], bar, n0 + 64, k0, t.e);
                            } else {
                                const int k0 = t.first + kb * GK;
                                tma_load_3d(a, &maps.a2[t.which], bar, m0, k0, 0);
                                tma_load_3d(a + OP_BYTES / 2, &maps.a2[t.which], bar, m0 + 64, k0, 0);
                                tma_load_3d(b, &maps.b2, bar, n0, k0, 0);
                                tma_load_3d(b + OP_BYTES / 2, &maps.b2, bar, n0 + 64, k0, 0);
                            }
                        }
                        if (left < GK) {
                            tail_flight = true;
                            flight &= ~(1u << stage);
                        } else {
                            flight |= 1u << stage;
                            phases = (phases & ~(1u << stage)) | (phase << stage);
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                if (!ok) break;
                if (left < GK) {
                    // the last rows belong to the next expert: zeroed in both operands (an
                    // infinity there must not meet a zero here), then the stage is full
                    const bool got = wait_bounded(tail_bar, tail_phase, abort_flag, g.status);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    tail_flight = false;
                    tail_phase ^= 1u;
                    const int pieces = (GK - left) * 8;     // 16 bytes each, the rows of a half tile are 128 bytes
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint8_t* half = (h < 2 ? sA : sB) + stage * OP_BYTES + (h & 1) * (OP_BYTES / 2);
                        for (int i = lane; i < pieces; i += 32)
                            *reinterpret_cast<uint4*>(half + left * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fb);
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // this CTA's copies still in flight (after an abort nobody consumes them)
        if (lane == 0) {
            for (int s = 0; s < STAGES; ++s)
                if ((flight >> s) & 1) wait_drain(full0 + 8 * s, (phases >> s) & 1);
            if (tail_flight) wait_drain(tail_bar, tail_phase);
        }
        __syncwarp();
    } else if (warp == 1 && rank == 1) {
        // ---------------- relay: the odd CTA's filled stages to the even CTA ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            while (ok && w.next(g, t)) {
                for (int kb = 0; kb < t.blocks; ++kb) {
                    if (!wait_bounded(full0 + 8 * stage, phase, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    // (a stage whose rows were zeroed here: those writes go along)
                    if (t.family && t.last - t.first - kb * GK < GK) mbar_arrive_remote(full0 + 8 * stage, 0);
                    else mbar_arrive_remote_relaxed(full0 + 8 * stage, 0);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (even CTA) ----------------
        if (lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, aphase = 0;
            bool ok = true;
            constexpr bool FWD = MODE != BACKWARD;
            while (ok && w.next(g, t)) {
                const bool fam_b = !FWD && t.family;
                const uint32_t idesc =
                    idesc_f16kind(2 * GM, 256, !FWD, g.dtype == MUON_F16) | (fam_b ? (1u << 15) : 0u);
                for (int from = 0; ok && from < t.blocks; from += MAX_BLOCKS) {
                    const int upto = min(from + MAX_BLOCKS, t.blocks);
                    if (!wait_bounded(acce0 + 8 * acc, aphase ^ 1u, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(acc * 256);
                    for (int kb = from; kb < upto; ++kb) {
                        if (!wait_bounded(full0 + 8 * stage, phase, abort_flag, g.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a = smem_u32(sA + stage * OP_BYTES), b = smem_u32(sB + stage * OP_BYTES);
#pragma unroll
                        for (int kk = 0; kk < GK / 16; ++kk) {
                            const uint64_t ad = fam_b ? sdesc(a + kk * 2048, GK * 128, 1024) : sdesc(a + kk * 32, 16, 1024);
                            const uint64_t bd = FWD ? sdesc(b + kk * 32, 16, 1024) : sdesc(b + kk * 2048, GK * 128, 1024);
                            tc_mma2_bf16(d, ad, bd, idesc, (kb > from || kk > 0) ? 1u : 0u);
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
        int groups = 0, acc = 0;
        uint32_t aphase = 0;
        bool ok = true;
        while (ok && w.next(g, t)) {
            // rows and columns of the result, and the matrix of its output
            const int rows = t.family ? g.rows_b : t.last, cols = t.family ? g.cols_b : g.cols_a;
            const int z = t.family ? t.e : 0, z_rows = t.family ? g.rows_b : g.rows;
            const int r0 = (t.family ? 0 : t.first) + t.tm * 2 * GM + rank * GM + q * 32;
            const int o = t.family ? 1 + t.which : 0;
            constexpr int W = MODE == FWD_GLU ? 2 : 4;      // chunks of a warp
            const int n0 = t.tn * (MODE == FWD_GLU ? GM : 2 * GM);
            if (t.blocks == 0) {
                // nothing to sum (an expert without rows, rows behind the last expert)
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = 0.f;
                for (int ch = W * half; ch < W * half + W; ++ch) {
                    const int c0 = n0 + ch * 32;
                    if (c0 >= cols || r0 >= rows) break;
                    store_chunk(g, &maps.out[o], g.out[o], rows, cols, r0, c0, z, z_rows, v, stage, groups);
                    if (MODE == FWD_GLU && g.save) {
                        store_chunk(g, &maps.out[1], g.out[1], rows, cols, r0, c0, z, z_rows, v, stage, groups);
                        store_chunk(g, &maps.out[2], g.out[2], rows, cols, r0, c0, z, z_rows, v, stage, groups);
                    }
                }
                continue;
            }
            for (int from = 0; from < t.blocks; from += MAX_BLOCKS) {
                const bool got = wait_bounded(accf0 + 8 * acc, aphase, abort_flag, g.status);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
                const bool more = from + MAX_BLOCKS < t.blocks;
                // this thread's running sums: its row of the CTA's, 256 columns
                float* part = g.part + ((size_t)blockIdx.x * GM + q * 32 + lane) * 256;
                // columns at `at` of the accumulator, with the parts before
                auto sums = [&](int at, float(&v)[32]) {
                    tmem_ld32(lanes + (uint32_t)at, v);
                    if (from) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(part + at + k);
                            v[k] += f.x;
                            v[k + 1] += f.y;
                            v[k + 2] += f.z;
                            v[k + 3] += f.w;
                        }
                    }
                    if (more) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(part + at + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                };
#pragma unroll 1
                for (int ch = W * half; ch < W * half + W; ++ch) {
                    const int c0 = n0 + ch * 32;
                    if (c0 >= cols || r0 >= rows) break;
                    float v[32];
                    if (MODE == FWD_GLU) {
                        float uv[32];
                        sums(ch * 32, v);
                        sums(GM + ch * 32, uv);
                        if (more) continue;
                        if (g.save) {
                            store_chunk(g, &maps.out[1], g.out[1], rows, cols, r0, c0, z, z_rows, v, stage, groups);
                            store_chunk(g, &maps.out[2], g.out[2], rows, cols, r0, c0, z, z_rows, uv, stage, groups);
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = uv[k] * activate<false>(v[k], g.act, nullptr);
                    } else {
                        sums(ch * 32, v);
                        if (more) continue;
                    }
                    store_chunk(g, &maps.out[o], g.out[o], rows, cols, r0, c0, z, z_rows, v, stage, groups);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 1) mbar_arrive_remote(acce0 + 8 * acc, 0);
                    else mbar_arrive(acce0 + 8 * acc);
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
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
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
    g.tiles_n = (int)((cols_a + tile_cols - 1) / tile_cols);
    g.seg_blocks = blocks_of(k);
    g.segs = segs;
    g.nb = nb;
    g.rows_b = (int)rows_b;
    g.cols_b = (int)cols_b;
    g.tiles_mb = (int)((rows_b + 2 * GM - 1) / (2 * GM));
    g.tiles_nb = (int)((cols_b + 2 * GM - 1) / (2 * GM));
    *most = (g.a_on ? ((int64_t)g.rows / (2 * GM) + g.experts + 1) * g.tiles_n : 0) +
            (int64_t)g.experts * nb * g.tiles_mb * g.tiles_nb;
    // (their results alone, 128 KB a tile, are more than the device holds)
    return *most > 1 << 30 ? fail(MUON_ENOMEM, "products of more than 2^30 tiles") : MUON_OK;
}

// Whether a contraction of this launch can take more than one part.
bool in_parts(const ExpArgs& g) {
    return (g.a_on && g.segs * g.seg_blocks > MAX_BLOCKS) || (g.nb && blocks_of(g.rows) > MAX_BLOCKS);
}

template <int MODE>
cudaError_t clusters_at_once(int device, int* n) {
    static OncePer<int, int> fits;          // by device: pairs resident at once
    return fits.get(device, n, [&](int& v) {
        cudaError_t e = cudaFuncSetAttribute(expert_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, EXP_SMEM);
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
        e = cudaOccupancyMaxActiveClusters(&v, expert_kernel<MODE>, &cfg);
        return e == cudaSuccess && v < 1 ? cudaErrorInvalidConfiguration : e;
    });
}

template <int MODE>
int launch_expert(const ExpMaps& maps, const ExpArgs& g, int64_t most, double work, const DevCtx& dc, cudaStream_t s) {
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
    note_launch_begin(KC_GLU, s);
    e = cudaLaunchKernelEx(&cfg, expert_kernel<MODE>, maps, g);
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
    Operand* const ops[3] = {&X, &G, &U};
    if (pads && (r = glu_prepare(ops, 3, static_cast<char*>(scratch) + part, nullptr, dc.sms, s))) return r;
    G.rows = U.rows = ffn;
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{h, ffn}; g.out[1] = GluOut{gate, ffn}; g.out[2] = GluOut{up, ffn};
    g.tma_out = tma_ok(h, ffn) && tma_ok(gate, ffn) && tma_ok(up, ffn);
    bool ok = map_in(&maps.a[0], X, dtype, GK, GM) && map_in(&maps.b[0], G, dtype, GK, GM, num_experts) &&
              map_in(&maps.b[1], U, dtype, GK, GM, num_experts);
    for (int i = 0; ok && g.tma_out && i < (g.save ? 3 : 1); ++i) ok = map_out(&maps.out[i], g.out[i], dtype, rows, ffn);
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
    Operand X{x, rows, hidden, hidden}, G{w_gate, num_experts * ffn, hidden, hidden}, U{w_up, num_experts * ffn, hidden, hidden};
    const int64_t ldw = pad8(ffn);
    const size_t half = align_up((size_t)rows * ldw * 2, 256);
    size_t part = 0;
    if ((r = part_bytes<BACKWARD>(g, most, dc, &part))) return r;
    if ((r = scratch_check(scratch, scratch_bytes, part + 2 * half + padded_bytes(X) + padded_bytes(G) + padded_bytes(U))))
        return r;
    char* at = static_cast<char*>(scratch);
    g.part = reinterpret_cast<float*>(at);
    GluGradArgs ga;
    ga.dh = dh; ga.gate = gate; ga.up = up;
    ga.dg = at + part; ga.du = at + part + half;
    ga.rows = rows; ga.ffn = (int)ffn; ga.pieces = (int)(ldw / 8);
    ga.dtype = dtype; ga.act = act;
    ga.vec = tma_ok(dh, ffn) && tma_ok(gate, ffn) && tma_ok(up, ffn);
    Operand* const ops[3] = {&X, &G, &U};
    if ((r = glu_prepare(ops, 3, at + part + 2 * half, &ga, dc.sms, s))) return r;
    G.rows = U.rows = ffn;
    const Operand DG{ga.dg, rows, ffn, ldw}, DU{ga.du, rows, ffn, ldw};
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{dx, hidden}; g.out[1] = GluOut{dw_gate, hidden}; g.out[2] = GluOut{dw_up, hidden};
    g.tma_out = tma_ok(dx, hidden) && tma_ok(dw_gate, hidden) && tma_ok(dw_up, hidden);
    bool ok = map_in(&maps.a[0], DG, dtype, GK, GM) && map_in(&maps.a[1], DU, dtype, GK, GM) &&
              map_in(&maps.b[0], G, dtype, 64, GK, num_experts) && map_in(&maps.b[1], U, dtype, 64, GK, num_experts) &&
              map_in(&maps.a2[0], DG, dtype, 64, GK) && map_in(&maps.a2[1], DU, dtype, 64, GK) &&
              map_in(&maps.b2, X, dtype, 64, GK);
    if (ok && g.tma_out && dx) ok = map_out(&maps.out[0], g.out[0], dtype, rows, hidden);
    if (ok && g.tma_out && dw_gate)
        ok = map_out(&maps.out[1], g.out[1], dtype, ffn, hidden, num_experts) &&
             map_out(&maps.out[2], g.out[2], dtype, ffn, hidden, num_experts);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
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
    Operand* const ops[2] = {&X, &W};
    if (pads && (r = glu_prepare(ops, 2, static_cast<char*>(scratch) + part, nullptr, dc.sms, s))) return r;
    W.rows = out;
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{y, out};
    g.tma_out = tma_ok(y, out);
    bool ok = map_in(&maps.a[0], X, dtype, GK, GM) && map_in(&maps.b[0], W, dtype, GK, GM, num_experts);
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
    Operand X{x, rows, in, in}, W{w, num_experts * out, in, in}, D{dy, rows, out, out};
    size_t part = 0;
    if ((r = part_bytes<BACKWARD>(g, most, dc, &part))) return r;
    const size_t pads = padded_bytes(X) + padded_bytes(W) + padded_bytes(D);
    if ((r = scratch_check(scratch, scratch_bytes, part + pads))) return r;
    g.part = static_cast<float*>(scratch);
    Operand* const ops[3] = {&X, &W, &D};
    if (pads && (r = glu_prepare(ops, 3, static_cast<char*>(scratch) + part, nullptr, dc.sms, s))) return r;
    W.rows = out;
    ExpMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{dx, in}; g.out[1] = GluOut{dw, in};
    g.tma_out = tma_ok(dx, in) && tma_ok(dw, in);
    bool ok = map_in(&maps.a[0], D, dtype, GK, GM) && map_in(&maps.b[0], W, dtype, 64, GK, num_experts) &&
              map_in(&maps.a2[0], D, dtype, 64, GK) && map_in(&maps.b2, X, dtype, 64, GK);
    if (ok && g.tma_out && dx) ok = map_out(&maps.out[0], g.out[0], dtype, rows, in);
    if (ok && g.tma_out && dw) ok = map_out(&maps.out[1], g.out[1], dtype, out, in, num_experts);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    return launch_expert<BACKWARD>(maps, g, most, ((dx ? 2.0 : 0.0) + (dw ? 2.0 : 0.0)) * (double)rows * in * out, dc, s);
} MUON_CATCH_ALL
