// Gated feed-forward block: both projections, the activation and the product in
// one kernel, and its backward pass.  Weights as a training step keeps them for
// the Muon update: w_gate and w_up are ffn x hidden, row-major.
//
//   forward   G = X Wg^T, U = X Wu^T, H = act(G) U
//   backward  dG = dH U act'(G), dU = dH act(G)
//             dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X
//
// Products run on 2-SM tcgen05 pairs (M = 256, N = 256, fp32 accumulation in
// TMEM, two accumulators so that a tile's epilogue runs under the next tile's
// products), fed by TMA through a ring of six 32 KB stages per CTA.  Bound: the
// tensor pipe under the power cap.  Forward 8192 x 4096 x 14336 bf16 1.50-1.69
// PFLOP/s by box and load (0.88-0.99 of the sustained cuBLAS rate), the backward
// products of 4096 x 2048 x 8192 1.57.
//
// Forward: a pair's tile is 256 tokens x 128 ffn columns of BOTH projections.
// The even CTA loads the 128 rows of Wg and the odd CTA the same rows of Wu as
// the two halves of the N = 256 operand, so G occupies accumulator columns
// 0..127 and U columns 128..255 of the same rows, and the epilogue forms
// act(G) U from registers; G and U leave rounded only if the caller keeps them.
//
// Backward: one elementwise launch writes dG and dU (16-bit: the operands that
// the tensor core takes at this rate; the one rounding beside the results', after
// which the gradients' error against fp64 is 0.0023 in bf16 and 0.00029 in fp16,
// from 0.0017 and 0.00021 by the results' rounding alone), then one persistent launch
// runs all three products: dX as one contraction over 2 ffn (first dG Wg, then
// dU Wu, in one accumulator), dWg and dWu with both operands read MN-major, so
// nothing is transposed in memory.
#include "host.h"
#include "epilogue.cuh"
#include "tc_ptx.cuh"

#include <cfloat>

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
constexpr int NBARS = 2 * STAGES + 5;
constexpr int GLU_SMEM = STAGES * STAGE_BYTES + NEPI * 2 * OUT_BYTES + NBARS * 8 + 16 + 1024;
static_assert(GLU_SMEM <= 232448, "shared memory per CTA");
// Row pairs of tiles that share their B tiles in L2: forward 8192 x 4096 x 14336
// 1144 us, with groups of 4, 8 and 32 1172, 1152 and 1201 (one box, at the fast
// end of 1144-1280).
constexpr int GROUP = 16;

enum Act : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// act(g), and act'(g) where asked for.  Written so that large finite |g| give 0,
// 1 or g, never an infinity times zero.
template <bool GRAD>
__device__ __forceinline__ float activate(float g, int act, float* grad) {
    if (act == ACT_GELU) {
        const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
        if (GRAD) *grad = fmaf(g * expf(-0.5f * g * g), 0.3989422804014327f, cdf);
        return g * cdf;
    }
    if (act == ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = sigmoid(2 u)
        const float k2 = 1.5957691216057308f;
        const float s = 1.0f / (1.0f + __expf(-k2 * g * fmaf(0.044715f * g, g, 1.0f)));
        if (GRAD) {
            const float c = fminf(fmaxf(g, -30.f), 30.f);
            *grad = fmaf(c * s * (1.0f - s), k2 * fmaf(0.134145f * c, c, 1.0f), s);
        }
        return g * s;
    }
    const float s = 1.0f / (1.0f + __expf(-g));
    if (GRAD) *grad = s * fmaf(g, 1.0f - s, 1.0f);
    return g * s;
}

// One output matrix: rows x cols, row-major with pitch ld.
struct GluOut {
    void* p;
    int64_t ld;
};

// One family of tiles: rows x cols outputs over kblocks k-blocks.
struct GluTiles {
    int rows, cols;             // of the output
    int tiles_m, tiles_n;       // pairs of row blocks, column tiles
    int seg_blocks, segs;       // k-blocks of one segment (one A and B map each), segments
    int count;                  // units of one output: tiles, times splits
    int splits;                 // parts the k-blocks are cut into
};

struct GluArgs {
    int dtype;
    int act;
    int save;                   // forward: G and U leave too
    int tma_out;                // outputs leave through tile stores
    GluTiles a, b;              // forward: a; backward: a = dX, b = dWg and dWu
    int nb;                     // tiles of family b (both outputs)
    int extra;                  // tiles of b a cluster with one tile of a less takes first
    GluOut out[3];              // H, G, U or dX, dWg, dWu
    float* part;                // dX in splits > 1 parts: [splits][rows][ldp] partial sums
    float* part_w;              // dWg and dWu likewise: [2][splits][rows][ldp]
    int64_t ldp;
    int* status;
};

struct GluMaps {
    CUtensorMap a[2], b[2];     // family a: operands by segment (forward: b = Wg, Wu)
    CUtensorMap a2[2], b2;      // family b: dG, dU read MN-major; X
    CUtensorMap out[3];
};

struct Tile {
    int family, which;          // 0: a, 1: b; output index
    int tm, tn;
    int split, kb0, kb1;        // its k-blocks
};

// j-th tile of cluster c.  Family a's tiles go round-robin, the clusters left
// with one fewer then take `extra` of family b's, and the rest of family b goes
// round-robin starting with those: with a's tiles the longer ones, every
// cluster ends within one tile of b of the others.
__device__ __forceinline__ bool tile_of(const GluArgs& g, int c, int P, int j, Tile& t) {
    const int r = g.a.count % P, mine = g.a.count / P + (c < r ? 1 : 0);
    int l;
    if (j < mine) {
        l = c + j * P;
        t.family = 0;
        t.which = 0;
    } else {
        j -= mine;
        int id;
        const int light = r ? P - r : 0, first = light * g.extra;
        if (light && c >= r) {
            id = j < g.extra ? (c - r) + j * light : first + (c - r) + (j - g.extra) * P;
        } else {
            id = first + (light ? light + c : c) + j * P;
        }
        if (id >= g.nb) return false;
        t.family = 1;
        t.which = 1 + id / g.b.count;
        l = id % g.b.count;
    }
    const GluTiles& f = t.family ? g.b : g.a;
    const int all = f.tiles_m * f.tiles_n, blocks = f.segs * f.seg_blocks;
    t.split = l / all;
    l -= t.split * all;
    t.kb0 = (int)((int64_t)blocks * t.split / f.splits);
    t.kb1 = (int)((int64_t)blocks * (t.split + 1) / f.splits);
    const int per = GROUP * f.tiles_n, grp = l / per, first = grp * GROUP;
    const int size = min(GROUP, f.tiles_m - first);
    l -= grp * per;
    t.tm = first + l % size;
    t.tn = l / size;
    return true;
}

// One warp's 32 x 32 chunk (rows r0 + lane, columns c0 ..) of an output.
__device__ __forceinline__ void store_chunk(const GluArgs& g, const CUtensorMap* map, const GluOut& o, int rows, int cols,
                                            int r0, int c0, const float (&v)[32], uint8_t* stage, int& groups) {
    const int lane = threadIdx.x & 31;
    if (g.tma_out) {
        if (groups >= 2) {              // the store that last used this buffer has read it
            if (lane == 0) bulk_wait_read1();
            __syncwarp();
        }
        uint8_t* buf = stage + (groups & 1) * OUT_BYTES;
        // 64-byte swizzle: 16-byte piece k of row r at k ^ ((r / 2) % 4)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(buf + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
                pack8_h(v + 8 * k, g.dtype == MUON_F16);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, smem_u32(buf), c0, r0, 0);
            bulk_commit();
        }
        ++groups;
        return;
    }
    // rows that do not start on 16 bytes: through the same buffer, a row's 32 columns per store
    uint8_t* buf = stage;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(buf + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = pack8_h(v + 8 * k, g.dtype == MUON_F16);
    __syncwarp();
    if (c0 + lane < cols) {
        uint16_t* p = static_cast<uint16_t*>(o.p) + (int64_t)r0 * o.ld + c0 + lane;
        const int n = min(32, rows - r0);
#pragma unroll 8
        for (int i = 0; i < n; ++i)
            p[(int64_t)i * o.ld] = *reinterpret_cast<const uint16_t*>(
                buf + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
    }
}

template <bool FWD>
__global__ void __launch_bounds__(GT, 1)
glu_kernel(const __grid_constant__ GluMaps maps, const __grid_constant__ GluArgs g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * OP_BYTES;
    uint8_t* sOut = sB + STAGES * OP_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + NEPI * 2 * OUT_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, accf0 = empty0 + 8 * STAGES;
    const uint32_t acce0 = accf0 + 16, drain_bar = acce0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int c = (int)cluster_idx(), P = (int)cluster_count();

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

    Tile t;
    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            int issued[STAGES];
#pragma unroll
            for (int s = 0; s < STAGES; ++s) issued[s] = -1;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int j = 0; ok && tile_of(g, c, P, j, t); ++j) {
                const GluTiles& f = (!FWD && t.family) ? g.b : g.a;
                const int m0 = t.tm * 2 * GM + rank * GM;
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * stage;
                    const uint32_t a = smem_u32(sA + stage * OP_BYTES), b = smem_u32(sB + stage * OP_BYTES);
                    const int seg = kb >= f.seg_blocks ? 1 : 0;
                    const int k0 = (kb - seg * f.seg_blocks) * GK;
                    mbar_expect_tx(fb, STAGE_BYTES);
                    if (FWD) {
                        tma_load_3d(a, &maps.a[0], fb, k0, m0, 0);
                        tma_load_3d(b, &maps.b[rank], fb, k0, t.tn * GM, 0);    // 128 rows of Wg or of Wu
                    } else {
                        const int n0 = t.tn * 2 * GM + rank * GM;
                        if (t.family == 0) {
                            tma_load_3d(a, &maps.a[seg], fb, k0, m0, 0);
                        } else {
                            tma_load_3d(a, &maps.a2[t.which - 1], fb, m0, k0, 0);
                            tma_load_3d(a + OP_BYTES / 2, &maps.a2[t.which - 1], fb, m0 + 64, k0, 0);
                        }
                        const CUtensorMap* mb = t.family == 0 ? &maps.b[seg] : &maps.b2;
                        tma_load_3d(b, mb, fb, n0, k0, 0);
                        tma_load_3d(b + OP_BYTES / 2, mb, fb, n0 + 64, k0, 0);
                    }
                    issued[stage] = (int)phase;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // this CTA's copies still in flight (after an abort nobody consumes them)
#pragma unroll
            for (int s = 0; s < STAGES; ++s)
                if (issued[s] >= 0) wait_drain(full0 + 8 * s, (uint32_t)issued[s]);
        }
        __syncwarp();
    } else if (warp == 1 && rank == 1) {
        // ---------------- relay: the odd CTA's filled stages to the even CTA ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int j = 0; ok && tile_of(g, c, P, j, t); ++j) {
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!wait_bounded(full0 + 8 * stage, phase, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_remote_relaxed(full0 + 8 * stage, 0);
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
            for (int j = 0; ok && tile_of(g, c, P, j, t); ++j) {
                const bool fam_b = !FWD && t.family;
                const uint32_t idesc =
                    idesc_f16kind(2 * GM, 256, !FWD, g.dtype == MUON_F16) | (fam_b ? (1u << 15) : 0u);
                if (!wait_bounded(acce0 + 8 * acc, aphase ^ 1u, abort_flag, g.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * 256);
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
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
                        tc_mma2_bf16(d, ad, bd, idesc, (kb > t.kb0 || kk > 0) ? 1u : 0u);
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
        for (int j = 0; tile_of(g, c, P, j, t); ++j) {
            const GluTiles& f = (!FWD && t.family) ? g.b : g.a;
            const int r0 = t.tm * 2 * GM + rank * GM + q * 32;
            const bool ok = wait_bounded(accf0 + 8 * acc, aphase, abort_flag, g.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
            if (FWD) {
#pragma unroll 1
                for (int ch = 2 * half; ch < 2 * half + 2; ++ch) {
                    const int c0 = t.tn * GM + ch * 32;
                    if (c0 >= f.cols || r0 >= f.rows) break;
                    float gv[32], uv[32];
                    tmem_ld32(lanes + (uint32_t)(ch * 32), gv);
                    tmem_ld32(lanes + (uint32_t)(GM + ch * 32), uv);
                    if (g.save) {
                        store_chunk(g, &maps.out[1], g.out[1], f.rows, f.cols, r0, c0, gv, stage, groups);
                        store_chunk(g, &maps.out[2], g.out[2], f.rows, f.cols, r0, c0, uv, stage, groups);
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) uv[k] *= activate<false>(gv[k], g.act, nullptr);
                    store_chunk(g, &maps.out[0], g.out[0], f.rows, f.cols, r0, c0, uv, stage, groups);
                }
            } else {
#pragma unroll 1
                for (int ch = 4 * half; ch < 4 * half + 4; ++ch) {
                    const int c0 = t.tn * 2 * GM + ch * 32;
                    if (c0 >= f.cols || r0 >= f.rows) break;
                    float v[32];
                    tmem_ld32(lanes + (uint32_t)(ch * 32), v);
                    if (f.splits > 1) {
                        const int64_t plane = t.family ? (int64_t)(t.which - 1) * f.splits + t.split : t.split;
                        if (r0 + lane < f.rows)     // ldp is a multiple of 32
                            store_row_run<32>(t.family ? g.part_w : g.part, (plane * f.rows + r0 + lane) * g.ldp + c0, v,
                                              MUON_F32);
                        continue;
                    }
                    store_chunk(g, &maps.out[t.which], g.out[t.which], f.rows, f.cols, r0, c0, v, stage, groups);
                }
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
// forward for few tokens: the weights are the rows of the products
// ---------------------------------------------------------------------------
//
// With at most FEW_TOKENS tokens the call is a reading of both weights, so they
// take the M side: a tile is R rows of Wg (accumulator lanes 0 .. R-1) and the
// same R rows of Wu (lanes 64 ..), the tokens are the N columns (16 .. 64), and
// the ring's stages of FEW_SUB k-blocks keep the copies of one CTA per SM
// running.  R divides the ffn rows evenly over the SMs: the smallest number of
// rows per SM over R = 8, 16, ..., 64 (14336 rows on 152 SMs: R = 48, two tiles
// each).  G and U of one ffn row sit in different lanes; U goes through shared
// memory.  Bound: HBM.  One token through 4096 x 14336 (235 MB): 39 us, 6.0 TB/s,
// 0.88 of the copy rate; with one k-block per stage 50 us (a stage costs about
// 340 ns whatever it holds), as 256 x 128 tiles of the other kernel 86 us.  At
// 128 tokens the other kernel is as fast (72 us) or faster (2048 x 8192: 31
// against 36 us; at 64 tokens 31 against 29).
constexpr int FEW_TOKENS = 64;
constexpr int FEW_SUB = 2;           // k-blocks of a stage
constexpr int FEW_STAGES = 6;
constexpr int FEW_EPI = 4;
constexpr int FEW_T = 64 + 32 * FEW_EPI;
constexpr int FEW_BARS = 2 * FEW_STAGES + 5;
constexpr int FEW_FIXED = 64 * 33 * 4 + FEW_BARS * 8 + 16 + 1024;

struct FewArgs {
    int dtype, act, save;
    int tokens, ffn, kblocks;
    int n;                      // tokens rounded up to 16
    int R, tiles, stages;
    GluOut out[3];              // H, G, U
    int* status;
};

__global__ void __launch_bounds__(FEW_T, 1)
glu_few_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
               const __grid_constant__ CUtensorMap mu, const __grid_constant__ FewArgs g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int block_bytes = OP_BYTES + g.n * 128, stage_bytes = FEW_SUB * block_bytes, S = g.stages;
    float(*up)[33] = reinterpret_cast<float(*)[33]>(smem + S * stage_bytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * stage_bytes + 64 * 33 * 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + FEW_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * FEW_STAGES, accf0 = empty0 + 8 * FEW_STAGES;
    const uint32_t acce0 = accf0 + 16, drain_bar = acce0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf0 + 8 * i, 1);
            mbar_init(acce0 + 8 * i, FEW_EPI);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 2 * FEW_TOKENS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(FEW_SUB * (2 * g.R * 128 + g.n * 128));
            uint32_t flight = 0, phases = 0;        // per stage: a copy was issued, and its phase
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < g.tiles && ok; t += gridDim.x) {
                for (int kb = 0; kb < g.kblocks; ++kb) {
                    if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * stage, a = smem_u32(smem + stage * stage_bytes);
                    mbar_expect_tx(fb, bytes);
#pragma unroll
                    for (int i = 0; i < FEW_SUB; ++i) {
                        const uint32_t at = a + i * block_bytes;
                        const int k0 = (kb * FEW_SUB + i) * GK;
                        tma_load_3d(at, &mg, fb, k0, t * g.R, 0);
                        tma_load_3d(at + OP_BYTES / 2, &mu, fb, k0, t * g.R, 0);
                        tma_load_3d(at + OP_BYTES, &mx, fb, k0, 0, 0);
                    }
                    flight |= 1u << stage;
                    phases = (phases & ~(1u << stage)) | (phase << stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < S; ++s)
                if ((flight >> s) & 1) wait_drain(full0 + 8 * s, (phases >> s) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_f16kind(GM, g.n, false, g.dtype == MUON_F16);
            int stage = 0, acc = 0;
            uint32_t phase = 0, aphase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < g.tiles && ok; t += gridDim.x) {
                if (!wait_bounded(acce0 + 8 * acc, aphase ^ 1u, abort_flag, g.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int kb = 0; kb < g.kblocks; ++kb) {
                    if (!wait_bounded(full0 + 8 * stage, phase, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < FEW_SUB; ++i) {
                        const uint32_t a = smem_u32(smem + stage * stage_bytes + i * block_bytes), b = a + OP_BYTES;
#pragma unroll
                        for (int kk = 0; kk < GK / 16; ++kk)
                            tc_mma_bf16(tmem + (uint32_t)(acc * FEW_TOKENS), sdesc(a + kk * 32, 16, 1024),
                                        sdesc(b + kk * 32, 16, 1024), idesc, (kb > 0 || i > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc_commit(empty0 + 8 * stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                tc_commit(accf0 + 8 * acc);
                acc ^= 1;
                if (acc == 0) aphase ^= 1u;
            }
            if (!ok) {
                tc_commit(drain_bar);
                wait_drain(drain_bar, 0);
            }
        }
        __syncwarp();
    } else {
        // warps 2 .. 5: lane quarters 2, 3 (U) and 0, 1 (G)
        const int q = warp & 3, r = (q & 1) * 32 + lane;        // row of the tile
        const bool is_up = q >= 2, f16 = g.dtype == MUON_F16;
        auto bar4 = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        int acc = 0;
        uint32_t aphase = 0;
        for (int t = blockIdx.x; t < g.tiles; t += gridDim.x) {
            // the four warps go on together, whichever of them saw the wait give up
            const bool got = wait_bounded(accf0 + 8 * acc, aphase, abort_flag, g.status);
            int all;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                         : "=r"(all) : "r"((uint32_t)got) : "memory");
            if (!all) break;
            tc_fence_after();
            const int f = t * g.R + r;
            const bool mine = r < g.R && f < g.ffn;
            for (int n0 = 0; n0 < g.tokens; n0 += 32) {
                float v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * FEW_TOKENS + n0), v);
                const int n = min(32, g.tokens - n0);
                if (is_up) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) up[r][k] = v[k];
                }
                bar4();
                if (g.save && mine) {
                    const GluOut& o = g.out[is_up ? 2 : 1];
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k < n) st_elem(o.p, (int64_t)(n0 + k) * o.ld + f, v[k], f16 ? MUON_F16 : MUON_BF16);
                }
                if (!is_up && mine) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k < n)
                            st_elem(g.out[0].p, (int64_t)(n0 + k) * g.out[0].ld + f,
                                    activate<false>(v[k], g.act, nullptr) * up[r][k], f16 ? MUON_F16 : MUON_BF16);
                }
                bar4();                     // U's buffer is free again
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce0 + 8 * acc);
            acc ^= 1;
            if (acc == 0) aphase ^= 1u;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * FEW_TOKENS);
    }
}

// dG = dH U act'(G) and dU = dH act(G), written at a pitch of whole 16-byte
// pieces (zeros beyond ffn), eight columns per thread and step.  Bound by HBM:
// three matrices read, two written.  3280 x 7504 (246 MB): 33 us, 7.4 TB/s with
// the last writes still in L2; with the activation chosen per element and two
// pieces per step it was 45 us, most of the difference instructions to fetch.
// Rows that start anywhere, 3282 x 7507 beside the padding of three operands of
// 287 columns: 59 us, from 65 with eight 2-byte loads per piece; the padding of
// 333 + 2 x 2731 rows of 1001 columns alone 12.4 -> 9.1.
struct GluGradArgs {
    const void* dh;
    const void* gate;
    const void* up;
    void* dg;
    void* du;
    int64_t rows;
    int ffn, pieces;            // columns, 16-byte pieces of a workspace row
    int dtype, act;
    int vec;                    // the inputs' rows start on 16 bytes too
};

// Columns c .. c + 7 of a row of a dense matrix of `n` 16-bit elements whose
// rows start anywhere (zeros from `cols` on), read as the two aligned 16-byte
// vectors that hold them and shifted into place.  Vectors that would reach
// outside the matrix, at its two ends, are left to by_elements().  Loads and
// shifts are apart so that a thread's loads leave together.
struct Shifted {
    const uint16_t* r;
    int off;                    // elements past the first vector's start
    uint4 q0, q1;
    __device__ __forceinline__ bool at(const void* p, int64_t n, int64_t e) {
        const uint16_t* base = static_cast<const uint16_t*>(p);
        r = base + e;
        off = (int)(reinterpret_cast<uintptr_t>(r) & 15) / 2;
        return e >= off && e - off + 16 <= n;
    }
    __device__ __forceinline__ void load() {
        q0 = *reinterpret_cast<const uint4*>(r - off);
        q1 = *(reinterpret_cast<const uint4*>(r - off) + 1);
    }
    __device__ __forceinline__ uint4 get(int left) const {
        uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        const bool by4 = off & 4, by2 = off & 2;
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = by4 ? w[k + 2] : w[k];
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = by2 ? w[k + 1] : w[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = __funnelshift_r(w[k], w[k + 1], (off & 1) * 16);
            w[k] = 2 * k + 1 < left ? w[k] : 2 * k < left ? w[k] & 0xFFFFu : 0u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 by_elements(int left) const {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t l = 2 * k < left ? r[2 * k] : 0u, h = 2 * k + 1 < left ? r[2 * k + 1] : 0u;
            w[k] = l | (h << 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// i / pieces for i < n, in 32 bits where they do (a 64-bit division costs more
// than the piece).
__device__ __forceinline__ int64_t row_of(int64_t i, int64_t n, int pieces) {
    return n <= INT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)pieces) : i / pieces;
}

template <int ACT>
__device__ __forceinline__ void glu_grad_piece(const GluGradArgs& a, int64_t i, const uint4& qd, const uint4& qg,
                                               const uint4& qu) {
    const bool f16 = a.dtype == MUON_F16;
    float d[8], g[8], u[8];
    unpack8_h(qd, d, f16);
    unpack8_h(qg, g, f16);
    unpack8_h(qu, u, f16);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // a gate that its rounding took out of fp16's range: the limits of act and
        // act', as at the largest finite number (NaN stays)
        if (fabsf(g[k]) > FLT_MAX) g[k] = copysignf(FLT_MAX, g[k]);
        float s;
        const float act = activate<true>(g[k], ACT, &s);
        g[k] = d[k] * u[k] * s;
        u[k] = d[k] * act;
    }
    static_cast<uint4*>(a.dg)[i] = pack8_h(g, f16);
    static_cast<uint4*>(a.du)[i] = pack8_h(u, f16);
}

// One copy of the arithmetic per loop: the eight activations are most of the
// kernel's instructions, and a launch of a few microseconds is spent fetching them.
template <int ACT>
__device__ __forceinline__ void glu_grad(const GluGradArgs& a) {
    const int64_t n = a.rows * a.pieces, step = (int64_t)gridDim.x * 256;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    if (a.vec) {                            // aligned rows are one dense run of pieces, loaded a piece ahead
        const uint4 *d = static_cast<const uint4*>(a.dh), *g = static_cast<const uint4*>(a.gate),
                    *u = static_cast<const uint4*>(a.up);
        uint4 qd = __ldcs(d + i), qg = __ldcs(g + i), qu = __ldcs(u + i);
#pragma unroll 1
        while (true) {
            const int64_t at = i;
            const uint4 cd = qd, cg = qg, cu = qu;
            i += step;
            if (i < n) {
                qd = __ldcs(d + i);
                qg = __ldcs(g + i);
                qu = __ldcs(u + i);
            }
            glu_grad_piece<ACT>(a, at, cd, cg, cu);
            if (i >= n) return;
        }
    }
    const int64_t all = a.rows * a.ffn;
#pragma unroll 1
    for (; i < n; i += step) {
        const int64_t row = row_of(i, n, a.pieces);
        const int c = (int)(i - row * a.pieces) * 8, left = a.ffn - c;
        const int64_t e = row * a.ffn + c;
        Shifted d, g, u;
        const bool id = d.at(a.dh, all, e), ig = g.at(a.gate, all, e), iu = u.at(a.up, all, e);
        uint4 qd, qg, qu;
        if (id && ig && iu) {
            d.load();
            g.load();
            u.load();
            qd = d.get(left);
            qg = g.get(left);
            qu = u.get(left);
        } else {
            qd = d.by_elements(left);
            qg = g.by_elements(left);
            qu = u.by_elements(left);
        }
        glu_grad_piece<ACT>(a, i, qd, qg, qu);
    }
}

// Up to three matrices of 16-bit elements to pitches the copy engine can address.
struct PadArgs {
    const void* src[3];
    void* dst[3];
    int64_t rows[3];
    int cols, n;
};
// What a call needs before its products, in one launch: operands blockIdx.y <
// pads.n padded, and (backward) blockIdx.y == pads.n dG and dU.
template <int ACT>
__global__ void __launch_bounds__(256) glu_prepare_kernel(const __grid_constant__ PadArgs a,
                                                          const __grid_constant__ GluGradArgs g) {
    pdl_wait();
    pdl_trigger();
    const int o = blockIdx.y, pieces = (a.cols + 7) / 8;
    if (o == a.n) {
        glu_grad<ACT>(g);
        return;
    }
    const int64_t n = a.rows[o] * pieces, all = a.rows[o] * a.cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = row_of(i, n, pieces);
        const int c = (int)(i - row * pieces) * 8, left = a.cols - c;
        Shifted v;
        const bool in = v.at(a.src[o], all, row * a.cols + c);
        if (in) v.load();
        static_cast<uint4*>(a.dst[o])[i] = in ? v.get(left) : v.by_elements(left);
    }
}

// A result from its partial sums, added in the order of the parts.
struct PartSumArgs {
    const float* part;
    void* out;
    int64_t rows, ldp;
    int cols, splits, dtype;
};
__global__ void __launch_bounds__(256) part_sum_kernel(const __grid_constant__ PartSumArgs a) {
    pdl_wait();
    pdl_trigger();
    const int64_t plane = a.rows * a.ldp;
    for (int64_t row = (int64_t)blockIdx.x; row < a.rows; row += gridDim.x) {
        for (int c = blockIdx.y * 256 + threadIdx.x; c < a.cols; c += gridDim.y * 256) {
            const float* p = a.part + row * a.ldp + c;
            float s = 0.f;
#pragma unroll 4
            for (int k = 0; k < a.splits; ++k) s += p[k * plane];
            st_elem(a.out, row * a.cols + c, s, a.dtype);
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t MAX_SIDE = 1 << 20;
constexpr int64_t MAX_TOKENS = 1 << 24;
constexpr int SPLIT_BLOCKS = 8;     // k-blocks a part of dX keeps at least
constexpr int SUM_COST = 12;        // the sum of dX's parts, in k-blocks' time
// The accumulators truncate: a product of same-signed terms comes out short by
// 6.4e-9 per term (measured: 2.7e-5 at 2^12 terms, 4.2e-4 at 2^16, 6.7e-3 at
// 2^20), which passes fp16's half ulp beyond 2^16.  The backward pass cuts longer
// contractions (tokens, 2 ffn) into parts of at most MAX_BLOCKS k-blocks, whose
// fp32 sums are added in round-to-nearest.
constexpr int MAX_BLOCKS = 1024;

struct Operand {
    const void* p;
    int64_t rows, cols, ld;
};

bool tma_ok(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

// A caller's matrix as the copy engine can read it: itself, or (rows that do not
// start on 16 bytes) a padded copy at `at` in the workspace.
size_t padded_bytes(const Operand& o) {
    return tma_ok(o.p, o.ld) ? 0 : align_up((size_t)o.rows * pad8(o.cols) * 2, 256);
}
// Points the operands that need it at padded copies and makes these, with dG and
// dU where `g` is given, in one launch.
int prepare(Operand* const* ops, char* at, const GluGradArgs* g, int sms, cudaStream_t s) {
    PadArgs p;
    GluGradArgs ga;
    std::memset(&p, 0, sizeof p);
    std::memset(&ga, 0, sizeof ga);
    int64_t blocks = 1;
    for (int i = 0; i < 3; ++i) {
        Operand& o = *ops[i];
        const size_t b = padded_bytes(o);
        if (!b) continue;
        p.src[p.n] = o.p;
        p.dst[p.n] = at;
        p.rows[p.n] = o.rows;
        p.cols = (int)o.cols;               // the three share it
        ++p.n;
        o.ld = pad8(o.cols);
        blocks = std::max(blocks, (o.rows * (pad8(o.cols) / 8) + 255) / 256);
        o.p = at;
        at += b;
    }
    if (g) {
        ga = *g;
        blocks = std::max(blocks, (g->rows * g->pieces + 255) / 256);
    }
    const unsigned parts = (unsigned)p.n + (g ? 1u : 0u);
    if (!parts) return MUON_OK;
    note_launch_begin(g ? KC_GLU : KC_OTHER, s);
    auto kern = ga.act == ACT_GELU        ? glu_prepare_kernel<ACT_GELU>
                : ga.act == ACT_GELU_TANH ? glu_prepare_kernel<ACT_GELU_TANH>
                                          : glu_prepare_kernel<ACT_SILU>;
    cudaError_t e = launch_pdl(kern, dim3((unsigned)std::min<int64_t>(blocks, (int64_t)sms * 8), parts), dim3(256),
                               0, s, p, ga);
    note_launch_end(g ? KC_GLU : KC_OTHER, 0.0, s);
    if (e != cudaSuccess) return cuda_fail(e, "operand preparation launch");
    return MUON_OK;
}

bool map_in(CUtensorMap* m, const Operand& o, int dtype, uint32_t box_cols, uint32_t box_rows) {
    return make_map(m, o.p, dtype, (uint64_t)o.cols, (uint64_t)o.rows, 1, (uint64_t)o.ld, 0, box_cols, box_rows);
}

// 32 x 32 chunks in 64-byte swizzled rows.
bool map_out(CUtensorMap* m, const GluOut& o, int dtype, int64_t rows, int64_t cols) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
    cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.ld * 2 * (cuuint64_t)rows};
    cuuint32_t box[3] = {32, 32, 1}, elem[3] = {1, 1, 1};
    return fn(m, dtype == MUON_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, o.p, dims,
              strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

GluTiles tiles(int64_t rows, int64_t cols, int64_t tile_cols, int64_t k, int segs) {
    GluTiles t;
    t.rows = (int)rows;
    t.cols = (int)cols;
    t.tiles_m = (int)((rows + 2 * GM - 1) / (2 * GM));
    t.tiles_n = (int)((cols + tile_cols - 1) / tile_cols);
    t.seg_blocks = (int)((k + GK - 1) / GK);
    t.segs = segs;
    t.count = t.tiles_m * t.tiles_n;
    t.splits = 1;
    return t;
}

// A tile's time in k-blocks: one of few costs what its 256 x 256 results take to
// leave, about 8 k-blocks' time.
int tile_cost(const GluTiles& t, int splits) { return std::max(8, t.segs * t.seg_blocks / splits); }

// Tiles of family b that the clusters with one fewer of family a take first.
int extra_of(int na, int nb, int P, int ca, int cb) {
    const int r = na % P;
    return r ? std::min(nb / (P - r), (ca + cb / 2) / cb) : 0;
}

// Parts that keep an accumulator's rounding below the results'.
int least_splits(const GluTiles& t) { return (t.segs * t.seg_blocks + MAX_BLOCKS - 1) / MAX_BLOCKS; }

// Parts of dX's contraction.  dX has few tiles and a long contraction (2 ffn)
// when the tokens are few: the number of parts, of SPLIT_BLOCKS k-blocks at
// least, with which the last cluster of tile_of()'s schedule ends first, the
// partial sums' own launch counted as SUM_COST (333 tokens, 1001 x 2731:
// 8 parts instead of the 9 that fit, products 27.2 -> 23.1 us; one token, 1235 x
// 4575: 31.0 -> 26.0).
int dx_splits(const GluTiles& a, const GluTiles& b, int nb, int P) {
    const int blocks = a.segs * a.seg_blocks, from = least_splits(a);
    const int most = std::max(from, std::min(P / a.count, blocks / SPLIT_BLOCKS));
    const int cb = tile_cost(b, b.splits);
    int best = from;
    int64_t least = INT64_MAX;
    for (int s = from; s <= most; ++s) {
        const int na = a.count * s, ca = tile_cost(a, s), r = na % P, light = r ? P - r : 0;
        const int extra = extra_of(na, nb, P, ca, cb), rest = nb - light * extra;
        const int64_t full = (na + P - 1) / P;      // tiles of a where no cluster has one fewer, or of those that have more
        const int64_t heavy = full * ca + (int64_t)((rest - light + P - 1) / P) * cb;
        const int64_t few = light ? (full - 1) * ca + (int64_t)(extra + (rest + P - 1) / P) * cb : 0;
        const int64_t end = std::max(heavy, few) + (s > 1 ? SUM_COST : 0);
        if (end < least) {
            least = end;
            best = s;
        }
    }
    return best;
}

template <bool FWD>
cudaError_t launch_glu(GluMaps& maps, GluArgs& g, int device, cudaStream_t s) {
    auto kern = glu_kernel<FWD>;
    static OncePer<int, int> fits;          // by device: pairs resident at once
    int most = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(GT);
    cfg.dynamicSmemBytes = GLU_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t err = fits.get(device, &most, [&](int& n) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GLU_SMEM);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2);
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        return e == cudaSuccess && n < 1 ? cudaErrorInvalidConfiguration : e;
    });
    if (err != cudaSuccess) return err;
    const int P = (int)std::min<int64_t>(most, (int64_t)g.a.count + g.nb);
    g.extra = extra_of(g.a.count, g.nb, P, tile_cost(g.a, g.a.splits), tile_cost(g.b, g.b.splits));
    cfg.gridDim = dim3((unsigned)(2 * P));
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, g);
}

int launch_few(const Operand& X, const Operand& W, const Operand& U, FewArgs& g, const DevCtx& dc, cudaStream_t s) {
    static OncePer<int, int> attr;          // by device
    const int sms = dc.sms;
    int set = 0;
    const cudaError_t err = attr.get(dc.device, &set, [](int&) {
        return cudaFuncSetAttribute(glu_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    });
    if (err != cudaSuccess) return cuda_fail(err, "cudaFuncSetAttribute");
    g.n = (g.tokens + 15) / 16 * 16;
    int64_t best = INT64_MAX;
    for (int R = 64; R >= 8; R -= 8) {
        const int64_t n = ((int64_t)g.ffn + R - 1) / R, rows = (n + sms - 1) / sms * R;
        if (rows < best) {
            best = rows;
            g.R = R;
            g.tiles = (int)n;
        }
    }
    const int stage_bytes = FEW_SUB * (OP_BYTES + g.n * 128);
    g.stages = std::min(FEW_STAGES, (232448 - FEW_FIXED) / stage_bytes);
    CUtensorMap mx, mg, mu;
    if (!map_in(&mx, X, g.dtype, GK, (uint32_t)g.n) || !map_in(&mg, W, g.dtype, GK, (uint32_t)g.R) ||
        !map_in(&mu, U, g.dtype, GK, (uint32_t)g.R))
        return fail(MUON_ECUDA, "tensor map creation failed");
    note_launch_begin(KC_GLU, s);
    cudaError_t e = launch_pdl(glu_few_kernel, dim3((unsigned)std::min(g.tiles, sms)), dim3(FEW_T),
                               (size_t)(g.stages * stage_bytes + FEW_FIXED), s, mx, mg, mu, g);
    note_launch_end(KC_GLU, 4.0 * g.tokens * (double)X.cols * g.ffn, s);
    if (e != cudaSuccess) return cuda_fail(e, "glu forward launch");
    return MUON_OK;
}

int glu_check(int64_t tokens, int64_t hidden, int64_t ffn, int dtype, int act) {
    if (!is_half(dtype)) return fail(MUON_EDTYPE, "dtype %d: MUON_BF16 or MUON_F16", dtype);
    if (act < ACT_SILU || act > ACT_GELU_TANH) return fail(MUON_EINVAL, "activation %d", act);
    if (tokens < 0 || tokens > MAX_TOKENS) return fail(MUON_EINVAL, "tokens outside [0, 2^24]");
    if (hidden < 1 || hidden > MAX_SIDE || ffn < 1 || ffn > MAX_SIDE)
        return fail(MUON_EINVAL, "hidden and ffn outside [1, 2^20]");
    return MUON_OK;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" int muon_glu_forward(const void* x, const void* w_gate, const void* w_up, void* h, void* gate, void* up,
                                int64_t tokens, int64_t hidden, int64_t ffn, int dtype, int act, void* stream) try {
    int r = glu_check(tokens, hidden, ffn, dtype, act);
    if (r) return r;
    if ((gate == nullptr) != (up == nullptr)) return fail(MUON_EINVAL, "gate and up: both or neither");
    if (tokens == 0) return MUON_OK;
    if (!x || !w_gate || !w_up || !h) return fail(MUON_EINVAL, "NULL argument");
    for (const void* p : {x, w_gate, w_up, (const void*)h, (const void*)gate, (const void*)up})
        if (reinterpret_cast<uintptr_t>(p) & 1) return fail(MUON_EINVAL, "pointer not aligned to its element");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Operand X{x, tokens, hidden, hidden}, G{w_gate, ffn, hidden, hidden}, U{w_up, ffn, hidden, hidden};
    if (const size_t need = padded_bytes(X) + padded_bytes(G) + padded_bytes(U)) {
        Workspace* w = nullptr;
        if ((r = ws_get(dc.device, s, need, &w))) return r;
        Operand* const ops[3] = {&X, &G, &U};
        if ((r = prepare(ops, w->base, nullptr, dc.sms, s))) return r;
    }
    if (tokens <= FEW_TOKENS) {
        FewArgs f;
        std::memset(&f, 0, sizeof f);
        f.dtype = dtype; f.act = act; f.save = gate != nullptr;
        f.tokens = (int)tokens; f.ffn = (int)ffn; f.kblocks = (int)((hidden + FEW_SUB * GK - 1) / (FEW_SUB * GK));
        f.out[0] = GluOut{h, ffn}; f.out[1] = GluOut{gate, ffn}; f.out[2] = GluOut{up, ffn};
        f.status = dc.status;
        return launch_few(X, G, U, f, dc, s);
    }
    GluArgs g;
    GluMaps maps;
    std::memset(&g, 0, sizeof g);
    std::memset(&maps, 0, sizeof maps);
    g.dtype = dtype; g.act = act; g.save = gate != nullptr;
    g.a = tiles(tokens, ffn, GM, hidden, 1);
    g.b = g.a;
    g.status = dc.status;
    g.out[0] = GluOut{h, ffn}; g.out[1] = GluOut{gate, ffn}; g.out[2] = GluOut{up, ffn};
    g.tma_out = tma_ok(h, ffn) && tma_ok(gate, ffn) && tma_ok(up, ffn);
    bool ok = map_in(&maps.a[0], X, dtype, GK, GM) && map_in(&maps.b[0], G, dtype, GK, GM) &&
              map_in(&maps.b[1], U, dtype, GK, GM);
    for (int i = 0; ok && g.tma_out && i < (g.save ? 3 : 1); ++i) ok = map_out(&maps.out[i], g.out[i], dtype, tokens, ffn);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    note_launch_begin(KC_GLU, s);
    cudaError_t e = launch_glu<true>(maps, g, dc.device, s);
    note_launch_end(KC_GLU, 4.0 * (double)tokens * hidden * ffn, s);
    if (e != cudaSuccess) return cuda_fail(e, "glu forward launch");
    return MUON_OK;
} MUON_CATCH_ALL

extern "C" int muon_glu_backward(const void* x, const void* w_gate, const void* w_up, const void* gate, const void* up,
                                 const void* dh, void* dx, void* dw_gate, void* dw_up, int64_t tokens, int64_t hidden,
                                 int64_t ffn, int dtype, int act, void* stream) try {
    int r = glu_check(tokens, hidden, ffn, dtype, act);
    if (r) return r;
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return fail(MUON_EINVAL, "dw_gate and dw_up: both or neither");
    if (!dx && !dw_gate) return MUON_OK;
    if (tokens > 0 && (!x || !w_gate || !w_up || !gate || !up || !dh)) return fail(MUON_EINVAL, "NULL argument");
    for (const void* p : {x, w_gate, w_up, gate, up, dh, (const void*)dx, (const void*)dw_gate, (const void*)dw_up})
        if (reinterpret_cast<uintptr_t>(p) & 1) return fail(MUON_EINVAL, "pointer not aligned to its element");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0) {                      // no token: the weights' gradients are zero
        if (dw_gate) {
            MUON_CUDA(cudaMemsetAsync(dw_gate, 0, (size_t)(ffn * hidden) * 2, s));
            MUON_CUDA(cudaMemsetAsync(dw_up, 0, (size_t)(ffn * hidden) * 2, s));
        }
        return MUON_OK;
    }
    Operand X{x, tokens, hidden, hidden}, G{w_gate, ffn, hidden, hidden}, U{w_up, ffn, hidden, hidden};
    const int64_t ldw = pad8(ffn);
    const size_t half = align_up((size_t)tokens * ldw * 2, 256);
    GluArgs g;
    std::memset(&g, 0, sizeof g);
    g.dtype = dtype; g.act = act;
    g.status = dc.status;
    g.a = tiles(tokens, hidden, 2 * GM, ffn, 2);
    g.b = tiles(ffn, hidden, 2 * GM, tokens, 1);
    g.b.splits = least_splits(g.b);
    // (their results alone, 128 KB a tile, are more than the device holds)
    if ((int64_t)g.a.count * least_splits(g.a) + (int64_t)2 * g.b.count * g.b.splits > 1 << 30)
        return fail(MUON_ENOMEM, "products of more than 2^30 tiles");
    g.b.count *= g.b.splits;
    g.nb = dw_gate ? 2 * g.b.count : 0;
    g.a.splits = dx_splits(g.a, g.b, g.nb, dc.sms / 2);
    g.a.count *= g.a.splits;
    if (!dx) g.a.count = 0;
    g.ldp = (hidden + 31) / 32 * 32;
    const size_t part = dx && g.a.splits > 1 ? align_up((size_t)g.a.splits * tokens * g.ldp * 4, 256) : 0;
    const size_t plane_w = (size_t)g.b.splits * ffn * g.ldp;
    const size_t part_w = dw_gate && g.b.splits > 1 ? align_up(2 * plane_w * 4, 256) : 0, parts = part + part_w;
    Workspace* w = nullptr;
    if ((r = ws_get(dc.device, s, 2 * half + parts + padded_bytes(X) + padded_bytes(G) + padded_bytes(U), &w))) return r;
    g.part = reinterpret_cast<float*>(w->base + 2 * half);
    g.part_w = reinterpret_cast<float*>(w->base + 2 * half + part);
    GluGradArgs ga;
    ga.dh = dh; ga.gate = gate; ga.up = up;
    ga.dg = w->base; ga.du = w->base + half;
    ga.rows = tokens; ga.ffn = (int)ffn; ga.pieces = (int)(ldw / 8);
    ga.dtype = dtype; ga.act = act;
    ga.vec = tma_ok(dh, ffn) && tma_ok(gate, ffn) && tma_ok(up, ffn);
    Operand* const ops[3] = {&X, &G, &U};
    if ((r = prepare(ops, w->base + 2 * half + parts, &ga, dc.sms, s))) return r;
    const Operand DG{ga.dg, tokens, ffn, ldw}, DU{ga.du, tokens, ffn, ldw};
    GluMaps maps;
    std::memset(&maps, 0, sizeof maps);
    g.out[0] = GluOut{dx, hidden}; g.out[1] = GluOut{dw_gate, hidden}; g.out[2] = GluOut{dw_up, hidden};
    g.tma_out = tma_ok(dx, hidden) && tma_ok(dw_gate, hidden) && tma_ok(dw_up, hidden);
    bool ok = map_in(&maps.a[0], DG, dtype, GK, GM) && map_in(&maps.a[1], DU, dtype, GK, GM) &&
              map_in(&maps.b[0], G, dtype, 64, GK) && map_in(&maps.b[1], U, dtype, 64, GK) &&
              map_in(&maps.a2[0], DG, dtype, 64, GK) && map_in(&maps.a2[1], DU, dtype, 64, GK) &&
              map_in(&maps.b2, X, dtype, 64, GK);
    if (ok && g.tma_out && dx) ok = map_out(&maps.out[0], g.out[0], dtype, tokens, hidden);
    if (ok && g.tma_out && dw_gate)
        ok = map_out(&maps.out[1], g.out[1], dtype, ffn, hidden) && map_out(&maps.out[2], g.out[2], dtype, ffn, hidden);
    if (!ok) return fail(MUON_ECUDA, "tensor map creation failed");
    note_launch_begin(KC_GLU, s);
    cudaError_t e = launch_glu<false>(maps, g, dc.device, s);
    note_launch_end(KC_GLU, (dx ? 4.0 : 0.0) * tokens * (double)hidden * ffn + (dw_gate ? 4.0 : 0.0) * tokens * (double)hidden * ffn, s);
    if (e != cudaSuccess) return cuda_fail(e, "glu backward launch");
    const PartSumArgs sums[3] = {{g.part, dx, tokens, g.ldp, (int)hidden, g.a.splits, dtype},
                                 {g.part_w, dw_gate, ffn, g.ldp, (int)hidden, g.b.splits, dtype},
                                 {g.part_w + plane_w, dw_up, ffn, g.ldp, (int)hidden, g.b.splits, dtype}};
    for (int i = 0; i < 3; ++i) {
        if (!(i ? part_w : part)) continue;
        note_launch_begin(KC_GLU, s);
        e = launch_pdl(part_sum_kernel,
                       dim3((unsigned)std::min<int64_t>(sums[i].rows, 65535),
                            (unsigned)std::min<int64_t>((hidden + 255) / 256, 64)),
                       dim3(256), 0, s, sums[i]);
        note_launch_end(KC_GLU, 0.0, s);
        if (e != cudaSuccess) return cuda_fail(e, "glu partial sum launch");
    }
    return MUON_OK;
} MUON_CATCH_ALL
