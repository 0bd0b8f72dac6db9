// Losses over the vocabulary with their gradients, the start of a training
// step's backward pass: distillation from a teacher's top logits, the clipped
// policy loss with a KL term, and the preference loss of paired sequences.
//
// One row x of V logits, z = x / T, q = softmax(z).  Every loss here has a row
// gradient of the form  dz_v = alpha q_v - t_v  with a sparse t (the sampled
// token, or the teacher's k entries), so a row needs its maximum and its sum
// of exponentials, a handful of gathered logits, and one pass that writes
// alpha q_v - t_v.  Arithmetic is fp32 whatever the logits' type; the gradient
// is rounded once, on its store.
//
//   distillation  KL = sum_j p_j (log p_j - log q_j) over the teacher's set S,
//                 plus p_r (log p_r - log q_r) for everything else as one class
//                 when the teacher's own log-sum-exp is given.
//                 dKL/dz_v = P q_v - p_v in S,  (P - p_r / q_r) q_v outside,
//                 P = sum p (+ p_r).  loss = w T^2 KL, dx = w T dKL/dz.
//                 q_r is summed over the entries outside S, not as 1 - q(S),
//                 which cancels once the student is sure.
//   policy        l = z_a - lse, r = exp(l - old),
//                 L = -min(r A, clip(r) A) + b (exp(ref - l) - (ref - l) - 1),
//                 dL/dl = -r A where not clipped, + b (1 - exp(ref - l)).
//   preference    a row's factor needs the log-probabilities of its whole pair:
//                 one launch takes every row's statistics, one sums the
//                 sequences and writes each row's factor, one writes gradients.
//
// The exponent is taken of (x - max x) / T, never of x / T - max / T: rows whose
// logits are all the type's lowest value stay finite for T < 1.
#include "host.h"
#include "epilogue.cuh"
#include "tc_ptx.cuh"

namespace muon {

namespace {

enum LossMode : int { LM_POLICY = 0, LM_DISTILL = 1, LM_STATS = 2 };

struct RowStats {       // one row of the preference loss between its launches
    float mx, inv_s;    // q_v = exp2((x_v - mx) c2) * inv_s
    float logp;
    float coef;         // d loss / d logp, 0 for rows outside the loss
};

// One entry of a teacher's list as the row kernel needs it.
struct alignas(16) Listed {
    int id;                     // -1: padding
    float p;                    // the teacher's probability
    float psum;                 // p of every entry with this index at its first one, -1 at the others
    int pad;
};

struct RowLossArgs {
    const void* logits;
    void* grad;                 // may be the logits themselves
    int64_t ld, ldg;            // row pitches in elements
    int64_t rows;
    int vocab;
    int same_align;             // grad rows sit on the same 16-byte phase as the logits' rows
    float c2;                   // log2(e) / T
    float inv_t, t;
    const float* weights;       // per row, or null (1)
    float* loss;
    // tokens (policy, statistics)
    const void* tokens;
    int tok64;
    // policy
    const float* old_logp;
    const float* ref_logp;
    const float* adv;
    float lo, hi, kl;           // clip range of the ratio, KL coefficient
    float* logp;
    // distillation
    const void* tidx;
    const void* tval;
    const float* tlse;
    int k, tidx64, tval_dtype;
    Listed* listed;             // [rows][k], written by teacher_kernel
    float2* teacher;            // [rows]: the listed probability, sum p log p
    // preference
    RowStats* stats;
};

__device__ __forceinline__ int64_t ld_index(const void* p, int64_t i, int is64) {
    return is64 ? reinterpret_cast<const int64_t*>(p)[i] : (int64_t) reinterpret_cast<const int32_t*>(p)[i];
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int E = 4;
    static constexpr uint32_t NONE = 0xFF800000u;       // a word of -inf
    static __device__ __forceinline__ float ld(const float* p) { return *p; }
    static __device__ __forceinline__ void st(float* p, float v) { *p = v; }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&v)[4]) {
        v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
        v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ float vmax(const uint4& q) {
        return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    static constexpr uint32_t NONE = 0xFF80FF80u;
    static __device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&v)[8]) { unpack8_h(q, v, false); }
    static __device__ __forceinline__ float vmax(const uint4& q) {
        auto h = [](const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) { return pack8_h(v, false); }
};
template <>
struct Vec<__half> {
    static constexpr int E = 8;
    static constexpr uint32_t NONE = 0xFC00FC00u;
    static __device__ __forceinline__ float ld(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ void st(__half* p, float v) { *p = __float2half_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&v)[8]) { unpack8_h(q, v, true); }
    static __device__ __forceinline__ float vmax(const uint4& q) {
        auto h = [](const uint32_t& w) { return *reinterpret_cast<const __half2*>(&w); };
        const __half2 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) { return pack8_h(v, true); }
};

// What the policy loss needs of one row besides its logits.
struct PolicyRow {
    float w, adv, old, ref;
};

// The policy loss of one row from its log-probability: loss and dL/dlogp.
__device__ __forceinline__ void policy_row(const RowLossArgs& a, const PolicyRow& p, float lp, float& loss, float& dl) {
    const float r = a.old_logp ? expf(lp - p.old) : 1.0f;
    const float rc = fminf(fmaxf(r, a.lo), a.hi);
    // an advantage of 0 takes the term out, also where the ratio has left fp32's range
    const float u = p.adv == 0.f && r == r ? 0.f : r * p.adv, uc = rc * p.adv;
    loss = -fminf(u, uc);
    dl = u <= uc ? -u : 0.f;
    if (a.kl != 0.f) {
        const float x = p.ref - lp;
        // exp(x) - x - 1 cancels for small x: expm1 keeps it
        const float em = expm1f(x);
        loss += a.kl * (em - x);
        dl -= a.kl * em;
    }
    // min and max drop a NaN: a row without a distribution, or a NaN among its
    // values, has no loss either
    if (lp != lp || u != u) loss = dl = lp + u;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Pairs of fp32 values in one 64-bit register, two per instruction.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// v <- exp2((v + nr) c2)
template <int E>
__device__ __forceinline__ void exp_vec(uint64_t (&v)[E / 2], uint64_t nr, uint64_t c2) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const float2 z = unpair(mul2(add2(v[j], nr), c2));
        v[j] = pair2(ex2(z.x), ex2(z.y));
    }
}
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& q, uint64_t (&v)[Vec<T>::E / 2]) {
    float f[Vec<T>::E];
    Vec<T>::unpack(q, f);
#pragma unroll
    for (int j = 0; j < Vec<T>::E / 2; ++j) v[j] = pair2(f[2 * j], f[2 * j + 1]);
}
template <int E>
__device__ __forceinline__ void split_pairs(const uint64_t (&v)[E / 2], float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const float2 z = unpair(v[j]);
        f[2 * j] = z.x;
        f[2 * j + 1] = z.y;
    }
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes into shared memory if `on` (predicated: no branch in the walks)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
                 "l"(src), "r"((int)on)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most n (0 .. 3) of the thread's copy groups are pending.
__device__ __forceinline__ void cp_async_wait(int n) {
    if (n == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// 16 bytes to the same shared-memory offset of CTA `rank`, counted on its mbarrier.
__device__ __forceinline__ void st_async_f4(uint32_t local, uint32_t bar, uint32_t rank, const float4& v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(bar), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
                 : "memory");
}

// ---------------------------------------------------------------------------
// one reading: the row rests in shared memory between its two walks
// ---------------------------------------------------------------------------
//
// A row belongs to a cluster of C CTAs (C = 1 up to 26624 16-bit logits), CTA r
// holding its r-th part in shared memory, SLOTS x NT vectors of 16 bytes as a
// rule, four CTAs per SM.  The first walk takes the maximum and the sums; warp 0
// brings them together, exchanges them with the other CTAs of the cluster
// (distributed shared memory, an mbarrier per row parity), forms the loss and
// hands the gradient's factors to the other warps; the second walk takes the
// exponentials again (cheaper than the registers to keep them in) and stores
// the gradient, so every logit is read from memory once.  What is per row is
// done by one warp: at ten vectors per thread and row, a per-row step of every
// warp costs as many instructions as a vector or two of each thread.  For the
// same reason the walks have no branch per vector (slots beyond the part read
// as -inf, copies and stores are predicated): 65536 bf16 logits 502 -> 466 us
// for 9155 rows.
//
// Bound: the policy loss by HBM for fp32 (131072 logits: 5.9 TB/s of logits and
// gradients, 0.87 of the copy rate), for 16-bit types by the walks' instructions
// and the waits between them (5.2 TB/s, 0.77: twice the logits per byte; issue
// slots 61 % busy, DRAM 63 %, the largest stall the barriers).  The statistics
// alone read at 4.3-5.5 TB/s.
// Other forms measured for 65536 bf16 logits, 1.2 GB: one CTA per row with the
// second walk reading L2 again 498 us (and 603 at 131072, where the rows in
// flight no longer fit L2), the exponentials kept in registers over a cluster
// 819, a ring of eight vectors per thread 590.
//
// Thread t owns the vectors t, t + NT, ... of the part: it copies them in
// (cp.async), reads them twice, and as soon as the second walk has taken a slot
// it starts the copy of the next row's vector into it: no barrier guards the
// slots, and up to a whole part per CTA is in flight.  Copies complete by
// quarters of the part.
//
// The vectors are those aligned in memory; what a row has before the first and
// after the last of them (odd vocabularies, sliced heads: at most 2 (E - 1)
// logits) is taken one logit per thread by the first CTA.
//
// A thread's exponents are taken against a reference that follows the maximum
// only when a logit exceeds it by more than 40 powers of two, so the sums stay
// far from overflow and the rescaling branch is rare; the row's maximum becomes
// the reference when the threads' sums are brought together.
constexpr int SLOTS = 13;
constexpr int MAX_CLUSTER = 16;
constexpr float REBASE = 40.0f;     // exponent (base 2) beyond which the reference moves

struct Sums {
    float ref, limit;       // reference (negated), and the logit from which it moves
    float s, si;            // sums of exponentials: outside the teacher's set (or all), inside
    float top;              // the maximum
};

// Takes a new maximum; returns whether the reference moved.
__device__ __forceinline__ bool follow(Sums& z, float vm, float c2, float step) {
    z.top = fmaxf(z.top, vm);
    if (!(vm > z.limit)) return false;
    const float f = z.limit == -INFINITY ? 1.0f : ex2((-z.ref - vm) * c2);
    z.s *= f;
    z.si *= f;
    z.ref = -vm;
    z.limit = vm + step;
    return true;
}

// Partial sums of a warp's lanes, one per lane (maximum, s, si), as one.
__device__ __forceinline__ float3 merge_lanes(float top, float s, float si, float c2, bool set) {
    float3 r;
    r.x = warp_max(top);
    const float f = top == -INFINITY ? 0.f : ex2((top - r.x) * c2);     // 0 x NaN stays NaN
    r.y = warp_sum(s * f);
    r.z = set ? warp_sum(si * f) : 0.f;
    return r;
}

// Bytes of a row's listing in shared memory (rows with a remainder class): for
// each vector of the part the listed logits, a bit each, and for each entry
// whether it leads its vector.
__host__ __device__ constexpr int listing_bytes(int per, int k) { return (per + 15) / 16 * 16 + (k + 127) / 128 * 16; }

// A warp's run of 16-byte vectors of 16-bit values, lane l's at g + 16 l bytes,
// where g lies o bytes after a 16-byte boundary (o even, not 0) and lanes from
// nact on have none.  The vector before a lane's own comes from its neighbour, so
// all but the run's ends leave as aligned 16-byte stores; lane 0 writes the run's
// first 16 - o bytes, the lane after the last (lane 0 after 31) its last o, in
// powers of two.  0.6 GB of bf16 logits at 50001 with a gradient of another pitch,
// policy loss: 777 us stored by elements, 331 so (245 where the rows agree).
__device__ __forceinline__ void store_run(uint8_t* g, const uint4& q, int nact, int o) {
    const int lane = threadIdx.x & 31, src = (lane + 31) & 31;
    uint32_t w[8] = {__shfl_sync(0xffffffffu, q.x, src), __shfl_sync(0xffffffffu, q.y, src),
                     __shfl_sync(0xffffffffu, q.z, src), __shfl_sync(0xffffffffu, q.w, src), q.x, q.y, q.z, q.w};
    const int from = 16 - o;
    const bool by8 = from & 8, by4 = from & 4;
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = by8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = by4 ? w[k + 1] : w[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], (from & 2) * 8);
    uint8_t* at = g - o;
    if (lane > 0 && lane < nact) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    if (nact > 0 && (lane == 0 || lane == nact)) {
        if (lane == 0) {                        // bytes o .. 15
            const int p4 = (o + 3) & ~3, p8 = (p4 + 7) & ~7;
            if (o & 2)
                *reinterpret_cast<uint16_t*>(at + o) =
                    (uint16_t)((o & 8 ? (o & 4 ? w[3] : w[2]) : (o & 4 ? w[1] : w[0])) >> 16);
            if (p4 & 4) *reinterpret_cast<uint32_t*>(at + p4) = p4 & 8 ? w[3] : w[1];
            if (p8 == 8) *reinterpret_cast<uint2*>(at + 8) = make_uint2(w[2], w[3]);
        }
        if (lane == (nact & 31)) {              // bytes 0 .. o - 1 of what follows the run
            uint8_t* end = lane == 0 ? at + 512 : at;
            if (o & 8) *reinterpret_cast<uint2*>(end) = make_uint2(w[0], w[1]);
            if (o & 4) *reinterpret_cast<uint32_t*>(end + (o & 8)) = o & 8 ? w[2] : w[0];
            if (o & 2)
                *reinterpret_cast<uint16_t*>(end + (o & 12)) =
                    (uint16_t)(o & 8 ? (o & 4 ? w[3] : w[2]) : (o & 4 ? w[1] : w[0]));
        }
    }
}

struct PartArgs {
    int csize;              // CTAs per row
    int per;                // vectors of a row per CTA, at most SLOTS NT
    int* status;
};

// In distillation one warp of the CTA is for the listed entries, so that the
// walks stay free of them: the first walk leaves out whole vectors that hold one
// (their other logits are summed by that warp), and the second stores all
// logits alike, the listed ones' gradients following once it is through.
// Listings are kept for three rows in turn.  (A row's own is read before the
// first barrier of its pass alone, and the next one's written between the two
// barriers, so fewer would do.)  The warp's loads run a row ahead (cp.async),
// since its chain of steps is what the walks would wait for.
// Measured for 64 entries, 1.2 GB of logits at 65536: bf16 568 us (3.9-4.2 TB/s:
// two or three CTAs per SM are too few warps, 24 % active, to cover the waits;
// issue slots and DRAM 54 % busy each), fp32 467 (5.1 TB/s).  More entries cost:
// 4096 rows of 131072 bf16 logits 474 us with 64, 0.88 ms with 256, 5.9 ms with
// 1024 (with the rest's class 0.49, 1.16 and 8.7).  Listed logits handled inside the walks took 1.0-1.1 ms (branches
// that a fifth of a warp's vectors take, and partial sectors).
constexpr int TEACHERS = 3;
template <int MODE>
constexpr int TEACHER = MODE == LM_DISTILL ? 32 : 0;

template <typename T, int MODE, int NT>
__global__ void __launch_bounds__(NT + TEACHER<MODE>, 1024 / (NT + TEACHER<MODE>))
row_loss_kernel(const __grid_constant__ RowLossArgs a, const __grid_constant__ PartArgs pa) {
    constexpr int E = Vec<T>::E, NW = NT / 32, QUARTERS = 4;
    constexpr bool GRAD = MODE != LM_STATS, SET = MODE == LM_DISTILL;
    extern __shared__ __align__(16) uint8_t dyn8[];
    uint4* ring = reinterpret_cast<uint4*>(dyn8);       // [slots][NT]
    __shared__ float4 red[2][NW + 1];
    __shared__ __align__(16) float4 part[2][MAX_CLUSTER * (SET ? 2 : 1)];
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ float4 factors;                          // maximum, factors of e inside and outside S (policy: the token's
                                                        // gradient, factor of e), factor of t
    __shared__ float3 cross;                            // distillation: of this part, sum p (x - ref), sum p, ref
    __shared__ uint32_t odd_of_row[TEACHERS];           // which of the row's odd logits are listed
    __shared__ int abort_flag;
    const int V = a.vocab, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int csize = pa.csize, per = pa.per;
    const int rank = csize > 1 ? (int)tc::cluster_ctarank() : 0;
    const int64_t G = gridDim.x / csize, row0 = blockIdx.x / csize;
    const int slots = (per + NT - 1) / NT, quarter = (slots + QUARTERS - 1) / QUARTERS;
    const float c2 = a.c2, step = REBASE / c2;
    const uint64_t c22 = pair2(c2, c2);
    const bool rest_class = SET && a.tlse != nullptr;
    // of the row's entries: themselves (two rows), the vectors that hold their logits, the logits
    Listed* entries = reinterpret_cast<Listed*>(dyn8 + (size_t)slots * NT * 16);
    uint4* vecs = reinterpret_cast<uint4*>(entries + 2 * a.k);
    float* sx = reinterpret_cast<float*>(vecs + a.k);
    auto listing = [&](int buf) {
        return reinterpret_cast<uint8_t*>(sx) + (a.k + 3) / 4 * 16 + (size_t)buf * listing_bytes(per, a.k);
    };
    if (t == 0) {
        tc::mbar_init(smem_addr(&bars[0]), 1);
        tc::mbar_init(smem_addr(&bars[1]), 1);
        abort_flag = 0;
        tc::fence_mbar_init();
    }
    __syncthreads();
    if (csize > 1) tc::cluster_sync();                  // the cluster's barriers exist before anything targets them
    pdl_wait();
    pdl_trigger();

    auto row_live = [&](int64_t row) -> bool {
        if (row >= a.rows) return false;
        bool live = !a.weights || a.weights[row] != 0.f;
        if (MODE != LM_DISTILL) {
            const int64_t tok = ld_index(a.tokens, row, a.tok64);
            live = live && tok >= 0 && tok < V;
        }
        return live;
    };
    // whether `row`, the sequence's next, is live: 32 rows are looked up at a time
    uint32_t window = 0;
    int taken = 0;
    auto live_next = [&](int64_t row) -> bool {
        if ((taken & 31) == 0) window = __ballot_sync(0xffffffffu, row_live(row + (int64_t)lane * G));
        return (window >> (taken++ & 31)) & 1;
    };
    // geometry of a row: logits before its first vector, vectors of this CTA
    auto head_of = [&](const T* x) { return min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T)); };
    auto count_of = [&](int head) { return max(0, min(per, (V - head) / E - rank * per)); };
    // an odd logit of a row (the first CTA's first threads), -1 if none
    auto odd_of = [&](int head) -> int {
        if (rank != 0 || t >= 2 * E) return -1;
        if (t < head) return t;
        const int at = head + (V - head) / E * E + (t - head);
        return at < V ? at : -1;
    };

    // the thread that has logit `at` as its odd one, -1: none
    auto odd_thread = [&](int head, int at) {
        const int tail = head + (V - head) / E * E;
        return at < head ? at : at >= tail ? head + at - tail : -1;
    };

    // the row in the loss after the one worked on: its vectors are copied in as slots fall free
    const T* lx = nullptr;
    const T* lp = nullptr;                              // this thread's first vector of it
    int lhead = 0, lcount = 0;                          // its odd logits in front, the CTA's vectors of it
    float lodd = -INFINITY;                             // this thread's odd logit of it (warp 0)
    int64_t lrow = row0 - G;
    const uint32_t slot0 = smem_addr(ring + t);
    auto issue = [&](int u) {
        cp_async16(slot0 + u * (NT * 16), lp + u * (NT * E), t + u * NT < lcount);
    };
    const bool walker = !SET || warp < NW;
    // lists entry j0 + lane of row lrow, of index id, in buffer buf
    auto list = [&](int buf, int j0, int id) {
        uint8_t* flags = listing(buf);
        uint32_t* leads = reinterpret_cast<uint32_t*>(flags + (per + 15) / 16 * 16);
        const int part0 = lhead + rank * per * E, tail = lhead + (V - lhead) / E * E, at = id - part0;
        const bool in = id >= 0 && at >= 0 && at < lcount * E;
        const int vec = in ? at / E : 0;
        const uint32_t same = __match_any_sync(0xffffffffu, in ? vec : -1 - lane);
        const bool lead = in && flags[vec] == 0 && lane == __ffs(same) - 1;
        const uint32_t word = __ballot_sync(0xffffffffu, lead);
        if (lane == 0) leads[j0 >> 5] = word;
        if (in) atomicOr(reinterpret_cast<uint32_t*>(flags) + (vec >> 2), 1u << ((vec & 3) * 8 + at % E));
        else if (id >= 0 && rank == 0 && (id < lhead || id >= tail))
            atomicOr(&odd_of_row[buf], 1u << (id < lhead ? id : lhead + id - tail));
        __syncwarp();
    };

    // One pass per row in the loss, and one before the first that only fetches:
    // the row after the current one is found, the rows between, which are not
    // in the loss, get their zeros, and every per-row step appears once.
    int par = 1, nbuf = 0;
    uint32_t phase[2] = {0, 0};
    int64_t row = -1;
    do {
        par ^= 1;
        const int head = lhead, count = lcount;     // the row whose vectors are in the ring
        const int part0 = head + rank * per * E;    // the part's first logit
        const float odd = lodd;
        T* g = reinterpret_cast<T*>(a.grad) + row * a.ldg;
        int tok = 0;
        float xt = 0.f;
        float2 teacher = make_float2(0.f, 0.f);
        PolicyRow pr{1.0f, 0.f, 0.f, 0.f};
        if (row >= 0) {
            if (MODE != LM_DISTILL) tok = (int)ld_index(a.tokens, row, a.tok64);
            if (warp == 0) {                // under the first walk, for the step between the barriers
                if (MODE != LM_DISTILL) xt = Vec<T>::ld(lx + tok);
                if (MODE != LM_STATS && a.weights) pr.w = a.weights[row];
                if (SET) teacher = a.teacher[row];
                if (MODE == LM_POLICY) {
                    pr.adv = a.adv[row];
                    if (a.old_logp) pr.old = a.old_logp[row];
                    if (a.kl != 0.f) pr.ref = a.ref_logp[row];
                }
            }
        }
        const int buf = nbuf;                       // of the teacher's buffers
        nbuf = nbuf == TEACHERS - 1 ? 0 : nbuf + 1;
        const uint8_t* flags = listing(SET ? buf : 0);
        for (lrow += G; lrow < a.rows && !live_next(lrow); lrow += G) {
            if (GRAD && walker) {
                T* z = reinterpret_cast<T*>(a.grad) + lrow * a.ldg;
                const int h = head_of(z), n = count_of(h), at = odd_of(h);
                z += h + (int64_t)rank * per * E;
                for (int i = t; i < n; i += NT) *reinterpret_cast<uint4*>(z + i * E) = make_uint4(0, 0, 0, 0);
                if (at >= 0) Vec<T>::st(reinterpret_cast<T*>(a.grad) + lrow * a.ldg + at, 0.f);
            }
            if (rank == 0 && t == 0) {
                if (MODE == LM_STATS) a.stats[lrow] = RowStats{0.f, 0.f, 0.f, 0.f};
                else a.loss[lrow] = 0.f;
                if (MODE == LM_POLICY) a.logp[lrow] = 0.f;
            }
        }
        lcount = 0;
        if (lrow < a.rows) {
            lx = reinterpret_cast<const T*>(a.logits) + lrow * a.ld;
            lhead = head_of(lx);
            lcount = count_of(lhead);
            lp = lx + lhead + (int64_t)(rank * per + t) * E;
            if (warp == 0) {
                const int at = odd_of(lhead);
                lodd = at >= 0 ? Vec<T>::ld(lx + at) : -INFINITY;
            }
        }
        auto put_sums = [&](const Sums& z) {
            const float wm = warp_max(z.top);
            const float f = z.limit == -INFINITY ? 0.f : ex2((-z.ref - wm) * c2);
            const float s = warp_sum(z.s * f);
            const float si = rest_class ? warp_sum(z.si * f) : 0.f;
            if (lane == 0) red[par][warp] = make_float4(wm, s, si, 0.f);
        };
        // The entries' warp: the next row's entries start to come in; this row's
        // entries and the vectors of their logits have, since the last pass.
        const int tail = head + (V - head) / E * E;
        const Listed* here = entries + par * a.k;
        Listed* next_entries = entries + (par ^ 1) * a.k;
        // whether this CTA holds logit id: in its vectors, or (the first CTA) beside them
        auto held = [&](int id) {
            return (id >= part0 && id < part0 + count * E) || (rank == 0 && id >= 0 && (id < head || id >= tail));
        };
        if (!walker) {
            if (lrow < a.rows)
                for (int j = lane; j < a.k; j += 32) cp_async16(smem_addr(next_entries + j), a.listed + lrow * a.k + j, true);
            cp_async_commit();
            cp_async_wait(1);
            if (row >= 0) {
                const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld;
                const uint32_t* leads = reinterpret_cast<const uint32_t*>(flags + (per + 15) / 16 * 16);
                Sums z{0.f, -INFINITY, 0.f, 0.f, -INFINITY};    // of the vectors that the walk leaves out
                float top = -INFINITY;
                for (int j0 = 0; j0 < a.k; j0 += 32) {
                    const int j = j0 + lane, id = j < a.k ? here[j].id : -1;
                    if (held(id)) {
                        const float xj = Vec<T>::ld(id >= part0 && id < part0 + count * E
                                                        ? reinterpret_cast<const T*>(vecs + j) + (id - part0) % E : x + id);
                        sx[j] = xj;
                        top = fmaxf(top, xj);
                    }
                    if (rest_class && ((leads[j0 >> 5] >> lane) & 1)) {
                        const uint32_t f = flags[(id - part0) / E];
                        const uint4 raw = vecs[j];
                        follow(z, Vec<T>::vmax(raw), c2, step);
                        float v[E];
                        Vec<T>::unpack(raw, v);
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float ev = ex2((v[i] + z.ref) * c2);
                            if ((f >> i) & 1) z.si += ev;
                            else z.s += ev;
                        }
                    }
                }
                top = warp_max(top);
                const float ref = top == -INFINITY ? 0.f : top;
                float d = 0.f, ps = 0.f;
                for (int j = lane; j < a.k; j += 32) {
                    const float p = here[j].p;
                    if (p != 0.f && held(here[j].id)) {     // also where it is NaN
                        d += p * (sx[j] - ref);
                        ps += p;
                    }
                }
                d = warp_sum(d);
                ps = warp_sum(ps);
                if (lane == 0) cross = make_float3(d, ps, ref);
                if (rest_class) put_sums(z);
                else if (lane == 0) red[par][NW] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
            }
        }
        if (row >= 0) {
        if (walker) {
        // first walk
        Sums z{0.f, -INFINITY, 0.f, 0.f, -INFINITY};
        uint64_t ref2 = pair2(0.f, 0.f), sum2 = ref2;
        // slots beyond the part read as -inf
        for (int u = count / NT; u < slots; ++u)
            if (t + u * NT >= count) ring[u * NT + t] = make_uint4(Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE);
#pragma unroll
        for (int qd = 0; qd < QUARTERS; ++qd) {
            // pending behind this quarter: the row's later ones, and (statistics) the next row's earlier ones
            cp_async_wait(GRAD ? QUARTERS - 1 - qd : QUARTERS - 1);
            const int end = min(slots, (qd + 1) * quarter);
#pragma unroll 1
            for (int u = qd * quarter; u < end; ++u) {
                const uint4 raw = ring[u * NT + t];
                const float vm = Vec<T>::vmax(raw);
                z.top = fmaxf(z.top, vm);
                if (vm > z.limit) {
                    const float2 h = unpair(sum2);
                    z.s = h.x + h.y;
                    follow(z, vm, c2, step);
                    sum2 = pair2(z.s, 0.f);
                    ref2 = pair2(z.ref, z.ref);
                }
                uint64_t v[E / 2];
                unpack_pairs<T>(raw, v);
                exp_vec<E>(v, ref2, c22);
                // (flags beyond the part are another listing's bytes: those slots add nothing either way)
                if (!rest_class || flags[min(t + u * NT, per - 1)] == 0) {
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) sum2 = add2(sum2, v[j]);
                }
                if (!GRAD) issue(u);
            }
            if (!GRAD) cp_async_commit();
        }
        {
            const float2 h = unpair(sum2);
            z.s = h.x + h.y;
        }
        if (t < 2 * E && rank == 0) {
            follow(z, odd, c2, step);
            const float e = ex2((odd + z.ref) * c2);
            if (rest_class && ((odd_of_row[buf] >> t) & 1)) z.si += e;
            else z.s += e;
        }
        put_sums(z);
        }
        __syncthreads();
        if (warp == 0) {
            const float4 r = lane < NW + (SET ? 1 : 0) ? red[par][lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            float3 q = merge_lanes(r.x, r.y, r.z, c2, SET);
            float3 dp = SET ? cross : make_float3(0.f, 0.f, 0.f);
            if (csize > 1) {
                // the token's logit travels along: it has been read before any CTA's gradient can replace it
                const uint32_t bar = smem_addr(&bars[par]);
                if (lane == 0) tc::mbar_expect_tx(bar, (uint32_t)((SET ? 32 : 16) * csize));
                __syncwarp();
                if (lane < csize) {
                    st_async_f4(smem_addr(&part[par][rank]), bar, (uint32_t)lane, make_float4(q.x, q.y, q.z, xt));
                    if (SET)
                        st_async_f4(smem_addr(&part[par][MAX_CLUSTER + rank]), bar, (uint32_t)lane,
                                    make_float4(dp.x, dp.y, dp.z, 0.f));
                }
                tc::wait_bounded(bar, phase[par], &abort_flag, pa.status);
                phase[par] ^= 1u;
                __syncwarp();
                const float4 c = lane < csize ? part[par][lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
                if (SET) {
                    const float4 e = lane < csize ? part[par][MAX_CLUSTER + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                    dp = make_float3(e.x, e.y, e.z);
                }
                q = merge_lanes(c.x, c.y, c.z, c2, SET);
            } else if (SET && lane > 0) {
                dp = make_float3(0.f, 0.f, 0.f);
            }
            const float m = q.x, all = q.y + q.z, log_s = ::logf(all), inv_s = 1.0f / all;
            const bool writes = rank == 0 && lane == 0;
            if (MODE == LM_STATS) {
                if (writes) a.stats[row] = RowStats{m, inv_s, (xt - m) * a.inv_t - log_s, 0.f};
            } else {
                const float w = pr.w;
                if (MODE == LM_POLICY) {
                    const float lt = (xt - m) * a.inv_t - log_s;
                    float loss, dl;
                    policy_row(a, pr, lt, loss, dl);
                    if (writes) {
                        a.loss[row] = w * loss;
                        a.logp[row] = lt;
                    }
                    const float scale = w * dl * a.inv_t;
                    // the token's gradient, everyone's factor of e
                    if (lane == 0)
                        factors = make_float4(m, fmaf(-scale * inv_s, ex2((xt - m) * c2), scale), -scale * inv_s, scale);
                } else {
                    float rest = 0.f, share = 0.f, kl = 0.f;
                    const float mass = teacher.x;
                    if (rest_class) {
                        const float qr = q.y * inv_s;
                        rest = 1.0f - mass;
                        if (!(rest > 0.f && qr > 0.f)) rest = 0.f;
                        else {
                            share = rest / qr;
                            kl = rest * ::logf(share);
                        }
                    }
                    // sum p (log p - log q) = sum p log p - sum p ((x - m) / T - log s), the parts' sums
                    // taken against references of their own
                    float dm = 0.f;
                    if (dp.y != 0.f) dm = dp.x + dp.y * (dp.z - m);
                    dm = warp_sum(dm);
                    const float ps = warp_sum(dp.y);
                    if (ps != 0.f) kl += teacher.y - dm * a.inv_t + ps * log_s;
                    // a row without a distribution has no loss, with nothing listed either
                    if (writes) a.loss[row] = all > 0.f ? w * a.t * a.t * kl : NAN;
                    const float scale = w * a.t;
                    if (lane == 0)
                        factors = make_float4(m, scale * (mass + rest) * inv_s, scale * (mass + rest - share) * inv_s, scale);
                }
            }
        }
        }
        if (!walker) {
            cp_async_wait(0);
            if (rest_class && lrow < a.rows) {
                // the next row's listing, while warp 0 brings this row's sums together
                uint8_t* to = listing(nbuf);
                for (int i = lane; i < (per + 15) / 16; i += 32) reinterpret_cast<uint4*>(to)[i] = make_uint4(0, 0, 0, 0);
                if (lane == 0) odd_of_row[nbuf] = 0;
                __syncwarp();
                for (int j0 = 0; j0 < a.k; j0 += 32) list(nbuf, j0, j0 + lane < a.k ? next_entries[j0 + lane].id : -1);
            }
        }
        if (GRAD) __syncthreads();
        const float4 fac = factors;
        const float m = fac.x, scale = fac.w;
        if (!walker) {
            // the vectors that hold the next row's listed logits
            if (lrow < a.rows) {
                const int next0 = lhead + rank * per * E;
                for (int j = lane; j < a.k; j += 32) {
                    const int at = next_entries[j].id - next0;
                    cp_async16(smem_addr(vecs + j), lx + next0 + (at >= 0 ? at / E * E : 0), at >= 0 && at < lcount * E);
                }
            }
            cp_async_commit();
            if (row >= 0) {
                // the listed gradients of this part, once the second walk is through (an index listed
                // twice counts twice, at its first entry)
                asm volatile("bar.sync 1, %0;" ::"n"(NT + 32) : "memory");
                for (int j = lane; j < a.k; j += 32) {
                    const Listed q = here[j];
                    if (held(q.id) && !(q.psum < 0.f))
                        Vec<T>::st(g + q.id, fac.y * ex2((sx[j] - m) * c2) - scale * q.psum);
                }
            }
            row = lrow;
            continue;
        }
        // second walk: out q everywhere, the token's entry on the way
        const uint64_t out2 = pair2(fac.z, fac.z);
        const uint64_t ref2 = pair2(-m, -m);
        T* gp = g + part0 + t * E;
        const int off = a.same_align ? 0 : (int)(reinterpret_cast<uintptr_t>(gp) & 15);
        // (`run`: rows whose gradient lies elsewhere between 16-byte boundaries, in a loop of their own:
        // the aligned one with both in it took 4-10 % longer)
        auto slot = [&](int u, bool run) {
            const int i = t + u * NT;
            if (GRAD && row >= 0) {
                uint64_t v[E / 2];
                float f[E];
                unpack_pairs<T>(ring[i], v);
                exp_vec<E>(v, ref2, c22);
#pragma unroll
                for (int j = 0; j < E / 2; ++j) v[j] = mul2(v[j], out2);
                split_pairs<E>(v, f);
                const uint4 packed = Vec<T>::pack(f);
                if (run) {
                    if (sizeof(T) == 2) {
                        store_run(reinterpret_cast<uint8_t*>(gp + u * (NT * E)), packed, min(32, count - (i - lane)), off);
                    } else if (i < count) {
#pragma unroll
                        for (int j = 0; j < E; ++j) Vec<T>::st(gp + u * (NT * E) + j, f[j]);
                    }
                } else if (SET) {
                    // evict-first in distillation alone, where it measured 565-629 -> 536-579 us for 1.2 GB
                    // of 16-bit logits; no difference in the policy loss
                    if (i < count) __stcs(reinterpret_cast<uint4*>(gp + u * (NT * E)), packed);
                } else {
                    if (i < count) *reinterpret_cast<uint4*>(gp + u * (NT * E)) = packed;
                }
            }
            issue(u);
        };
#pragma unroll
        for (int qd = 0; qd < QUARTERS && (GRAD || row < 0); ++qd) {
            const int end = min(slots, (qd + 1) * quarter);
            if (GRAD && off != 0) {
#pragma unroll 1
                for (int u = qd * quarter; u < end; ++u) slot(u, true);
            } else {
#pragma unroll 1
                for (int u = qd * quarter; u < end; ++u) slot(u, false);
            }
            cp_async_commit();
        }
        if (GRAD && warp == 0 && row >= 0) {
            const int at = odd_of(head);
            if (at >= 0) Vec<T>::st(g + at, ex2((odd - m) * c2) * fac.z);
        }
        if (MODE == LM_POLICY && row >= 0) {
            // the token's own entry over what its warp stored
            __syncwarp();
            const int at = tok - part0;
            const bool vec = at >= 0 && at < count * E;
            if (vec ? t == at / E % NT : rank == 0 && t == odd_thread(head, tok)) Vec<T>::st(g + tok, fac.y);
        }
        if (SET && row >= 0) asm volatile("bar.arrive 1, %0;" ::"n"(NT + 32) : "memory");
        row = lrow;
    } while (row < a.rows);
    cp_async_wait(0);
    if (csize > 1) {
        __syncthreads();
        tc::cluster_sync();                 // no CTA leaves while another may still write to its shared memory
    }
}

// The teacher's side of every row, a warp per row: its softmax over the listed
// entries (or against its own log-sum-exp), and repeated indices brought
// together (looked for, in k^2 steps, only where two entries of a row share a bit
// of a 32768-bit map: 6 % of rows without a repeat at k = 64, all at 1024).  The student's logits at the entries are left to the row's own CTAs,
// which read them while they read the row: gathered here, from all over the
// logits at once, they took 0.4 ms for 9155 x 64.
constexpr int TW = 4;                       // warps of a CTA
__global__ void __launch_bounds__(32 * TW) teacher_kernel(const __grid_constant__ RowLossArgs a) {
    __shared__ __align__(16) uint32_t seen[TW][1024];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    for (int64_t row = (int64_t)blockIdx.x * TW + warp; row < a.rows; row += (int64_t)gridDim.x * TW) {
        if (a.weights && a.weights[row] == 0.f) continue;
        auto entry = [&](int j, float& v) {
            const int64_t id = ld_index(a.tidx, row * a.k + j, a.tidx64);
            const bool ok = id >= 0 && id < a.vocab;
            v = ok ? ld_elem(a.tval, row * a.k + j, a.tval_dtype) : -INFINITY;
            return ok ? (int)id : -1;
        };
        float tm = 0.f, lse = 0.f, v;
        if (a.tlse) {
            lse = a.tlse[row];
        } else {
            tm = -INFINITY;
            for (int j = lane; j < a.k; j += 32) {
                entry(j, v);
                tm = fmaxf(tm, v);
            }
            tm = warp_max(tm);
        }
        for (int i = lane; i < 256; i += 32) reinterpret_cast<uint4*>(seen[warp])[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
        float s = 0.f;
        bool again = false;
        for (int j = lane; j < a.k; j += 32) {
            const int id = entry(j, v);
            if (id < 0) continue;
            s += expf((v - tm) * a.inv_t - lse);
            const uint32_t bit = 1u << (id & 31);
            again = (atomicOr(&seen[warp][(id >> 5) & 1023], bit) & bit) || again;
        }
        s = warp_sum(s);
        again = __any_sync(0xffffffffu, again);
        if (!a.tlse) {
            lse = ::logf(s);
            s = s > 0.f || s != s ? 1.0f : 0.f;         // nothing listed: no distribution, no loss
        }
        Listed* out = a.listed + row * a.k;
        float plp = 0.f;
        for (int j = lane; j < a.k; j += 32) {
            Listed e;
            e.id = entry(j, v);
            const float lp = e.id >= 0 ? (v - tm) * a.inv_t - lse : -INFINITY;
            e.p = e.psum = expf(lp);
            e.pad = 0;
            if (e.p != 0.f) plp += e.p * lp;
            out[j] = e;
        }
        plp = warp_sum(plp);
        if (again) {
            __syncwarp();
            for (int j = lane; j < a.k; j += 32) {
                const int id = out[j].id;
                float sum = 0.f;
                bool first = true;
                for (int n = 0; n < a.k; ++n) {
                    if (out[n].id == id) {
                        sum += out[n].p;
                        first = first && n >= j;
                    }
                }
                out[j].psum = first ? sum : -1.0f;
            }
        }
        if (lane == 0) a.teacher[row] = make_float2(s, plp);
        __syncwarp();
    }
}

// Gradient rows of the preference loss, coef ([v = token] - q_v): a stream over
// all logits, a CTA per GC vectors of a row.  Rows are taken last first: the
// statistics' launch read them in order, so the last ones are still in L2.
constexpr int GC = 2048, GU = 4;        // vectors per CTA, in flight per thread
template <typename T, bool SAME>        // the gradient's rows on the logits' 16-byte phase
__global__ void __launch_bounds__(256, 4) row_grad_kernel(const __grid_constant__ RowLossArgs a, int chunks) {
    constexpr int E = Vec<T>::E;
    const int V = a.vocab, t = threadIdx.x;
    const uint64_t c22 = pair2(a.c2, a.c2);
    pdl_wait();
    pdl_trigger();
    for (int64_t b = blockIdx.x; b < a.rows * chunks; b += gridDim.x) {
        const int64_t back = b / chunks, row = a.rows - 1 - back;
        const int chunk = (int)(b - back * chunks);
        const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld;
        T* g = reinterpret_cast<T*>(a.grad) + row * a.ldg;
        const RowStats st = a.stats[row];
        const bool on = st.coef != 0.f;     // also where it is NaN
        // the aligned vectors of the row that is read (of the gradient's where it is only cleared)
        const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(on ? x : g) & 15)) & 15) / (int)sizeof(T));
        const int nv = (V - head) / E, end = min(nv, (chunk + 1) * GC);
        const int tok = on ? (int)ld_index(a.tokens, row, a.tok64) : -1;
        const float f = -st.coef * st.inv_s;
        const uint64_t f2 = pair2(f, f), ref2 = pair2(-st.mx, -st.mx);
        const int off = SAME || !on ? 0 : (int)(reinterpret_cast<uintptr_t>(g + head) & 15);
        for (int i0 = chunk * GC + t; (SAME ? i0 : i0 - (t & 31)) < end; i0 += GU * 256) {   // (whole warps, for store_run)
            uint4 q[GU];
#pragma unroll
            for (int u = 0; u < GU; ++u)
                if (on && i0 + u * 256 < end) q[u] = *reinterpret_cast<const uint4*>(x + head + (int64_t)(i0 + u * 256) * E);
#pragma unroll
            for (int u = 0; u < GU; ++u) {
                const int v0 = head + (i0 + u * 256) * E;
                const bool mine = i0 + u * 256 < end;
                if (SAME ? mine : i0 + u * 256 - (t & 31) < end) {
                    float r[E];
                    if (on) {
                        uint64_t v[E / 2];
                        unpack_pairs<T>(q[u], v);
                        exp_vec<E>(v, ref2, c22);
#pragma unroll
                        for (int j = 0; j < E / 2; ++j) v[j] = mul2(v[j], f2);
                        split_pairs<E>(v, r);
                        if ((unsigned)(tok - v0) < (unsigned)E) {
#pragma unroll
                            for (int j = 0; j < E; ++j)
                                if (v0 + j == tok) r[j] += st.coef;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < E; ++j) r[j] = 0.f;
                    }
                    if (off == 0) {
                        if (mine) *reinterpret_cast<uint4*>(g + v0) = Vec<T>::pack(r);
                    } else if (sizeof(T) == 2) {
                        store_run(reinterpret_cast<uint8_t*>(g + v0), Vec<T>::pack(r), min(32, end - (i0 + u * 256 - (t & 31))), off);
                    } else if (mine) {
#pragma unroll
                        for (int j = 0; j < E; ++j) Vec<T>::st(g + v0 + j, r[j]);
                    }
                }
            }
        }
        // what the row has before and after its vectors
        if (chunk == 0 && t < 2 * E) {
            const int at = t < head ? t : head + nv * E + (t - head);
            if (at < V) Vec<T>::st(g + at, on ? fmaf(f, ex2((Vec<T>::ld(x + at) - st.mx) * a.c2), at == tok ? st.coef : 0.f) : 0.f);
        }
    }
}

struct PairArgs {
    RowStats* stats;
    int64_t rows;
    const void* bounds;         // 2 pairs + 1 row offsets
    int bounds64;
    const float* ref_logp;      // per sequence, or null
    const float* weights;       // per pair, or null
    float beta, margin, smoothing;
    int average;
    float* seq_logp;
    float* loss;
};

// One CTA per pair, half of it per sequence: both sequence values (fp64 sums in
// a fixed order), the pair's loss, and the factor of every row of the pair.  A
// row in the loss is one whose statistics say so (inv_s != 0).
constexpr int PT = 512;
__global__ void __launch_bounds__(PT) pair_kernel(const __grid_constant__ PairArgs a) {
    constexpr int HT = PT / 2;
    __shared__ double rs[PT / 32];
    __shared__ int rn[PT / 32];
    const int64_t pair = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = threadIdx.x / HT, t = threadIdx.x % HT;
    pdl_wait();
    pdl_trigger();
    auto bound = [&](int i) {
        const int64_t v = ld_index(a.bounds, 2 * pair + i, a.bounds64);
        return v < 0 ? (int64_t)0 : (v > a.rows ? a.rows : v);
    };
    const int64_t b0 = bound(c), b1 = bound(c + 1);
    const float w = a.weights ? a.weights[pair] : 1.0f;
    double ref = 0.0;
    if (a.ref_logp) ref = (double)a.ref_logp[2 * pair] - (double)a.ref_logp[2 * pair + 1];
    double s = 0;
    int n = 0;
    for (int64_t r = b0 + t; r < b1; r += HT) {
        const RowStats st = a.stats[r];
        if (st.inv_s != 0.f) {
            s += (double)st.logp;
            ++n;
        }
    }
    for (int o = 16; o; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane == 0) {
        rs[warp] = s;
        rn[warp] = n;
    }
    __syncthreads();
    double val[2] = {0.0, 0.0};
    int cnt[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < PT / 32; ++i) {
        val[i / (HT / 32)] += rs[i];
        cnt[i / (HT / 32)] += rn[i];
    }
    if (a.average)
        for (int i = 0; i < 2; ++i) val[i] = cnt[i] > 0 ? val[i] / cnt[i] : 0.0;
    const float h = (float)((double)a.beta * (val[0] - val[1] - ref) - (double)a.margin);
    // -log sigmoid(h) and -log sigmoid(-h), each by itself (their difference h
    // may be infinite, or all that is left of the smaller one), and sigmoid(h),
    // sigmoid(-h) without overflow
    const float e = expf(-fabsf(h)), near = log1pf(e);
    const float big = 1.0f / (1.0f + e), small = e * big;
    const float sp = h >= 0.f ? big : small, sn = h >= 0.f ? small : big;
    float loss = 0.f, dh = -(1.0f - a.smoothing) * sn;
    if (a.smoothing != 1.f) loss = (1.0f - a.smoothing) * (fmaxf(-h, 0.f) + near);
    if (a.smoothing != 0.f) {
        loss += a.smoothing * (fmaxf(h, 0.f) + near);
        dh += a.smoothing * sp;
    }
    if (h != h) loss = dh = h;
    const bool on = w != 0.f;
    if (t == 0) {
        a.seq_logp[2 * pair + c] = (float)val[c];
        if (c == 0) a.loss[pair] = on ? w * loss : 0.f;
    }
    const float share = a.average ? (cnt[c] > 0 ? 1.0f / (float)cnt[c] : 0.f) : 1.0f;
    const float coef = on ? (c ? -1.0f : 1.0f) * w * dh * a.beta * share : 0.f;
    for (int64_t r = b0 + t; r < b1; r += HT)
        if (a.stats[r].inv_s != 0.f) a.stats[r].coef = coef;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t MAX_VOCAB = 1 << 19;
constexpr int MAX_TEACHER = 1024;

// Shared memory of a row's CTA: its part of the row, and for distillation the
// listings of three rows.
template <typename T, int MODE, int NT>
size_t row_smem(int per, int k) {
    size_t b = (size_t)((per + NT - 1) / NT) * NT * 16;
    if (MODE == LM_DISTILL) b += (size_t)TEACHERS * listing_bytes(per, k) + 48 * (size_t)k + (size_t)(k + 3) / 4 * 16;
    return b;
}

// Shared memory of a part in distillation, and what a CTA may have.
constexpr size_t PART_SMEM = 85000, MAX_SMEM = 220000;

template <typename T, int MODE, int NT>
cudaError_t launch_part(const RowLossArgs& a, int64_t nv, int csize, const DevCtx& dc, cudaStream_t s) {
    auto kern = row_loss_kernel<T, MODE, NT>;
    static OncePer<int, int> attrs;                         // by device
    int set = 0;
    cudaError_t err = attrs.get(dc.device, &set, [&](int&) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MAX_SMEM);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e;
    });
    if (err != cudaSuccess) return err;
    PartArgs pa;
    pa.csize = csize;
    pa.per = (int)((nv + csize - 1) / csize);
    pa.status = dc.status;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)csize);
    cfg.blockDim = dim3(NT + TEACHER<MODE>);
    cfg.dynamicSmemBytes = row_smem<T, MODE, NT>(pa.per, a.k);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)csize;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    // clusters resident at once with what a CTA keeps (a teacher's entries
    // included), by device, cluster size and kilobytes
    static OncePer<std::tuple<int, int, int>, int> fits;
    const int kb = (int)((cfg.dynamicSmemBytes + 1023) / 1024);
    int n = 0;
    err = fits.get({dc.device, csize, kb}, &n, [&](int& v) {
        cfg.attrs = at + 1;
        cfg.numAttrs = 1;
        cudaLaunchConfig_t most = cfg;
        most.dynamicSmemBytes = std::min((size_t)kb * 1024, MAX_SMEM);
        cudaError_t e = cudaOccupancyMaxActiveClusters(&v, kern, &most);
        if (e == cudaSuccess && v < 1) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess)
            muon::logf(2, "row loss mode %d: %d threads, %d CTAs per row, %d vectors each, %zu bytes, %d clusters", MODE,
                       NT, csize, pa.per, most.dynamicSmemBytes, v);
        return e;
    });
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3((unsigned)(csize * std::min<int64_t>(a.rows, n)));
    // A launch whose clusters walk several rows each waits for the one before it
    // to end: placed beside its last CTAs, clusters may leave holes that one of
    // them does not fit, and its rows then follow as a wave of their own (measured
    // behind teacher_kernel: 0.64 ms became 1.0).
    const bool early = pdl_enabled() && a.rows <= n;
    cfg.attrs = early ? at : at + 1;
    cfg.numAttrs = early ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, pa);
}


// How a launch divides its rows: 128-thread CTAs for rows of up to SLOTS vectors
// per thread of theirs; else 256-thread CTAs, as few per row as hold it with four
// CTAs on an SM (16 at most, then with more shared memory each), twice as many
// while the rows alone would leave SMs idle and a thread keeps four vectors.
// Four CTAs of 256 threads beat two of 512 (a CTA's wait between its walks is
// hidden by the others): 131072 bf16 logits 530 -> 482 us for 1.2 GB of logits,
// fp32 459 -> 423; eight of 128 with twice the slots took 567 and 501.
// Distillation, with more to keep per CTA, takes powers of two and two or three
// CTAs on an SM: for the same 1.2 GB, fp32 131072 by 8 CTAs 480 us, by 12 (four
// on an SM) 503, by 10 584; fp32 65536 by 4 465, by 5 566, by 6 488; bf16 50001
// by 2 565, by 3 610; bf16 131072 by 4 629, by 6 606, by 8 608.
template <typename T, int MODE>
cudaError_t launch_mode(const RowLossArgs& a, const DevCtx& dc, cudaStream_t s) {
    constexpr int NT = 256 - TEACHER<MODE>, SMALL = 128 - TEACHER<MODE>;
    const int64_t nv = std::max(1, a.vocab / Vec<T>::E);       // whole vectors of a row at most
    if (nv <= SLOTS * SMALL) return launch_part<T, MODE, SMALL>(a, nv, 1, dc, s);
    auto smem = [&](int c) { return row_smem<T, MODE, NT>((int)((nv + c - 1) / c), a.k); };
    int c = 1;
    if (MODE == LM_DISTILL)
        while (c < MAX_CLUSTER && smem(c) > PART_SMEM) c *= 2;
    else
        c = (int)std::min<int64_t>(MAX_CLUSTER, (nv + SLOTS * NT - 1) / (SLOTS * NT));
    while (c <= 4 && a.rows * c < dc.sms && nv > (int64_t)c * 4 * NT) c *= 2;
    return launch_part<T, MODE, NT>(a, nv, c, dc, s);
}

template <typename T>
cudaError_t launch_rows(const RowLossArgs& a, int mode, const DevCtx& dc, cudaStream_t s) {
    if (mode == LM_POLICY) return launch_mode<T, LM_POLICY>(a, dc, s);
    if (mode == LM_STATS) return launch_mode<T, LM_STATS>(a, dc, s);
    return launch_mode<T, LM_DISTILL>(a, dc, s);
}

template <typename T>
cudaError_t launch_grad(const RowLossArgs& a, cudaStream_t s) {
    const int chunks = std::max(1, (a.vocab / Vec<T>::E + GC - 1) / GC);
    return launch_pdl(a.same_align ? row_grad_kernel<T, true> : row_grad_kernel<T, false>, dim3((unsigned)std::min<int64_t>(a.rows * chunks, 1 << 30)), dim3(256), 0, s, a,
                      chunks);
}

cudaError_t dispatch_rows(const RowLossArgs& a, int mode, int dtype, const DevCtx& dc, cudaStream_t s) {
    if (dtype == MUON_F32) return launch_rows<float>(a, mode, dc, s);
    if (dtype == MUON_BF16) return launch_rows<__nv_bfloat16>(a, mode, dc, s);
    return launch_rows<__half>(a, mode, dc, s);
}

cudaError_t dispatch_grad(const RowLossArgs& a, int dtype, cudaStream_t s) {
    if (dtype == MUON_F32) return launch_grad<float>(a, s);
    if (dtype == MUON_BF16) return launch_grad<__nv_bfloat16>(a, s);
    return launch_grad<__half>(a, s);
}

bool valid_index(int d) { return d == MUON_I32 || d == MUON_I64; }

// The checks every loss makes of its logits and gradient; fills the shared
// fields.  Nothing is enqueued.
int row_args(RowLossArgs& a, const void* logits, int64_t ld, int64_t rows, int64_t vocab, int dtype, float temperature,
             void* grad, int64_t ld_grad) {
    std::memset(&a, 0, sizeof a);
    if (!valid_dtype(dtype)) return fail(MUON_EDTYPE, "logits dtype %d", dtype);
    if (rows < 0 || rows > INT32_MAX) return fail(MUON_EINVAL, "rows outside [0, 2^31)");
    if (vocab < 1 || vocab > MAX_VOCAB) return fail(MUON_EINVAL, "vocab outside [1, 2^19]");
    if (ld < vocab || ld_grad < vocab) return fail(MUON_EINVAL, "row pitch below vocab");
    if (ld > INT64_MAX / 8 / std::max<int64_t>(rows, 1) || ld_grad > INT64_MAX / 8 / std::max<int64_t>(rows, 1))
        return fail(MUON_EINVAL, "byte range overflows");
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature))
        return fail(MUON_EINVAL, "temperature must be positive and finite");
    if (rows == 0) return MUON_OK;
    if (!logits || !grad) return fail(MUON_EINVAL, "NULL logits or grad");
    const size_t es = esize(dtype);
    const uintptr_t pl = reinterpret_cast<uintptr_t>(logits), pg = reinterpret_cast<uintptr_t>(grad);
    if (pl % es || pg % es) return fail(MUON_EINVAL, "pointer not aligned to its element");
    if (pl == pg && ld != ld_grad) return fail(MUON_EINVAL, "gradient in place of the logits needs their row pitch");
    const uintptr_t ll = ((uintptr_t)(rows - 1) * ld + vocab) * es, lg = ((uintptr_t)(rows - 1) * ld_grad + vocab) * es;
    if (pl != pg && pl < pg + lg && pg < pl + ll)
        return fail(MUON_EINVAL, "logits and gradient overlap without being the same matrix");
    a.logits = logits; a.grad = grad; a.ld = ld; a.ldg = ld_grad;
    a.rows = rows; a.vocab = (int)vocab;
    a.same_align = ((pl - pg) % 16 == 0) && (((uint64_t)ld * es - (uint64_t)ld_grad * es) % 16 == 0);
    a.c2 = (float)(1.4426950408889634 / (double)temperature);
    a.inv_t = (float)(1.0 / (double)temperature);
    a.t = temperature;
    if (!std::isfinite(a.c2)) return fail(MUON_EINVAL, "temperature must be positive and finite");
    return MUON_OK;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" int muon_distill_loss(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int dtype,
                                 const void* teacher_idx, int idx_dtype, const void* teacher_logits,
                                 int teacher_dtype, int64_t k, const float* teacher_lse, const float* weights,
                                 float temperature, float* loss, void* grad, int64_t ld_grad, void* stream) try {
    RowLossArgs a;
    int r = row_args(a, logits, ld, rows, vocab, dtype, temperature, grad, ld_grad);
    if (r) return r;
    if (!valid_index(idx_dtype)) return fail(MUON_EDTYPE, "index dtype %d", idx_dtype);
    if (!valid_dtype(teacher_dtype)) return fail(MUON_EDTYPE, "teacher dtype %d", teacher_dtype);
    if (k < 1 || k > MAX_TEACHER) return fail(MUON_EINVAL, "k outside [1, %d]", MAX_TEACHER);
    if (rows == 0) return MUON_OK;
    if (!teacher_idx || !teacher_logits || !loss) return fail(MUON_EINVAL, "NULL argument");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.tidx = teacher_idx; a.tidx64 = idx_dtype == MUON_I64;
    a.tval = teacher_logits; a.tval_dtype = teacher_dtype;
    a.tlse = teacher_lse; a.k = (int)k;
    a.weights = weights; a.loss = loss;
    const size_t listed = align_up(sizeof(Listed) * (size_t)rows * (size_t)k, 256);
    Workspace* w = nullptr;
    if ((r = ws_get(dc.device, s, listed + sizeof(float2) * (size_t)rows, &w))) return r;
    a.listed = reinterpret_cast<Listed*>(w->base);
    a.teacher = reinterpret_cast<float2*>(w->base + listed);
    const dim3 tg((unsigned)std::min<int64_t>((rows + TW - 1) / TW, (int64_t)dc.sms * 12));
    note_launch_begin(KC_LOSS, s);
    cudaError_t e = launch_pdl(teacher_kernel, tg, dim3(32 * TW), 0, s, a);
    note_launch_end(KC_LOSS, 0.0, s);
    if (e != cudaSuccess) return cuda_fail(e, "teacher launch");
    note_launch_begin(KC_LOSS, s);
    e = dispatch_rows(a, LM_DISTILL, dtype, dc, s);
    note_launch_end(KC_LOSS, 2.0 * (double)rows * vocab * esize(dtype), s);
    if (e != cudaSuccess) return cuda_fail(e, "distillation launch");
    return MUON_OK;
} MUON_CATCH_ALL

extern "C" int muon_policy_loss(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int dtype,
                                const void* tokens, int token_dtype, const float* advantages, const float* old_logp,
                                const float* ref_logp, const float* weights, float temperature, float clip_low,
                                float clip_high, float kl_coef, float* loss, float* logp, void* grad, int64_t ld_grad,
                                void* stream) try {
    RowLossArgs a;
    int r = row_args(a, logits, ld, rows, vocab, dtype, temperature, grad, ld_grad);
    if (r) return r;
    if (!valid_index(token_dtype)) return fail(MUON_EDTYPE, "token dtype %d", token_dtype);
    if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !std::isfinite(kl_coef))
        return fail(MUON_EINVAL, "clip_low in [0, 1], clip_high >= 0 and a finite kl_coef are needed");
    if (rows == 0) return MUON_OK;
    if (!tokens || !advantages || !loss || !logp) return fail(MUON_EINVAL, "NULL argument");
    if (kl_coef != 0.f && !ref_logp) return fail(MUON_EINVAL, "a KL term needs ref_logp");
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.tokens = tokens; a.tok64 = token_dtype == MUON_I64;
    a.adv = advantages; a.old_logp = old_logp; a.ref_logp = ref_logp;
    a.weights = weights;
    a.lo = (float)(1.0 - (double)clip_low); a.hi = (float)(1.0 + (double)clip_high); a.kl = kl_coef;
    a.loss = loss; a.logp = logp;
    note_launch_begin(KC_LOSS, s);
    cudaError_t e = dispatch_rows(a, LM_POLICY, dtype, dc, s);
    note_launch_end(KC_LOSS, 2.0 * (double)rows * vocab * esize(dtype), s);
    if (e != cudaSuccess) return cuda_fail(e, "policy loss launch");
    return MUON_OK;
} MUON_CATCH_ALL

extern "C" int muon_preference_loss(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int dtype,
                                    const void* tokens, int token_dtype, const void* seq_bounds, int bounds_dtype,
                                    int64_t pairs, const float* ref_logp, const float* weights, float beta,
                                    float margin, float label_smoothing, int average, float* loss, float* seq_logp,
                                    void* grad, int64_t ld_grad, void* stream) try {
    RowLossArgs a;
    int r = row_args(a, logits, ld, rows, vocab, dtype, 1.0f, grad, ld_grad);
    if (r) return r;
    if (!valid_index(token_dtype) || !valid_index(bounds_dtype))
        return fail(MUON_EDTYPE, "index dtypes %d / %d", token_dtype, bounds_dtype);
    if (pairs < 0 || pairs > INT32_MAX / 2) return fail(MUON_EINVAL, "pairs outside [0, 2^30)");
    if (!std::isfinite(beta) || !std::isfinite(margin) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
        return fail(MUON_EINVAL, "finite beta and margin and label_smoothing in [0, 1] are needed");
    if (pairs > 0 && (!seq_bounds || !loss || !seq_logp)) return fail(MUON_EINVAL, "NULL argument");
    if (rows > 0 && !tokens) return fail(MUON_EINVAL, "NULL tokens");
    if (rows == 0 && pairs == 0) return MUON_OK;
    DevCtx dc;
    if ((r = get_dev(dc))) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Workspace* w = nullptr;
    if ((r = ws_get(dc.device, s, std::max<size_t>(256, sizeof(RowStats) * (size_t)rows), &w))) return r;
    a.stats = reinterpret_cast<RowStats*>(w->base);
    a.tokens = tokens; a.tok64 = token_dtype == MUON_I64;
    const double bytes = (double)rows * vocab * esize(dtype);
    cudaError_t e;
    if (rows > 0) {
        note_launch_begin(KC_LOSS, s);
        e = dispatch_rows(a, LM_STATS, dtype, dc, s);
        note_launch_end(KC_LOSS, bytes, s);
        if (e != cudaSuccess) return cuda_fail(e, "preference statistics launch");
    }
    if (pairs > 0) {
        PairArgs p;
        p.stats = a.stats; p.rows = rows;
        p.bounds = seq_bounds; p.bounds64 = bounds_dtype == MUON_I64;
        p.ref_logp = ref_logp; p.weights = weights;
        p.beta = beta; p.margin = margin; p.smoothing = label_smoothing; p.average = average != 0;
        p.seq_logp = seq_logp; p.loss = loss;
        note_launch_begin(KC_LOSS, s);
        e = launch_pdl(pair_kernel, dim3((unsigned)pairs), dim3(PT), 0, s, p);
        note_launch_end(KC_LOSS, 0.0, s);
        if (e != cudaSuccess) return cuda_fail(e, "preference pair launch");
    }
    if (rows > 0) {
        note_launch_begin(KC_LOSS, s);
        e = dispatch_grad(a, dtype, s);
        note_launch_end(KC_LOSS, 2.0 * bytes, s);
        if (e != cudaSuccess) return cuda_fail(e, "preference gradient launch");
    }
    return MUON_OK;
} MUON_CATCH_ALL
