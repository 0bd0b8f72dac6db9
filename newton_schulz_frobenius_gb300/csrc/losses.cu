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

namespace muon {

namespace {

enum LossMode : int { LM_POLICY = 0, LM_DISTILL = 1, LM_STATS = 2 };

struct RowStats {       // one row of the preference loss between its launches
    float mx, inv_s;    // q_v = exp2((x_v - mx) c2) * inv_s
    float logp;
    float coef;         // d loss / d logp, 0 for rows outside the loss
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

// A row is walked in 16-byte vectors aligned in memory: vector i holds the
// elements E i - shift .. E i - shift + E - 1, where shift is how many elements
// the row starts after a 16-byte boundary (odd vocabularies, sliced heads).
// Elements outside [0, V) are never touched; they read as -inf.
template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int v0, int vocab) {
    constexpr int E = Vec<T>::E;
    if (v0 >= 0 && v0 + E <= vocab) return *reinterpret_cast<const uint4*>(row + v0);
    float x[E];
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = (v0 + j >= 0 && v0 + j < vocab) ? Vec<T>::ld(row + v0 + j) : -INFINITY;
    return Vec<T>::pack(x);
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int v0, int vocab, const float (&x)[Vec<T>::E], bool aligned) {
    constexpr int E = Vec<T>::E;
    if (aligned && v0 >= 0 && v0 + E <= vocab) {
        *reinterpret_cast<uint4*>(row + v0) = Vec<T>::pack(x);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (v0 + j >= 0 && v0 + j < vocab) Vec<T>::st(row + v0 + j, x[j]);
    }
}

template <int NW>
__device__ __forceinline__ float block_sum(float v, float* red) {
    __syncthreads();            // red may still be read from the previous reduction
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += red[i];
    return s;
}

template <int NW>
__device__ __forceinline__ float block_max(float v, float* red) {
    __syncthreads();
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) s = fmaxf(s, red[i]);
    return s;
}

template <typename T, int NT>
__device__ __forceinline__ void zero_row(T* row, int vocab) {
    constexpr int E = Vec<T>::E;
    const int shift = row_shift(row);
    const int nv = (vocab + shift + E - 1) / E;
    float z[E];
#pragma unroll
    for (int j = 0; j < E; ++j) z[j] = 0.f;
    for (int i = threadIdx.x; i < nv; i += NT) store_vec<T>(row, i * E - shift, vocab, z, true);
}

// The policy loss of one row from its log-probability: loss and dL/dlogp.
__device__ __forceinline__ void policy_row(const RowLossArgs& a, int64_t row, float lp, float& loss, float& dl) {
    const float adv = a.adv[row];
    const float r = a.old_logp ? expf(lp - a.old_logp[row]) : 1.0f;
    const float rc = fminf(fmaxf(r, a.lo), a.hi);
    const float u = r * adv, uc = rc * adv;
    loss = -fminf(u, uc);
    dl = (u <= uc || u != u) ? -u : 0.f;
    if (a.kl != 0.f) {
        const float x = a.ref_logp[row] - lp;
        // exp(x) - x - 1 cancels for small x: expm1 keeps it
        const float em = expm1f(x);
        loss += a.kl * (em - x);
        dl -= a.kl * em;
    }
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

// v <- exp2((v + nr) c2), two values per add and multiply; returns their sum.
template <int E>
__device__ __forceinline__ float exp_vec(float (&v)[E], float nr, float c2) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        asm("{\n\t.reg .b64 x, r, c;\n\t"
            "mov.b64 x, {%0, %1};\n\tmov.b64 r, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
            "add.rn.f32x2 x, x, r;\n\tmul.rn.f32x2 x, x, c;\n\t"
            "mov.b64 {%0, %1}, x;\n\t}"
            : "+f"(v[j]), "+f"(v[j + 1])
            : "f"(nr), "f"(c2));
        v[j] = ex2(v[j]);
        v[j + 1] = ex2(v[j + 1]);
        asm("{\n\t.reg .b64 s, x;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\t"
            "add.rn.f32x2 s, s, x;\n\tmov.b64 {%0, %1}, s;\n\t}"
            : "+f"(s.x), "+f"(s.y)
            : "f"(v[j]), "f"(v[j + 1]));
    }
    return s.x + s.y;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster; orders shared and global accesses before and after.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_f4(uint32_t local, uint32_t rank, const float4& v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// ---------------------------------------------------------------------------
// one reading: the row rests in shared memory between its two walks
// ---------------------------------------------------------------------------
//
// A row belongs to a cluster of C CTAs (C = 1 up to 53248 16-bit logits), CTA r
// holding its r-th part in shared memory, SLOTS x NT vectors of 16 bytes at
// most, two CTAs per SM.  The first walk takes the maximum and the sums, the
// CTAs of a cluster exchange theirs through distributed shared memory, and the
// second walk takes the exponentials again (cheaper than the registers to keep
// them in) and stores the gradient, so every logit is read from memory once.
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
    float s, so;            // sum of exponentials, the part outside the teacher's set
    float top;              // the maximum
};

__device__ __forceinline__ void follow(Sums& z, float vm, float c2, float step) {
    z.top = fmaxf(z.top, vm);
    if (vm > z.limit) {
        const float f = z.limit == -INFINITY ? 1.0f : ex2((-z.ref - vm) * c2);
        z.s *= f;
        z.so *= f;
        z.ref = -vm;
        z.limit = vm + step;
    }
}

// Partial sums of a warp's lanes, one per lane (maximum, s, so), as one.
__device__ __forceinline__ float3 merge_lanes(float top, float s, float so, float c2, bool rest) {
    float3 r;
    r.x = warp_max(top);
    const float f = top == -INFINITY ? 0.f : ex2((top - r.x) * c2);     // 0 x NaN stays NaN
    r.y = warp_sum(s * f);
    r.z = rest ? warp_sum(so * f) : 0.f;
    return r;
}

// Which of the cluster's next 32 rows are in the loss, refreshed every 32 rows.
struct LiveWindow {
    uint32_t bits;
    int n;                  // rows of the cluster's sequence already taken from it
};

__host__ __device__ constexpr int bit_words(int logits) { return (logits + 31) / 32; }

struct PartArgs {
    int csize;              // CTAs per row
    int per;                // vectors of a row per CTA, at most SLOTS NT
};

template <typename T, int MODE, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT)
row_loss_kernel(const __grid_constant__ RowLossArgs a, const __grid_constant__ PartArgs pa) {
    constexpr int E = Vec<T>::E, NW = NT / 32, QUARTERS = 4;
    constexpr bool GRAD = MODE != LM_STATS;
    extern __shared__ __align__(16) uint8_t dyn8[];
    uint4* ring = reinterpret_cast<uint4*>(dyn8);       // [slots][NT]
    __shared__ float4 red[2][NW];
    __shared__ float4 part[2][MAX_CLUSTER];
    __shared__ float tred[NW], tred_m[NW], lred[NW];
    const int V = a.vocab, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int csize = pa.csize, per = pa.per;
    const int rank = csize > 1 ? (int)cluster_rank() : 0;
    const int64_t G = gridDim.x / csize, row0 = blockIdx.x / csize;
    const int slots = (per + NT - 1) / NT, quarter = (slots + QUARTERS - 1) / QUARTERS;
    const float c2 = a.c2, step = REBASE / c2;
    // distillation: the teacher's entries; with a remainder class, the bitmap of its set in this part
    int* sidx = reinterpret_cast<int*>(dyn8 + (size_t)slots * NT * 16);
    float* slp = reinterpret_cast<float*>(sidx + a.k);
    float* sp = slp + a.k;
    float* sx = sp + a.k;
    uint32_t* bits = reinterpret_cast<uint32_t*>(sx + a.k);
    const bool rest_class = MODE == LM_DISTILL && a.tlse != nullptr;
    pdl_wait();
    pdl_trigger();
    if (rest_class)
        for (int i = t; i < bit_words(per * E); i += NT) bits[i] = 0;
    if (csize > 1) cluster_barrier();                   // every CTA of the cluster runs before any writes to it

    auto row_live = [&](int64_t row) -> bool {
        if (row >= a.rows) return false;
        bool live = !a.weights || a.weights[row] != 0.f;
        if (MODE != LM_DISTILL) {
            const int64_t tok = ld_index(a.tokens, row, a.tok64);
            live = live && tok >= 0 && tok < V;
        }
        return live;
    };
    auto window = [&](LiveWindow& w, int64_t row) -> bool {     // whether `row`, the sequence's next, is live
        if ((w.n & 31) == 0) w.bits = __ballot_sync(0xffffffffu, row_live(row + (int64_t)lane * G));
        return (w.bits >> (w.n++ & 31)) & 1;
    };
    // geometry of a row: logits before its first vector, vectors of this CTA
    auto head_of = [&](const T* x) { return min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T)); };
    auto count_of = [&](int head) { return max(0, min(per, (V - head) / E - rank * per)); };
    // this thread's odd logit of a row (the first CTA's threads), -1 if none
    auto odd_of = [&](int head) -> int {
        if (rank != 0 || t >= 2 * E) return -1;
        if (t < head) return t;
        const int at = head + (V - head) / E * E + (t - head);
        return at < V ? at : -1;
    };

    // the row in the loss after the one worked on: its vectors are copied in as slots fall free
    LiveWindow lw{0, 0}, pw{0, 0};
    int64_t lrow = row0;
    const T* lx = nullptr;
    const T* lp = nullptr;                              // this thread's first vector of it
    int lcount = 0;                                     // the CTA's vectors of it
    float lodd = -INFINITY;                             // this thread's odd logit of it
    auto advance = [&]() {
        while (lrow < a.rows && !window(lw, lrow)) lrow += G;
        lcount = 0;
        lodd = -INFINITY;
        if (lrow < a.rows) {
            lx = reinterpret_cast<const T*>(a.logits) + lrow * a.ld;
            const int head = head_of(lx);
            lcount = count_of(head);
            lp = lx + head + (int64_t)(rank * per + t) * E;
            const int odd = odd_of(head);
            if (odd >= 0) lodd = Vec<T>::ld(lx + odd);
        }
    };
    const uint32_t slot0 = smem_addr(ring + t);
    auto issue = [&](int u) {
        if (t + u * NT < lcount) cp_async16(slot0 + u * (NT * 16), lp + u * (NT * E));
    };
    advance();
#pragma unroll
    for (int qd = 0; qd < QUARTERS; ++qd) {
        for (int u = qd * quarter; u < min(slots, (qd + 1) * quarter); ++u) issue(u);
        cp_async_commit();
    }

    int par = 0;
    for (int64_t row = row0; row < a.rows; row += G) {
        T* g = reinterpret_cast<T*>(a.grad) + row * a.ldg;
        if (!window(pw, row)) {
            if (GRAD) {
                const int head = head_of(g), n = count_of(head), odd = odd_of(head);
                T* gp = g + head + (int64_t)rank * per * E;
                for (int i = t; i < n; i += NT) *reinterpret_cast<uint4*>(gp + i * E) = make_uint4(0, 0, 0, 0);
                if (odd >= 0) Vec<T>::st(g + odd, 0.f);
            }
            if (rank == 0 && t == 0) {
                if (MODE == LM_STATS) a.stats[row] = RowStats{0.f, 0.f, 0.f, 0.f};
                else a.loss[row] = 0.f;
                if (MODE == LM_POLICY) a.logp[row] = 0.f;
            }
            continue;
        }
        const T* x = lx;                    // the row whose vectors are in the ring
        const int head = head_of(x), count = lcount;
        const float odd = lodd;
        const float w = a.weights ? a.weights[row] : 1.0f;
        int tok = 0;
        float xt = 0.f;
        if (MODE != LM_DISTILL) {
            tok = (int)ld_index(a.tokens, row, a.tok64);
            xt = Vec<T>::ld(x + tok);
        }
        float tm = 0.f, lse = 0.f;
        const int part0 = head + rank * per * E;        // the part's first logit; its bit is 0
        bool odd_in = false;                            // the thread's odd logit is in the teacher's set
        if (MODE == LM_DISTILL) {
            lse = a.tlse ? a.tlse[row] : 0.f;
            __syncthreads();                // the previous row's use of the entries is over
            float wm = -INFINITY;
            for (int j = t; j < a.k; j += NT) {
                const int64_t id = ld_index(a.tidx, row * a.k + j, a.tidx64);
                const bool ok = id >= 0 && id < V;
                const float tv = ok ? ld_elem(a.tval, row * a.k + j, a.tval_dtype) : -INFINITY;
                sidx[j] = ok ? (int)id : -1;
                slp[j] = tv;
                sx[j] = ok ? Vec<T>::ld(x + id) : 0.f;
                const int at = (int)id - part0;
                if (ok && rest_class && at >= 0 && at < count * E) atomicOr(&bits[at >> 5], 1u << (at & 31));
                wm = fmaxf(wm, tv);
            }
            wm = warp_max(wm);
            if (lane == 0) tred_m[warp] = wm;
            __syncthreads();
            if (!a.tlse) tm = warp_max(lane < NW ? tred_m[lane] : -INFINITY);
            float s = 0.f;
            for (int j = t; j < a.k; j += NT)
                if (sidx[j] >= 0) s += expf((slp[j] - tm) * a.inv_t - lse);
            s = warp_sum(s);
            if (lane == 0) tred[warp] = s;
            if (rest_class && odd_of(head) >= 0)
                for (int j = 0; j < a.k; ++j) odd_in = odd_in || sidx[j] == odd_of(head);
        }
        lrow += G;
        advance();
        // first walk
        Sums z{0.f, -INFINITY, 0.f, 0.f, -INFINITY};
#pragma unroll
        for (int qd = 0; qd < QUARTERS; ++qd) {
            // pending behind this quarter: the row's later ones, and (statistics) the next row's earlier ones
            if (!GRAD || qd == 0) cp_async_wait<3>();
            else if (qd == 1) cp_async_wait<2>();
            else if (qd == 2) cp_async_wait<1>();
            else cp_async_wait<0>();
            const int end = min(slots, (qd + 1) * quarter);
#pragma unroll 2
            for (int u = qd * quarter; u < end; ++u) {
                if (t + u * NT < count) {
                    const uint4 raw = ring[u * NT + t];
                    follow(z, Vec<T>::vmax(raw), c2, step);
                    float v[E];
                    Vec<T>::unpack(raw, v);
                    const float sv = exp_vec<E>(v, z.ref, c2);
                    z.s += sv;
                    if (rest_class) {
                        const int i = (t + u * NT) * E;
                        const uint32_t k = (bits[i >> 5] >> (i & 31)) & ((1u << E) - 1);
                        if (k == 0) {
                            z.so += sv;
                        } else {
#pragma unroll
                            for (int j = 0; j < E; ++j)
                                if (!((k >> j) & 1)) z.so += v[j];
                        }
                    }
                }
                if (!GRAD) issue(u);
            }
            if (!GRAD) cp_async_commit();
        }
        if (t < 2 * E) {
            follow(z, odd, c2, step);
            const float e = ex2((odd + z.ref) * c2);
            z.s += e;
            if (!odd_in) z.so += e;
        }
        float3 q;
        {
            const float wm = warp_max(z.top);
            const float f = z.limit == -INFINITY ? 0.f : ex2((-z.ref - wm) * c2);
            const float s = warp_sum(z.s * f);
            const float so = rest_class ? warp_sum(z.so * f) : 0.f;
            if (lane == 0) red[par][warp] = make_float4(wm, s, so, 0.f);
            __syncthreads();
            const float4 r = lane < NW ? red[par][lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            if (csize == 1) {
                q = merge_lanes(r.x, r.y, r.z, c2, rest_class);
            } else {
                if (warp == 0) {
                    q = merge_lanes(r.x, r.y, r.z, c2, rest_class);
                    if (t < csize) st_cluster_f4(smem_addr(&part[par][rank]), (uint32_t)t, make_float4(q.x, q.y, q.z, 0.f));
                }
                cluster_barrier();
                const float4 c = lane < csize ? part[par][lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
                q = merge_lanes(c.x, c.y, c.z, c2, rest_class);
            }
        }
        par ^= 1;
        const float m = q.x, log_s = ::logf(q.y), inv_s = 1.0f / q.y;
        float in = 0.f, out = 0.f;          // factors of q inside and outside S
        float scale = 0.f;                  // factor of the sparse part
        if (MODE == LM_STATS) {
            if (rank == 0 && t == 0) a.stats[row] = RowStats{m, inv_s, (xt - m) * a.inv_t - log_s, 0.f};
            continue;
        } else if (MODE == LM_POLICY) {
            const float lp_tok = (xt - m) * a.inv_t - log_s;
            float loss, dl;
            policy_row(a, row, lp_tok, loss, dl);
            if (rank == 0 && t == 0) {
                a.loss[row] = w * loss;
                a.logp[row] = lp_tok;
            }
            scale = w * dl * a.inv_t;
            out = -scale * inv_s;
        } else {
            const float ts = warp_sum(lane < NW ? tred[lane] : 0.f);
            const float mass = a.tlse ? ts : (ts > 0.f || ts != ts ? 1.0f : 0.f);
            const float tsub = a.tlse ? lse : ::logf(ts);
            float rest = 0.f, share = 0.f, kl = 0.f;
            if (a.tlse) {
                const float qr = q.z * inv_s;
                rest = 1.0f - mass;
                if (!(rest > 0.f && qr > 0.f)) rest = 0.f;
                else {
                    share = rest / qr;
                    kl = rest * ::logf(share);
                }
            }
            float part_kl = 0.f;
            for (int j = t; j < a.k; j += NT) {
                const float lpj = sidx[j] >= 0 ? (slp[j] - tm) * a.inv_t - tsub : -INFINITY;
                const float p = expf(lpj);
                sp[j] = p;
                if (p > 0.f) part_kl += p * (lpj - ((sx[j] - m) * a.inv_t - log_s));
                else if (p != p) part_kl = p;
            }
            part_kl = warp_sum(part_kl);
            if (lane == 0) lred[warp] = part_kl;
            scale = w * a.t;
            in = scale * (mass + rest) * inv_s;
            out = scale * (mass + rest - share) * inv_s;
            __syncthreads();
            if (rank == 0 && warp == 0) {
                part_kl = warp_sum(lane < NW ? lred[lane] : 0.f);
                if (t == 0) a.loss[row] = w * a.t * a.t * (kl + part_kl);
            }
        }
        // second walk: out q everywhere, the token's entry on the way
        T* gp = g + part0 + t * E;
        const int tok_at = tok - part0;     // within the part's vectors, if there
#pragma unroll
        for (int qd = 0; qd < QUARTERS; ++qd) {
            const int end = min(slots, (qd + 1) * quarter);
#pragma unroll 2
            for (int u = qd * quarter; u < end; ++u) {
                const int i = t + u * NT;
                if (i < count) {
                    float v[E];
                    Vec<T>::unpack(ring[i], v);
                    exp_vec<E>(v, -m, c2);
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] *= out;
                    if (MODE == LM_POLICY && (unsigned)(tok_at - i * E) < (unsigned)E) {
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            if (i * E + j == tok_at) v[j] += scale;
                    }
                    if (a.same_align) {
                        *reinterpret_cast<uint4*>(gp + u * (NT * E)) = Vec<T>::pack(v);
                    } else {
#pragma unroll
                        for (int j = 0; j < E; ++j) Vec<T>::st(gp + u * (NT * E) + j, v[j]);
                    }
                }
                issue(u);
            }
            cp_async_commit();
        }
        if (odd_of(head) >= 0) {
            const int at = odd_of(head);
            Vec<T>::st(g + at, ex2((odd - m) * c2) * out + (MODE == LM_POLICY && at == tok ? scale : 0.f));
        }
        if (MODE == LM_DISTILL) {
            __syncthreads();                // the listed entries' own values go over what the walk stored
            for (int j = t; j < a.k; j += NT) {
                const int id = sidx[j], at = id - part0;
                const bool vec = at >= 0 && at < count * E;
                // an odd logit (before the vectors, or after the row's last) is the first CTA's
                const bool end = rank == 0 && (id < head || id >= head + (V - head) / E * E);
                if (id < 0 || !(vec || end)) continue;
                float psum = 0.f;           // an index the teacher lists twice counts twice
                bool leads = true;
                for (int n = 0; n < a.k; ++n) {
                    if (sidx[n] == id) {
                        psum += sp[n];
                        leads = leads && n >= j;
                    }
                }
                if (leads) Vec<T>::st(g + id, in * ex2((sx[j] - m) * c2) - scale * psum);
                if (rest_class && vec) bits[at >> 5] = 0;
            }
        }
    }
    cp_async_wait<0>();
    if (csize > 1) cluster_barrier();       // no CTA leaves while another may still write to its shared memory
}

constexpr int UNROLL = 4;          // vectors of a gradient row in flight per thread

// Gradient rows of the preference loss: coef ([v = token] - q_v).
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) row_grad_kernel(const __grid_constant__ RowLossArgs a) {
    constexpr int E = Vec<T>::E;
    pdl_wait();
    pdl_trigger();
    const int V = a.vocab;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld;
        T* g = reinterpret_cast<T*>(a.grad) + row * a.ldg;
        const RowStats st = a.stats[row];
        if (st.coef == 0.f) {
            zero_row<T, NT>(g, V);
            continue;
        }
        const int tok = (int)ld_index(a.tokens, row, a.tok64);
        const int shift = row_shift(x);
        const int nv = (V + shift + E - 1) / E;
        const float f = -st.coef * st.inv_s;
        for (int i0 = threadIdx.x; i0 < nv; i0 += UNROLL * NT) {
            uint4 q[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (i0 + u * NT < nv) q[u] = load_vec<T>(x, (i0 + u * NT) * E - shift, V);
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int v0 = (i0 + u * NT) * E - shift;
                if (i0 + u * NT < nv) {
                    float v[E];
                    Vec<T>::unpack(q[u], v);
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = f * ex2((v[j] - st.mx) * a.c2);
                    if ((unsigned)(tok - v0) < (unsigned)E) {
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            if (v0 + j == tok) v[j] += st.coef;
                    }
                    store_vec<T>(g, v0, V, v, a.same_align != 0);
                }
            }
        }
    }
}

struct PairArgs {
    RowStats* stats;
    int64_t rows;
    const void* tokens;
    int tok64, vocab;
    const void* bounds;         // 2 pairs + 1 row offsets
    int bounds64;
    const float* ref_logp;      // per sequence, or null
    const float* weights;       // per pair, or null
    float beta, margin, smoothing;
    int average;
    float* seq_logp;
    float* loss;
};

// One CTA per pair: both sequence values (fp64 sums in a fixed order), the
// pair's loss, and the factor of every row of the pair.
__global__ void __launch_bounds__(256) pair_kernel(const __grid_constant__ PairArgs a) {
    __shared__ double rs[8];
    __shared__ int rn[8];
    pdl_wait();
    pdl_trigger();
    const int64_t pair = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double val[2];
    float share[2];
    int64_t b[3];
    for (int i = 0; i < 3; ++i) {
        int64_t v = ld_index(a.bounds, 2 * pair + i, a.bounds64);
        b[i] = v < 0 ? 0 : (v > a.rows ? a.rows : v);
    }
    for (int c = 0; c < 2; ++c) {
        double s = 0;
        int n = 0;
        for (int64_t r = b[c] + threadIdx.x; r < b[c + 1]; r += 256) {
            const int64_t tok = ld_index(a.tokens, r, a.tok64);
            if (tok >= 0 && tok < a.vocab) {
                s += (double)a.stats[r].logp;
                ++n;
            }
        }
        for (int o = 16; o; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        __syncthreads();
        if (lane == 0) {
            rs[warp] = s;
            rn[warp] = n;
        }
        __syncthreads();
        s = 0;
        n = 0;
        for (int i = 0; i < 8; ++i) {
            s += rs[i];
            n += rn[i];
        }
        share[c] = a.average ? (n > 0 ? 1.0f / (float)n : 0.f) : 1.0f;
        val[c] = a.average ? (n > 0 ? s / n : 0.0) : s;
        if (threadIdx.x == 0) a.seq_logp[2 * pair + c] = (float)val[c];
    }
    double d = val[0] - val[1];
    if (a.ref_logp) d -= (double)a.ref_logp[2 * pair] - (double)a.ref_logp[2 * pair + 1];
    const float h = (float)((double)a.beta * d - (double)a.margin);
    const float w = a.weights ? a.weights[pair] : 1.0f;
    // -log sigmoid(h), and sigmoid(h), sigmoid(-h) without overflow
    const float t = expf(-fabsf(h));
    const float soft = fmaxf(-h, 0.f) + log1pf(t);
    const float big = 1.0f / (1.0f + t), small = t * big;
    const float sp = h >= 0.f ? big : small, sn = h >= 0.f ? small : big;
    float loss = (1.0f - a.smoothing) * soft, dh = -(1.0f - a.smoothing) * sn;
    if (a.smoothing != 0.f) {
        loss += a.smoothing * (soft + h);
        dh += a.smoothing * sp;
    }
    if (h != h) loss = dh = h;
    const bool on = w != 0.f;
    if (threadIdx.x == 0) a.loss[pair] = on ? w * loss : 0.f;
    for (int c = 0; c < 2; ++c) {
        const float coef = on ? (c ? -1.0f : 1.0f) * w * dh * a.beta * share[c] : 0.f;
        for (int64_t r = b[c] + threadIdx.x; r < b[c + 1]; r += 256) {
            const int64_t tok = ld_index(a.tokens, r, a.tok64);
            if (tok >= 0 && tok < a.vocab) a.stats[r].coef = coef;
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t MAX_VOCAB = (int64_t)MAX_CLUSTER * SLOTS * 512 * 4;   // fp32: 425984
constexpr int MAX_TEACHER = 1024;

constexpr int SMALL_NT = 128;           // threads of a CTA whose whole row fits SLOTS x 128 vectors; else 512

// Shared memory of a row's CTA: its part of the row, and for distillation the
// teacher's entries and the bitmap of its set.
template <typename T, int MODE, int NT>
size_t row_smem(int per, int k, bool rest) {
    size_t b = (size_t)((per + NT - 1) / NT) * NT * 16;
    if (MODE == LM_DISTILL) b += 16 * (size_t)k + (rest ? 4 * (size_t)bit_words(per * Vec<T>::E) : 0);
    return b;
}

template <typename T, int MODE, int NT>
cudaError_t launch_part(const RowLossArgs& a, int64_t nv, int csize, cudaStream_t s) {
    auto kern = row_loss_kernel<T, MODE, NT>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [&] {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)row_smem<T, MODE, NT>(SLOTS * NT, MAX_TEACHER, true));
        if (err == cudaSuccess) err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (err != cudaSuccess) return err;
    PartArgs pa;
    pa.csize = csize;
    pa.per = (int)((nv + csize - 1) / csize);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)csize);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = row_smem<T, MODE, NT>(pa.per, a.k, a.tlse != nullptr);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)csize;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    // clusters resident at once, by cluster size and slots
    static std::atomic<int> fits[MAX_CLUSTER + 1][SLOTS + 1];
    std::atomic<int>& fit = fits[csize][(pa.per + NT - 1) / NT];
    int n = fit.load();
    if (n == 0) {
        cfg.attrs = at + 1;
        cfg.numAttrs = 1;
        cudaLaunchConfig_t most = cfg;
        most.dynamicSmemBytes = row_smem<T, MODE, NT>((pa.per + NT - 1) / NT * NT, MODE == LM_DISTILL ? 256 : 0, true);
        cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &most);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        fit.store(n);
    }
    cfg.gridDim = dim3((unsigned)(csize * std::min<int64_t>(a.rows, n)));
    cfg.attrs = pdl_enabled() ? at : at + 1;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, pa);
}

// How a launch divides its rows: 128-thread CTAs for rows of up to 13 x 128
// vectors; else 512-thread CTAs, as few per row as hold it, twice as many while
// the rows alone would leave SMs idle and a CTA keeps two vectors per thread.
template <typename T, int MODE>
cudaError_t launch_mode(const RowLossArgs& a, int sms, cudaStream_t s) {
    constexpr int E = Vec<T>::E;
    const int64_t nv = std::max(1, a.vocab / E);       // whole vectors of a row at most
    if (nv <= SLOTS * SMALL_NT) return launch_part<T, MODE, SMALL_NT>(a, nv, 1, s);
    int c = (int)((nv + SLOTS * 512 - 1) / (SLOTS * 512));
    while (c <= 4 && a.rows * c < sms && nv > (int64_t)c * 1024) c *= 2;
    return launch_part<T, MODE, 512>(a, nv, c, s);
}

template <typename T>
cudaError_t launch_rows(const RowLossArgs& a, int mode, int sms, cudaStream_t s) {
    if (mode == LM_POLICY) return launch_mode<T, LM_POLICY>(a, sms, s);
    if (mode == LM_STATS) return launch_mode<T, LM_STATS>(a, sms, s);
    return launch_mode<T, LM_DISTILL>(a, sms, s);
}

template <typename T>
cudaError_t launch_grad(const RowLossArgs& a, int sms, cudaStream_t s) {
    if (a.vocab <= SMALL_NT * UNROLL * Vec<T>::E)
        return launch_pdl(row_grad_kernel<T, 128>, dim3((unsigned)std::min<int64_t>(a.rows, (int64_t)sms * 8)), dim3(128),
                          0, s, a);
    return launch_pdl(row_grad_kernel<T, 512>, dim3((unsigned)std::min<int64_t>(a.rows, (int64_t)sms * 2)), dim3(512), 0,
                      s, a);
}

cudaError_t dispatch_rows(const RowLossArgs& a, int mode, int dtype, int sms, cudaStream_t s) {
    if (dtype == MUON_F32) return launch_rows<float>(a, mode, sms, s);
    if (dtype == MUON_BF16) return launch_rows<__nv_bfloat16>(a, mode, sms, s);
    return launch_rows<__half>(a, mode, sms, s);
}

cudaError_t dispatch_grad(const RowLossArgs& a, int dtype, int sms, cudaStream_t s) {
    if (dtype == MUON_F32) return launch_grad<float>(a, sms, s);
    if (dtype == MUON_BF16) return launch_grad<__nv_bfloat16>(a, sms, s);
    return launch_grad<__half>(a, sms, s);
}

bool valid_index(int d) { return d == MUON_I32 || d == MUON_I64; }

// The checks every loss makes of its logits and gradient; fills the shared
// fields.  Nothing is enqueued.
int row_args(RowLossArgs& a, const void* logits, int64_t ld, int64_t rows, int64_t vocab, int dtype, float temperature,
             void* grad, int64_t ld_grad) {
    std::memset(&a, 0, sizeof a);
    if (!valid_dtype(dtype)) return fail(MUON_EDTYPE, "logits dtype %d", dtype);
    if (rows < 0 || rows > INT32_MAX) return fail(MUON_EINVAL, "rows outside [0, 2^31)");
    if (vocab < 1 || vocab > MAX_VOCAB) return fail(MUON_EINVAL, "vocab outside [1, %lld]", (long long)MAX_VOCAB);
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
    note_launch_begin(KC_LOSS, s);
    cudaError_t e = dispatch_rows(a, LM_DISTILL, dtype, dc.sms, s);
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
    cudaError_t e = dispatch_rows(a, LM_POLICY, dtype, dc.sms, s);
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
        e = dispatch_rows(a, LM_STATS, dtype, dc.sms, s);
        note_launch_end(KC_LOSS, bytes, s);
        if (e != cudaSuccess) return cuda_fail(e, "preference statistics launch");
    }
    if (pairs > 0) {
        PairArgs p;
        p.stats = a.stats; p.rows = rows;
        p.tokens = tokens; p.tok64 = a.tok64; p.vocab = (int)vocab;
        p.bounds = seq_bounds; p.bounds64 = bounds_dtype == MUON_I64;
        p.ref_logp = ref_logp; p.weights = weights;
        p.beta = beta; p.margin = margin; p.smoothing = label_smoothing; p.average = average != 0;
        p.seq_logp = seq_logp; p.loss = loss;
        note_launch_begin(KC_LOSS, s);
        e = launch_pdl(pair_kernel, dim3((unsigned)pairs), dim3(256), 0, s, p);
        note_launch_end(KC_LOSS, 0.0, s);
        if (e != cudaSuccess) return cuda_fail(e, "preference pair launch");
    }
    if (rows > 0) {
        note_launch_begin(KC_LOSS, s);
        e = dispatch_grad(a, dtype, dc.sms, s);
        note_launch_end(KC_LOSS, 2.0 * bytes, s);
        if (e != cudaSuccess) return cuda_fail(e, "preference gradient launch");
    }
    return MUON_OK;
} MUON_CATCH_ALL
