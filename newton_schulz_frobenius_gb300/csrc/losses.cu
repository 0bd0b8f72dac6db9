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

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

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
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) { return pack8_h(v, false); }
};
template <>
struct Vec<__half> {
    static constexpr int E = 8;
    static __device__ __forceinline__ float ld(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ void st(__half* p, float v) { *p = __float2half_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&v)[8]) { unpack8_h(q, v, true); }
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
__device__ __forceinline__ void load_vec(const T* row, int v0, int vocab, float (&x)[Vec<T>::E]) {
    constexpr int E = Vec<T>::E;
    if (v0 >= 0 && v0 + E <= vocab) {
        Vec<T>::unpack(*reinterpret_cast<const uint4*>(row + v0), x);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = (v0 + j >= 0 && v0 + j < vocab) ? Vec<T>::ld(row + v0 + j) : -INFINITY;
    }
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

constexpr int LT = 512;         // threads of a row
constexpr int LNW = LT / 32;

// Two walks over the row, one CTA per row: first the online maximum and sum,
// then the gradient.
template <typename T, int MODE>
__global__ void __launch_bounds__(LT) row_loss_kernel(const __grid_constant__ RowLossArgs a) {
    constexpr int E = Vec<T>::E;
    extern __shared__ uint32_t dyn[];       // distillation: bitmap of S, then indices and p
    __shared__ float red[LNW];
    pdl_wait();
    pdl_trigger();
    const int V = a.vocab;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld;
        T* g = reinterpret_cast<T*>(a.grad) + row * a.ldg;
        const float w = a.weights ? a.weights[row] : 1.0f;
        int64_t tok = 0;
        bool live = (w != 0.f);
        if (MODE != LM_DISTILL) {
            tok = ld_index(a.tokens, row, a.tok64);
            live = live && tok >= 0 && tok < V;
        }
        if (!live) {
            if (MODE != LM_STATS) zero_row<T, LT>(g, V);
            if (threadIdx.x == 0) {
                if (MODE == LM_STATS) a.stats[row] = RowStats{0.f, 0.f, 0.f, 0.f};
                else a.loss[row] = 0.f;
                if (MODE == LM_POLICY) a.logp[row] = 0.f;
            }
            continue;
        }
        const int shift = row_shift(x);
        const int nv = (V + shift + E - 1) / E;
        // teacher's set
        const int words = (V + 31) / 32;
        uint32_t* bits = dyn;
        int* sidx = reinterpret_cast<int*>(dyn + words);
        float* sp = reinterpret_cast<float*>(sidx + a.k);
        float mass = 0.f, tsub = 0.f;       // sum of p; log p_j = t_j / T - tsub
        if (MODE == LM_DISTILL) {
            __syncthreads();
            for (int i = threadIdx.x; i < words; i += LT) bits[i] = 0;
            __syncthreads();
            float tm = -INFINITY;
            for (int j = threadIdx.x; j < a.k; j += LT) {
                const int64_t id = ld_index(a.tidx, row * a.k + j, a.tidx64);
                const bool ok = id >= 0 && id < V;
                const float t = ld_elem(a.tval, row * a.k + j, a.tval_dtype);
                sidx[j] = ok ? (int)id : -1;
                sp[j] = t;
                if (ok) {
                    atomicOr(&bits[id >> 5], 1u << (id & 31));
                    tm = fmaxf(tm, t);
                }
            }
            if (a.tlse) {
                tm = 0.f;
                tsub = a.tlse[row];
            } else {
                tm = block_max<LNW>(tm, red);
                float s = 0.f;
                for (int j = threadIdx.x; j < a.k; j += LT)
                    if (sidx[j] >= 0) s += expf((sp[j] - tm) * a.inv_t);
                tsub = ::logf(block_sum<LNW>(s, red));
            }
            // sp[j] becomes log p_j (entries that are not in the vocabulary drop out)
            float s = 0.f;
            for (int j = threadIdx.x; j < a.k; j += LT) {
                const float lp = sidx[j] >= 0 ? (sp[j] - tm) * a.inv_t - tsub : -INFINITY;
                sp[j] = lp;
                s += expf(lp);
            }
            mass = block_sum<LNW>(s, red);
        }
        // maximum and sums
        float m = -INFINITY;
        for (int i = threadIdx.x; i < nv; i += LT) {
            float v[E];
            load_vec<T>(x, i * E - shift, V, v);
#pragma unroll
            for (int j = 0; j < E; ++j) m = fmaxf(m, v[j]);
        }
        m = block_max<LNW>(m, red);
        float s = 0.f, so = 0.f;
        for (int i = threadIdx.x; i < nv; i += LT) {
            const int v0 = i * E - shift;
            float v[E];
            load_vec<T>(x, v0, V, v);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float e = (v0 + j >= 0 && v0 + j < V) ? exp2f((v[j] - m) * a.c2) : 0.f;
                s += e;
                if (MODE == LM_DISTILL && v0 + j >= 0 && v0 + j < V && !((bits[(v0 + j) >> 5] >> ((v0 + j) & 31)) & 1))
                    so += e;
            }
        }
        s = block_sum<LNW>(s, red);
        const float log_s = ::logf(s);
        const float inv_s = 1.0f / s;
        float in = 0.f, out = 0.f;          // factors of q inside and outside S
        float scale = 0.f;                  // factor of t
        if (MODE != LM_DISTILL) {
            const float lp = (Vec<T>::ld(x + tok) - m) * a.inv_t - log_s;
            if (MODE == LM_STATS) {
                if (threadIdx.x == 0) a.stats[row] = RowStats{m, inv_s, lp, 0.f};
                continue;
            }
            float loss, dl;
            policy_row(a, row, lp, loss, dl);
            if (threadIdx.x == 0) {
                a.loss[row] = w * loss;
                a.logp[row] = lp;
            }
            scale = w * dl * a.inv_t;
            in = out = -scale;
        } else {
            float rest = 0.f, share = 0.f, kl = 0.f;
            if (a.tlse) {
                const float qr = block_sum<LNW>(so, red) * inv_s;
                rest = 1.0f - mass;
                if (!(rest > 0.f && qr > 0.f)) rest = 0.f;
                else {
                    share = rest / qr;
                    kl = rest * ::logf(share);
                }
            }
            float part = 0.f;
            for (int j = threadIdx.x; j < a.k; j += LT) {
                const float lp = sp[j];
                const float p = expf(lp);
                if (p > 0.f) part += p * (lp - ((Vec<T>::ld(x + sidx[j]) - m) * a.inv_t - log_s));
                else if (p != p) part = p;
                sp[j] = p;
            }
            kl += block_sum<LNW>(part, red);        // also orders the gathers before the gradient's stores
            if (threadIdx.x == 0) a.loss[row] = w * a.t * a.t * kl;
            scale = w * a.t;
            in = scale * (mass + rest);
            out = scale * (mass + rest - share);
        }
        __syncthreads();
        // gradient
        for (int i = threadIdx.x; i < nv; i += LT) {
            const int v0 = i * E - shift;
            float v[E];
            load_vec<T>(x, v0, V, v);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int id = v0 + j;
                const float q = exp2f((v[j] - m) * a.c2) * inv_s;
                if (MODE == LM_POLICY) {
                    v[j] = in * q + (id == (int)tok ? scale : 0.f);
                } else if (id >= 0 && id < V && ((bits[id >> 5] >> (id & 31)) & 1)) {
                    float p = 0.f;          // an index the teacher lists twice counts twice
                    for (int n = 0; n < a.k; ++n)
                        if (sidx[n] == id) p += sp[n];
                    v[j] = in * q - scale * p;
                } else {
                    v[j] = out * q;
                }
            }
            store_vec<T>(g, v0, V, v, a.same_align != 0);
        }
    }
}

// Gradient rows of the preference loss: coef ([v = token] - q_v).
template <typename T>
__global__ void __launch_bounds__(LT) row_grad_kernel(const __grid_constant__ RowLossArgs a) {
    constexpr int E = Vec<T>::E;
    pdl_wait();
    pdl_trigger();
    const int V = a.vocab;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld;
        T* g = reinterpret_cast<T*>(a.grad) + row * a.ldg;
        const RowStats st = a.stats[row];
        if (st.coef == 0.f) {
            zero_row<T, LT>(g, V);
            continue;
        }
        const int tok = (int)ld_index(a.tokens, row, a.tok64);
        const int shift = row_shift(x);
        const int nv = (V + shift + E - 1) / E;
        const float f = -st.coef * st.inv_s;
        for (int i = threadIdx.x; i < nv; i += LT) {
            const int v0 = i * E - shift;
            float v[E];
            load_vec<T>(x, v0, V, v);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = fmaf(f, exp2f((v[j] - st.mx) * a.c2), v0 + j == tok ? st.coef : 0.f);
            store_vec<T>(g, v0, V, v, a.same_align != 0);
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

constexpr int64_t MAX_VOCAB = 1 << 20;
constexpr int MAX_TEACHER = 1024;

size_t distill_smem(int vocab, int k) { return 4 * ((size_t)(vocab + 31) / 32 + 2 * (size_t)k); }

template <typename T>
cudaError_t launch_rows(const RowLossArgs& a, int mode, int sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(a.rows, (int64_t)sms * 4);
    if (mode == LM_POLICY) return launch_pdl(row_loss_kernel<T, LM_POLICY>, dim3(grid), dim3(LT), 0, s, a);
    if (mode == LM_STATS) return launch_pdl(row_loss_kernel<T, LM_STATS>, dim3(grid), dim3(LT), 0, s, a);
    const size_t smem = distill_smem(a.vocab, a.k);
    cudaError_t e = cudaFuncSetAttribute(row_loss_kernel<T, LM_DISTILL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)distill_smem((int)MAX_VOCAB, MAX_TEACHER));
    if (e != cudaSuccess) return e;
    return launch_pdl(row_loss_kernel<T, LM_DISTILL>, dim3(grid), dim3(LT), smem, s, a);
}

template <typename T>
cudaError_t launch_grad(const RowLossArgs& a, int sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(a.rows, (int64_t)sms * 4);
    return launch_pdl(row_grad_kernel<T>, dim3(grid), dim3(LT), 0, s, a);
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
    if (vocab < 1 || vocab > MAX_VOCAB) return fail(MUON_EINVAL, "vocab outside [1, 2^20]");
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
