// Dropout whose mask is a function of the element's index, a seed and an
// offset, and is never stored: y = residual + x m / (1 - p).
//
// Random bits: the Philox4x32 generator with ten rounds (J. Salmon, M. Moraes,
// R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).  Key:
// the seed; counter: the index of an eight-element block (64 bits) and the offset
// (64 bits).  The 128 bits of a counter are eight numbers of 16 bits, one for
// each element, so p counts in steps of 2^-16; an element stays where its number
// is at least p 65536.  32 bits each would double the generator's work, which at
// 16 bits hides under the copies: 67 M bf16 elements onto a residual (403 MB) 58 us, at
// the copy rate; without one (268 MB) 45 us, 0.89 of it, the generator's multiplications
// showing.  One block per thread and step with the key's steps taken for each, the type
// chosen per access, was 95 us.  Tensors off 16 bytes go by elements, 16 bytes apart from
// lane to lane: the same elements 128 us with or without a residual (fp32 179 and 200; on 16
// bytes 76 and 113).
#include "host.h"
#include "epilogue.cuh"

namespace muon {

namespace {

constexpr int DT = 256;

struct DropArgs {
    const void* x;
    const void* add;            // residual or null
    void* y;
    int64_t n;
    const int64_t* state;       // device {seed, offset}, or null: the two below
    uint64_t seed, offset;
    uint32_t cut;               // p 65536, in the upper half of a word
    float scale;
    int dtype;
};

// Eight 16-bit numbers of each of two blocks, two to a word, the even element in
// the low half.
__device__ __forceinline__ void philox2(uint64_t b0, uint64_t b1, uint64_t seed, uint64_t offset, uint4& r0, uint4& r1) {
    uint32_t c[2][4] = {{(uint32_t)b0, (uint32_t)(b0 >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)},
                        {(uint32_t)b1, (uint32_t)(b1 >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)}};
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint64_t p = (uint64_t)0xD2511F53u * c[j][0], q = (uint64_t)0xCD9E8D57u * c[j][2];
            c[j][0] = (uint32_t)(q >> 32) ^ c[j][1] ^ k0;
            c[j][2] = (uint32_t)(p >> 32) ^ c[j][3] ^ k1;
            c[j][1] = (uint32_t)q;
            c[j][3] = (uint32_t)p;
        }
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    r0 = make_uint4(c[0][0], c[0][1], c[0][2], c[0][3]);
    r1 = make_uint4(c[1][0], c[1][1], c[1][2], c[1][3]);
}

// Eight elements from their 16-byte pieces (one, of fp32 two) and back.
template <int DTYPE>
__device__ __forceinline__ void load8(const void* p, int64_t b, float (&v)[8]) {
    const uint4* q = static_cast<const uint4*>(p);
    if constexpr (DTYPE == MUON_F32) {
        const uint4 lo = q[2 * b], hi = q[2 * b + 1];
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
    } else {
        unpack8_h(q[b], v, DTYPE == MUON_F16);
    }
}

template <int DTYPE>
__device__ __forceinline__ void store8(void* p, int64_t b, const float (&v)[8]) {
    uint4* q = static_cast<uint4*>(p);
    if constexpr (DTYPE == MUON_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            q[2 * b + h] = make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                                      __float_as_uint(v[4 * h + 3]));
    } else {
        q[b] = pack8_h(v, DTYPE == MUON_F16);
    }
}

// A dropped element is 0 whatever it was (infinities and NaN too).  A word holds
// two numbers; compared with cut << 16 the upper one needs no shift.
template <bool ADD>
__device__ __forceinline__ void drop8(const DropArgs& a, const uint4& bits, float (&x)[8], const float (&add)[8]) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t r = k & 1 ? w[k / 2] : w[k / 2] << 16;
        x[k] = r >= a.cut ? (ADD ? fmaf(x[k], a.scale, add[k]) : x[k] * a.scale) : (ADD ? add[k] : 0.f);
    }
}

template <int DTYPE, bool VEC, bool ADD>
__global__ void __launch_bounds__(DT) dropout_kernel(const __grid_constant__ DropArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint64_t seed = a.state ? (uint64_t)a.state[0] : a.seed, offset = a.state ? (uint64_t)a.state[1] : a.offset;
    const int64_t blocks = (a.n + 7) / 8, whole = VEC ? a.n / 8 : 0;
    // two blocks per thread, 256 apart: their loads leave together, and the key's
    // ten steps are taken once
    int64_t b = (int64_t)blockIdx.x * 2 * DT + threadIdx.x;
    const int64_t end = min(blocks, ((int64_t)blockIdx.x + 1) * 2 * DT);
    float x[8], add[8];
    if (b + DT < whole) {
        float x2[8], add2[8];
        load8<DTYPE>(a.x, b, x);
        load8<DTYPE>(a.x, b + DT, x2);
        if (ADD) {
            load8<DTYPE>(a.add, b, add);
            load8<DTYPE>(a.add, b + DT, add2);
        }
        uint4 r, r2;
        philox2((uint64_t)b, (uint64_t)b + DT, seed, offset, r, r2);
        drop8<ADD>(a, r, x, add);
        drop8<ADD>(a, r2, x2, add2);
        store8<DTYPE>(a.y, b, x);
        store8<DTYPE>(a.y, b + DT, x2);
        return;
    }
    // the last blocks, and elements that are no aligned pieces
#pragma unroll 1
    for (; b < end; b += DT) {
        const int n = (int)min((int64_t)8, a.n - 8 * b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = k < n ? ld_elem(a.x, 8 * b + k, DTYPE) : 0.f;
            add[k] = ADD && k < n ? ld_elem(a.add, 8 * b + k, DTYPE) : 0.f;
        }
        uint4 bits, unused;
        philox2((uint64_t)b, (uint64_t)b, seed, offset, bits, unused);
        drop8<ADD>(a, bits, x, add);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) st_elem(a.y, 8 * b + k, x[k], DTYPE);
    }
}

template <int DTYPE>
auto dropout_form(bool vec, bool add) {
    return vec ? (add ? dropout_kernel<DTYPE, true, true> : dropout_kernel<DTYPE, true, false>)
               : (add ? dropout_kernel<DTYPE, false, true> : dropout_kernel<DTYPE, false, false>);
}

// p = 1: the residual, or zeros.
int drop_all(const void* residual, void* y, size_t bytes, cudaStream_t s) {
    if (!residual) MUON_CUDA(cudaMemsetAsync(y, 0, bytes, s));
    else if (residual != y) MUON_CUDA(cudaMemcpyAsync(y, residual, bytes, cudaMemcpyDeviceToDevice, s));
    return MUON_OK;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" int muon_dropout(const void* x, const void* residual, void* y, int64_t n, int dtype, double p,
                            int64_t seed, int64_t offset, const int64_t* state, void* stream) try {
    if (!valid_dtype(dtype)) return fail(MUON_EDTYPE, "dtype %d", dtype);
    if (n < 0 || n > ((int64_t)1 << 40)) return fail(MUON_EINVAL, "n outside [0, 2^40]");
    if (!(p >= 0.0 && p <= 1.0)) return fail(MUON_EINVAL, "p outside [0, 1]");
    if (n == 0) return MUON_OK;
    if (!x || !y) return fail(MUON_EINVAL, "NULL argument");
    for (const void* q : {x, residual, (const void*)y})
        if (reinterpret_cast<uintptr_t>(q) & (esize(dtype) - 1)) return fail(MUON_EINVAL, "pointer not aligned to its element");
    if (reinterpret_cast<uintptr_t>(state) & 7) return fail(MUON_EINVAL, "pointer not aligned to its element");
    DevCtx dc;
    int r = get_dev(dc);
    if (r) return r;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    DropArgs a;
    a.x = x; a.add = residual; a.y = y; a.n = n; a.dtype = dtype;
    a.state = state;
    a.seed = (uint64_t)seed; a.offset = (uint64_t)offset;
    const double cut = std::floor(p * 65536.0 + 0.5);
    if (cut >= 65536.0) return drop_all(residual, y, (size_t)n * esize(dtype), s);
    a.cut = (uint32_t)cut << 16;
    a.scale = (float)(65536.0 / (65536.0 - cut));
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(y)) & 15) == 0;
    const int64_t ctas = ((n + 7) / 8 + 2 * DT - 1) / (2 * DT);
    auto kern = dtype == MUON_F32    ? dropout_form<MUON_F32>(vec, residual != nullptr)
                : dtype == MUON_BF16 ? dropout_form<MUON_BF16>(vec, residual != nullptr)
                                     : dropout_form<MUON_F16>(vec, residual != nullptr);
    note_launch_begin(KC_OTHER, s);
    const cudaError_t e = launch_pdl(kern,
                                     dim3((unsigned)ctas), dim3(DT), 0, s, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "dropout launch");
} MUON_CATCH_ALL
