// Dropout whose mask is a function of the element's index, a seed and an
// offset, and is never stored: y = residual + x m / (1 - p).
//
// Random bits: the Philox4x32 generator with ten rounds (J. Salmon, M. Moraes,
// R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).  Key:
// the seed; counter: the index of an eight-element block (64 bits) and the offset
// (64 bits).  The 128 bits of a counter are eight numbers of 16 bits, one for
// each element, so p counts in steps of 2^-16; an element stays where its number
// is at least p 65536.  32 bits each would double the generator's work, which at
// 16 bits hides under the loads.
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
    uint32_t cut;               // p 65536
    float scale;
    int dtype;
};

// Eight 16-bit numbers of block b, two to a word, the even element in the low half.
__device__ __forceinline__ uint4 philox(uint64_t b, uint64_t seed, uint64_t offset) {
    uint32_t c0 = (uint32_t)b, c1 = (uint32_t)(b >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)q;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// A dropped element is 0 whatever it was (infinities and NaN too).
__device__ __forceinline__ void drop8(const DropArgs& a, const uint4& bits, const float (&x)[8], const float (&add)[8],
                                      float (&y)[8]) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t r = k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xFFFFu;
        y[k] = r >= a.cut ? fmaf(x[k], a.scale, add[k]) : add[k];
    }
}

template <bool VEC>
__global__ void __launch_bounds__(DT) dropout_kernel(const __grid_constant__ DropArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint64_t seed = a.state ? (uint64_t)a.state[0] : a.seed, offset = a.state ? (uint64_t)a.state[1] : a.offset;
    const int64_t blocks = (a.n + 7) / 8, step = (int64_t)gridDim.x * DT;
    for (int64_t b = (int64_t)blockIdx.x * DT + threadIdx.x; b < blocks; b += step) {
        float x[8], add[8], y[8];
        const int n = (int)min((int64_t)8, a.n - 8 * b);
#pragma unroll
        for (int k = 0; k < 8; ++k) add[k] = x[k] = 0.f;
        if (VEC && n == 8) {
            load_row_run<8>(a.x, 8 * b, x, a.dtype);
            if (a.add) load_row_run<8>(a.add, 8 * b, add, a.dtype);
        } else {
            for (int k = 0; k < 8; ++k) {
                if (k < n) x[k] = ld_elem(a.x, 8 * b + k, a.dtype);
                if (k < n && a.add) add[k] = ld_elem(a.add, 8 * b + k, a.dtype);
            }
        }
        drop8(a, philox((uint64_t)b, seed, offset), x, add, y);
        if (VEC && n == 8) {
            store_row_run<8>(a.y, 8 * b, y, a.dtype);
        } else {
            for (int k = 0; k < 8; ++k)
                if (k < n) st_elem(a.y, 8 * b + k, y[k], a.dtype);
        }
    }
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
    a.cut = (uint32_t)std::floor(p * 65536.0 + 0.5);
    a.scale = a.cut < 65536u ? (float)(65536.0 / (65536.0 - a.cut)) : 0.f;
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(y)) & 15) == 0;
    const int64_t ctas = ((n + 7) / 8 + DT - 1) / DT;
    note_launch_begin(KC_OTHER, s);
    const cudaError_t e = launch_pdl(vec ? dropout_kernel<true> : dropout_kernel<false>,
                                     dim3((unsigned)std::min<int64_t>(ctas, (int64_t)dc.sms * 8)), dim3(DT), 0, s, a);
    note_launch_end(KC_OTHER, 0.0, s);
    return e == cudaSuccess ? MUON_OK : cuda_fail(e, "dropout launch");
} MUON_CATCH_ALL
