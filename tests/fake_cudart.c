/*
 * A stand-in for the CUDA runtime under the library's host code: preloaded, it
 * answers the calls that a device would (no kernel runs) and keeps a log, so
 * that what the host asks of which device can be checked without a GPU.
 * Shared memory and cluster limits hold as on the device: a launch beyond what
 * was set for its kernel on its device is refused.
 */
#include <cuda_runtime_api.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static int device, capture, failing = -1;
static uintptr_t next_block = 0x100000000u;
static char text[1 << 20];
static size_t used;

void fake_set_device(int d) { device = d; }
void fake_set_capturing(int on) { capture = on; }
void fake_set_failing(int d) { failing = d; } /* a device whose kernels' attributes cannot be set */
void fake_clear(void) { used = 0; text[0] = 0; }
const char* fake_log(void) { return text; }

static void note(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    int n = vsnprintf(text + used, sizeof text - used, fmt, ap);
    va_end(ap);
    if (n > 0 && used + (size_t)n < sizeof text) used += (size_t)n;
}

/* what was set for a kernel on a device */
static struct { int device; const void* func; int smem, wide; } funcs[512];
static int nfuncs;
static int slot(const void* f) {
    for (int i = 0; i < nfuncs; ++i)
        if (funcs[i].device == device && funcs[i].func == f) return i;
    funcs[nfuncs].device = device;
    funcs[nfuncs].func = f;
    funcs[nfuncs].smem = 48 * 1024;
    funcs[nfuncs].wide = 0;
    return nfuncs++;
}

static unsigned cluster_of(const cudaLaunchConfig_t* c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
    return 1;
}
static cudaError_t check(const cudaLaunchConfig_t* c, const void* f) {
    const int i = slot(f);
    if (c->dynamicSmemBytes > (size_t)funcs[i].smem) return cudaErrorInvalidValue;
    if (cluster_of(c) > 8 && !funcs[i].wide) return cudaErrorInvalidClusterSize;
    return cudaSuccess;
}

cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetDeviceProperties(struct cudaDeviceProp* p, int d) {
    memset(p, 0, sizeof *p);
    snprintf(p->name, sizeof p->name, "fake %d", d);
    p->major = 10;
    p->minor = 3;
    p->multiProcessorCount = 152;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMalloc(void** p, size_t n) {
    *p = (void*)next_block;
    next_block += (n + 4095) / 4096 * 4096 + 4096;
    note("malloc %d %p %zu\n", device, *p, n);
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFree(void* p) { note("free %d %p\n", device, p); return cudaSuccess; }
cudaError_t CUDARTAPI cudaMemset(void* p, int v, size_t n) { (void)p; (void)v; (void)n; return cudaSuccess; }
cudaError_t CUDARTAPI cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) {
    (void)p; (void)v; (void)n; (void)s;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t s) {
    (void)s;
    return capture ? cudaErrorStreamCaptureUnsupported : cudaSuccess;
}
cudaError_t CUDARTAPI cudaStreamIsCapturing(cudaStream_t s, enum cudaStreamCaptureStatus* st) {
    (void)s;
    *st = capture ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
    const int i = slot(f);
    if (device == failing) return cudaErrorDevicesUnavailable;
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) funcs[i].smem = v;
    if (a == cudaFuncAttributeNonPortableClusterSizeAllowed) funcs[i].wide = v;
    note("attribute %d %p %d %d\n", device, f, (int)a, v);
    return cudaSuccess;
}
/* resident clusters of an SM's 228 KB, 1 KB kept per block, and 2048 threads */
cudaError_t CUDARTAPI cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
    const cudaError_t e = check(c, f);
    if (e != cudaSuccess) return e;
    int per = (int)(228 * 1024 / (c->dynamicSmemBytes + 1024));
    if (per > (int)(2048 / c->blockDim.x)) per = (int)(2048 / c->blockDim.x);
    *n = 152 * per / (int)cluster_of(c);
    note("occupancy %d %p %zu %u %d\n", device, f, c->dynamicSmemBytes, cluster_of(c), *n);
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
    (void)args;
    const cudaError_t e = check(c, f);
    note("launch %d %p %zu %u %u %d\n", device, f, c->dynamicSmemBytes, cluster_of(c), c->gridDim.x, (int)e);
    return e;
}
cudaError_t CUDARTAPI cudaMallocHost(void** p, size_t n) {
    *p = calloc(1, n);
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFreeHost(void* p) { free(p); return cudaSuccess; }
cudaError_t CUDARTAPI cudaMemcpyAsync(void* d, const void* s, size_t n, enum cudaMemcpyKind k, cudaStream_t st) {
    (void)d; (void)s; (void)n; (void)k; (void)st;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaEventCreate(cudaEvent_t* e) { *e = (cudaEvent_t)1; return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventCreateWithFlags(cudaEvent_t* e, unsigned f) { (void)f; *e = (cudaEvent_t)1; return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventDestroy(cudaEvent_t e) { (void)e; return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventRecord(cudaEvent_t e, cudaStream_t s) { (void)e; (void)s; return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventSynchronize(cudaEvent_t e) { (void)e; return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventElapsedTime(float* ms, cudaEvent_t a, cudaEvent_t b) {
    (void)a; (void)b;
    *ms = 1.0f;
    return cudaSuccess;
}
static int encode_tiled(void) { return 0; }
cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned int version,
                                                       unsigned long long flags,
                                                       enum cudaDriverEntryPointQueryResult* q) {
    (void)name; (void)version; (void)flags;
    *fn = (void*)encode_tiled;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
