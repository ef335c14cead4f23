// A stand-in for the CUDA runtime on the host, for tests of what the library launches and how: linked with the library's
// objects in place of the runtime, it runs nothing and records every launch.  "Device" memory is host memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

namespace {
struct Launch {
    std::string kernel;                          // mangled name
    unsigned grid, block, cluster;
    int overlap;                                 // launched with programmatic stream serialization
    void* stream;
};
std::mutex mu;
std::map<const void*, std::string>& names() { static std::map<const void*, std::string> m; return m; }
std::vector<Launch>& launches() { static std::vector<Launch> v; return v; }
int largest_cluster = 16, sms = 152, no_memory = 0;
thread_local struct { dim3 grid, block; size_t smem; cudaStream_t st; } call;

CUresult encode_tiled(CUtensorMap* m, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                      const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                      CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    memset(m, 0, sizeof *m);
    return CUDA_SUCCESS;
}
void record(const void* f, dim3 grid, dim3 block, cudaStream_t st, const cudaLaunchAttribute* attrs, unsigned n) {
    Launch l = {"", grid.x, block.x, 1, 0, st};
    for (unsigned i = 0; i < n; ++i) {
        if (attrs[i].id == cudaLaunchAttributeClusterDimension) l.cluster = attrs[i].val.clusterDim.x;
        if (attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
            l.overlap = attrs[i].val.programmaticStreamSerializationAllowed;
    }
    std::lock_guard<std::mutex> lk(mu);
    l.kernel = names()[f];
    launches().push_back(l);
}
}  // namespace

extern "C" {
// ---- for the tests
void fake_set_largest_cluster(int n) { largest_cluster = n; }
void fake_set_no_memory(int on) { no_memory = on; }
int fake_launch_count() { return (int)launches().size(); }
void fake_clear() { launches().clear(); }
const char* fake_launch(int i, unsigned* grid, unsigned* block, unsigned* cluster, int* overlap) {
    const Launch& l = launches()[i];
    *grid = l.grid; *block = l.block; *cluster = l.cluster; *overlap = l.overlap;
    return l.kernel.c_str();
}

// ---- registration and launches, as compiled code calls them
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
    std::lock_guard<std::mutex> lk(mu);
    names()[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* host) {
    *k = (cudaKernel_t)const_cast<void*>(host);
    return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
    call = {grid, block, smem, st};
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* st) {
    *grid = call.grid; *block = call.block; *smem = call.smem;
    *(cudaStream_t*)st = call.st;
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3 block, void**, size_t, cudaStream_t st) {
    record((const void*)k, grid, block, st, nullptr, 0);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    record(f, c->gridDim, c->blockDim, c->stream, c->attrs, c->numAttrs);
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension && (int)c->attrs[i].val.clusterDim.x > largest_cluster)
            return cudaErrorLaunchOutOfResources;
    return cudaSuccess;
}

// ---- the runtime's calls
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "error"; }
const char* cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : (a == cudaDevAttrComputeCapabilityMinor ? 3 : sms);
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
    int size = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) size = (int)c->attrs[i].val.clusterDim.x;
    *n = size > largest_cluster ? 0 : sms / size;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    *p = (void*)encode_tiled;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) {
    *p = no_memory ? nullptr : aligned_alloc(256, (n + 255) / 256 * 256);
    return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaMemset(void* p, int v, size_t n) { memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
    *s = cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = nullptr; return cudaErrorInvalidSymbol; }
}
