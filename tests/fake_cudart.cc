// fake_cudart.cc -- the CUDA runtime calls that libgemm.so makes, as a host without a
// GPU can answer them: one GB300, device memory at made-up addresses, launches that do
// nothing. The n-th launch (or kernel attribute) from now on fails when it is asked
// to, and leaves its error the way the runtime does: until somebody reads it with
// cudaGetLastError(). Loaded before libgemm.so with its symbols global
// (tests/test_failed_launches.py drives it).
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstring>

namespace {
cudaError_t last = cudaSuccess;
long launches = 0, fail_launch = -1, attributes = 0, fail_attribute = -1;
long allocated = 0, freed = 0;

cudaError_t left(cudaError_t e) {
    if (e != cudaSuccess) last = e;
    return e;
}
cudaError_t launch() {
    return left(launches++ == fail_launch ? cudaErrorLaunchOutOfResources : cudaSuccess);
}
cudaError_t attribute() {
    return left(attributes++ == fail_attribute ? cudaErrorInvalidValue : cudaSuccess);
}
CUresult encode(...) { return CUDA_SUCCESS; }
}  // namespace

extern "C" {

// what a test asks: counts from zero, and which launch or attribute fails (-1: none)
void fake_reset(long launch_to_fail, long attribute_to_fail) {
    last = cudaSuccess;
    launches = attributes = allocated = freed = 0;
    fail_launch = launch_to_fail;
    fail_attribute = attribute_to_fail;
}
int fake_last_error() { return (int)last; }
long fake_launches() { return launches; }
long fake_attributes() { return attributes; }
long fake_live_allocations() { return allocated - freed; }

cudaError_t cudaGetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaGetDevice(int* device) { return *device = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int) {
    return *value = 0, cudaSuccess;
}
cudaError_t cudaGetDeviceProperties(cudaDeviceProp* p, int) {
    std::memset(p, 0, sizeof(*p));
    p->major = 10;
    p->minor = 3;
    p->multiProcessorCount = 152;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** at, const void*) {
    return *at = reinterpret_cast<void*>(0x7000), cudaSuccess;
}
cudaError_t cudaMemPoolCreate(cudaMemPool_t* pool, const cudaMemPoolProps*) {
    return *pool = reinterpret_cast<cudaMemPool_t>(0x10), cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void*) { return cudaSuccess; }
cudaError_t cudaMallocFromPoolAsync(void** at, size_t, cudaMemPool_t, cudaStream_t) {
    ++allocated;
    return *at = reinterpret_cast<void*>(0x1000000), cudaSuccess;
}
cudaError_t cudaFreeAsync(void*, cudaStream_t) { return ++freed, cudaSuccess; }
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
    return *s = reinterpret_cast<cudaStream_t>(0x20), cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t, unsigned long long* id) { return *id = 1, cudaSuccess; }
// in a capture, so that no scratch is kept across calls
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* status) {
    return *status = cudaStreamCaptureStatusActive, cudaSuccess;
}
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
    return *e = reinterpret_cast<cudaEvent_t>(0x30), cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void*) {
    std::memset(a, 0, sizeof(*a));
    a->type = cudaMemoryTypeDevice;
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) {
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
    std::memset(a, 0, sizeof(*a));
    a->numRegs = 168;  // of gemm_xent's kernels, which are launched with no other number
    return attribute();
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return attribute(); }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
    return *n = 76, attribute();
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t,
                                                                   unsigned) {
    return *n = 1, attribute();
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    *fn = reinterpret_cast<void*>(&encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return launch(); }
// a launch by <<<>>>
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, cudaStream_t) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
    *grid = *block = dim3(1);
    *smem = 0;
    *static_cast<void**>(stream) = nullptr;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* kernel, const void* at) {
    return *kernel = reinterpret_cast<cudaKernel_t>(const_cast<void*>(at)), cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) {
    return launch();
}

}  // extern "C"
