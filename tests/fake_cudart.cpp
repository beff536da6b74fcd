// A stand-in for the CUDA runtime, for tests of the library's host code without a GPU (linked with the library's own
// objects in place of the runtime).  It keeps what the host code relies on: function attributes belong to the
// current device, a launch that they do not allow fails, an error stays until it is asked for, and a device places
// clusters up to a size of its own.  Nothing runs; fake_* functions set it up and tell what was launched.
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <string.h>

#include <map>
#include <string>
#include <utility>
#include <vector>

namespace {
int device = 0, max_cluster = 16, failing_attributes = 0, failing_launches = 0;
cudaError_t last = cudaSuccess;
struct Attributes {
    int dynamic_smem = 48 * 1024, non_portable = 0;
};
std::map<std::pair<int, const void*>, Attributes> attributes;
std::map<const void*, std::string> names;
struct Launch {
    std::string name;
    int cluster;
};
std::vector<Launch> launches;

cudaError_t result(cudaError_t e) {
    if (e != cudaSuccess) last = e;
    return e;
}
int cluster_of(const cudaLaunchConfig_t* c) {
    int n = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension)
            n = c->attrs[i].val.clusterDim.x * c->attrs[i].val.clusterDim.y * c->attrs[i].val.clusterDim.z;
    return n;
}
bool allowed(const cudaLaunchConfig_t* c, const void* f) {
    const Attributes& a = attributes[{device, f}];
    const int n = cluster_of(c);
    return static_cast<int>(c->dynamicSmemBytes) <= a.dynamic_smem && (n <= 8 || a.non_portable);
}
CUresult encode(CUtensorMap* m, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                CUtensorMapFloatOOBfill) {
    memset(m, 0, sizeof(*m));
    return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
void fake_reset(int dev, int cluster) {
    device = dev;
    max_cluster = cluster;
    failing_attributes = failing_launches = 0;
    last = cudaSuccess;
    launches.clear();
}
void fake_fail(int n_attributes, int n_launches) {
    failing_attributes = n_attributes;
    failing_launches = n_launches;
}
int fake_launches(void) { return static_cast<int>(launches.size()); }
const char* fake_launch_name(int i) { return launches[i].name.c_str(); }
int fake_launch_cluster(int i) { return launches[i].cluster; }

cudaError_t cudaGetDevice(int* d) {
    *d = device;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr attr, int) {
    *v = attr == cudaDevAttrMultiProcessorCount ? 152 : 0;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int v) {
    if (failing_attributes > 0) {
        --failing_attributes;
        return result(cudaErrorInvalidValue);
    }
    Attributes& a = attributes[{device, f}];
    if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) a.dynamic_smem = v;
    if (attr == cudaFuncAttributeNonPortableClusterSizeAllowed) a.non_portable = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
    *n = 0;
    if (!allowed(c, f)) return result(cudaErrorInvalidClusterSize);
    *n = cluster_of(c) <= max_cluster ? 8 : 0;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
    *n = 2;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    if (failing_launches > 0) {
        --failing_launches;
        return result(cudaErrorLaunchOutOfResources);
    }
    if (!allowed(c, f)) return result(cudaErrorInvalidValue);
    if (cluster_of(c) > max_cluster) return result(cudaErrorInvalidClusterSize);
    launches.push_back({names[f], cluster_of(c)});
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    *p = reinterpret_cast<void*>(&encode);
    if (q) *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
    *p = reinterpret_cast<void*>(0x1000);
    return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }

// what nvcc's host stubs call to register their kernels
void** __cudaRegisterFatBinary(void*) {
    static void* handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*) {
    names[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
    *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
}
