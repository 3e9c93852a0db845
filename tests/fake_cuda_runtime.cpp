// fake_cuda_runtime.cpp -- a CUDA runtime for tests of the library's host side on a
// machine without a GPU.  It runs no kernel: it keeps what is asked of it, and
// answers as the runtime does where the tests look.
//   * several devices, one current (fake_set_device);
//   * the limit of a kernel's dynamic shared memory belongs to a device, and a
//     launch that asks for more than it fails;
//   * clusters that fit at once, by device (fake_set_clusters);
//   * fake_fail(name, skip, n): after `skip` more calls of a function, n of them fail.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstdlib>
#include <cstring>
#include <map>
#include <set>
#include <string>
#include <utility>

namespace {

constexpr int kDevices = 4;
int g_device = 0;
int g_clusters[kDevices] = {152, 152, 152, 152};
std::map<std::string, std::pair<int, int>> g_fail;    // calls to skip, then to fail
std::map<std::pair<int, const void *>, int> g_smem;   // limits by device and kernel
std::set<std::pair<int, const void *>> g_blocks;      // allocations by device
std::map<const void *, std::string> g_names;
unsigned char g_symbols[kDevices][64];

struct Launch {
    char kernel[256];
    int device, grid[3], block, smem, cluster, pdl;
};
Launch g_launch[64];
int g_launches = 0;

bool fails(const char *name)
{
    auto i = g_fail.find(name);
    if (i == g_fail.end()) return false;
    if (i->second.first > 0) {
        --i->second.first;
        return false;
    }
    return i->second.second-- > 0;
}

}  // namespace

extern "C" {

void fake_set_device(int d) { g_device = d; }
void fake_set_clusters(int d, int n) { g_clusters[d] = n; }
void fake_fail(const char *name, int skip, int n) { g_fail[name] = {skip, n}; }
int fake_launches(void) { return g_launches; }
const void *fake_launch(int i) { return &g_launch[i]; }
void fake_forget_launches(void) { g_launches = 0; }
int fake_blocks(int d)
{
    int n = 0;
    for (const auto &b : g_blocks) n += b.first == d;
    return n;
}

cudaError_t cudaGetDevice(int *d)
{
    *d = g_device;
    return fails("cudaGetDevice") ? cudaErrorUnknown : cudaSuccess;
}

#undef cudaGetDeviceProperties
cudaError_t cudaGetDeviceProperties(cudaDeviceProp *p, int)
{
    if (fails("cudaGetDeviceProperties")) return cudaErrorUnknown;
    std::memset(p, 0, sizeof *p);
    p->multiProcessorCount = 152, p->major = 10, p->minor = 3, p->sharedMemPerBlockOptin = 227 * 1024;
    return cudaSuccess;
}

cudaError_t cudaGetLastError(void) { return cudaSuccess; }

cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute attr, int value)
{
    if (fails("cudaFuncSetAttribute")) return cudaErrorUnknown;
    if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) g_smem[{g_device, f}] = value;
    return cudaSuccess;
}

cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c)
{
    if (fails("cudaOccupancyMaxActiveClusters")) return cudaErrorUnknown;
    const auto s = g_smem.find({g_device, f});
    const size_t most = s == g_smem.end() ? 48 * 1024 : s->second;
    if (c->dynamicSmemBytes > most) return cudaErrorInvalidValue;
    *n = g_clusters[g_device] / static_cast<int>(c->attrs[0].val.clusterDim.x);
    return cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **)
{
    if (fails("cudaLaunchKernelExC")) return cudaErrorUnknown;
    const auto s = g_smem.find({g_device, f});
    const size_t most = s == g_smem.end() ? 48 * 1024 : s->second;
    if (c->dynamicSmemBytes > most) return cudaErrorInvalidValue;
    if (g_launches < 64) {
        Launch &l = g_launch[g_launches++];
        std::memset(&l, 0, sizeof l);
        std::strncpy(l.kernel, g_names[f].c_str(), sizeof l.kernel - 1);
        l.device = g_device, l.block = static_cast<int>(c->blockDim.x), l.smem = static_cast<int>(c->dynamicSmemBytes);
        l.grid[0] = static_cast<int>(c->gridDim.x), l.grid[1] = static_cast<int>(c->gridDim.y), l.grid[2] = static_cast<int>(c->gridDim.z);
        for (unsigned i = 0; i < c->numAttrs; ++i) {
            if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) l.cluster = static_cast<int>(c->attrs[i].val.clusterDim.x);
            if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization) l.pdl = 1;
        }
    }
    return cudaSuccess;
}

cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s)
{
    *s = cudaStreamCaptureStatusNone;
    return cudaSuccess;
}

// (a pool's handle is its device)
cudaError_t cudaMemPoolCreate(cudaMemPool_t *p, const cudaMemPoolProps *props)
{
    if (fails("cudaMemPoolCreate")) return cudaErrorUnknown;
    *p = reinterpret_cast<cudaMemPool_t>(static_cast<uintptr_t>(props->location.id + 1));
    return cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void *)
{
    return fails("cudaMemPoolSetAttribute") ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaMemPoolDestroy(cudaMemPool_t) { return cudaSuccess; }
static cudaError_t take(void **p, size_t n, int device)
{
    *p = std::malloc(n ? n : 1);
    g_blocks.insert({device, *p});
    return cudaSuccess;
}
cudaError_t cudaMallocFromPoolAsync(void **p, size_t n, cudaMemPool_t pool, cudaStream_t)
{
    if (fails("cudaMallocFromPoolAsync")) return cudaErrorMemoryAllocation;
    return take(p, n, static_cast<int>(reinterpret_cast<uintptr_t>(pool)) - 1);
}
cudaError_t cudaMallocAsync(void **p, size_t n, cudaStream_t)
{
    return fails("cudaMallocAsync") ? cudaErrorMemoryAllocation : take(p, n, g_device);
}
cudaError_t cudaFreeAsync(void *p, cudaStream_t)
{
    for (int d = 0; d < kDevices; ++d) g_blocks.erase({d, p});
    std::free(p);
    return cudaSuccess;
}

cudaError_t cudaGetSymbolAddress(void **p, const void *)
{
    if (fails("cudaGetSymbolAddress")) return cudaErrorUnknown;
    *p = g_symbols[g_device];
    return cudaSuccess;
}
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void *d, const void *, size_t n, size_t, cudaMemcpyKind)
{
    std::memset(d, 0, n);
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
#undef cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned)
{
    *n = 1;
    return cudaSuccess;
}

static CUresult encode(CUtensorMap *, ...) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *r)
{
    *f = reinterpret_cast<void *>(&encode), *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

// What the compiler's host code calls when the library is loaded, and to launch.
void **__cudaRegisterFatBinary(void *)
{
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *f, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *, int *)
{
    g_names[f] = name;
}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f)
{
    *k = reinterpret_cast<cudaKernel_t>(const_cast<void *>(f));
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }

}  // extern "C"
