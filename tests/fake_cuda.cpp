// A CUDA runtime for tests without a GPU: it launches nothing and notes what it is asked for. The
// dense operators' objects link against it in place of the runtime (tests/fake_cuda.py).
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <cudaTypedefs.h>

#include <map>
#include <string>
#include <vector>

namespace {

struct Launch {
  std::string kernel;
  int device;
};

std::map<const void *, std::string> g_names;          // kernels by their host address
std::map<std::pair<const void *, int>, int> g_smem;   // what each may ask for, per device
std::vector<Launch> g_launches;
int g_device = 0;
int g_maps = 0, g_refused = -1;  // tensor maps asked for; the one that is refused
int g_fail_attribute = 0;        // attribute calls still to fail
int g_attribute_calls = 0;

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t rank, void *base,
                const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  if (g_maps++ == g_refused) return CUDA_ERROR_INVALID_VALUE;
  if (!base || (reinterpret_cast<uintptr_t>(base) & 15u)) return CUDA_ERROR_INVALID_VALUE;
  for (cuuint32_t i = 0; i < rank; ++i)
    if (dims[i] == 0 || box[i] == 0 || box[i] > 256) return CUDA_ERROR_INVALID_VALUE;
  for (cuuint32_t i = 0; i + 1 < rank; ++i)
    if (strides[i] % 16 || strides[i] >> 40) return CUDA_ERROR_INVALID_VALUE;
  return CUDA_SUCCESS;
}

}  // namespace

namespace coll {
// api.cu looks it up through the runtime
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() { return encode; }
}  // namespace coll

extern "C" {

void fake_reset(int refused_map) {
  g_launches.clear();
  g_maps = 0;
  g_refused = refused_map;
}
void fake_device(int d) { g_device = d; }
void fake_fail_attributes(int n) { g_fail_attribute = n; }
int fake_attribute_calls(void) { return g_attribute_calls; }
int fake_maps(void) { return g_maps; }
int fake_launches(void) { return (int)g_launches.size(); }
const char *fake_launch_kernel(int i) { return g_launches[i].kernel.c_str(); }
int fake_launch_device(int i) { return g_launches[i].device; }

cudaError_t cudaGetDevice(int *d) {
  *d = g_device;
  return cudaSuccess;
}

cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int value) {
  ++g_attribute_calls;
  if (g_fail_attribute > 0) {
    --g_fail_attribute;
    return cudaErrorInvalidValue;
  }
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_smem[{f, g_device}] = value;
  return cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
  const auto it = g_smem.find({f, g_device});
  const size_t most = it == g_smem.end() ? 48 * 1024 : it->second;
  const bool grid = c->gridDim.x && c->gridDim.y && c->gridDim.z && c->gridDim.x <= 0x7FFFFFFFu &&
                    c->gridDim.y <= 65535 && c->gridDim.z <= 65535;
  if (c->dynamicSmemBytes > most) return cudaErrorInvalidValue;
  if (!grid) return cudaErrorInvalidConfiguration;
  g_launches.push_back({g_names[f], g_device});
  return cudaSuccess;
}

cudaError_t cudaGetLastError(void) { return cudaSuccess; }

// what nvcc's host code registers at load
void **__cudaRegisterFatBinary(void *) {
  static void *handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *,
                            uint3 *, dim3 *, dim3 *, int *) {
  g_names[host] = name;
}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void *) { return 1; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) {
  *k = (cudaKernel_t)f;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) {
  return cudaErrorNotSupported;  // the dense operators launch with attributes
}

}  // extern "C"
