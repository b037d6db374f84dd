// Counts what the library's host-side caches ask of the driver, with a driver
// of its own: two rounds over the buffers of 40 layers, and over 96 kernels.
// Prints: encodes of round one and two, wrong maps, attribute calls of round
// one and two, map slots of another shape that came back wrong.
#include <cstdio>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

static int g_encodes = 0, g_attributes = 0;

static CUresult fake_encode(CUtensorMap* map, CUtensorMapDataType, cuuint32_t rank, void* base, const cuuint64_t* dims,
                            const cuuint64_t*, const cuuint32_t* box, const cuuint32_t*, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  ++g_encodes;
  std::memset(map, 0, sizeof(*map));
  std::memcpy(map, &base, sizeof(base));
  std::memcpy(reinterpret_cast<char*>(map) + 8, dims, rank * sizeof(*dims));
  std::memcpy(reinterpret_cast<char*>(map) + 48, box, rank * sizeof(*box));
  return CUDA_SUCCESS;
}
static CUresult fake_ctx(CUcontext* c) {
  *c = reinterpret_cast<CUcontext>(0x10);
  return CUDA_SUCCESS;
}
static CUresult fake_ctx_id(CUcontext, unsigned long long* id) {
  *id = 7;
  return CUDA_SUCCESS;
}

extern "C" {
cudaError_t cudaGetDriverEntryPoint(const char* name, void** p, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *q = cudaDriverEntryPointSuccess;
  *p = !std::strcmp(name, "cuCtxGetCurrent") ? (void*)fake_ctx
       : !std::strcmp(name, "cuCtxGetId")    ? (void*)fake_ctx_id
                                             : (void*)fake_encode;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 148;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  ++g_attributes;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return cudaSuccess; }
}

#include "host_cache.cu"

int main() {
  int encodes[2], attributes[2], wrong = 0;
  for (int round = 0; round < 2; ++round) {
    const int e0 = g_encodes, a0 = g_attributes;
    for (int layer = 0; layer < 40; ++layer)
      for (int which = 0; which < 4; ++which) {  // caches of two shapes: keys and values, rows and scales
        void* base = reinterpret_cast<void*>(0x7f0000000000ull + (uint64_t)layer * 0x4000000 + which * 0x1000000);
        const uint64_t dims[3] = {64, (uint64_t)(16 << which), 1000}, strides[2] = {128, 4096};
        const uint32_t box[3] = {64, 16, 1};
        CUtensorMap m;
        if (!csa::encode_tensor_map(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
          return 1;
        wrong += std::memcmp(&m, &base, sizeof(base)) != 0 || std::memcmp(reinterpret_cast<char*>(&m) + 8, dims, sizeof(dims)) != 0;
      }
    for (int k = 0; k < 96; ++k)
      if (csa::set_max_smem(reinterpret_cast<void*>(0x1000 + 64 * (uint64_t)k), 200000) != cudaSuccess) return 1;
    encodes[round] = g_encodes - e0;
    attributes[round] = g_attributes - a0;
  }
  // more of them than there are places: still the right ones
  for (int i = 0; i < 5000; ++i) {
    void* base = reinterpret_cast<void*>(0x1000ull * (i % 1700 + 1));
    const uint64_t dims[2] = {64, (uint64_t)(i % 3 + 1)}, strides[1] = {128};
    const uint32_t box[2] = {64, 1};
    CUtensorMap m;
    csa::encode_tensor_map(&m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    wrong += std::memcmp(&m, &base, sizeof(base)) != 0 || std::memcmp(reinterpret_cast<char*>(&m) + 8, dims, sizeof(dims)) != 0;
  }
  std::printf("%d %d %d %d %d\n", encodes[0], encodes[1], attributes[0], attributes[1], wrong);
  return 0;
}
