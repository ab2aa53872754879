// A stand-in for the CUDA runtime and the kernel launchers, host code only: it
// is linked with the library's boundary (csrc/api.cu) into a library of its own,
// so that a test sees which device was current at each launch, and what a
// launcher was given, without a GPU.
#include <cuda_runtime.h>
#include <stdlib.h>
#include <string.h>

int atomicOr(int*, int);  // named in device code, which is not compiled here
template <typename Kernel>
cudaError_t cudaFuncSetAttribute(Kernel* kernel, cudaFuncAttribute a, int v) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), a, v);
}

#include "../token_sparse_denoising_layer_b200/csrc/internal.h"

namespace {

int current = 0;    // the calling thread's current device
int n_launches = 0;
int n_strays = 0;   // launches made while another device than the context's was current
int attr_device = -1;  // device that was current when a kernel's attribute was last set
hsa::RopeFreqs freqs;

cudaError_t launch(const hsa::Ctx& c) {
  ++n_launches;
  if (current != c.device) ++n_strays;
  return cudaSuccess;
}

void no_kernel() {}

}  // namespace

extern "C" {

void fake_set_device(int d) { current = d; }
int fake_device() { return current; }
int fake_launches() { return n_launches; }
int fake_strays() { return n_strays; }
const uint64_t* fake_turns() { return freqs.turns; }

// Device on which the limit was raised for a context of `device` (-1: it was not).
int fake_ensure_smem_limit(int device) {
  static std::atomic<uint64_t> done{0};
  attr_device = -1;
  if (hsa::ensure_smem_limit(no_kernel, 1000, device, done) != cudaSuccess) return -2;
  return attr_device;
}

cudaError_t cudaGetDevice(int* d) { return *d = current, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return current = d, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 148, cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t) { return *p = aligned_alloc(64, 64), cudaSuccess; }
cudaError_t cudaFree(void* p) { return free(p), cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void* d, const void*, size_t n, cudaMemcpyKind) { return memset(d, 0, n), cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventCreate(cudaEvent_t*) { return cudaErrorNotSupported; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float* ms, cudaEvent_t, cudaEvent_t) { return *ms = 0.f, cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "fake"; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPoint(const char*, void**, unsigned long long, cudaDriverEntryPointQueryResult*) {
  return cudaErrorNotSupported;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return attr_device = current, cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}

hsa_status hsa_select_groups_static(const float*, const float*, int, const int*, int, uint8_t*, void*) {
  return HSA_ERR_CUDA;
}

}  // extern "C"

namespace hsa {

cudaError_t launch_schedule(const Ctx& c, int, const uint8_t*, uint8_t*, int32_t*, int32_t*) { return launch(c); }
cudaError_t launch_score(const Ctx& c, const float*, const float*, float*) { return launch(c); }
cudaError_t launch_select(const Ctx& c, const float*, uint8_t*) { return launch(c); }
cudaError_t launch_selftest_timeout(const Ctx& c, uint64_t) { return launch(c); }
cudaError_t launch_euler(const Ctx& c, float*, float*, float*, const float*, const uint8_t*, float, float, float*) {
  return launch(c);
}
cudaError_t launch_ln_gather(const Ctx& c, const float*, const int32_t*, int, void*, const float*, const float*) {
  return launch(c);
}
cudaError_t launch_kv_scatter(const Ctx& c, const void*, const void*, int, const int32_t*, int, void*, void*) {
  return launch(c);
}
cudaError_t launch_embed(const Ctx& c, const float*, const float*, const int32_t*, int, float*) { return launch(c); }
cudaError_t launch_head(const Ctx& c, const float*, const float*, const int32_t*, int, float*) { return launch(c); }
cudaError_t launch_gemm(const Ctx& c, const GemmArgs&, std::string*) { return launch(c); }
cudaError_t launch_gemm_s8(const Ctx& c, const GemmArgs&, std::string*) { return launch(c); }
cudaError_t launch_attention(const Ctx& c, const void*, int, const void*, const void*, int, void*, std::string*) {
  return launch(c);
}
cudaError_t launch_rope_table(const Ctx& c, const RopeFreqs& f, const int32_t*, int, float*) {
  freqs = f;
  return launch(c);
}
cudaError_t launch_rope(const Ctx& c, const void*, int64_t, bool, int, int, const float*, int, int, const int32_t*,
                        bool, bool, void*, int64_t) {
  return launch(c);
}
cudaError_t launch_qk_norm_rope(const Ctx& c, const hsa_qk_rope&, const QkRows&) { return launch(c); }
cudaError_t launch_quant_rows(const Ctx& c, const void*, bool, int, int, int64_t, int8_t*, int64_t, float*) {
  return launch(c);
}
cudaError_t launch_ln_gather_quant(const Ctx& c, const float*, const int32_t*, int, int8_t*, float*, const float*,
                                   const float*) {
  return launch(c);
}
cudaError_t launch_cross_attention(const Ctx& c, const hsa_cross_args&, std::string*) { return launch(c); }

}  // namespace hsa
