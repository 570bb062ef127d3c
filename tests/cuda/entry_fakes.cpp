// entry_fakes.cpp — test-only stand-ins for the CUDA runtime and for the kernels'
// launches, so that the C entry points of cross-attention and of the heads' norm and
// rotation run on a machine without a GPU, past their first CUDA call.  Nothing is
// launched; a call that gets as far as that counts as one launch.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "attn_bwd.h"
#include "attn_fwd.h"
#include "attn_host.h"
#include "cross_few.h"
#include "cross_join.h"
#include "rope_impl.h"

#define FAKE extern "C" __attribute__((visibility("default")))

namespace {
int g_sms = 152, g_fail = 0, g_launches = 0;
int g_status[2];
CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
cudaError_t launched() {
  ++g_launches;
  return cudaSuccess;
}
}  // namespace

// The SMs of the device; `fail`: its queries end with that error instead.
FAKE void fake_device(int sms, int fail) { g_sms = sms, g_fail = fail, g_launches = 0; }
FAKE int fake_launches() { return g_launches; }
FAKE int fake_cuda_error() { return ea::g_last_cuda_error; }

extern "C" {
cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int) {
  if (g_fail) return static_cast<cudaError_t>(g_fail);
  *value = g_sms;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* found) {
  *fn = reinterpret_cast<void*>(&encode);
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}

namespace ea {
attn_status_t current_status_words(int** status) {
  *status = g_status;
  return ATTN_OK;
}
cudaError_t cross_few_launch(const FewParams&, bool, cudaStream_t) { return launched(); }
cudaError_t cross_small_bwd_launch(const SmallBwdParams&, int, bool, cudaStream_t) { return launched(); }
cudaError_t fwd1qp_launch(const Fwd1QParams&, int, int, bool, cudaStream_t) { return launched(); }
cudaError_t fwd1q_launch(const Fwd1QParams&, int, int, bool, cudaStream_t) { return launched(); }
cudaError_t cross_bwd_launch(const BwdParams&, int, bool, cudaStream_t) { return launched(); }
cudaError_t bwd256_launch(const BwdParams&, int, bool, cudaStream_t) { return launched(); }
cudaError_t join_fwd_launch(const JoinFwdParams&, bool, cudaStream_t) { return launched(); }
cudaError_t join_sum_launch(const JoinSumParams*, int, bool, cudaStream_t) { return launched(); }
cudaError_t rope_fwd_launch(const RopeParams&, RopeShape, bool, int, cudaStream_t) { return launched(); }
cudaError_t rope_bwd_launch(const RopeParams&, RopeShape, bool, int, cudaStream_t) { return launched(); }
// as the kernels' own, divides by what is resident
int rope_plan(RopeParams& p, RopeShape, bool, int sms) { return (p.N + sms - 1) / sms; }
int rope_most_ctas(int sms) { return 3 * sms; }
}  // namespace ea
