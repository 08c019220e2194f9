// Test infrastructure: one wavefront runs one sparse 8-bit matrix instruction on
// operands given lane by lane, so a GPU test can compare the hardware's lane
// mapping with the lane-level model the CPU tests drive the 8-bit layout through.
//   p24probe_smfmac64_f8: v_smfmac_f32_32x32x64_fp8_fp8, A = a[64][16]
//     (compressed e4m3 values), B = b[64][32] e4m3, index word idx[64], zero
//     accumulator; d[64][16] fp32 in the instruction's output lane order.
// Returns 0, or -1 if the launch failed.  All pointers are device pointers.
#include <hip/hip_runtime.h>
#include <stdint.h>

typedef int i32x4v __attribute__((ext_vector_type(4)));
typedef int i32x8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

__global__ __launch_bounds__(64) void k_smfmac_f8(const int* a, const int* b, const uint32_t* idx, float* d) {
  const int l = threadIdx.x;
  i32x4v av;
  i32x8v bv;
  for (int i = 0; i < 4; ++i) av[i] = a[l * 4 + i];
  for (int i = 0; i < 8; ++i) bv[i] = b[l * 8 + i];
  f16v acc = {};
  acc = __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(av, bv, acc, (int)idx[l], 0, 0);
  for (int i = 0; i < 16; ++i) d[l * 16 + i] = acc[i];
}

extern "C" __attribute__((visibility("default"))) int p24probe_smfmac64_f8(const void* a, const void* b,
                                                                          const uint32_t* idx, float* d,
                                                                          void* stream) {
  hipLaunchKernelGGL(k_smfmac_f8, dim3(1), dim3(64), 0, (hipStream_t)stream, (const int*)a, (const int*)b, idx, d);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
