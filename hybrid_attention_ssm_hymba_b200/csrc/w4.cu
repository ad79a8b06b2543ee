// w4.cu -- weights in 4 bits with group scales, w[n, k] = q[n, k] * scales[n, k / group]:
// quantised, read back, and multiplied with a few rows (a generation step's products).
#include "paged.cuh"

namespace hy {
namespace {

// Eight weights per lane; the group / 8 lanes of a group share its maximum by shuffles.
template <typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const T* __restrict__ w, uint32_t* __restrict__ q4,
                                                          float* __restrict__ scales, long long n8, int group) {
  pdl_trigger();
  pdl_wait();
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int lpg = group / 8;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (i < n8) {
    Vec8<T> v;
    v.load(w + i * 8);
    v.to_f32(f);
  }
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
  for (int o = lpg >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (i >= n8) return;
  const float most = fmaxf(m, 1.17549435e-38f), r = __fdiv_rn(7.f, most);
  uint32_t u = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // t is within 7 * 2^-22 of 7 w / most: only next to a half does the exact quotient decide
    // (and where 7 / most overflows, which leaves t - c no number)
    const float t = f[e] * r;
    float c = rintf(t);
    if (!(fabsf(t - c) <= 0.49999f)) c = static_cast<float>(rint(7.0 * f[e] / static_cast<double>(most)));
    u |= static_cast<uint32_t>(static_cast<int>(c) + 8) << (4 * e);
  }
  q4[i] = u;
  if ((i % lpg) == 0) scales[i / lpg] = fmaxf(__fdiv_rn(m, 7.f), 1.17549435e-38f);
}

template <typename T>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(const uint32_t* __restrict__ q4,
                                                            const float* __restrict__ scales, T* __restrict__ w,
                                                            long long n8, int group) {
  pdl_trigger();
  pdl_wait();
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n8) return;
  const uint32_t u = q4[i];
  const float s = scales[i / (group / 8)];
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(static_cast<int>((u >> (4 * e)) & 15u) - 8) * s;
  Vec8<T> v;
  v.from_f32(f);
  v.store(w + i * 8);
}

// One warp per (n, m): every lane takes eight consecutive k at a time.
template <typename T>
__global__ void __launch_bounds__(256) gemm_w4_simple(const T* __restrict__ a, const uint32_t* __restrict__ q4,
                                                      const float* __restrict__ scales, T* __restrict__ c, int M,
                                                      int N, int K, int group) {
  pdl_trigger();
  pdl_wait();
  const long long wid = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (wid >= static_cast<long long>(M) * N) return;
  const int n = static_cast<int>(wid / M), m = static_cast<int>(wid % M);
  float acc = 0.f;
  for (int k8 = lane; k8 < K / 8; k8 += 32) {
    const uint32_t u = q4[static_cast<long long>(n) * (K / 8) + k8];
    const float s = scales[static_cast<long long>(n) * (K / group) + k8 / (group / 8)];
    Vec8<T> v;
    float f[8], t = 0.f;
    v.load(a + static_cast<long long>(m) * K + k8 * 8);
    v.to_f32(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) t = fmaf(static_cast<float>(static_cast<int>((u >> (4 * e)) & 15u) - 8), f[e], t);
    acc = fmaf(t, s, acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) c[static_cast<long long>(m) * N + n] = from_f<T>(acc);
}

unsigned blocks_for(long long items, int per) { return static_cast<unsigned>((items + per - 1) / per); }

}  // namespace

cudaError_t launch_quantize_w4(const void* w, void* q4, float* scales, int N, int K, int group, bool bf16,
                               cudaStream_t st) {
  const long long n8 = static_cast<long long>(N) * K / 8;
  return bf16 ? launch(quantize_w4_kernel<__nv_bfloat16>, dim3(blocks_for(n8, 256)), dim3(256), 0, st,
                       static_cast<const __nv_bfloat16*>(w), static_cast<uint32_t*>(q4), scales, n8, group)
              : launch(quantize_w4_kernel<float>, dim3(blocks_for(n8, 256)), dim3(256), 0, st,
                       static_cast<const float*>(w), static_cast<uint32_t*>(q4), scales, n8, group);
}

cudaError_t launch_dequantize_w4(const void* q4, const float* scales, void* w, int N, int K, int group, bool bf16,
                                 cudaStream_t st) {
  const long long n8 = static_cast<long long>(N) * K / 8;
  return bf16 ? launch(dequantize_w4_kernel<__nv_bfloat16>, dim3(blocks_for(n8, 256)), dim3(256), 0, st,
                       static_cast<const uint32_t*>(q4), scales, static_cast<__nv_bfloat16*>(w), n8, group)
              : launch(dequantize_w4_kernel<float>, dim3(blocks_for(n8, 256)), dim3(256), 0, st,
                       static_cast<const uint32_t*>(q4), scales, static_cast<float*>(w), n8, group);
}

cudaError_t launch_gemm_w4(const void* a, const void* q4, const float* scales, void* c, int M, int N, int K, int group,
                           bool bf16, cudaStream_t st) {
  const unsigned grid = blocks_for(static_cast<long long>(M) * N, 8);
  return bf16 ? launch(gemm_w4_simple<__nv_bfloat16>, dim3(grid), dim3(256), 0, st,
                       static_cast<const __nv_bfloat16*>(a), static_cast<const uint32_t*>(q4), scales,
                       static_cast<__nv_bfloat16*>(c), M, N, K, group)
              : launch(gemm_w4_simple<float>, dim3(grid), dim3(256), 0, st, static_cast<const float*>(a),
                       static_cast<const uint32_t*>(q4), scales, static_cast<float*>(c), M, N, K, group);
}

}  // namespace hy
