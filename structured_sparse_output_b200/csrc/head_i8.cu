// head_i8.cu -- the dense head in 8-bit integers on sm_100a.
//
// Row quantisation (weights: one scale per label; features: one per sample):
// s = max|x| / 127 rounded once to fp32, q = the exact quotient x / s rounded half
// to even.  Product: z[b, h] = (sum_f qx[b, f] qw[h, f]) * (sx[b] * sw[h]), the sum
// exact in 32 bits.
#include "common.cuh"

namespace haste {
namespace head8 {

constexpr int kThreads = 256;
constexpr int kMaxN = 131072;  // 127 * 127 * kMaxN < 2^31

__host__ __device__ inline int pitch(int n) { return (n + 15) / 16 * 16; }

// x / s rounded half to even, clamped to +-127, for s > 0 (127 s is about the
// row's maximum, or s lost bits as a subnormal).  The rounded fp32 quotient can
// land on the wrong side of a half; the remainder x - q s is exact in fp32 (a
// multiple of half an ulp of s, at most about s), so it decides.
__device__ __forceinline__ int quantise(float x, float s) {
  float q = rintf(__fdiv_rn(x, s));
  if (fabsf(q) > 127.f) return q > 0.f ? 127 : -127;
  const float r2 = 2.f * fmaf(-q, s, x);
  const bool odd = ((int)q & 1) != 0;
  if (r2 > s || (r2 == s && odd)) q += 1.f;
  else if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// One CTA per row.  A row with a NaN or an infinity gets the scale NaN and zeros.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(const T* __restrict__ x, int n, int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
  __shared__ float red[kThreads / 32];
  const int64_t r = blockIdx.x;
  const int ld = pitch(n);
  const T* xr = x + r * n;
  float m = 0.f;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const float v = fabsf(Elem<T>::to_f(xr[i]));
    m = v <= m ? m : v < INFINITY ? v : INFINITY;  // NaN counts as infinite
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, red[i]);
  const float s = m < INFINITY ? __fdiv_rn(m, 127.f) : NAN;
  for (int i = threadIdx.x; i < ld; i += blockDim.x)
    q[r * ld + i] = (int8_t)(i < n && s > 0.f ? quantise(Elem<T>::to_f(xr[i]), s) : 0);
  if (threadIdx.x == 0) scale[r] = s;
}

// One thread per logit.
template <typename O>
__global__ void __launch_bounds__(128) k_head_i8(int H, int ld, const int8_t* __restrict__ qx,
                                                 const float* __restrict__ sx, const int8_t* __restrict__ qw,
                                                 const float* __restrict__ sw, O* __restrict__ out) {
  const int64_t h = blockIdx.x * 128ll + threadIdx.x, b = blockIdx.y;
  if (h >= H) return;
  const int* x4 = reinterpret_cast<const int*>(qx + b * ld);
  const int* w4 = reinterpret_cast<const int*>(qw + h * ld);
  int acc = 0;
  for (int i = 0; i < ld / 4; ++i) acc = __dp4a(x4[i], w4[i], acc);
  out[b * H + h] = Elem<O>::from_f((float)acc * (sx[b] * sw[h]));
}

template <typename T>
cudaError_t launch_quantize(int64_t rows, int n, const void* x, int8_t* q, float* scale, cudaStream_t st) {
  k_quantize_rows<T><<<(unsigned)rows, kThreads, 0, st>>>(static_cast<const T*>(x), n, q, scale);
  return cudaGetLastError();
}

template <typename O>
cudaError_t launch_product(int B, int H, int ld, const int8_t* qx, const float* sx, const int8_t* qw, const float* sw,
                           void* out, cudaStream_t st) {
  k_head_i8<O><<<dim3((unsigned)((H + 127) / 128), B), 128, 0, st>>>(H, ld, qx, sx, qw, sw, static_cast<O*>(out));
  return cudaGetLastError();
}

}  // namespace head8
}  // namespace haste
