// logprob.cu -- softmax reading of a layer's logits on sm_100a: log probabilities
// of given labels, entropy and top alternatives of every row, and the gradient.
//
// Row z[0..N) (a masked label is -inf): m = max z, S = sum e^(z-m),
// T = sum e^(z-m) (m-z);  lse = m + log S,  log p_j = (z_j - m) - log S,
// entropy = log S + T / S (two terms >= 0: nothing cancels).
// Rank order of the alternatives: larger logit first, equal logits by smaller id.
// Gradient: dz_j = sum_{i: id_i = j} g_i - p_j (sum_i g_i + gH (log p_j + entropy)).
#include "common.cuh"

namespace haste {
namespace logprob {

constexpr int kThreads = 256;

struct Args {
  const void* logits;  // [B, N]
  int64_t N;
  const int32_t* row_ptr;  // NULL: no given labels
  const int32_t* ids;
  int64_t nnz;
  int k;
  float* logp;
  float* lse;
  float* entropy;
  float* top_logp;
  int32_t* top_id;
};

struct GradArgs {
  const void* logits;
  int64_t N;
  const float* lse;
  const float* entropy;
  const int32_t* row_ptr;
  const int32_t* ids;
  int64_t nnz;
  const float* d_logp;
  const float* d_entropy;
  void* d_logits;
};

// A whole number that orders (z, id) as the alternatives are ranked: larger z
// first (-0 as 0, NaN as -inf), then smaller id.  0 is below every pair.
__device__ __forceinline__ uint64_t rank_key(float z, uint32_t id) {
  z = z == z ? z + 0.f : -INFINITY;
  const uint32_t u = __float_as_uint(z);
  const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)o << 32) | (uint32_t)~id;
}
__device__ __forceinline__ uint32_t key_id(uint64_t key) { return ~(uint32_t)key; }
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

// The given labels of row b: [begin, end) of the lists, within [0, nnz] whatever
// row_ptr holds.
__device__ __forceinline__ void row_list(const int32_t* row_ptr, int64_t nnz, int64_t b, int64_t& begin,
                                         int64_t& end) {
  begin = end = 0;
  if (!row_ptr) return;
  begin = row_ptr[b];
  end = row_ptr[b + 1];
  begin = begin < 0 ? 0 : begin > nnz ? nnz : begin;
  end = end < begin ? begin : end > nnz ? nnz : end;
}

template <typename Op, typename V>
__device__ __forceinline__ V block_reduce(V v, V* red, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < (int)blockDim.x / 32; ++i) v = op(v, red[i]);
  return v;
}

// One CTA per row; the row is read once for the maximum, once for the sums and
// once for each alternative.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_logprob(Args a) {
  __shared__ float red_f[kThreads / 32];
  __shared__ uint64_t red_u[kThreads / 32];
  const int64_t b = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + b * a.N;
  auto fmx = [](float x, float y) { return fmaxf(x, y); };
  auto add = [](float x, float y) { return x + y; };
  float m = -INFINITY, bad = 0.f;
  for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
    const float v = Elem<T>::to_f(z[j]);
    m = fmaxf(m, v);
    if (!(v < INFINITY)) bad = 1.f;  // NaN or +inf
  }
  m = block_reduce(m, red_f, fmx);
  bad = block_reduce(bad, red_f, fmx);
  float S = 0.f, Tt = 0.f;
  if (m > -INFINITY)
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float d = Elem<T>::to_f(z[j]) - m, e = expf(d);
      S += e;
      if (e > 0.f) Tt -= e * d;
    }
  S = block_reduce(S, red_f, add);
  Tt = block_reduce(Tt, red_f, add);
  const float logS = bad > 0.f ? NAN : logf(S);
  const bool none = m == -INFINITY && !(bad > 0.f);
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[b] = none ? -INFINITY : m + logS;
    if (a.entropy) a.entropy[b] = none ? 0.f : logS + Tt / S;
  }
  auto logp = [&](float v) { return none ? -INFINITY : (v - m) - logS; };
  int64_t p0, p1;
  row_list(a.row_ptr, a.nnz, b, p0, p1);
  for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) {
    const int64_t id = a.ids[p];
    a.logp[p] = id >= 0 && id < a.N ? logp(Elem<T>::to_f(z[id])) : NAN;
  }
  uint64_t last = ~0ull;
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = 0;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const uint64_t key = rank_key(Elem<T>::to_f(z[j]), (uint32_t)j);
      if (key < last && key > best) best = key;
    }
    last = block_reduce(best, red_u, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
    if (threadIdx.x == 0) {
      a.top_id[b * a.k + r] = (int32_t)key_id(last);
      a.top_logp[b * a.k + r] = logp(key_value(last));
    }
  }
}

// One CTA per (row, run of columns): the dense term of its columns, then the
// given labels that fall into them.
constexpr int kGradCols = 2048;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_logprob_grad(GradArgs a) {
  __shared__ float red[kThreads / 32];
  const int64_t b = blockIdx.y;
  const T* z = static_cast<const T*>(a.logits) + b * a.N;
  T* dz = static_cast<T*>(a.d_logits) + b * a.N;
  const int64_t c0 = (int64_t)blockIdx.x * kGradCols, c1 = c0 + kGradCols < a.N ? c0 + kGradCols : a.N;
  int64_t p0, p1;
  row_list(a.row_ptr, a.nnz, b, p0, p1);
  float G = 0.f;
  for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x)
    if (a.ids[p] >= 0 && a.ids[p] < a.N) G += a.d_logp[p];
  G = block_reduce(G, red, [](float x, float y) { return x + y; });
  const float lse = a.lse[b];
  const bool none = lse == -INFINITY;
  const float gH = a.d_entropy ? a.d_entropy[b] : 0.f, H = a.d_entropy ? a.entropy[b] : 0.f;
  auto dense = [&](float v) {
    const float lp = v - lse, p = expf(lp);
    return p == 0.f ? 0.f : -p * (G + gH * (lp + H));
  };
  for (int64_t j = c0 + threadIdx.x; j < c1; j += blockDim.x)
    dz[j] = Elem<T>::from_f(none ? 0.f : dense(Elem<T>::to_f(z[j])));
  __syncthreads();
  if (none) return;
  for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) {
    const int64_t id = a.ids[p];
    if (id < c0 || id >= c1) continue;
    float g = 0.f;
    bool first = true;
    for (int64_t q = p0; q < p1; ++q)
      if (a.ids[q] == id) {
        if (q < p) first = false;
        g += a.d_logp[q];
      }
    if (first) dz[id] = Elem<T>::from_f(g + dense(Elem<T>::to_f(z[id])));
  }
}

template <typename T>
cudaError_t launch(int B, const Args& a, cudaStream_t st) {
  k_logprob<T><<<B, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grad(int B, const GradArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.N + kGradCols - 1) / kGradCols), B);
  k_logprob_grad<T><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace logprob
}  // namespace haste
