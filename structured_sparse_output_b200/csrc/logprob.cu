// logprob.cu -- softmax reading of a layer's logits on sm_100a: log probabilities
// of given labels, entropy and top alternatives of every row, and the gradient.
//
// Row z[0..N) (a masked label is -inf): m = max z, S = sum e^(z-m),
// T = sum e^(z-m) (m-z);  lse = m + log S,  log p_j = (z_j - m) - log S,
// entropy = log S + T / S (two terms >= 0: nothing cancels).  Segments of a row
// join by rescaling S and T to the common maximum.
// Rank order of the alternatives: larger logit first, equal logits by smaller id.
// Gradient: dz_j = sum_{i: id_i = j} g_i - p_j (sum_i g_i + gH (log p_j + entropy)).
#include "common.cuh"

namespace haste {
namespace logprob {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxK = 64;
constexpr int kV = 4;        // 16-byte vectors per thread: a segment of 64 bytes a thread, held in registers
constexpr int kGroups = 128;  // groups of threads whose maxima bound the k-th best logit

struct Args {
  const void* logits;  // [B, N]
  int64_t N;
  const int32_t* row_ptr;  // NULL: no given labels
  const int32_t* ids;
  int64_t nnz;
  int k;
  int n_seg;  // segments of a row
  float* logp;
  float* lse;
  float* entropy;
  float* top_logp;
  int32_t* top_id;
  float4* part;    // [B, n_seg] (m, S, T): partial sums when n_seg > 1
  uint64_t* keys;  // [B, n_seg, k] rank keys of the segment's best, descending, 0 = none
};

struct GradArgs {
  const void* logits;
  int64_t N;
  int n_seg;
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

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// The vectors of a row: 16-byte pieces of memory, the first and last of which may
// reach beyond the row (rows start where they start: an odd N leaves only every
// eighth bf16 row on a boundary).
template <typename T>
struct Row {
  static constexpr int kE = 16 / sizeof(T);  // elements of a vector
  const T* z;
  int64_t N;
  int head;  // elements of the first vector before the row
  __device__ Row(const void* base, int64_t b, int64_t n) : z(static_cast<const T*>(base) + b * n), N(n) {
    head = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
  }
  // column of the first element of vector v (negative in the first vector of a row off the boundary)
  __device__ int64_t column(int64_t v) const { return v * kE - head; }
  __device__ uint4 load(int64_t v) const {
    const int64_t j = column(v);
    if (j >= 0 && j + kE <= N) return *reinterpret_cast<const uint4*>(z + j);
    constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
    uint32_t u[4] = {kNone, kNone, kNone, kNone};
    if (j < N)
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (j + i >= 0 && j + i < N) {
          if constexpr (sizeof(T) == 2) {
            const uint32_t s = __bfloat16_as_ushort(z[j + i]);
            u[i / 2] = (i & 1) ? (u[i / 2] & 0xffffu) | (s << 16) : (u[i / 2] & 0xffff0000u) | s;
          } else {
            u[i] = __float_as_uint(z[j + i]);
          }
        }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <typename T>
__device__ __forceinline__ void unpack(const uint4& r, float (&v)[16 / sizeof(T)]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(u[i]);
    }
  }
}
// Vectors that a row of N elements can touch, given where the first row starts.
template <typename T>
inline int64_t row_vectors(int64_t N, bool on_boundary) {
  constexpr int kE = 16 / sizeof(T);
  return N % kE == 0 ? N / kE + (on_boundary ? 0 : 1) : (N + kE - 2) / kE + 1;
}

// The largest tau such that at least k of the block's keys are >= tau, and exactly
// k when the keys are distinct; key[i] = 0 does not count.  At least k must exist.
template <int kN>
__device__ __forceinline__ uint64_t kth_key(const uint64_t (&key)[kN], int k) {
  uint64_t tau = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t c = tau | (1ull << bit);
    int n = 0;
    if constexpr (kN == 1) {
      n = __syncthreads_count(key[0] >= c);
    } else {
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) mine += key[i] >= c;
      // counts of up to kN per thread: one vote per bit of the count
#pragma unroll
      for (int s = 0; (1 << s) <= kN; ++s) n += __syncthreads_count((mine >> s) & 1) << s;
    }
    if (n >= k) tau = c;
    if (n == k) break;
  }
  return tau;
}

// What a row needs besides its sums, from m, S and T of the whole row.
struct RowStats {
  float m, log_s;
  bool none;
  __device__ float logp(float v) const { return none ? -INFINITY : (v - m) - log_s; }
};
__device__ __forceinline__ RowStats row_stats(float m, float S) {
  RowStats r;
  r.m = m;
  r.none = m == -INFINITY;
  r.log_s = m < INFINITY ? logf(S) : NAN;  // a NaN or +inf in the row
  return r;
}
template <typename T>
__device__ __forceinline__ void write_row(const Args& a, int64_t b, const T* z, const RowStats& r, float S, float Tt) {
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[b] = r.none ? -INFINITY : r.m + r.log_s;
    if (a.entropy) a.entropy[b] = r.none ? 0.f : r.log_s + Tt / S;
  }
  int64_t p0, p1;
  row_list(a.row_ptr, a.nnz, b, p0, p1);
  for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) {
    const int64_t id = a.ids[p];
    a.logp[p] = id >= 0 && id < a.N ? r.logp(Elem<T>::to_f(z[id])) : NAN;
  }
}

// One CTA per segment of a row.  The segment stays in registers: its maximum, then
// its sums and its k best.  The k-th largest of the maxima of 128 groups of threads
// is a lower bound of the k-th best logit, so only the few logits at or above it
// compete; where too many do (long runs of equal logits), or a NaN hides a maximum,
// the k-th best thread maximum decides, above which lie at most k threads' logits.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 8) k_logprob(Args a) {
  constexpr int kE = 16 / sizeof(T), kWarps = kThreads / 32, kLanes = kThreads / kGroups;
  constexpr int kCand = kMaxK * kV * kE;  // the logits of k threads
  __shared__ float warp_m[kWarps], warp_s[kWarps], warp_t[kWarps];
  __shared__ __align__(16) float group_m[kGroups];
  __shared__ float tau_s;
  __shared__ int n_cand;
  __shared__ uint64_t cand[kCand];
  const int64_t b = blockIdx.x / a.n_seg;
  const int seg = blockIdx.x % a.n_seg, t = threadIdx.x;
  const Row<T> row(a.logits, b, a.N);
  const int64_t v0 = (int64_t)seg * (kThreads * kV) + t;

  uint4 raw[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) raw[i] = row.load(v0 + i * kThreads);
  if (t == 0) n_cand = 0;
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    float v[kE];
    unpack<T>(raw[i], v);
#pragma unroll
    for (int e = 0; e < kE; ++e) mine = max_nan(mine, v[e]);
  }
  float g = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o == kLanes && t % kLanes == 0) group_m[t / kLanes] = g;
    g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
  }
  if ((t & 31) == 0) warp_m[t >> 5] = g;
  __syncthreads();
  float m = warp_m[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) m = max_nan(m, warp_m[i]);

  // the k-th largest group maximum
  if (a.k > 0 && t < kGroups) {
    const float v = group_m[t];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < kGroups; i += 4) {
      const float4 o = *reinterpret_cast<const float4*>(&group_m[i]);
      rank += (o.x > v || (o.x == v && i < t)) + (o.y > v || (o.y == v && i + 1 < t)) +
              (o.z > v || (o.z == v && i + 2 < t)) + (o.w > v || (o.w == v && i + 3 < t));
    }
    if (rank == a.k - 1) tau_s = v;
  }
  float S = 0.f, Tt = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    float v[kE];
    unpack<T>(raw[i], v);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float d = fmaxf(v[e] - m, -200.f), x = ex2(d * kLog2e);  // -inf: e^-200 is 0 in fp32
      S += x;
      Tt = fmaf(-x, d, Tt);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, o);
    Tt += __shfl_xor_sync(0xffffffffu, Tt, o);
  }
  if ((t & 31) == 0) {
    warp_s[t >> 5] = S;
    warp_t[t >> 5] = Tt;
  }
  __syncthreads();
  S = Tt = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    S += warp_s[i];
    Tt += warp_t[i];
  }
  const RowStats st = row_stats(m, S);
  if (a.n_seg == 1) write_row(a, b, row.z, st, S, Tt);
  else if (t == 0) a.part[blockIdx.x] = make_float4(m, S, Tt, 0.f);
  if (a.k == 0) return;

  // the competing logits; a thread holds one only if its maximum does
  auto collect = [&](auto keep) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t j = row.column(v0 + i * kThreads);
      float v[kE];
      unpack<T>(raw[i], v);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (j + e >= 0 && j + e < a.N && keep(v[e], (uint32_t)(j + e))) {
          const int at = atomicAdd(&n_cand, 1);
          if (at < kCand) cand[at] = rank_key(v[e], (uint32_t)(j + e));
        }
    }
  };
  const bool odd = !(m == m);  // a NaN: the group maxima bound nothing
  if (!odd) {
    const float tau = tau_s;
    if (mine >= tau) collect([&](float v, uint32_t) { return v >= tau; });
  }
  __syncthreads();
  int c = n_cand;
  if (odd || c > 256) {
    uint64_t best[1] = {0};
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t j = row.column(v0 + i * kThreads);
      float v[kE];
      unpack<T>(raw[i], v);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (j + e >= 0 && j + e < a.N) {
          const uint64_t key = rank_key(v[e], (uint32_t)(j + e));
          if (key > best[0]) best[0] = key;
        }
    }
    const int live = __syncthreads_count(best[0] != 0);
    const uint64_t tau = live > a.k ? kth_key(best, a.k) : 1;
    __syncthreads();
    if (t == 0) n_cand = 0;
    __syncthreads();
    if (best[0] >= tau) collect([&](float v, uint32_t id) { return rank_key(v, id) >= tau; });
    __syncthreads();
    c = n_cand;
  }
  uint64_t* keys = a.keys + (int64_t)blockIdx.x * a.k;
  auto emit = [&](int rank, uint64_t key) {
    if (a.n_seg == 1) {
      a.top_id[b * a.k + rank] = (int32_t)key_id(key);
      a.top_logp[b * a.k + rank] = st.logp(key_value(key));
    } else {
      keys[rank] = key;
    }
  };
  for (int i = t; i < c; i += kThreads) {
    const uint64_t key = cand[i];
    int rank = 0;
    for (int j = 0; j < c; ++j) rank += cand[j] > key;
    if (rank < a.k) emit(rank, key);
  }
  if (a.n_seg > 1)  // a short last segment
    for (int r = c + t; r < a.k; r += kThreads) keys[r] = 0;
}

// One CTA per row joins its segments.
constexpr int kJoinThreads = 512;
constexpr int kJoinCand = kMaxK * kMaxK;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) k_logprob_join(Args a) {
  __shared__ float red[3][kJoinThreads / 32];
  __shared__ uint64_t cand[kJoinCand];
  __shared__ uint64_t best[kMaxK];
  __shared__ int n_cand, n_best;
  const int64_t b = blockIdx.x;
  const int t = threadIdx.x, n = a.n_seg, k = a.k;
  const float4* part = a.part + b * n;
  float m = -INFINITY;
  for (int i = t; i < n; i += kJoinThreads) m = max_nan(m, part[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((t & 31) == 0) red[0][t >> 5] = m;
  if (t == 0) n_cand = n_best = 0;
  __syncthreads();
  for (int i = 0; i < kJoinThreads / 32; ++i) m = max_nan(m, red[0][i]);
  float S = 0.f, Tt = 0.f;
  for (int i = t; i < n; i += kJoinThreads) {
    const float4 p = part[i];
    if (p.x > -INFINITY) {
      const float d = p.x - m, w = expf(d);
      S += w * p.y;
      Tt += w * (p.z - p.y * fmaxf(d, -200.f));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, o);
    Tt += __shfl_xor_sync(0xffffffffu, Tt, o);
  }
  if ((t & 31) == 0) {
    red[1][t >> 5] = S;
    red[2][t >> 5] = Tt;
  }
  __syncthreads();
  S = Tt = 0.f;
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    S += red[1][i];
    Tt += red[2][i];
  }
  const RowStats st = row_stats(m, S);
  write_row(a, b, static_cast<const T*>(a.logits) + b * a.N, st, S, Tt);
  if (k == 0) return;
  // with more segments than alternatives, only the segments whose best is among the
  // k best of the segments' bests hold any
  const uint64_t* keys = a.keys + b * n * k;
  uint64_t tau = 1;
  if (n > k) {
    uint64_t top = 0;  // k-th largest of the heads, each thread's heads in turn
    uint64_t lo = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t c = lo | (1ull << bit);
      int cnt = 0;
      for (int i0 = 0; i0 < n; i0 += kJoinThreads) cnt += __syncthreads_count(i0 + t < n && keys[(int64_t)(i0 + t) * k] >= c);
      if (cnt >= k) lo = c;
      if (cnt == k) break;
    }
    top = lo;
    tau = top > 0 ? top : 1;
  }
  for (int64_t i = t; i < (int64_t)n * k; i += kJoinThreads) {
    const uint64_t key = keys[i];
    if (key >= tau) cand[atomicAdd(&n_cand, 1)] = key;
  }
  __syncthreads();
  const int c = n_cand;
  constexpr int kPer = kJoinCand / kJoinThreads;
  uint64_t mine[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine[i] = i * kJoinThreads + t < c ? cand[i * kJoinThreads + t] : 0;
  const uint64_t last = kth_key(mine, k);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (mine[i] >= last && mine[i] != 0) best[atomicAdd(&n_best, 1)] = mine[i];
  __syncthreads();
  if (t < k) {
    const uint64_t key = best[t];
    int rank = 0;
    for (int j = 0; j < k; ++j) rank += best[j] > key;
    a.top_id[b * k + rank] = (int32_t)key_id(key);
    a.top_logp[b * k + rank] = st.logp(key_value(key));
  }
}

// One CTA per segment of a row: the dense term, then the given labels in it.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 8) k_logprob_grad(GradArgs a) {
  constexpr int kE = 16 / sizeof(T);
  const int64_t b = blockIdx.x / a.n_seg;
  const int seg = blockIdx.x % a.n_seg, t = threadIdx.x;
  const Row<T> row(a.logits, b, a.N);
  T* dz = static_cast<T*>(a.d_logits) + b * a.N;
  const int64_t v0 = (int64_t)seg * (kThreads * kV) + t;
  uint4 raw[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) raw[i] = row.load(v0 + i * kThreads);
  const float lse = a.lse[b];
  const bool none = lse == -INFINITY;
  const float gH = a.d_entropy ? a.d_entropy[b] : 0.f, H = a.d_entropy ? a.entropy[b] : 0.f;
  int64_t p0, p1;
  row_list(a.row_ptr, a.nnz, b, p0, p1);
  float G = 0.f;  // every warp sums the list in the same order
  for (int64_t p = p0 + (t & 31); p < p1; p += 32) {
    const int64_t id = a.ids[p];
    if (id >= 0 && id < a.N) G += a.d_logp[p];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) G += __shfl_xor_sync(0xffffffffu, G, o);
  auto dense = [&](float v) {
    const float lp = v - lse, p = ex2(lp * kLog2e);
    return p == 0.f ? 0.f : -p * fmaf(gH, lp + H, G);
  };
  // the output may sit on the 16-byte boundary differently from the input
  const bool vec = ((reinterpret_cast<uintptr_t>(row.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int64_t j = row.column(v0 + i * kThreads);
    if (j >= a.N) break;
    float v[kE];
    unpack<T>(raw[i], v);
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] = none ? 0.f : dense(v[e]);
    if (vec && j >= 0 && j + kE <= a.N) {
      uint4 o;
      if constexpr (sizeof(T) == 2)
        o = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      else
        o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      *reinterpret_cast<uint4*>(dz + j) = o;
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (j + e >= 0 && j + e < a.N) dz[j + e] = Elem<T>::from_f(v[e]);
    }
  }
  if (p0 == p1 || none) return;
  __syncthreads();
  const int64_t c0 = row.column((int64_t)seg * (kThreads * kV)), c1 = c0 + (int64_t)kThreads * kV * kE;
  for (int64_t p = p0 + t; p < p1; p += kThreads) {
    const int64_t id = a.ids[p];
    if (id < 0 || id >= a.N || id < c0 || id >= c1) continue;
    float g = 0.f;
    bool first = true;
    for (int64_t q = p0; q < p1; ++q)
      if (a.ids[q] == id) {
        if (q < p) first = false;
        g += a.d_logp[q];
      }
    if (first) dz[id] = Elem<T>::from_f(g + dense(Elem<T>::to_f(row.z[id])));
  }
}

// Threads of a segment's CTA: rows that 128 threads hold whole take one such CTA.
inline int seg_threads(int64_t vectors) { return vectors <= 128 * kV ? 128 : 512; }
inline int64_t segments(int64_t vectors) {
  const int64_t per = (int64_t)seg_threads(vectors) * kV;
  return (vectors + per - 1) / per;
}

template <typename T>
cudaError_t launch(int B, int threads, const Args& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)B * a.n_seg);
  if (threads == 128) k_logprob<T, 128><<<grid, 128, 0, st>>>(a);
  else k_logprob<T, 512><<<grid, 512, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_join(int B, const Args& a, cudaStream_t st) {
  k_logprob_join<T><<<B, kJoinThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grad(int B, int threads, const GradArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)B * a.n_seg);
  if (threads == 128) k_logprob_grad<T, 128><<<grid, 128, 0, st>>>(a);
  else k_logprob_grad<T, 512><<<grid, 512, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace logprob
}  // namespace haste
