// logprob.cu -- softmax reading of a layer's logits on sm_100a: log probabilities
// of given labels, entropy and top alternatives of every row, and the gradient.
//
// Row z[0..N) (a masked label is -inf): m = max z, S = sum e^(z-m),
// T = sum e^(z-m) (m-z);  lse = m + log S,  log p_j = (z_j - m) - log S,
// entropy = log S + T / S (two terms >= 0: nothing cancels).  Segments of a row
// join by rescaling S and T to the common maximum.
// Rank order of the alternatives: larger logit first, equal logits by smaller id.
// Gradient: dz_j = sum_{i: id_i = j} g_i - p_j (sum_i g_i + gH (log p_j + entropy)).
//
// Times in this file are of one call among others in a CUDA graph on the same inputs, those
// of less than about 60 MB in L2; a program's calls one by one take up to 7 % longer at the
// largest sizes (256 x 670,208: 76 us where 70 stand here, the gradient 117 for 110).
#include <cfloat>

#include "common.cuh"
#include "launch.cuh"

namespace haste {
namespace logprob {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxK = 64;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kV = 4;                     // 16-byte vectors of a thread in a block of a row
constexpr int kBlock = kThreads * kV;     // vectors of a block: 16 KB of a row
constexpr int kCap = 128;                 // competing logits that a warp keeps
constexpr int kRoom = 96;                 // and how many at most after it drops some
constexpr int kRing = 2;                  // blocks in flight or in use
constexpr int kList = 128;                // vectors that a warp notes before it looks into them
constexpr int kMaxRuns = 1024;            // runs of a row
constexpr int kFew = 16;                  // alternatives for which the bound is raised less often

struct Args {
  const void* logits;  // [B, N]
  int64_t N;
  const int32_t* row_ptr;  // NULL: no given labels
  const int32_t* ids;
  int64_t nnz;
  int k;
  int n_run;  // runs that a row is split into, one CTA each
  // Rows too short to give k groups of threads a logit: the bound takes groups of one
  // thread, or (a few hundred logits) every logit is ranked without one.
  int thin, rank_all;
  float* logp;
  float* lse;
  float* entropy;
  float* top_logp;
  int32_t* top_id;
  float4* part;    // [B, n_run] (mu, S, Y): the runs' sums when n_run > 1
  uint64_t* keys;  // [B, n_run, k] rank keys of the run's best, descending, 0 = none
};

struct GradArgs {
  const void* logits;
  int64_t N;
  int n_run;
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
__device__ __forceinline__ uint32_t rank_value(float z) {
  z = z == z ? z + 0.f : -INFINITY;
  const uint32_t u = __float_as_uint(z);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t rank_key(float z, uint32_t id) {
  return ((uint64_t)rank_value(z) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ uint32_t key_id(uint64_t key) { return ~(uint32_t)key; }
__device__ __forceinline__ float key_value(uint64_t key) {  // -inf for what is below every pair
  const uint32_t o = (uint32_t)(key >> 32);
  if (o < 0x007fffffu) return -INFINITY;
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {  // 2^x, 0 below the normal numbers
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 numbers in one register pair: one instruction adds or multiplies both.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f2 p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 ex2_2(f2 p) {
  float a, b;
  unpair(p, a, b);
  return pair(ex2(a), ex2(b));
}

// The given labels of row b: [begin, end) of the lists, within [0, nnz] whatever
// row_ptr holds.
__device__ __forceinline__ void row_list(const int32_t* row_ptr, int64_t nnz, int64_t b, int64_t& begin,
                                         int64_t& end) {
  begin = end = 0;
  if (!row_ptr) return;
  begin = __ldcg(row_ptr + b);
  end = __ldcg(row_ptr + b + 1);
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
  uint32_t N;
  int head;  // elements of the first vector before the row
  __device__ Row(const void* base, int64_t b, int64_t n) : z(static_cast<const T*>(base) + b * n), N((uint32_t)n) {
    head = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
  }
  // column of the first element of vector v (negative in the first vector of a row off the boundary)
  __device__ int64_t column(uint32_t v) const { return (int64_t)v * kE - head; }
  __device__ bool whole(int64_t j) const { return j >= 0 && j + kE <= (int64_t)N; }
  __device__ uint4 load(uint32_t v) const {
    const int64_t j = column(v);
    if (whole(j)) return *reinterpret_cast<const uint4*>(z + j);
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

// The k-th largest of the block's keys (kN per thread, distinct but for 0, which
// does not count; at least k of them), or a lower bound that k keys reach and no
// other: digits of 8 bits from the top, each by a histogram of the keys that share
// the digits before.
template <int kN>
__device__ uint64_t kth_key(const uint64_t (&key)[kN], int k, int* hist, int* found) {
  uint64_t prefix = 0, mask = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      // one addition for the lanes that share a digit: most do in the first digits
      const bool in = key[i] != 0 && (key[i] & mask) == prefix;
      const int digit = in ? (int)(key[i] >> shift) & 255 : 256;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && (int)(threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane l: bins 8 (31 - l) .. + 7, so that a prefix sum counts from the top
      const int* bin = hist + 8 * (31 - threadIdx.x);
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += bin[i];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)threadIdx.x >= o) upto += v;
      }
      int above = upto - mine;
      if (above < k && upto >= k) {
        int i = 7;
        while (above + bin[i] < k) above += bin[i--];
        found[0] = 8 * (31 - threadIdx.x) + i;
        found[1] = k - above;
        found[2] = bin[i] == k - above;
      }
    }
    __syncthreads();
    prefix |= (uint64_t)found[0] << shift;
    mask |= (uint64_t)255 << shift;
    k = found[1];
    if (found[2]) break;
  }
  return prefix;
}

// What a row needs besides its sums, from m, S and T of the whole row (S = 0 only
// where every logit is -inf: the largest contributes 1).
struct RowStats {
  float m, log_s;
  bool none;
  __device__ float logp(float v) const { return none ? -INFINITY : (v - m) - log_s; }
};
__device__ __forceinline__ RowStats row_stats(float m, float S) {
  RowStats r;
  r.m = m;
  r.none = S == 0.f;
  r.log_s = logf(S);  // NaN for a NaN or +inf in the row
  return r;
}
// The given labels of a row: each thread's first one is loaded early, since its logit
// is found through two loads before it.  (From L2: the join loads them before it waits
// for the kernel before it.)
template <typename T, int kStep>
struct Given {  // for kStep threads of a row
  int64_t begin, end;
  int t;
  float z;  // of entry begin + t; NaN for an id outside the row
  __device__ float logit(const Args& a, const T* row, int64_t p) const {
    const int64_t id = __ldcg(a.ids + p);
    return id >= 0 && id < a.N ? Elem<T>::to_f(__ldcg(row + id)) : NAN;
  }
  __device__ Given(const Args& a, int64_t b, const T* row) {
    row_list(a.row_ptr, a.nnz, b, begin, end);
    t = threadIdx.x % kStep;
    z = begin + t < end ? logit(a, row, begin + t) : 0.f;
  }
  // What a row gives besides its alternatives.
  __device__ void write(const Args& a, int64_t b, const T* row, const RowStats& r, float S, float Tt) const {
    if (t == 0) {
      if (a.lse) a.lse[b] = r.none ? -INFINITY : r.m + r.log_s;
      if (a.entropy) a.entropy[b] = r.none ? 0.f : r.log_s + Tt / S;
    }
    for (int64_t p = begin + t; p < end; p += kStep) {
      const float v = p == begin + t ? z : logit(a, row, p);
      a.logp[p] = v == v ? r.logp(v) : NAN;
    }
  }
};

// Competing logits of one warp: the keys at or above `tau`, of which fewer than k
// can be beaten by the others.
struct Keep {
  int n;
  bool strict;  // k kept keys reach tau: a later equal logit, of a larger id, is beaten
  uint64_t tau;
  // The value that a logit has to reach from here on.
  __device__ float bar() const { return key_value(strict ? ((tau >> 32) + 1) << 32 : tau); }
  __device__ void raise(uint64_t to) {
    if (to > tau) {
      tau = to;
      strict = false;
    }
  }
};
// -inf and NaN compete only where a run has fewer than k other logits.
constexpr uint64_t kFinite = (uint64_t)0x00800000u << 32;

// Raise tau until at most kRoom of the warp's keys reach it, and still k do.
__device__ __noinline__ Keep shrink(uint64_t* buf, Keep s, int k) {
  const int lane = threadIdx.x & 31;
  uint64_t key[kCap / 32];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kCap / 32; ++i) key[i] = i * 32 + lane < s.n ? buf[i * 32 + lane] : 0;
  uint64_t c = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t up = c | (1ull << bit);
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < kCap / 32; ++i) cnt += __popc(__ballot_sync(0xffffffffu, key[i] >= up));
    if (cnt >= k) c = up;
    if (cnt >= k && cnt <= kRoom) break;
  }
  int at = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kCap / 32; ++i) {
    const bool in = key[i] >= c && key[i] != 0;
    const uint32_t who = __ballot_sync(0xffffffffu, in);
    if (in) buf[at + __popc(who & ((1u << lane) - 1))] = key[i];
    at += __popc(who);
  }
  __syncwarp();
  return Keep{at, c >= s.tau || s.strict, c > s.tau ? c : s.tau};
}

// Add the logits of one vector of every lane (of those with `live`) that reach tau.
template <typename T>
__device__ __noinline__ Keep take(uint64_t* buf, Keep s, uint4 raw, bool live, int64_t j, uint32_t N, int k) {
  constexpr int kE = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  uint32_t hit = 0;
  if (live) {
    const float bar = s.bar();
    float v[kE];
    unpack<T>(raw, v);
#pragma unroll
    for (int e = 0; e < kE; ++e) hit |= v[e] >= bar ? 1u << e : 0u;
  }
  while (__any_sync(0xffffffffu, hit != 0)) {
    uint64_t key = 0;
    if (hit) {
      const int e = __ffs(hit) - 1, wi = sizeof(T) == 2 ? e >> 1 : e;
      hit &= hit - 1;
      uint32_t u = wi == 0 ? raw.x : wi == 1 ? raw.y : wi == 2 ? raw.z : raw.w;
      if (sizeof(T) == 2) u = (e & 1) ? u & 0xffff0000u : u << 16;
      const int64_t col = j + e;
      if (col >= 0 && col < (int64_t)N) key = rank_key(__uint_as_float(u), (uint32_t)col);
    }
    uint32_t who = __ballot_sync(0xffffffffu, key >= s.tau);
    if (s.n + __popc(who) > kCap) {
      s = shrink(buf, s, k);
      who = __ballot_sync(0xffffffffu, key >= s.tau);
    }
    if (key >= s.tau) buf[s.n + __popc(who & ((1u << lane) - 1))] = key;
    s.n += __popc(who);
  }
  return s;
}

// A lower bound of the k-th best of what the block's threads have seen, from their
// maxima: the k-th largest of the maxima of kG groups of threads (k <= kG), as a
// rank value without its low 8 bits, which tell equal maxima apart.
template <int kG>
__device__ __forceinline__ uint32_t bound_of(float mx, int k, uint32_t* group, uint32_t* out) {
  constexpr int kL = kThreads / kG, kPart = kG / kL;  // lanes of a group, groups that a lane compares with
  const int t = threadIdx.x;
#pragma unroll
  for (int o = 1; o < kL; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const uint32_t mine = (rank_value(mx) & ~255u) | (uint32_t)(t / kL);
  if (t % kL == 0) group[t / kL] = mine;
  __syncthreads();
  int above = 0;
#pragma unroll
  for (int i = 0; i < kPart; i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(&group[t % kL * kPart + i]);
    above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
  }
#pragma unroll
  for (int o = 1; o < kL; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
  if (above == k - 1 && t % kL == 0) *out = mine & ~255u;
  __syncthreads();
  return *out;
}

// The same for a row that only the first 128 threads hold a vector of: groups of one.
__device__ __noinline__ uint32_t bound_thin(float mx, int k, uint32_t* group, uint32_t* out) {
  const int t = threadIdx.x;
  const uint32_t mine = (rank_value(mx) & ~255u) | (uint32_t)(t & 127);
  if (t < 128) group[t] = mine;
  __syncthreads();
  if (t < 128) {
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < 128; i += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&group[i]);
      above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    }
    if (above == k - 1) *out = mine & ~255u;
  }
  __syncthreads();
  return *out;
}

// The k largest of the keys that the block's threads hold (kN each, distinct but
// for 0, at least min(k, their number) wanted): emit(rank, key), by any thread.
template <int kN, typename Emit>
__device__ void emit_best(const uint64_t (&key)[kN], int k, int* hist, int* found, uint64_t* best, int* n_best,
                          Emit emit) {
  const uint64_t tau = kth_key(key, k, hist, found);
  if (threadIdx.x == 0) *n_best = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (key[i] != 0 && key[i] >= tau) best[atomicAdd(n_best, 1)] = key[i];
  __syncthreads();
  if ((int)threadIdx.x < k) {
    const uint64_t mine = best[threadIdx.x];
    int rank = 0;
    for (int i = 0; i < k; ++i) rank += best[i] > mine;
    emit(rank, mine);
  }
}

// References beyond it take y = (z - mu) log2(e): R would lose more than 2^-7.
constexpr float kFar = 65536.f;

// Sums around a finite reference mu, in powers of two: y = z log2(e) - R with R =
// fl(mu log2(e)), S = sum 2^y, Y = sum 2^y y.  One fused multiply-add gives y; what R
// lost in rounding is put back once, by settle().
struct Sums {
  float mu, R, S, Y;
  // R is rounded by itself: fused into a later subtraction, it would not be the R of y
  __device__ explicit Sums(float m) : mu(m), S(0.f), Y(0.f) { R = __fmul_rn(m, kLog2e); }
  // What R lost: y is (z - mu) log2(e) + lost().  Nothing beyond kFar, where y has no R.
  __device__ float lost() const { return fabsf(mu) < kFar ? fmaf(mu, kLog2e, -R) : 0.f; }
  __device__ void move(float to) {  // to >= mu
    const Sums next(to);
    // where one of the two lies beyond kFar, the sums take on what its y has and theirs not
    const float far = (mu - to) * kLog2e + (next.lost() - lost());
    const float d = fmaxf(fabsf(mu) < kFar && fabsf(to) < kFar ? R - next.R : far, -300.f), w = ex2(d);
    Y = w * fmaf(S, d, Y);
    S *= w;
    mu = to;
    R = next.R;
  }
  // S = sum e^(z - mu) and T = sum e^(z - mu) (mu - z)
  __device__ float settle() {
    const float d = lost(), w = ex2(-d);
    S *= w;
    return -kLn2 * fmaf(-d, S, w * Y);
  }
};

// -inf counts as `lo`, whose 2^y is 0: the sums then meet no infinity times 0.  A
// multiple of mu goes into the distance so that lo differs from mu in bf16, too.
__device__ __forceinline__ float floor_of(float mu) { return mu - fmaxf(200.f, 0.02f * fabsf(mu)); }

// A vector's logits as pairs, raised to the floor before they are widened: two at a
// time in bf16 (max keeps a NaN).
template <typename T>
__device__ __forceinline__ void raised(const uint4& raw, float lo, f2 (&v)[8 / sizeof(T)]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 lo2 = __float2bfloat162_rn(lo);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&u[i]), lo2);
      const uint32_t c = *reinterpret_cast<const uint32_t*>(&r);
      v[i] = pair(__uint_as_float(c << 16), __uint_as_float(c & 0xffff0000u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = pair(max_nan(__uint_as_float(u[2 * i]), lo), max_nan(__uint_as_float(u[2 * i + 1]), lo));
  }
}
// The largest logit of kN vectors; NaN is passed over.
template <typename T, int kN>
__device__ __forceinline__ float max_of(const uint4 (&r)[kN]) {
  if constexpr (sizeof(T) == 2) {
    auto h = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
    __nv_bfloat162 m = h(r[0].x);
#pragma unroll
    for (int i = 0; i < kN; ++i) m = __hmax2(m, __hmax2(__hmax2(h(r[i].x), h(r[i].y)), __hmax2(h(r[i].z), h(r[i].w))));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[i].x), __uint_as_float(r[i].y)),
                         fmaxf(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
    return m;
  }
}

// The sums of one vector around a reference beyond kFar, and before any is known.
template <typename T>
__device__ __noinline__ float2 far_sums(uint4 raw, float mu) {
  constexpr int kE = 16 / sizeof(T);
  float v[kE], S = 0.f, Y = 0.f;
  unpack<T>(raw, v);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float y = max_nan((v[e] - mu) * kLog2e, -300.f), x = ex2(y);
    S += x;
    Y = fmaf(x, y, Y);
  }
  return make_float2(S, Y);
}

// Add kN vectors, of which no logit is above s.mu, to the sums.
template <typename T, int kN>
__device__ __forceinline__ void add(Sums& s, const uint4 (&raw)[kN]) {
  constexpr int kP = 8 / sizeof(T);
  if (fabsf(s.mu) < kFar) {
    const f2 L = pair(kLog2e, kLog2e), R = pair(-s.R, -s.R);
    const float lo = floor_of(s.mu);
    f2 S2 = 0, Y2 = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      f2 v[kP];
      raised<T>(raw[i], lo, v);
#pragma unroll
      for (int e = 0; e < kP; ++e) {
        const f2 y = fma2(v[e], L, R), x = ex2_2(y);
        S2 = add2(S2, x);
        Y2 = fma2(x, y, Y2);
      }
    }
    float x, y;
    unpair(S2, x, y);
    s.S += x + y;
    unpair(Y2, x, y);
    s.Y += x + y;
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float2 r = far_sums<T>(raw[i], s.mu);
      s.S += r.x;
      s.Y += r.y;
    }
  }
}

// Fewer than k logits of columns [j0, j1) are above -inf (`have` of them): the first of
// the others, -inf or NaN, follow.  By one warp; gives the alternatives found.
template <typename T, typename Emit>
__device__ __forceinline__ int fill_others(const Row<T>& row, int64_t j0, int64_t j1, int have, int k, Emit emit) {
  const int lane = threadIdx.x & 31;
  int r = have;
  for (int64_t j = j0 + lane; r < k && j - lane < j1; j += 32) {
    const bool other = j < j1 && !(Elem<T>::to_f(row.z[j]) > -INFINITY);
    const uint32_t who = __ballot_sync(0xffffffffu, other);
    const int at = r + __popc(who & ((1u << lane) - 1));
    if (other && at < k) emit(at, rank_key(-INFINITY, (uint32_t)j));
    r += __popc(who);
  }
  return r;
}

// Look into the vectors that a warp noted (numbers within the run, which starts at
// vector v0 of the row): those from `kept` on are still in the ring.
template <typename T>
__device__ __noinline__ Keep look(uint64_t* buf, Keep s, const uint32_t* list, int n_list, const Row<T> row, uint32_t v0,
                                  const uint4* ring, uint32_t kept, int k) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  for (int i = 0; i < n_list; i += 32) {
    const bool live = i + lane < n_list;
    const uint32_t at = list[live ? i + lane : i], v = v0 + at;
    s = take<T>(buf, s, at >= kept ? ring[at % (kRing * kBlock)] : row.load(v), live, row.column(v), row.N, k);
  }
  __syncwarp();
  return s;
}

// One CTA per run of a row, block by block; every thread copies its vectors of the
// next block into its own slots of shared memory (cp.async, no barrier), which costs
// no registers.  The threads' maxima bound the k-th best logit from below: over the
// first block and again after 4, 16 .. blocks (more than 16 alternatives: after 2, 4,
// 8 .. and at the end; raising the bound costs two barriers, about 0.4 us, and leaves
// fewer logits to rank).  A warp notes the vectors whose maximum reaches the bound of
// the time, and looks into them at the end (or when its list is full).  -inf does not
// compete: where a run has fewer than k other logits, its first -inf or NaN follow.
// 256 x 670,208 bf16 logits: 58 us without alternatives (5.9 TB/s, 90% of a copy's
// rate; issuing the sums' instructions takes 80% of the cycles), 70 us with 5 (the
// starts and ends of the runs, of which 4 CTAs share an SM).  Rows read three times by
// one CTA each took 2.6 ms; whole segments in registers 245 us (half of the time in
// barriers and first loads); exponents of scalar fp32 98 us where pairs take 76.
// Rows of one block take 4 us, most of it launch, first load and barriers.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_logprob(Args a) {
  constexpr int kE = 16 / sizeof(T);
  __shared__ uint4 ring[kRing][kV][kThreads];
  __shared__ float red[3][kWarps];
  __shared__ __align__(16) uint32_t group[128];
  __shared__ uint32_t tau_s;
  __shared__ int n_keep[kWarps], hist[256], found[3], n_best;
  __shared__ uint64_t keep_buf[kWarps][kCap];
  __shared__ uint32_t noted[kWarps][kList];
  __shared__ uint64_t best[kMaxK];
  const int64_t b = blockIdx.x / a.n_run;
  const int run = blockIdx.x % a.n_run, t = threadIdx.x, w = t >> 5, lane = t & 31;
  const Row<T> row(a.logits, b, a.N);
  const int n_blocks = (int)((a.N + row.head + kE * (int64_t)kBlock - 1) / (kE * (int64_t)kBlock));
  const int blk0 = (int)((int64_t)run * n_blocks / a.n_run), blk1 = (int)((int64_t)(run + 1) * n_blocks / a.n_run);
  const uint32_t run0 = (uint32_t)blk0 * kBlock, v0 = run0 + t;
  wait_for_stream();
  let_next_start();
  // blocks [in0, in1) lie whole inside the row
  const int in0 = row.head ? 1 : 0, in1 = (int)((a.N + row.head) / (kE * (int64_t)kBlock));
  const uint4* src = reinterpret_cast<const uint4*>(row.z - row.head) + v0;
  uint32_t v_next = v0;  // vector of the next request
  auto request = [&](int blk) {
    if (blk < blk1) {
      uint4(*to)[kThreads] = ring[(blk - blk0) % kRing];
      if (blk >= in0 && blk < in1) {
#pragma unroll
        for (int i = 0; i < kV; ++i) cp_async16(smem_u32(&to[i][t]), src + i * kThreads, 16);
      } else {
#pragma unroll 1
        for (int i = 0; i < kV; ++i) {
          const uint32_t v = v_next + i * kThreads;
          if (row.whole(row.column(v))) cp_async16(smem_u32(&to[i][t]), src + i * kThreads, 16);
          else to[i][t] = row.load(v);
        }
      }
      src += kBlock;
      v_next += kBlock;
    }
    cp_async_commit();
  };
  request(blk0);
  request(blk0 + 1);
  const Given<T, kThreads> given(a.n_run == 1 ? a : Args{}, b, row.z);
  cp_async_wait_group<1>();
  uint4 cur[kV];
  float vm;  // of this thread's vectors of the block
  auto read = [&](int blk) {
    uint4(*at)[kThreads] = ring[(blk - blk0) % kRing];
#pragma unroll
    for (int i = 0; i < kV; ++i) cur[i] = at[i][t];
    vm = max_of<T>(cur);
  };
  read(blk0);
  float mx = blk0 < blk1 ? vm : -INFINITY;  // of what this thread has seen
  if (a.rank_all)
    for (uint32_t j = t; j < row.N; j += kThreads) (&keep_buf[0][0])[j] = rank_key(Elem<T>::to_f(row.z[j]), j);
  float m = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][w] = m;
  Keep keep{0, false, kFinite};
  float tau_f = INFINITY;
  auto raise = [&] {
    keep.raise((uint64_t)(a.k <= kFew ? bound_of<64>(mx, a.k, group, &tau_s)
                                      : bound_of<128>(mx, a.k, group, &tau_s)) << 32);
    tau_f = keep.bar();
  };
  if (a.k == 0 || a.rank_all) {
    __syncthreads();
  } else if (a.thin) {
    keep.raise((uint64_t)bound_thin(mx, a.k, group, &tau_s) << 32);
    tau_f = keep.bar();
  } else {
    raise();
  }
  int n_noted = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) m = fmaxf(m, red[0][i]);
  Sums s(m < INFINITY ? fmaxf(m, -FLT_MAX) : 0.f);
  if (!(m < INFINITY)) s.S = NAN;  // +inf: the row is NaN

#pragma unroll 1
  for (int blk = blk0; blk < blk1; ++blk) {
    if (blk > blk0) {
      cp_async_wait_group<1>();
      read(blk);
      const int seen = blk - blk0;
      if (a.k > 0 && seen > 1 && (seen & (seen - 1)) == 0 && (a.k > kFew || (seen & 0x55555555))) raise();
      mx = fmaxf(mx, vm);
      if (vm > s.mu) {
        if (vm < INFINITY) s.move(vm);
        else s.S = NAN;
      }
    }
    if (__any_sync(0xffffffffu, vm >= tau_f) && a.k > 0 && !a.rank_all) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const uint32_t at = (uint32_t)((blk - blk0) * kBlock + i * kThreads + t);
        const bool in = max_of<T, 1>({cur[i]}) >= tau_f;
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        if (n_noted + __popc(who) > kList) {
          keep = look<T>(keep_buf[w], keep, noted[w], n_noted, row, run0, nullptr, ~0u, a.k);
          tau_f = keep.bar();
          n_noted = 0;
        }
        if (in) noted[w][n_noted + __popc(who & ((1u << lane) - 1))] = at;
        n_noted += __popc(who);
      }
    }
    add<T>(s, cur);
    request(blk + kRing);
  }
  cp_async_wait_all();
  uint64_t* flat = a.rank_all ? &keep_buf[0][0] : reinterpret_cast<uint64_t*>(ring);  // once every thread is through its blocks
  if (a.k > 0 && !a.rank_all) {
    if (a.k > kFew && blk1 - blk0 > 1) raise();
    keep = look<T>(keep_buf[w], keep, noted[w], n_noted, row, run0, &ring[0][0][0],
                   (uint32_t)max(blk1 - blk0 - kRing, 0) * kBlock, a.k);
  }

  // join the threads' sums around the run's maximum
  float mu = s.mu;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
  __syncthreads();
  if (lane == 0) {
    red[0][w] = mu;
    n_keep[w] = keep.n;
  }
  __syncthreads();
  int c = 0, at = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    mu = fmaxf(mu, red[0][i]);
    if (i == w) at = c;
    c += n_keep[i];
  }
  s.move(mu);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
    s.Y += __shfl_xor_sync(0xffffffffu, s.Y, o);
  }
  if (lane == 0) {
    red[1][w] = s.S;
    red[2][w] = s.Y;
  }
  if (a.rank_all) {
    c = (int)row.N;
  } else if (c <= kThreads) {
    for (int i = lane; i < keep.n; i += 32) flat[at + i] = keep_buf[w][i];
  }
  __syncthreads();
  s.S = s.Y = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    s.S += red[1][i];
    s.Y += red[2][i];
  }
  if (a.n_run > 1 && t == 0) a.part[blockIdx.x] = make_float4(mu, s.S, s.Y, 0.f);
  const float Tt = s.settle();
  const RowStats st = row_stats(mu, s.S);
  if (a.n_run == 1) given.write(a, b, row.z, st, s.S, Tt);
  if (a.k == 0) return;

  uint64_t* keys = a.keys + (int64_t)blockIdx.x * a.k;
  auto emit = [&](int rank, uint64_t key) {
    if (a.n_run == 1) {
      a.top_id[b * a.k + rank] = (int32_t)key_id(key);
      a.top_logp[b * a.k + rank] = st.logp(key_value(key));
    } else {
      keys[rank] = key;
    }
  };
  if (c <= kThreads) {  // few: each counts the keys above it
    if (t < c) {
      const uint64_t key = flat[t];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < c; ++j) rank += flat[j] > key;
      if (rank < a.k) emit(rank, key);
    }
    if (c < a.k && w == 0) {
      const int64_t j0 = max(row.column(run0), (int64_t)0);
      const int64_t j1 = min(row.column((uint32_t)blk1 * kBlock), a.N);
      int r = fill_others(row, j0, j1, c, a.k, emit);
      if (a.n_run > 1)  // a short last run
        for (r += lane; r < a.k; r += 32) keys[r] = 0;
    }
  } else {
    uint64_t key[kCap / 32];
#pragma unroll
    for (int i = 0; i < kCap / 32; ++i)
      key[i] = a.rank_all                  ? (i * kThreads + t < c ? flat[i * kThreads + t] : 0)
               : i * 32 + lane < keep.n ? keep_buf[w][i * 32 + lane]
                                        : 0;
    emit_best(key, a.k, hist, found, best, &n_best, emit);
  }
}

// One CTA per row joins its runs (2 us beside the runs without alternatives, about 8 us
// for 3 rows of 128 runs with 64 alternatives).
constexpr int kJoinThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads, 1) k_logprob_join(Args a) {
  __shared__ float red[3][kJoinThreads / 32];
  __shared__ uint64_t cand[kMaxK * kMaxK];
  __shared__ uint64_t best[kMaxK];
  __shared__ int n_cand, n_best, n_lists, lists[kMaxK], hist[256], found[3];
  __shared__ uint64_t tau_s;
  const int64_t b = blockIdx.x;
  const int t = threadIdx.x, n = a.n_run, k = a.k;
  // the labels and the logits were complete before the runs' kernel let this one start
  const T* row = static_cast<const T*>(a.logits) + b * a.N;
  const Given<T, kJoinThreads> given(a, b, row);
  wait_for_stream();
  let_next_start();
  const float4* part = a.part + b * n;
  constexpr int kPer = kMaxRuns / kJoinThreads;
  float4 p[kPer];
  float mu = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] = i * kJoinThreads + t < n ? part[i * kJoinThreads + t] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    mu = fmaxf(mu, p[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
  if ((t & 31) == 0) red[0][t >> 5] = mu;
  if (t == 0) n_cand = n_lists = 0;
  __syncthreads();
  for (int i = 0; i < kJoinThreads / 32; ++i) mu = fmaxf(mu, red[0][i]);
  Sums s(mu);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (p[i].y != 0.f) {  // NaN too
      Sums r(p[i].x);
      r.S = p[i].y;
      r.Y = p[i].z;
      r.move(mu);
      s.S += r.S;
      s.Y += r.Y;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
    s.Y += __shfl_xor_sync(0xffffffffu, s.Y, o);
  }
  if ((t & 31) == 0) {
    red[1][t >> 5] = s.S;
    red[2][t >> 5] = s.Y;
  }
  __syncthreads();
  s.S = s.Y = 0.f;
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    s.S += red[1][i];
    s.Y += red[2][i];
  }
  const float Tt = s.settle();
  const RowStats st = row_stats(mu, s.S);
  given.write(a, b, row, st, s.S, Tt);
  if (k == 0) return;
  // A bound that few keys beside the k best reach.  Up to k runs: the smallest of the
  // runs' ceil(k / n)-th bests, since k keys are as large.  More: the k-th largest of
  // the runs' bests, below which a run holds nothing.
  const uint64_t* keys = a.keys + b * n * k;
  uint64_t tau = 1;
  int m = n;  // runs that are looked into
  if (n > k && n * k > kJoinThreads) {
    uint64_t head[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) head[i] = i * kJoinThreads + t < n ? keys[(int64_t)(i * kJoinThreads + t) * k] : 0;
    tau = kth_key(head, k, hist, found);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (head[i] != 0 && head[i] >= tau) lists[atomicAdd(&n_lists, 1)] = i * kJoinThreads + t;
    m = k;
    __syncthreads();
  } else if (n <= k) {
    if (t < 32) {
      uint64_t low = ~0ull;
      for (int i = t; i < n; i += 32) {
        const uint64_t key = keys[(int64_t)i * k + (k + n - 1) / n - 1];
        low = key < low ? key : low;  // 0 where a short run ends before
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, low, o);
        low = other < low ? other : low;
      }
      if (t == 0) tau_s = low;
    }
    __syncthreads();
    tau = tau_s > 0 ? tau_s : 1;
  }
  constexpr int kPerCand = kMaxK * kMaxK / kJoinThreads;
  uint64_t got[kPerCand];
#pragma unroll
  for (int i = 0; i < kPerCand; ++i) {
    const int at = i * kJoinThreads + t;
    got[i] = 0;
    if (at < m * k) got[i] = keys[(int64_t)(m < n ? lists[at / k] : at / k) * k + at % k];
  }
#pragma unroll
  for (int i = 0; i < kPerCand; ++i)
    if (got[i] != 0 && got[i] >= tau) cand[atomicAdd(&n_cand, 1)] = got[i];
  __syncthreads();
  const int c = n_cand;
  auto emit = [&](int rank, uint64_t key) {
    a.top_id[b * k + rank] = (int32_t)key_id(key);
    a.top_logp[b * k + rank] = st.logp(key_value(key));
  };
  if (c <= kJoinThreads) {  // few: each counts the keys above it
    if (t < c) {
      const uint64_t key = cand[t];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < c; ++j) rank += cand[j] > key;
      if (rank < k) emit(rank, key);
    }
  } else {
    emit_best(got, k, hist, found, best, &n_best, emit);
  }
}

// As bound_of, by one warp: the k-th largest maximum of 32 kP groups of a row's vectors (k
// of which hold one), or 0.
template <typename T, int kN, int kP>
__device__ __forceinline__ uint32_t bound_rows(const uint4 (&raw)[kN], int k) {
  const int lane = threadIdx.x & 31;
  float mx[kP];
  uint32_t mine[kP];
  int above[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    mx[p] = -INFINITY;
#pragma unroll
    for (int i = p; i < kN; i += kP) mx[p] = fmaxf(mx[p], max_of<T, 1>({raw[i]}));
    mine[p] = (rank_value(mx[p]) & ~127u) | (uint32_t)(p * 32 + lane);
    above[p] = 0;
  }
#pragma unroll 4
  for (int l = 0; l < 32; ++l)
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const uint32_t o = __shfl_sync(0xffffffffu, mine[p], l);
#pragma unroll
      for (int q = 0; q < kP; ++q) above[q] += o > mine[q];
    }
  uint32_t bound = 0;
#pragma unroll
  for (int p = 0; p < kP; ++p)
    if (above[p] == k - 1) bound = mine[p] & ~127u;
  return __reduce_max_sync(0xffffffffu, bound);
}

// The n <= 32 kP keys of a warp: each counts those above it.
template <int kP, typename Emit>
__device__ __forceinline__ void rank_kept(const uint64_t* buf, int n, int k, Emit emit) {
  const int lane = threadIdx.x & 31;
  uint64_t key[kP];
  int rank[kP] = {};
#pragma unroll
  for (int p = 0; p < kP; ++p) key[p] = p * 32 + lane < n ? buf[p * 32 + lane] : 0;
#pragma unroll 4
  for (int j = 0; j < n; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(buf + j);
#pragma unroll
    for (int p = 0; p < kP; ++p) rank[p] += (o.x > key[p]) + (o.y > key[p]);
  }
#pragma unroll
  for (int p = 0; p < kP; ++p)
    if (key[p] != 0 && rank[p] < k) emit(rank[p], key[p]);
}

// A warp per row, its kN vectors a lane in registers: no barrier, and 12 to 36 rows under
// way on an SM.  A row's latency bounds it (load, the dependent loads of its labels, the
// bound, ranking): 20,000 x 1,000 bf16 in 10 us without labels or alternatives (4.0 TB/s;
// by CTAs 120), 27 with 2 labels and 5 alternatives (200).  Vectors that hold something
// are read again (from L1) rather than picked from registers: unrolled over the registers
// the selection took 34.
constexpr int kRowWarps = 4;
template <typename T, int kN>
__global__ void __launch_bounds__(32 * kRowWarps) k_logprob_rows(Args a, int B) {
  __shared__ __align__(16) uint64_t keep_buf[kRowWarps][kCap];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = (int64_t)blockIdx.x * kRowWarps + w;
  wait_for_stream();
  let_next_start();
  if (b >= B) return;
  const Row<T> row(a.logits, b, a.N);
  uint4 raw[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) raw[i] = row.load(i * 32 + lane);
  const Given<T, 32> given(a, b, row.z);
  const float mx = max_of<T>(raw);
  float m = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  Sums s(m < INFINITY ? fmaxf(m, -FLT_MAX) : 0.f);
  if (!(m < INFINITY)) s.S = NAN;
  add<T>(s, raw);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
    s.Y += __shfl_xor_sync(0xffffffffu, s.Y, o);
  }
  const float Tt = s.settle();
  const RowStats st = row_stats(s.mu, s.S);
  given.write(a, b, row.z, st, s.S, Tt);
  if (a.k == 0) return;

  // what competes: all of up to kCap logits; else those from a bound on, the k-th largest
  // maximum of kG groups of vectors
  uint64_t* buf = keep_buf[w];
  Keep keep{0, false, kFinite};
  if (a.N <= kCap) {
    for (uint32_t j = lane; j < row.N; j += 32) buf[j] = rank_key(Elem<T>::to_f(row.z[j]), j);
    keep.n = (int)row.N;
  } else {
    keep.raise((uint64_t)(a.k <= 8    ? bound_rows<T, kN, 1>(raw, a.k)
                          : a.k <= 32 ? bound_rows<T, kN, 2>(raw, a.k)
                                      : bound_rows<T, kN, 4>(raw, a.k)) << 32);
    const float bar = keep.bar();
    uint32_t want = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) want |= max_of<T, 1>({raw[i]}) >= bar ? 1u << i : 0u;
    while (__any_sync(0xffffffffu, want != 0)) {  // every lane its next vector
      const uint32_t v = (uint32_t)(want ? __ffs(want) - 1 : 0) * 32 + lane;
      keep = take<T>(buf, keep, row.load(v), want != 0, row.column(v), row.N, a.k);
      keep.strict = false;  // smaller ids may follow
      want &= want - 1;
    }
  }
  auto emit = [&](int rank, uint64_t key) {
    a.top_id[b * a.k + rank] = (int32_t)key_id(key);
    a.top_logp[b * a.k + rank] = st.logp(key_value(key));
  };
  if (lane == 0 && keep.n < kCap) buf[keep.n] = 0;  // keys are read in pairs
  __syncwarp();
  if (keep.n <= 32) rank_kept<1>(buf, keep.n, a.k, emit);
  else if (keep.n <= 64) rank_kept<2>(buf, keep.n, a.k, emit);
  else rank_kept<kCap / 32>(buf, keep.n, a.k, emit);
  if (keep.n < a.k) fill_others(row, 0, a.N, keep.n, a.k, emit);
}

// The dense term of a row's gradient, by its definition: for single labels, and for rows
// whose lse lies beyond kFar.  An fp32 lse is too coarse there to hold log S (of a row of
// the type's lowest value it holds nothing of it); `lack` is what it lacks.
struct Term {
  float lse, H, gH, G, lack;
  __device__ bool none() const { return lse == -INFINITY; }
  __device__ bool near() const { return fabsf(lse) < kFar || lse != lse; }
  __device__ float at(float v) const {
    const float lp = (v - lse) - lack, p = ex2(lp * kLog2e);
    return p == 0.f || none() ? 0.f : -p * fmaf(gH, lp + H, G);
  }
};
// The terms of vectors [v0, v1) of a row beyond kFar (or of nothing but -inf), by the kStep
// threads of the row's warp or of one of its CTAs; gives the row's `lack`, the log of its
// sum of e^(z - lse), which they take over the whole row.
template <typename T, int kStep>
__device__ __noinline__ float far_terms(const Row<T> row, T* dz, uint32_t v0, uint32_t v1, Term f) {
  constexpr int kE = Row<T>::kE;
  const uint32_t t = threadIdx.x % kStep, n_vec = (uint32_t)((row.N + (int64_t)row.head + kE - 1) / kE);
  if (fabsf(f.lse) < INFINITY) {
    double S = 0.;
    for (uint32_t v = t; v < n_vec; v += kStep) S += far_sums<T>(row.load(v), f.lse).x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    if constexpr (kStep > 32) {
      __shared__ double part[kStep / 32];
      if (t % 32 == 0) part[t / 32] = S;
      __syncthreads();
      S = 0.;
      for (int i = 0; i < kStep / 32; ++i) S += part[i];
    }
    if (S > 0.) f.lack = logf((float)S);
  }
  for (uint32_t v = v0 + t; v < min(v1, n_vec); v += kStep) {
    const int64_t j = row.column(v);
    float z[kE];
    unpack<T>(row.load(v), z);
    for (int e = 0; e < kE; ++e)
      if (j + e >= 0 && j + e < row.N) dz[j + e] = Elem<T>::from_f(f.at(z[e]));
  }
  return f.lack;
}

// The same for vectors of a row within kFar.  With y = z log2(e) - R, R = fl(lse log2(e)) and
// e = lse log2(e) - R, which an fma gives exactly, p = 2^(y - e) and log p = ln2 (y - e):
// the term is -2^y (A + C y) with A and C of the row.
template <typename T>
struct Dense {
  static constexpr int kE = 16 / sizeof(T), kP = kE / 2;
  float lo;
  f2 R2, A2, C2;
  __device__ explicit Dense(const Term& f) : lo(floor_of(f.lse)) {
    const float R = f.lse * kLog2e, e0 = fmaf(f.lse, kLog2e, -R), w = -ex2(-e0);
    const float A = w * fmaf(f.gH, fmaf(-kLn2, e0, f.H), f.G), C = w * f.gH * kLn2;
    R2 = pair(-R, -R);
    A2 = pair(A, A);
    C2 = pair(C, C);
  }
  __device__ void of(const uint4& raw, float (&v)[kE]) const {
    const f2 L2 = pair(kLog2e, kLog2e);
    f2 x[kP];
    raised<T>(raw, lo, x);
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      const f2 y = fma2(x[e], L2, R2);
      unpair(mul2(ex2_2(y), fma2(y, C2, A2)), v[2 * e], v[2 * e + 1]);
    }
  }
};
template <typename T>
__device__ __forceinline__ uint4 packed(const float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// A warp's part of the sum over a row's list, and whether that part ascends.
__device__ __forceinline__ float list_sum(const GradArgs& a, int64_t p0, int64_t p1, int first, int step, bool& ascending) {
  float G = 0.f;
  ascending = true;
  for (int64_t p = p0 + first; p < p1; p += step) {
    const int64_t id = a.ids[p];
    if (id >= 0 && id < a.N) G += a.d_logp[p];
    ascending &= p + 1 == p1 || id < a.ids[p + 1];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) G += __shfl_xor_sync(0xffffffffu, G, o);
  return G;
}

// The given labels of columns [c0, c1), by kStep threads whose dense terms there are
// written.  In a list that ascends each label is given once.  In any other a label that
// may be given again (it shares its bit of `again` with a second entry) is looked for in
// the whole list by its warp, and its first entry takes the sum.  (Every label looked for
// by its thread: 256 x 8,192, 1,024 shuffled labels a row, 154 us against 8.3; in
// ascending order 6.0.  Lists of many repeats are slower for it: 256 rows of 50 labels
// given 400 times 77 us, 9,000 labels 68, against 33.)
template <typename T, int kStep, uint32_t kBits>
__device__ __forceinline__ void put_given(const GradArgs& a, const Row<T>& row, T* dz, const Term& term, int64_t p0,
                                          int64_t p1, int64_t c0, int64_t c1, bool ascending, uint32_t* once,
                                          uint32_t* again) {
  auto sync = [] {
    if constexpr (kStep == 32) __syncwarp();
    else __syncthreads();
  };
  const int t = threadIdx.x % kStep;
  sync();  // the dense term is written
  auto put = [&](int64_t id, float g) { dz[id] = Elem<T>::from_f(g + term.at(Elem<T>::to_f(row.z[id]))); };
  if (ascending) {
    for (int64_t p = p0 + t; p < p1; p += kStep) {
      const int64_t id = a.ids[p];
      if (id >= c0 && id < c1) put(id, a.d_logp[p]);
    }
    return;
  }
  for (int i = t; i < (int)(kBits / 32); i += kStep) once[i] = again[i] = 0;
  sync();
  for (int64_t p = p0 + t; p < p1; p += kStep) {
    const int64_t id = a.ids[p];
    if (id < c0 || id >= c1) continue;
    const uint32_t at = (uint32_t)id % kBits, bit = 1u << at % 32;
    if (atomicOr(&once[at / 32], bit) & bit) atomicOr(&again[at / 32], bit);
  }
  sync();
  for (int64_t q0 = p0 + (t & ~31); q0 < p1; q0 += kStep) {
    const int64_t p = q0 + (t & 31), id = p < p1 ? a.ids[p] : -1;
    const uint32_t at = (uint32_t)id % kBits;
    const bool here = id >= c0 && id < c1, maybe = here && (again[at / 32] >> at % 32 & 1);
    if (here && !maybe) put(id, a.d_logp[p]);
    bool look_for = maybe;
    if constexpr (kStep == 32) {  // a bit a label, in the list's order: only its first entry still finds it in `once`
      look_for = maybe && (once[at / 32] >> at % 32 & 1);
      const uint32_t same = __match_any_sync(0xffffffffu, look_for ? (int)id : -1 - t);
      look_for = look_for && __ffs(same) - 1 == t;
      __syncwarp();
      if (look_for) atomicAnd(&once[at / 32], ~(1u << at % 32));
      __syncwarp();
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, look_for); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      const int label = __shfl_sync(0xffffffffu, (int)id, l);
      bool first = true;
      float g = 0.f;
      for (int64_t q = kStep == 32 ? q0 : p0; q < p1; q += 4 * 32) {
        bool hit[4];
        uint32_t who[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t r = q + i * 32 + (t & 31);
          hit[i] = r < p1 && a.ids[r] == label;
        }
        if (!__any_sync(0xffffffffu, hit[0] || hit[1] || hit[2] || hit[3])) continue;
        int64_t at0 = q;  // the first entry among these that gives the label
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          who[i] = __ballot_sync(0xffffffffu, hit[i]);
          if (who[i]) at0 = q + i * 32 + __ffs(who[i]) - 1;
        }
        first = at0 >= q0 + l;
        if (!first) break;
        float add[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) add[i] = hit[i] ? a.d_logp[q + i * 32 + (t & 31)] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          for (; who[i]; who[i] &= who[i] - 1) g += __shfl_sync(0xffffffffu, add[i], __ffs(who[i]) - 1);
      }
      if (first && (t & 31) == l) put(label, g);
    }
  }
}

// One CTA per run of a row: the dense term of its blocks, then the given labels in
// them.  Bound by memory: 256 x 670,208 bf16 in 110 us, 6.2 TB/s read and written, 95%
// of a copy's rate.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_logprob_grad(GradArgs a) {
  constexpr int kE = 16 / sizeof(T);
  constexpr uint32_t kBits = 32768;
  __shared__ uint32_t once[kBits / 32], again[kBits / 32];
  const int64_t b = blockIdx.x / a.n_run;
  const int run = blockIdx.x % a.n_run, t = threadIdx.x;
  const Row<T> row(a.logits, b, a.N);
  T* dz = static_cast<T*>(a.d_logits) + b * a.N;
  const int n_blocks = (int)((a.N + row.head + kE * (int64_t)kBlock - 1) / (kE * (int64_t)kBlock));
  const int blk0 = (int)((int64_t)run * n_blocks / a.n_run), blk1 = (int)((int64_t)(run + 1) * n_blocks / a.n_run);
  const int in0 = row.head ? 1 : 0, in1 = (int)((a.N + row.head) / (kE * (int64_t)kBlock));
  const uint4* at_row = reinterpret_cast<const uint4*>(row.z - row.head) + t;
  wait_for_stream();
  let_next_start();
  uint4 raw[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) raw[i] = row.load((uint32_t)blk0 * kBlock + t + i * kThreads);
  const float lse = a.lse[b];
  const float gH = a.d_entropy ? a.d_entropy[b] : 0.f, H = a.d_entropy ? a.entropy[b] : 0.f;
  int64_t p0, p1;
  row_list(a.row_ptr, a.nnz, b, p0, p1);
  // every warp sums the list, in the same order; long ones are split over the warps
  // (64 x 32,768, 4,096 labels a row: 12.0 us against 21.0)
  __shared__ float g_warp[kWarps];
  const bool split = p1 - p0 > 4 * 32;
  bool ascending;
  float G = list_sum(a, p0, p1, split ? t : t & 31, split ? kThreads : 32, ascending);
  if (split) {
    if ((t & 31) == 0) g_warp[t >> 5] = G;
    ascending = __syncthreads_and(ascending);
    G = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) G += g_warp[i];
  } else {
    ascending = __all_sync(0xffffffffu, ascending);
  }
  Term term{lse, H, gH, G, 0.f};
  if (term.near()) {
    const Dense<T> dense(term);
    // the output may sit on the 16-byte boundary differently from the input
    const bool vec = ((reinterpret_cast<uintptr_t>(row.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
    uint4* out_row = reinterpret_cast<uint4*>(dz - row.head) + t;
    for (int blk = blk0; blk < blk1; ++blk) {
      const bool more = blk + 1 < blk1, inside = blk + 1 >= in0 && blk + 1 < in1;
      const bool whole = vec && blk >= in0 && blk < in1;
      const uint32_t v0 = (uint32_t)blk * kBlock + t;
      const uint4* next = at_row + (int64_t)(blk + 1) * kBlock;
      uint4* out = out_row + (int64_t)blk * kBlock;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        float v[kE];
        dense.of(raw[i], v);
        if (more) raw[i] = inside ? next[i * kThreads] : row.load(v0 + kBlock + i * kThreads);
        if (whole) {
          out[i * kThreads] = packed<T>(v);
        } else {
          const int64_t j = row.column(v0 + i * kThreads);
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (j + e >= 0 && j + e < a.N) dz[j + e] = Elem<T>::from_f(v[e]);
        }
      }
    }
  } else {
    term.lack = far_terms<T, kThreads>(row, dz, (uint32_t)blk0 * kBlock, (uint32_t)blk1 * kBlock, term);
  }
  if (p0 == p1 || term.none()) return;
  put_given<T, kThreads, kBits>(a, row, dz, term, p0, p1, max(row.column((uint32_t)blk0 * kBlock), (int64_t)0),
                                min(row.column((uint32_t)blk1 * kBlock), a.N), ascending, once, again);
}

// A warp per row, its kN vectors a lane in registers: 20,000 x 1,000 bf16 in 14.9 us, 5.4
// TB/s read and written (21 us, 3.8 TB/s, from and to HBM).  4, 7 or 8 CTAs an SM (4,000 x 2,000 f32 with entropies, 16 vectors a
// lane: 15.5 us against 17.4 without that bound on the registers).
template <typename T, int kN>
__global__ void __launch_bounds__(32 * kRowWarps, kN == 16 ? 4 : kN == 8 ? 7 : 8) k_logprob_grad_rows(GradArgs a, int B) {
  constexpr int kE = 16 / sizeof(T);
  constexpr uint32_t kBits = 32 * kN * kE;  // one for each label
  __shared__ uint32_t once[kRowWarps][kBits / 32], again[kRowWarps][kBits / 32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = (int64_t)blockIdx.x * kRowWarps + w;
  wait_for_stream();
  let_next_start();
  if (b >= B) return;
  const Row<T> row(a.logits, b, a.N);
  T* dz = static_cast<T*>(a.d_logits) + b * a.N;
  uint4 raw[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) raw[i] = row.load(i * 32 + lane);
  const float lse = a.lse[b];
  const float gH = a.d_entropy ? a.d_entropy[b] : 0.f, H = a.d_entropy ? a.entropy[b] : 0.f;
  int64_t p0, p1;
  row_list(a.row_ptr, a.nnz, b, p0, p1);
  bool ascending;
  const float G = list_sum(a, p0, p1, lane, 32, ascending);
  ascending = __all_sync(0xffffffffu, ascending);
  Term term{lse, H, gH, G, 0.f};
  if (term.near()) {
    const Dense<T> dense(term);
    const bool vec = ((reinterpret_cast<uintptr_t>(row.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t j = row.column(i * 32 + lane);
      float v[kE];
      dense.of(raw[i], v);
      if (vec && row.whole(j)) {
        *reinterpret_cast<uint4*>(dz + j) = packed<T>(v);
      } else if (j < a.N) {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (j + e >= 0 && j + e < a.N) dz[j + e] = Elem<T>::from_f(v[e]);
      }
    }
  } else {
    term.lack = far_terms<T, 32>(row, dz, 0, ~0u, term);
  }
  if (p0 == p1 || term.none()) return;
  put_given<T, 32, kBits>(a, row, dz, term, p0, p1, 0, a.N, ascending, once[w], again[w]);
}

// Blocks that a row of N elements can touch: of logits at this address, or (NULL)
// wherever they start.
template <typename T>
inline int64_t row_blocks(const void* logits, int64_t N) {
  constexpr int64_t kE = 16 / sizeof(T);
  const bool on = logits && reinterpret_cast<uintptr_t>(logits) % 16 == 0 && N % kE == 0;
  return (N + (on ? 0 : kE - 1) - 1) / (kE * kBlock) + 1;
}
// Runs of a row: `ctas` CTAs in all, at least `least` blocks each.
inline int64_t runs(int B, int64_t blocks, int64_t ctas, int64_t least) {
  const int64_t want = (ctas + B - 1) / B;
  const int64_t n = blocks / least < want ? blocks / least : want;
  return n < 1 ? 1 : n > kMaxRuns ? kMaxRuns : n;
}
// Whole rows where that leaves the SMs busy or a row is short: the start of a run
// and the join cost as much as several blocks.  Measured with 5 alternatives, whole
// against split: 256 x 65,536 bf16 13.1 and 20.4 us, 256 x 131,072 20.1 and 25.2 us,
// 64 x 40,000 8.2 and 10.5 us, 64 x 65,536 9.9 and 10.7 us, 100 x 65,536 10.2 and 12.5
// us; but 1 x 65,536 9.6 and 6.9 us, 256 x 670,208 (4 runs) 87 and 73 us.
// One block a run (the last half a block to one and a half, so that none is empty
// wherever the rows start) where that leaves no more CTAs than SMs: 8 x 65,536 bf16 7.2
// us with 5 alternatives, 10.0 with 64, against 8.5 and 11.4 in runs of two.
// The numbers of CTAs (888 and 3,552 are six and 24 a SM) are a B200's and not the device's:
// the workspace's size follows from them, and a host without a GPU may ask for it.
constexpr int64_t kSpread = 148;
inline int64_t forward_runs(int B, int64_t blocks, int64_t row_bytes) {
  if (blocks <= 4 || (B >= 64 && blocks <= 8) || (B >= 128 && blocks <= 16)) return 1;
  const int64_t single = (row_bytes + 8 * kBlock) / (16 * kBlock);
  if (single <= kSpread / B) return single;
  return runs(B, blocks, 888, 2);
}
// The gradient has nothing to join: short runs, of which many are in flight (256 x
// 670,208 bf16: 109 us with 14 a row, 117 with 7, 133 with one block each).
inline int64_t grad_runs(int B, int64_t blocks) { return runs(B, blocks, 3552, 1); }

// Vectors that a lane holds where a warp takes a row: 0 where a row has too many.
template <typename T>
int lane_vectors(const void* logits, int64_t N) {
  const int64_t most = row_vectors<T>(N, reinterpret_cast<uintptr_t>(logits) % 16 == 0);
  return most <= 128 ? 4 : most <= 256 ? 8 : most <= 512 ? 16 : 0;
}
// Samples from which on a warp takes a row of that many vectors a lane: it has more to
// do one after another than a CTA, but an SM holds 12 to 36 of them against 4 CTAs.
// bf16, the CTAs' times second: 64 x 1,000 with 5 alternatives 5.3 and 5.5 us, with 20
// 6.4 and 6.0; 512 x 1,000 with 20 7.1 and 8.8, with 64 10.7 and 10.4; 20,000 x 1,000
// with 5 27 and 200; 64 x 2,000 with 1 4.8 and 5.3, with 5 6.1 and 5.5, 256 x 2,000 5.9
// and 6.1; 256 x 4,000 with 5 7.0 and 6.0, 512 x 4,000 7.9 and 8.0.  Rows of up to kCap
// labels always: 256 x 100 5.3 and 5.9.
template <typename T>
int warp_rows_from(int vecs, int64_t N, int k) {
  if (N <= kCap) return 1;
  if (k > 32) return 1024;
  if (vecs == 4) return k <= 8 || N * (int)sizeof(T) <= 1024 ? 1 : 256;
  return vecs == 8 ? (k <= 2 ? 1 : 256) : 512;
}
template <typename T>
cudaError_t launch(int B, Args a, cudaStream_t st) {
  const int vecs = lane_vectors<T>(a.logits, a.N);
  // every alternative needs a vector of its own for the bound
  const bool bounded = a.N <= kCap || a.N / (16 / (int)sizeof(T)) >= a.k;
  if (vecs > 0 && bounded && B >= warp_rows_from<T>(vecs, a.N, a.k)) {
    const unsigned grid = (unsigned)((B + (int64_t)kRowWarps - 1) / kRowWarps);
    if (vecs == 4) return launch_early(k_logprob_rows<T, 4>, grid, 32 * kRowWarps, 0, st, a, B);
    if (vecs == 8) return launch_early(k_logprob_rows<T, 8>, grid, 32 * kRowWarps, 0, st, a, B);
    return launch_early(k_logprob_rows<T, 16>, grid, 32 * kRowWarps, 0, st, a, B);
  }
  a.thin = a.N / (16 / (int)sizeof(T)) < 2 * a.k;  // up to 16 alternatives: a warp has taken the row
  a.rank_all = a.k > 0 && a.n_run == 1 && a.N / (16 / (int)sizeof(T)) < a.k;
  return launch_early(k_logprob<T>, (unsigned)(B * (int64_t)a.n_run), kThreads, 0, st, a);
}
template <typename T>
cudaError_t launch_join(int B, const Args& a, cudaStream_t st) {
  return launch_early(k_logprob_join<T>, (unsigned)B, kJoinThreads, 0, st, a);
}
template <typename T>
cudaError_t launch_grad(int B, const GradArgs& a, cudaStream_t st) {
  // a warp a row: 1 x 1,000 bf16 in 2.5 us (3.3 by a CTA), 20,000 x 1,000 in 14.9 (152);
  // 1 x 2,000 fp32 in 3.4 (2.9), 256 x 2,000 in 3.9 (3.9), 512 x 2,000 in 3.9 (5.4)
  const int vecs = lane_vectors<T>(a.logits, a.N);
  const unsigned grid = (unsigned)((B + (int64_t)kRowWarps - 1) / kRowWarps);
  if (vecs == 4) return launch_early(k_logprob_grad_rows<T, 4>, grid, 32 * kRowWarps, 0, st, a, B);
  if (vecs == 8) return launch_early(k_logprob_grad_rows<T, 8>, grid, 32 * kRowWarps, 0, st, a, B);
  if (vecs == 16 && B >= 512) return launch_early(k_logprob_grad_rows<T, 16>, grid, 32 * kRowWarps, 0, st, a, B);
  return launch_early(k_logprob_grad<T>, (unsigned)(B * (int64_t)a.n_run), kThreads, 0, st, a);
}

}  // namespace logprob
}  // namespace haste
