// head_i8.cu -- the dense head in 8-bit integers on sm_100a.
//
// Row quantisation (weights: one scale per label; features: one per sample):
// s = max|x| / 127 rounded once to fp32, q = the exact quotient x / s rounded half
// to even.  Product: z[b, h] = (float)(sum_f qx[b, f] qw[h, f]) * (sx[b] * sw[h]),
// the sum exact in 32 bits (tcgen05 kind::i8).
//
// Times in this file are of one call among others in a CUDA graph on the same inputs; a
// program's calls one by one take longer at the largest size (512 x 131,072 x 1024: 90 us
// where 76 stand here).
#include "common.cuh"
#include "launch.cuh"

namespace haste {
namespace head8 {

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

// 8 of a row's elements as 8-bit integers.  x inv + 1.5 * 2^23 rounds x / s to a whole
// number in the low bits of the sum, inv being 1 / s to an ulp; the exact remainder
// then moves a quotient that fell on the wrong side of a half (half the row's maximum
// lies next to 63.5, and bf16 rows meet it often).  Scales too small for a reciprocal
// (inv = 0) take the division above.  131,072 rows of 1,024 bf16 values take 140 us (their
// bytes 61 at a copy's rate; the corrections' instructions bound it), 256 of 768 1.9 us.
// (Divisions throughout took 249 us, and 4 us for a single row.)
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float s, float inv) {
  constexpr float kM = 12582912.f;
  uint32_t b[8];
  if (inv != 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = fmaf(x[j], inv, kM), r = fmaf(kM - t, s, x[j]), r2 = r + r;
      b[j] = __float_as_uint(t);
      const bool odd = b[j] & 1;
      if (r2 > s || (r2 == s && odd)) ++b[j];
      if (r2 < -s || (r2 == -s && odd)) --b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = (uint32_t)quantise(x[j], s);
  }
  uint2 w;
  w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return w;
}

// 8 consecutive elements of a row as fp32, 0 past its end; vec: the row starts on
// a 16-byte boundary and holds whole vectors of 8.
template <typename T>
__device__ __forceinline__ void load8(const T* __restrict__ row, int i, int n, bool vec, float (&v)[8]) {
  if (vec && i + 8 <= n) {
    if constexpr (sizeof(T) == 2) {
      const uint4 r = *reinterpret_cast<const uint4*>(row + i);
      const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(row + i), b = *reinterpret_cast<const float4*>(row + i + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < n ? Elem<T>::to_f(row[i + j]) : 0.f;
  }
}

// The largest magnitude so far; a NaN counts as infinite.
__device__ __forceinline__ float row_max(float m, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(v[j]);
    m = a <= m ? m : a < INFINITY ? a : INFINITY;
  }
  return m;
}
// A row's scale, from its largest magnitude (infinite: NaN, and every q = 0).
struct RowScale {
  float s, inv;
  __device__ explicit RowScale(float m) {
    s = m < INFINITY ? __fdiv_rn(m, 127.f) : NAN;
    inv = s > 1e-30f ? __fdiv_rn(1.f, s) : 0.f;
  }
  __device__ uint2 quantised(const float (&v)[8]) const { return s > 0.f ? quantise8(v, s, inv) : make_uint2(0, 0); }
};

// One row per group of kWarps warps; every lane holds kKeep runs of 8 elements of
// its row (rows of up to 256 kWarps kKeep elements are read once), longer rows are
// read again from L2.  A row with a NaN or an infinity gets the scale NaN and zeros.
constexpr int kQThreads = 256, kKeep = 4;
constexpr int64_t kManyRows = 4096;
template <typename T, int kWarps>
__global__ void __launch_bounds__(kQThreads) k_quantize_rows(const T* __restrict__ x, int64_t rows, int n, bool vec,
                                                             int8_t* __restrict__ q, float* __restrict__ scale) {
  // what came before is complete before the kernel after this one may start: that
  // one reads its weights without waiting for more
  wait_for_stream();
  let_next_start();
  __shared__ float red[kQThreads / 32];
  constexpr int kRowThreads = 32 * kWarps;
  const int64_t r = (int64_t)blockIdx.x * (kQThreads / kRowThreads) + threadIdx.x / kRowThreads;
  const int t = threadIdx.x % kRowThreads;
  const bool live = r < rows;
  const int ld = pitch(n);
  const T* xr = x + (live ? r : 0) * n;
  float keep[kKeep][8];
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < kKeep; ++c)
    if (c * kRowThreads * 8 < n) load8(xr, (c * kRowThreads + t) * 8, n, vec, keep[c]);
#pragma unroll
  for (int c = 0; c < kKeep; ++c)
    if (c * kRowThreads * 8 < n) m = row_max(m, keep[c]);
  for (int i = (kKeep * kRowThreads + t) * 8; i < n; i += kRowThreads * 8) {
    float v[8];
    load8(xr, i, n, vec, v);
    m = row_max(m, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) m = fmaxf(m, red[threadIdx.x / kRowThreads * kWarps + i]);
  }
  if (!live) return;
  const RowScale s(m);
  if (t == 0) scale[r] = s.s;
  auto put = [&](int i, const float (&v)[8]) { *reinterpret_cast<uint2*>(q + r * ld + i) = s.quantised(v); };
#pragma unroll
  for (int c = 0; c < kKeep; ++c) {
    const int i = (c * kRowThreads + t) * 8;
    if (i < ld) put(i, keep[c]);
  }
  for (int i = (kKeep * kRowThreads + t) * 8; i < ld; i += kRowThreads * 8) {
    float v[8];
    load8(xr, i, n, vec, v);
    put(i, v);
  }
}

template <typename T, int kWarps>
cudaError_t launch_quantize_t(int64_t rows, int n, const T* x, bool vec, int8_t* q, float* scale, cudaStream_t st) {
  constexpr int kRows = kQThreads / 32 / kWarps;
  auto kern = k_quantize_rows<T, kWarps>;
  // the product's split of an SM's memory, so that its CTAs can move in beside this kernel's
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_once(done, reinterpret_cast<const void*>(kern), cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)((rows + kRows - 1) / kRows), kQThreads, 0, st, x, rows, n, vec, q, scale);
}

template <typename T>
cudaError_t launch_quantize(int64_t rows, int n, const void* x, int8_t* q, float* scale, cudaStream_t st) {
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && n % 8 == 0;
  const T* xp = static_cast<const T*>(x);
  // a warp per row where its registers hold the row and the rows fill the SMs; more
  // warps, which end sooner, for the rows of a batch (one row of 768: 2.2 and 1.6 us)
  if (n <= 256 * kKeep && rows >= kManyRows) return launch_quantize_t<T, 1>(rows, n, xp, vec, q, scale, st);
  if (n <= 2 * 256 * kKeep) return launch_quantize_t<T, 4>(rows, n, xp, vec, q, scale, st);
  return launch_quantize_t<T, 8>(rows, n, xp, vec, q, scale, st);
}

// ------------------------------------------------------------- the product
// Persistent CTAs over tiles of 128 labels x BN samples.  The labels are the M
// rows of the MMA (TMEM lanes), so that a warp's store of one sample covers 32
// consecutive logits, and a batch of one still fills the instruction's M.
//   warp 0     TMA producer: 128-byte runs of K of the weight and feature tiles
//              into a ring of NS stages (128B swizzle)
//   warp 1     MMA issuer: kind::i8, K = 32 per instruction, into one of two
//              TMEM accumulators of BN columns
//   warps 2-9  epilogue: warp (q, half) reads lane quarter q of its half of the
//              columns, scales and stores
// 512 x 131,072 x 1024 to bf16: 76 us, 1.8 Pop/s, against 41 us for its bytes at a
// copy's rate.  The MMAs alone take 49 us (199 clocks for 128 x 256 x 32), the whole
// without loads 65 and without the epilogue 58: staging 48 KB for 4 MMAs, the MMAs and
// the epilogue's TMEM reads share an SM's ports.  Up to some hundred samples the
// weights' bytes bound it: 32 x 131,072 x 1024 in 29 us, 4.9 TB/s.
constexpr int kThreads = 320;
constexpr int kML = 128;      // labels per tile
constexpr int kKB = 128;      // K bytes per stage
constexpr int kMaxStages = 8;
constexpr int kMaxBH = 1 << 30;  // B and H: tile coordinates are 32-bit
constexpr int kMaxTiles = 1 << 30;  // a tile's number and the next one's of its CTA fit 32 bits
// Tiles of the narrowest form a batch of B can take.
inline int64_t max_tiles(int64_t B, int64_t H) { return (H + kML - 1) / kML * ((B + 15) / 16); }

struct Args {
  int B, H, nk;  // nk: K stages of a tile
  int n_bt, n_tiles;
  const float* sx;  // [B], readable up to a multiple of 256
  const float* sw;
  void* out;
};

template <int BN>
constexpr int stages() {
  constexpr int fit = 200 * 1024 / ((kML + BN) * kKB);
  return fit < kMaxStages ? fit : kMaxStages;
}
template <int BN>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)stages<BN>() * (kML + BN) * kKB + 512 + 8 * (BN / 2) * 4;
}

__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Signed 8-bit operands, both K-major, 32-bit integer accumulator.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// 32 lanes x kN consecutive columns of 32-bit integers, in flight until landed() is called
// on them.
template <int kN>
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, int (&r)[kN]) {
  static_assert(kN == 8 || kN == 16 || kN == 32, "columns of one load");
  if constexpr (kN == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  } else if constexpr (kN == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  }
}
// Waits for the loads in flight.  The columns are passed on from behind the wait, so that no
// use of them, a conversion in registers included, can be placed before it.
template <int kN>
__device__ __forceinline__ void landed(int (&r)[kN]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < kN; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (*abort_flag) return false;
  if (!mbar_wait(bar, parity, g_wait_limit_ns)) {
    *abort_flag = 1;
    return false;
  }
  return true;
}

// One warp's share of a finished tile: kCols samples from b0 on of the 32 labels of
// its TMEM lane quarter (this lane's label is h), scaled and stored.  The next columns
// leave TMEM while these are stored.
template <typename O, int kCols>
__device__ __forceinline__ void store_tile(const Args& a, uint32_t src, int h, int b0, const float* sxs) {
  constexpr int CH = kCols < 32 ? kCols : 32, kChunks = kCols / CH;
  const int lane = threadIdx.x & 31;
  O* out = static_cast<O*>(a.out);
  const float sw = h < a.H ? a.sw[h] : 0.f;
  // bf16 logits of two neighbouring labels leave as one 4-byte store when every row
  // starts on one (two 2-byte stores of a warp cover the same 64 bytes)
  const bool pairs = sizeof(O) == 2 && (a.H & 1) == 0 && (reinterpret_cast<uintptr_t>(out) & 3) == 0;
  const bool all = h - lane + 32 <= a.H;
  const int n_c = min(kChunks, (a.B - b0 + CH - 1) / CH);
  int v[2][CH];
  if (n_c > 0) tmem_ld_async(src, v[0]);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    if (c >= n_c) break;
    const int(&sum)[CH] = v[c & 1];
    landed(v[c & 1]);
    if (c + 1 < kChunks && c + 1 < n_c) tmem_ld_async(src + (uint32_t)((c + 1) * CH), v[(c + 1) & 1]);
    float z[CH];
#pragma unroll
    for (int i = 0; i < CH; i += 4) {
      const float4 sx = *reinterpret_cast<const float4*>(sxs + c * CH + i);
      z[i] = (float)sum[i] * (sx.x * sw);
      z[i + 1] = (float)sum[i + 1] * (sx.y * sw);
      z[i + 2] = (float)sum[i + 2] * (sx.z * sw);
      z[i + 3] = (float)sum[i + 3] * (sx.w * sw);
    }
    const int left = a.B - b0 - c * CH;  // samples from this column on
    O* row = out + (int64_t)(b0 + c * CH) * a.H + h;
    if (pairs) {
      // even lanes store this label and the next for column i, odd ones the previous
      // label and this one for column i + 1
      const bool odd = lane & 1, in = all || h < a.H;
      O* at = row + (odd ? (int64_t)a.H - 1 : 0);
      const int64_t step = 2 * (int64_t)a.H;
#pragma unroll
      for (int i = 0; i < CH; i += 2, at += step) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? z[i] : z[i + 1], 1);
        const uint32_t pk = odd ? pack_bf16x2(got, z[i + 1]) : pack_bf16x2(z[i], got);
        if (in && i + (odd ? 1 : 0) < left) *reinterpret_cast<uint32_t*>(at) = pk;
      }
    } else if (h < a.H) {
#pragma unroll
      for (int i = 0; i < CH; ++i, row += a.H)
        if (i < left) *row = Elem<O>::from_f(z[i]);
    }
  }
}

// A warp's copy of its samples' scales.
__device__ __forceinline__ void copy_scales(float* sxs, const float* sx, int n) {
  __syncwarp();
  for (int i = threadIdx.x & 31; i < n; i += 32) sxs[i] = sx[i];
  __syncwarp();
}

template <typename O, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_head_i8(Args a, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int NS = stages<BN>();
  constexpr uint32_t kA = kML * kKB, kB = BN * kKB;
  constexpr uint32_t kTmemCols = 2 * BN;
  const uint32_t base = align1024(smem_u32(smem));
  auto SA = [&](int st) -> uint32_t { return base + (uint32_t)st * (kA + kB); };
  auto SB = [&](int st) -> uint32_t { return SA(st) + kA; };
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (base - smem_u32(smem)) + NS * (kA + kB));
  uint64_t* full = bars;                 // [NS] tiles landed
  uint64_t* empty = full + kMaxStages;   // [NS] tiles read (MMA commit)
  uint64_t* acc_full = empty + kMaxStages;  // [2] accumulator complete
  uint64_t* acc_empty = acc_full + 2;       // [2] accumulator read (8 epilogue warps)
  uint64_t* done = acc_empty + 2;           // every MMA of the CTA finished
  uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_w) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_x) : "memory");
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8);
    }
    mbar_init(done, 1);
    // a limit shorter than one sleep: every warp's first wait runs out at once
    *abort_flag = g_wait_limit_ns < kWaitSuspendNs;
    if (*abort_flag) record_error(kErrTimeout);
    fence_mbar_init();
  }
  if (w == 1) {
    tmem_alloc(tslot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  let_next_start();

  if (w == 0) {
    if (lane == 0) {
      // the weights do not depend on the quantisation kernel before this one: its
      // end is awaited only before the first feature tile
      bool waited = false;
      int st = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.n_tiles && ok; t += gridDim.x) {
        const int h0 = t / a.n_bt * kML, b0 = t % a.n_bt * BN;
        for (int k = 0; k < a.nk; ++k) {
          if (!wait_or_abort(&empty[st], ph ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          ++issued;
          mbar_arrive_expect_tx(&full[st], kA + kB);
          tma_load_2d(SA(st), &tm_w, k * kKB, h0, &full[st]);
          if (!waited) {
            wait_for_stream();
            waited = true;
          }
          tma_load_2d(SB(st), &tm_x, k * kKB, b0, &full[st]);
          if (++st == NS) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // no copy may still be landing when the CTA exits
      for (int j = issued > NS ? issued - NS : 0; j < issued; ++j) mbar_wait(&full[j % NS], (j / NS) & 1);
    }
  } else if (w == 1) {
    constexpr uint32_t idesc = idesc_i8(kML, BN);
    int st = 0, ph = 0, it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < a.n_tiles && ok; t += gridDim.x, ++it) {
      const int ac = it & 1;
      if (!__all_sync(0xffffffffu, wait_or_abort(&acc_empty[ac], ((it >> 1) & 1) ^ 1, abort_flag))) break;
      tc_fence_after();
      for (int k = 0; k < a.nk; ++k) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&full[st], ph, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t ad = make_sdesc(SA(st), 16, 1024, kLayoutSw128), bd = make_sdesc(SB(st), 16, 1024, kLayoutSw128);
#pragma unroll
          for (int kk = 0; kk < kKB / 32; ++kk)
            mma_i8(tmem + (uint32_t)(ac * BN), ad + 2 * kk, bd + 2 * kk, idesc, (k > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&empty[st]);
          if (k + 1 == a.nk) mma_commit(&acc_full[ac]);
        }
        __syncwarp();
        if (++st == NS) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (lane == 0) mma_commit(done);  // also after an abort: TMEM is freed only once the MMAs end
    __syncwarp();
  } else {
    wait_for_stream();
    constexpr int kCols = BN / 2;
    const int q = w & 3, half = (w - 2) >> 2;
    float* sxs = reinterpret_cast<float*>(smem + (base - smem_u32(smem)) + NS * (kA + kB) + 512) + (w - 2) * kCols;
    int it = 0, b_have = -1;
    for (int t = blockIdx.x; t < a.n_tiles; t += gridDim.x, ++it) {
      const int ac = it & 1;
      const int h = t / a.n_bt * kML + q * 32 + lane, b0 = t % a.n_bt * BN + half * kCols;
      if (b0 != b_have) {
        copy_scales(sxs, a.sx + b0, kCols);
        b_have = b0;
      }
      if (!__all_sync(0xffffffffu, wait_or_abort(&acc_full[ac], (it >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      store_tile<O, kCols>(a, tmem + (uint32_t)(ac * BN + half * kCols) + ((uint32_t)(q * 32) << 16), h, b0, sxs);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ac]);
    }
    mbar_wait(done, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (w == 1) {
    mbar_wait(done, 0);
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------- the product of a few samples
// Up to 4 samples: one launch without tensor cores, whose latencies (quantisation,
// staging, MMA, TMEM) are most of a small call.  Every CTA quantises the samples into
// shared memory, its first weights already on the way; a warp takes 4 labels at a
// time, its lanes 16-byte pieces of their rows, and adds up 4-way byte products.
// One sample, 4,096 labels x 768: 2.7 us (5.7 through the tiles); 131,072 x 1024:
// 22.8 us, 5.9 TB/s (28.1).  Each sample adds its own shared-memory reads and byte
// products: 4 samples take 4.2 us (5.6) and 28.7 (28.2), 8 would take 5.9 and 44.
constexpr int kFewThreads = 256, kFewLabels = 4, kFewBytes = 32768;

struct FewArgs {
  int B, H, d;
  bool vec;  // rows of x start on 16 bytes and hold whole vectors of 8
  const int8_t* w;
  const float* sw;
  void* out;
};

template <typename O, typename T, int BT>
__global__ void __launch_bounds__(kFewThreads, 2) k_head_i8_few(FewArgs a, const T* __restrict__ x) {
  extern __shared__ __align__(16) uint8_t few_smem[];  // [BT][ld]
  __shared__ uint32_t row_max_bits[BT];
  __shared__ float sxs[BT];
  constexpr int kRounds = 2;  // 512-byte runs of 4 labels' rows in registers
  const int t = threadIdx.x, lane = t & 31, ld = pitch(a.d), n16 = ld / 16;
  const int n_warps = gridDim.x * (kFewThreads / 32), first = blockIdx.x * (kFewThreads / 32) + (t >> 5);
  const int groups = (a.H + kFewLabels - 1) / kFewLabels;
  wait_for_stream();
  let_next_start();
  uint4 wv[kFewLabels][kRounds];
  auto fetch = [&](int g, int c) {  // 16-byte pieces c + lane, c + 32 + lane of group g's rows
#pragma unroll
    for (int l = 0; l < kFewLabels; ++l) {
      const int h = min(g * kFewLabels + l, a.H - 1);
      const uint4* row = reinterpret_cast<const uint4*>(a.w + (int64_t)h * ld);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int p = c + r * 32 + lane;
        wv[l][r] = p < n16 ? row[p] : make_uint4(0, 0, 0, 0);
      }
    }
  };
  if (first < groups) fetch(first, 0);

  // the samples, 8 elements at a time; past the last one zeros
  if (t < BT) row_max_bits[t] = 0;
  __syncthreads();
  const int runs = ld / 8;
  for (int i = t; i < a.B * runs; i += kFewThreads) {
    float v[8];
    load8(x + (int64_t)(i / runs) * a.d, i % runs * 8, a.d, a.vec, v);
    atomicMax(&row_max_bits[i / runs], __float_as_uint(row_max(0.f, v)));
  }
  __syncthreads();
  for (int i = t; i < BT * runs; i += kFewThreads) {
    const int b = i / runs;
    uint2 q = make_uint2(0, 0);
    if (b < a.B) {
      const RowScale s(__uint_as_float(row_max_bits[b]));
      float v[8];
      load8(x + (int64_t)b * a.d, i % runs * 8, a.d, a.vec, v);
      q = s.quantised(v);
      if (i % runs == 0) sxs[b] = s.s;
    }
    *reinterpret_cast<uint2*>(few_smem + b * ld + i % runs * 8) = q;
  }
  __syncthreads();

  O* out = static_cast<O*>(a.out);
  for (int g = first; g < groups; g += n_warps) {
    int acc[kFewLabels][BT] = {};
    for (int c = 0; c < n16; c += 32 * kRounds) {
      if (c > 0) fetch(g, c);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int p = c + r * 32 + lane;
        if (c + r * 32 >= n16) break;
#pragma unroll
        for (int b = 0; b < BT; ++b) {
          const uint4 xv = *reinterpret_cast<const uint4*>(few_smem + b * ld + (p < n16 ? p : 0) * 16);
#pragma unroll
          for (int l = 0; l < kFewLabels; ++l) {
            acc[l][b] = __dp4a((int)wv[l][r].x, (int)xv.x, acc[l][b]);
            acc[l][b] = __dp4a((int)wv[l][r].y, (int)xv.y, acc[l][b]);
            acc[l][b] = __dp4a((int)wv[l][r].z, (int)xv.z, acc[l][b]);
            acc[l][b] = __dp4a((int)wv[l][r].w, (int)xv.w, acc[l][b]);
          }
        }
      }
    }
    if (g + n_warps < groups) fetch(g + n_warps, 0);
    int mine = 0;  // of label lane % 4 and sample lane / 4
#pragma unroll
    for (int l = 0; l < kFewLabels; ++l)
#pragma unroll
      for (int b = 0; b < BT; ++b) {
        const int s = __reduce_add_sync(0xffffffffu, acc[l][b]);
        if (lane == b * kFewLabels + l) mine = s;
      }
    const int h = g * kFewLabels + lane % kFewLabels, b = lane / kFewLabels;
    if (b < a.B && b < BT && h < a.H) out[(int64_t)b * a.H + h] = Elem<O>::from_f((float)mine * (sxs[b] * a.sw[h]));
  }
}

// 2D map of rows of ld bytes in boxes of 128 bytes x box_rows (128B swizzle), zeros
// past the edges.
inline cudaError_t tmap_i8(CUtensorMap* tm, const void* base, uint64_t ld, uint64_t rows, uint32_t box_rows) {
  tail2::EncodeTiledFn enc = tail2::encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {ld, rows}, strides[1] = {ld};
  const cuuint32_t box[2] = {kKB, box_rows}, estr[2] = {1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename O, int BN>
cudaError_t launch_product_t(Args a, int ld, const int8_t* qx, const int8_t* qw, int sms, cudaStream_t st) {
  a.n_bt = (a.B + BN - 1) / BN;
  a.n_tiles = (a.H + kML - 1) / kML * a.n_bt;
  CUtensorMap tm_w, tm_x;
  cudaError_t e = tmap_i8(&tm_w, qw, ld, a.H, kML);
  if (e == cudaSuccess) e = tmap_i8(&tm_x, qx, ld, a.B, BN);
  auto kern = k_head_i8<O, BN>;
  static std::atomic<uint64_t> done{0};
  if (e == cudaSuccess)
    e = set_once(done, reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<BN>());
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)(a.n_tiles < sms ? a.n_tiles : sms), kThreads, smem_bytes<BN>(), st, a, tm_w, tm_x);
}

// Where the tiles are slower: up to 16,384 labels (two launches against one), and one
// or two samples of rows long enough to occupy a warp's lanes (1 x 131,072 x 1024 22.8
// and 28.1 us, but x 256 11.9 and 10.1 us).  In between the two forms change places where
// the rule does not (x 512 13.6 and 15.3 us for one sample, 16.6 and 15.3 for two; x 768 18.5
// and 22.3, 21.7 and 22.5).  Three and four samples of more than 1,024
// features take as long as the tiles, or longer (4 x 16,384 x 4096: 24 and 18 us).
inline int few_samples(int B) { return B <= 2 ? B : 4; }
inline bool few(int B, int H, int ld) {
  if (B > 4 || few_samples(B) * ld > kFewBytes) return false;
  return B <= 2 ? H <= 16384 || ld >= 768 : H <= 16384 && ld <= 1024;
}

template <typename O, typename T, int BT>
cudaError_t launch_few_t(const FewArgs& a, const T* x, int sms, cudaStream_t st) {
  const int per_cta = kFewLabels * kFewThreads / 32, want = (a.H + per_cta - 1) / per_cta;
  return launch_early(k_head_i8_few<O, T, BT>, (unsigned)(want < 2 * sms ? want : 2 * sms), kFewThreads,
                      (size_t)BT * pitch(a.d), st, a, x);
}
template <typename O, typename T>
cudaError_t launch_few(int B, int H, int d, const void* x, const int8_t* qw, const float* sw, void* out, int sms,
                       cudaStream_t st) {
  const FewArgs a{B, H, d, reinterpret_cast<uintptr_t>(x) % 16 == 0 && d % 8 == 0, qw, sw, out};
  const T* xp = static_cast<const T*>(x);
  switch (few_samples(B)) {
    case 1: return launch_few_t<O, T, 1>(a, xp, sms, st);
    case 2: return launch_few_t<O, T, 2>(a, xp, sms, st);
    default: return launch_few_t<O, T, 4>(a, xp, sms, st);
  }
}

// Samples per tile: the width (not above the batch's, rounded up) whose rounds of tiles
// over the SMs stage the fewest bytes, 128 + BN rows a tile.  Measured against the
// others at d = 768: 256 x 16,384 labels 10.6 us with 256 (12.1 with 128, 16.0 with
// 64), 256 x 8,192 8.4 us with 128 (10.3 with 64).
inline int tile_samples(int B, int H, int sms) {
  const int64_t lt = (H + kML - 1) / kML;
  int best = 16;
  int64_t least = INT64_MAX;
  for (int bn = 16; bn <= 256; bn *= 2) {
    const int64_t rounds = (lt * ((B + bn - 1) / bn) + sms - 1) / sms, rows = rounds * (kML + bn);
    if (rows <= least) {
      best = bn;
      least = rows;
    }
    if (bn >= B) break;
  }
  return best;
}

template <typename O>
cudaError_t launch_product(int B, int H, int ld, const int8_t* qx, const float* sx, const int8_t* qw, const float* sw,
                           void* out, int sms, cudaStream_t st) {
  Args a{};
  a.B = B;
  a.H = H;
  a.nk = (ld + kKB - 1) / kKB;
  a.sx = sx;
  a.sw = sw;
  a.out = out;
  switch (tile_samples(B, H, sms)) {
    case 16: return launch_product_t<O, 16>(a, ld, qx, qw, sms, st);
    case 32: return launch_product_t<O, 32>(a, ld, qx, qw, sms, st);
    case 64: return launch_product_t<O, 64>(a, ld, qx, qw, sms, st);
    case 128: return launch_product_t<O, 128>(a, ld, qx, qw, sms, st);
    default: return launch_product_t<O, 256>(a, ld, qx, qw, sms, st);
  }
}

}  // namespace head8
}  // namespace haste
