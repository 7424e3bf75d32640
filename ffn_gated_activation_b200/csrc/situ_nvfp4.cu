// situ_nvfp4.cu -- NVFP4 storage of any matrix and the grouped NVFP4 product
// (include/situ_glu.h, situ_glu_nvfp4_*).
//
// The format (as situ_glu_fwd_nvfp4 writes it): with A the largest finite |x|
// of the matrix, each block of 16 elements of a row has the scale
// s_b = E4M3(amax_b 448 / A) and the codes E2M1(x 2688 / (A s_b)); a code q
// stands for q s_b A / 2688.

#include <type_traits>

#include "situ_host.cuh"

namespace {

#include "situ_fused_gemm.cuh"

// ---------------------------------------------------------------------------
// Storage
// ---------------------------------------------------------------------------
// One thread has one block of 16 elements: 32 (bf16) or 64 (fp32) bytes in, 8
// bytes of codes and a scale byte out, no exchange between lanes.  HBM
// bandwidth is the bound (2.56 bytes an element of bf16 where A is known, 4.56
// where the first pass has to find it).

constexpr int kStoreThreads = 256;

struct StoreArgs {
  const char* x;        // quantise: the matrix; dequantise: unused
  int64_t x_pitch;      // bytes
  char* data;
  int64_t data_pitch;
  uint8_t* scale;
  int64_t scale_pitch;
  const float* amax;
  unsigned int* amax_out;
  char* out;            // dequantise: the matrix
  int64_t out_pitch;
  int64_t rows;
  int64_t blocks;       // rows * per_row
  uint32_t per_row;     // blocks of 16 elements
  int wide;             // the matrix' vectors are 32-byte aligned
  int flat;             // no gaps between rows anywhere: one long row
};

// Row and column block of block i.
__device__ __forceinline__ void block_at(const StoreArgs& a, int64_t i, int64_t& row, int64_t& col) {
  if (a.flat) {
    row = 0;
    col = i;
  } else if (a.blocks <= 0xffffffffll) {
    const uint32_t r = static_cast<uint32_t>(i) / a.per_row;
    row = r;
    col = static_cast<uint32_t>(i) - r * a.per_row;
  } else {
    row = i / a.per_row;
    col = i - row * a.per_row;
  }
}

// The 16 elements of a block as fp32 pairs.
template <typename S>
__device__ __forceinline__ void load_block(const char* p, int wide, uint4 (&v)[8 / S::kPairs]) {
#pragma unroll
  for (int k = 0; k < 8 / S::kPairs; k += 2) {
    if (wide) {
      const U8 u = ld_stream32(p + k * kVecBytes);
      v[k] = u.a;
      v[k + 1] = u.b;
    } else {
      v[k] = ld_stream(p + k * kVecBytes);
      v[k + 1] = ld_stream(p + (k + 1) * kVecBytes);
    }
  }
}
template <typename S>
__device__ __forceinline__ float2 block_pair(const uint4 (&v)[8 / S::kPairs], int p) {
  return as_f2(S::pair(v[p / S::kPairs], p % S::kPairs));
}

// The largest magnitude of a block, NaN if there is one.
template <typename S>
__device__ __forceinline__ float block_max(const uint4 (&v)[8 / S::kPairs]) {
  if constexpr (S::kPairs == 4) {  // two bf16 at a time
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    }
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  } else {
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float2 f = block_pair<S>(v, p);
      m = max_nan(m, max_nan(fabsf(f.x), fabsf(f.y)));
    }
    return m;
  }
}

// The same of its finite elements.
template <typename S>
__device__ __forceinline__ float block_finite_max(const uint4 (&v)[8 / S::kPairs]) {
  float m = block_max<S>(v);
  if (m <= 3.402823466e38f) return m;
  m = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const float2 f = block_pair<S>(v, p);
    const float ax = fabsf(f.x), ay = fabsf(f.y);
    m = ax <= 3.402823466e38f ? fmaxf(m, ax) : m;  // false for NaN and infinity
    m = ay <= 3.402823466e38f ? fmaxf(m, ay) : m;
  }
  return m;
}

// Where block i of the matrix lies, and its elements.
template <typename S>
__device__ __forceinline__ void get_block(const StoreArgs& a, int64_t i, int64_t& row, int64_t& col,
                                          uint4 (&v)[8 / S::kPairs]) {
  block_at(a, i, row, col);
  load_block<S>(a.x + row * a.x_pitch + col * (8 / S::kPairs * kVecBytes), a.wide, v);
}

// The largest finite magnitude: per-thread maxima, one integer atomicMax per CTA
// (non-negative floats order as integers), so the result is order-free.
template <typename S>
__global__ void __launch_bounds__(kStoreThreads) situ_nvfp4_amax_kernel(const StoreArgs a) {
  float m = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kStoreThreads;
  int64_t i = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x, row;
  int64_t col;
  uint4 u[8 / S::kPairs], v[8 / S::kPairs];
  for (; i + step < a.blocks; i += 2 * step) {  // two blocks in flight
    get_block<S>(a, i, row, col, u);
    get_block<S>(a, i + step, row, col, v);
    m = fmaxf(m, fmaxf(block_finite_max<S>(u), block_finite_max<S>(v)));
  }
  if (i < a.blocks) {
    get_block<S>(a, i, row, col, u);
    m = fmaxf(m, block_finite_max<S>(u));
  }
  __shared__ unsigned int warp_max[kStoreThreads / 32];
  unsigned int bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = bits;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kStoreThreads / 32; ++w) bits = max(bits, warp_max[w]);
    if (bits != 0u) atomicMax(a.amax_out, bits);
  }
}

// Correctly rounded codes.  bf16 elements under an A of at most 12 significant
// bits (a bf16 tensor's own maximum, say): x 2688 has 13 bits, A s_b 16, and their
// quotient is either a midpoint of E2M1 or at least 2^-19 away from it.  One
// correction by the exact residual makes a quotient that fp32 can hold exact (P.
// Markstein, 1990), so ties come out as ties and nothing else crosses.
//
// In general the fp32 quotients below are within 2^-22 of the
// exact ones, so a code can differ from the exact quotient's only where moving
// the quotient by 2^-20 either way changes it; there the exact products on
// both sides of the midpoint are compared in double (all of them have at most
// 36 significant bits).
constexpr float kUp = 1.0f + 0x1p-20f, kDown = 1.0f - 0x1p-20f;

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
// E4M3(m 448 / big) for m >= 0; r is 448 / big rounded.
__device__ __forceinline__ uint32_t exact_scale(float m, float big, float r) {
  const float v = m * r;
  const uint32_t lo = e4m3_code(v * kDown), hi = e4m3_code(v * kUp);
  if (lo == hi) return lo;
  const double mid = 0.5 * (static_cast<double>(e4m3_value(lo)) + static_cast<double>(e4m3_value(hi)));
  const double left = static_cast<double>(m) * 448.0, right = mid * static_cast<double>(big);
  return left > right || (left == right && (hi & 1) == 0) ? hi : lo;
}
// The magnitude code of E2M1(m 2688 / (big s)) where lo and hi are the codes of
// the quotient moved down and up.
__device__ __forceinline__ uint32_t exact_code(float m, double big_s, uint32_t lo, uint32_t hi) {
  const uint32_t twice = 0xC8643210u;  // 2 x the magnitudes 0, .5, 1, 1.5, 2, 3, 4 of the codes 0 .. 6 (6 is 12: C)
  const double mid = 0.25 * (static_cast<double>((twice >> (4 * lo)) & 15u) + static_cast<double>((twice >> (4 * hi)) & 15u));
  const double left = static_cast<double>(m) * 2688.0, right = mid * big_s;
  return left > right || (left == right && (hi & 1) == 0) ? hi : lo;
}
// The codes of eight elements where `down` and `up` differ: a tie, as a rule (one
// element in a thousand of bf16 data), one element at a time.
__device__ __noinline__ uint32_t exact_codes(float2 f0, float2 f1, float2 f2, float2 f3, float big, float s, uint32_t down,
                                             uint32_t up) {
  const double big_s = static_cast<double>(big) * static_cast<double>(s);
  const float f[8] = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
  uint32_t diff = down ^ up;
  while (diff != 0) {
    const int at = (__ffs(static_cast<int>(diff)) - 1) & ~3;
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) m = at == 4 * p ? fabsf(f[p]) : m;
    const uint32_t code = exact_code(m, big_s, (down >> at) & 7u, (up >> at) & 7u);
    down = (down & ~(7u << at)) | (code << at);
    diff &= ~(15u << at);
  }
  return down;
}

// The tensor scale of a quantisation: A (2688 where it is 0 or not finite, S_enc
// = 1), and for a tiny A both sides times 2^80, exactly, so that 448 / A stays
// finite.
struct TensorScale {
  float lift, big, r448, s_enc;
  bool short_big;  // at most 12 significant bits
  __device__ __forceinline__ explicit TensorScale(float amax) {
    big = amax > 0.0f && amax <= 3.402823466e38f ? amax : 2688.0f;
    lift = big < 0x1p-60f ? 0x1p80f : 1.0f;
    big *= lift;
    r448 = 448.0f / big;
    s_enc = 2688.0f / big;
    short_big = (__float_as_uint(big) & 0xfffu) == 0 && big >= 0x1p-60f && big <= 0x1p60f && lift == 1.0f;
  }
};

// bf16 elements to +-cap, so that no product below is infinite and the residual of a
// saturated element keeps its sign.
__device__ __forceinline__ void clamp_block(uint4 (&v)[2], float cap) {
  const __nv_bfloat162 hi = __float2bfloat162_rn(cap), lo = __hneg2(hi);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&w[i]);
      x = __hmax2(__hmin2(x, hi), lo);
      w[i] = *reinterpret_cast<uint32_t*>(&x);
    }
  }
}

// GIVEN: elements may lie above A.
template <typename S, bool EXACT, bool GIVEN>
__device__ __forceinline__ void quantize_block(const StoreArgs& a, const TensorScale& t, int64_t row, int64_t col,
                                               uint4 (&v)[8 / S::kPairs]) {
  const float m = block_max<S>(v);
  const bool special = !(m <= 3.402823466e38f);
  const uint32_t sc = special ? 0x7fu : exact_scale(m * t.lift, t.big, t.r448);
  if (!EXACT && t.lift != 1.0f) {  // a power of two: exact in either type (too large is infinite, and saturates)
#pragma unroll
    for (int p = 0; p < 8; ++p)
      S::put(v[p / S::kPairs], p % S::kPairs, mul2(block_pair<S>(v, p), splat(t.lift)));
  }
  uint32_t q[2] = {0u, 0u};
  if (!special) {
    const float s = e4m3_value(sc);
    const float inv = s > 0.0f ? __fdividef(t.s_enc, s) : 0.0f;  // 2 ulp
    if constexpr (EXACT) {
      if constexpr (GIVEN && S::kPairs == 4) {
        if (m * inv > 16.0f) clamp_block(v, 16.0f / inv);  // far beyond the largest code, 6
      }
      const float2 d = splat(-(t.big * s)), r = splat(inv), r1 = splat(inv * (1.0f / 2688.0f));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 w[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 f = block_pair<S>(v, 4 * h + p);
          const float2 w0 = mul2(f, r);
          w[p] = fma2(fma2(w0, d, mul2(f, splat(2688.0f))), r1, w0);
        }
        q[h] = e2m1x8(w);
      }
    } else {
      const float2 up = splat(inv * kUp), down = splat(inv * kDown);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 u[4], d[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 f = block_pair<S>(v, 4 * h + p);
          u[p] = mul2(f, up);
          d[p] = mul2(f, down);
        }
        const uint32_t hi = e2m1x8(u), lo = e2m1x8(d);
        q[h] = lo;
        if (lo != hi)
          q[h] = exact_codes(block_pair<S>(v, 4 * h), block_pair<S>(v, 4 * h + 1), block_pair<S>(v, 4 * h + 2),
                             block_pair<S>(v, 4 * h + 3), t.big, s, lo, hi);
      }
    }
  }
  st_stream8(a.data + row * a.data_pitch + col * 8, make_uint2(q[0], q[1]));
  a.scale[row * a.scale_pitch + col] = static_cast<uint8_t>(sc);
}

// Blocks [0, blocks) from the end: what the pass before read last may still be in
// L2; a thread's next block is on its way while this one is coded.
template <typename S, bool EXACT, bool GIVEN>
__device__ __forceinline__ void quantize_blocks(const StoreArgs& a, const TensorScale& t, int64_t k, int64_t step) {
  int64_t row, next_row, col, next_col;
  if (k >= a.blocks) return;
  uint4 v[8 / S::kPairs], next[8 / S::kPairs];
  get_block<S>(a, a.blocks - 1 - k, row, col, v);
  for (;;) {
    k += step;
    const bool more = k < a.blocks;
    if (more) get_block<S>(a, a.blocks - 1 - k, next_row, next_col, next);
    quantize_block<S, EXACT, GIVEN>(a, t, row, col, v);
    if (!more) break;
#pragma unroll
    for (int i = 0; i < 8 / S::kPairs; ++i) v[i] = next[i];
    row = next_row;
    col = next_col;
  }
}

template <typename S, bool GIVEN>
__global__ void __launch_bounds__(kStoreThreads) situ_nvfp4_quantize_kernel(const StoreArgs a) {
  const TensorScale t(*a.amax);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kStoreThreads;
  if (std::is_same<S, Bf16>::value && t.short_big) quantize_blocks<S, true, GIVEN>(a, t, first, step);
  else quantize_blocks<S, false, GIVEN>(a, t, first, step);
}

// The two halves of a barrier that tells only that every CTA of the cluster has
// started: before it, the shared memory of another one may not be there yet.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_started() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A small matrix in one launch: a cluster of eight CTAs finds A, exchanges it
// through shared memory and quantises what it has just read (from L2).  Against a
// fill and two launches (bf16, us in a graph): 7168 blocks 3.9, 6.2; 16576 5.7, 6.2;
// 33152 8.3, 6.2.  Call by call, where the host is the bound, 13.3 and 17.0 up to
// 49280 blocks; the limit lies between the two.
constexpr int kSmallCtas = 8, kSmallThreads = 1024;
constexpr int64_t kSmallBlocks = 32768;  // blocks of 16
template <typename S>
__global__ void __cluster_dims__(kSmallCtas, 1, 1) __launch_bounds__(kSmallThreads) situ_nvfp4_small_kernel(const StoreArgs a) {
  __shared__ unsigned int warp_max[kSmallThreads / 32];
  __shared__ unsigned int cta_max[kSmallCtas];
  cluster_started();  // waited for before the first store to another CTA
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x, step = kSmallCtas * kSmallThreads;
  int64_t row;
  int64_t col;
  uint4 v[8 / S::kPairs];
  float m = 0.0f;
  for (int64_t i = first; i < a.blocks; i += step) {
    get_block<S>(a, i, row, col, v);
    m = fmaxf(m, block_finite_max<S>(v));
  }
  const unsigned int bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = bits;
  __syncthreads();
  cluster_wait_started();
  if (threadIdx.x < 32) {
    const unsigned int most = __reduce_max_sync(0xffffffffu, warp_max[threadIdx.x]);
    if (threadIdx.x < kSmallCtas)  // into slot `rank` of CTA threadIdx.x
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(&cta_max[cluster_rank()], threadIdx.x)), "r"(most)
                   : "memory");
  }
  cluster_sync();
  unsigned int most = 0;
#pragma unroll
  for (int c = 0; c < kSmallCtas; ++c) most = max(most, cta_max[c]);
  const float amax = __uint_as_float(most);
  if (first == 0) *reinterpret_cast<float*>(a.amax_out) = amax;
  const TensorScale t(amax);
  if (std::is_same<S, Bf16>::value && t.short_big) quantize_blocks<S, true, false>(a, t, first, step);
  else quantize_blocks<S, false, false>(a, t, first, step);
}

// Two E2M1 codes as an exact half2.
__device__ __forceinline__ float2 e2m1_pair(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <typename S>
__global__ void __launch_bounds__(kStoreThreads) situ_nvfp4_dequantize_kernel(const StoreArgs a) {
  const double unit = static_cast<double>(*a.amax) / 2688.0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kStoreThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x; i < a.blocks; i += step) {
    int64_t row;
    int64_t col;
    block_at(a, i, row, col);
    const uint2 q = ld_stream8(a.data + row * a.data_pitch + col * 8);
    const float s = static_cast<float>(unit * static_cast<double>(e4m3_value(a.scale[row * a.scale_pitch + col])));
    uint4 o[8 / S::kPairs];
#pragma unroll
    for (int p = 0; p < 8; ++p)
      S::put(o[p / S::kPairs], p % S::kPairs, mul2(e2m1_pair(((p < 4 ? q.x : q.y) >> (8 * (p & 3))) & 0xffu), splat(s)));
    char* out = a.out + row * a.out_pitch + col * (8 / S::kPairs * kVecBytes);
#pragma unroll
    for (int k = 0; k < 8 / S::kPairs; k += 2) {
      if (a.wide) {
        st_stream32(out + k * kVecBytes, o[k], o[k + 1]);
      } else {
        st_stream(out + k * kVecBytes, o[k]);
        st_stream(out + (k + 1) * kVecBytes, o[k + 1]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Grouped product
// ---------------------------------------------------------------------------
// out[r, n] = sum_k a[r, k] w_e[n, k] on the fp4 tensor cores
// (tcgen05.mma.kind::mxf4nvf4, a UE4M3 scale per 16 elements of k): the tensor
// cores multiply the codes by their block scales and add in fp32; the two
// tensor scales, one number per expert, are applied once in the epilogue.
//
// A cluster of two CTAs (tcgen05 cta_group::2), persistent over the output tiles of
// 256 rows and BN = 256 or 128 columns, numbered expert by expert as in
// situ_fused_gemm.cuh.  One product is M = 256, N = BN, k = 64: CTA r stages rows
// [128 r, 128 r + 128) of the A tile and its half of the B tile and holds
// accumulator rows [128 r, ...) in its TMEM.
//   * warp 0 streams the codes with TMA, a stage being 256 elements of k, i.e. a
//     128-byte swizzle row of A and of B;
//   * warps 6-9 write the block scales to TMEM, where the tensor cores read them
//     (32-lane x 4-column atoms: row r's four scales of a product at lane r % 32,
//     column r / 32), the same to each quarter of the lanes;
//   * warp 1 of CTA 0 issues four products a stage;
//   * warps 2-5 store the accumulator, one row a thread.
// Every wait is bounded as in situ_fused_gemm.cuh.
//
// Two SMs a tile: per operation of the tensor cores an SM then moves 5 / 8 of the
// operand bytes of one-SM tiles of 128 x 192, which spent 640 cycles a stage on
// them for 384 of products (8192 x 7168 x 4096: 177 us, this form 94 us; 8 x 7168 x
// 2048: 22, 16).  Scales by tcgen05.st: the tensor pipe takes about 55 cycles for
// each 512-byte tcgen05.cp and runs no product meanwhile (154 us that way).
//
// The scales of four stages come in one go, 64 bytes of each row (64-byte swizzle);
// lane l of each scale warp takes rows l, l + 32, ... of a stage and has in its
// registers just the TMEM columns of its lane.  Where every row of scales starts on
// 16 bytes they are a TMA box, issued in line with the codes; otherwise (rows of k /
// 16 bytes, k not a multiple of 256) warps 10 and 11 copy them, eight or four bytes
// at a time (8192 x 7168 x 4096: 97 and 119 us, by TMA 94 us; copied by the scale
// warps themselves, between their writes to TMEM, 114 and 132 us).
//
// The epilogue drains the accumulator to registers before it stores (bf16), so
// the next tile's products wait for the drain alone, and turns rows into whole
// 128-byte lines through shared memory (16384 x 1024 x 4096 with a 16-byte piece
// of 32 rows per store: 33 of 87 us).
//
// Waits poll with CTA scope; where the other CTA's work is waited for, one
// acquire at cluster scope follows.  (Polling with cluster scope empties L1 each
// time: 8192 x 7168 x 4096 took 253 us.)

namespace nvgemm {

using fc1::decode_tile;
using fc1::scan_experts;
using fc1::smem_desc_sw128;
using fc1::tc_fence_after;
using fc1::tc_fence_before;
using fc1::Tile;
using fc1::tma_load_2d;
using fc1::tma_load_2d_pair;
using fc1::tmem_ld16;
using fc1::tmem_ld_wait;
using fc1::umma_commit_pair;
using fc1::umma_commit_pair_local;
using fc1::wait_or_abort;

constexpr int kBM = 256;               // rows of a tile, 128 of them a CTA's
constexpr int kStageK = 256;           // elements of k per stage
constexpr int kStageRow = 128;         // their bytes
constexpr int kSteps = 4;              // products (k = 64) per stage
constexpr int kMaxExperts = 1024;
constexpr int kHeader = 256;
constexpr int kEpiWarps = 4;
constexpr int kScaleWarps = 4;         // one per quarter of the TMEM lanes
constexpr int kCopyWarps = 2;
constexpr int kThreads = 32 * (2 + kEpiWarps + kScaleWarps + kCopyWarps);
constexpr int kOutBytes = 32 * 128;    // a warp's piece of the output

// Sizes of a kernel with BN output columns per tile.
template <int BN>
struct Shape {
  static constexpr int kABytes = 128 * kStageRow, kBBytes = BN / 2 * kStageRow;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kAccs = 256 / BN;                      // accumulators
  static constexpr int kScaleRows = 128 + BN;                 // scales of a stage: A's rows, then B's
  static constexpr int kGroupBytes = kScaleRows * 64;         // of four stages
  static constexpr int kGroups = BN / 32;                     // TMEM columns of B's scales per step
  static constexpr int kScaleCols = kSteps * (4 + kGroups);   // of a stage
  static constexpr int kScaleBase = kAccs * BN;
  static constexpr int kSmem = kStages * kStageBytes + 2 * kGroupBytes + kEpiWarps * kOutBytes;
  static_assert(kScaleBase + kStages * kScaleCols <= 512, "TMEM overflows");
  // kind::mxf4nvf4: E2M1 A and B (bits 7-9, 10-11 = 1), K-major, N >> 3 at bits
  // 17-22, UE4M3 scales (bit 23 = 0), M >> 7 at bits 27-28, scale ids 0, k = 64.
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BN >> 3) << 17) | (2u << 27);
};

struct Args {
  const uint8_t* a_scale;
  int64_t a_scale_pitch;
  const uint8_t* w_scale;
  int64_t w_scale_pitch;
  const float* a_amax;
  const float* w_amax;
  int64_t w_amax_stride;
  const int64_t* offsets;
  int experts;
  int64_t tokens;
  int k, n;
  int scale_bytes;  // 16: the scales come by TMA; 8, 4: by copies of so many bytes
  char* out;
  int64_t out_pitch;
  int out_bf16;
};

__device__ __forceinline__ bool wait_or_abort_acquire(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (!wait_or_abort(bar, parity, abort_flag)) return false;
  (void)mbar_try_wait_cluster(bar, parity);  // completed already: the acquire alone
  return true;
}

// The whole warp comes here and one lane (`lead`) issues, so that the operands
// stay in uniform registers.
__device__ __forceinline__ void umma_nvfp4_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                                uint32_t sfb, uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(lead)
      : "memory");
}
// Arrive on an mbarrier of either CTA after TMEM writes that are complete
// or reads that are complete (tcgen05.wait) and fenced: nothing in memory hangs
// on the arrival, and a release at cluster scope would wait for the warp's loads
// and stores in flight as well (1000 and more cycles a stage).
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// The factor A_a A_w / 2688^2 as unit * lift.  Sums of products are 0 or lie in [2^-20,
// 2^54]; where the factor alone leaves the range in which fp32 keeps its precision,
// they are multiplied by a power of two first, which is exact.
__device__ __forceinline__ bool unit_in_range(double u) { return fabs(u) >= 0x1p-90 && fabs(u) <= 0x1p90; }
struct FarUnit {
  float unit, lift;
  __device__ __forceinline__ explicit FarUnit(double u) {
    lift = fabs(u) < 0x1p-90 ? 0x1p-100f : 0x1p64f;
    const double rest = u / static_cast<double>(lift);
    unit = static_cast<float>(rest);
    if (isinf(unit) && !isinf(u)) unit = copysignf(3.402823466e38f, unit);  // sums of 0 stay 0
  }
  __device__ __forceinline__ float operator()(uint32_t sum) const { return __uint_as_float(sum) * lift * unit; }
};
// Stores 128 bytes of each of a warp's 32 output rows, row0 + lane's in q:
// columns [c, c + 8 per_vec) of the tile, `per_vec` of them in 16 bytes, those
// below `cols` (a multiple of 8) and rows below the expert's end.  Through the
// warp's 4 KB of shared memory (16-byte chunks swizzled by the row), so that
// eight lanes write a row's line.
__device__ __forceinline__ void put_piece(unsigned char* piece, const Args& a, const Tile& tile, int64_t row0,
                                          const uint32_t* q, int c, int cols, int per_vec) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // the piece before is read
#pragma unroll
  for (int v = 0; v < 8; ++v)
    *reinterpret_cast<uint4*>(piece + lane * 128 + ((v ^ (lane & 7)) * 16)) =
        make_uint4(q[4 * v], q[4 * v + 1], q[4 * v + 2], q[4 * v + 3]);
  __syncwarp();
  const int v = lane & 7;
  if (c + v * per_vec < cols) {
    char* out = a.out + row0 * a.out_pitch + static_cast<int64_t>(tile.n0 + c + v * per_vec) * (16 / per_vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (row0 + r < tile.m_end)
        *reinterpret_cast<uint4*>(out + r * a.out_pitch) = lds16(piece + r * 128 + ((v ^ (r & 7)) * 16));
    }
  }
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Copies G bytes to shared memory of which `real` (0 to G) are read, the rest zero.
template <int G>
__device__ __forceinline__ void cp_async(unsigned char* dst, const uint8_t* src, int real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(G), "r"(real) : "memory");
}
// The copy warps' part of a group of scales: 64 bytes (four stages, from byte k0 of
// the row on) of `rows` rows, of which the first `left` exist and have `width` bytes;
// as the TMA box has them (16-byte chunks swizzled by (row / 2) % 4, zeros outside).
template <int G>
__device__ __forceinline__ void copy_scales(unsigned char* dst, const uint8_t* base, int64_t pitch, int64_t left, int rows,
                                            int k0, int width) {
  constexpr int kPer = 64 / G, kPass = 32 * kCopyWarps / kPer;  // pieces of a row, rows of a pass
  const int x = static_cast<int>(threadIdx.x) - (kThreads - 32 * kCopyWarps);
  const int off = x % kPer * G;
  const int in = max(0, min(G, width - k0 - off));
  const uint8_t* src = base + (x / kPer) * pitch + k0 + off;
#pragma unroll 4
  for (int r = x / kPer; r < rows; r += kPass, src += kPass * pitch) {
    const int real = r < left ? in : 0;
    cp_async<G>(dst + r * 64 + (((off >> 4) ^ ((r >> 1) & 3)) << 4) + (off & 15), real != 0 ? src : base, real);
  }
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    situ_nvfp4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                                const __grid_constant__ CUtensorMap tmap_as, const __grid_constant__ CUtensorMap tmap_ws,
                                const Args a) {
  using P = Shape<BN>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  unsigned char* ring = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  unsigned char* scales = ring + P::kStages * P::kStageBytes;
  unsigned char* pieces = scales + 2 * P::kGroupBytes;
  unsigned char* header = ring + P::kSmem;
  uint64_t* full = reinterpret_cast<uint64_t*>(header);
  uint64_t* empty = full + P::kStages;
  uint64_t* acc_full = empty + P::kStages;
  uint64_t* acc_empty = acc_full + P::kAccs;
  uint64_t* sf_full = acc_empty + P::kAccs;  // [2]: this CTA's scales of four stages
  uint64_t* sf_empty = sf_full + 2;
  uint64_t* drain = sf_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * P::kStages + 2 * P::kAccs + 5) * 8 + 8 <= kHeader, "header overflows");
  int64_t* lo = reinterpret_cast<int64_t*>(header + kHeader);
  int64_t* hi = lo + a.experts;
  int* first_tile = reinterpret_cast<int*>(hi + a.experts);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool own_scales = a.scale_bytes < 16;  // the copy warps bring them
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int cl = static_cast<int>(cluster_index()), ncl = static_cast<int>(cluster_count());
  const int n_tiles = (a.n + BN - 1) / BN;
  const int k_blocks = (a.k + kStageK - 1) / kStageK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(&full[s], 1 + 2 * kScaleWarps);  // CTA 0's: its TMA warp, both CTAs' scale warps and bytes
      mbar_init(&empty[s], 1);                       // CTA 0's commit, to both
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sf_full[b], own_scales ? 32 * kCopyWarps : 1);
      mbar_init(&sf_empty[b], kScaleWarps);
    }
    for (int b = 0; b < P::kAccs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * 32 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0) scan_experts<kBM>(a, n_tiles, lane, lo, hi, first_tile);
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = first_tile[a.experts];

  if (warp == 0) {
    // ---- codes and scales (both CTAs) ----
    int stage = 0, group = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int t = cl; ok && t < total; t += ncl) {
      const Tile tile = decode_tile<kBM>(t, first_tile, lo, hi, a.experts, n_tiles, BN);
      const int32_t arow = static_cast<int32_t>(tile.m0 + 128 * rank);
      const int32_t wrow = tile.expert * a.n + tile.n0 + static_cast<int32_t>(BN / 2 * rank);
      // a CTA none of whose rows exist multiplies what its ring holds, stored nowhere
      const bool second = tile.m_end - tile.m0 > 128;
      for (int kb = 0; kb < k_blocks; ++kb) {
        if (!own_scales && (kb & 3) == 0) {  // the scales of stages kb .. kb + 3
          const int b = group & 1;
          if (!wait_or_abort(&sf_empty[b], ((group >> 1) & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            unsigned char* sc = scales + b * P::kGroupBytes;
            mbar_arrive_expect_tx(&sf_full[b], P::kGroupBytes);
            tma_load_2d(sc, &tmap_as, kb * 16, arow, &sf_full[b]);
            tma_load_2d(sc + 128 * 64, &tmap_ws, kb * 16, tile.expert * a.n + tile.n0, &sf_full[b]);
          }
          __syncwarp();
          ++group;
        }
        if (!wait_or_abort(&empty[stage], phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          unsigned char* st = ring + stage * P::kStageBytes;
          const uint32_t bar = peer_addr(&full[stage], 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], (second ? 2 : 1) * P::kABytes + 2 * P::kBBytes);
          if (leader || second) tma_load_2d_pair(st, &tmap_a, kb * kStageRow, arow, bar);
          tma_load_2d_pair(st + P::kABytes, &tmap_w, kb * kStageRow, wrow, bar);
        }
        __syncwarp();
        issued |= 1u << stage;
        if (++stage == P::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      // Aborted: let this CTA's scales land, and CTA 0 wait for both CTAs' codes
      // (they count on its barriers); bounded.
      for (int g = group > 2 ? group - 2 : 0; g < group; ++g) {
        const unsigned long long t0 = global_timer_ns();
        while (!mbar_try_wait(&sf_full[g & 1], (g >> 1) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
    if (!ok && leader) {
      for (int s = 0; s < P::kStages; ++s) {
        if (!(issued & (1u << s))) continue;
        const uint32_t ph = (s < stage) ? phase : (phase ^ 1u);
        const unsigned long long t0 = global_timer_ns();
        while (!mbar_try_wait_cluster(&full[s], ph) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---- products (CTA 0) ----
      int stage = 0, b = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = cl; ok && t < total; t += ncl) {
        const uint32_t d = tmem_base + static_cast<uint32_t>(b * BN);
        if (!wait_or_abort_acquire(&acc_empty[b], acc_phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!wait_or_abort_acquire(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(ring + stage * P::kStageBytes);
          const uint64_t adesc = smem_desc_sw128(a_addr), bdesc = smem_desc_sw128(a_addr + P::kABytes);
          const uint32_t sfa = tmem_base + P::kScaleBase + static_cast<uint32_t>(stage * P::kScaleCols);
          const uint32_t sfb = sfa + kSteps * 4;
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
            umma_nvfp4_pair(d, adesc + 2 * s, bdesc + 2 * s, P::kIdesc, sfa + 4 * s, sfb + P::kGroups * s,
                            (kb | s) != 0 ? 1u : 0u, lane == 0);
          if (lane == 0) umma_commit_pair(&empty[stage]);
          __syncwarp();
          if (++stage == P::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (lane == 0) umma_commit_pair(&acc_full[b]);
        __syncwarp();
        if (++b == P::kAccs) {
          b = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok || *abort_flag) {
        if (lane == 0) umma_commit_pair_local(drain);
        __syncwarp();
        const unsigned long long t0 = global_timer_ns();
        while (!mbar_try_wait_cluster(drain, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    // ---- epilogue: one accumulator row per thread ----
    const int quarter = warp & 3;
    const double unit_a = static_cast<double>(*a.a_amax) / 2688.0;
    unsigned char* piece = pieces + (warp - 2) * kOutBytes;
    uint32_t acc_phase = 0;
    int b = 0;
    for (int t = cl; t < total; t += ncl) {
      const uint32_t empty_addr = peer_addr(&acc_empty[b], 0);
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(b * BN);
      const Tile tile = decode_tile<kBM>(t, first_tile, lo, hi, a.experts, n_tiles, BN);
      const double factor = unit_a * (static_cast<double>(a.w_amax[tile.expert * a.w_amax_stride]) / 2688.0);
      const float unit = static_cast<float>(factor);
      const bool far = !unit_in_range(factor);
      const int64_t row0 = tile.m0 + 128 * rank + quarter * 32;
      const int cols = min(BN, a.n - tile.n0);
      if (!wait_or_abort(&acc_full[b], acc_phase, abort_flag)) break;
      tc_fence_after();
      if (row0 >= tile.m_end) {  // none of the warp's rows exists
        tc_fence_before();
        mbar_arrive_remote_relaxed(empty_addr);
      } else if (far) {  // 128 bytes of the rows at a time; the factor worked out again takes no register till here
        const FarUnit scale(unit_a * (static_cast<double>(a.w_amax[tile.expert * a.w_amax_stride]) / 2688.0));
        const int per_vec = a.out_bf16 ? 8 : 4;
#pragma unroll 1
        for (int c = 0; c < cols; c += 8 * per_vec) {
          uint32_t q[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[16];
            if (a.out_bf16) {
              tmem_ld16(taddr + c + 32 * h, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int i = 0; i < 8; ++i) q[16 * h + i] = Bf16::pack(make_float2(scale(r[2 * i]), scale(r[2 * i + 1])));
              tmem_ld16(taddr + c + 32 * h + 16, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int i = 0; i < 8; ++i) q[16 * h + 8 + i] = Bf16::pack(make_float2(scale(r[2 * i]), scale(r[2 * i + 1])));
            } else {
              tmem_ld16(taddr + c + 16 * h, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int i = 0; i < 16; ++i) q[16 * h + i] = __float_as_uint(scale(r[i]));
            }
          }
          put_piece(piece, a, tile, row0, q, c, cols, per_vec);
        }
        tc_fence_before();
        mbar_arrive_remote_relaxed(empty_addr);
      } else if (a.out_bf16) {
        uint32_t q[BN / 2];
#pragma unroll
        for (int c = 0; c < BN; c += 16) {
          uint32_t r[16];
          tmem_ld16(taddr + c, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            q[c / 2 + i] = Bf16::pack(make_float2(__uint_as_float(r[2 * i]) * unit, __uint_as_float(r[2 * i + 1]) * unit));
        }
        tc_fence_before();
        mbar_arrive_remote_relaxed(empty_addr);
#pragma unroll
        for (int c = 0; c < BN; c += 64) put_piece(piece, a, tile, row0, &q[c / 2], c, cols, 8);
      } else {
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {  // uniform over the warp
          uint32_t r0[16], r1[16], q[32];
          tmem_ld16(taddr + c, r0);
          tmem_ld16(taddr + c + 16, r1);
          tmem_ld_wait(r0, r1);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            q[i] = __float_as_uint(__uint_as_float(r0[i]) * unit);
            q[16 + i] = __float_as_uint(__uint_as_float(r1[i]) * unit);
          }
          put_piece(piece, a, tile, row0, q, c, cols, 4);
        }
        tc_fence_before();
        mbar_arrive_remote_relaxed(empty_addr);
      }
      if (++b == P::kAccs) {
        b = 0;
        acc_phase ^= 1u;
      }
    }
  } else if (warp < 2 + kEpiWarps + kScaleWarps) {
    // ---- block scales (both CTAs): this CTA's rows of A, every column's of B ----
    const int quarter = warp & 3;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + P::kScaleBase;
    int stage = 0, group = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = cl; ok && t < total; t += ncl) {
      for (int kg = 0; ok && kg < k_blocks; kg += 4, ++group) {
        const int b = group & 1;
        if (!wait_or_abort(&sf_full[b], (group >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        for (int u = 0; u < 4 && kg + u < k_blocks; ++u) {
          if (!wait_or_abort(&empty[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // stage u's 16 bytes of row l: chunk u of the row's 64, swizzled by (row / 2) % 4
          const unsigned char* st = scales + b * P::kGroupBytes + lane * 64 + ((u ^ ((lane >> 1) & 3)) * 16);
          const uint32_t col = lanes + static_cast<uint32_t>(stage * P::kScaleCols);
          constexpr int kRowGroups = 4 + P::kGroups;
          uint4 q[kRowGroups];
#pragma unroll
          for (int c = 0; c < kRowGroups; ++c) q[c] = lds16(st + c * 2048);
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = word(q[i & 3], i >> 2);  // A: step i / 4, row group i % 4
          tmem_st16(col, r);
#pragma unroll
          for (int h = 0; h < P::kGroups / 4; ++h) {  // B: steps and groups in order
#pragma unroll
            for (int i = 0; i < 16; ++i)
              r[i] = word(q[4 + (16 * h + i) % P::kGroups], (16 * h + i) / P::kGroups);
            tmem_st16(col + 16 + 16 * h, r);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(peer_addr(&full[stage], 0));
          if (++stage == P::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&sf_empty[b]);  // the warp has read the group
      }
    }
  } else if (own_scales) {
    // ---- copies of the block scales whose rows TMA cannot read ----
    int group = 0;
    bool ok = true;
    for (int t = cl; ok && t < total; t += ncl) {
      const Tile tile = decode_tile<kBM>(t, first_tile, lo, hi, a.experts, n_tiles, BN);
      const int64_t arow = tile.m0 + 128 * rank, wrow = static_cast<int64_t>(tile.expert) * a.n + tile.n0;
      const int64_t aleft = tile.m_end - arow, wleft = a.n - tile.n0;
      const uint8_t* as = a.a_scale + (aleft > 0 ? arow : 0) * a.a_scale_pitch;
      const uint8_t* ws = a.w_scale + wrow * a.w_scale_pitch;
      for (int kg = 0; kg < k_blocks; kg += 4, ++group) {
        const int b = group & 1;
        if (!wait_or_abort(&sf_empty[b], ((group >> 1) & 1) ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        unsigned char* sc = scales + b * P::kGroupBytes;
        if (a.scale_bytes == 8) {
          copy_scales<8>(sc, as, a.a_scale_pitch, aleft, 128, kg * 16, a.k / 16);
          copy_scales<8>(sc + 128 * 64, ws, a.w_scale_pitch, wleft, BN, kg * 16, a.k / 16);
        } else {
          copy_scales<4>(sc, as, a.a_scale_pitch, aleft, 128, kg * 16, a.k / 16);
          copy_scales<4>(sc + 128 * 64, ws, a.w_scale_pitch, wleft, BN, kg * 16, a.k / 16);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sf_full[b])) : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // the CTA leaves with no copy in flight
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair's products or copies may touch its memory
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
}

// ---- host ---------------------------------------------------------------------

// 2-D byte tensor map of a matrix [rows, >= inner bytes] in boxes of `box_bytes`
// x `box_rows`, swizzled over the box's width (128: codes, 64: block scales).
situ_status_t byte_map(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t pitch, int box_bytes,
                       int box_rows) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return fail(SITU_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SITU_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return SITU_OK;
}

// Clusters of a kernel that the device holds at once, asked of the runtime once
// per device, kernel and shared-memory size.
situ_status_t max_clusters(const void* kernel, cudaLaunchConfig_t* cfg, int* clusters) {
  struct Entry {
    int dev;
    const void* kernel;
    size_t smem;
    int clusters;
  };
  static std::mutex mu;
  static Entry seen[64];
  static int n_seen = 0;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(err));
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_seen; ++i)
    if (seen[i].dev == dev && seen[i].kernel == kernel && seen[i].smem == cfg->dynamicSmemBytes) {
      *clusters = seen[i].clusters;
      return SITU_OK;
    }
  err = cudaOccupancyMaxActiveClusters(clusters, kernel, cfg);
  if (err != cudaSuccess || *clusters < 1) {
    (void)cudaGetLastError();  // the query's error is not sticky
    return fail(SITU_ERR_CUDA, "the device has no room for a cluster of two CTAs: %s", cudaGetErrorString(err));
  }
  if (n_seen < 64) seen[n_seen++] = {dev, kernel, cfg->dynamicSmemBytes, *clusters};
  return SITU_OK;
}

template <int BN>
situ_status_t launch(const void* a_data, int64_t a_pitch, const void* w_data, int64_t w_pitch, const Args& a,
                     cudaStream_t s) {
  using P = Shape<BN>;
  const void* kernel = reinterpret_cast<const void*>(situ_nvfp4_gemm_kernel<BN>);
  const int smem = 1024 + P::kSmem + kHeader + a.experts * 20 + 8;
  situ_status_t st = ensure_smem(kernel, smem);
  if (st != SITU_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  st = max_clusters(kernel, &cfg, &clusters);
  if (st != SITU_OK) return st;
  const int cap = g_max_ctas.load(std::memory_order_relaxed);
  if (cap > 0 && 2 * clusters > cap) clusters = cap < 2 ? 1 : cap / 2;
  // no more clusters than tiles there can be: every expert may end in a part of one
  const int64_t most = ((a.tokens + kBM - 1) / kBM + a.experts - 1) * ((a.n + BN - 1) / BN);
  if (clusters > most) clusters = static_cast<int>(most);
  const int64_t w_rows = static_cast<int64_t>(a.experts) * a.n;
  CUtensorMap ma, mw, mas = {}, mws = {};
  st = byte_map(&ma, a_data, a.k / 2, a.tokens, a_pitch, kStageRow, 128);
  if (st != SITU_OK) return st;
  st = byte_map(&mw, w_data, a.k / 2, w_rows, w_pitch, kStageRow, BN / 2);
  if (st != SITU_OK) return st;
  if (a.scale_bytes == 16) {
    st = byte_map(&mas, a.a_scale, a.k / 16, a.tokens, a.a_scale_pitch, 64, 128);
    if (st != SITU_OK) return st;
    st = byte_map(&mws, a.w_scale, a.k / 16, w_rows, a.w_scale_pitch, 64, BN);
    if (st != SITU_OK) return st;
  }
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, situ_nvfp4_gemm_kernel<BN>, ma, mw, mas, mws, a);
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "situ_glu_nvfp4_gemm launch: %s", cudaGetErrorString(err));
  return check_launch("situ_glu_nvfp4_gemm");
}

}  // namespace nvgemm

// Checks of a stored matrix' codes and scales (row pitches in bytes).
situ_status_t check_codes(const void* data, int64_t data_pitch, const void* scale, int64_t scale_pitch, int64_t rows,
                          int64_t cols, int data_align, int scale_align, const char* name) {
  if (data == nullptr || scale == nullptr) return fail(SITU_ERR_INVALID_ARG, "%s codes or scales are NULL", name);
  if (!span_fits(rows, data_pitch, cols / 2, 1) || !span_fits(rows, scale_pitch, cols / 16, 1))
    return fail(SITU_ERR_INVALID_ARG, "extent of %s overflows int64", name);
  if (!aligned(data, data_align) || data_pitch % data_align != 0 || !aligned(scale, scale_align) ||
      scale_pitch % scale_align != 0)
    return fail(SITU_ERR_MISALIGNED, "%s codes (%d bytes) or scales (%d) base or row pitch misaligned", name, data_align,
                scale_align);
  return SITU_OK;
}

Span bytes_span(const void* p, size_t n) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + n};
}

// Size checks shared by quantise and dequantise.
situ_status_t store_check(situ_dtype_t dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (!valid_dtype(dtype)) return fail(SITU_ERR_INVALID_ARG, "dtype %d is not a situ_dtype_t", (int)dtype);
  if (rows < 0) return fail(SITU_ERR_INVALID_ARG, "rows = %lld < 0", (long long)rows);
  if (cols <= 0 || cols % 16 != 0)
    return fail(SITU_ERR_INVALID_ARG, "cols must be a positive multiple of 16, got %lld", (long long)cols);
  if (cols > (int64_t(1) << 31)) return fail(SITU_ERR_UNSUPPORTED, "cols = %lld exceeds 2^31", (long long)cols);
  if (stride < cols) return fail(SITU_ERR_INVALID_ARG, "a row stride is shorter than its row");
  return SITU_OK;
}

void fill_store(StoreArgs* a, int64_t rows, int64_t cols, bool flat) {
  a->rows = rows;
  a->per_row = static_cast<uint32_t>(cols / 16);
  a->blocks = rows * (cols / 16);
  a->flat = flat;
}

// Whether every vector pair of a matrix is 32-byte aligned.
int wide_rows(const void* p, int64_t pitch) { return aligned(p, 32) && pitch % 32 == 0; }

}  // namespace

int nvfp4_device_status(int clear) { return unit_device_status(clear); }

extern "C" {

situ_status_t situ_glu_nvfp4_quantize(const void* x, situ_dtype_t dtype, int64_t rows, int64_t cols,
                                      int64_t x_row_stride, void* data, int64_t data_row_stride, void* scale,
                                      int64_t scale_row_stride, float* amax, int amax_given, void* stream) {
  tl_last_error[0] = '\0';
  situ_status_t st = store_check(dtype, rows, cols, x_row_stride);
  if (st != SITU_OK) return st;
  if (amax_given < 0 || amax_given > 2) return fail(SITU_ERR_INVALID_ARG, "amax_given must be 0, 1 or 2");
  const bool only = amax_given == 2;
  if (!only && (data_row_stride < cols / 2 || scale_row_stride < cols / 16))
    return fail(SITU_ERR_INVALID_ARG, "NVFP4 data or scale row pitch shorter than a row");
  if (amax == nullptr) return fail(SITU_ERR_INVALID_ARG, "amax is NULL");
  if (!aligned(amax, 4)) return fail(SITU_ERR_MISALIGNED, "amax not 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int es = elem_size(dtype);
  if (rows > 0) {
    if (x == nullptr) return fail(SITU_ERR_INVALID_ARG, "x is NULL");
    if (!span_fits(rows, x_row_stride, cols, es)) return fail(SITU_ERR_INVALID_ARG, "extent of x overflows int64");
    if (!aligned(x, 16) || (x_row_stride * es) % 16 != 0)
      return fail(SITU_ERR_MISALIGNED, "x base or row pitch not 16-byte aligned");
    if (!only) {
      st = check_codes(data, data_row_stride, scale, scale_row_stride, rows, cols, 8, 1, "NVFP4");
      if (st != SITU_OK) return st;
    }
    const Span in = matrix_span(x, rows, x_row_stride, cols, es);
    const Span outs[] = {bytes_span(amax, 4), only ? Span{0, 0} : matrix_span(data, rows, data_row_stride, cols / 2, 1),
                         only ? Span{0, 0} : matrix_span(scale, rows, scale_row_stride, cols / 16, 1)};
    for (int i = 0; i < 3; ++i) {
      if (overlap(outs[i], in)) return fail(SITU_ERR_INVALID_ARG, "an output overlaps x");
      for (int k = i + 1; k < 3; ++k)
        if (overlap(outs[i], outs[k])) return fail(SITU_ERR_INVALID_ARG, "outputs overlap each other");
    }
  }
  const bool bf = dtype == SITU_DTYPE_BF16;
  const bool small = amax_given == 0 && rows > 0 && rows <= kSmallBlocks / (cols / 16);
  if (amax_given != 1 && !small) {
    cudaError_t err = cudaMemsetAsync(amax, 0, sizeof(float), s);
    if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(err));
  }
  if (rows == 0) return SITU_OK;
  StoreArgs a{};
  a.x = static_cast<const char*>(x);
  a.x_pitch = x_row_stride * es;
  a.data = static_cast<char*>(data);
  a.data_pitch = data_row_stride;
  a.scale = static_cast<uint8_t*>(scale);
  a.scale_pitch = scale_row_stride;
  a.amax = amax;
  a.amax_out = reinterpret_cast<unsigned int*>(amax);
  a.wide = wide_rows(x, a.x_pitch);
  fill_store(&a, rows, cols,
             rows == 1 || (x_row_stride == cols &&
                           (only || (data_row_stride == cols / 2 && scale_row_stride == cols / 16))));
  if (small) {
    auto k = bf ? situ_nvfp4_small_kernel<Bf16> : situ_nvfp4_small_kernel<F32>;
    k<<<kSmallCtas, kSmallThreads, 0, s>>>(a);
    return check_launch("situ_glu_nvfp4_quantize (one launch)");
  }
  const int64_t ctas = (a.blocks + kStoreThreads - 1) / kStoreThreads;
  int grid = 0;
  if (amax_given != 1) {
    auto k = bf ? situ_nvfp4_amax_kernel<Bf16> : situ_nvfp4_amax_kernel<F32>;
    st = launch_grid(reinterpret_cast<const void*>(k), kStoreThreads, 0, ctas, &grid);
    if (st != SITU_OK) return st;
    k<<<grid, kStoreThreads, 0, s>>>(a);
    st = check_launch("situ_glu_nvfp4_quantize (amax)");
    if (st != SITU_OK || only) return st;
  }
  auto k = bf ? (amax_given != 0 ? situ_nvfp4_quantize_kernel<Bf16, true> : situ_nvfp4_quantize_kernel<Bf16, false>)
              : situ_nvfp4_quantize_kernel<F32, false>;  // whose codes saturate whatever A is
  st = launch_grid(reinterpret_cast<const void*>(k), kStoreThreads, 0, ctas, &grid);
  if (st != SITU_OK) return st;
  k<<<grid, kStoreThreads, 0, s>>>(a);
  return check_launch("situ_glu_nvfp4_quantize");
}

situ_status_t situ_glu_nvfp4_dequantize(const void* data, int64_t data_row_stride, const void* scale,
                                        int64_t scale_row_stride, const float* amax, int64_t rows, int64_t cols,
                                        void* out, situ_dtype_t dtype, int64_t out_row_stride, void* stream) {
  tl_last_error[0] = '\0';
  situ_status_t st = store_check(dtype, rows, cols, out_row_stride);
  if (st != SITU_OK) return st;
  if (data_row_stride < cols / 2 || scale_row_stride < cols / 16)
    return fail(SITU_ERR_INVALID_ARG, "NVFP4 data or scale row pitch shorter than a row");
  if (rows == 0) return SITU_OK;
  if (amax == nullptr || out == nullptr) return fail(SITU_ERR_INVALID_ARG, "amax or out is NULL");
  if (!aligned(amax, 4)) return fail(SITU_ERR_MISALIGNED, "amax not 4-byte aligned");
  const int es = elem_size(dtype);
  st = check_codes(data, data_row_stride, scale, scale_row_stride, rows, cols, 8, 1, "NVFP4");
  if (st != SITU_OK) return st;
  if (!span_fits(rows, out_row_stride, cols, es)) return fail(SITU_ERR_INVALID_ARG, "extent of out overflows int64");
  if (!aligned(out, 16) || (out_row_stride * es) % 16 != 0)
    return fail(SITU_ERR_MISALIGNED, "out base or row pitch not 16-byte aligned");
  const Span o = matrix_span(out, rows, out_row_stride, cols, es);
  if (overlap(o, matrix_span(data, rows, data_row_stride, cols / 2, 1)) ||
      overlap(o, matrix_span(scale, rows, scale_row_stride, cols / 16, 1)) || overlap(o, bytes_span(amax, 4)))
    return fail(SITU_ERR_INVALID_ARG, "out overlaps an input");
  StoreArgs a{};
  a.data = const_cast<char*>(static_cast<const char*>(data));
  a.data_pitch = data_row_stride;
  a.scale = const_cast<uint8_t*>(static_cast<const uint8_t*>(scale));
  a.scale_pitch = scale_row_stride;
  a.amax = amax;
  a.out = static_cast<char*>(out);
  a.out_pitch = out_row_stride * es;
  a.wide = wide_rows(out, a.out_pitch);
  fill_store(&a, rows, cols,
             rows == 1 || (out_row_stride == cols && data_row_stride == cols / 2 && scale_row_stride == cols / 16));
  auto k = dtype == SITU_DTYPE_BF16 ? situ_nvfp4_dequantize_kernel<Bf16> : situ_nvfp4_dequantize_kernel<F32>;
  // Two blocks a thread, as many CTAs as that takes: their turnover overlaps one's
  // stores with the next one's loads (bf16 57344 x 2048: 45 us, a loop of resident CTAs
  // 50 us).
  const int64_t ctas = (a.blocks + 2 * kStoreThreads - 1) / (2 * kStoreThreads);
  int grid = 0;
  if (g_max_ctas.load(std::memory_order_relaxed) <= 0 && ctas <= INT32_MAX) {
    grid = static_cast<int>(ctas);
  } else {
    st = launch_grid(reinterpret_cast<const void*>(k), kStoreThreads, 0, ctas, &grid);
    if (st != SITU_OK) return st;
  }
  k<<<grid, kStoreThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return check_launch("situ_glu_nvfp4_dequantize");
}

situ_status_t situ_glu_nvfp4_gemm(const void* a_data, int64_t a_data_row_stride, const void* a_scale,
                                  int64_t a_scale_row_stride, const float* a_amax, int64_t tokens, int64_t k,
                                  const void* w_data, int64_t w_data_row_stride, const void* w_scale,
                                  int64_t w_scale_row_stride, const float* w_amax, int64_t w_amax_stride,
                                  int64_t experts, int64_t n, const int64_t* offsets, void* out,
                                  situ_dtype_t out_dtype, int64_t out_row_stride, void* stream) {
  tl_last_error[0] = '\0';
  if (!valid_dtype(out_dtype)) return fail(SITU_ERR_INVALID_ARG, "out_dtype %d is not a situ_dtype_t", (int)out_dtype);
  if (tokens < 0) return fail(SITU_ERR_INVALID_ARG, "tokens = %lld < 0", (long long)tokens);
  if (k < 64 || k % 64 != 0)
    return fail(SITU_ERR_UNSUPPORTED, "k must be a positive multiple of 64, got %lld", (long long)k);
  if (n < 8 || n % 8 != 0)
    return fail(SITU_ERR_UNSUPPORTED, "n must be a positive multiple of 8, got %lld", (long long)n);
  if (experts < 1 || experts > nvgemm::kMaxExperts)
    return fail(SITU_ERR_UNSUPPORTED, "experts must be in [1, %d], got %lld", nvgemm::kMaxExperts, (long long)experts);
  if (tokens > INT32_MAX - 256 || n > INT32_MAX / experts - 256 || k > INT32_MAX - 256)
    return fail(SITU_ERR_UNSUPPORTED, "sizes exceed the 32-bit tensor-map coordinates");
  // tiles are numbered in 32 bits (the narrowest have 128 columns)
  if ((tokens / nvgemm::kBM + experts + 1) > INT32_MAX / (n / 128 + 1))
    return fail(SITU_ERR_UNSUPPORTED, "too many output tiles");
  if (offsets == nullptr && experts != 1) return fail(SITU_ERR_INVALID_ARG, "offsets is NULL with %lld experts", (long long)experts);
  if (a_data_row_stride < k / 2 || a_scale_row_stride < k / 16 || w_data_row_stride < k / 2 ||
      w_scale_row_stride < k / 16 || out_row_stride < n)
    return fail(SITU_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (w_amax_stride < 0) return fail(SITU_ERR_INVALID_ARG, "w_amax_stride < 0");
  if (tokens == 0) return SITU_OK;
  if (a_amax == nullptr || w_amax == nullptr || out == nullptr)
    return fail(SITU_ERR_INVALID_ARG, "a_amax, w_amax or out is NULL");
  if (!aligned(a_amax, 4) || !aligned(w_amax, 4) || (offsets != nullptr && !aligned(offsets, 8)))
    return fail(SITU_ERR_MISALIGNED, "a_amax, w_amax (4 bytes) or offsets (8) misaligned");
  situ_status_t st = check_codes(a_data, a_data_row_stride, a_scale, a_scale_row_stride, tokens, k, 16, 4, "a");
  if (st != SITU_OK) return st;
  st = check_codes(w_data, w_data_row_stride, w_scale, w_scale_row_stride, experts * n, k, 16, 4, "w");
  if (st != SITU_OK) return st;
  const int oes = elem_size(out_dtype);
  if (!span_fits(tokens, out_row_stride, n, oes) || !span_fits(experts, w_amax_stride, 1, 4))
    return fail(SITU_ERR_INVALID_ARG, "tensor extent overflows int64");
  if (!aligned(out, 16) || (out_row_stride * oes) % 16 != 0)
    return fail(SITU_ERR_MISALIGNED, "out base or row pitch not 16-byte aligned");
  const Span o = matrix_span(out, tokens, out_row_stride, n, oes);
  if (overlap(o, matrix_span(a_data, tokens, a_data_row_stride, k / 2, 1)) ||
      overlap(o, matrix_span(a_scale, tokens, a_scale_row_stride, k / 16, 1)) ||
      overlap(o, matrix_span(w_data, experts * n, w_data_row_stride, k / 2, 1)) ||
      overlap(o, matrix_span(w_scale, experts * n, w_scale_row_stride, k / 16, 1)) ||
      overlap(o, bytes_span(a_amax, 4)) || overlap(o, matrix_span(w_amax, experts, w_amax_stride, 1, 4)) ||
      (offsets != nullptr && overlap(o, bytes_span(offsets, static_cast<size_t>(experts + 1) * 8))))
    return fail(SITU_ERR_INVALID_ARG, "out overlaps an input");

  nvgemm::Args a{};
  a.a_scale = static_cast<const uint8_t*>(a_scale);
  a.a_scale_pitch = a_scale_row_stride;
  a.w_scale = static_cast<const uint8_t*>(w_scale);
  a.w_scale_pitch = w_scale_row_stride;
  a.a_amax = a_amax;
  a.w_amax = w_amax;
  a.w_amax_stride = w_amax_stride;
  a.offsets = offsets;
  a.experts = static_cast<int>(experts);
  a.tokens = tokens;
  a.k = static_cast<int>(k);
  a.n = static_cast<int>(n);
  a.scale_bytes = 4;
  for (int b = 8; b <= 16; b *= 2)
    if (aligned(a_scale, b) && aligned(w_scale, b) && a_scale_row_stride % b == 0 && w_scale_row_stride % b == 0)
      a.scale_bytes = b;
  a.out = static_cast<char*>(out);
  a.out_pitch = out_row_stride * oes;
  a.out_bf16 = out_dtype == SITU_DTYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  st = device_sm_count(&sms);
  if (st != SITU_OK) return st;
  // Tiles of 128 columns where every pair of SMs gets one of them at most (us, 128 and
  // 256 columns: 512 x 4096 x 4096 11.7, 13.4; 8 x 7168 x 2048 14.0, 16.1); from there
  // on the wider ones, with fewer operand bytes for the same products (2048 x 7168 x
  // 2048, 128 narrow tiles: 25.4, 18.3; 1024 x 2048 x 8192: 18.2, 15.1).
  const int64_t wide = ((tokens + nvgemm::kBM - 1) / nvgemm::kBM + experts - 1) * ((n + 255) / 256);
  if (4 * wide <= sms) return nvgemm::launch<128>(a_data, a_data_row_stride, w_data, w_data_row_stride, a, s);
  return nvgemm::launch<256>(a_data, a_data_row_stride, w_data, w_data_row_stride, a, s);
}

}  // extern "C"
