// situ_norm.cu -- residual addition + RMS norm in front of the experts
// (include/situ_glu.h, situ_glu_rms_norm_*): forward with native or MXFP8 rows,
// and the backward.
//
//   h = x + residual (rounded to the storage type),  q = 1 / sqrt(mean h^2 + eps)
//   y = h q w
//   d_x = grad_h + q g - h q^3 mean(g h),  g = grad_y w;   d_w = sum_t grad_y h q
//
// Every element is read and written once (8 bytes an element in bf16 either
// way, a dozen operations), so the bound is HBM bandwidth.  A row lives in the
// registers of its threads between its sum and its output: V 16-byte vectors
// per thread, thread t holding vectors t, t + n, ... of the row.

#include <initializer_list>
#include <type_traits>

#include "situ_host.cuh"

namespace {

constexpr int64_t kNormMaxRowBytes = 65536;  // eight vectors in each of 512 threads
// The most threads of a CTA with V vectors a thread (row_shape below).
template <int V, bool MX = false>
constexpr int kNormThreads = V == 8 || (MX && V == 2) ? 512 : 256;

struct NormArgs {
  const char* x;
  int64_t x_pitch;    // bytes, as every pitch here
  const char* res;    // NULL: none
  int64_t res_pitch;
  const void* w;
  int w_bf16;
  char* h;
  int64_t h_pitch;
  char* y;
  int64_t y_pitch;
  int64_t tokens;
  int vpr;            // 16-byte vectors of a row
  float eps, inv_hidden;
};

// The weights of vector j of a row as fp32 pairs.
template <typename S>
__device__ __forceinline__ void norm_weights(const void* w, int bf16, int j, float2 (&c)[S::kPairs]) {
  if (bf16) {
    const uint32_t* p = static_cast<const uint32_t*>(w) + static_cast<int64_t>(j) * S::kPairs;
    uint32_t q[S::kPairs];
    if constexpr (S::kPairs == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      q[0] = v.x, q[1] = v.y;
    }
#pragma unroll
    for (int k = 0; k < S::kPairs; ++k) c[k] = bf16x2_to_f2(q[k]);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + static_cast<int64_t>(j) * 2 * S::kPairs);
#pragma unroll
    for (int k = 0; k < S::kPairs; k += 2) {
      const float4 v = __ldg(p + k / 2);
      c[k] = make_float2(v.x, v.y);
      c[k + 1] = make_float2(v.z, v.w);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the threads of a row, in an order that the row's width alone fixes;
// every thread gets it.  A row of one warp needs no barrier; otherwise the CTA
// is the row, and `slot` alternates between two buffers so that one barrier a
// call suffices.
__device__ __forceinline__ float row_sum(float v, float* slot, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? slot[lane] : 0.0f);
}
// `BARRIER` names the barrier of the row's threads (0: the whole CTA).
template <int BARRIER = 0>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* slot, int warps) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"n"(BARRIER), "r"(warps * 32) : "memory");
  const int lane = threadIdx.x & 31;
  const float2 p = lane < warps ? slot[lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(p.x), warp_sum(p.y));
}

// A row whose mean square (with epsilon) leaves [kMeanLow, kMeanHigh] has squares, or
// products with powers of 1 / rms, that fp32 does not hold or not to its precision.  Its
// threads, which see the same mean, sum it once more with every element times a power
// of two that brings them all into range: the squares of a small row to at most 2^114
// in all, of the largest fp32 numbers to 2^110 (16384 of them), and the smallest
// element to 2^-59.
constexpr float kMeanLow = 0x1p-80f, kMeanHigh = 0x1p80f;
__device__ __forceinline__ bool mean_in_range(float mean) { return mean >= kMeanLow && mean <= kMeanHigh; }
__device__ __forceinline__ float range_scale(float mean) { return mean < kMeanLow ? 0x1p90f : 0x1p-80f; }

// What the backward needs of a row, from sums = (sum h^2, sum g h):
//   q       1 / rms
//   along   d_x = q g + along h,        along = -q q (q mean(g h))      of ordinary rows
//           d_x = q g + along (h q),    along = -q (q mean(g h))        of rows out of range,
// whose q q fp32 may not hold.  `lift`: the sums' h is the row's times it.
struct RowScale {
  float q, along;
  bool far;  // the mean is out of range
};
template <bool ONE_FORM = false>  // the second form for every row
__device__ __forceinline__ RowScale row_scale(const float2& sums, float mean, float inv_hidden) {
  const float q = rsqrtf(mean), t = q * (sums.y * inv_hidden);
  return {q, ONE_FORM ? -q * t : -q * (q * t), !mean_in_range(mean)};
}
__device__ __forceinline__ RowScale far_row_scale(const float2& sums, float inv_hidden, float eps, float lift) {
  const float u = rsqrtf(sums.x * inv_hidden + eps * lift * lift), q = u * lift;
  return {q, -q * (u * (sums.y * inv_hidden)), true};
}
// A pair of d_x (without grad_h) and of the terms of d_weight.
template <bool FAR>
__device__ __forceinline__ float2 norm_grad(const RowScale& k, const float2& h, const float2& g, const float2& w, float2& dw) {
  if constexpr (FAR) {
    const float2 n = mul2(h, splat(k.q));
    dw = fma2(g, n, dw);
    return fma2(mul2(g, splat(k.q)), w, mul2(n, splat(k.along)));
  } else {
    const float2 gq = mul2(g, splat(k.q));
    dw = fma2(gq, h, dw);
    return fma2(gq, w, mul2(h, splat(k.along)));
  }
}

// h = x + r in the storage type.
template <typename S>
__device__ __forceinline__ uint4 add_vec(const uint4& x, const uint4& r) {
  uint4 h;
#pragma unroll
  for (int p = 0; p < S::kPairs; ++p) S::put(h, p, add2(as_f2(S::pair(x, p)), as_f2(S::pair(r, p))));
  return h;
}

template <typename S, int V, bool RES, bool MX>
__global__ void __launch_bounds__(kNormThreads<V, MX>) situ_rms_norm_fwd_kernel(const NormArgs a, const MxOut m) {
  __shared__ float slots[2][32];
  const int nt = blockDim.x, warps = nt >> 5;
  int flip = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.tokens;
       row += static_cast<int64_t>(gridDim.x) * blockDim.y) {
    uint4 h[V];
    float2 acc = make_float2(0.0f, 0.0f);
    const char* xr = a.x + row * a.x_pitch;
    const char* rr = RES ? a.res + row * a.res_pitch : nullptr;
    uint4 r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = threadIdx.x + i * nt;
      if (j < a.vpr) {
        h[i] = ld_stream(xr + static_cast<int64_t>(j) * kVecBytes);
        if (RES) r[i] = ld_stream(rr + static_cast<int64_t>(j) * kVecBytes);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = threadIdx.x + i * nt;
      if (j < a.vpr) {
        if (RES) {
          h[i] = add_vec<S>(h[i], r[i]);
          st_stream(a.h + row * a.h_pitch + static_cast<int64_t>(j) * kVecBytes, h[i]);
        }
#pragma unroll
        for (int p = 0; p < S::kPairs; ++p) {
          const float2 f = as_f2(S::pair(h[i], p));
          acc = fma2(f, f, acc);
        }
      }
    }
    const float mean = row_sum(acc.x + acc.y, slots[flip], warps) * a.inv_hidden + a.eps;
    flip ^= 1;
    float q = rsqrtf(mean);
    if (!mean_in_range(mean)) {
      const float s = range_scale(mean);
      acc = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (static_cast<int>(threadIdx.x) + i * nt < a.vpr) {
#pragma unroll
          for (int p = 0; p < S::kPairs; ++p) {
            const float2 f = mul2(as_f2(S::pair(h[i], p)), splat(s));
            acc = fma2(f, f, acc);
            if (s > 1.0f) S::put(h[i], p, f);  // exact; 1 / rms itself may leave fp32
          }
        }
      }
      q = rsqrtf(row_sum(acc.x + acc.y, slots[flip], warps) * a.inv_hidden + a.eps * s * s);
      flip ^= 1;
      if (s < 1.0f) q *= s;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = threadIdx.x + i * nt;
      const bool in = j < a.vpr;
      float2 y[S::kPairs];
      if (in) {
        float2 w[S::kPairs];
        norm_weights<S>(a.w, a.w_bf16, j, w);
#pragma unroll
        for (int p = 0; p < S::kPairs; ++p) y[p] = mul2(mul2(as_f2(S::pair(h[i], p)), splat(q)), w[p]);
      } else {
#pragma unroll
        for (int p = 0; p < S::kPairs; ++p) y[p] = make_float2(0.0f, 0.0f);
      }
      if constexpr (MX) {  // every lane takes part in the block maxima
        mx_store_vec<S>(y, in, m.data + row * m.data_pitch, m.scale + row * m.scale_pitch, MxSlot<S>(j), m.rule);
      } else if (in) {
        uint4 o;
#pragma unroll
        for (int p = 0; p < S::kPairs; ++p) S::put(o, p, y[p]);
        st_stream(a.y + row * a.y_pitch + static_cast<int64_t>(j) * kVecBytes, o);
      }
    }
  }
}

// ---- backward -----------------------------------------------------------------
// d_weight is a sum over rows.  Chunk c of `chunks` holds rows c, c + chunks,
// ...; the CTA that has a chunk adds its rows' terms in registers (each thread
// has its own columns) and writes one fp32 row of partial sums; a second kernel
// adds the chunks in order.  Both orders depend on the shape alone.

// Chunks by the row's width: enough for the CTAs (or, in narrow rows, the warps)
// that share an SM, few enough that the partial rows stay a few per cent of the
// traffic (bf16 3000 x 16384: 136 us with 148 chunks, 141 with twice as many; 2000 x 7168: 25, 27).
constexpr int kNormMaxChunks = 2368;
int64_t norm_chunks(int64_t tokens, int64_t hidden) {
  const int64_t most = hidden <= 1024 ? kNormMaxChunks : hidden <= 4096 ? 592 : 148;
  return tokens < most ? tokens : most;
}

struct NormBwdArgs {
  const char* gy;
  int64_t gy_pitch;
  const char* gh;     // NULL: zero
  int64_t gh_pitch;
  const char* h;
  int64_t h_pitch;
  const void* w;
  int w_bf16;
  char* dx;
  int64_t dx_pitch;
  float* partials;    // [chunks][hidden], NULL: d_weight not wanted
  int64_t tokens;
  int64_t chunks;
  int vpr;
  float eps, inv_hidden;
};

// The sums of a row of which this thread has the vectors h and g, with h times s.
template <typename S, int V>
__device__ __forceinline__ float2 far_sums(const NormBwdArgs& a, int nt, const uint4 (&h)[V], const uint4 (&g)[V], float s) {
  float2 ss = make_float2(0.0f, 0.0f), gd = ss;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = threadIdx.x + i * nt;
    if (j < a.vpr) {
      float2 w[S::kPairs];
      norm_weights<S>(a.w, a.w_bf16, j, w);
#pragma unroll
      for (int p = 0; p < S::kPairs; ++p) {
        const float2 f = mul2(as_f2(S::pair(h[i], p)), splat(s));
        ss = fma2(f, f, ss);
        gd = fma2(mul2(as_f2(S::pair(g[i], p)), w[p]), f, gd);
      }
    }
  }
  return make_float2(ss.x + ss.y, gd.x + gd.y);
}

template <typename S, int V>
__global__ void __launch_bounds__(kNormThreads<V>) situ_rms_norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float2 slots[2][32];
  const int nt = blockDim.x, warps = nt >> 5;
  int flip = 0;
  // The thread's own columns' sums: registers, or (rows of eight vectors a
  // thread, whose sums would spill) the thread's words of shared memory.
  constexpr bool kInSmem = V == 8;
  // grad_h is loaded with the row (bf16 65536 x 1024: 92 us; loaded after the sums,
  // 133 us), but for eight vectors, which would spill.
  constexpr bool kEarly = V < 8;
  extern __shared__ float2 dw_smem[];
  float2 dw_reg[kInSmem ? 1 : V][S::kPairs];
  auto dw = [&](int i, int p) -> float2& {
    if constexpr (kInSmem) return dw_smem[(i * S::kPairs + p) * nt + threadIdx.x];
    else return dw_reg[i][p];
  };
  // The next row's vectors are loaded while this one is summed, up to two vectors a
  // thread (bf16 60000 x 256: 27 us, without 34; 40000 x 512: 29, 35); three or four
  // take the registers of other warps (40000 x 768: 52, without 47; 65536 x 1024: 101, 92).
  constexpr bool kAhead = V <= 2;
  auto load = [&](int64_t row, auto& h, auto& g, auto& gh) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = threadIdx.x + i * nt;
      if (j < a.vpr) {
        if (kEarly && a.gh != nullptr)
          gh[kEarly ? i : 0] = ld_stream(a.gh + row * a.gh_pitch + static_cast<int64_t>(j) * kVecBytes);
        h[i] = ld_stream(a.h + row * a.h_pitch + static_cast<int64_t>(j) * kVecBytes);
        g[i] = ld_stream(a.gy + row * a.gy_pitch + static_cast<int64_t>(j) * kVecBytes);
      }
    }
  };
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; c < a.chunks;
       c += static_cast<int64_t>(gridDim.x) * blockDim.y) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int p = 0; p < S::kPairs; ++p) dw(i, p) = make_float2(0.0f, 0.0f);
    uint4 next_h[kAhead ? V : 1], next_g[kAhead ? V : 1], next_gh[kAhead ? V : 1];
    if constexpr (kAhead) load(c, next_h, next_g, next_gh);
    for (int64_t row = c; row < a.tokens; row += a.chunks) {
      uint4 h[V], g[V], gh[kEarly ? V : 1];
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = next_h[i], g[i] = next_g[i], gh[i] = next_gh[i];
        if (row + a.chunks < a.tokens) load(row + a.chunks, next_h, next_g, next_gh);
      } else {
        load(row, h, g, gh);
      }
      float2 ss = make_float2(0.0f, 0.0f), gd = ss;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * nt;
        if (j < a.vpr) {
          float2 w[S::kPairs];
          norm_weights<S>(a.w, a.w_bf16, j, w);
#pragma unroll
          for (int p = 0; p < S::kPairs; ++p) {
            const float2 f = as_f2(S::pair(h[i], p));
            ss = fma2(f, f, ss);
            gd = fma2(mul2(as_f2(S::pair(g[i], p)), w[p]), f, gd);
          }
        }
      }
      const float2 sums = row_sum2(make_float2(ss.x + ss.y, gd.x + gd.y), slots[flip], warps);
      flip ^= 1;
      const float mean = sums.x * a.inv_hidden + a.eps;
      RowScale k = row_scale(sums, mean, a.inv_hidden);
      if (k.far) {
        const float lift = range_scale(mean);
        k = far_row_scale(row_sum2(far_sums<S>(a, nt, h, g, lift), slots[flip], warps), a.inv_hidden, a.eps, lift);
        flip ^= 1;
      }
      auto finish = [&](auto far) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int j = threadIdx.x + i * nt;
          if (j < a.vpr) {
            uint4 o;
            if (!kEarly && a.gh != nullptr) gh[0] = ld_stream(a.gh + row * a.gh_pitch + static_cast<int64_t>(j) * kVecBytes);
            const uint4& ghi = gh[kEarly ? i : 0];
            float2 w[S::kPairs];
            norm_weights<S>(a.w, a.w_bf16, j, w);
#pragma unroll
            for (int p = 0; p < S::kPairs; ++p) {
              float2 d = norm_grad<far.value>(k, as_f2(S::pair(h[i], p)), as_f2(S::pair(g[i], p)), w[p], dw(i, p));
              if (a.gh != nullptr) d = add2(d, as_f2(S::pair(ghi, p)));
              S::put(o, p, d);
            }
            st_stream(a.dx + row * a.dx_pitch + static_cast<int64_t>(j) * kVecBytes, o);
          }
        }
      };
      if (k.far) finish(std::true_type{});
      else finish(std::false_type{});
    }
    if (a.partials != nullptr) {
      float* out = a.partials + c * (static_cast<int64_t>(a.vpr) * 2 * S::kPairs);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * nt;
        if (j < a.vpr) {
          float4* p = reinterpret_cast<float4*>(out + static_cast<int64_t>(j) * 2 * S::kPairs);
#pragma unroll
          for (int k = 0; k < S::kPairs; k += 2)
            p[k / 2] = make_float4(dw(i, k).x, dw(i, k).y, dw(i, k + 1).x, dw(i, k + 1).y);
        }
      }
    }
  }
}

// The same with the rows staged by bulk copies: warp `warps` of the CTA keeps a
// ring of whole rows (h, grad_y, grad_h) filled, so the next rows' bytes are in
// flight while this one is summed; without it a CTA's loads wait for its sums
// (bf16 16384 x 7168: 286 us; staged 150 us, 6.3 TB/s).  V vectors a
// thread, the thread's weights and its columns' sums in registers; with four (rows of
// more than 1024 vectors) the sums leave no room, some of them spill, and the weights,
// which are larger than the L1 that the ring leaves, come from L2 twice a row: 3000 x
// 16384 takes 136 us, more than twice what HBM needs.
struct NormRing {
  int stages;
  int stage_bytes;
};

// The registers of the narrow rows' four CTAs an SM are asked for where the compiler
// would take more (bf16 32768 x 2048 with three: 108 us, four 98 us); two of 544
// threads have as many as four of 288.
template <int V>
constexpr int kRingThreads = V == 1 ? 288 : 544;
template <typename S, int V, bool GH>
constexpr int kRingCtas = V == 1 ? 4 : V == 2 && S::kPairs == 2 && !GH ? 2 : 0;
template <typename S, int V, bool GH>
__global__ void __launch_bounds__(kRingThreads<V>, kRingCtas<S, V, GH>) situ_rms_norm_bwd_ring_kernel(const NormBwdArgs a, const NormRing r) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float2 slots[2][32];
  __shared__ uint64_t full[8], empty[8];
  const int nt = blockDim.x - 32, warps = nt >> 5;
  const int row_bytes = a.vpr * kVecBytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < r.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], warps);
    }
    mbar_fence_init();
  }
  __syncthreads();
  int stage = 0;
  uint32_t phase = 0;
  if (static_cast<int>(threadIdx.x) >= nt) {
    // ---- copies: one lane ----
    if (threadIdx.x == static_cast<unsigned>(nt)) {
      uint32_t issued = 0;
      bool ok = true;
      for (int64_t c = blockIdx.x; ok && c < a.chunks; c += gridDim.x)
        for (int64_t row = c; row < a.tokens; row += a.chunks) {
          if (!mbar_wait(&empty[stage], phase ^ 1u)) {
            atomicExch(&g_device_status, kStatusWaitExpired);
            ok = false;
            break;
          }
          unsigned char* st = ring + stage * r.stage_bytes;
          mbar_arrive_expect_tx(&full[stage], (GH ? 3 : 2) * row_bytes);
          bulk_load(st, a.h + row * a.h_pitch, row_bytes, &full[stage]);
          bulk_load(st + row_bytes, a.gy + row * a.gy_pitch, row_bytes, &full[stage]);
          if (GH) bulk_load(st + 2 * row_bytes, a.gh + row * a.gh_pitch, row_bytes, &full[stage]);
          issued |= 1u << stage;
          if (++stage == r.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      // the CTA leaves with no copy in flight (a bounded wait, as all are)
      for (int s = 0; s < r.stages; ++s)
        if (issued & (1u << s)) mbar_wait(&full[s], s < stage ? phase : phase ^ 1u);
    }
    return;
  }
  // ---- sums and outputs ----
  // (four vectors a thread leave no registers for the weights: read twice a row)
  constexpr bool kKeep = V < 4;
  float2 kept[kKeep ? V : 1][S::kPairs], dw[V][S::kPairs];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = threadIdx.x + i * nt;
      if (j < a.vpr) norm_weights<S>(a.w, a.w_bf16, j, kept[i]);
    }
  }
  auto weights = [&](int i, float2 (&w)[S::kPairs]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int p = 0; p < S::kPairs; ++p) w[p] = kept[i][p];
    } else {
      norm_weights<S>(a.w, a.w_bf16, threadIdx.x + i * nt, w);
    }
  };
  // Rows of one vector a thread have the registers for both forms of the outputs (bf16
  // 32768 x 2048 without grad_h: 77 us, with the second form alone 79 us); wider ones
  // lose more to the other loop's (3000 x 16384 without: 100 us, with both 110 us).
  constexpr bool kOneForm = V > 1;
  int flip = 0;
  bool dead = false;  // a wait expired: the control flow goes on, without waits
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int p = 0; p < S::kPairs; ++p) dw[i][p] = make_float2(0.0f, 0.0f);
    for (int64_t row = c; row < a.tokens; row += a.chunks) {
      if (!dead && !mbar_wait(&full[stage], phase)) {
        atomicExch(&g_device_status, kStatusWaitExpired);
        dead = true;
      }
      const unsigned char* st = ring + stage * r.stage_bytes;
      uint4 h[V], g[V], gh[V];
      float2 ss = make_float2(0.0f, 0.0f), gd = ss;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * nt;
        if (j < a.vpr) {
          h[i] = lds16(st + j * kVecBytes);
          g[i] = lds16(st + row_bytes + j * kVecBytes);
          if (GH) gh[i] = lds16(st + 2 * row_bytes + j * kVecBytes);
        }
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[stage]);  // the warp has its vectors
      if (++stage == r.stages) {
        stage = 0;
        phase ^= 1u;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * nt;
        if (j < a.vpr) {
          float2 w[S::kPairs];
          weights(i, w);
#pragma unroll
          for (int p = 0; p < S::kPairs; ++p) {
            const float2 f = as_f2(S::pair(h[i], p));
            ss = fma2(f, f, ss);
            gd = fma2(mul2(as_f2(S::pair(g[i], p)), w[p]), f, gd);
          }
        }
      }
      const float2 sums = row_sum2<1>(make_float2(ss.x + ss.y, gd.x + gd.y), slots[flip], warps);
      flip ^= 1;
      const float mean = sums.x * a.inv_hidden + a.eps;
      RowScale k = row_scale<kOneForm>(sums, mean, a.inv_hidden);
      if (k.far) {
        const float lift = range_scale(mean);
        k = far_row_scale(row_sum2<1>(far_sums<S>(a, nt, h, g, lift), slots[flip], warps), a.inv_hidden, a.eps, lift);
        flip ^= 1;
      }
      auto finish = [&](auto far) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int j = threadIdx.x + i * nt;
          if (j < a.vpr) {
            uint4 o;
            float2 w[S::kPairs];
            weights(i, w);
#pragma unroll
            for (int p = 0; p < S::kPairs; ++p) {
              float2 d = norm_grad<far.value>(k, as_f2(S::pair(h[i], p)), as_f2(S::pair(g[i], p)), w[p], dw[i][p]);
              if (GH) d = add2(d, as_f2(S::pair(gh[i], p)));
              S::put(o, p, d);
            }
            st_stream(a.dx + row * a.dx_pitch + static_cast<int64_t>(j) * kVecBytes, o);
          }
        }
      };
      if (kOneForm || k.far) finish(std::true_type{});
      else finish(std::false_type{});
    }
    if (a.partials != nullptr) {
      float* out = a.partials + c * (static_cast<int64_t>(a.vpr) * 2 * S::kPairs);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * nt;
        if (j < a.vpr) {
          float4* p = reinterpret_cast<float4*>(out + static_cast<int64_t>(j) * 2 * S::kPairs);
#pragma unroll
          for (int k = 0; k < S::kPairs; k += 2)
            p[k / 2] = make_float4(dw[i][k].x, dw[i][k].y, dw[i][k + 1].x, dw[i][k + 1].y);
        }
      }
    }
  }
}

// d_weight[i] = sum of the chunks' partials: COLS columns a CTA, 1024 / COLS groups
// of chunks side by side, then the groups in order, 32 at a time.  The additions are
// in double, which costs nothing here: what is left of the error is the terms' and the
// chunks' own (fp32 2051 x 2048: 7.1e-8 in the 2-norm, with fp32 additions 1.5e-7).
// Launched so that it may be resident before the backward ends (its wait below is for
// the whole grid).
constexpr int kNormFinThreads = 1024;
template <int COLS>
__global__ void __launch_bounds__(kNormFinThreads)
    situ_rms_norm_dw_kernel(const float* partials, int64_t chunks, int hidden, void* d_w, int bf16) {
  constexpr int kGroups = kNormFinThreads / COLS, kParts = kGroups / 32;
  __shared__ double part[kGroups][COLS];
  const int c0 = threadIdx.x % COLS, grp = threadIdx.x / COLS;
  const int col = blockIdx.x * COLS + c0;
  double s = 0.0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (col < hidden) {
#pragma unroll 4
    for (int64_t c = grp; c < chunks; c += kGroups) s += static_cast<double>(__ldcg(partials + c * hidden + col));
  }
  part[grp][c0] = s;
  __syncthreads();
  double t = 0.0;
  if (grp < kParts) {
#pragma unroll
    for (int g = 0; g < 32; ++g) t += part[grp * 32 + g][c0];
  }
  if (kParts > 1) {
    __syncthreads();
    if (grp < kParts) part[grp][c0] = t;
    __syncthreads();
    t = 0.0;
    if (grp == 0) {
#pragma unroll
      for (int g = 0; g < kParts; ++g) t += part[g][c0];
    }
  }
  if (grp == 0 && col < hidden) {
    if (bf16)
      static_cast<__nv_bfloat16*>(d_w)[col] = __double2bfloat16(t);
    else
      static_cast<float*>(d_w)[col] = static_cast<float>(t);
  }
}

// ---- host ---------------------------------------------------------------------

// Threads and vectors per thread of a row of `vpr` vectors.  Up to 128 vectors a
// row is one warp's, so that no barrier parts its sum from its output; wider rows
// take a CTA of as few warps as leave two (then four, then eight) vectors a thread.
// MXFP8 rows, with more arithmetic per vector, keep two up to 1024 vectors (bf16
// 16384 x 7168, time of the forward: 150 us against 160 us with four; native rows
// 157 us against 140 us) and one vector is slower (32768 x 2048: 87 us, two 78 us).
struct RowShape {
  int v, threads, rows;  // rows: rows of one CTA (one warp each)
};
RowShape row_shape(int vpr, bool mx) {
  if (vpr <= 128) return {(vpr + 31) / 32, 32, 8};
  const int v = vpr <= (mx ? 1024 : 512) ? 2 : vpr <= 1024 ? 4 : 8;
  return {v, ((vpr + v - 1) / v + 31) / 32 * 32, 1};
}

// Checks shared by the three entry points.
situ_status_t norm_check(situ_dtype_t dtype, int64_t tokens, int64_t hidden, situ_dtype_t weight_dtype, double eps) {
  if (!valid_dtype(dtype) || !valid_dtype(weight_dtype))
    return fail(SITU_ERR_INVALID_ARG, "a dtype is not a situ_dtype_t");
  if (tokens < 0) return fail(SITU_ERR_INVALID_ARG, "tokens = %lld < 0", (long long)tokens);
  if (hidden <= 0) return fail(SITU_ERR_INVALID_ARG, "hidden = %lld <= 0", (long long)hidden);
  if (hidden > kNormMaxRowBytes / elem_size(dtype))
    return fail(SITU_ERR_UNSUPPORTED, "hidden = %lld exceeds %lld", (long long)hidden,
                (long long)(kNormMaxRowBytes / elem_size(dtype)));
  if (!std::isfinite(eps) || eps < 0.0) return fail(SITU_ERR_INVALID_ARG, "epsilon must be finite and >= 0");
  if ((hidden * elem_size(dtype)) % kVecBytes != 0)
    return fail(SITU_ERR_MISALIGNED, "hidden * element size (%lld bytes) is not a multiple of 16",
                (long long)(hidden * elem_size(dtype)));
  return SITU_OK;
}

int norm_weight_align(situ_dtype_t dtype, situ_dtype_t weight_dtype) {
  const int a = kVecBytes / elem_size(dtype) * elem_size(weight_dtype);
  return a < 16 ? a : 16;
}

// A row-pitched matrix argument: its stride, extent and alignment.
struct Matrix {
  const void* p;
  int64_t stride, width;
  int es;
  const char* name;
};
situ_status_t check_matrices(std::initializer_list<Matrix> ms, int64_t rows) {
  for (const Matrix& m : ms) {
    if (m.p == nullptr) return fail(SITU_ERR_INVALID_ARG, "%s is NULL", m.name);
    if (!span_fits(rows, m.stride, m.width, m.es)) return fail(SITU_ERR_INVALID_ARG, "extent of %s overflows int64", m.name);
    if (!aligned(m.p, 16) || (m.stride * m.es) % 16 != 0)
      return fail(SITU_ERR_MISALIGNED, "%s base or row pitch not 16-byte aligned", m.name);
  }
  return SITU_OK;
}
Span span_of(const Matrix& m, int64_t rows) { return matrix_span(m.p, rows, m.stride, m.width, m.es); }

using NormRingKernel = void (*)(NormBwdArgs, NormRing);
template <typename S>
NormRingKernel pick_norm_ring(int v, bool gh) {
  switch (v) {
    case 1: return gh ? situ_rms_norm_bwd_ring_kernel<S, 1, true> : situ_rms_norm_bwd_ring_kernel<S, 1, false>;
    case 2: return gh ? situ_rms_norm_bwd_ring_kernel<S, 2, true> : situ_rms_norm_bwd_ring_kernel<S, 2, false>;
    default: return gh ? situ_rms_norm_bwd_ring_kernel<S, 4, true> : situ_rms_norm_bwd_ring_kernel<S, 4, false>;
  }
}

// Launch of the staged backward: one CTA per SM for rows of more than 256 threads,
// four for narrower ones, each with its share of the shared memory (bf16 8191 x
// 4096: 51 us, with two 56 us; 32768 x 1536: 77 us, with two 90 us).
situ_status_t launch_norm_ring(const NormBwdArgs& a, bool bf, cudaStream_t s) {
  const int v = a.vpr <= 256 ? 1 : a.vpr <= 1024 ? 2 : 4;
  const int nt = ((a.vpr + v - 1) / v + 31) / 32 * 32;
  const int ctas = nt > 256 ? 1 : 4;
  NormRing r;
  r.stage_bytes = (a.gh != nullptr ? 3 : 2) * a.vpr * kVecBytes;
  r.stages = (208 * 1024 / ctas) / r.stage_bytes;
  if (r.stages > 8) r.stages = 8;
  const int smem = r.stages * r.stage_bytes;
  NormRingKernel k = bf ? pick_norm_ring<Bf16>(v, a.gh != nullptr) : pick_norm_ring<F32>(v, a.gh != nullptr);
  situ_status_t st = ensure_smem(reinterpret_cast<const void*>(k), smem);
  if (st != SITU_OK) return st;
  int grid = 0;
  st = launch_grid(reinterpret_cast<const void*>(k), nt + 32, smem, a.chunks, &grid);
  int sms = 0;
  if (st == SITU_OK) st = device_sm_count(&sms);
  if (st != SITU_OK) return st;
  if (grid > ctas * sms) grid = ctas * sms;
  k<<<grid, nt + 32, smem, s>>>(a, r);
  return check_launch("situ_glu_rms_norm_bwd");
}

using NormFwdKernel = void (*)(NormArgs, MxOut);
template <typename S, bool MX>
NormFwdKernel pick_norm_fwd(int v, bool res) {
  switch (v) {
    case 1: return res ? situ_rms_norm_fwd_kernel<S, 1, true, MX> : situ_rms_norm_fwd_kernel<S, 1, false, MX>;
    case 2: return res ? situ_rms_norm_fwd_kernel<S, 2, true, MX> : situ_rms_norm_fwd_kernel<S, 2, false, MX>;
    case 3: return res ? situ_rms_norm_fwd_kernel<S, 3, true, MX> : situ_rms_norm_fwd_kernel<S, 3, false, MX>;
    case 4: return res ? situ_rms_norm_fwd_kernel<S, 4, true, MX> : situ_rms_norm_fwd_kernel<S, 4, false, MX>;
    default: return res ? situ_rms_norm_fwd_kernel<S, 8, true, MX> : situ_rms_norm_fwd_kernel<S, 8, false, MX>;
  }
}
using NormBwdKernel = void (*)(NormBwdArgs);
template <typename S>
NormBwdKernel pick_norm_bwd(int v) {
  switch (v) {
    case 1: return situ_rms_norm_bwd_kernel<S, 1>;
    case 2: return situ_rms_norm_bwd_kernel<S, 2>;
    case 3: return situ_rms_norm_bwd_kernel<S, 3>;
    case 4: return situ_rms_norm_bwd_kernel<S, 4>;
    default: return situ_rms_norm_bwd_kernel<S, 8>;
  }
}

// The forward with native rows (mx == NULL) or MXFP8 rows.
situ_status_t norm_fwd_entry(const void* x, situ_dtype_t dtype, int64_t tokens, int64_t hidden, int64_t x_row_stride,
                             const void* residual, int64_t residual_row_stride, const void* weight,
                             situ_dtype_t weight_dtype, double epsilon, void* h, int64_t h_row_stride, void* y,
                             int64_t y_row_stride, const MxOut* mx, void* stream, const char* what) {
  tl_last_error[0] = '\0';
  situ_status_t st = norm_check(dtype, tokens, hidden, weight_dtype, epsilon);
  if (st != SITU_OK) return st;
  if (mx != nullptr) {
    if (mx->rule != SITU_MX_RULE_OCP && mx->rule != SITU_MX_RULE_CEIL)
      return fail(SITU_ERR_INVALID_ARG, "rule %d is not a situ_mx_rule_t", mx->rule);
    if (hidden % kMxBlock != 0)
      return fail(SITU_ERR_INVALID_ARG, "MXFP8 outputs need hidden a multiple of %d, got %lld", kMxBlock,
                  (long long)hidden);
    if (mx->data_pitch < hidden || mx->scale_pitch < hidden / kMxBlock)
      return fail(SITU_ERR_INVALID_ARG, "MXFP8 data or scale row pitch shorter than a row");
  }
  if ((residual == nullptr) != (h == nullptr))
    return fail(SITU_ERR_INVALID_ARG, "residual and h go together: both or neither may be NULL");
  const bool res = residual != nullptr;
  if (x_row_stride < hidden || (res && (residual_row_stride < hidden || h_row_stride < hidden)) ||
      (mx == nullptr && y_row_stride < hidden))
    return fail(SITU_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (tokens == 0) return SITU_OK;
  const int es = elem_size(dtype);
  const Matrix mxx = {x, x_row_stride, hidden, es, "x"};
  const Matrix mr = res ? Matrix{residual, residual_row_stride, hidden, es, "residual"} : mxx;
  const Matrix my = mx != nullptr ? Matrix{mx->data, mx->data_pitch, hidden, 1, "y_data"}
                                  : Matrix{y, y_row_stride, hidden, es, "y"};
  const Matrix mh = res ? Matrix{h, h_row_stride, hidden, es, "h"} : my;
  st = check_matrices({mxx, mr, my, mh}, tokens);
  if (st != SITU_OK) return st;
  if (mx != nullptr) {
    if (mx->scale == nullptr) return fail(SITU_ERR_INVALID_ARG, "y_scale is NULL");
    if (!span_fits(tokens, mx->scale_pitch, hidden / kMxBlock, 1))
      return fail(SITU_ERR_INVALID_ARG, "extent of y_scale overflows int64");
  }
  if (weight == nullptr) return fail(SITU_ERR_INVALID_ARG, "weight is NULL");
  if (!aligned(weight, norm_weight_align(dtype, weight_dtype)))
    return fail(SITU_ERR_MISALIGNED, "weight must be %d-byte aligned", norm_weight_align(dtype, weight_dtype));
  const Span ins[] = {span_of(mxx, tokens), span_of(mr, tokens),
                      matrix_span(weight, 1, hidden, hidden, elem_size(weight_dtype))};
  Span outs[3] = {span_of(my, tokens)};
  int n_outs = 1;
  if (res) outs[n_outs++] = span_of(mh, tokens);
  if (mx != nullptr) outs[n_outs++] = matrix_span(mx->scale, tokens, mx->scale_pitch, hidden / kMxBlock, 1);
  for (int i = 0; i < n_outs; ++i) {
    for (const Span& s : ins)
      if (overlap(outs[i], s)) return fail(SITU_ERR_INVALID_ARG, "an output overlaps an input");
    for (int k = i + 1; k < n_outs; ++k)
      if (overlap(outs[i], outs[k])) return fail(SITU_ERR_INVALID_ARG, "outputs overlap each other");
  }

  NormArgs a{};
  a.x = static_cast<const char*>(x);
  a.x_pitch = x_row_stride * es;
  a.res = static_cast<const char*>(residual);
  a.res_pitch = res ? residual_row_stride * es : 0;
  a.w = weight;
  a.w_bf16 = weight_dtype == SITU_DTYPE_BF16;
  a.h = static_cast<char*>(h);
  a.h_pitch = res ? h_row_stride * es : 0;
  a.y = static_cast<char*>(y);
  a.y_pitch = mx == nullptr ? y_row_stride * es : 0;
  a.tokens = tokens;
  a.vpr = static_cast<int>(hidden * es / kVecBytes);
  a.eps = static_cast<float>(epsilon);
  a.inv_hidden = static_cast<float>(1.0 / static_cast<double>(hidden));
  const RowShape rs = row_shape(a.vpr, mx != nullptr);
  const bool bf = dtype == SITU_DTYPE_BF16;
  NormFwdKernel k = mx != nullptr ? (bf ? pick_norm_fwd<Bf16, true>(rs.v, res) : pick_norm_fwd<F32, true>(rs.v, res))
                                  : (bf ? pick_norm_fwd<Bf16, false>(rs.v, res) : pick_norm_fwd<F32, false>(rs.v, res));
  int grid = 0;
  const int64_t groups = (tokens + rs.rows - 1) / rs.rows;
  const int cap = g_max_ctas.load(std::memory_order_relaxed);
  // Native rows of 128 vectors and more: a CTA per group of rows, whose turnover
  // overlaps one row's stores with the next one's loads (bf16 16384 x 7168: 140 us, a
  // loop of resident CTAs 153 us; 65536 x 1024: 82, 93).  Narrower rows and MXFP8
  // ones do better in the loop (60000 x 256: 19, 22; MXFP8 16384 x 7168: 162, 170).
  if (mx == nullptr && a.vpr >= 128 && cap <= 0 && groups <= INT32_MAX) {
    grid = static_cast<int>(groups);
  } else {
    st = launch_grid(reinterpret_cast<const void*>(k), rs.threads * rs.rows, 0, groups, &grid);
    if (st != SITU_OK) return st;
  }
  k<<<grid, dim3(rs.threads, rs.rows), 0, static_cast<cudaStream_t>(stream)>>>(a, mx != nullptr ? *mx : MxOut{});
  return check_launch(what);
}

}  // namespace

int norm_device_status(int clear) { return unit_device_status(clear); }

extern "C" {

situ_status_t situ_glu_rms_norm_fwd(const void* x, situ_dtype_t dtype, int64_t tokens, int64_t hidden,
                                    int64_t x_row_stride, const void* residual, int64_t residual_row_stride,
                                    const void* weight, situ_dtype_t weight_dtype, double epsilon, void* h,
                                    int64_t h_row_stride, void* y, int64_t y_row_stride, void* stream) {
  return norm_fwd_entry(x, dtype, tokens, hidden, x_row_stride, residual, residual_row_stride, weight, weight_dtype,
                        epsilon, h, h_row_stride, y, y_row_stride, nullptr, stream, "situ_glu_rms_norm_fwd");
}

situ_status_t situ_glu_rms_norm_fwd_mxfp8(const void* x, situ_dtype_t dtype, int64_t tokens, int64_t hidden,
                                          int64_t x_row_stride, const void* residual, int64_t residual_row_stride,
                                          const void* weight, situ_dtype_t weight_dtype, double epsilon, void* h,
                                          int64_t h_row_stride, void* y_data, int64_t y_data_row_stride,
                                          void* y_scale, int64_t y_scale_row_stride, situ_mx_rule_t rule,
                                          void* stream) {
  const MxOut m{static_cast<char*>(y_data), y_data_row_stride, static_cast<uint8_t*>(y_scale), y_scale_row_stride,
                static_cast<int>(rule)};
  return norm_fwd_entry(x, dtype, tokens, hidden, x_row_stride, residual, residual_row_stride, weight, weight_dtype,
                        epsilon, h, h_row_stride, nullptr, 0, &m, stream, "situ_glu_rms_norm_fwd_mxfp8");
}

size_t situ_glu_rms_norm_bwd_workspace_bytes(int64_t tokens, int64_t hidden, int want_dweight) {
  if (!want_dweight || tokens <= 0 || hidden <= 0 || hidden > kNormMaxRowBytes / 2) return 0;
  return (static_cast<size_t>(norm_chunks(tokens, hidden)) * static_cast<size_t>(hidden) * sizeof(float) + 255) / 256 * 256;
}

situ_status_t situ_glu_rms_norm_bwd(const void* grad_y, int64_t grad_y_row_stride, const void* grad_h,
                                    int64_t grad_h_row_stride, const void* h, situ_dtype_t dtype, int64_t tokens,
                                    int64_t hidden, int64_t h_row_stride, const void* weight,
                                    situ_dtype_t weight_dtype, double epsilon, void* d_x, int64_t d_x_row_stride,
                                    void* d_weight, void* workspace, size_t workspace_bytes, void* stream) {
  tl_last_error[0] = '\0';
  situ_status_t st = norm_check(dtype, tokens, hidden, weight_dtype, epsilon);
  if (st != SITU_OK) return st;
  if (grad_y_row_stride < hidden || h_row_stride < hidden || d_x_row_stride < hidden ||
      (grad_h != nullptr && grad_h_row_stride < hidden))
    return fail(SITU_ERR_INVALID_ARG, "a row stride is shorter than its row");
  const int es = elem_size(dtype), wes = elem_size(weight_dtype);
  if (d_weight != nullptr && !aligned(d_weight, wes))
    return fail(SITU_ERR_MISALIGNED, "d_weight not aligned to its element");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (d_weight != nullptr) {
      cudaError_t err = cudaMemsetAsync(d_weight, 0, static_cast<size_t>(hidden) * wes, s);
      if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(err));
    }
    return SITU_OK;
  }
  const Matrix mg = {grad_y, grad_y_row_stride, hidden, es, "grad_y"};
  const Matrix mhh = {h, h_row_stride, hidden, es, "h"};
  const Matrix mgh = grad_h != nullptr ? Matrix{grad_h, grad_h_row_stride, hidden, es, "grad_h"} : mg;
  const Matrix md = {d_x, d_x_row_stride, hidden, es, "d_x"};
  st = check_matrices({mg, mhh, mgh, md}, tokens);
  if (st != SITU_OK) return st;
  if (weight == nullptr) return fail(SITU_ERR_INVALID_ARG, "weight is NULL");
  if (!aligned(weight, norm_weight_align(dtype, weight_dtype)))
    return fail(SITU_ERR_MISALIGNED, "weight must be %d-byte aligned", norm_weight_align(dtype, weight_dtype));
  const size_t need = situ_glu_rms_norm_bwd_workspace_bytes(tokens, hidden, d_weight != nullptr);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(SITU_ERR_INVALID_ARG, "workspace of %zu bytes needed, got %zu", need,
                  workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
    if (!aligned(workspace, 16)) return fail(SITU_ERR_MISALIGNED, "workspace not 16-byte aligned");
  }
  const Span ins[] = {span_of(mg, tokens), span_of(mhh, tokens), span_of(mgh, tokens),
                      matrix_span(weight, 1, hidden, hidden, wes)};
  Span outs[3] = {span_of(md, tokens)};
  int n_outs = 1;
  if (d_weight != nullptr) {
    outs[n_outs++] = matrix_span(d_weight, 1, hidden, hidden, wes);
    const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
    outs[n_outs++] = {ws, ws + need};
  }
  for (int i = 0; i < n_outs; ++i) {
    for (const Span& sp : ins)
      if (overlap(outs[i], sp)) return fail(SITU_ERR_INVALID_ARG, "an output overlaps an input");
    for (int k = i + 1; k < n_outs; ++k)
      if (overlap(outs[i], outs[k])) return fail(SITU_ERR_INVALID_ARG, "outputs overlap each other");
  }

  NormBwdArgs a{};
  a.gy = static_cast<const char*>(grad_y);
  a.gy_pitch = grad_y_row_stride * es;
  a.gh = static_cast<const char*>(grad_h);
  a.gh_pitch = grad_h != nullptr ? grad_h_row_stride * es : 0;
  a.h = static_cast<const char*>(h);
  a.h_pitch = h_row_stride * es;
  a.w = weight;
  a.w_bf16 = weight_dtype == SITU_DTYPE_BF16;
  a.dx = static_cast<char*>(d_x);
  a.dx_pitch = d_x_row_stride * es;
  a.partials = d_weight != nullptr ? static_cast<float*>(workspace) : nullptr;
  a.tokens = tokens;
  a.chunks = norm_chunks(tokens, hidden);
  a.vpr = static_cast<int>(hidden * es / kVecBytes);
  a.eps = static_cast<float>(epsilon);
  a.inv_hidden = static_cast<float>(1.0 / static_cast<double>(hidden));
  const bool bf = dtype == SITU_DTYPE_BF16;
  // Staged rows from 129 vectors up to 2048, of which two or more fit in shared
  // memory.  Narrower rows have a warp each and enough of them in flight (bf16 65536 x
  // 1024: 92 us, staged 100; 40000 x 512: 29, staged 51); of the wider ones nearly all
  // gain from the ring (16384 x 7168: 150 us, direct 286; 8191 x 4096: 48, 52; 32768 x
  // 1536: 75, 78; 32768 x 2048 with grad_h 98, 92, without 78, 82).
  if (a.vpr > 128 && a.vpr <= 2048) {
    st = launch_norm_ring(a, bf, s);
  } else {
    const RowShape rs = row_shape(a.vpr, false);
    NormBwdKernel k = bf ? pick_norm_bwd<Bf16>(rs.v) : pick_norm_bwd<F32>(rs.v);
    const int smem = rs.v == 8 ? rs.v * rs.threads * (kVecBytes / es) * 4 : 0;
    if (smem > 48 * 1024) {
      st = ensure_smem(reinterpret_cast<const void*>(k), smem);
      if (st != SITU_OK) return st;
    }
    int grid = 0;
    st = launch_grid(reinterpret_cast<const void*>(k), rs.threads * rs.rows, smem, (a.chunks + rs.rows - 1) / rs.rows,
                     &grid);
    if (st != SITU_OK) return st;
    k<<<grid, dim3(rs.threads, rs.rows), smem, s>>>(a);
    st = check_launch("situ_glu_rms_norm_bwd");
  }
  if (st != SITU_OK || d_weight == nullptr) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int cols = hidden <= 1024 ? 8 : 32;
  cfg.gridDim = dim3(static_cast<unsigned>((hidden + cols - 1) / cols));
  cfg.blockDim = dim3(kNormFinThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err =
      cudaLaunchKernelEx(&cfg, cols == 8 ? situ_rms_norm_dw_kernel<8> : situ_rms_norm_dw_kernel<32>,
                         static_cast<const float*>(a.partials), a.chunks, static_cast<int>(hidden), d_weight,
                         weight_dtype == SITU_DTYPE_BF16 ? 1 : 0);
  if (err != cudaSuccess)
    return fail(SITU_ERR_CUDA, "situ_glu_rms_norm_bwd (d_weight) launch: %s", cudaGetErrorString(err));
  return check_launch("situ_glu_rms_norm_bwd (d_weight)");
}

}  // extern "C"
