// situ_moe.cu -- the whole expert layer for the few tokens of a decoding step
// (include/situ_glu.h, situ_glu_moe_fwd), in two kernels.
//
//   a[t, e] = SiTU-GLU(W1_e x[t]) w[t, e],   y[t] = sum_e W2_e a[t, e]
//
// A decoding step reads 6 hidden inter bytes of weights per active expert and
// does a few operations with each, so the bound is the HBM bandwidth of the
// weights: every weight is read once, straight from HBM into the registers
// that feed the tensor cores.  The weights are the 16-row operand of
// mma.m16n8k16 (the tokens fill its eight columns), so one instruction serves
// up to eight tokens of an expert; with these row counts the products are a
// few per cent of the tensor rate and never the limit.
//
// A unit of work is 16 weight rows of one expert against all of that expert's
// tokens: kernel 1 takes 8 gate rows with their 8 up rows (one thread then
// holds G and U of the same column and applies the activation at once), kernel
// 2 takes 16 rows of W2_e.  The four warps of a CTA split the sum over k in
// 64-wide chunks and add their parts through shared memory in warp order.
//
// Which tokens an expert has is worked out by every CTA from the token's
// choices: a 64-bit token mask per expert, and a running count over the
// experts.  Entry (e, t), the count's value plus the rank of t in e's mask,
// numbers the rows of the intermediate buffers.  A choice that names an expert
// twice is one entry with the sum of the weights: the layer is linear in them.
//
// Kernel 2 leaves one fp32 row per entry; the CTA that completes the last
// expert of a 16-column group (a counter per group) adds each token's rows in
// the order of its choices.  No sum depends on which CTA ran when.

#include "situ_host.cuh"

namespace {

constexpr int kMoeThreads = 128;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopk = 16;
constexpr int kMoeMaxExperts = 1024;
constexpr int64_t kMoeMaxDim = 32768;
constexpr int kMoeChunk = 64;  // k elements of one warp step

struct MoeArgs {
  const char* x;
  int64_t x_pitch;           // bytes
  const int64_t* ids;
  int64_t ids_stride;        // elements
  const void* weights;       // NULL: 1
  int64_t weights_stride;    // elements
  int weights_bf16;
  const char* w1;
  int64_t w1_pitch;          // bytes
  const char* w2;
  int64_t w2_pitch;          // bytes
  char* y;
  int64_t y_pitch;           // bytes
  __nv_bfloat16* act;        // [entries][2][inter]: the rounded activations, then the remainders
  float* part;               // [entries][hidden]
  int* done;                 // [hidden / 16] experts completed
  int tokens, topk, experts, hidden, inter;
  Coeffs c;
};

// The call's routing, in shared memory.
struct MoePlan {
  unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
  uint16_t start[kMoeMaxExperts];           // first entry of each expert
  uint16_t active[kMoeMaxTokens * kMoeMaxTopk];  // experts that have a token, rising
  int16_t id[kMoeMaxTokens * kMoeMaxTopk];  // [token][choice], -1: none
  float w[kMoeMaxTokens * kMoeMaxTopk];
  int warp_active[kMoeWarps], warp_entries[kMoeWarps];
  int n_active;
};

__device__ __forceinline__ void moe_plan(const MoeArgs& a, MoePlan& p) {
  const int n = a.tokens * a.topk;
  for (int e = threadIdx.x; e < a.experts; e += kMoeThreads) p.mask[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kMoeThreads) {
    const int t = i / a.topk, j = i - t * a.topk;
    const int64_t id = a.ids[t * a.ids_stride + j];
    const bool in = id >= 0 && id < a.experts;
    p.id[i] = static_cast<int16_t>(in ? id : -1);
    float w = 1.0f;
    if (a.weights != nullptr) {
      const int64_t at = t * a.weights_stride + j;
      w = a.weights_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.weights)[at])
                         : static_cast<const float*>(a.weights)[at];
    }
    p.w[i] = w;
    if (in) atomicOr(&p.mask[id], 1ull << t);
  }
  __syncthreads();
  // running counts over the experts: each thread a run of them, then the warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (a.experts + kMoeThreads - 1) / kMoeThreads;
  const int e0 = min(a.experts, static_cast<int>(threadIdx.x) * per), e1 = min(a.experts, e0 + per);
  int act = 0, ent = 0;
  for (int e = e0; e < e1; ++e) {
    const int c = __popcll(p.mask[e]);
    act += c > 0;
    ent += c;
  }
  int act_incl = act, ent_incl = ent;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int va = __shfl_up_sync(0xffffffffu, act_incl, o), ve = __shfl_up_sync(0xffffffffu, ent_incl, o);
    if (lane >= o) {
      act_incl += va;
      ent_incl += ve;
    }
  }
  if (lane == 31) {
    p.warp_active[warp] = act_incl;
    p.warp_entries[warp] = ent_incl;
  }
  __syncthreads();
  int run_a = act_incl - act, run_e = ent_incl - ent;
  for (int w = 0; w < warp; ++w) {
    run_a += p.warp_active[w];
    run_e += p.warp_entries[w];
  }
  for (int e = e0; e < e1; ++e) {
    const int c = __popcll(p.mask[e]);
    p.start[e] = static_cast<uint16_t>(run_e);
    if (c > 0) p.active[run_a++] = static_cast<uint16_t>(e);
    run_e += c;
  }
  if (threadIdx.x == kMoeThreads - 1) p.n_active = run_a;
  __syncthreads();
}

// The weight of entry (e, t): the sum over the token's choices that name e.
__device__ __forceinline__ float moe_weight(const MoeArgs& a, const MoePlan& p, int e, int t) {
  float w = 0.0f;
  for (int j = 0; j < a.topk; ++j)
    if (p.id[t * a.topk + j] == e) w += p.w[t * a.topk + j];
  return w;
}

// The k-th set bit of a token mask (k < its count).
__device__ __forceinline__ int mask_token(unsigned long long m, int k) {
  for (int i = 0; i < k; ++i) m &= m - 1;
  return __ffsll(static_cast<long long>(m)) - 1;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D[16 x 8 NT] += A[16 x k] B[8 NT x k]^T over this warp's chunks.  Thread
// (g, t) = (lane / 4, lane % 4) loads the 16-byte vectors t of rows g and g + 8
// of A and row g of each B tile; since the sum may run over k in any order, the
// four words of a vector serve as the k pairs (2t, 2t + 8) of two instructions,
// the same for A and B.  U chunks are requested before any is used.  PARTS: B
// rows come as a value and its remainder, `part` bytes apart.
template <int NT, int PARTS, int U>
__device__ __forceinline__ void mma_rows(float (&acc)[NT][4], const char* a_lo, const char* a_hi, const char* const (&b)[NT],
                                         int64_t part, int chunks, int warp) {
#pragma unroll 1
  for (int c0 = warp; c0 < chunks; c0 += kMoeWarps * U) {
    uint4 lo[U][2], hi[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kMoeWarps;
      if (c < chunks) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          lo[u][v] = ld_stream(a_lo + c * (kMoeChunk * 2) + v * 64);
          hi[u][v] = ld_stream(a_hi + c * (kMoeChunk * 2) + v * 64);
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) lo[u][v] = hi[u][v] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kMoeWarps;
      if (c >= chunks) break;  // the same for the whole warp
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint4 bv = make_uint4(0, 0, 0, 0);
            if (b[n] != nullptr) bv = *reinterpret_cast<const uint4*>(b[n] + q * part + c * (kMoeChunk * 2) + v * 64);
            mma_bf16(acc[n], lo[u][v].x, hi[u][v].x, lo[u][v].y, hi[u][v].y, bv.x, bv.y);
            mma_bf16(acc[n], lo[u][v].z, hi[u][v].z, lo[u][v].w, hi[u][v].w, bv.z, bv.w);
          }
    }
  }
}

// The warps' parts of a unit, added in warp order: warp w's sum for tile n of
// lane l at red[(w * 8 + n) * 32 + l].  Tile n's total goes to warp n % 4.
template <int NT>
__device__ __forceinline__ void put_parts(float4* red, const float (&acc)[NT][4], int warp, int lane) {
#pragma unroll
  for (int n = 0; n < NT; ++n) red[(warp * 8 + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
}
__device__ __forceinline__ float4 sum_parts(const float4* red, int n, int lane) {
  float4 s = red[n * 32 + lane];
#pragma unroll
  for (int w = 1; w < kMoeWarps; ++w) {
    const float4 v = red[(w * 8 + n) * 32 + lane];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  return s;
}

template <int NT, int U>
__device__ __forceinline__ void fc1_unit(const MoeArgs& a, const MoePlan& p, float4* red, int e, int col0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const unsigned long long mask = p.mask[e];
  const int count = __popcll(mask);
  const char* rows[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    rows[n] = n * 8 + g < count ? a.x + mask_token(mask, n * 8 + g) * a.x_pitch + t * 16 : nullptr;
  const char* gate = a.w1 + (static_cast<int64_t>(e) * 2 * a.inter + col0 + g) * a.w1_pitch + t * 16;
  float acc[NT][4] = {};
  mma_rows<NT, 1, U>(acc, gate, gate + static_cast<int64_t>(a.inter) * a.w1_pitch, rows, 0, a.hidden / kMoeChunk, warp);
  put_parts<NT>(red, acc, warp, lane);
}

// v as the sum of two bf16 numbers, `apart` elements from each other: 16 bits of
// its significand (an infinite rounding has no remainder).
__device__ __forceinline__ void put_split(__nv_bfloat16* out, int apart, float v) {
  const __nv_bfloat16 hi = __float2bfloat16(v);
  const float rest = v - __bfloat162float(hi);
  out[0] = hi;
  out[apart] = __float2bfloat16(isfinite(rest) ? rest : 0.0f);
}

template <int GATE, bool HAS_LB>
__global__ void __launch_bounds__(kMoeThreads, 4) situ_moe_fc1_kernel(const MoeArgs a) {
  __shared__ MoePlan plan;
  __shared__ float4 red[kMoeWarps * 8 * 32];
  for (int i = blockIdx.x * kMoeThreads + threadIdx.x; i < a.hidden / 16; i += gridDim.x * kMoeThreads) a.done[i] = 0;
  moe_plan(a, plan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int blocks = a.inter / 8, units = plan.n_active * blocks;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int e = plan.active[u / blocks], col0 = (u % blocks) * 8;
    const unsigned long long mask = plan.mask[e];
    const int count = __popcll(mask), tiles = (count + 7) / 8;
    if (tiles == 1) fc1_unit<1, 4>(a, plan, red, e, col0);
    else if (tiles == 2) fc1_unit<2, 2>(a, plan, red, e, col0);
    else if (tiles <= 4) fc1_unit<4, 2>(a, plan, red, e, col0);
    else fc1_unit<8, 1>(a, plan, red, e, col0);
    __syncthreads();
    for (int n = warp; n < tiles; n += kMoeWarps) {
      const float4 s = sum_parts(red, n, lane);  // G of tokens 2t, 2t + 1, then U
      const int k0 = n * 8 + 2 * t;
      if (k0 < count) {
        const bool two = k0 + 1 < count;
        const float2 w = make_float2(moe_weight(a, plan, e, mask_token(mask, k0)),
                                     two ? moe_weight(a, plan, e, mask_token(mask, k0 + 1)) : 0.0f);
        const Bits2 gb = {__float_as_uint(s.x), __float_as_uint(s.y)};
        const Bits2 ub = {__float_as_uint(s.z), __float_as_uint(s.w)};
        const float2 v = fwd_pair_abs<GATE, HAS_LB, F32>(gb, ub, mul2(w, splat(a.c.bb)), a.c);
        __nv_bfloat16* out = a.act + static_cast<int64_t>(plan.start[e] + k0) * 2 * a.inter + col0 + g;
        put_split(out, a.inter, v.x);
        if (two) put_split(out + 2 * a.inter, a.inter, v.y);
      }
    }
    __syncthreads();
  }
}

template <int NT, int U>
__device__ __forceinline__ void fc2_unit(const MoeArgs& a, const MoePlan& p, float4* red, int e, int row0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int count = __popcll(p.mask[e]);
  const char* rows[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    rows[n] = n * 8 + g < count
                  ? reinterpret_cast<const char*>(a.act + static_cast<int64_t>(p.start[e] + n * 8 + g) * 2 * a.inter) + t * 16
                  : nullptr;
  const char* w = a.w2 + (static_cast<int64_t>(e) * a.hidden + row0 + g) * a.w2_pitch + t * 16;
  float acc[NT][4] = {};
  mma_rows<NT, 2, U>(acc, w, w + 8 * a.w2_pitch, rows, static_cast<int64_t>(a.inter) * 2, a.inter / kMoeChunk, warp);
  put_parts<NT>(red, acc, warp, lane);
}

__global__ void __launch_bounds__(kMoeThreads, 4) situ_moe_fc2_kernel(const MoeArgs a) {
  __shared__ MoePlan plan;
  __shared__ float4 red[kMoeWarps * 8 * 32];
  __shared__ int last;
  moe_plan(a, plan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int blocks = a.hidden / 16, units = plan.n_active * blocks;
  if (plan.n_active == 0) {  // no token has an expert
    for (int b = blockIdx.x; b < blocks; b += gridDim.x)
      for (int i = threadIdx.x; i < a.tokens * 16; i += kMoeThreads)
        *reinterpret_cast<__nv_bfloat16*>(a.y + (i / 16) * a.y_pitch + (b * 16 + i % 16) * 2) = __float2bfloat16(0.0f);
    return;
  }
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int e = plan.active[u / blocks], block = u % blocks, row0 = block * 16;
    const int count = __popcll(plan.mask[e]), tiles = (count + 7) / 8;
    if (tiles == 1) fc2_unit<1, 4>(a, plan, red, e, row0);
    else if (tiles == 2) fc2_unit<2, 2>(a, plan, red, e, row0);
    else if (tiles <= 4) fc2_unit<4, 2>(a, plan, red, e, row0);
    else fc2_unit<8, 1>(a, plan, red, e, row0);
    __syncthreads();
    for (int n = warp; n < tiles; n += kMoeWarps) {
      const float4 s = sum_parts(red, n, lane);  // row g of tokens 2t, 2t + 1, then row g + 8
      const int k0 = n * 8 + 2 * t;
      if (k0 < count) {
        float* out = a.part + static_cast<int64_t>(plan.start[e] + k0) * a.hidden + row0 + g;
        out[0] = s.x;
        out[8] = s.z;
        if (k0 + 1 < count) {
          out[a.hidden] = s.y;
          out[a.hidden + 8] = s.w;
        }
      }
    }
    // the CTA that completes the group's last expert adds the tokens' rows
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&a.done[block], 1) == plan.n_active - 1;
    __syncthreads();
    if (last) {
      __threadfence();
      for (int i = threadIdx.x; i < a.tokens * 16; i += kMoeThreads) {
        const int tok = i / 16, col = row0 + i % 16;
        float s = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
          const int id = plan.id[tok * a.topk + j];
          bool first = id >= 0;
          for (int k = 0; k < j; ++k) first = first && plan.id[tok * a.topk + k] != id;
          if (first) {
            const int entry = plan.start[id] + __popcll(plan.mask[id] & ((1ull << tok) - 1));
            s += __ldcg(a.part + static_cast<int64_t>(entry) * a.hidden + col);
          }
        }
        *reinterpret_cast<__nv_bfloat16*>(a.y + tok * a.y_pitch + col * 2) = __float2bfloat16(s);
      }
    }
  }
}

// ---- host ---------------------------------------------------------------------

struct MoeWorkspace {
  size_t act, part, done;  // bytes of each part, multiples of 256
};
MoeWorkspace moe_workspace(int64_t tokens, int64_t topk, int64_t hidden, int64_t inter) {
  auto up = [](int64_t b) { return static_cast<size_t>((b + 255) / 256 * 256); };
  return {up(tokens * topk * inter * 4), up(tokens * topk * hidden * 4), up(hidden / 16 * 4)};
}

using MoeKernel = void (*)(MoeArgs);
template <bool LB>
MoeKernel pick_moe_fc1(int gate) {
  switch (gate) {
    case kGateSquare: return situ_moe_fc1_kernel<kGateSquare, LB>;
    case kGateEqual: return situ_moe_fc1_kernel<kGateEqual, LB>;
    case kGateRoot: return situ_moe_fc1_kernel<kGateRoot, LB>;
    default: return situ_moe_fc1_kernel<kGateGeneric, LB>;
  }
}

}  // namespace

int moe_device_status(int clear) { return unit_device_status(clear); }

extern "C" {

size_t situ_glu_moe_workspace_bytes(int64_t tokens, int64_t topk, int64_t hidden, int64_t inter) {
  if (tokens <= 0 || tokens > kMoeMaxTokens || topk <= 0 || topk > kMoeMaxTopk || hidden <= 0 || hidden > kMoeMaxDim ||
      inter <= 0 || inter > kMoeMaxDim)
    return 0;
  const MoeWorkspace w = moe_workspace(tokens, topk, hidden, inter);
  return w.act + w.part + w.done;
}

situ_status_t situ_glu_moe_fwd(const void* x, int64_t tokens, int64_t hidden, int64_t x_row_stride,
                               const int64_t* topk_ids, int64_t topk, int64_t topk_ids_row_stride,
                               const void* topk_weights, situ_dtype_t weights_dtype, int64_t topk_weights_row_stride,
                               const void* w1, int64_t experts, int64_t inter, int64_t w1_row_stride, const void* w2,
                               int64_t w2_row_stride, double beta, int has_linear_beta, double linear_beta, void* y,
                               int64_t y_row_stride, void* workspace, size_t workspace_bytes, void* stream) {
  tl_last_error[0] = '\0';
  if (!finite_positive(beta)) return fail(SITU_ERR_INVALID_ARG, "beta must be finite and > 0");
  if (has_linear_beta != 0 && has_linear_beta != 1)
    return fail(SITU_ERR_INVALID_ARG, "has_linear_beta must be 0 or 1");
  if (has_linear_beta && !finite_positive(linear_beta))
    return fail(SITU_ERR_INVALID_ARG, "linear_beta must be finite and > 0");
  if (topk_weights != nullptr && !valid_dtype(weights_dtype))
    return fail(SITU_ERR_INVALID_ARG, "weights_dtype %d is not a situ_dtype_t", (int)weights_dtype);
  if (tokens < 0) return fail(SITU_ERR_INVALID_ARG, "tokens = %lld < 0", (long long)tokens);
  if (tokens > kMoeMaxTokens)
    return fail(SITU_ERR_UNSUPPORTED, "tokens = %lld exceeds %d: group the rows by expert and call situ_glu_fc1_fwd",
                (long long)tokens, kMoeMaxTokens);
  if (topk < 1 || topk > kMoeMaxTopk)
    return fail(SITU_ERR_UNSUPPORTED, "topk must be in [1, %d], got %lld", kMoeMaxTopk, (long long)topk);
  if (experts < 1 || experts > kMoeMaxExperts)
    return fail(SITU_ERR_UNSUPPORTED, "experts must be in [1, %d], got %lld", kMoeMaxExperts, (long long)experts);
  if (hidden < kMoeChunk || hidden % kMoeChunk != 0 || hidden > kMoeMaxDim || inter < kMoeChunk ||
      inter % kMoeChunk != 0 || inter > kMoeMaxDim)
    return fail(SITU_ERR_UNSUPPORTED, "hidden and inter must be positive multiples of %d up to %lld, got %lld and %lld",
                kMoeChunk, (long long)kMoeMaxDim, (long long)hidden, (long long)inter);
  if (x_row_stride < hidden || topk_ids_row_stride < topk ||
      (topk_weights != nullptr && topk_weights_row_stride < topk) || w1_row_stride < hidden ||
      w2_row_stride < inter || y_row_stride < hidden)
    return fail(SITU_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (tokens == 0) return SITU_OK;
  if (x == nullptr || topk_ids == nullptr || w1 == nullptr || w2 == nullptr || y == nullptr)
    return fail(SITU_ERR_INVALID_ARG, "x, topk_ids, w1, w2 or y is NULL");
  const int wes = topk_weights != nullptr ? elem_size(weights_dtype) : 1;
  if (!span_fits(tokens, x_row_stride, hidden, 2) || !span_fits(tokens, topk_ids_row_stride, topk, 8) ||
      (topk_weights != nullptr && !span_fits(tokens, topk_weights_row_stride, topk, wes)) ||
      !span_fits(experts * 2 * inter, w1_row_stride, hidden, 2) ||
      !span_fits(experts * hidden, w2_row_stride, inter, 2) || !span_fits(tokens, y_row_stride, hidden, 2))
    return fail(SITU_ERR_INVALID_ARG, "tensor extent overflows int64");
  if (!aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) || !aligned(y, 16) || (x_row_stride * 2) % 16 != 0 ||
      (w1_row_stride * 2) % 16 != 0 || (w2_row_stride * 2) % 16 != 0 || (y_row_stride * 2) % 16 != 0 ||
      !aligned(topk_ids, 8) || (topk_weights != nullptr && !aligned(topk_weights, wes)))
    return fail(SITU_ERR_MISALIGNED, "x, w1, w2, y (16 bytes), topk_ids (8) or topk_weights base or row pitch misaligned");
  const MoeWorkspace w = moe_workspace(tokens, topk, hidden, inter);
  const size_t need = w.act + w.part + w.done;
  if (workspace == nullptr || workspace_bytes < need)
    return fail(SITU_ERR_INVALID_ARG, "workspace of %zu bytes needed, got %zu", need,
                workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
  if (!aligned(workspace, 16)) return fail(SITU_ERR_MISALIGNED, "workspace not 16-byte aligned");
  const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
  const Span outs[] = {matrix_span(y, tokens, y_row_stride, hidden, 2), {ws, ws + need}};
  const Span ins[] = {matrix_span(x, tokens, x_row_stride, hidden, 2),
                      matrix_span(topk_ids, tokens, topk_ids_row_stride, topk, 8),
                      topk_weights != nullptr ? matrix_span(topk_weights, tokens, topk_weights_row_stride, topk, wes)
                                              : Span{0, 0},
                      matrix_span(w1, experts * 2 * inter, w1_row_stride, hidden, 2),
                      matrix_span(w2, experts * hidden, w2_row_stride, inter, 2)};
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (overlap(o, i)) return fail(SITU_ERR_INVALID_ARG, "y or workspace overlaps an input");
  if (overlap(outs[0], outs[1])) return fail(SITU_ERR_INVALID_ARG, "y overlaps workspace");

  MoeArgs a{};
  a.x = static_cast<const char*>(x);
  a.x_pitch = x_row_stride * 2;
  a.ids = topk_ids;
  a.ids_stride = topk_ids_row_stride;
  a.weights = topk_weights;
  a.weights_stride = topk_weights_row_stride;
  a.weights_bf16 = topk_weights != nullptr && weights_dtype == SITU_DTYPE_BF16;
  a.w1 = static_cast<const char*>(w1);
  a.w1_pitch = w1_row_stride * 2;
  a.w2 = static_cast<const char*>(w2);
  a.w2_pitch = w2_row_stride * 2;
  a.y = static_cast<char*>(y);
  a.y_pitch = y_row_stride * 2;
  char* base = static_cast<char*>(workspace);
  a.act = reinterpret_cast<__nv_bfloat16*>(base);
  a.part = reinterpret_cast<float*>(base + w.act);
  a.done = reinterpret_cast<int*>(base + w.act + w.part);
  a.tokens = static_cast<int>(tokens);
  a.topk = static_cast<int>(topk);
  a.experts = static_cast<int>(experts);
  a.hidden = static_cast<int>(hidden);
  a.inter = static_cast<int>(inter);
  int gate = kGateGeneric;
  fill_coeffs(beta, has_linear_beta, linear_beta, &a.c, &gate);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t most = experts < tokens * topk ? experts : tokens * topk;  // experts that can be active
  MoeKernel k1 = has_linear_beta ? pick_moe_fc1<true>(gate) : pick_moe_fc1<false>(gate);
  int grid = 0;
  situ_status_t st = launch_grid(reinterpret_cast<const void*>(k1), kMoeThreads, 0, most * (inter / 8), &grid);
  if (st != SITU_OK) return st;
  k1<<<grid, kMoeThreads, 0, s>>>(a);
  st = check_launch("situ_glu_moe_fwd (FC1)");
  if (st != SITU_OK) return st;
  st = launch_grid(reinterpret_cast<const void*>(situ_moe_fc2_kernel), kMoeThreads, 0, most * (hidden / 16), &grid);
  if (st != SITU_OK) return st;
  situ_moe_fc2_kernel<<<grid, kMoeThreads, 0, s>>>(a);
  return check_launch("situ_glu_moe_fwd (FC2)");
}

}  // extern "C"
