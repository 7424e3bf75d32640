// situ_moe.cu -- the whole expert layer for the few tokens of a decoding step
// (include/situ_glu.h, situ_glu_moe_fwd), in two kernels.
//
//   a[t, e] = SiTU-GLU(W1_e x[t]) w[t, e],   y[t] = sum_e W2_e a[t, e]
//
// A decoding step reads 6 hidden inter bytes of weights per active expert and
// does a few operations with each, so the bound is the HBM bandwidth of the
// weights: every weight is read once.  The tensor cores take them from shared
// memory where TMA puts them (tcgen05.mma, the weights as the row operand, the
// tokens as the few columns), so no thread touches a weight.
//
// A unit of work is 128 weight rows of one expert: in kernel 1 64 gate rows and
// the 64 up rows of the same columns, in kernel 2 128 rows of W2_e.  Each SM has
// one CTA with a contiguous run of units, and one warp streams their rows, a 32
// KB stage at a time, through a ring with the token rows of the same k: kernel 1
// multiplies every token of the call (those that are not the expert's cost
// columns that the product has anyway), kernel 2 the expert's entries.  128 rows
// are the tensor cores' tallest product and need the fewest of them, four for 16
// KB; units of 32 or 64 rows would share out more evenly, but one warp issues
// twice and four times the products and falls behind HBM.  The SMs that get a
// unit less leave their bandwidth to the others.
//
// What this design is for (7168 x 2048, top 8, one token / 4096 x 1024, 64 slots,
// 32 experts): weights loaded straight into the registers of mma.sync drain at
// every unit's end (153 / 218 us); staged in shared memory and multiplied with
// mma.sync, the warps' loads of the token rows wait behind the ring's copies, and
// with those staged too the eight warps take longer over a stage than HBM does
// (139 / 224 us).  This one takes 128 / 154 us, 5.5 and 5.2 TB/s of weights.
//
// Which tokens an expert has is worked out by every CTA from the token's
// choices: a 64-bit token mask per expert, and a running count over the
// experts.  Entry (e, t), the count's value plus the rank of t in e's mask,
// numbers the rows of the intermediate buffers.  A choice that names an expert
// twice is one entry with the sum of the weights: the layer is linear in them.
//
// Kernel 1 leaves an entry's activations as two bf16 rows, the rounding and its
// remainder; they are two columns of kernel 2's product, added in its epilogue.
// Kernel 2 leaves one fp32 row per entry; the CTA that completes the last expert
// of a group of 128 columns (a counter per group) adds each token's rows in the
// order of its choices.  No sum depends on which CTA ran when.  Kernel 2 may
// start before kernel 1 has ended: its weights do not wait for the activations.

#include "situ_host.cuh"

namespace {

#include "situ_fused_gemm.cuh"

constexpr int kMoeThreads = 192;  // copies, products, four warps of epilogue
constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopk = 16;
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxEntries = kMoeMaxTokens * kMoeMaxTopk;
constexpr int64_t kMoeMaxDim = 32768;
constexpr int kMoeChunk = 64;                        // k elements of a 128-byte swizzle row
constexpr int kMoeRows = 128;                        // weight rows of a unit
constexpr int kMoeChunks = 2;                        // of a stage
constexpr int kMoeTileBytes = kMoeRows * kMoeChunk * 2;           // one chunk's weights
constexpr int kMoeWeightBytes = kMoeChunks * kMoeTileBytes;       // of a stage
constexpr int kMoeTile = 16;                         // entries of one box of kernel 2 (32 columns)
constexpr int kMoeMaxStages = 8;
constexpr int kMoeTmemCols = 512;                    // two sets of accumulators, 256 columns each
constexpr int kMoeSmem = 227 * 1024;

struct MoeArgs {
  const int64_t* ids;
  int64_t ids_stride;        // elements
  const void* weights;       // NULL: 1
  int64_t weights_stride;    // elements
  int weights_bf16;
  char* y;
  int64_t y_pitch;           // bytes
  __nv_bfloat16* act;        // [entries][2][inter]: the rounded activations, then the remainders
  float* part;               // [entries][hidden]
  int* done;                 // [column groups] experts completed
  int tokens, topk, experts, hidden, inter;
  Coeffs c;
};

// The call's routing, in shared memory.
struct MoePlan {
  unsigned long long mask[kMoeMaxExperts];  // tokens of each expert
  float weight[kMoeMaxEntries];             // of each entry
  uint16_t start[kMoeMaxExperts + 1];       // first entry of each expert
  uint16_t active[kMoeMaxEntries];          // experts that have a token, rising
  int16_t id[kMoeMaxEntries];               // [token][choice] its expert, then its entry; -1: none or named before
  int complete[128];                        // kernel 2: column groups whose experts are all done
  int warp_active[kMoeThreads / 32], warp_entries[kMoeThreads / 32];
  int n_active, most;                       // most: entries of the expert that has the most
  float up[2][16][64];                      // kernel 1: the up halves of 16 tokens, for the gate halves' warps
};

__device__ __forceinline__ int64_t moe_id(const MoeArgs& a, int t, int j) {
  const int64_t id = a.ids[t * a.ids_stride + j];
  return id >= 0 && id < a.experts ? id : -1;
}

__device__ __forceinline__ void moe_plan(const MoeArgs& a, MoePlan& p) {
  const int n = a.tokens * a.topk;
  for (int e = threadIdx.x; e < a.experts; e += kMoeThreads) p.mask[e] = 0;
  if (threadIdx.x == 0) p.most = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kMoeThreads) {
    const int t = i / a.topk, j = i - t * a.topk;
    const int64_t id = moe_id(a, t, j);
    bool first = id >= 0;
    for (int k = 0; k < j; ++k) first = first && moe_id(a, t, k) != id;
    p.id[i] = static_cast<int16_t>(first ? id : -1);
    if (first) atomicOr(&p.mask[id], 1ull << t);
  }
  __syncthreads();
  // running counts over the experts: each thread a run of them, then the warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (a.experts + kMoeThreads - 1) / kMoeThreads;
  const int e0 = min(a.experts, static_cast<int>(threadIdx.x) * per), e1 = min(a.experts, e0 + per);
  int act = 0, ent = 0, most = 0;
  for (int e = e0; e < e1; ++e) {
    const int c = __popcll(p.mask[e]);
    act += c > 0;
    ent += c;
    most = max(most, c);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMax(&p.most, most);
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
  if (threadIdx.x == kMoeThreads - 1) {
    p.n_active = run_a;
    p.start[a.experts] = static_cast<uint16_t>(run_e);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kMoeThreads) {
    const int id = p.id[i];
    if (id < 0) continue;
    const int t = i / a.topk;
    const int entry = p.start[id] + __popcll(p.mask[id] & ((1ull << t) - 1));
    p.id[i] = static_cast<int16_t>(entry);
    float w = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
      if (moe_id(a, t, j) != id) continue;
      const int64_t at = t * a.weights_stride + j;
      w += a.weights == nullptr  ? 1.0f
           : a.weights_bf16 != 0 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.weights)[at])
                                 : static_cast<const float*>(a.weights)[at];
    }
    p.weight[entry] = w;
  }
  __syncthreads();
}

// v as the sum of two bf16 numbers, `apart` elements from each other: 16 bits of
// its significand (an infinite rounding has no remainder).
__device__ __forceinline__ void put_split(__nv_bfloat16* out, int apart, float v) {
  const __nv_bfloat16 hi = __float2bfloat16(v);
  const float rest = v - __bfloat162float(hi);
  out[0] = hi;
  out[apart] = __float2bfloat16(isfinite(rest) ? rest : 0.0f);
}

// The two columns' products as one.  The values' column alone says what an infinite or
// NaN weight gives: times a remainder, which may be 0 or of the other sign, it says
// something else.
__device__ __forceinline__ float join_split(float value, float rest) { return isfinite(value) ? value + rest : value; }

// A box of rows of k elements [k0, ...): [chunk of 64 elements][row][128 bytes],
// the 16-byte pieces of a row swizzled by the row.
__device__ __forceinline__ void moe_box(uint32_t dst, const CUtensorMap* map, int32_t row, int32_t chunk, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(smem_u32(bar))
      : "memory");
}

// D[128 x n] (+)= A[128 x 16] B[n x 16]^T, bf16 in, fp32 out.  Operands by their
// shared-memory descriptors: one is 16 bytes further on for every 1 added to it.
// The whole warp comes here, one lane (`lead`) issues: operands that are the same
// for the warp stay in uniform registers, where the instruction wants them.
// (Descriptors computed anew for every product: 70 to 270 cycles each, 152 / 187
// us for the calls above.)
__device__ __forceinline__ void moe_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                        uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t moe_idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// A unit's k is spread over accumulators of a set, stage by stage: the tensor cores cut
// off what does not fit into an fp32 accumulator instead of rounding it, so that every
// addition takes a little of the sum away (activations of 7168 x 2048 in the 2-norm:
// 1.23e-5 off with one accumulator of 448 additions, 2.7e-6 with eight).  One
// accumulator for each eight stages of 64 additions, as far as the set's columns go
// (more would cost: 3 tokens of 1024 x 512 16.5 us with one each way, 16.9 with
// eight).  Columns from one accumulator to the next:
constexpr int kMoeSet = kMoeTmemCols / 2;
__device__ __forceinline__ int moe_apart(int columns, int steps) {
  const int room = columns <= 32 ? 32 : columns <= 64 ? 64 : 128;
  const int wish = steps <= 8 ? kMoeSet : steps <= 16 ? kMoeSet / 2 : steps <= 32 ? kMoeSet / 4 : kMoeSet / 8;
  return max(room, wish);
}
// 16 columns of the sum of the accumulators that a unit of `steps` stages has used.
__device__ __forceinline__ void moe_load16(uint32_t taddr, int apart, int steps, float (&sum)[16]) {
  uint32_t r[16];
  fc1::tmem_ld16(taddr, r);
  fc1::tmem_ld_wait(r);
#pragma unroll
  for (int j = 0; j < 16; ++j) sum[j] = __uint_as_float(r[j]);
#pragma unroll 1
  for (int at = apart; at < min(kMoeSet, steps * apart); at += apart) {
    fc1::tmem_ld16(taddr + at, r);
    fc1::tmem_ld_wait(r);
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[j] += __uint_as_float(r[j]);
  }
}

// First unit of CTA i of `grid` when `units` are shared out in runs.
__device__ __forceinline__ int moe_first(int units, int i, int grid) {
  return static_cast<int>(static_cast<int64_t>(units) * i / grid);
}

// The ring, before barriers and plan (whose last member kernel 2 does without).
__host__ __device__ constexpr int moe_ring(bool fc2) {
  const int tail = 256 + static_cast<int>(fc2 ? offsetof(MoePlan, up) : sizeof(MoePlan));
  return kMoeSmem - 1024 - (tail + 1023) / 1024 * 1024;
}

// Columns of kernel 1's product: the call's tokens; of kernel 2's largest: two per
// entry of the expert that has the most, which the plan knows.
__host__ __device__ constexpr int moe_columns(int entries, bool fc2) {
  return (entries + kMoeTile - 1) / kMoeTile * kMoeTile * (fc2 ? 2 : 1);
}
__host__ __device__ constexpr int moe_stage_bytes(int entries, bool fc2) {
  return kMoeWeightBytes + moe_columns(entries, fc2) * kMoeChunk * 2 * kMoeChunks;
}
__host__ __device__ constexpr int moe_stages(int entries, bool fc2) {
  const int s = moe_ring(fc2) / moe_stage_bytes(entries, fc2);
  return s < kMoeMaxStages ? s : kMoeMaxStages;
}
static_assert(moe_stages(kMoeMaxTokens, true) >= 3, "the ring is too short");

// Shared memory: the ring (1024-byte aligned), the barriers, the plan.
struct MoeSmem {
  uint32_t ring;
  uint64_t *full, *empty, *acc_full, *acc_empty, *drain;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  MoePlan* plan;
};
__device__ __forceinline__ MoeSmem moe_smem(unsigned char* raw, int ring_bytes) {
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  MoeSmem m;
  m.ring = smem_u32(base);
  m.full = reinterpret_cast<uint64_t*>(base + ring_bytes);
  m.empty = m.full + kMoeMaxStages;
  m.acc_full = m.empty + kMoeMaxStages;
  m.acc_empty = m.acc_full + 2;
  m.drain = m.acc_empty + 2;
  m.tmem_slot = reinterpret_cast<uint32_t*>(m.drain + 1);
  m.abort_flag = reinterpret_cast<volatile int*>(m.tmem_slot + 1);
  m.plan = reinterpret_cast<MoePlan*>(base + ring_bytes + 256);
  return m;
}

// Columns col .. col + 3 of y: warp q's tokens q, q + 4, ..., TOKENS of them and 16
// of their rows at a time, so that as many loads are in flight.  The CTA that completes
// a group of columns is among the last to end, and all the others wait for it (4096 x
// 1024, 64 slots, top 4 of 32: 171 us with the loads of one token in flight, 154 us
// with eight tokens'; for one token eight would be mostly idle work, 125 and 129 us).
template <int TOKENS>
__device__ __forceinline__ void moe_sum(const MoeArgs& a, const MoePlan& plan, int col, int q) {
  constexpr int kUnroll = 16 / TOKENS;
  for (int t0 = q; t0 < a.tokens; t0 += 4 * TOKENS) {
    float4 s[TOKENS];
#pragma unroll
    for (int n = 0; n < TOKENS; ++n) s[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll kUnroll
    for (int j = 0; j < a.topk; ++j) {
#pragma unroll
      for (int n = 0; n < TOKENS; ++n) {
        const int t = t0 + 4 * n, entry = t < a.tokens ? plan.id[t * a.topk + j] : -1;
        const float4 p =
            __ldcg(reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(entry >= 0 ? entry : 0) * a.hidden + col));
        if (entry >= 0) s[n].x += p.x, s[n].y += p.y, s[n].z += p.z, s[n].w += p.w;
      }
    }
#pragma unroll
    for (int n = 0; n < TOKENS; ++n)
      if (t0 + 4 * n < a.tokens)
        *reinterpret_cast<uint2*>(a.y + (t0 + 4 * n) * a.y_pitch + col * 2) =
            make_uint2(Bf16::pack(make_float2(s[n].x, s[n].y)), Bf16::pack(make_float2(s[n].z, s[n].w)));
  }
}

// Both kernels: FC2 false is W1 with the activation, true W2 with the sums.
template <bool FC2, int GATE, bool HAS_LB>
__global__ void __launch_bounds__(kMoeThreads, 1)
    situ_moe_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_b,
                    const MoeArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const MoeSmem m = moe_smem(smem_raw, moe_ring(FC2));
  const MoePlan& plan = *m.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (!FC2) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * kMoeThreads + threadIdx.x; i * kMoeRows < a.hidden; i += gridDim.x * kMoeThreads) a.done[i] = 0;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMoeMaxStages; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&m.acc_full[b], 1);
      mbar_init(&m.acc_empty[b], 128);
    }
    mbar_init(m.drain, 1);
    *m.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(m.tmem_slot)),
                 "r"(kMoeTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fc1::tc_fence_before();
  moe_plan(a, *m.plan);
  fc1::tc_fence_after();
  const uint32_t tmem = *m.tmem_slot;
  const int widest = FC2 ? plan.most : a.tokens;
  const int stages = moe_stages(widest, FC2), stage_bytes = moe_stage_bytes(widest, FC2);

  // Kernel 1: expert by expert.  Kernel 2: column group by column group, every expert.
  const int n_active = plan.n_active, k = FC2 ? a.inter : a.hidden;
  const int blocks = FC2 ? (a.hidden + kMoeRows - 1) / kMoeRows : a.inter / (kMoeRows / 2), units = n_active * blocks;
  const int u0 = moe_first(units, blockIdx.x, gridDim.x), u1 = moe_first(units, blockIdx.x + 1, gridDim.x);
  const int steps = (k + kMoeChunks * kMoeChunk - 1) / (kMoeChunks * kMoeChunk);  // stages of a unit
  struct Unit {
    int expert, block, row;   // row: the first of its weight rows
    int start, count, tiles;  // the expert's entries, and the products of kernel 2 they take
    int b_bytes;              // of a stage's columns
  };
  constexpr int tile_bytes = 2 * kMoeTile * kMoeChunk * 2 * kMoeChunks;  // columns of 16 entries
  auto unit = [&](int u) -> Unit {
    Unit v;
    v.block = FC2 ? u / n_active : u % blocks;
    v.expert = plan.active[FC2 ? u - v.block * n_active : u / blocks];
    v.row = FC2 ? v.expert * a.hidden + v.block * kMoeRows : v.expert * 2 * a.inter + v.block * (kMoeRows / 2);
    v.start = plan.start[v.expert];
    v.count = plan.start[v.expert + 1] - v.start;
    v.tiles = (v.count + kMoeTile - 1) / kMoeTile;
    v.b_bytes = FC2 ? v.tiles * tile_bytes : stage_bytes - kMoeWeightBytes;
    return v;
  };

  if (warp == 0) {
    // ---- copies ----
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    // one stage of a unit: its weights (with the announcement of all the bytes), then its columns
    auto weights = [&](const Unit& v, int step, int st) {
      const uint32_t at = m.ring + st * stage_bytes;
      mbar_arrive_expect_tx(&m.full[st], kMoeWeightBytes + v.b_bytes);
      if constexpr (FC2) {
        moe_box(at, &tmap_w, v.row, step * kMoeChunks, &m.full[st]);
      } else {  // a chunk's gate rows, then its up rows
#pragma unroll
        for (int c = 0; c < kMoeChunks; ++c) {
          moe_box(at + c * kMoeTileBytes, &tmap_w, v.row, step * kMoeChunks + c, &m.full[st]);
          moe_box(at + c * kMoeTileBytes + kMoeTileBytes / 2, &tmap_w, v.row + a.inter, step * kMoeChunks + c, &m.full[st]);
        }
      }
    };
    auto columns = [&](const Unit& v, int step, int st) {
      const uint32_t at = m.ring + st * stage_bytes + kMoeWeightBytes;
      if constexpr (FC2) {
        for (int c = 0; c < kMoeChunks; ++c)  // a chunk's columns of all the expert's entries side by side
          for (int i = 0; i < v.tiles; ++i)
            moe_box(at + (c * v.tiles + i) * (tile_bytes / kMoeChunks), &tmap_b, 2 * (v.start + i * kMoeTile),
                    step * kMoeChunks + c, &m.full[st]);
      } else {
        moe_box(at, &tmap_b, 0, step * kMoeChunks, &m.full[st]);
      }
    };
    int u = u0, step = 0;  // the next stage to send
    if constexpr (FC2) {  // the first stages' weights are sent before kernel 1's end
      const int early = min(stages, (u1 - u0) * steps);
      if (lane == 0) {
        Unit v{};
        for (int i = 0, x = u0, y = 0; i < early; ++i) {
          if (y == 0) v = unit(x);
          weights(v, y, i);
          if (++y == steps) y = 0, ++x;
        }
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");  // kernel 1's activations
      asm volatile("fence.proxy.async;" ::: "memory");
      Unit v{};
      for (int i = 0; i < early; ++i) {
        if (step == 0) v = unit(u);
        if (lane == 0) columns(v, step, i);
        if (++step == steps) step = 0, ++u;
      }
      __syncwarp();
      issued = (1u << early) - 1;
      stage = early % stages;
      phase = early == stages ? 1u : 0u;
    }
    bool ok = true;
    for (; ok && u < u1; ++u, step = 0) {
      const Unit v = unit(u);
      for (; step < steps; ++step) {
        if (!fc1::wait_or_abort(&m.empty[stage], phase ^ 1u, m.abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          weights(v, step, stage);
          columns(v, step, stage);
        }
        __syncwarp();
        issued |= 1u << stage;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok)  // aborted: let the copies this warp issued land (bounded) before the CTA exits
      for (int s = 0; s < stages; ++s)
        if (issued & (1u << s)) mbar_wait(&m.full[s], s < stage ? phase : phase ^ 1u);
  } else if (warp == 1) {
    // ---- products ----
    int stage = 0, it = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int u = u0; ok && u < u1; ++u, ++it) {
      const int b = it & 1;
      if (!fc1::wait_or_abort(&m.acc_empty[b], ((acc_phase >> b) & 1u) ^ 1u, m.abort_flag)) {
        ok = false;
        break;
      }
      fc1::tc_fence_after();
      const uint32_t d0 = tmem + static_cast<uint32_t>(b * kMoeSet);
      const int n_cols = FC2 ? unit(u).tiles * 2 * kMoeTile : moe_columns(a.tokens, false);
      const uint32_t idesc = moe_idesc(n_cols);
      const uint64_t t_chunk = n_cols * (kMoeChunk * 2 / 16);
      const int apart = moe_apart(n_cols, steps);
      int at_col = 0;            // of the stage's accumulator in the set
      uint32_t accumulate = 0;   // once every accumulator has had a stage
      for (int step = 0; step < steps; ++step) {
        if (!fc1::wait_or_abort(&m.full[stage], phase, m.abort_flag)) {
          ok = false;
          break;
        }
        fc1::tc_fence_after();
        const uint32_t d = d0 + static_cast<uint32_t>(at_col);
        const uint32_t at = m.ring + stage * stage_bytes;
        const uint64_t w = fc1::smem_desc_sw128(at);
        const uint64_t t = fc1::smem_desc_sw128(at + kMoeWeightBytes);
#pragma unroll
        for (int c = 0; c < kMoeChunks; ++c)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            moe_mma(d, w + (c * kMoeTileBytes + s * 32) / 16, t + c * t_chunk + s * 2, idesc,
                    (c | s) != 0 ? 1u : accumulate, lane == 0);
        if ((at_col += apart) == kMoeSet) {
          at_col = 0;
          accumulate = 1;
        }
        if (lane == 0) fc1::umma_commit(&m.empty[stage]);
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) fc1::umma_commit(&m.acc_full[b]);
      __syncwarp();
      acc_phase ^= 1u << b;
    }
    if (!ok || *m.abort_flag) {
      // Aborted: wait (bounded) for this warp's products before TMEM is freed.
      if (lane == 0) fc1::umma_commit(m.drain);
      __syncwarp();
      mbar_wait(m.drain, 0);
    }
  } else {
    // ---- epilogue: one accumulator row per thread ----
    const int q = warp & 3, row = q * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if constexpr (FC2) asm volatile("griddepcontrol.wait;" ::: "memory");  // kernel 1's counters
    uint32_t acc_phase = 0;
    int it = 0, turn = 0;
    bool ok = true;  // false: a wait gave up; the barriers below are still met
    for (int u = u0; u < u1; ++u, ++it) {
      const int b = it & 1;
      const Unit v = unit(u);
      if (ok && !fc1::wait_or_abort(&m.acc_full[b], (acc_phase >> b) & 1u, m.abort_flag)) ok = false;
      __syncwarp();
      fc1::tc_fence_after();
      const uint32_t taddr = lanes + static_cast<uint32_t>(b * kMoeSet);
      const int apart = moe_apart(FC2 ? v.tiles * 2 * kMoeTile : moe_columns(a.tokens, false), steps);
      if constexpr (FC2) {
        float* out = a.part + static_cast<int64_t>(v.start) * a.hidden + v.block * kMoeRows + row;
        const bool in = v.block * kMoeRows + row < a.hidden;
#pragma unroll 1
        for (int i = 0; i < v.count; i += 8) {  // eight entries, the value's and the remainder's columns
          float r[16];
          moe_load16(taddr + 2 * i, apart, steps, r);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (in && i + j < v.count)
              out[static_cast<int64_t>(i + j) * a.hidden] = join_split(r[2 * j], r[2 * j + 1]);
          __syncwarp();
        }
      } else {
        // rows 0 .. 63 are the gate halves, 64 .. 127 the up halves of the same columns
        const unsigned long long mask = plan.mask[v.expert];
        __nv_bfloat16* out = a.act + static_cast<int64_t>(v.start) * 2 * a.inter + v.block * (kMoeRows / 2) + (row & 63);
        int entry = 0;
#pragma unroll 1
        for (int t = 0; t < a.tokens; t += 16) {
          const uint32_t some = static_cast<uint32_t>(mask >> t) & 0xffffu;
          if (some == 0) continue;
          float r[16];
          moe_load16(taddr + t, apart, steps, r);
          float(&up)[16][64] = m.plan->up[turn & 1];
          ++turn;
          if (q >= 2) {
#pragma unroll
            for (int j = 0; j < 16; ++j) up[j][row & 63] = r[j];
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (q < 2) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {  // two tokens at a time, the expert's among them stored
              const uint32_t two = (some >> j) & 3u;
              if (two == 0) continue;
              const float2 w = make_float2(two & 1u ? plan.weight[v.start + entry] : 0.0f,
                                           two & 2u ? plan.weight[v.start + entry + (two & 1u)] : 0.0f);
              const float2 y =
                  fwd_pair_abs<GATE, HAS_LB, F32>({__float_as_uint(r[j]), __float_as_uint(r[j + 1])}, {__float_as_uint(up[j][row]), __float_as_uint(up[j + 1][row])},
                                                  mul2(w, splat(a.c.bb)), a.c);
              __nv_bfloat16* o = out + static_cast<int64_t>(entry) * 2 * a.inter;
              if (two & 1u) put_split(o, a.inter, y.x);
              if (two & 2u) put_split(o + (two & 1u) * 2 * a.inter, a.inter, y.y);
              entry += __popc(two);
            }
          }
          __syncwarp();
        }
      }
      fc1::tc_fence_before();
      mbar_arrive(&m.acc_empty[b]);
      acc_phase ^= 1u << b;
    }
    if constexpr (FC2) {
      const int thread = threadIdx.x - 64;
      if (n_active == 0) {  // no token has an expert
        for (int64_t i = blockIdx.x * 128 + thread; i < static_cast<int64_t>(a.tokens) * a.hidden; i += gridDim.x * 128)
          *reinterpret_cast<__nv_bfloat16*>(a.y + i / a.hidden * a.y_pitch + i % a.hidden * 2) = __float2bfloat16(0.0f);
      } else if (u0 < u1) {
        // Count this CTA's experts of each of its column groups; where they were the
        // last, the group's rows are complete and each token's are added here.
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int b0 = u0 / n_active, groups = (u1 - 1) / n_active - b0 + 1;
        for (int base = 0; base < groups; base += 128) {
          const int some = min(128, groups - base);
          if (thread < some) {
            const int b = b0 + base + thread;
            const int mine = min(u1, (b + 1) * n_active) - max(u0, b * n_active);
            m.plan->complete[thread] = mine == n_active || atomicAdd(&a.done[b], mine) + mine == n_active;
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
          __threadfence();
          for (int gi = 0; gi < some; ++gi) {
            const int col = (b0 + base + gi) * kMoeRows + (thread & 31) * 4;
            if (!plan.complete[gi] || col >= a.hidden) continue;
            if (a.tokens > 16)
              moe_sum<8>(a, plan, col, thread >> 5);
            else
              moe_sum<2>(a, plan, col, thread >> 5);
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
        }
      }
    }
  }

  fc1::tc_fence_before();
  __syncthreads();
  fc1::tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kMoeTmemCols) : "memory");
}

// ---- host ---------------------------------------------------------------------

struct MoeWorkspace {
  size_t act, part, done;  // bytes of each part, multiples of 256
};
MoeWorkspace moe_workspace(int64_t tokens, int64_t topk, int64_t hidden, int64_t inter) {
  auto up = [](int64_t b) { return static_cast<size_t>((b + 255) / 256 * 256); };
  return {up(tokens * topk * inter * 4), up(tokens * topk * hidden * 4), up((hidden + kMoeRows - 1) / kMoeRows * 4)};
}

// [rows, k] bf16 as [k / 64][rows][64], boxes of `box_chunks` x `box_rows` x 64
// elements with the 128-byte swizzle.
situ_status_t moe_map(CUtensorMap* m, const void* base, int64_t rows, int64_t k, int64_t pitch_elems, int box_rows,
                      int box_chunks) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return fail(SITU_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {kMoeChunk, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(k / kMoeChunk)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch_elems) * 2, kMoeChunk * 2};
  const cuuint32_t box[3] = {kMoeChunk, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_chunks)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SITU_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return SITU_OK;
}

using MoeKernel = void (*)(const CUtensorMap, const CUtensorMap, const MoeArgs);
template <bool LB>
MoeKernel pick_moe_fc1(int gate) {
  switch (gate) {
    case kGateSquare: return situ_moe_kernel<false, kGateSquare, LB>;
    case kGateEqual: return situ_moe_kernel<false, kGateEqual, LB>;
    case kGateRoot: return situ_moe_kernel<false, kGateRoot, LB>;
    default: return situ_moe_kernel<false, kGateGeneric, LB>;
  }
}

struct MoeCall {
  const void *x, *w1, *w2;
  int64_t x_stride, w1_stride, w2_stride, experts;
  bool lb;
  int gate;
};

situ_status_t launch_moe(const MoeArgs& a, const MoeCall& c, cudaStream_t s) {
  CUtensorMap mw1, mx, mw2, ma;
  situ_status_t st = moe_map(&mw1, c.w1, c.experts * 2 * a.inter, a.hidden, c.w1_stride, kMoeRows / 2, 1);
  if (st != SITU_OK) return st;
  st = moe_map(&mx, c.x, a.tokens, a.hidden, c.x_stride, moe_columns(a.tokens, false), kMoeChunks);
  if (st != SITU_OK) return st;
  st = moe_map(&mw2, c.w2, c.experts * a.hidden, a.inter, c.w2_stride, kMoeRows, kMoeChunks);
  if (st != SITU_OK) return st;
  st = moe_map(&ma, a.act, static_cast<int64_t>(a.tokens) * a.topk * 2, a.inter, a.inter, 2 * kMoeTile, 1);
  if (st != SITU_OK) return st;
  const MoeKernel k1 = c.lb ? pick_moe_fc1<true>(c.gate) : pick_moe_fc1<false>(c.gate);
  const MoeKernel k2 = situ_moe_kernel<true, kGateGeneric, false>;
  const int64_t most = c.experts < static_cast<int64_t>(a.tokens) * a.topk ? c.experts : a.tokens * a.topk;
  int grid = 0;
  st = ensure_smem(reinterpret_cast<const void*>(k1), kMoeSmem);
  if (st != SITU_OK) return st;
  st = ensure_smem(reinterpret_cast<const void*>(k2), kMoeSmem);
  if (st != SITU_OK) return st;
  st = launch_grid(reinterpret_cast<const void*>(k1), kMoeThreads, kMoeSmem, most * (a.inter / (kMoeRows / 2)), &grid);
  if (st != SITU_OK) return st;
  k1<<<grid, kMoeThreads, kMoeSmem, s>>>(mw1, mx, a);
  st = check_launch("situ_glu_moe_fwd (FC1)");
  if (st != SITU_OK) return st;
  st = launch_grid(reinterpret_cast<const void*>(k2), kMoeThreads, kMoeSmem, most * ((a.hidden + kMoeRows - 1) / kMoeRows), &grid);
  if (st != SITU_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, k2, mw2, ma, a);
  if (err != cudaSuccess) return fail(SITU_ERR_CUDA, "situ_glu_moe_fwd (FC2) launch: %s", cudaGetErrorString(err));
  return check_launch("situ_glu_moe_fwd (FC2)");
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
  if (experts * 2 * inter > INT32_MAX || experts * hidden > INT32_MAX)
    return fail(SITU_ERR_UNSUPPORTED, "sizes exceed the 32-bit tensor-map coordinates");
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
  a.ids = topk_ids;
  a.ids_stride = topk_ids_row_stride;
  a.weights = topk_weights;
  a.weights_stride = topk_weights_row_stride;
  a.weights_bf16 = topk_weights != nullptr && weights_dtype == SITU_DTYPE_BF16;
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
  const MoeCall c = {x, w1, w2, x_row_stride, w1_row_stride, w2_row_stride, experts, has_linear_beta != 0, gate};
  return launch_moe(a, c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
