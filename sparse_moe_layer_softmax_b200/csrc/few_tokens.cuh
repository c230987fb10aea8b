// The whole MoE layer for a few tokens (1 .. kFewTokens) in one persistent cooperative kernel.
//
// The layer is the one of "Muse Spark Open: Norm-Preserving Gates Are Not a Norm Guarantee"
// (sections "Latent experts" and "Residual gates") and, without latent projections, of "816 billion
// parameters, and only 42 billion show up for each token" ("The math"), optionally with a low-rank
// adapter per token beside the two latent projections:
//   l = u W_g^T, top-k;  z = C_pre(P_down u + s B A u);  a = SiLU(W_gate z) * (W_up z);  o = W_d a;
//   y = sum_j w_j I_gamma(o_j);  b = P_up y + s B' A' y;  out = alpha r + beta b.
//
// What bounds it: at this size the layer is a stream of weights, each read once (944 MB for one
// token of the Muse layer, about 5.9 GB for eight), with one multiply-add per weight and token.
// So everything is arranged around that stream never pausing:
//   - One CTA per SM.  A producer warp walks this CTA's weight tiles of every stage of the layer in
//     order and copies them into one shared-memory ring with bulk copies; it never waits for the
//     arithmetic of a stage, only for ring slots and, once, for the routing.  While the CTAs wait
//     for one another between stages, the ring fills with the next stage's weights.
//   - A tile is 16 weight rows; eight consumer warps split its reduction, each accumulating with
//     m16n8k16 tensor-core products: 16 weight rows on M and the tokens on N = 8.  The stream asks for
//     one such instruction per SM about every 12 clocks, far below what the warp-level tensor path
//     delivers, and operands come straight from the ring without staging accumulators in TMEM.
//     The reduction index is permuted the same way in both operands, so that every fragment is a
//     16-byte shared-memory load.
//   - For SwiGLU a tile holds 8 gate rows and the same 8 features' up rows, which meet in one thread.
//   - Stages are separated by grid barriers (arrive early, wait late) on counters in the workspace.
//
// Precision: every intermediate (z, a, o, y, b) stays in fp32, and enters the tensor cores as a pair
// of bf16 values hi + lo (16 bits of mantissa); only the layer output is rounded to bf16.  (With
// input_norm the branch input u is rounded to bf16, as in the batch path, since the router's selection
// depends on it.)  The second product costs tensor-core time that the stream leaves idle.
#pragma once

#include "common.cuh"
#include "kernels_simt.cuh"

namespace moe {

constexpr int kFewTokens = 8;                  // tokens on the MMA's N side
constexpr int kFewSlots = kFewTokens * kMaxTopK;
constexpr int kFewWarps = 8;                   // consumer warps
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewRows = 16;                   // weight rows per tile
constexpr int kFewRowBytes = 1024;             // bytes of each row in one ring stage
// Rows lie 64 bytes (mod 128) apart, so the eight 16-byte loads of a quarter-warp phase (two rows,
// four 16-byte columns) fall into distinct banks.
constexpr int kFewRowPitch = kFewRowBytes + 64;
constexpr int kFewStageBytes = kFewRows * kFewRowPitch;
constexpr int kFewMaxStages = 12;
constexpr int kFewMaxRank = 128;
constexpr int kFewRedPitch = 10;               // floats per row of a partial tile (no bank conflicts)
constexpr int kFewRedFloats = kFewWarps * kFewRows * kFewRedPitch;
constexpr int kFewBarriers = 8;                // grid-barrier counters, 64 bytes apart

struct FewParams {
  int T, d, L, E, H, n, k;      // E: expert width (L, or d without latent projections)
  int swiglu, pre_norm, expert_norm, resid_mode, gate_mode, input_norm, post_norm;
  int wk_seg;                   // segments of length d in a router row (3: split fp32 weights)
  float eps, eps_block, tau, floor_, routed_scale, logit_mult;
  const void *u, *r;
  const void *w_router, *p_down, *p_up, *w_gu, *w_down;
  const float *gamma_pre, *gamma_expert, *resid_g, *logit_bias, *sel_bias, *gamma_in, *gamma_post;
  // adapters (nA == 0: none)
  int nA, rank;
  const uint16_t *down_a, *down_b, *up_a, *up_b;
  const float* scale;
  const int32_t* token_adapter;
  // outputs
  void* out;
  float* logits_out;            // optional
  int32_t* idx_out;             // optional
  float* w_out;                 // optional
  // workspace
  unsigned* bar;                // [kFewBarriers * 16], zeroed before the launch
  float* logits;                // [T, n] pre-activation
  float* z;                     // [T, L]
  float* a;                     // [T*k, H]
  float* s;                     // [T*k, E] scaled expert outputs (1 + gamma) o
  float* ss;                    // [T*k, E/16] partial sums of squares of s
  float* y;                     // [T, E]
  float* v_down;                // [T, rank]
  float* v_up;                  // [T, rank]
  float* b;                     // [T, d] (post_norm)
  float* bss;                   // [T, d/16] (post_norm)
  int stages;                   // ring stages
  int act_bytes;                // activation region of shared memory
};

// Routing tables every CTA keeps in shared memory.
struct FewTables {
  int idx[kFewSlots];
  float w[kFewSlots];
  int dist;                            // distinct selected experts
  int expert[kFewSlots];               // ascending
  int count[kFewSlots];                // slots routed to that expert (at most T)
  uint8_t slot[kFewSlots][kFewTokens]; // those slots, in token order
  int own[256];
  // adapters: the distinct ones the tokens use, and each token's (-1: none)
  int ndist_ad;
  int ad[kFewTokens];
  int tok_ad[kFewTokens];
  float inv[kMaxTopK];
  float red[kFewWarps][kFewTokens];
  float norm[kFewTokens];
  int abort_;
};

enum FewPhase : int { FEW_IN = 0, FEW_UP1 = 1, FEW_DOWN2 = 2, FEW_OUT = 3 };

// One 16-row weight tile: row i < split starts at base + i * ld, row i >= split at
// base2 + (i - split) * ld (elements); rows past `valid` repeat the last valid row.
struct FewTile {
  const char* base;
  const char* base2;
  long ld_bytes;
  int split, valid;
  int seg_len, segs;   // reduction: segs segments of seg_len, each against activation columns 0..
  int kind;            // what the epilogue does
  int r0;              // first row (feature, expert or rank index) of the tile
  int e;               // index into the distinct experts / adapters
};
enum FewKind : int { FEW_ROUTER, FEW_AD_DOWN, FEW_LATENT, FEW_GATEUP, FEW_EXPERT_OUT, FEW_AD_UP,
                     FEW_LAYER_OUT };

template <bool kF32>
struct FewTiles {
  const FewParams& p;
  const FewTables& tb;
  static constexpr int kEs = kF32 ? 4 : 2;

  __device__ int per_expert(int phase) const {
    return phase == FEW_UP1 ? (p.swiglu ? p.H / 8 : p.H / 16) : p.E / 16;
  }
  __device__ int ad_tiles() const { return p.nA ? (p.rank + 15) / 16 : 0; }
  __device__ int lead_tiles(int phase) const {  // tiles other CTAs wait for before the phase's others
    return (phase == FEW_IN ? (p.n + 15) / 16 : 0) + tb.ndist_ad * ad_tiles();
  }
  __device__ int total(int phase) const {
    switch (phase) {
      case FEW_IN: return lead_tiles(phase) + p.L / 16;
      case FEW_UP1:
      case FEW_DOWN2: return tb.dist * per_expert(phase);
      default: return p.L ? lead_tiles(phase) + p.d / 16 : 0;
    }
  }
  // This CTA's tiles: contiguous runs of the expert stages (at most a few experts per CTA), strided
  // ones of the dense stages, so that their leading tiles start at once on as many CTAs.
  __device__ void range(int phase, int& i, int& end, int& step) const {
    const int N = total(phase);
    if (phase == FEW_UP1 || phase == FEW_DOWN2) {
      i = static_cast<int>(static_cast<long>(blockIdx.x) * N / gridDim.x);
      end = static_cast<int>(static_cast<long>(blockIdx.x + 1) * N / gridDim.x);
      step = 1;
    } else {
      i = static_cast<int>(blockIdx.x);
      end = N;
      step = static_cast<int>(gridDim.x);
    }
  }
  __device__ FewTile rows(const void* w, long row0, long ld, int valid) const {
    FewTile t;
    t.base = static_cast<const char*>(w) + row0 * ld * kEs;
    t.base2 = t.base;
    t.ld_bytes = ld * kEs;
    t.split = kFewRows;
    t.valid = min(valid, kFewRows);
    t.seg_len = static_cast<int>(ld);
    t.segs = 1;
    t.e = 0;
    return t;
  }
  __device__ FewTile get(int phase, int i) const {
    FewTile t;
    if (phase == FEW_IN) {
      const int nr = (p.n + 15) / 16, na = tb.ndist_ad * ad_tiles();
      if (i < nr) {
        t = rows(p.w_router, i * 16l, static_cast<long>(p.wk_seg) * p.d, p.n - i * 16);
        t.seg_len = p.d;
        t.segs = p.wk_seg;
        t.kind = FEW_ROUTER;
        t.r0 = i * 16;
      } else if (i < nr + na) {
        const int j = i - nr, q = j / ad_tiles(), r0 = (j - q * ad_tiles()) * 16;
        t = rows(p.down_a, static_cast<long>(tb.ad[q]) * p.rank + r0, p.d, p.rank - r0);
        t.kind = FEW_AD_DOWN;
        t.r0 = r0;
        t.e = q;
      } else {
        t.r0 = (i - nr - na) * 16;
        const int r0 = t.r0;
        t = rows(p.p_down, r0, p.d, 16);
        t.kind = FEW_LATENT;
        t.r0 = r0;
      }
    } else if (phase == FEW_UP1 || phase == FEW_DOWN2) {
      const int per = per_expert(phase), q = i / per, j = i - q * per;
      const long e = tb.expert[q];
      if (phase == FEW_DOWN2) {
        t = rows(p.w_down, e * p.E + j * 16, p.H, 16);
        t.kind = FEW_EXPERT_OUT;
        t.r0 = j * 16;
      } else if (p.swiglu) {
        t = rows(p.w_gu, e * 2 * p.H + j * 8, p.E, 16);
        t.base2 = t.base + static_cast<long>(p.H) * t.ld_bytes;
        t.split = 8;
        t.kind = FEW_GATEUP;
        t.r0 = j * 8;
      } else {
        t = rows(p.w_gu, e * p.H + j * 16, p.E, 16);
        t.kind = FEW_GATEUP;
        t.r0 = j * 16;
      }
      t.e = q;
    } else {
      const int na = tb.ndist_ad * ad_tiles();
      if (i < na) {
        const int q = i / ad_tiles(), r0 = (i - q * ad_tiles()) * 16;
        t = rows(p.up_a, static_cast<long>(tb.ad[q]) * p.rank + r0, p.L, p.rank - r0);
        t.kind = FEW_AD_UP;
        t.r0 = r0;
        t.e = q;
      } else {
        const int r0 = (i - na) * 16;
        t = rows(p.p_up, r0, p.L, 16);
        t.kind = FEW_LAYER_OUT;
        t.r0 = r0;
      }
    }
    return t;
  }
};

__device__ __forceinline__ void few_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
}

// Grid barrier b: every consumer thread calls arrive once (its earlier global writes are then
// published), and every consumer thread calls wait before it reads what other CTAs wrote.
__device__ __forceinline__ void few_arrive(unsigned* bar, int b) {
  few_bar();
  if (threadIdx.x == 0) {
    __threadfence();
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(bar + b * 16) : "memory");
  }
}
__device__ __forceinline__ void few_wait(unsigned* bar, int b, volatile int* abort_) {
  if (threadIdx.x == 0 && !*abort_) {
    const long long t0 = clock64();
    unsigned v;
    for (;;) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar + b * 16) : "memory");
      if (v >= gridDim.x) break;
      if (clock64() - t0 > kWaitBudgetClocks) {
        latch_status(MOE_ERR_TIMEOUT);
        *abort_ = 1;
        break;
      }
    }
    __threadfence();
  }
  few_bar();
}

__device__ __forceinline__ void few_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The activations a stage multiplies, in shared memory: rows of K values.  bf16 layers: one plane
// (exact bf16 inputs) or two (hi, lo); fp32 layers: fp32 rows.
struct FewAct {
  char* base;
  int pitch;      // bytes per row
  int plane;      // bytes from the hi to the lo plane, 0: no lo plane
};
template <bool kF32>
__device__ __forceinline__ FewAct few_act(char* base, int rows, int K, bool split) {
  FewAct a;
  a.base = base;
  a.pitch = kF32 ? K * 4 + 16 : K * 2 + 64;
  a.plane = (!kF32 && split) ? rows * a.pitch : 0;
  return a;
}
// Stores 4 fp32 values at columns c .. c+3 (c % 4 == 0) of a row.
template <bool kF32>
__device__ __forceinline__ void few_act_put4(const FewAct& a, int row, int c, float4 v) {
  char* at = a.base + row * a.pitch;
  if constexpr (kF32) {
    *reinterpret_cast<float4*>(at + c * 4) = v;
  } else {
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float h0 = round_bf16(f[2 * i]), h1 = round_bf16(f[2 * i + 1]);
      hi[i] = pack_bf16x2(h0, h1);
      // an infinite value has no remainder (inf - inf is NaN)
      lo[i] = pack_bf16x2(isinf(h0) ? 0.0f : f[2 * i] - h0, isinf(h1) ? 0.0f : f[2 * i + 1] - h1);
    }
    *reinterpret_cast<uint2*>(at + c * 2) = make_uint2(hi[0], hi[1]);
    if (a.plane) *reinterpret_cast<uint2*>(at + a.plane + c * 2) = make_uint2(lo[0], lo[1]);
  }
}

// One warp's share of a stage: 32-value blocks (fp32: 4-value blocks) warp, warp + 8, ... of the
// chunk's kw columns, added into acc (m16n8 fragment: rows lane/4 and lane/4 + 8, tokens
// 2 (lane%4) and + 1).  arow: this lane's activation row (token lane/4; fp32: unused) at the chunk's
// first column, nullptr for a column without a token.
__device__ __forceinline__ void few_chunk_bf16(const char* stage, int kw, const char* arow, int plane,
                                               int warp, int lane, float (&acc)[4]) {
  const int g = lane >> 2, t = lane & 3;
  const char* w0 = stage + g * kFewRowPitch + t * 16;
  float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
  for (int kb = warp; kb < kw / 32; kb += kFewWarps) {
    const uint4 x = *reinterpret_cast<const uint4*>(w0 + kb * 64);
    const uint4 y = *reinterpret_cast<const uint4*>(w0 + 8 * kFewRowPitch + kb * 64);
    uint4 h = zero;
    if (arow) h = *reinterpret_cast<const uint4*>(arow + kb * 64 + t * 16);
    few_mma(d, x.x, y.x, x.y, y.y, h.x, h.y);
    few_mma(d, x.z, y.z, x.w, y.w, h.z, h.w);
    if (plane) {
      uint4 l = zero;
      if (arow) l = *reinterpret_cast<const uint4*>(arow + plane + kb * 64 + t * 16);
      few_mma(d, x.x, y.x, x.y, y.y, l.x, l.y);
      few_mma(d, x.z, y.z, x.w, y.w, l.z, l.w);
    }
  }
  // The chunk's short sums are added in fp32 registers: the tensor core's own accumulation
  // truncates, which over a whole row would cost the router's logits a digit.
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += d[i];
}
__device__ __forceinline__ void few_chunk_f32(const char* stage, int kw, const char* x0,
                                              const char* x1, int warp, int lane, float (&acc)[4]) {
  const int g = lane >> 2;
  const char* w0 = stage + g * kFewRowPitch;
  const float4 zero = make_float4(0, 0, 0, 0);
  for (int kb = warp; kb < kw / 4; kb += kFewWarps) {
    const float4 wa = *reinterpret_cast<const float4*>(w0 + kb * 16);
    const float4 wb = *reinterpret_cast<const float4*>(w0 + 8 * kFewRowPitch + kb * 16);
    const float4 xa = x0 ? *reinterpret_cast<const float4*>(x0 + kb * 16) : zero;
    const float4 xb = x1 ? *reinterpret_cast<const float4*>(x1 + kb * 16) : zero;
    acc[0] = fmaf(wa.x, xa.x, fmaf(wa.y, xa.y, fmaf(wa.z, xa.z, fmaf(wa.w, xa.w, acc[0]))));
    acc[1] = fmaf(wa.x, xb.x, fmaf(wa.y, xb.y, fmaf(wa.z, xb.z, fmaf(wa.w, xb.w, acc[1]))));
    acc[2] = fmaf(wb.x, xa.x, fmaf(wb.y, xa.y, fmaf(wb.z, xa.z, fmaf(wb.w, xa.w, acc[2]))));
    acc[3] = fmaf(wb.x, xb.x, fmaf(wb.y, xb.y, fmaf(wb.z, xb.z, fmaf(wb.w, xb.w, acc[3]))));
  }
}

// Top-k of token t by one warp, into the tables (and CTA 0's copies to the caller's buffers); the
// rules are those of moe_route: descending keys, ties to the lower index, a NaN key below every
// other and latched.
__device__ __forceinline__ void few_topk(const FewParams& p, FewTables& tb, int t, int lane) {
  uint32_t key[kMaxExperts / 32];
  float pay[kMaxExperts / 32];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0u;
    pay[i] = 0.0f;
    if (e < p.n) {
      float l = __ldcg(&p.logits[static_cast<size_t>(t) * p.n + e]);
      float kf = l;
      if (p.gate_mode == MOE_GATE_SIGMOID) {
        l = 1.0f / (1.0f + expf(-l));
        kf = l + (p.sel_bias ? p.sel_bias[e] : 0.0f);
      }
      if (p.logits_out && blockIdx.x == 0) p.logits_out[static_cast<size_t>(t) * p.n + e] = l;
      pay[i] = l;
      if (kf != kf) {
        bad = true;
        kf = -INFINITY;
        pay[i] = p.gate_mode == MOE_GATE_SIGMOID ? 0.0f : -INFINITY;
      }
      key[i] = ordered_key(kf);
    }
  }
  float top_s[kMaxTopK];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    top_s[j] = 0.0f;
    if (j >= p.k) continue;
    uint32_t bk = 0u;
    int bi = 0x7fffffff;
    float bp = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i)
      if (key[i] > bk) { bk = key[i]; bi = lane + 32 * i; bp = pay[i]; }
    const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
    const uint32_t win =
        __reduce_min_sync(0xffffffffu, bk == m ? static_cast<uint32_t>(bi) : 0xffffffffu);
    top_s[j] = __shfl_sync(0xffffffffu, bp, static_cast<int>(win & 31u));
    // k <= n, and every candidate's key is above 0: some candidate is always left
    if (lane == 0) tb.idx[t * p.k + j] = min(static_cast<int>(win), p.n - 1);
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i)
      if (static_cast<uint32_t>(lane + 32 * i) == win) key[i] = 0u;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    if (blockIdx.x == 0 && (bad || !(fabsf(top_s[0]) <= 3.0e38f))) latch_status(MOE_ERR_DEVICE_CHECK);
    const bool sig = p.gate_mode == MOE_GATE_SIGMOID;
    float ex[kMaxTopK];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      ex[j] = j < p.k ? (sig ? top_s[j] : expf(top_s[j] - top_s[0])) : 0.0f;
      sum += ex[j];
    }
    const float denom = sig ? sum + 1e-15f : sum;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j)
      if (j < p.k) tb.w[t * p.k + j] = ex[j] / denom * p.routed_scale;
  }
}

// The layer.  Grid: one CTA per SM, cooperative (every CTA resident).
template <bool kF32>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const FewParams p) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  char* act_mem = reinterpret_cast<char*>(few_smem);
  char* ring = act_mem + p.act_bytes;
  float* red = reinterpret_cast<float*>(ring + p.stages * kFewStageBytes);
  float* s_v = red + 2 * kFewRedFloats;  // [T][rank] adapter inner products
  __shared__ FewTables tb;
  __shared__ __align__(8) uint64_t full[kFewMaxStages], empty[kFewMaxStages], routed;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = p.T, k = p.k;
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], kFewWarps); }
    mbar_init(&routed, 1);
    fence_barrier_init();
    tb.abort_ = 0;
    tb.dist = 0;
    tb.ndist_ad = 0;
  }
  if (tid < kFewTokens) {
    int a = p.nA && tid < T ? p.token_adapter[tid] : -1;
    if (a < -1 || a >= p.nA) {
      if (blockIdx.x == 0) latch_status(MOE_ERR_DEVICE_CHECK);
      a = -1;
    }
    tb.tok_ad[tid] = a;
  }
  __syncthreads();
  if (p.nA) {
    if (tid == 0) {
      for (int t = 0; t < T; ++t) {
        const int a = tb.tok_ad[t];
        bool seen = a < 0;
        for (int q = 0; q < tb.ndist_ad; ++q) seen = seen || tb.ad[q] == a;
        if (!seen) tb.ad[tb.ndist_ad++] = a;
      }
    }
    __syncthreads();
  }
  const FewTiles<kF32> tiles{p, tb};
  volatile int* abort_ = &tb.abort_;

  if (warp == kFewWarps) {
    // -------------------------------------------------------------- producer
    constexpr int kEs = kF32 ? 4 : 2;
    uint32_t stage = 0, phase_bit = 0, issued = 0, parities = 0;
    bool ok = true;
    for (int ph = FEW_IN; ph <= FEW_OUT && ok; ++ph) {
      if (ph == FEW_UP1) ok = mbar_wait(&routed, 0);
      if (!ok) break;
      int i, end, step;
      tiles.range(ph, i, end, step);
      for (; i < end && ok; i += step) {
        const FewTile t = tiles.get(ph, i);
        const int row = min(lane, t.valid - 1);
        const char* src = row < t.split ? t.base + row * t.ld_bytes
                                        : t.base2 + (row - t.split) * t.ld_bytes;
        for (int seg = 0; seg < t.segs && ok; ++seg) {
          const int seg_bytes = t.seg_len * kEs;
          for (int o = 0; o < seg_bytes; o += kFewRowBytes) {
            const int bytes = min(kFewRowBytes, seg_bytes - o);
            if (!mbar_wait(&empty[stage], phase_bit ^ 1)) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(bytes) * kFewRows);
            __syncwarp();
            if (lane < kFewRows)
              bulk_load(ring + stage * kFewStageBytes + lane * kFewRowPitch,
                        src + static_cast<long>(seg) * seg_bytes + o, static_cast<uint32_t>(bytes),
                        &full[stage]);
            issued |= 1u << stage;
            parities = (parities & ~(1u << stage)) | (phase_bit << stage);
            if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase_bit ^= 1; }
          }
        }
      }
    }
    if (!ok) *abort_ = 1;
    // No copy may still be landing in shared memory when the CTA exits.
    for (int s = 0; s < p.stages; ++s)
      if (issued >> s & 1) mbar_wait(&full[s], parities >> s & 1);
    return;
  }

  // ---------------------------------------------------------------- consumers
  uint32_t stage = 0, phase_bit = 0;
  int red_buf = 0;
  // Runs one tile through the ring; on return the 16 x 8 tile's partial sums of every warp lie in
  // the returned buffer.  arow of column c is rows[c]'s activation row, or none.
  auto run_tile = [&](const FewTile& t, const FewAct& act, int my_row, int row0, int row1) -> const float* {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kPer = kFewRowBytes / (kF32 ? 4 : 2);
    for (int seg = 0; seg < t.segs; ++seg) {
      for (int k0 = 0; k0 < t.seg_len; k0 += kPer) {
        if (!*abort_ && !mbar_wait(&full[stage], phase_bit)) *abort_ = 1;
        const char* st = ring + stage * kFewStageBytes;
        const int kw = min(kPer, t.seg_len - k0);
        if constexpr (kF32) {
          const char* x0 = row0 >= 0 ? act.base + row0 * act.pitch + k0 * 4 : nullptr;
          const char* x1 = row1 >= 0 ? act.base + row1 * act.pitch + k0 * 4 : nullptr;
          few_chunk_f32(st, kw, x0, x1, warp, lane, acc);
        } else {
          const char* ar = my_row >= 0 ? act.base + my_row * act.pitch + k0 * 2 : nullptr;
          few_chunk_bf16(st, kw, ar, act.plane, warp, lane, acc);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase_bit ^= 1; }
      }
    }
    float* rb = red + red_buf * kFewRedFloats;
    red_buf ^= 1;
    float* mine = rb + warp * kFewRows * kFewRedPitch;
    const int g = lane >> 2, c = (lane & 3) * 2;
    *reinterpret_cast<float2*>(mine + g * kFewRedPitch + c) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(mine + (g + 8) * kFewRedPitch + c) = make_float2(acc[2], acc[3]);
    few_bar();
    return rb;
  };
  auto tile_sum = [&](const float* rb, int row, int col) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) v += rb[(w * kFewRows + row) * kFewRedPitch + col];
    return v;
  };
  const int er = tid & 15, ec = tid >> 4;  // epilogue: tile row and column (threads 0 .. 127)
  const int g8 = lane >> 2, t2 = (lane & 3) * 2;

  // Residual gate and store of one output value.
  auto resid_out = [&](int t, int f, float b) {
    if constexpr (!kF32) {
      float x = b;
      if (p.resid_mode != MOE_RESID_NONE) {
        const float r = bf16_to_f32(static_cast<const uint16_t*>(p.r)[static_cast<size_t>(t) * p.d + f]);
        const float g = p.resid_g[f];
        if (p.resid_mode == MOE_RESID_MUSE_GATE) {
          const float beta = 1.0f / (1.0f + expf(-g / p.tau));
          const float alpha = sqrtf(fmaxf(1.0f / (1.0f + expf(g / p.tau)) * (1.0f + beta), p.floor_));
          x = fmaf(alpha, r, beta * b);
        } else {
          x = fmaf(g, b, r);
        }
      }
      static_cast<uint16_t*>(p.out)[static_cast<size_t>(t) * p.d + f] = f32_to_bf16(x);
    }
  };

  // u (or C_in(r)) to shared memory
  FewAct act = few_act<kF32>(act_mem, T, p.d, false);
  {
    const void* src = p.input_norm ? p.r : p.u;
    const int vec = p.d * (kF32 ? 4 : 2) / 16;
    for (int t = 0; t < T; ++t) {
      const uint4* row = static_cast<const uint4*>(src) + static_cast<size_t>(t) * vec;
      char* dst = act.base + t * act.pitch;
      for (int i = tid; i < vec; i += 32 * kFewWarps) *reinterpret_cast<uint4*>(dst + i * 16) = row[i];
    }
    few_bar();
    if constexpr (!kF32) {
      if (p.input_norm && warp < T) {  // one warp per token
        uint16_t* row = reinterpret_cast<uint16_t*>(act.base + warp * act.pitch);
        float ss = 0.0f;
        for (int i = lane; i < p.d; i += 32) { const float x = bf16_to_f32(row[i]); ss = fmaf(x, x, ss); }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = 1.0f / sqrtf(ss / p.d + p.eps_block);
        for (int i = lane; i < p.d; i += 32)
          row[i] = f32_to_bf16((1.0f + p.gamma_in[i]) * (bf16_to_f32(row[i]) * inv));
      }
      few_bar();
    }
  }
  const int tok_row = g8 < T ? g8 : -1, tok_row0 = t2 < T ? t2 : -1, tok_row1 = t2 + 1 < T ? t2 + 1 : -1;

  // The adapter term of row f for token t (0 without an adapter): sum over the rank in fp32.
  auto adapter_term = [&](const uint16_t* bmat, int rows, int f, int t) {
    const int a = tb.tok_ad[t];
    float v = 0.0f;
    if (a >= 0) {
      const uint16_t* br = bmat + (static_cast<size_t>(a) * rows + f) * p.rank;
      for (int r0 = 0; r0 < p.rank; r0 += 8) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(br + r0));
        const uint16_t* h = reinterpret_cast<const uint16_t*>(&q);
#pragma unroll
        for (int j = 0; j < 8; ++j) v = fmaf(bf16_to_f32(h[j]), s_v[t * p.rank + r0 + j], v);
      }
    }
    return v;
  };
  auto load_v = [&](const float* v) {
    for (int i = tid; i < T * p.rank; i += 32 * kFewWarps) s_v[i] = __ldcg(&v[i]);
    few_bar();
  };
  // Inner products of an adapter tile: scale * (A x), for the tokens that use this adapter.
  auto put_v = [&](const FewTile& t, const float* rb, float* v) {
    if (tid < 128 && ec < T && er < t.valid && tb.tok_ad[ec] == tb.ad[t.e])
      v[ec * p.rank + t.r0 + er] = p.scale[tb.ad[t.e]] * tile_sum(rb, er, ec);
  };

  // -------------------------------------------------------------- router, adapters' A, latent down
  {
    int i, end, step;
    tiles.range(FEW_IN, i, end, step);
    const int lead = tiles.lead_tiles(FEW_IN);
    for (; i < lead; i += step) {
      const FewTile t = tiles.get(FEW_IN, i);
      const float* rb = run_tile(t, act, tok_row, tok_row0, tok_row1);
      if (t.kind == FEW_ROUTER) {
        const int e = t.r0 + er;
        if (tid < 128 && ec < T && e < p.n) {
          float l = tile_sum(rb, er, ec);
          if (p.gate_mode == MOE_GATE_SIGMOID) l *= p.logit_mult;
          p.logits[static_cast<size_t>(ec) * p.n + e] = l + (p.logit_bias ? p.logit_bias[e] : 0.0f);
        }
      } else {
        put_v(t, rb, p.v_down);
      }
    }
    few_arrive(p.bar, 0);
    bool have_v = tb.ndist_ad == 0;
    for (; i < end; i += step) {
      const FewTile t = tiles.get(FEW_IN, i);
      const float* rb = run_tile(t, act, tok_row, tok_row0, tok_row1);
      if (!have_v) {
        few_wait(p.bar, 0, abort_);
        load_v(p.v_down);
        have_v = true;
      }
      if (tid < 128 && ec < T) {
        float v = tile_sum(rb, er, ec);
        if (tb.ndist_ad) v += adapter_term(p.down_b, p.L, t.r0 + er, ec);
        p.z[static_cast<size_t>(ec) * p.L + t.r0 + er] = v;
      }
    }
    few_arrive(p.bar, 1);
  }

  // -------------------------------------------------------------- routing tables
  few_wait(p.bar, 0, abort_);
  if (warp < T) few_topk(p, tb, warp, lane);
  few_bar();
  {
    // distinct experts in ascending order, each with its slots in token order (thread = expert)
    const int slots = T * k;
    int cnt = 0;
    uint8_t mine[kFewTokens];
    for (int s = 0; s < slots; ++s)
      if (tb.idx[s] == tid && cnt < kFewTokens) mine[cnt++] = static_cast<uint8_t>(s);
    tb.own[tid] = cnt;
    few_bar();
    if (cnt > 0) {
      int at = 0;
      for (int e = 0; e < tid; ++e) at += tb.own[e] > 0;
      tb.expert[at] = tid;
      tb.count[at] = cnt;
      for (int q = 0; q < cnt; ++q) tb.slot[at][q] = mine[q];
    }
    if (tid == 255) {
      int at = 0;
      for (int e = 0; e < 256; ++e) at += tb.own[e] > 0;
      tb.dist = at;
    }
    if (blockIdx.x == 0 && tid < slots) {
      if (p.idx_out) p.idx_out[tid] = tb.idx[tid];
      if (p.w_out) p.w_out[tid] = tb.w[tid];
    }
    few_bar();
    if (tid == 0) mbar_arrive(&routed);
  }

  // -------------------------------------------------------------- z (C_pre) to shared memory
  if (p.L) {
    few_wait(p.bar, 1, abort_);
    act = few_act<kF32>(act_mem, T, p.E, true);
    if (p.pre_norm) {
      float ss[kFewTokens];
#pragma unroll
      for (int t = 0; t < kFewTokens; ++t) {
        ss[t] = 0.0f;
        if (t < T)
          for (int c = tid * 4; c < p.E; c += 128 * kFewWarps) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.z + static_cast<size_t>(t) * p.E + c));
            ss[t] += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss[t] += __shfl_xor_sync(0xffffffffu, ss[t], o);
        if (lane == 0) tb.red[warp][t] = ss[t];
      }
      few_bar();
      if (tid < T) {
        float v = 0.0f;
        for (int w = 0; w < kFewWarps; ++w) v += tb.red[w][tid];
        tb.norm[tid] = 1.0f / sqrtf(v / p.E + p.eps);
      }
      few_bar();
    }
    for (int t = 0; t < T; ++t) {
      const float inv = p.pre_norm ? tb.norm[t] : 1.0f;
      for (int c = tid * 4; c < p.E; c += 128 * kFewWarps) {
        float4 v = __ldcg(reinterpret_cast<const float4*>(p.z + static_cast<size_t>(t) * p.E + c));
        if (p.pre_norm) {
          const float4 g = *reinterpret_cast<const float4*>(p.gamma_pre + c);
          v.x *= inv * (1.0f + g.x); v.y *= inv * (1.0f + g.y);
          v.z *= inv * (1.0f + g.z); v.w *= inv * (1.0f + g.w);
        }
        few_act_put4<kF32>(act, t, c, v);
      }
    }
    few_bar();
  }

  // -------------------------------------------------------------- experts, first product
  {
    int i, end, step;
    tiles.range(FEW_UP1, i, end, step);
    for (; i < end; i += step) {
      const FewTile t = tiles.get(FEW_UP1, i);
      const int m = tb.count[t.e];
      auto tok = [&](int c) { return c < m ? tb.slot[t.e][c] / k : -1; };
      const float* rb = run_tile(t, act, tok(g8), tok(t2), tok(t2 + 1));
      if (p.swiglu) {
        if (tid < 64) {
          const int row = tid & 7, col = tid >> 3;
          if (col < m) {
            const float g = tile_sum(rb, row, col), up = tile_sum(rb, row + 8, col);
            p.a[static_cast<size_t>(tb.slot[t.e][col]) * p.H + t.r0 + row] = g / (1.0f + expf(-g)) * up;
          }
        }
      } else if (tid < 128 && ec < m) {
        const float v = tile_sum(rb, er, ec);
        // NaN stays NaN (fmaxf would drop it)
        p.a[static_cast<size_t>(tb.slot[t.e][ec]) * p.H + t.r0 + er] = v < 0.0f ? 0.0f : v;
      }
    }
    few_arrive(p.bar, 2);
  }

  // -------------------------------------------------------------- experts, second product
  few_wait(p.bar, 2, abort_);
  {
    int i, end, step, loaded = -1;
    tiles.range(FEW_DOWN2, i, end, step);
    act = few_act<kF32>(act_mem, T, p.H, true);
    for (; i < end; i += step) {
      const FewTile t = tiles.get(FEW_DOWN2, i);
      const int m = tb.count[t.e];
      if (t.e != loaded) {  // this expert's rows (every warp is past the previous tile's products)
        for (int c = 0; c < m; ++c) {
          const float* row = p.a + static_cast<size_t>(tb.slot[t.e][c]) * p.H;
          for (int j = tid * 4; j < p.H; j += 128 * kFewWarps)
            few_act_put4<kF32>(act, c, j, __ldcg(reinterpret_cast<const float4*>(row + j)));
        }
        few_bar();
        loaded = t.e;
      }
      const float* rb = run_tile(t, act, g8 < m ? g8 : -1, t2 < m ? t2 : -1, t2 + 1 < m ? t2 + 1 : -1);
      if (tid < 128) {
        const int f = t.r0 + er;
        float v = 0.0f;
        if (ec < m) {
          v = tile_sum(rb, er, ec);
          if (p.expert_norm) v *= 1.0f + p.gamma_expert[f];
          p.s[static_cast<size_t>(tb.slot[t.e][ec]) * p.E + f] = v;
        }
        if (p.expert_norm) {
          float q = v * v;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          if (er == 0 && ec < m)
            p.ss[static_cast<size_t>(tb.slot[t.e][ec]) * (p.E / 16) + t.r0 / 16] = q;
        }
      }
    }
    few_arrive(p.bar, 3);
  }

  // -------------------------------------------------------------- I_gamma and the weighted sum
  few_wait(p.bar, 3, abort_);
  {
    const int cols = 32 * kFewWarps, blocks = (p.E + cols - 1) / cols;
    for (int unit = blockIdx.x; unit < T * blocks; unit += gridDim.x) {
      const int t = unit / blocks, c = (unit - t * blocks) * cols + tid;
      if (warp < k) {
        float inv = 1.0f;
        if (p.expert_norm) {
          const float* part = p.ss + static_cast<size_t>(t * k + warp) * (p.E / 16);
          float q = 0.0f;
          for (int j = lane; j < p.E / 16; j += 32) q += __ldcg(&part[j]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          inv = 1.0f / sqrtf(q / p.E + p.eps);
        }
        if (lane == 0) tb.inv[warp] = inv;
      }
      few_bar();
      if (c < p.E) {
        float y = 0.0f;
        for (int j = 0; j < k; ++j)
          y = fmaf(tb.w[t * k + j],
                   __ldcg(&p.s[static_cast<size_t>(t * k + j) * p.E + c]) * tb.inv[j], y);
        if (p.L) p.y[static_cast<size_t>(t) * p.E + c] = y;
        else if (kF32) static_cast<float*>(p.out)[static_cast<size_t>(t) * p.E + c] = y;
        else static_cast<uint16_t*>(p.out)[static_cast<size_t>(t) * p.E + c] = f32_to_bf16(y);
      }
      few_bar();
    }
  }
  if (!p.L) return;
  few_arrive(p.bar, 4);
  few_wait(p.bar, 4, abort_);

  // -------------------------------------------------------------- adapters' A', latent up, residual
  act = few_act<kF32>(act_mem, T, p.L, true);
  for (int t = 0; t < T; ++t)
    for (int c = tid * 4; c < p.L; c += 128 * kFewWarps)
      few_act_put4<kF32>(act, t, c, __ldcg(reinterpret_cast<const float4*>(p.y + static_cast<size_t>(t) * p.L + c)));
  few_bar();
  {
    int i, end, step;
    tiles.range(FEW_OUT, i, end, step);
    const int lead = tiles.lead_tiles(FEW_OUT);
    for (; i < lead; i += step) {
      const FewTile t = tiles.get(FEW_OUT, i);
      put_v(t, run_tile(t, act, tok_row, tok_row0, tok_row1), p.v_up);
    }
    bool have_v = tb.ndist_ad == 0;
    if (!have_v) few_arrive(p.bar, 5);
    for (; i < end; i += step) {
      const FewTile t = tiles.get(FEW_OUT, i);
      const float* rb = run_tile(t, act, tok_row, tok_row0, tok_row1);
      if (!have_v) {
        few_wait(p.bar, 5, abort_);
        load_v(p.v_up);
        have_v = true;
      }
      if (tid < 128) {
        const int f = t.r0 + er;
        float v = 0.0f;
        if (ec < T) {
          v = tile_sum(rb, er, ec);
          if (tb.ndist_ad) v += adapter_term(p.up_b, p.d, f, ec);
          if (p.post_norm) {
            v *= 1.0f + p.gamma_post[f];
            p.b[static_cast<size_t>(ec) * p.d + f] = v;
          } else {
            resid_out(ec, f, v);
          }
        }
        if (p.post_norm) {
          float q = v * v;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          if (er == 0 && ec < T) p.bss[static_cast<size_t>(ec) * (p.d / 16) + t.r0 / 16] = q;
        }
      }
    }
  }
  if (!p.post_norm) return;

  // -------------------------------------------------------------- output norm, residual
  few_arrive(p.bar, 6);
  few_wait(p.bar, 6, abort_);
  const int cols = 32 * kFewWarps, blocks = (p.d + cols - 1) / cols;
  for (int unit = blockIdx.x; unit < T * blocks; unit += gridDim.x) {
    const int t = unit / blocks, c = (unit - t * blocks) * cols + tid;
    float q = 0.0f;
    for (int j = tid; j < p.d / 16; j += 32 * kFewWarps)
      q += __ldcg(&p.bss[static_cast<size_t>(t) * (p.d / 16) + j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    if (lane == 0) tb.red[warp][0] = q;
    few_bar();
    q = 0.0f;
    for (int w = 0; w < kFewWarps; ++w) q += tb.red[w][0];
    const float inv = 1.0f / sqrtf(q / p.d + p.eps_block);
    if (c < p.d) resid_out(t, c, __ldcg(&p.b[static_cast<size_t>(t) * p.d + c]) * inv);
    few_bar();
  }
}

}  // namespace moe
