// Dense projection of a few rows (at most 64: a decode batch) with its reduction split over the
// CTAs of a thread-block cluster: the latent down-projection z_raw = u P_down^T and the latent
// up-projection with the residual gate, out = alpha * r + beta * dtype(y P_up^T) ("Muse Spark
// Open: Norm-Preserving Gates Are Not a Norm Guarantee", sections "Latent experts" and
// "Residual gates").
//
// At this size the weight stream is the whole cost (67 MB per projection), and the 128-row weight
// tiles of a 4096- or 8192-wide output number only 32 or 64, fewer than the SMs.  So each
// 128-feature tile is shared by the S CTAs of one cluster, CTA s streaming k-blocks
// [s K/S, (s+1) K/S) into its own TMEM accumulator (swapped orientation: 128 weight rows on the
// MMA's M side, the batch's rows on N).  The CTAs then add their fp32 partial tiles through
// distributed shared memory, in the fixed order s = 0, 1, ..., S-1, each finishing 128/S of the
// features: no partial sums go out to HBM and no second kernel runs.
//   - TMA loads without multicast; every mbarrier wait is bounded; the cluster barriers are
//     reached by every thread of every CTA, also after a wait ran out.
//   - The partial tile [rows][128] fp32 reuses the operand ring once the MMAs have finished.
#pragma once

#include "few_tokens.cuh"
#include "gemm_tc.cuh"

namespace moe {

constexpr int kSplitBN = 64;      // rows of the batch on the MMA's N side (all of them)
constexpr int kSplitStages = 8;
constexpr int kSplitMaxCluster = 8;
using SplitShape = GemmShape<true, kSplitBN, EPI_STORE>;

// Ring stages: with adapters fewer, to make room for their inner products and terms (120 KB in flight
// on each of 128 SMs is still more than the memory system holds).
template <class Adapt>
constexpr int split_stages() { return Adapt::kOn ? 5 : kSplitStages; }
template <class Adapt>
constexpr int gemm_splitk_smem_bytes() {
  return split_stages<Adapt>() * SplitShape::kStageBytes + 1024 + 256;
}
static_assert(kSplitBN * 128 * 4 <= 5 * SplitShape::kStageBytes, "the partial tile fits in the operand ring");

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t caddr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(caddr)
               : "memory");
  return v;
}

// Low-rank adapters of the batch's rows: row t adds B_a v_t, a = which[t], v_t the sum of the partial
// inner products v[s, t, :] (already scaled) that the kernel just before this one writes.
constexpr int kSplitAdaptParts = 4;
constexpr int kSplitAdaptThreads = 256;  // that make the terms: the 128 epilogue threads and 128 more
__device__ __forceinline__ void split_adapt_bar() {
  asm volatile("bar.sync 2, %0;" ::"n"(kSplitAdaptThreads) : "memory");
}
struct SplitAdapt {
  static constexpr bool kOn = true;
  const float* v;          // [kSplitAdaptParts, rows, rank]
  const uint16_t* b;       // [n, Nout, rank]
  const int32_t* which;    // [rows]
  int n, rank;
};
// Shared memory of the terms: v as hi and lo bf16 planes [kSplitBN][rank rounded up to 32, + 32], the
// terms [kSplitBN][64 + 4] fp32, the rows grouped by adapter, and a buffer of the adapters' B rows.
__host__ __device__ constexpr int split_adapt_pitch(int rank) { return (rank + 31) / 32 * 64 + 64; }  // bytes
constexpr int kSplitTermPitch = 68;
struct __align__(16) SplitRows {  // the batch's rows grouped by adapter, in order of the adapters' first rows
  int a[kSplitBN];            // a row's adapter, -1: none
  int row[kSplitBN];          // the grouped rows
  int adapter[kSplitBN];      // a group's adapter
  int first[kSplitBN + 4];    // where a group's rows begin (and the end of the last)
  int start[kSplitBN];        // per row that leads a group: where its group begins
  int leaders[2], taken[2];   // per warp of rows
};
// Bytes of that buffer: 40 KB at the largest rank, and what v leaves at smaller ones.  (64 adapters of rank 16
// then need no second filling of it: 30.3 -> 29.1 us a call.)
__host__ __device__ constexpr int split_b_bytes(int rank) {
  return 40 * 1024 + 2 * kSplitBN * (split_adapt_pitch(MOE_ADAPTER_MAX_RANK) - split_adapt_pitch(rank));
}
constexpr int split_adapt_smem(int rank) {
  return 2 * kSplitBN * split_adapt_pitch(rank) + kSplitBN * kSplitTermPitch * 4 +
         static_cast<int>(sizeof(SplitRows)) + split_b_bytes(rank);
}

// The adapter terms B_a v_t of this CTA's 128/NS features for every row, into s_term[row][feature].  Runs
// in kSplitAdaptThreads threads while the tile's weights stream in, and behind that stream every load
// takes about 3 us: what counts is how few of them wait for one another.  So the rows are grouped by
// adapter, the adapters' B rows come in as one bulk copy each (a part of B is contiguous), as many as
// half a buffer holds while the other half is in use, and v's partial sums as one batch of loads; then
// m16n8k16 products put 16 features on M, eight of an adapter's rows on N and the rank on K.  (Loading B
// into fragments adapter by adapter, 64 adapters of rank 16 took 60 us; a thread to 8 features on the
// CUDA cores, 12 of rank 64 also 60.)
// v enters as hi + lo, so the term keeps fp32's accuracy to 2^-17.
template <int NS>
__device__ __forceinline__ void splitk_adapt(const SplitAdapt& ad, const GemmParams& p, uint32_t rank,
                                             int ft, char* smem, uint64_t* b_full) {
  constexpr int kFs = 128 / NS;
  const int et = static_cast<int>(threadIdx.x) - 64, warp = et >> 5, lane = et & 31;
  const int pitch = split_adapt_pitch(ad.rank), kpad = (ad.rank + 31) / 32 * 32;
  char* s_v = smem;
  const int plane = kSplitBN * pitch;
  float* s_term = reinterpret_cast<float*>(smem + 2 * plane);
  SplitRows& r = *reinterpret_cast<SplitRows*>(s_term + kSplitBN * kSplitTermPitch);
  char* s_b = reinterpret_cast<char*>(&r + 1);
  const int f0 = ft * 128 + static_cast<int>(rank) * kFs;
  const int b_half = split_b_bytes(ad.rank) / 2, b_bytes = kFs * ad.rank * 2, fit = b_half / b_bytes;  // adapters in half of the buffer

  if (et < kSplitBN) {
    int a = -1;
    if (et < p.M) {
      a = ad.which[et];
      if (a < 0 || a >= ad.n) a = -1;
    }
    r.a[et] = a;
  }
  for (int i = et; i < kSplitBN * kSplitTermPitch; i += kSplitAdaptThreads) s_term[i] = 0.0f;
  split_adapt_bar();
  // Grouping, a thread to a row: a group begins after the sizes of the groups led by earlier rows.
  // (One warp walking over the rows, and one thread issuing the copies, took 34 us for 64 adapters.)
  int lead = 0, mine = -1, size = 0, incl = 0;
  unsigned long long same = 0;
  if (et < kSplitBN) {
    mine = r.a[et];
#pragma unroll
    for (int j = 0; j < kSplitBN; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(&r.a[j]);
      const unsigned f = (v.x == mine) | (v.y == mine) << 1 | (v.z == mine) << 2 | (v.w == mine) << 3;
      same |= static_cast<unsigned long long>(f) << j;
    }
    lead = mine >= 0 && __ffsll(static_cast<long long>(same)) - 1 == et;
    size = lead ? __popcll(same) : 0;
  }
  const unsigned leaders = __ballot_sync(0xffffffffu, lead);
  incl = size;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31 && warp < 2) {
    r.leaders[warp] = __popc(leaders);
    r.taken[warp] = incl;
  }
  split_adapt_bar();
  const int groups = r.leaders[0] + r.leaders[1], rows = r.taken[0] + r.taken[1];
  if (lead) {
    const int gid = (warp ? r.leaders[0] : 0) + __popc(leaders & ((1u << lane) - 1u));
    const int begin = (warp ? r.taken[0] : 0) + incl - size;
    r.adapter[gid] = mine;
    r.first[gid] = begin;
    r.start[et] = begin;
  }
  if (et == 0) r.first[groups] = rows;
  split_adapt_bar();
  if (mine >= 0)
    r.row[r.start[__ffsll(static_cast<long long>(same)) - 1] + __popcll(same & ((1ull << et) - 1ull))] = et;
  // Copies of the B rows of round k's adapters [k fit, k fit + fit) into half k & 1 of the buffer, a thread
  // to an adapter.  (A copy may land before its bytes are expected: the phase ends with the one arrival.)
  auto fetch = [&](int k) {
    const int m = min(fit, groups - k * fit);
    if (m <= 0) return;
    if (et == 0) mbar_arrive_expect_tx(&b_full[k & 1], static_cast<uint32_t>(m) * b_bytes);
    for (int i = et; i < m; i += kSplitAdaptThreads)
      bulk_load(s_b + (k & 1) * b_half + i * b_bytes,
                ad.b + (static_cast<size_t>(r.adapter[k * fit + i]) * p.Nout + f0) * ad.rank,
                static_cast<uint32_t>(b_bytes), &b_full[k & 1]);
  };
  fetch(0);
  fetch(1);
  pdl_wait();  // v
  // Four columns of a row at a time, two of them and all their parts in flight; the padding of the rank
  // to whole 32s is zero.
  const int vec = ad.rank / 4, pad = (kpad - ad.rank) / 4;
  for (int i = et; i < p.M * pad; i += kSplitAdaptThreads) {
    char* at = s_v + i / pad * pitch + (ad.rank + i % pad * 4) * 2;
    *reinterpret_cast<uint2*>(at) = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(at + plane) = make_uint2(0, 0);
  }
  for (int i = et; i < p.M * vec; i += 2 * kSplitAdaptThreads) {
    float4 part[2][kSplitAdaptParts];
    int t[2], c[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = i + u * kSplitAdaptThreads;
      t[u] = x < p.M * vec ? x / vec : -1;
      c[u] = (x - t[u] * vec) * 4;
      const bool has = t[u] >= 0 && r.a[max(t[u], 0)] >= 0;
#pragma unroll
      for (int s = 0; s < kSplitAdaptParts; ++s) {
        part[u][s] = make_float4(0, 0, 0, 0);
        if (has)
          part[u][s] = __ldcg(reinterpret_cast<const float4*>(
              ad.v + (static_cast<size_t>(s) * p.M + t[u]) * ad.rank + c[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (t[u] < 0) continue;
      float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kSplitAdaptParts; ++s) {
        f[0] += part[u][s].x; f[1] += part[u][s].y; f[2] += part[u][s].z; f[3] += part[u][s].w;
      }
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float h0 = round_bf16(f[2 * j]), h1 = round_bf16(f[2 * j + 1]);
        hi[j] = pack_bf16x2(h0, h1);  // a non-finite value has no remainder
        lo[j] = pack_bf16x2(isfinite(h0) ? f[2 * j] - h0 : 0.0f, isfinite(h1) ? f[2 * j + 1] - h1 : 0.0f);
      }
      *reinterpret_cast<uint2*>(s_v + t[u] * pitch + c[u] * 2) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(s_v + plane + t[u] * pitch + c[u] * 2) = make_uint2(lo[0], lo[1]);
    }
  }
  split_adapt_bar();
  const int g = lane >> 2, q = lane & 3;
  const uint32_t v0 = smem_u32(s_v) + q * 16, b0 = smem_u32(s_b) + g * ad.rank * 2 + q * 16;
  bool ok = true;
  for (int g0 = 0, round = 0; g0 < groups; g0 += fit, ++round) {
    ok = ok && mbar_wait(&b_full[round & 1], round >> 1 & 1);
    const int pairs = min(fit, groups - g0) * (kFs / 16);
    // (adapter, 16-feature tile), a warp at a time
    for (int w = warp; w < pairs; w += kSplitAdaptThreads / 32) {
      const int gi = w / (kFs / 16), mt = w % (kFs / 16), gr = g0 + gi;
      const int r0 = r.first[gr], r1 = r.first[gr + 1];
      const uint32_t b = b0 + (round & 1) * b_half + gi * b_bytes + mt * 32 * ad.rank;
      for (int c0 = r0; c0 < r1; c0 += 8) {  // eight rows on N
        const bool has = c0 + g < r1;
        const uint32_t v = v0 + (has ? r.row[c0 + g] : 0) * pitch;
        float d[2][4] = {};
        for (int s = 0; s * 32 < ad.rank; ++s) {
          const uint4 zero = make_uint4(0, 0, 0, 0);
          uint4 x = zero, y = zero, h = zero, l = zero;
          if (s * 32 + q * 8 < ad.rank) {
            x = lds128(b + s * 64);
            y = lds128(b + 16 * ad.rank + s * 64);
          }
          if (has) {
            h = lds128(v + s * 64);
            l = lds128(v + plane + s * 64);
          }
          few_mma(d[0], x.x, y.x, x.y, y.y, h.x, h.y);
          few_mma(d[1], x.x, y.x, x.y, y.y, l.x, l.y);
          few_mma(d[0], x.z, y.z, x.w, y.w, h.z, h.w);
          few_mma(d[1], x.z, y.z, x.w, y.w, l.z, l.w);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = c0 + 2 * q + j;
          if (c < r1) {
            float* o = s_term + r.row[c] * kSplitTermPitch + mt * 16 + g;
            o[0] = d[0][j] + d[1][j];
            o[8] = d[0][2 + j] + d[1][2 + j];
          }
        }
      }
    }
    if (g0 + 2 * fit < groups) {
      split_adapt_bar();  // every warp is done with this half
      fetch(round + 2);
    }
  }
}

// Reduce + epilogue of one CTA of a cluster of NS: CTA `rank` finishes features
// [rank * 128/NS, (rank + 1) * 128/NS) of feature tile `ft` for every row, in vectors of 8
// features.  Thread (group g, row lane r) of the 128 epilogue threads takes features g*8 .. g*8+7
// of that part and rows r, r + nr, ... (8/NS rows); all of its loads (the NS partial tiles through
// distributed shared memory, the residual rows) are issued before the first sum, and the partials
// are added in the order s = 0, 1, ..., NS-1.
template <int kEpi, int NS, bool kAdd>
__device__ __forceinline__ void splitk_reduce(const GemmParams& p, const float* part, uint32_t rank,
                                              int ft, const float* term) {
  constexpr int kFs = 128 / NS, kGroups = kFs / 8, kNr = 128 / kGroups, kRows = kSplitBN / kNr;
  static_assert(kRows * kNr == kSplitBN && kGroups * 8 == kFs, "reduce layout");
  const int et = static_cast<int>(threadIdx.x) - 64;
  const int g = et % kGroups, r0 = et / kGroups;
  const int fl = static_cast<int>(rank) * kFs + g * 8;  // first feature within the tile
  const int col = ft * 128 + fl;
  float4 cur[NS][kRows][2];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const uint32_t base = cluster_addr(part, static_cast<uint32_t>(s));
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const int row = r0 + q * kNr;
      if (row < p.M) {
        const uint32_t off = base + static_cast<uint32_t>((row * 128 + fl) * 4);
        cur[s][q][0] = ld_cluster_f32x4(off);
        cur[s][q][1] = ld_cluster_f32x4(off + 16);
      }
    }
  }
  const bool has_r = kEpi == EPI_RESGATE && p.resid_mode != MOE_RESID_NONE;
  uint4 rv[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    const int row = r0 + q * kNr;
    rv[q] = make_uint4(0, 0, 0, 0);
    if (row < p.M && has_r)
      rv[q] = __ldg(reinterpret_cast<const uint4*>(p.resid + static_cast<size_t>(row) * p.Nout + col));
  }
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = 0.0f;
    b[j] = 1.0f;
    if constexpr (kEpi == EPI_RESGATE) {
      const float gg = p.gparam ? p.gparam[col + j] : 0.0f;
      if (p.resid_mode == MOE_RESID_MUSE_GATE) {
        b[j] = sigmoidf_(gg / p.tau);
        a[j] = sqrtf(fmaxf(sigmoidf_(-gg / p.tau) * (1.0f + b[j]), p.floor_));
      } else if (p.resid_mode == MOE_RESID_LITERAL) {
        a[j] = 1.0f;
        b[j] = gg;
      }
    }
  }
  uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    const int row = r0 + q * kNr;
    if (row >= p.M) continue;
    float v[8] = {cur[0][q][0].x, cur[0][q][0].y, cur[0][q][0].z, cur[0][q][0].w,
                  cur[0][q][1].x, cur[0][q][1].y, cur[0][q][1].z, cur[0][q][1].w};
#pragma unroll
    for (int s = 1; s < NS; ++s) {
      v[0] += cur[s][q][0].x; v[1] += cur[s][q][0].y; v[2] += cur[s][q][0].z; v[3] += cur[s][q][0].w;
      v[4] += cur[s][q][1].x; v[5] += cur[s][q][1].y; v[6] += cur[s][q][1].z; v[7] += cur[s][q][1].w;
    }
    const uint16_t* rh = reinterpret_cast<const uint16_t*>(&rv[q]);
    uint4 o;
    uint16_t* oh = reinterpret_cast<uint16_t*>(&o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = v[j];
      if constexpr (kAdd) x += term[row * kSplitTermPitch + g * 8 + j];
      if constexpr (kEpi == EPI_RESGATE)
        x = __fmaf_rn(a[j], bf16_to_f32(rh[j]), __fmul_rn(b[j], round_bf16(x)));
      oh[j] = f32_to_bf16(x);
    }
    *reinterpret_cast<uint4*>(out + static_cast<size_t>(row) * p.Nout + col) = o;
  }
}

// kEpi: EPI_STORE (out = dtype(sum)) or EPI_RESGATE (out = dtype(alpha r + beta dtype(sum))).
// Grid: (Nout / 128) * S CTAs in clusters of S (2 <= S <= 8, S divides K / 64); rows p.M <= kSplitBN.
template <class Adapt>
constexpr int split_threads() { return Adapt::kOn ? 64 + kSplitAdaptThreads : kGemmThreads; }
template <int kEpi, class Adapt = NoAdapt>
// (With adapters two CTAs' worth of registers at most: room for the inner products' CTAs beside this one.)
__global__ void __launch_bounds__(split_threads<Adapt>(), Adapt::kOn ? 2 : 1)
    gemm_splitk_cluster_kernel(const __grid_constant__ CUtensorMap tmX,
                               const __grid_constant__ CUtensorMap tmW, const GemmParams p,
                               const Adapt ad) {
  static_assert(kEpi == EPI_STORE || kEpi == EPI_RESGATE, "dense projection epilogues");
  using S = SplitShape;
  constexpr int kStages = split_stages<Adapt>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  float* part = reinterpret_cast<float*>(tiles);  // after the MMAs: [kSplitBN rows][128 features]
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + kStages * S::kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* b_full = tfull + 1;  // adapters: the B rows in either half of their buffer have landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_full + 2);

  char* s_adapt = reinterpret_cast<char*>(tiles) + kStages * S::kStageBytes + 256;  // adapters only

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int ns = static_cast<int>(cluster_nctarank());
  const int ft = static_cast<int>(blockIdx.x) / ns;
  const int kbs = p.K / S::kBK / ns;
  const int kb0 = static_cast<int>(rank) * kbs;

  // Setup that reads nothing an earlier kernel writes runs before the dependency wait.
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    mbar_init(tfull, 1);
    mbar_init(&b_full[0], 1);
    mbar_init(&b_full[1], 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kSplitBN);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  // With adapters the kernel before this one only makes their inner products, and started once
  // everything before it was complete: x may be read at once.
  if (!Adapt::kOn) pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    uint32_t stage = 0, phase = 0;
    uint32_t last_parity[kStages];
    bool issued[kStages];
#pragma unroll
    for (int s = 0; s < kStages; ++s) { issued[s] = false; last_parity[s] = 0; }
    for (int kb = kb0; kb < kb0 + kbs; ++kb) {
      if (!mbar_wait(&empty[stage], phase ^ 1)) break;
      uint8_t* sa = tiles + stage * S::kStageBytes;
      mbar_arrive_expect_tx(&full[stage], S::kStageBytes);
      tma_load_2d(&tmW, &full[stage], sa, kb * S::kBK, ft * 128);
      tma_load_2d(&tmX, &full[stage], sa + S::kABytes, kb * S::kBK, 0);
      issued[stage] = true;
      last_parity[stage] = phase;
      if (++stage == kStages) { stage = 0; phase ^= 1; }
    }
    // No copy may still be landing in the ring once the partial tile is written there.
    for (int s = 0; s < kStages; ++s)
      if (issued[s]) mbar_wait(&full[s], last_parity[s]);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0;
    for (int kb = kb0; kb < kb0 + kbs; ++kb) {
      if (!mbar_wait(&full[stage], phase)) break;
      tc_fence_after();
      const uint32_t a_addr = smem_u32(tiles + stage * S::kStageBytes);
      const uint32_t b_addr = a_addr + S::kABytes;
#pragma unroll
      for (int k = 0; k < S::kBK / 16; ++k)
        tc_mma_bf16(tmem_base, smem_desc_k128(a_addr + 32 * k), smem_desc_k128(b_addr + 32 * k),
                    S::kIdesc, (kb > kb0 || k > 0) ? 1u : 0u);
      tc_commit(&empty[stage]);
      if (++stage == kStages) { stage = 0; phase ^= 1; }
    }
    // Arrives when every MMA issued above has finished (and with them every operand load the
    // producer issued, each of which an MMA waited for), so the ring may be overwritten; the
    // issuer waits for it too, so no MMA is in flight when TMEM is released.
    tc_commit(tfull);
    mbar_wait(tfull, 0);
  } else if (warp >= 2) {
    // ------------------------------------------------------------ partial tile to shared memory
    const int q = warp & 3;  // TMEM lane quarter: features 32q .. 32q + 31
    if constexpr (Adapt::kOn) {
      switch (ns) {
        case 2: splitk_adapt<2>(ad, p, rank, ft, s_adapt, b_full); break;
        case 4: splitk_adapt<4>(ad, p, rank, ft, s_adapt, b_full); break;
        default: splitk_adapt<8>(ad, p, rank, ft, s_adapt, b_full); break;
      }
    }
    if (warp < 6) {
      mbar_wait(tfull, 0);
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const int f = q * 32 + lane;
#pragma unroll 1
      for (int j0 = 0; j0 < kSplitBN; j0 += 16) {
        float v[16];
        tmem_ld16(tb + j0, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(j0 + i) * 128 + f] = v[i];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // every CTA's partial tile is complete and visible to the cluster

  if (warp >= 2 && warp < 6) {
    // ------------------------------------------------------------ reduce + epilogue
    const float* term = nullptr;  // the adapters' terms
    if constexpr (Adapt::kOn) term = reinterpret_cast<const float*>(s_adapt + 2 * kSplitBN * split_adapt_pitch(ad.rank));
    switch (ns) {
      case 2: splitk_reduce<kEpi, 2, Adapt::kOn>(p, part, rank, ft, term); break;
      case 4: splitk_reduce<kEpi, 4, Adapt::kOn>(p, part, rank, ft, term); break;
      default: splitk_reduce<kEpi, 8, Adapt::kOn>(p, part, rank, ft, term); break;
    }
  }
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while a peer may still read its partial tile
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kSplitBN);
  }
}

}  // namespace moe
