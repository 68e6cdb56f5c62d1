// decode_paged_sm100.cuh -- split-KV Skip-Softmax decode over a paged cache:
// bf16 pages, and what the 4-bit kernel (decode_paged4_sm100.cuh) shares.
//
// The rule is that of the contiguous decode: a decode tile is 64 keys and the
// G = Hq / Hkv query heads of one kv head, the heads take one joint decision,
// every split starts from m_run = -inf, and the splits merge by log-sum-exp.
//
// One CTA per (split, kv head, sequence): a producer warp follows the block
// table and streams tiles into shared memory, four consumer warps own 16 of a
// tile's 64 keys each.  The contractions run as m16n8k16 tensor-core products
// with the KEYS in the 16-row dimension and the heads in the 8-column one:
//   S^T[16 keys, 8 heads] = K Q^T,   O^T[d, 8 heads] += V^T P^T,
// so eight heads fill the instruction (16-row query tiles would leave half of
// it empty), and one 8x8 transpose of the packed P turns the first product's
// result into the second's operand (P in two bf16 parts, so that it is as good
// as the contiguous decode's, which holds it in fp32).  Each warp keeps O^T of its own keys in
// registers; the warps merge once per split.  (tcgen05 has no use here: the
// kernel is bound by HBM.)
//
// Without a threshold (SKIP = false) K and V tiles are fetched together, no
// warp ever waits for another, and the softmax reference of a warp moves only
// when a score exceeds it by 2^8.  With one, the warps exchange their tile
// maxima (one named barrier a tile), all take the same decision, and the V
// tile is fetched after it, kLag tiles ahead of its use; a skipped tile costs
// no V bytes.  64 sequences of 16K-32K (8 kv heads, d = 128): 896 us, 7.2 TB/s,
// without a threshold; at factor 500 (63 % skipped) 650 us, 6.8 TB/s of what it
// reads (699 us where calls on three such caches take turns).
#pragma once

#include "kvcache_sm100.cuh"
#include "skip_rule.cuh"

namespace sskip {

struct PagedDecodeParams {
  const __nv_bfloat16* q;      // [B, Hq, D]
  const int* seqlens;          // [B]
  PagedRows c;
  float* o_part;               // [B, Hq, S, D]
  float* lse_part;             // [B, Hq, S], natural log
  __nv_bfloat16* o;            // [B, Hq, D]
  float* lse;                  // [B, Hq]
  unsigned long long* counts;  // {skipped, visited} or null
  uint8_t* tile_state;         // [B, Hkv, n_k_max] or null
  int B, Hq, Hkv, G, S, n_k_max;
  int clustered;               // the S splits of a head are one cluster, which merges them
  float scale_log2, tsf;
};

constexpr int kPgTile = 64;
constexpr int kPgWarps = 4;                          // consumer warps
constexpr int kPgThreads = (kPgWarps + 1) * 32;
constexpr int kPgLag = 2;                            // P.V runs this many tiles behind the vote

// A split's result for the merge over its cluster: lse and the normalised O of
// its heads, in shared memory that nothing else uses any more.
template <int D>
struct PagedPart {
  float lse[8], o[8][D];
};

template <int D>
struct PagedCfg {
  static constexpr int kTileBytes = kPgTile * D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;  // of K and of V
  static constexpr int kCtas = 2;                   // per SM
  static constexpr int kK = 0;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kMax = kV + kStages * kTileBytes;        // [2][8][W] fp32
  static constexpr int kStat = kMax + 2 * 8 * kPgWarps * 4;     // [W][8] (m, l)
  static constexpr int kIds = kStat + kPgWarps * 8 * 8;         // [stages][4] pages of a tile
  static constexpr int kBar = kIds + kStages * 16;
  static constexpr int kTotal = kBar + 4 * kStages * 8 + 16;
  static constexpr int kAlloc = kTotal + 1024;                  // the ring starts 1024-aligned
  static constexpr int kPart = kPgWarps * 8 * (D + 4) * 4;      // behind the merge of the warps
  static_assert(kPart + (int)sizeof(PagedPart<D>) <= kMax, "both merges fit the rings");
  static_assert(kStages > kPgLag, "a V slot is free again when its next tile is voted on");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What the rounding of a pair to bf16 left over, in bf16.
__device__ __forceinline__ uint32_t pack_rest(float x, float y, uint32_t rounded) {
  return pack_bf16x2(x - __uint_as_float(rounded << 16), y - __uint_as_float(rounded & 0xFFFF0000u));
}

// The splits of a head merged by the cluster they are, each CTA writing its
// share of the columns: one launch and no trip through memory where a call is
// short.  All threads of all its CTAs call, also of those whose split was empty
// or gave up (they left lse = -inf).
template <int D>
__device__ __forceinline__ void paged_cluster_merge(const PagedDecodeParams& p,
                                                    const PagedPart<D>* part, size_t head0, int tid,
                                                    int threads) {
  __syncwarp();
  cluster_sync();  // every CTA's part is written
  const uint32_t lse0 = smem_u32(part->lse), o0 = smem_u32(part->o);
  for (int i = (int)cluster_rank() * threads + tid; i < p.G * D; i += p.S * threads) {
    const int h = i / D;
    float l[8], mx = -INFINITY;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      l[s] = s < p.S ? ld_cluster(lse0 + h * 4, s) : -INFINITY;
      mx = fmaxf(mx, l[s]);
    }
    float sum = 0.f, o = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s >= p.S || l[s] == -INFINITY) continue;  // an empty split left no O
      const float w = __expf(l[s] - mx);
      sum += w;
      o = fmaf(w, ld_cluster(o0 + i * 4, s), o);
    }
    // Every split empty (a sequence of length 0): O = 0 and lse = -inf.  A split
    // of NaN has a NaN lse, which the maximum drops and the sum keeps.
    p.o[head0 * D + i] = __float2bfloat16_rn(sum == 0.f ? 0.f : o / sum);
    if (i % D == 0) p.lse[head0 + h] = sum == 0.f ? -INFINITY : mx + __logf(sum);
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another may read its shared memory
}

// What a split without tiles leaves: nothing for the merge to weigh, or (with
// one split) the empty sequence's O = 0 and lse = -inf.
template <int D>
__device__ __forceinline__ void paged_empty_split(const PagedDecodeParams& p, PagedPart<D>* part,
                                                  size_t head0, int split, int tid, int threads) {
  if (p.S == 1) {
    for (int i = tid; i < p.G * D; i += threads) p.o[head0 * D + i] = __float2bfloat16_rn(0.f);
    if (tid < p.G) p.lse[head0 + tid] = -INFINITY;
  } else if (p.clustered) {
    if (tid < 8) part->lse[tid] = -INFINITY;
  } else if (tid < p.G) {
    p.lse_part[(head0 + tid) * p.S + split] = -INFINITY;
  }
}

// How the lanes of a warp share a tile's copies.  A tile of 64 rows comes in
// 64 / rows copies (one when a page holds a tile), a bf16 row of 128 values in
// two 128-byte-wide halves, and K and V tiles may go out together: every copy
// is one lane's, so issuing a tile costs the warp one pass through the code.
struct PagedLane {
  int shift, rows, row_shift, npt;  // page size, rows of a copy, copies of a tile
  int sub, half, val;               // this lane's copy, half, and K (0) or V (1)
  __device__ __forceinline__ PagedLane(const PagedRows& c, int lane) {
    shift = c.page_shift;
    row_shift = min(shift, 6);
    rows = 1 << row_shift;
    npt = kPgTile >> row_shift;
    sub = lane & 3;
    half = (lane >> 2) & 1;
    val = (lane >> 3) & 1;
  }
  // Copies of tile j that hold a key: those behind the last one are not fetched.
  __device__ __forceinline__ int copies(int j, int len) const {
    return min(npt, (len - j * kPgTile + rows - 1) >> row_shift);
  }
  // Row of the pools (pages, heads and rows flattened) of this lane's copy.
  __device__ __forceinline__ long long row(int j, int page, int Hkv, int kvh) const {
    const int off = (j * kPgTile + sub * rows) & ((1 << shift) - 1);
    return (((long long)page * Hkv + kvh) << shift) + off;
  }
  __device__ __forceinline__ int slot(int j) const { return (j * kPgTile + sub * rows) >> shift; }
};

// A page outside the pool is latched and read as page 0.
__device__ __forceinline__ int paged_checked(const PagedRows& c, int page) {
  if (page >= 0 && page < c.num_pages) return page;
  latch_status(kStatusInvalidArg);
  return 0;
}

// row_passes_log2 for a positive threshold, without its branches (only
// (-inf) - (-inf) needs a word of its own).  The maxima come from max_nan: a tile
// with a NaN score, or one behind it in its split, has a NaN here, is below no
// border and is kept, so that the NaN reaches the outputs.
__device__ __forceinline__ bool paged_head_passes(float local, float run, float log2_t, bool idle) {
  return idle | (local == -INFINITY) | (local - run < log2_t);
}

struct PagedCell {
  int d;
  float x;
};

// Merge W warps' O^T, references m (log2 units) and row sums l of heads 2 c,
// 2 c + 1 (the same at every g), and write the split, or the result when it is the only
// one.  cell(mt, i): column and value of accumulator i of row tile mt.  red:
// W * 8 * (D + 4) floats of shared memory that nothing else uses any more.
template <int D, int W, typename Cell>
__device__ __forceinline__ void paged_merge_warps(const PagedDecodeParams& p, float* red,
                                                  float2* stat, size_t head0, int split, int tid,
                                                  const float (&m)[2], const float (&l)[2],
                                                  PagedPart<D>* part, Cell cell) {
  constexpr int RS = D + 4;  // row stride of the merge buffer: spreads the banks
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const PagedCell e = cell(mt, i);
      red[(warp * 8 + 2 * c + (i & 1)) * RS + e.d] = e.x;
    }
  if (g == 0) {
    stat[warp * 8 + 2 * c] = make_float2(m[0], l[0]);
    stat[warp * 8 + 2 * c + 1] = make_float2(m[1], l[1]);
  }
  named_bar_sync(1, W * 32);
  for (int i = tid; i < p.G * D; i += W * 32) {
    const int h = i / D, d = i % D;
    float2 st[W];
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      st[w] = stat[w * 8 + h];
      mx = fmaxf(mx, st[w].x);
    }
    float sum = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float e = st[w].x == -INFINITY ? 0.f : ex2_approx(st[w].x - mx);
      sum = fmaf(e, st[w].y, sum);
      o = fmaf(e, red[(w * 8 + h) * RS + d], o);
    }
    const float lse = (mx + __log2f(sum)) * 0.69314718055994531f;
    if (p.S == 1) {
      // Scores that are all -inf: O = 0, as the merges of several splits leave it.
      p.o[(head0 + h) * D + d] = __float2bfloat16_rn(sum == 0.f ? 0.f : o / sum);
      if (d == 0) p.lse[head0 + h] = lse;
    } else if (p.clustered) {
      part->o[h][d] = o / sum;
      if (d == 0) part->lse[h] = lse;
    } else {
      p.o_part[((head0 + h) * p.S + split) * D + d] = o / sum;
      if (d == 0) p.lse_part[(head0 + h) * p.S + split] = lse;
    }
  }
}

template <int D, bool SKIP>
__global__ void __launch_bounds__(kPgThreads, PagedCfg<D>::kCtas)
    decode_paged_kernel(const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const PagedDecodeParams p) {
  using C = PagedCfg<D>;
  constexpr int NS = C::kStages;
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBar + 4 * NS * 8);
  int* ids = reinterpret_cast<int*>(smem + C::kIds);
  const uint32_t k_smem = smem_u32(smem + C::kK), v_smem = smem_u32(smem + C::kV);
  auto kfull = [&](int s) { return smem_u32(&bars[s]); };
  auto kfree = [&](int s) { return smem_u32(&bars[NS + s]); };
  auto vfull = [&](int s) { return smem_u32(&bars[2 * NS + s]); };
  auto vfree = [&](int s) { return smem_u32(&bars[3 * NS + s]); };
  if (tid == 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    for (int s = 0; s < NS; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(kfree(s), kPgWarps);
      mbar_init(vfull(s), 1);
      mbar_init(vfree(s), kPgWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }

  wait_for_previous_kernel();
  launch_dependents();
  // seqlens[b] lies in [0, max_pages * P]: another length is latched and
  // clamped, so that no page number is read outside the sequence's table row.
  const int cap = p.c.max_pages << p.c.page_shift;
  const int Lraw = p.seqlens[b];
  if ((Lraw < 0 || Lraw > cap) && tid == 0 && split == 0 && kvh == 0)
    latch_status(kStatusInvalidArg);
  const int Lb = min(max(Lraw, 0), cap);
  const int n_k = (Lb + kPgTile - 1) / kPgTile;
  const int c_per = (n_k + p.S - 1) / p.S;
  const int j0 = split * c_per;
  const int ntiles = max(0, min(n_k, j0 + c_per) - j0);
  const size_t head0 = (size_t)b * p.Hq + (size_t)kvh * p.G;

  auto* part = reinterpret_cast<PagedPart<D>*>(smem + C::kPart);
  if (ntiles == 0) {
    paged_empty_split<D>(p, part, head0, split, tid, kPgThreads);
    if (p.clustered) paged_cluster_merge<D>(p, part, head0, tid, kPgThreads);
    return;
  }
  __syncthreads();

  // A whole warp: tile j's copies of K (val = 0) or V into ring slot s; each
  // lane brings the page of its copy.
  const PagedLane ln(p.c, lane);
  const uint32_t copy_bytes = (uint32_t)ln.rows * 128;  // of one half
  auto fetch = [&](int val, bool on, int j, int s, int page) {
    const uint32_t bar = val ? vfull(s) : kfull(s);
    const uint32_t dst = (val ? v_smem : k_smem) + s * C::kTileBytes;
    const int n = ln.copies(j, Lb);
    const bool ok = dev_check(j < n_k && n >= 1 && n <= 4 && s < NS);
    if (on && ln.sub == 0 && ln.half == 0) {
      if (ok) mbar_arrive_expect_tx(bar, n * copy_bytes * (D / 64));
      else mbar_arrive(bar);  // the phase completes without data
    }
    __syncwarp();
    if (on && ok && ln.sub < n && ln.half < D / 64)
      tma_load_2d(dst + ln.half * (kPgTile * 128) + ln.sub * copy_bytes, val ? &map_v : &map_k, bar,
                  ln.half * 64, (int)ln.row(j, page, p.Hkv, kvh));
  };

  if (warp == kPgWarps) {
    // ------------------------------------------------------------ producer
    const int* table = p.c.block_table + (size_t)b * p.c.max_pages;
    const int val = SKIP ? 0 : ln.val;
    const bool mine = lane < (SKIP ? 8 : 16) && ln.half < D / 64;
    // The page of this lane's copy of a tile, loaded a tile ahead.
    auto page_of = [&](int j) {
      return mine && j < n_k && ln.sub < ln.copies(j, Lb) ? table[ln.slot(j)] : 0;
    };
    int issued = 0, s = 0, par = 1, next = page_of(j0);
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int j = j0 + t, page = paged_checked(p.c, next);
      next = page_of(j + 1);
      if (t >= NS) ok = mbar_wait(val ? vfree(s) : kfree(s), par, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (SKIP && mine && ln.half == 0) ids[s * 4 + ln.sub] = page;
      __syncwarp();
      fetch(val, mine, j, s, page);
      issued = t + 1;
      if (++s == NS) { s = 0; par ^= 1; }
    }
    __syncthreads();
    if (*abort_flag && lane == 0) {  // wait out the copies in flight before the CTA exits
      int no_abort = 0;
      for (int i = 0; i < NS; ++i)
        if (issued > i) {
          mbar_wait(kfull(i), ((issued - 1 - i) / NS) & 1, &no_abort);
          if (!SKIP) mbar_wait(vfull(i), ((issued - 1 - i) / NS) & 1, &no_abort);
        }
    }
    __syncwarp();
    if (p.clustered) paged_cluster_merge<D>(p, part, head0, tid, kPgThreads);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  // Q^T fragments: head g, the d's that the K fragments hold at this lane.
  uint32_t qf[MT][2];
  {
    const __nv_bfloat16* q = p.q + (head0 + g) * D;
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = kt * 16 + i * 8 + 2 * c;
        qf[kt][i] = g < p.G ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
      }
  }
  float* wmax = reinterpret_cast<float*>(smem + C::kMax);
  const bool idle[2] = {2 * c >= p.G, 2 * c + 1 >= p.G};  // padding heads always pass
  const float log2_t = SKIP ? (float)log2((double)p.tsf / (double)Lb) : -INFINITY;

  float acc[MT][4];                 // O^T
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2 c, 2 c + 1
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

  // Scores of this warp's 16 keys of tile t, in log2 units: s[0..1] key g,
  // s[2..3] key g + 8, heads 2 c and 2 c + 1; keys past the end -> -inf.
  auto scores = [&](int t, float (&s)[4]) {
    const int valid = Lb - (j0 + t) * kPgTile - warp * 16;  // of the 16
    const uint8_t* tile = smem + C::kK + (t % NS) * C::kTileBytes;
    const uint32_t base = smem_u32(tile) + warp * 16 * 128;
    const int row = (lane & 7) + ((lane >> 3) & 1) * 8, ch = lane >> 4;
    float x[2][4] = {};
#pragma unroll
    for (int kt = 0; kt < MT; ++kt) {
      const int chunk = kt * 2 + ch;
      uint32_t a[4];
      ldsm4(base + (chunk >> 3) * (kPgTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), a);
      mma16816(x[kt & 1], a[0], a[1], a[2], a[3], qf[kt][0], qf[kt][1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = x[0][i] + x[1][i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s[i] = (g + (i >> 1) * 8 < valid) ? s[i] * p.scale_log2 : -INFINITY;
  };

  // O^T = a O^T + V^T P^T over this warp's 16 keys of tile t, from ring slot t % NS.
  auto accumulate = [&](int t, const float (&pr)[4], float a0, float a1) {
    const int valid = Lb - (j0 + t) * kPgTile - warp * 16;
    uint8_t* tile = smem + C::kV + (t % NS) * C::kTileBytes;
    if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][0] *= a0; acc[i][1] *= a1; acc[i][2] *= a0; acc[i][3] *= a1;
      }
    }
    if (valid <= 0) return;
    if (valid < 16) {  // rows behind the last key: P is 0 there, V may be NaN
      for (int i = lane; i < (16 - valid) * 8; i += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          *reinterpret_cast<uint4*>(tile + h * (kPgTile * 128) +
                                    (warp * 16 + valid + (i >> 3)) * 128 + (i & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    // P goes into the product as two bf16 parts, its rounding and the rest's
    // (within 2^-16 of each weight): twice the products, in the shadow of HBM
    // (64 x 16K-32K 896 us with one part or two, factor 500 647 and 650).
    const uint32_t h0 = pack_bf16x2(pr[0], pr[1]), h1 = pack_bf16x2(pr[2], pr[3]);
    const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
    const uint32_t r0 = transpose8x8(pack_rest(pr[0], pr[1], h0));
    const uint32_t r1 = transpose8x8(pack_rest(pr[2], pr[3], h1));
    const uint32_t base = smem_u32(tile) + warp * 16 * 128;
    const int row = (lane & 7) + (lane >> 4) * 8, ch = (lane >> 3) & 1;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int chunk = mt * 2 + ch;
      uint32_t a[4];
      ldsm4_t(base + (chunk >> 3) * (kPgTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4),
              a);
      mma16816(acc[mt], a[0], a[1], a[2], a[3], b0, b1);
      mma16816(acc[mt], a[0], a[1], a[2], a[3], r0, r1);
    }
  };

  int n_skipped = 0;
  uint32_t v_used = 0, v_par = 0;  // warp 0: V slots in use, parity of their last copy
  if constexpr (!SKIP) {
    for (int t = 0; t < ntiles; ++t) {
      const int s = t % NS;
      mbar_wait(kfull(s), (t / NS) & 1, abort_flag);
      float x[4];
      scores(t, x);
      __syncwarp();
      if (lane == 0) mbar_arrive(kfree(s));
      // The reference moves only when a score is 2^8 above it: P stays below
      // 2^8 and most tiles need no exchange between the lanes.
      float a[2] = {1.f, 1.f};
      float top[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
      if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
          const float mn = fmaxf(m[i], top[i]);
          a[i] = (m[i] == -INFINITY) ? 0.f : ex2_approx(m[i] - mn);
          m[i] = mn;
          l[i] *= a[i];
        }
      }
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ref = m[i & 1] == -INFINITY ? 0.f : m[i & 1];
        pr[i] = ex2_approx(x[i] - ref);
        l[i & 1] += pr[i];
      }
      if (p.tile_state && tid == 0)
        p.tile_state[((size_t)b * p.Hkv + kvh) * p.n_k_max + j0 + t] = 1;
      mbar_wait(vfull(s), (t / NS) & 1, abort_flag);
      accumulate(t, pr, a[0], a[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(vfree(s));
    }
  } else {
    float pr[kPgLag][4], al[kPgLag][2];
    uint32_t kept = 0, v_phase = 0;  // kept: bit 0 the last tile, bit 1 the one before
#pragma unroll
    for (int i = 0; i < kPgLag; ++i) {
      pr[i][0] = pr[i][1] = pr[i][2] = pr[i][3] = 0.f;
      al[i][0] = al[i][1] = 1.f;
    }
    for (int t = 0; t < ntiles + kPgLag; ++t) {
      const bool live = t < ntiles;
      float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      int page = 0;
      if (live) {
        const int s = t % NS;
        mbar_wait(kfull(s), (t / NS) & 1, abort_flag);
        if (warp == 0) page = ids[s * 4 + ln.sub];
        scores(t, x);
        __syncwarp();
        if (lane == 0) mbar_arrive(kfree(s));
        float top[2] = {max_nan(x[0], x[2]), max_nan(x[1], x[3])};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top[i] = max_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
          if (g == 0) wmax[((t & 1) * 8 + 2 * c + i) * kPgWarps + warp] = top[i];
        }
      }
      named_bar_sync(1, kPgWarps * 32);  // maxima of tile t published; P.V of t - 1 - kLag done
      float np[4] = {0.f, 0.f, 0.f, 0.f}, na[2] = {1.f, 1.f};
      bool keep = false;
      if (live) {
        float top[2];
        bool pass = true;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(&wmax[((t & 1) * 8 + 2 * c + i) * kPgWarps]);
          top[i] = max_nan(max_nan(w.x, w.y, w.z), w.w);
          pass &= paged_head_passes(top[i], m[i], log2_t, idle[i]);
        }
        keep = !__all_sync(0xffffffffu, pass);
        if (keep) {
          if (warp == 0) {
            const bool go = __all_sync(0xffffffffu, !*abort_flag);
            fetch(1, go && lane < 8, j0 + t, t % NS, page);
            if (go) {
              v_used |= 1u << (t % NS);
              v_par ^= 1u << (t % NS);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = max_nan(m[i], top[i]);
            na[i] = (m[i] == -INFINITY) ? 0.f : ex2_approx(m[i] - mn);
            m[i] = mn;
            l[i] *= na[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            np[i] = ex2_approx(x[i] - (m[i & 1] == -INFINITY ? 0.f : m[i & 1]));
            l[i & 1] += np[i];
          }
        } else {
          n_skipped += 1;
        }
        if (p.tile_state && tid == 0)
          p.tile_state[((size_t)b * p.Hkv + kvh) * p.n_k_max + j0 + t] = keep ? 1 : 2;
      }
      const int u = t - kPgLag;
      if (u >= 0 && ((kept >> (kPgLag - 1)) & 1)) {
        const int s = u % NS;
        mbar_wait(vfull(s), (v_phase >> s) & 1, abort_flag);
        v_phase ^= 1u << s;
        accumulate(u, pr[kPgLag - 1], al[kPgLag - 1][0], al[kPgLag - 1][1]);
      }
      kept = (kept << 1) | (keep ? 1u : 0u);
#pragma unroll
      for (int i = kPgLag - 1; i >= 0; --i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[i][k] = i ? pr[i - 1][k] : np[k];
        al[i][0] = i ? al[i - 1][0] : na[0];
        al[i][1] = i ? al[i - 1][1] : na[1];
      }
    }
  }

  // ---- merge the warps; write the split.
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  __syncthreads();  // with the producer: every warp is past its last use of the rings
  if (*abort_flag) {
    if (SKIP && tid == 0) {
      int no_abort = 0;
      for (int s = 0; s < NS; ++s)
        if ((v_used >> s) & 1) mbar_wait(vfull(s), ((v_par >> s) & 1) ^ 1, &no_abort);
    }
    if (p.clustered) {
      if (tid < 8) part->lse[tid] = -INFINITY;
      paged_cluster_merge<D>(p, part, head0, tid, kPgThreads);
    }
    return;
  }
  paged_merge_warps<D, kPgWarps>(p, reinterpret_cast<float*>(smem),
                                 reinterpret_cast<float2*>(smem + C::kStat), head0, split, tid, m,
                                 l, part, [&](int mt, int i) {
                                   return PagedCell{mt * 16 + g + (i >> 1) * 8, acc[mt][i]};
                                 });
  if (tid == 0 && p.counts) {
    atomicAdd(&p.counts[0], (unsigned long long)n_skipped);
    atomicAdd(&p.counts[1], (unsigned long long)ntiles);
  }
  if (p.clustered) paged_cluster_merge<D>(p, part, head0, tid, kPgThreads);
}

// Merge the splits of one (sequence, query head).
template <int D>
__global__ void __launch_bounds__(128) decode_paged_combine_kernel(const PagedDecodeParams p) {
  const size_t bh = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* lp = p.lse_part + bh * p.S;
  __shared__ float w_s[64];
  __shared__ float red[4][D];
  __shared__ float sum_s;
  wait_for_previous_kernel();
  launch_dependents();
  if (warp == 0) {
    const float a = lane < p.S ? lp[lane] : -INFINITY;
    const float e = lane + 32 < p.S ? lp[lane + 32] : -INFINITY;
    float mx = fmaxf(a, e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float wa = a == -INFINITY ? 0.f : __expf(a - mx);
    const float we = e == -INFINITY ? 0.f : __expf(e - mx);
    float sum = wa + we;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w_s[lane] = wa;
    w_s[lane + 32] = we;
    if (lane == 0) {
      sum_s = sum;
      // Every split empty (a sequence of length 0): O = 0 and lse = -inf.  A split
      // of NaN has a NaN lse, which the maximum drops and the sum keeps.
      p.lse[bh] = sum == 0.f ? -INFINITY : mx + __logf(sum);
    }
  }
  __syncthreads();
  constexpr int V = D / 32;  // columns of a lane
  float o[V] = {};
  for (int s = warp; s < p.S; s += 4) {
    const float w = w_s[s];
    if (w == 0.f) continue;  // an empty split wrote no partial
    const float* part = p.o_part + (bh * p.S + s) * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(w, part[i], o[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) red[warp][lane * V + i] = o[i];
  __syncthreads();
  for (int d = tid; d < D; d += 128) {
    const float x = red[0][d] + red[1][d] + red[2][d] + red[3][d];
    const float sum = sum_s;
    p.o[bh * D + d] = __float2bfloat16_rn(sum == 0.f ? 0.f : x / sum);
  }
}

}  // namespace sskip
