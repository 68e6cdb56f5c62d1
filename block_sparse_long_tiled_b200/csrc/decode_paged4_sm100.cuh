// decode_paged4_sm100.cuh -- the split-KV Skip-Softmax decode over 4-bit pages.
//
// The rule, the grid and the products are those of the bf16 kernel
// (decode_paged_sm100.cuh); what differs is what bounds it.  A tile is a
// quarter of the bytes, so the instructions that widen the codes decide: a
// consumer warp therefore owns WHOLE tiles (tile t belongs to warp t mod 4),
// which spreads everything that is not widening -- waits, the reference check,
// the vote -- over 64 keys instead of 16.
//
// Keys: S = sum over groups of sc (q . (n - 8)) + (8 sc + mn) sum(q).  The codes
// enter the tensor cores as the exact bf16 integers n - 8; a group's scale
// multiplies its 32-term product in fp32; the last term is one more product,
// of the record's own (sc, mn) pairs with (8 sum q, sum q) split into three
// bf16 parts that together hold its 24 bits.
// Values: the group's scale joins P before the rounding to bf16, the part that
// does not depend on the code, P (8 sc + mn), is summed in fp32.
//
// With a threshold the warps take one decision for four tiles at a time: each
// publishes its tile's maxima, and after one named barrier all walk the four
// tiles in order under the rule.  The scores wait in shared memory for the V
// tile, which is fetched after the decision and used one round later.
#pragma once

#include "decode_paged_sm100.cuh"

namespace sskip {

constexpr int kP4Warps = 4;                      // consumer warps
constexpr int kP4Threads = (kP4Warps + 1) * 32;

template <int D, bool SKIP>
struct Paged4Cfg {
  static constexpr int kTileBytes = 4 * Kv4<D>::kRecord;
  static constexpr int kNK = 2 * kP4Warps;           // ring slots of K
  static constexpr int kNV = 2 * kP4Warps;
  static constexpr int kCtas = 2;                    // per SM
  static constexpr int kK = 0;
  static constexpr int kV = kK + kNK * kTileBytes;
  static constexpr int kS = kV + kNV * kTileBytes;  // [W][2][64][8] fp32 scores
  static constexpr int kMax = kS + (SKIP ? kP4Warps * 2 * kPgTile * 8 * 4 : 0);  // [2][8][W]
  static constexpr int kStat = kMax + 2 * 8 * kP4Warps * 4;    // [W][8] (m, l)
  static constexpr int kIds = kStat + kP4Warps * 8 * 8;        // [NK][4] pages of a tile
  static constexpr int kBar = kIds + kNK * 16;
  static constexpr int kTotal = kBar + 2 * (kNK + kNV) * 8 + 16;
  static_assert(kP4Warps * 8 * (D + 4) * 4 <= kS, "the merge of the warps fits the rings");
  // Every slot belongs to one warp: only then does that warp wait for the
  // slot's phases one after the other, and no parity can be an older phase's.
  static_assert(kNK % kP4Warps == 0 && kNV % kP4Warps == 0, "a slot's tiles belong to one warp");
};

// The four pairs of a 4-bit word as bf16 pairs n - 8: the code under the
// exponent of 128 is 128 + n, and taking 136 away is exact.
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t (&r)[4]) {
  const __nv_bfloat162 bias = __halves2bfloat162(__ushort_as_bfloat16(0x4308),
                                                 __ushort_as_bfloat16(0x4308));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), bias);
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// N words of shared memory, aligned to N * 4 bytes (N = 2 or 4).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

template <int D, bool SKIP>
__global__ void __launch_bounds__(kP4Threads, Paged4Cfg<D, SKIP>::kCtas)
    decode_paged4_kernel(const PagedDecodeParams p) {
  using C = Paged4Cfg<D, SKIP>;
  constexpr int NK = C::kNK, NV = C::kNV, W = kP4Warps;
  constexpr int NG = D / 32;   // groups of a row
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  constexpr int REC = Kv4<D>::kRecord, CODES = Kv4<D>::kCodes;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

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
  if (ntiles == 0) {
    paged_empty_split<D>(p, head0, split, tid, kP4Threads);
    return;
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBar + 2 * (NK + NV) * 8);
  int* ids = reinterpret_cast<int*>(smem + C::kIds);
  const uint32_t k_smem = smem_u32(smem + C::kK), v_smem = smem_u32(smem + C::kV);
  auto kfull = [&](int s) { return smem_u32(&bars[s]); };
  auto kfree = [&](int s) { return smem_u32(&bars[NK + s]); };
  auto vfull = [&](int s) { return smem_u32(&bars[2 * NK + s]); };
  auto vfree = [&](int s) { return smem_u32(&bars[2 * NK + NV + s]); };
  if (tid == 0) {
    for (int s = 0; s < 2 * (NK + NV); ++s) mbar_init(smem_u32(&bars[s]), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  // A whole warp: tile j's copies of K (val = 0) or V into ring slot s; each
  // lane brings the page of its copy.
  const PagedLane ln(p.c, lane);
  const uint32_t copy_bytes = (uint32_t)(ln.rows >> 4) * REC;
  auto fetch = [&](int val, bool on, int j, int s, int page) {
    const uint32_t bar = val ? vfull(s) : kfull(s);
    const uint32_t dst = (val ? v_smem : k_smem) + s * C::kTileBytes;
    const int n = ln.copies(j, Lb);
    const bool ok = dev_check(j < n_k && n >= 1 && n <= 4 && s < (val ? NV : NK));
    if (on && ln.sub == 0 && ln.half == 0) {
      if (ok) mbar_arrive_expect_tx(bar, n * copy_bytes);
      else mbar_arrive(bar);  // the phase completes without data
    }
    __syncwarp();
    if (on && ok && ln.sub < n && ln.half == 0)
      bulk_load(dst + ln.sub * copy_bytes,
                (val ? p.c.v_pages : p.c.k_pages) + ln.row(j, page, p.Hkv, kvh) * (REC / 16),
                copy_bytes, bar);
  };

  if (warp == W) {
    // ------------------------------------------------------------ producer
    const int* table = p.c.block_table + (size_t)b * p.c.max_pages;
    const int val = SKIP ? 0 : ln.val;
    const bool mine = lane < (SKIP ? 8 : 16) && ln.half == 0;
    // The page of this lane's copy of a tile, loaded a tile ahead.
    auto page_of = [&](int j) {
      return mine && j < n_k && ln.sub < ln.copies(j, Lb) ? __ldg(table + ln.slot(j)) : 0;
    };
    static_assert(SKIP || NK == NV, "one slot counter for both rings");
    int issued = 0, s = 0, par = 1, next = page_of(j0);
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int j = j0 + t, page = paged_checked(p.c, next);
      next = page_of(j + 1);
      if (t >= NK) ok = mbar_wait(val ? vfree(s) : kfree(s), par, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (SKIP && mine) ids[s * 4 + ln.sub] = page;
      __syncwarp();
      fetch(val, mine, j, s, page);
      issued = t + 1;
      if (++s == NK) { s = 0; par ^= 1; }
    }
    __syncthreads();
    if (*abort_flag && lane == 0) {  // wait out the copies in flight before the CTA exits
      int no_abort = 0;
      for (int i = 0; i < NK; ++i)
        if (issued > i) {
          mbar_wait(kfull(i), ((issued - 1 - i) / NK) & 1, &no_abort);
          if (!SKIP) mbar_wait(vfull(i), ((issued - 1 - i) / NK) & 1, &no_abort);
        }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  // Q^T fragments of head g: the d's that the key words hold at this lane.
  uint32_t qf[MT][2];
  uint32_t zf[3] = {0u, 0u, 0u};  // (8 sum q, sum q) of group c, in three bf16 parts
  {
    const __nv_bfloat16* q = p.q + (head0 + g) * D;
#pragma unroll
    for (int kt = 0; kt < MT; ++kt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = (kt >> 1) * 32 + 8 * c + 2 * ((kt & 1) * 2 + i);
        qf[kt][i] = g < p.G ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
      }
    float mine = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = qf[2 * gr + (i >> 1)][i & 1];
        s += __uint_as_float(w << 16) + __uint_as_float(w & 0xFFFF0000u);
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (c == gr) mine = s;
    }
    float x = 8.f * mine, y = mine;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      zf[i] = pack_bf16x2(x, y);
      x -= __uint_as_float(zf[i] << 16);
      y -= __uint_as_float(zf[i] & 0xFFFF0000u);
    }
  }
  const float log2_t = SKIP ? (float)log2((double)p.tsf / (double)Lb) : -INFINITY;
  const float sl = p.scale_log2;

  float acc[MT][4];    // O^T
  float zacc[NG][2];   // sum of p (8 sc + mn)
  float l[2] = {0.f, 0.f};  // heads 2 c, 2 c + 1
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
  for (int i = 0; i < NG; ++i) zacc[i][0] = zacc[i][1] = 0.f;

  // Logits (before sm_scale) of a record's 16 keys: x[0..1] key g, x[2..3] key
  // g + 8, heads 2 c and 2 c + 1; the keys from `valid` on -> -inf.
  auto scores = [&](const uint8_t* rec, int valid, float (&x)[4]) {
    uint32_t wa[NG], wb[NG], pa[NG], pb[NG];
    lds_words<NG>(wa, rec + g * (D / 2) + c * NG * 4);
    lds_words<NG>(wb, rec + (g + 8) * (D / 2) + c * NG * 4);
    lds_words<NG>(pa, rec + CODES + g * NG * 4);
    lds_words<NG>(pb, rec + CODES + (g + 8) * NG * 4);
    const uint32_t z0 = *reinterpret_cast<const uint32_t*>(rec + CODES + (g * NG + (c % NG)) * 4);
    const uint32_t z1 = *reinterpret_cast<const uint32_t*>(rec + CODES + ((g + 8) * NG + (c % NG)) * 4);
    x[0] = x[1] = x[2] = x[3] = 0.f;
    mma16816(x, z0, z1, z0, z1, zf[0], zf[1]);
    mma16816(x, z0, z1, z0, z1, zf[2], 0u);
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      uint32_t a[4], e[4];
      widen_codes(wa[gr], a);
      widen_codes(wb[gr], e);
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      mma16816(y, a[0], e[0], a[1], e[1], qf[2 * gr][0], qf[2 * gr][1]);
      mma16816(y, a[2], e[2], a[3], e[3], qf[2 * gr + 1][0], qf[2 * gr + 1][1]);
      const float sa = __uint_as_float(pa[gr] << 16), sb = __uint_as_float(pb[gr] << 16);
      x[0] = fmaf(sa, y[0], x[0]);
      x[1] = fmaf(sa, y[1], x[1]);
      x[2] = fmaf(sb, y[2], x[2]);
      x[3] = fmaf(sb, y[3], x[3]);
    }
    if (valid < 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (g + (i >> 1) * 8 >= valid) x[i] = -INFINITY;
    }
  };

  // O^T += V^T P^T over a record's 16 keys.
  auto accumulate = [&](const uint8_t* rec, int valid, const float (&pr)[4]) {
    uint32_t w0[NG], w1[NG], pa[NG], pb[NG];
    lds_words<NG>(w0, rec + lane * NG * 4);
    lds_words<NG>(w1, rec + (32 + lane) * NG * 4);
    lds_words<NG>(pa, rec + CODES + g * NG * 4);
    lds_words<NG>(pb, rec + CODES + (g + 8) * NG * 4);
    if (valid < 16) {
      // Behind the last key the record holds what an earlier sequence left:
      // its codes are numbers, its scales need not be.
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        if (g >= valid) pa[gr] = 0u;
        if (g + 8 >= valid) pb[gr] = 0u;
      }
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const float sa = __uint_as_float(pa[gr] << 16), sb = __uint_as_float(pb[gr] << 16);
      const float za = fmaf(8.f, sa, __uint_as_float(pa[gr] & 0xFFFF0000u));
      const float zb = fmaf(8.f, sb, __uint_as_float(pb[gr] & 0xFFFF0000u));
      zacc[gr][0] = fmaf(pr[0], za, fmaf(pr[2], zb, zacc[gr][0]));
      zacc[gr][1] = fmaf(pr[1], za, fmaf(pr[3], zb, zacc[gr][1]));
      // The scale joins P before its rounding to bf16 (2^-8 of the product).
      const uint32_t b0 = transpose8x8(pack_bf16x2(pr[0] * sa, pr[1] * sa));
      const uint32_t b1 = transpose8x8(pack_bf16x2(pr[2] * sb, pr[3] * sb));
      uint32_t a[4], e[4];
      widen_codes(w0[gr], a);
      widen_codes(w1[gr], e);
      mma16816(acc[2 * gr], a[0], a[1], e[0], e[1], b0, b1);
      mma16816(acc[2 * gr + 1], a[2], a[3], e[2], e[3], b0, b1);
    }
  };

  auto rescale = [&](float a0, float a1) {
    if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][0] *= a0; acc[i][1] *= a1; acc[i][2] *= a0; acc[i][3] *= a1;
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) { zacc[i][0] *= a0; zacc[i][1] *= a1; }
      l[0] *= a0;
      l[1] *= a1;
    }
  };

  float m[2] = {-INFINITY, -INFINITY};  // reference of heads 2 c, 2 c + 1, in log2 units
  int n_skipped = 0;
  // SKIP: this warp's two V slots: fetched into (and the parity of the last
  // copy), and the phase to wait for next.
  uint32_t v_used = 0, v_par = 0, v_phase = 0;
  if constexpr (!SKIP) {
    float mm[2] = {0.f, 0.f};  // m, or 0 while it is -inf
    int ks = warp, kp = 0, vs = warp, vp = 0;
    for (int t = warp; t < ntiles; t += W) {
      mbar_wait(kfull(ks), kp, abort_flag);
      mbar_wait(vfull(vs), vp, abort_flag);
      const int left = Lb - (j0 + t) * kPgTile;
      const uint8_t* krec = smem + C::kK + ks * C::kTileBytes;
      const uint8_t* vrec = smem + C::kV + vs * C::kTileBytes;
#pragma unroll 1
      for (int i = 0; i < 4 && i * 16 < left; ++i) {
        float x[4];
        scores(krec + i * REC, left - i * 16, x);
        // The reference moves only when a score is 2^8 above it: P stays
        // below 2^8 and most records need no exchange between the lanes.
        float top[2] = {fmaxf(x[0], x[2]) * sl, fmaxf(x[1], x[3]) * sl};
        if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
          float a[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
              top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
            const float mn = fmaxf(m[h], top[h]);
            a[h] = (m[h] == -INFINITY) ? 0.f : ex2_approx(m[h] - mn);
            m[h] = mn;
            mm[h] = mn == -INFINITY ? 0.f : mn;
          }
          rescale(a[0], a[1]);
        }
        float pr[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          pr[h] = ex2_approx(fmaf(x[h], sl, -mm[h & 1]));
          l[h & 1] += pr[h];
        }
        accumulate(vrec + i * REC, left - i * 16, pr);
      }
      if (p.tile_state && lane == 0)
        p.tile_state[((size_t)b * p.Hkv + kvh) * p.n_k_max + j0 + t] = 1;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(kfree(ks));
        mbar_arrive(vfree(vs));
      }
      ks += W; if (ks >= NK) { ks -= NK; kp ^= 1; }
      vs += W; if (vs >= NV) { vs -= NV; vp ^= 1; }
    }
  } else {
    float* wmax = reinterpret_cast<float*>(smem + C::kMax);
    float* sbuf = reinterpret_cast<float*>(smem + C::kS) + warp * 2 * kPgTile * 8;
    float m_prev[2] = {0.f, 0.f}, a_prev[2] = {1.f, 1.f};  // of the round before
    bool kept_prev = false;
    const int rounds = (ntiles + W - 1) / W;
    int ks = warp, kp = 0;
    for (int r = 0; r <= rounds; ++r) {
      const int t = r * W + warp;
      const bool live = t < ntiles;
      bool keep = false;
      float a[2] = {1.f, 1.f}, mm[2] = {0.f, 0.f};
      if (r < rounds) {
        int page = 0;
        if (live) {
          mbar_wait(kfull(ks), kp, abort_flag);
          page = ids[ks * 4 + ln.sub];
          const int left = Lb - (j0 + t) * kPgTile;
          const uint8_t* krec = smem + C::kK + ks * C::kTileBytes;
          float* sb = sbuf + (r & 1) * kPgTile * 8;
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
          for (int i = 0; i < 4 && i * 16 < left; ++i) {
            float x[4];
            scores(krec + i * REC, left - i * 16, x);
            *reinterpret_cast<float2*>(sb + (i * 16 + g) * 8 + 2 * c) = make_float2(x[0], x[1]);
            *reinterpret_cast<float2*>(sb + (i * 16 + g + 8) * 8 + 2 * c) = make_float2(x[2], x[3]);
            top[0] = fmaxf(top[0], fmaxf(x[0], x[2]));
            top[1] = fmaxf(top[1], fmaxf(x[1], x[3]));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(kfree(ks));
          ks += W; if (ks >= NK) { ks -= NK; kp ^= 1; }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
              top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
            if (g == 0) wmax[((r & 1) * 8 + 2 * c + h) * W + warp] = top[h] * sl;
          }
        }
        named_bar_sync(1, W * 32);  // the maxima of round r are published
        float tw[2][W];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v = *reinterpret_cast<const float4*>(&wmax[((r & 1) * 8 + 2 * c + h) * W]);
          tw[h][0] = v.x; tw[h][1] = v.y; tw[h][2] = v.z; tw[h][3] = v.w;
        }
        const float start[2] = {m[0], m[1]};
#pragma unroll
        for (int i = 0; i < W; ++i) {
          if (r * W + i >= ntiles) break;
          bool pass = true;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (2 * c + h < p.G) pass = pass && row_passes_log2(tw[h][i], m[h], log2_t, true);
          const bool kept = !__all_sync(0xffffffffu, pass);
          if (kept) {
            m[0] = fmaxf(m[0], tw[0][i]);
            m[1] = fmaxf(m[1], tw[1][i]);
          }
          if (i == warp) keep = kept;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[h] = start[h] == m[h] ? 1.f : (start[h] == -INFINITY ? 0.f : ex2_approx(start[h] - m[h]));
          mm[h] = m[h] == -INFINITY ? 0.f : m[h];
        }
        if (live) {
          if (keep) {
            const bool go = __all_sync(0xffffffffu, !*abort_flag);
            fetch(1, go && lane < 8, j0 + t, (r & 1) * W + warp, page);
            if (go) {
              v_used |= 1u << (r & 1);
              v_par ^= 1u << (r & 1);
            }
          } else {
            n_skipped += 1;
          }
          if (p.tile_state && lane == 0)
            p.tile_state[((size_t)b * p.Hkv + kvh) * p.n_k_max + j0 + t] = keep ? 1 : 2;
        }
      }
      if (r > 0) {  // round r - 1: its V tile has had a round's time to arrive
        rescale(a_prev[0], a_prev[1]);
        if (kept_prev) {
          const int u = (r - 1) & 1, left = Lb - (j0 + t - W) * kPgTile;
          mbar_wait(vfull(u * W + warp), (v_phase >> u) & 1, abort_flag);
          v_phase ^= 1u << u;
          const uint8_t* vrec = smem + C::kV + (u * W + warp) * C::kTileBytes;
          const float* sb = sbuf + u * kPgTile * 8;
#pragma unroll 1
          for (int i = 0; i < 4 && i * 16 < left; ++i) {
            const float2 x0 = *reinterpret_cast<const float2*>(sb + (i * 16 + g) * 8 + 2 * c);
            const float2 x1 = *reinterpret_cast<const float2*>(sb + (i * 16 + g + 8) * 8 + 2 * c);
            float pr[4];
            pr[0] = ex2_approx(fmaf(x0.x, sl, -m_prev[0]));
            pr[1] = ex2_approx(fmaf(x0.y, sl, -m_prev[1]));
            pr[2] = ex2_approx(fmaf(x1.x, sl, -m_prev[0]));
            pr[3] = ex2_approx(fmaf(x1.y, sl, -m_prev[1]));
            l[0] += pr[0] + pr[2];
            l[1] += pr[1] + pr[3];
            accumulate(vrec + i * REC, left - i * 16, pr);
          }
        }
      }
      kept_prev = keep;
#pragma unroll
      for (int h = 0; h < 2; ++h) { a_prev[h] = a[h]; m_prev[h] = mm[h]; }
    }
  }

  // ---- merge the warps; write the split.
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        zacc[gr][i] += __shfl_xor_sync(0xffffffffu, zacc[gr][i], o);
  __syncthreads();  // with the producer: every warp is past its last use of the rings
  if (*abort_flag) {
    if (SKIP && lane == 0) {
      int no_abort = 0;
      for (int u = 0; u < 2; ++u)
        if ((v_used >> u) & 1) mbar_wait(vfull(u * W + warp), ((v_par >> u) & 1) ^ 1, &no_abort);
    }
    return;
  }
  paged_merge_warps<D, W>(
      p, reinterpret_cast<float*>(smem), reinterpret_cast<float2*>(smem + C::kStat), head0, split,
      tid, m, l, [&](int mt, int i) {
        return PagedCell{(mt >> 1) * 32 + 4 * g + 2 * (mt & 1) + (i >> 1),
                         acc[mt][i] + zacc[mt >> 1][i & 1]};
      });
  if (lane == 0 && p.counts) {
    atomicAdd(&p.counts[0], (unsigned long long)n_skipped);
    if (tid == 0) atomicAdd(&p.counts[1], (unsigned long long)ntiles);
  }
}

}  // namespace sskip
