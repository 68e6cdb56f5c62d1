// decode_paged4_sm100.cuh -- the split-KV Skip-Softmax decode over 4-bit pages.
//
// The rule, the grid and the products are those of the bf16 kernel
// (decode_paged_sm100.cuh); what differs is what bounds it.  A tile is 0.31 of
// the bytes, so the instructions that widen the codes decide, and the kernel is
// laid out to spend few others and to keep many warps at it: there is no
// producer, every warp owns WHOLE tiles and fetches them itself into a slot
// that only it uses, so that waits, reference checks and votes spread over 64
// keys, and the other warps of its sub-partition (three without a threshold,
// two with one) cover the time a tile takes to arrive.  A call of two CTAs an SM
// at most, without a threshold, has too few warps for that: there (DEEP) a warp
// has two slots, one arriving while it works on the other (128K keys, 8 kv heads,
// 18 splits 76 -> 59 us, 37 splits 53 -> 47).  Measured at 64
// sequences of 16K-32K (8 kv heads, d = 128, no threshold): half tiles in two
// slots and 12 warps an SM 448 us, whole tiles in one slot 434, with 16 warps
// 429; as it stands 397 us, 5.1 TB/s, at 320 instructions for 16 keys of a head
// (55 % of the issue slots; 362 us with every tile in L2).
//
// Codes.  A bf16 whose sign and upper seven exponent bits are 0 is its low byte
// times 2^-133: the subnormals and the first binade are evenly spaced.  So a
// mask alone turns two nibbles of a word into the bf16 operands n 2^-133 and
// 16 n 2^-133, and a shift by 8 and two masks do the other two: five
// instructions for eight codes, exactly, with no bias to take off.  Q and P
// carry 2^48 each, which keeps every product and sum a normal fp32 number
// (2^-85 times what it stands for), and the 16 goes into Q (or, for the
// values, into the result's rows).  Measured clocks of a sub-partition for one
// instruction of a warp: logic, shifts, packed bf16 arithmetic 2, the 8x8
// transpose 4, m16n8k16 bf16 8, m16n8k32 e4m3 24.  The logic pipe is the
// fullest.  Same workload, other things equal: 583 us with e4m3 operands, 504
// with the codes as 128 + n and a subtraction, 473 with these, 450 with full
// and last records apart.
//
// Keys: S = sum over groups of sc (q . n) + mn sum(q).  A group's scale multiplies
// its 32-term product in fp32; the last term is one more product, of the
// record's own (sc, mn) pairs with (0, sum q) in three bf16 parts that hold its
// 24 bits.
//
// Values: O = sum of P' (n - 8) + P (8 sc + mn) with P' = P sc, the group's scale
// joining P before its rounding to bf16.  The -8 (it halves what that rounding
// costs) is one more product for each group, of the number 8 with the same
// rounded P'; the part that does not depend on the code is, for d = 128, one
// more product, of the record's (sc, mn) pairs with P in bf16 (for d = 64, where
// a key's pairs do not fill a row of an 8x8 matrix, a sum in fp32).
//
// With a threshold the warps go in rounds of four tiles.  Each works out its
// tile's scores, which wait in shared memory; then a record of every kept tile
// of the ROUND BEFORE, so that a tile few warps would keep busy is shared by
// all; then it publishes its tile's maxima, and after the round's one barrier
// all walk the four tiles in order under the rule (a head a lane).  The barrier
// also says that the V slots are read, and a kept tile's V is fetched behind it.
// Factor 500 (63 % skipped), same workload: 370 us; 395 with a kept tile's V
// worked on by its own warp, 391 with the barrier ahead of the V work and a
// second one, 490 with 15 or 16 warps of 136 or 128 registers an SM.
#pragma once

#include <type_traits>

#include "decode_paged_sm100.cuh"

namespace sskip {

constexpr int kP4Warps = 4;
constexpr int kP4Threads = kP4Warps * 32;

template <int D, bool SKIP, bool DEEP>
struct Paged4Cfg {
  static constexpr int kBytes = 4 * Kv4<D>::kRecord;          // of a tile
  // Per SM: as many as registers and shared memory hold without slowing the
  // code (d = 64, 64 x 16K-32K: 247 us with five, 262 with four, 253 with six;
  // at factor 500 263 with four, 297 with three, 267 with five).
  static constexpr int kCtas = DEEP ? 2 : (SKIP ? 3 : 4) + (D == 64 ? 1 : 0);
  static constexpr int kSlots = DEEP ? 2 : 1;                 // tiles of a warp
  static constexpr int kK = 0;                                // [W][kSlots] tiles
  static constexpr int kV = kK + kP4Warps * kSlots * kBytes;
  static constexpr int kS = kV + kP4Warps * kSlots * kBytes;           // [2][W][64][8] fp32 scores
  static constexpr int kMax = kS + (SKIP ? kP4Warps * 2 * kPgTile * 8 * 4 : 0);  // [2][8][W]
  // The two merges reuse the slots and the scores.
  static constexpr int kPart = kP4Warps * 8 * (D + 4) * 4;
  static constexpr int kMerge = kPart + (int)sizeof(PagedPart<D>);
  static constexpr int kStat = (kMax > kMerge ? kMax : kMerge) + 2 * 8 * kP4Warps * 4;
  static constexpr int kBar = kStat + kP4Warps * 8 * 8;       // [W]: a tile's K and V, or K, V apart
  static constexpr int kTotal = kBar + kP4Warps * 2 * 8 + 16;
};

constexpr uint32_t kEights = 0x00080008u;              // a pair of 8s, in units of 2^-133
constexpr float kP4Up = 281474976710656.f;            // 2^48: on Q and P
constexpr float kP4Log = 48.f;
constexpr float kP4Unit = 2.5849394142282115e-26f;     // 2^-85: what a product stands for
constexpr float kP4PerUnit = 3.8685626227668134e25f;   // 2^85

// The four pairs of a 4-bit word as bf16 pairs, n 2^-133 (even) and
// 16 n 2^-133 (odd nibbles).
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t v = w >> 8;
  r[0] = w & 0x000F000Fu;
  r[1] = w & 0x00F000F0u;
  r[2] = v & 0x000F000Fu;
  r[3] = v & 0x00F000F0u;
}

// D = A B, without an accumulator to clear first.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm2_t(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr)
               : "memory");
}

// N words at a shared-memory address, aligned to N * 4 bytes (N = 1, 2 or 4).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

template <int D, bool SKIP, bool DEEP>
__global__ void __launch_bounds__(kP4Threads, Paged4Cfg<D, SKIP, DEEP>::kCtas)
    decode_paged4_kernel(const PagedDecodeParams p) {
  using C = Paged4Cfg<D, SKIP, DEEP>;
  static_assert(!(SKIP && DEEP), "a threshold has one tile of keys in flight");
  constexpr int W = kP4Warps, UNIT = kPgTile, NREC = UNIT / 16;
  constexpr int NG = D / 32;   // groups of a row
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  constexpr int REC = Kv4<D>::kRecord, CODES = Kv4<D>::kCodes;
  constexpr bool ZMMA = NG == 4;  // a key's (sc, mn) pairs are 8 values of 16 bits
  extern __shared__ __align__(1024) uint8_t smem[];
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const uint32_t bars = smem_u32(smem + C::kBar) + warp * 2 * 8;  // this warp's
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBar + W * 2 * 8);
  // Shared-memory addresses (32 bits: the loads' arithmetic stays short).
  const uint32_t kbuf = smem_u32(smem + C::kK) + warp * C::kSlots * C::kBytes;
  const uint32_t vbuf = smem_u32(smem + C::kV) + warp * C::kSlots * C::kBytes;
  if (lane == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 8, 1);
    if (warp == 0) *abort_flag = 0;
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
    paged_empty_split<D>(p, part, head0, split, tid, kP4Threads);
    if (p.clustered) paged_cluster_merge<D>(p, part, head0, tid, kP4Threads);
    return;
  }
  const int key0 = j0 * kPgTile;                              // of the split
  const int keys = min(Lb, (j0 + ntiles) * kPgTile) - key0;
  __syncthreads();

  // ---- the copies of a tile: one when a page holds it, else 64 / P, of which
  // those behind the last key are not fetched.  Every copy is one lane's (lanes
  // 0 .. 3 K, lanes 4 .. 7 V), which follows its own first key through the split
  // and looks a copy's page up well before it issues the copy.
  const int* table = p.c.block_table + (size_t)b * p.c.max_pages;
  const int shift = p.c.page_shift, row_shift = min(shift, 6), rows = 1 << row_shift;
  const int sub = lane & 3, end = key0 + keys;
  const uint32_t copy_bytes = (uint32_t)(rows >> 4) * REC;
  const bool copies = lane < 8 && sub < (UNIT >> row_shift);
  const uint8_t* pool = ((lane & 4) ? p.c.v_pages : p.c.k_pages) +
                        ((size_t)kvh << shift) * (REC / 16);
  const uint32_t page_bytes = (uint32_t)(p.Hkv << shift) * (REC / 16);
  const uint32_t dst = ((lane & 4) ? vbuf : kbuf) + sub * copy_bytes;
  // key: this lane's first key of a tile.  The number is looked at when its copy
  // is issued, not here: the look-up is a trip to memory.
  auto page_at = [&](int key) { return copies && key < end ? table[key >> shift] : 0; };
  // The tile whose first key (of lane sub = 0) is k0, this lane's being `key`.
  // which: bit 0 K, bit 1 V; slot: of the warp's.  Called by the whole warp, on a
  // slot whose last copies have arrived.
  auto fetch = [&](int k0, int key, int page, int which, uint32_t bar, int slot) {
    const bool ok = dev_check(k0 < end);
    if (lane == 0) {
      const uint32_t n = (uint32_t)min(UNIT, (end - k0 + rows - 1) >> row_shift << row_shift);
      if (ok) mbar_arrive_expect_tx(bar, (n >> 4) * REC * (which == 3 ? 2 : 1));
      else mbar_arrive(bar);  // the phase completes without data
    }
    __syncwarp();
    if (ok && copies && key < end && ((which >> (lane >> 2)) & 1)) {
      if ((uint32_t)page >= (uint32_t)p.c.num_pages) {
        latch_status(kStatusInvalidArg);  // read as page 0
        page = 0;
      }
      bulk_load(dst + slot * C::kBytes,
                pool + (size_t)page * page_bytes +
                    (uint32_t)(key & ((1 << shift) - 1)) * (uint32_t)(REC / 16),
                copy_bytes, bar);
    }
  };
  // A wait that gives up is the same for the whole warp; what it waited for
  // stays in flight and its slot is not fetched into again.
  auto await = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
  };

  int u = warp;  // this warp's next tile of the split
  constexpr int STEP = W * UNIT;
  int key = key0 + u * UNIT + sub * rows;  // this lane's first key of the next tile to fetch
  int page = page_at(key), next_page = 0;  // of that tile and the one after it
  bool k_inflight = false;                 // SKIP: K's tile
  // This warp's next tile, `tile` of the split, into a slot that has been read,
  // and the look-up for the one after it (ahead of the copies where another tile
  // is there to work on: 4 splits of 128K keys 178 us and 167; else behind them:
  // 64 x 16K-32K 400 us and 397).
  auto fetch_next = [&](int tile, int slot) {
    if (DEEP) next_page = page_at(key + STEP);
    fetch(key0 + tile * UNIT, key, page, SKIP ? 1 : 3, bars + slot * 8, slot);
    k_inflight = true;
    if (!DEEP) next_page = page_at(key + STEP);
  };
  auto step = [&] {
    key += STEP;
    page = next_page;
  };
  if (u < ntiles) {
    fetch_next(u, 0);
    if (DEEP && u + W < ntiles) {
      step();
      fetch_next(u + W, 1);
    }
  }

  // ---- Q^T of head g: the d's that the key words hold at this lane, times 2^48
  // (even nibbles) or 2^44 (odd ones): a power of two, so still exact.
  const int g = lane >> 2, c = lane & 3;
  uint32_t qf[MT][2];
  uint32_t zf[3] = {0u, 0u, 0u};  // (0, sum q) of group c, in three bf16 parts
  {
    const __nv_bfloat16* q = p.q + (head0 + g) * D;
    float mine = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      float x[8], s = 0.f;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (g < p.G) w = *reinterpret_cast<const uint4*>(q + gr * 32 + c * 8);
      bf16x8_to_f32(w, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float up = (i & 1) ? kP4Up / 16.f : kP4Up;
        qf[2 * gr + (i >> 1)][i & 1] = pack_bf16x2(x[2 * i] * up, x[2 * i + 1] * up);
        s += x[2 * i] + x[2 * i + 1];
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (c == gr) mine = s * kP4Unit;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      zf[i] = pack_bf16x2(0.f, mine);
      mine -= __uint_as_float(zf[i] & 0xFFFF0000u);
    }
  }
  const float sl = p.scale_log2 * kP4PerUnit, per_sl = kP4Unit / p.scale_log2;
  const float log2_t = SKIP ? (float)log2((double)p.tsf / (double)Lb) : -INFINITY;

  float acc[MT][4];                // O^T of the codes, in units of 2^-133
  // 8 sum of P', in the same units: a group in an accumulator of its own, the
  // same in every row, or (four groups) group gr in rows 4 gr .. 4 gr + 3 of one,
  // which saves twelve registers of a kernel that has none to spare (407 us and
  // 398; 24 bytes a thread are spilled all the same).
  constexpr int NE = NG == 4 ? 1 : NG;
  float eight[NE][4];
  // Sum of p (8 sc + mn), or (ZMMA) of p sc and p mn: rows 2 g' and 2 g' + 1 of
  // a product's result, the other eight rows not used.
  float zacc[ZMMA ? 2 : NG][2];
  float l[2] = {0.f, 0.f};         // heads 2 c, 2 c + 1
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
  for (int i = 0; i < (ZMMA ? 2 : NG); ++i) zacc[i][0] = zacc[i][1] = 0.f;
#pragma unroll
  for (int i = 0; i < NE; ++i) eight[i][0] = eight[i][1] = eight[i][2] = eight[i][3] = 0.f;
  const uint32_t e_lo = lane < 16 ? kEights : 0u, e_hi = lane >= 16 ? kEights : 0u;

  // Where this lane's words of a record are.
  const uint32_t key_at = g * (D / 2) + c * NG * 4, value_at = lane * NG * 4;
  const uint32_t pair_at = CODES + g * NG * 4, own_at = pair_at + (c % NG) * 4;

  // A record is worked on as a full one or (last) as one with `valid` < 16 keys.
  constexpr std::false_type full;
  constexpr std::true_type last;

  // Logits (before sm_scale, times 2^-85) of a record's 16 keys: x[0..1] key g, x[2..3] key
  // g + 8, heads 2 c and 2 c + 1; the keys from `valid` on -> -inf.
  auto scores = [&](auto tail, uint32_t rec, int valid, float (&x)[4]) {
    uint32_t wa[NG], wb[NG], pa[NG], pb[NG];
    uint32_t z0[1], z1[1];
    lds_words<NG>(wa, rec + key_at);
    lds_words<NG>(wb, rec + key_at + 8 * (D / 2));
    lds_words<NG>(pa, rec + pair_at);
    lds_words<NG>(pb, rec + pair_at + 8 * NG * 4);
    lds_words<1>(z0, rec + own_at);
    lds_words<1>(z1, rec + own_at + 8 * NG * 4);
    mma16816_zero(x, z0[0], z1[0], z0[0], z1[0], zf[0], zf[1]);
    mma16816(x, z0[0], z1[0], z0[0], z1[0], zf[2], 0u);
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      uint32_t a[4], e[4];
      widen_codes(wa[gr], a);
      widen_codes(wb[gr], e);
      float y[4];
      mma16816_zero(y, a[0], e[0], a[1], e[1], qf[2 * gr][0], qf[2 * gr][1]);
      mma16816(y, a[2], e[2], a[3], e[3], qf[2 * gr + 1][0], qf[2 * gr + 1][1]);
      const float sa = __uint_as_float(pa[gr] << 16), sb = __uint_as_float(pb[gr] << 16);
      x[0] = fmaf(sa, y[0], x[0]);
      x[1] = fmaf(sa, y[1], x[1]);
      x[2] = fmaf(sb, y[2], x[2]);
      x[3] = fmaf(sb, y[3], x[3]);
    }
    if constexpr (tail.value) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (g + (i >> 1) * 8 >= valid) x[i] = -INFINITY;
    }
  };

  // O^T += V^T P^T over a record's 16 keys.
  auto accumulate = [&](auto tail, uint32_t rec, int valid, const float (&pr)[4]) {
    if constexpr (tail.value) {
      // Behind the last key the record holds what an earlier sequence left:
      // its codes are numbers, its scales need not be.  The slot is not
      // fetched into again: this is the sequence's last record.
      for (int i = valid * NG + lane; i < 16 * NG; i += 32)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(rec + CODES + i * 4), "r"(0u) : "memory");
      __syncwarp();
    }
    uint32_t w0[NG], w1[NG], pa[NG], pb[NG];
    lds_words<NG>(w0, rec + value_at);
    lds_words<NG>(w1, rec + value_at + 32 * NG * 4);
    lds_words<NG>(pa, rec + pair_at);
    lds_words<NG>(pb, rec + pair_at + 8 * NG * 4);
    if constexpr (ZMMA) {
      uint32_t t0, t1;
      ldsm2_t(rec + CODES + (lane & 15) * 16, t0, t1);
      float z[4] = {zacc[0][0], zacc[0][1], zacc[1][0], zacc[1][1]};
      // (P in bf16 here too; in two parts 411 us for 397.)
      mma16816(z, t0, 0u, t1, 0u, transpose8x8(pack_bf16x2(pr[0], pr[1])),
               transpose8x8(pack_bf16x2(pr[2], pr[3])));
      zacc[0][0] = z[0]; zacc[0][1] = z[1]; zacc[1][0] = z[2]; zacc[1][1] = z[3];
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const float sa = __uint_as_float(pa[gr] << 16), sb = __uint_as_float(pb[gr] << 16);
      if constexpr (!ZMMA) {
        const float za = fmaf(8.f, sa, __uint_as_float(pa[gr] & 0xFFFF0000u));
        const float zb = fmaf(8.f, sb, __uint_as_float(pb[gr] & 0xFFFF0000u));
        zacc[gr][0] = fmaf(pr[0], za, fmaf(pr[2], zb, zacc[gr][0]));
        zacc[gr][1] = fmaf(pr[1], za, fmaf(pr[3], zb, zacc[gr][1]));
      }
      // The scale joins P before its rounding to bf16 (2^-8 of the product at
      // most, where 4 bits leave a value off by a thirtieth of its group's spread).
      // In two bf16 parts, as over bf16 pages, the calls' error against 64 bits
      // falls from 1.9 to 1.7 thousandths, O's own rounding, and 64 x 16K-32K takes
      // 498 us for 397 (factor 500: 404 for 370).
      const uint32_t b0 = transpose8x8(pack_bf16x2(pr[0] * sa, pr[1] * sa));
      const uint32_t b1 = transpose8x8(pack_bf16x2(pr[2] * sb, pr[3] * sb));
      uint32_t a[4], e[4];
      widen_codes(w0[gr], a);
      widen_codes(w1[gr], e);
      mma16816(acc[2 * gr], a[0], a[1], e[0], e[1], b0, b1);
      mma16816(acc[2 * gr + 1], a[2], a[3], e[2], e[3], b0, b1);
      if constexpr (NE == 1) {
        const uint32_t e8 = (gr & 1) ? e_hi : e_lo;
        if (gr < 2) mma16816(eight[0], e8, 0u, e8, 0u, b0, b1);
        else mma16816(eight[0], 0u, e8, 0u, e8, b0, b1);
      } else {
        mma16816(eight[gr], kEights, kEights, kEights, kEights, b0, b1);
      }
    }
  };

  auto rescale = [&](float a0, float a1) {
    if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][0] *= a0; acc[i][1] *= a1; acc[i][2] *= a0; acc[i][3] *= a1;
      }
#pragma unroll
      for (int i = 0; i < (ZMMA ? 1 : NG); ++i) { zacc[i][0] *= a0; zacc[i][1] *= a1; }
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        eight[i][0] *= a0; eight[i][1] *= a1; eight[i][2] *= a0; eight[i][3] *= a1;
      }
      l[0] *= a0;
      l[1] *= a1;
    }
  };

  float m[2] = {-INFINITY, -INFINITY};  // reference of heads 2 c, 2 c + 1, in log2 units
  int n_skipped = 0;
  if constexpr (!SKIP) {
    // What follows from m: the score (in units of 1 / sl) that moves it, and the
    // exponent's offset 48 - m (48 while m is -inf).
    float move_at[2] = {-INFINITY, -INFINITY}, off[2] = {kP4Log, kP4Log};
    auto record = [&](auto tail, uint32_t krec, uint32_t vrec, int valid) {
      float x[4];
      scores(tail, krec, valid, x);
      // The reference moves only when a score is 2^8 above it: P stays below
      // 2^8 (times 2^48) and most records need no exchange between the lanes.
      float top[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
      if (__any_sync(0xffffffffu, (top[0] > move_at[0]) | (top[1] > move_at[1]))) {
        float a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
          const float mn = fmaxf(m[h], top[h] * sl);
          a[h] = m[h] == mn ? 1.f : (m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - mn));
          m[h] = mn;
          move_at[h] = (mn + 8.f) * per_sl;
          off[h] = mn == -INFINITY ? kP4Log : kP4Log - mn;
        }
        rescale(a[0], a[1]);
      }
      float pr[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) pr[h] = ex2_approx(fmaf(x[h], sl, off[h & 1]));
      l[0] += pr[0] + pr[2];
      l[1] += pr[1] + pr[3];
      accumulate(tail, vrec, valid, pr);
    };
    auto slot_of = [](int i) { return DEEP ? i & 1 : 0; };          // of the warp's tile i
    auto phase_of = [](int i) { return (uint32_t)((DEEP ? i >> 1 : i) & 1); };
    int n = 0;  // tiles done
    for (; u < ntiles; u += W, ++n) {
      const int slot = slot_of(n);
      if (!await(bars + slot * 8, phase_of(n))) break;
      const uint32_t kt = kbuf + slot * C::kBytes, vt = vbuf + slot * C::kBytes;
      const int left = keys - u * UNIT;
      if (left >= UNIT) {
#pragma unroll 1
        for (int i = 0; i < NREC; ++i) record(full, kt + i * REC, vt + i * REC, 16);
      } else {
#pragma unroll 1
        for (int i = 0; i * 16 < left; ++i) record(last, kt + i * REC, vt + i * REC, left - i * 16);
      }
      if (p.tile_state && lane == 0)
        p.tile_state[((size_t)b * p.Hkv + kvh) * p.n_k_max + j0 + u] = 1;
      __syncwarp();  // every lane is past its reads of the slot
      if (u + C::kSlots * W < ntiles) {
        step();
        fetch_next(u + C::kSlots * W, slot);
      }
    }
    // Gave up: wait out this warp's copies, of tile u and (two slots) the one
    // after it, before the CTA exits.
    for (int i = 0; i < C::kSlots && u < ntiles; ++i, ++n, u += W) {
      int no_abort = 0;
      mbar_wait(bars + slot_of(n) * 8, phase_of(n), &no_abort);
    }
  } else {
    float* wmax = reinterpret_cast<float*>(smem + C::kMax);
    constexpr int SB = kPgTile * 8;  // a tile's scores: 64 keys, 8 heads
    float* sbuf = reinterpret_cast<float*>(smem + C::kS) + g * 8 + 2 * c;
    const uint32_t vbars = smem_u32(smem + C::kBar) + 8, vbase = smem_u32(smem + C::kV) + warp * REC;
    float m_prev[2] = {0.f, 0.f}, a_prev[2] = {1.f, 1.f};  // of the round before
    float mw = -INFINITY;  // the running maximum of head lane & 7, which the rule is walked on
    bool v_inflight = false;
    uint32_t k_count = 0;                // K tiles waited for
    uint32_t kept_prev = 0, v_parity = 0;  // a bit a warp: V fetched; phase of the next wait for it
    int vkey = 0;  // this lane's first key of the round's tile
    const int rounds = (ntiles + W - 1) / W;
    const bool idle = (lane & 7) >= p.G;  // padding heads always pass
    for (int r = 0; r <= rounds; ++r, u += W) {
      const bool live = u < ntiles;
      float top[2] = {-INFINITY, -INFINITY};
      int vpage = 0;
      if (live) {
        const bool there = k_inflight && await(bars, k_count & 1);
        if (there) { k_inflight = false; ++k_count; }
        const int left = keys - u * UNIT;
        float* sb = sbuf + (r & 1) * W * SB + warp * SB;
        auto record = [&](auto tail, int i) {
          float x[4];
          scores(tail, kbuf + i * REC, left - i * 16, x);
          *reinterpret_cast<float2*>(sb + i * 128) = make_float2(x[0], x[1]);
          *reinterpret_cast<float2*>(sb + i * 128 + 64) = make_float2(x[2], x[3]);
          top[0] = max_nan(top[0], x[0], x[2]);
          top[1] = max_nan(top[1], x[1], x[3]);
        };
        if (left >= UNIT) {
#pragma unroll 2  // 371 us, 379 one by one, 376 by four
          for (int i = 0; i < NREC; ++i) record(full, i);
        } else {
#pragma unroll 1
          for (int i = 0; i * 16 < left; ++i) record(last, i);
        }
        __syncwarp();  // every lane is past its reads of the slot
        vpage = page;
        vkey = key;
        if (u + W < ntiles && there) {
          step();
          fetch_next(u + W, 0);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top[h] = max_nan(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
      }
      // The kept tiles of round r - 1, whose V tiles have had these scores'
      // time to arrive: a record of each for every warp.
      rescale(a_prev[0], a_prev[1]);
      const float off[2] = {kP4Log - m_prev[0], kP4Log - m_prev[1]};
#pragma unroll 1
      for (uint32_t todo = kept_prev; todo; todo &= todo - 1) {
        const int i = __ffs(todo) - 1;
        if (!await(vbars + i * 16, (v_parity >> i) & 1)) break;
        v_parity ^= 1u << i;
        if (i == warp) v_inflight = false;
        const int valid = keys - ((r - 1) * W + i) * UNIT - warp * 16;  // of this warp's record
        const float* sb = sbuf + ((r - 1) & 1) * W * SB + i * SB + warp * 128;
        auto record = [&](auto tail) {
          const float2 x0 = *reinterpret_cast<const float2*>(sb);
          const float2 x1 = *reinterpret_cast<const float2*>(sb + 64);
          float pr[4];
          pr[0] = ex2_approx(fmaf(x0.x, sl, off[0]));
          pr[1] = ex2_approx(fmaf(x0.y, sl, off[1]));
          pr[2] = ex2_approx(fmaf(x1.x, sl, off[0]));
          pr[3] = ex2_approx(fmaf(x1.y, sl, off[1]));
          l[0] += pr[0] + pr[2];
          l[1] += pr[1] + pr[3];
          accumulate(tail, vbase + i * C::kBytes, valid, pr);
        };
        if (valid >= 16) record(full);
        else if (valid > 0) record(last);
      }
      if (r == rounds) break;
      if (g == 0) {
        wmax[((r & 1) * 8 + 2 * c) * W + warp] = top[0] * sl;  // -inf: no such tile
        wmax[((r & 1) * 8 + 2 * c + 1) * W + warp] = top[1] * sl;
      }
      // The maxima of round r are published, and the V slots of round r - 1 read.
      named_bar_sync(1, W * 32);
      // The rule, tile after tile, a head a lane (four lanes the same); a dead
      // tile's maxima are -inf and pass.
      const float4 v = *reinterpret_cast<const float4*>(&wmax[((r & 1) * 8 + (lane & 7)) * W]);
      const float tw[W] = {v.x, v.y, v.z, v.w};
      uint32_t kept = 0;
      const float start = mw;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const bool keep = !__all_sync(0xffffffffu, paged_head_passes(tw[i], mw, log2_t, idle));
        mw = keep ? max_nan(mw, tw[i]) : mw;
        kept |= keep ? 1u << i : 0u;
      }
      a_prev[0] = a_prev[1] = 1.f;
      if (kept) {
        const float aw = start == mw ? 1.f : (start == -INFINITY ? 0.f : ex2_approx(start - mw));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a_prev[h] = __shfl_sync(0xffffffffu, aw, 2 * c + h);
          m[h] = __shfl_sync(0xffffffffu, mw, 2 * c + h);
          m_prev[h] = m[h] == -INFINITY ? 0.f : m[h];
        }
      }
      if (live) {
        const bool keep = (kept >> warp) & 1;
        if (!keep) n_skipped += 1;
        if (p.tile_state && lane == 0)
          p.tile_state[((size_t)b * p.Hkv + kvh) * p.n_k_max + j0 + u] = keep ? 1 : 2;
        if (keep && !v_inflight) {
          fetch(key0 + u * UNIT, vkey, vpage, 2, bars + 8, 0);
          v_inflight = true;
        }
      }
      kept_prev = kept;
    }
    {  // a wait gave up: wait out this warp's copies before the CTA exits
      int no_abort = 0;
      if (k_inflight) mbar_wait(bars, k_count & 1, &no_abort);
      if (v_inflight) mbar_wait(bars + 8, (v_parity >> warp) & 1, &no_abort);
    }
  }

  __syncthreads();  // every warp is past its last use of the slots
  if (*abort_flag) {
    if (p.clustered) {
      if (tid < 8) part->lse[tid] = -INFINITY;
      paged_cluster_merge<D>(p, part, head0, tid, kP4Threads);
    }
    return;
  }

  // ---- merge the warps; write the split.
  auto sum_keys = [&](float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  float z[NG][2];  // what does not come from the codes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      if constexpr (ZMMA)
        z[gr][h] = fmaf(8.f, __shfl_sync(0xffffffffu, zacc[0][h], 8 * gr + c),
                        __shfl_sync(0xffffffffu, zacc[0][h], 8 * gr + 4 + c));
      else
        z[gr][h] = sum_keys(zacc[gr][h]);
      const float e8 = NE == 1 ? __shfl_sync(0xffffffffu, eight[0][(gr >> 1) * 2 + h], (gr & 1) * 16 + c)
                               : eight[gr % NE][h];
      z[gr][h] -= e8 * kP4PerUnit * kP4Up;
    }
    l[h] = sum_keys(l[h]);
    m[h] -= kP4Log;  // what l, z and the codes' part are relative to
  }
  paged_merge_warps<D, W>(
      p, reinterpret_cast<float*>(smem), reinterpret_cast<float2*>(smem + C::kStat), head0, split,
      tid, m, l, part, [&](int mt, int i) {
        // 2^133 in two steps; the odd rows' codes came 16 times too large
        const float o = acc[mt][i] * kP4PerUnit * ((i >> 1) ? kP4Up / 16.f : kP4Up);
        return PagedCell{(mt >> 1) * 32 + 4 * g + 2 * (mt & 1) + (i >> 1),
                         o + z[mt >> 1][i & 1]};
      });
  if (lane == 0 && p.counts) {
    atomicAdd(&p.counts[0], (unsigned long long)n_skipped);
    if (tid == 0) atomicAdd(&p.counts[1], (unsigned long long)ntiles);
  }
  if (p.clustered) paged_cluster_merge<D>(p, part, head0, tid, kP4Threads);
}

}  // namespace sskip
