// kvcache_sm100.cuh -- filling and reading back the paged key/value cache.
//
// Append: what lies between a layer's projections and its attention, in one
// pass over the rows.  Per query and key head an optional RMS norm, then the
// rotation by position, then the row goes where it is read next: the decode's
// or the prefill's layout, and for keys and values the pages of the cache.
//
//   y = x rsqrt(mean(x^2) + eps) w;   (a, b) -> (a cos - b sin, a sin + b cos)
//
// Everything is fp32 between the bf16 load and the one rounding at the store
// (to bf16, or to the 4-bit form): no rounding sits between norm and rotation.
//
// Angles.  A frequency is kept as a 64-bit fixed-point fraction of a turn per
// position, so position * frequency modulo 2^64 is the angle modulo one turn,
// exact at any position: no fp32 product whose error grows with the position,
// and no table that grows with the context.
//
// The work is HBM traffic (a row is read once and written once or twice).
// D / 16 lanes hold one head's row as two 16-byte pieces a lane; the pieces
// are chosen so that a lane owns both members of its eight pairs in either
// pairing, so the rotation needs no exchange.  A token's rot / 2 sines and
// cosines are worked out once, one or two a lane, and shared.  Large calls give
// a token to one warp, which walks its heads and loads the next rows ahead of
// the arithmetic of the current ones; small ones give a token a CTA, every
// group of heads a warp of its own.  16K tokens (32 + 8 heads of 128, all rows
// out and into the cache) take 81 us, 5.8 TB/s of rows in and out, more than
// half of it writes; into 4-bit pages (q out only) 88 us, bound by the codes'
// instructions (79 % of the issue slots).  64 tokens take 2.4 us.
#pragma once

#include <cstdint>

#include "kv4_sm100.cuh"
#include "sm100_ptx.cuh"

namespace sskip {

struct PagedRows {             // where rows of the cache live
  uint8_t* k_pages;            // [num_pages, Hkv, P, D] bf16 or [num_pages, Hkv, P / 16, record]
  uint8_t* v_pages;
  const int* block_table;      // [B, max_pages]
  int B, Hkv, num_pages, page_shift, max_pages;
};

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;          // [T, H, D] rows, token stride below
  long long q_stride, k_stride, v_stride;  // elements
  const int *seq_ids, *positions;          // [T]
  const __nv_bfloat16 *q_weight, *k_weight;  // [D] or null
  float eps;
  const unsigned long long* turns;         // [rot / 2], 2^-64 turns per position
  int rot_chunks;                          // rot / 16: lanes of a head that rotate
  int interleaved;
  float attn_factor;
  __nv_bfloat16 *q_out, *k_out, *v_out;    // [T / out_len, H, out_len, D] or null
  int out_len, T, Hq;
  PagedRows c;
};

struct GatherParams {
  const int *seq_ids, *positions;
  __nv_bfloat16 *k_out, *v_out;            // [T / out_len, Hkv, out_len, D]
  int out_len, T, warps_per_token;
  PagedRows c;
};

constexpr int kKvThreads = 128;      // of a gather
constexpr int kAppendMaxWarps = 12;  // of a token with a CTA to itself
constexpr int kAppendAlone = 4;      // tokens of a CTA whose warps have one each

// Page and offset of a token's row; false for a padding token (negative
// sequence) or an index outside the table, which is latched.
__device__ __forceinline__ bool locate_row(const PagedRows& c, int seq, int pos, int* page,
                                           int* off) {
  if (seq < 0) return false;
  const int slot = pos >> c.page_shift;
  if (seq >= c.B || pos < 0 || slot >= c.max_pages) {
    latch_status(kStatusInvalidArg);
    return false;
  }
  *page = c.block_table[(size_t)seq * c.max_pages + slot];
  *off = pos & ((1 << c.page_shift) - 1);
  if (*page < 0 || *page >= c.num_pages) {
    latch_status(kStatusInvalidArg);
    return false;
  }
  return true;
}

__device__ __forceinline__ uint4 load_raw(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint4*>(p);
}

__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float (&x)[8]) {
  uint4 w;
  w.x = pack_bf16x2(x[0], x[1]);
  w.y = pack_bf16x2(x[2], x[3]);
  w.z = pack_bf16x2(x[4], x[5]);
  w.w = pack_bf16x2(x[6], x[7]);
  *reinterpret_cast<uint4*>(p) = w;
}

// Cosine and sine of position * turns: the top 32 bits of the wrapped product
// are the angle in 2^-32 turns; the nearest quarter turn comes off in integers
// and the rest, within an eighth of a turn, is exact enough in fp32.
__device__ __forceinline__ void turn_cos_sin(long long pos, unsigned long long turns, float scale,
                                             float& c, float& s) {
  const uint32_t u = (uint32_t)(((unsigned long long)pos * turns) >> 32);
  const uint32_t quarter = (u + (1u << 29)) >> 30;
  const int rest = (int)(u - (quarter << 30));
  float sn, cs;
  sincospif((float)rest * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: units of pi
  const bool odd = quarter & 1;
  float cc = odd ? sn : cs, ss = odd ? cs : sn;
  if (quarter == 1 || quarter == 2) cc = -cc;
  if (quarter == 2 || quarter == 3) ss = -ss;
  c = cc * scale;
  s = ss * scale;
}

// ALONE: a warp has a token to itself (else the CTA has one).
template <int D, bool Q4, bool ALONE>
__global__ void __launch_bounds__(ALONE ? kAppendAlone * 32 : kAppendMaxWarps * 32, ALONE ? 7 : 2)
    kv_append_kernel(const AppendParams p) {
  constexpr int LH = D / 16;       // lanes per head
  constexpr int HW = 32 / LH;      // heads a warp holds at a time
  wait_for_previous_kernel();
  // cosine and sine of pair 8 j + e at e LH + j
  __shared__ float tabs[ALONE ? kAppendAlone : 1][2][D / 2];
  const int lane = threadIdx.x & 31, j = lane % LH, hs = lane / LH;
  const int warp = ALONE ? 0 : threadIdx.x >> 5, warps = ALONE ? 1 : blockDim.x >> 5;
  const int t = ALONE ? blockIdx.x * kAppendAlone + (threadIdx.x >> 5) : blockIdx.x;
  if (ALONE && t >= p.T) return;
  auto& tab = tabs[ALONE ? threadIdx.x >> 5 : 0];
  const int pos = p.positions ? p.positions[t] : 0;
  const int seq = p.seq_ids ? p.seq_ids[t] : 0;
  // The lane's pairs 8 j .. 8 j + 7: in chunks (j, j + rot / 16) when pairs are
  // half the rotated part apart, in (2 j, 2 j + 1) when they are neighbours or
  // not rotated at all.
  const bool turns = j < p.rot_chunks;
  const bool apart = turns && !p.interleaved;
  const int m0 = apart ? j : 2 * j, m1 = apart ? j + p.rot_chunks : 2 * j + 1;

  const int Hkv = p.c.Hkv, units = p.Hq + 2 * Hkv;
  // kind 0: query, 1: key, 2: value
  auto kind_of = [&](int u) { return u < p.Hq ? 0 : (u < p.Hq + Hkv ? 1 : 2); };
  auto head_of = [&](int u, int kind) {
    return kind == 0 ? u : (kind == 1 ? u - p.Hq : u - p.Hq - Hkv);
  };
  uint4 r0, r1;
  auto load = [&](int u) {
    r0 = r1 = make_uint4(0u, 0u, 0u, 0u);
    if (u < units) {
      const int kind = kind_of(u);
      const __nv_bfloat16* row =
          (kind == 0 ? p.q + (size_t)t * p.q_stride
                     : (kind == 1 ? p.k + (size_t)t * p.k_stride : p.v + (size_t)t * p.v_stride)) +
          (size_t)head_of(u, kind) * D;
      r0 = load_raw(row + m0 * 8);
      r1 = load_raw(row + m1 * 8);
    }
  };
  const bool cached = p.c.k_pages != nullptr;
  if (seq < 0) return;  // padding: all of the token's threads
  load(warp * HW + hs);
  int page = 0, off = 0;
  if (cached && !locate_row(p.c, seq, pos, &page, &off)) return;
  for (int i = ALONE ? lane : threadIdx.x; i < p.rot_chunks * 8; i += ALONE ? 32 : blockDim.x) {
    float c, s;
    turn_cos_sin(pos, p.turns[i], p.attn_factor, c, s);
    tab[0][(i & 7) * LH + (i >> 3)] = c;
    tab[1][(i & 7) * LH + (i >> 3)] = s;
  }
  if (ALONE) __syncwarp();
  else __syncthreads();
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = turns ? tab[0][e * LH + j] : 1.f;
    sn[e] = turns ? tab[1][e * LH + j] : 0.f;
  }
  const size_t ob = (size_t)(t / p.out_len), oi = (size_t)(t % p.out_len);
  const bool any_norm = p.q_weight || p.k_weight;

  for (int u0 = warp * HW; u0 < units; u0 += warps * HW) {
    const int u = u0 + hs;
    const bool live = u < units;
    const int kind = kind_of(u), h = head_of(u, kind);
    float x0[8], x1[8];
    bf16x8_to_f32(r0, x0);
    bf16x8_to_f32(r1, x1);
    load(u + warps * HW);  // the next rows, while these are worked on
    if (any_norm) {
      const __nv_bfloat16* w = kind == 0 ? p.q_weight : p.k_weight;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
#pragma unroll
      for (int o = LH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (kind < 2 && w != nullptr) {
        const float r = rsqrtf(ss * (1.0f / D) + p.eps);
        float w0[8], w1[8];
        bf16x8_to_f32(load_raw(w + m0 * 8), w0);
        bf16x8_to_f32(load_raw(w + m1 * 8), w1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x0[e] = x0[e] * r * w0[e];
          x1[e] = x1[e] * r * w1[e];
        }
      }
    }
    if (turns && kind < 2) {
      if (apart) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = x0[e], b = x1[e];
          x0[e] = a * cs[e] - b * sn[e];
          x1[e] = a * sn[e] + b * cs[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x0[2 * e], b = x0[2 * e + 1], c = x1[2 * e], d = x1[2 * e + 1];
          x0[2 * e] = a * cs[e] - b * sn[e];
          x0[2 * e + 1] = a * sn[e] + b * cs[e];
          x1[2 * e] = c * cs[4 + e] - d * sn[4 + e];
          x1[2 * e + 1] = c * sn[4 + e] + d * cs[4 + e];
        }
      }
    }
    __nv_bfloat16* out = kind == 0 ? p.q_out : (kind == 1 ? p.k_out : p.v_out);
    if (live && out) {
      const int H = kind == 0 ? p.Hq : Hkv;
      __nv_bfloat16* o = out + ((ob * H + h) * (size_t)p.out_len + oi) * D;
      store_chunk(o + m0 * 8, x0);
      store_chunk(o + m1 * 8, x1);
    }
    if constexpr (Q4) {
      // Whole warps come here (the group statistics are exchanged by shuffles);
      // a warp with no key or value head has nothing to write.
      if (__any_sync(0xffffffffu, live && kind > 0)) {
        uint8_t* base = kind == 2 ? p.c.v_pages : p.c.k_pages;
        uint8_t* rec = base + ((((size_t)page * Hkv + (kind == 0 ? 0 : h)) << (p.c.page_shift - 4)) +
                               (off >> 4)) * Kv4<D>::kRecord;
        kv4_store_row<D>(rec, off & 15, kind == 2, live && kind > 0, p.interleaved ? 0 : p.rot_chunks,
                         apart, m0, m1, x0, x1);
      }
    } else if (cached && live && kind > 0) {
      __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(kind == 1 ? p.c.k_pages : p.c.v_pages);
      __nv_bfloat16* o = base + ((((size_t)page * Hkv + h) << p.c.page_shift) + off) * D;
      store_chunk(o + m0 * 8, x0);
      store_chunk(o + m1 * 8, x1);
    }
  }
}

// Rows of the cache back as bf16, in the prefill's or the decode's layout.
template <int D, bool Q4>
__global__ void __launch_bounds__(kKvThreads) kv_gather_kernel(const GatherParams p) {
  constexpr int LH = D / 16, HW = 32 / LH;
  wait_for_previous_kernel();
  const int gw = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  const int t = gw / p.warps_per_token, part = gw - t * p.warps_per_token;
  if (t >= p.T) return;
  const int lane = threadIdx.x & 31, j = lane % LH, hs = lane / LH;
  int page, off;
  if (!locate_row(p.c, p.seq_ids[t], p.positions[t], &page, &off)) return;
  const size_t ob = (size_t)(t / p.out_len), oi = (size_t)(t % p.out_len);
  const int units = 2 * p.c.Hkv;
  for (int u = part * HW + hs; u < units; u += p.warps_per_token * HW) {
    const bool val = u >= p.c.Hkv;
    const int h = val ? u - p.c.Hkv : u;
    const uint8_t* base = val ? p.c.v_pages : p.c.k_pages;
    __nv_bfloat16* o =
        (val ? p.v_out : p.k_out) + ((ob * p.c.Hkv + h) * (size_t)p.out_len + oi) * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = j + i * LH;
      if constexpr (Q4) {
        const uint8_t* rec = base + ((((size_t)page * p.c.Hkv + h) << (p.c.page_shift - 4)) +
                                     (off >> 4)) * Kv4<D>::kRecord;
        float x[8];
        kv4_load_chunk<D>(rec, off & 15, val, m, x);
        store_chunk(o + m * 8, x);
      } else {
        const uint4* row = reinterpret_cast<const uint4*>(
            base + ((((size_t)page * p.c.Hkv + h) << p.c.page_shift) + off) * (D * 2));
        reinterpret_cast<uint4*>(o)[m] = row[m];
      }
    }
  }
}

}  // namespace sskip
