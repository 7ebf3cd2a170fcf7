// One 16-row page of one kv head in shared memory, for the window attend's mma.sync kernel: scores
// S^T = K Q^T and O^T += V^T P^T with the keys as the MMA's M (scores) and K (output) dimension and
// NT n8-tiles of query columns (a column = one query head of one row of the group).
//
// A page in shared memory: bf16 [4 quarter rows: K lo, K hi, V lo, V hi][16 rows][128 B] and fp8 [K, V][16
// rows][128 B], 128B-swizzled; NVFP4 the K slot (1152 B) and the V slot as stored.
//
// A lane (hh = lane / 4, c = lane % 4) holds scores of keys hh, hh + 8 in columns 2c, 2c + 1 of a
// tile, and V^T fragments of keys 2c, 2c + 1 (first half of the MMA's k) and 2c + 8, 2c + 9.
#pragma once

#include "pbs_device.cuh"

namespace pbs {
namespace wp {

template <int FMT>
constexpr int kPageBytes = FMT == PBS_KV_BF16 ? 8192 : FMT == PBS_KV_FP8_E4M3 ? 4096 : 2304;
constexpr int kNvfp4Slot = 1152;

// Byte offset of the 128-byte line of page row r, quarter q of a bf16 row / half q of an fp8 row.
__device__ __forceinline__ uint32_t line_off(int r, int q) { return q * 2048 + r * 128; }

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Four e4m3 bytes to two f16x2 words, eight e2m1 codes to four (exact). The converts take a byte or a half
// of their source register for free; shifting it down first would double the work of the pipe that converts
// (16 lanes a clock).
__device__ __forceinline__ void e4m3x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ void e2m1x8(uint32_t x, uint32_t (&w)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\tcvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
      : "r"(x));
}

// First of the two dims (the second is +8 for bf16, +2 otherwise) of Q fragment word w of k-step j:
// the order in which page_scores feeds K's dims to the MMA.
template <int FMT>
__device__ __forceinline__ int q_dim(int j, int w, int c) {
  if (FMT == PBS_KV_BF16) return 16 * j + 2 * c + 8 * w;
  if (FMT == PBS_KV_FP8_E4M3) return 16 * j + 4 * c + 2 * w;
  return 32 * c + 4 * j + 2 * w;
}

// Scores of the pages at st[0..NP): s[page][tile][..]. The pages' chains interleave. q(t, j): the Q fragment of
// tile t and k-step j.
template <int FMT, int NP, int NT, typename Q>
__device__ __forceinline__ void page_scores(const uint32_t (&st)[NP], Q q, int lane, float (&s)[NP][NT][4]) {
  const int hh = lane >> 2, c = lane & 3;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) s[i][t][0] = s[i][t][1] = s[i][t][2] = s[i][t][3] = 0.f;
  if (FMT == PBS_KV_BF16) {
    const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
    const int hi = lane >> 4;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int chunk = 2 * (j & 3) + hi;
      uint2 qj[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) qj[t] = q(t, j);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t af[4];
        ldsm_x4(st[i] + line_off(key, j >> 2) + ((chunk ^ (key & 7)) << 4), af);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_bf16(s[i][t], af, qj[t].x, qj[t].y);
      }
    }
  } else if (FMT == PBS_KV_FP8_E4M3) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint2 qj[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) qj[t] = q(t, j);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t w0 = lds32(st[i] + line_off(hh, 0) + ((j ^ hh) << 4) + 4 * c);
        const uint32_t w1 = lds32(st[i] + line_off(hh + 8, 0) + ((j ^ hh) << 4) + 4 * c);
        uint32_t af[4];
        e4m3x4(w0, af[0], af[2]);
        e4m3x4(w1, af[1], af[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(s[i][t], af, qj[t].x, qj[t].y);
      }
    }
  } else {
    uint4 k0[NP], k1[NP];
    uint32_t s0lo[NP], s0hi[NP], s1lo[NP], s1hi[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      k0[i] = lds128(st[i] + hh * 64 + 16 * c);
      k1[i] = lds128(st[i] + (hh + 8) * 64 + 16 * c);
      const uint32_t sc0 = e4m3x2_to_f16x2(lds16(st[i] + 1024 + hh * 8 + 2 * c));
      const uint32_t sc1 = e4m3x2_to_f16x2(lds16(st[i] + 1024 + (hh + 8) * 8 + 2 * c));
      s0lo[i] = prmt(sc0, sc0, 0x1010);
      s0hi[i] = prmt(sc0, sc0, 0x3232);
      s1lo[i] = prmt(sc1, sc1, 0x1010);
      s1hi[i] = prmt(sc1, sc1, 0x3232);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint2 qj[2][NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        qj[0][t] = q(t, j);
        qj[1][t] = q(t, j + 1);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t sa = j < 4 ? s0lo[i] : s0hi[i], sb = j < 4 ? s1lo[i] : s1hi[i];
        uint32_t a[4], b[4];
        e2m1x8(word_of(k0[i], j >> 1), a);
        e2m1x8(word_of(k1[i], j >> 1), b);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t af[4] = {hmul2(a[2 * h], sa), hmul2(b[2 * h], sb), hmul2(a[2 * h + 1], sa), hmul2(b[2 * h + 1], sb)};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(s[i][t], af, qj[h][t].x, qj[h][t].y);
        }
      }
    }
  }
}

// The 16-bit words of a V^T fragment whose keys are in `bits` (bit n = key n of the page), this
// lane's keys only: x for the MMA's first 8 keys (2c, 2c + 1), y for the last 8.
__device__ __forceinline__ uint2 key_words(uint32_t bits, int c) {
  const uint32_t a = bits >> (2 * c), b = bits >> (2 * c + 8);
  return make_uint2(((a & 1u) ? 0xffffu : 0u) | ((a & 2u) ? 0xffff0000u : 0u),
                    ((b & 1u) ? 0xffffu : 0u) | ((b & 2u) ? 0xffff0000u : 0u));
}

// V^T fragment of output-dim tile i (16 dims x 16 keys) of a page.
template <int FMT>
struct VPage {
  uint32_t st;
  int lane;
  uint4 a8[FMT == PBS_KV_FP8_E4M3 ? 4 : 1];  // fp8: keys 2c, 2c + 1, 2c + 8, 2c + 9, 16 dims from 16 hh
  uint32_t w4[4][4];                         // NVFP4: the fragments of 4 tiles ..
  uint32_t sab, scd;                         // .. before their scales (keys 2c, 2c + 1 | 2c + 8, 2c + 9)

  __device__ __forceinline__ VPage(uint32_t stage, int lane_) : st(stage), lane(lane_) {
    const int hh = lane >> 2, c = lane & 3;
    if (FMT == PBS_KV_FP8_E4M3) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int key = 2 * c + (q & 1) + 8 * (q >> 1);
        a8[q] = lds128(st + line_off(key, 1) + ((hh ^ (key & 7)) << 4));
      }
    } else if (FMT == PBS_KV_NVFP4) {
      const uint32_t vs0 = st + kNvfp4Slot + 1024;
      sab = e4m3x2_to_f16x2(lds8(vs0 + (2 * c) * 8 + hh) | (lds8(vs0 + (2 * c + 1) * 8 + hh) << 8));
      scd = e4m3x2_to_f16x2(lds8(vs0 + (2 * c + 8) * 8 + hh) | (lds8(vs0 + (2 * c + 9) * 8 + hh) << 8));
    }
  }

  // Tiles 4 half .. 4 half + 3 (NVFP4: unpacks their 8-dim words; elsewhere nothing to do).
  __device__ __forceinline__ void begin(int half) {
    if (FMT != PBS_KV_NVFP4) return;
    const int hh = lane >> 2, c = lane & 3;
    const uint32_t vc0 = st + kNvfp4Slot + 8 * hh + 4 * half;
    const uint32_t A = lds32(vc0 + (2 * c) * 64), B = lds32(vc0 + (2 * c + 1) * 64);
    const uint32_t C = lds32(vc0 + (2 * c + 8) * 64), D = lds32(vc0 + (2 * c + 9) * 64);
    // a byte of the interleaved words holds one dim of two keys: what one f16x2 word of the fragment wants
    e2m1x8((A & 0x0F0F0F0Fu) | ((B & 0x0F0F0F0Fu) << 4), w4[0]);
    e2m1x8(((A >> 4) & 0x0F0F0F0Fu) | (B & 0xF0F0F0F0u), w4[1]);
    e2m1x8((C & 0x0F0F0F0Fu) | ((D & 0x0F0F0F0Fu) << 4), w4[2]);
    e2m1x8(((C >> 4) & 0x0F0F0F0Fu) | (D & 0xF0F0F0F0u), w4[3]);
  }

  __device__ __forceinline__ void tile(int i, uint32_t (&vf)[4]) const {
    if (FMT == PBS_KV_BF16) {
      const int mi = lane >> 3;
      const int key = (lane & 7) + 8 * (mi >> 1), chunk = 2 * (i & 3) + (mi & 1);
      ldsm_x4_trans(st + line_off(key, 2 + (i >> 2)) + ((chunk ^ (key & 7)) << 4), vf);
    } else if (FMT == PBS_KV_FP8_E4M3) {
      const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
      e4m3x4(prmt(word_of(a8[0], i >> 1), word_of(a8[1], i >> 1), sel), vf[0], vf[1]);
      e4m3x4(prmt(word_of(a8[2], i >> 1), word_of(a8[3], i >> 1), sel), vf[2], vf[3]);
    } else {
      const int b = i & 3;
      vf[0] = hmul2(w4[0][b], sab);
      vf[1] = hmul2(w4[1][b], sab);
      vf[2] = hmul2(w4[2][b], scd);
      vf[3] = hmul2(w4[3][b], scd);
    }
  }
};

// P^T as the MMA's B operand. bf16 V: P as bf16 hi + lo (two MMAs: P keeps 16 bits), hi cut and lo above zero
// where P is (by 2^-126 at least), so that an infinite V is not multiplied by a zero or by both signs; fp8 /
// NVFP4: V exact in f16, P in f16 (2^-11).
template <int FMT, int NT>
struct PFrag {
  uint32_t b0[NT], b1[NT], l0[NT], l1[NT];
  __device__ __forceinline__ explicit PFrag(const float (&p)[NT][4]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (FMT == PBS_KV_BF16) {
        float lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          lo[i] = fminf(fmaxf(p[t][i] - bf16_hi(__float_as_uint(p[t][i])), 0x1p-126f), p[t][i]);
        b0[t] = movmatrix_trans(__byte_perm(__float_as_uint(p[t][0]), __float_as_uint(p[t][1]), 0x7632));
        b1[t] = movmatrix_trans(__byte_perm(__float_as_uint(p[t][2]), __float_as_uint(p[t][3]), 0x7632));
        l0[t] = movmatrix_trans(pack_bf16(lo[0], lo[1]));
        l1[t] = movmatrix_trans(pack_bf16(lo[2], lo[3]));
      } else {
        b0[t] = movmatrix_trans(pack_f16(p[t][0], p[t][1]));
        b1[t] = movmatrix_trans(pack_f16(p[t][2], p[t][3]));
      }
    }
  }
  __device__ __forceinline__ void mma(int t, float (&o)[4], const uint32_t (&vf)[4]) const {
    if (FMT == PBS_KV_BF16) {
      mma_bf16(o, vf, b0[t], b1[t]);
      mma_bf16(o, vf, l0[t], l1[t]);
    } else {
      mma_f16(o, vf, b0[t], b1[t]);
    }
  }
};

// O^T += V^T P^T of one page, p[tile][..] laid out as page_scores returns it.
template <int FMT, int NT>
__device__ __forceinline__ void page_pv(uint32_t st, const float (&p)[NT][4], int lane, float (&o)[NT][8][4]) {
  const PFrag<FMT, NT> pf(p);
  VPage<FMT> v(st, lane);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if ((i & 3) == 0) v.begin(i >> 2);
    uint32_t vf[4];
    v.tile(i, vf);
#pragma unroll
    for (int t = 0; t < NT; ++t) pf.mma(t, o[t][i], vf);
  }
}

// Infinities or NaN in the words of 16-bit pairs (bf16, or f16).
template <int FMT>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  constexpr uint32_t kExp = FMT == PBS_KV_BF16 ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = FMT == PBS_KV_BF16 ? 0x00800080u : 0x04000400u;
  return ((x & kExp) + kOne) & 0x80008000u;  // an exponent of ones carries into the sign's place
}

// The same for a page that the group's rows see in part: `any` are the keys that some row sees; `same`: every
// row sees just those. V of the others is cleared in registers before it meets P, since 0 * NaN is NaN. Where
// the rows differ, a key that one sees and another does not has P = 0 for the latter, which a finite V leaves at
// 0; only when such a page holds a V that is not finite does it go row by row, each row's product added to its own
// columns. bits(r): the keys row r sees; row_of: the lane's columns' rows.
template <int FMT, int NT, typename Bits>
__device__ __forceinline__ void page_pv_masked(uint32_t st, const float (&p)[NT][4], int lane, float (&o)[NT][8][4],
                                               uint32_t any, bool same, int rows, Bits bits,
                                               const int (&row_of)[NT][2]) {
  // (each pass reads V anew: nothing but O lives across them)
  bool finite = true;
  if (!same) {
    const uint2 m = key_words(any, lane & 3);
    VPage<FMT> v(st, lane);
    uint32_t bad = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & 3) == 0) v.begin(i >> 2);
      uint32_t vf[4];
      v.tile(i, vf);
      bad |= not_finite<FMT>(vf[0] & m.x) | not_finite<FMT>(vf[1] & m.x) | not_finite<FMT>(vf[2] & m.y) |
             not_finite<FMT>(vf[3] & m.y);
    }
    finite = !__any_sync(0xffffffffu, bad != 0u);
  }
  const int passes = finite ? 1 : rows;
#pragma unroll 1
  for (int r = 0; r < passes; ++r) {
    const PFrag<FMT, NT> pf(p);
    const uint2 m = key_words(finite ? any : bits(r), lane & 3);
    VPage<FMT> v(st, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & 3) == 0) v.begin(i >> 2);
      uint32_t vf[4];
      v.tile(i, vf);
      vf[0] &= m.x;
      vf[1] &= m.x;
      vf[2] &= m.y;
      vf[3] &= m.y;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        pf.mma(t, x, vf);
        const bool y0 = finite || row_of[t][0] == r, y1 = finite || row_of[t][1] == r;
        o[t][i][0] = y0 ? o[t][i][0] + x[0] : o[t][i][0];
        o[t][i][1] = y1 ? o[t][i][1] + x[1] : o[t][i][1];
        o[t][i][2] = y0 ? o[t][i][2] + x[2] : o[t][i][2];
        o[t][i][3] = y1 ? o[t][i][3] + x[3] : o[t][i][3];
      }
    }
  }
}

// Output dims of accumulator words 0/1 and 2/3 of o[..][i].
template <int FMT>
__device__ __forceinline__ int o_dim(int i, int half, int hh) {
  return FMT == PBS_KV_BF16 ? 16 * i + hh + 8 * half : 16 * hh + 2 * i + half;
}

}  // namespace wp
}  // namespace pbs
