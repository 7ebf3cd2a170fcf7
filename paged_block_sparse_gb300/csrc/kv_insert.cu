// K/V insert: the K and V rows of new tokens into the pages of the cache, in the cache's format.
//
// For token n and kv head g, with block = slot / 128 and page = block * block_page_stride +
// (slot % 128) / 16, row = slot % 16:
//   bf16   the 128 + 128 elements as they are,
//   fp8    e4m3(x / scale), round to nearest even, saturating at +-448 (NaN stays NaN),
//   NVFP4  per 16 elements: s = e4m3(max |x / scale| / 6), code = e2m1(x / scale / s); s = 0 (a
//          group of zeros, or too small for e4m3) stores zeros. Infinities saturate; a NaN makes
//          its group's scale NaN, so the 16 values read back as NaN (e2m1 has none).
// x / scale is x * (1 / scale) with the reciprocal rounded to fp32 by the host (2^-24 next to
// e4m3's 2^-4 and e2m1's 2^-2); x / s is a true division, the codes' borders depend on it.
//
// An HBM copy with a few conversions per element: one warp per (token, kv heads in chunks of
// kHeads), lanes 0-15 hold K and 16-31 V, 8 elements (16 bytes of bf16) each, so a head's row is
// one 512-byte read per side and one 512 / 256 / 2 x 64-byte write. kHeads heads per warp are
// loaded before the first is converted (bytes in flight). Measured: 22528 tokens x 8 heads to fp8
// (139 MB) 20.4 us on the device = the copy rate, 24.6 us a call; 64 tokens 5 us.
#include "pbs_device.cuh"
#include "pbs_internal.h"

namespace pbs {
namespace {

constexpr int kWarps = 8;
constexpr int kHeads = 4;
constexpr int kNvfp4Slot = 1152;

// Eight bf16 elements of this lane's side.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int64_t stride) {
  if (kVec) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(__ldg(p + 2 * i * stride)) |
           (static_cast<uint32_t>(__ldg(p + (2 * i + 1) * stride)) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two floats to e4m3 (first to the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two floats to e2m1 (first to the low nibble), nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tmov.b16 %0, {b, 0};\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

template <int FMT, bool kVec>
__global__ void __launch_bounds__(kWarps * 32) kv_insert_kernel(const KvInsertArgs a) {
  const int lane = threadIdx.x & 31;
  const int chunks = (a.num_kv_heads + kHeads - 1) / kHeads;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.num_tokens) * chunks) return;
  const int n = static_cast<int>(w / chunks), h0 = static_cast<int>(w % chunks) * kHeads;
  const int64_t slot = __ldg(a.slot_mapping + static_cast<int64_t>(n) * a.slot_stride);
  if (slot < 0) return;  // padding
  const int64_t block = slot / kSparseBlock;
  const int64_t page = block < a.num_pages ? block * a.block_page_stride + (slot % kSparseBlock) / kPageRows
                                           : a.num_pages;
  if (page >= a.num_pages) {
    if (lane == 0) set_err(a.err_word, PBS_DEVERR_SLOT_OOB);
    return;
  }
  const int row = static_cast<int>(slot % kPageRows);
  const int side = lane >> 4, c = lane & 15;  // side 0: K, 1: V; elements 8c .. 8c + 7
  const uint16_t* src = side ? a.v + n * a.v_row_stride + 8 * c * a.v_dim_stride
                             : a.k + n * a.k_row_stride + 8 * c * a.k_dim_stride;
  const int64_t head_stride = side ? a.v_head_stride : a.k_head_stride;
  const int64_t dim_stride = side ? a.v_dim_stride : a.k_dim_stride;
  const float inv = side ? a.inv_v_scale : a.inv_k_scale;
  uint4 x[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (h0 + i < a.num_kv_heads) x[i] = load8<kVec>(src + (h0 + i) * head_stride, dim_stride);
  uint8_t* dst = a.kv_cache + page * a.page_stride_bytes;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int g = h0 + i;
    if (g >= a.num_kv_heads) break;
    if (FMT == PBS_KV_BF16) {
      *reinterpret_cast<uint4*>(dst + (g * kPageRows + row) * 512 + side * 256 + 16 * c) = x[i];
      continue;
    }
    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(u[j]) * inv;
      f[2 * j + 1] = bf16_hi(u[j]) * inv;
    }
    if (FMT == PBS_KV_FP8_E4M3) {
      *reinterpret_cast<uint2*>(dst + (g * kPageRows + row) * 256 + side * 128 + 8 * c) =
          make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16), e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
    } else {
      // the 16-element group is this lane's 8 elements and its neighbour's
      float mx = 0.f;
      bool nan = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mx = fmaxf(mx, fabsf(f[j]));
        nan |= f[j] != f[j];
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      nan |= __shfl_xor_sync(0xffffffffu, nan, 1) != 0;
      const uint32_t sb = nan ? 0x7fu : e4m3x2(mx * (1.0f / 6.0f), 0.f) & 0xffu;
      float s;
      {
        const uint32_t h = e4m3x2_to_f16x2(sb);
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(s) : "r"(h));
      }
      uint32_t code = 0;
      if (s > 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code |= e2m1x2(__fdiv_rn(f[2 * j], s), __fdiv_rn(f[2 * j + 1], s)) << (8 * j);
      }
      uint8_t* sl = dst + (2 * g + side) * kNvfp4Slot;
      *reinterpret_cast<uint32_t*>(sl + row * 64 + 4 * c) = code;
      if ((c & 1) == 0) sl[1024 + row * 8 + (c >> 1)] = static_cast<uint8_t>(sb);
    }
  }
}

template <int FMT>
cudaError_t launch_fmt(const KvInsertArgs& a, bool vec, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(a.num_tokens) * ((a.num_kv_heads + kHeads - 1) / kHeads);
  const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
  if (vec) kv_insert_kernel<FMT, true><<<grid, kWarps * 32, 0, stream>>>(a);
  else kv_insert_kernel<FMT, false><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_insert(const KvInsertArgs& a, cudaStream_t stream) {
  // 16-byte loads when every row of K and V starts on a 16-byte boundary with unit dim stride
  const bool vec = a.k_dim_stride == 1 && a.v_dim_stride == 1 && a.k_row_stride % 8 == 0 && a.v_row_stride % 8 == 0 &&
                   a.k_head_stride % 8 == 0 && a.v_head_stride % 8 == 0 &&
                   reinterpret_cast<uintptr_t>(a.k) % 16 == 0 && reinterpret_cast<uintptr_t>(a.v) % 16 == 0;
  switch (a.kv_dtype) {
    case PBS_KV_BF16: return launch_fmt<PBS_KV_BF16>(a, vec, stream);
    case PBS_KV_FP8_E4M3: return launch_fmt<PBS_KV_FP8_E4M3>(a, vec, stream);
    case PBS_KV_NVFP4: return launch_fmt<PBS_KV_NVFP4>(a, vec, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pbs
