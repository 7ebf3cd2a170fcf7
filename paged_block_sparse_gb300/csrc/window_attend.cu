// Window attend with sinks over the paged cache: every key n <= p of the query's request with
// n > p - window (or any n when window is 0) or n < num_sinks.
//
// One CTA per (row, query head), four warps striding over the visible keys, one key at a time:
// lane l holds dims 4l .. 4l + 3. fp32 throughout, online softmax per warp, one merge.
#include "pbs_device.cuh"
#include "pbs_internal.h"

namespace pbs {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float half_of(uint32_t h2, int hi) {
  float f;
  const uint16_t h = static_cast<uint16_t>(hi ? h2 >> 16 : h2);
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return f;
}

// Dims 4l .. 4l + 3 of K (side 0) or V (side 1) of a page row.
__device__ __forceinline__ void load4(const uint8_t* page, int fmt, int g, int row, int side, int lane, float (&x)[4]) {
  if (fmt == PBS_KV_BF16) {
    const uint2 w = *reinterpret_cast<const uint2*>(page + (g * kPageRows + row) * 512 + side * 256 + lane * 8);
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  } else if (fmt == PBS_KV_FP8_E4M3) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(page + (g * kPageRows + row) * 256 + side * 128 + lane * 4);
    const uint32_t a = e4m3x2_to_f16x2(w), b = e4m3x2_to_f16x2(w >> 16);
    x[0] = half_of(a, 0); x[1] = half_of(a, 1); x[2] = half_of(b, 0); x[3] = half_of(b, 1);
  } else {
    const uint8_t* sl = page + (2 * g + side) * 1152;
    const uint32_t w = *reinterpret_cast<const uint16_t*>(sl + row * 64 + lane * 2);
    const float s = half_of(e4m3x2_to_f16x2(sl[1024 + row * 8 + (lane >> 2)]), 0);
    const uint32_t a = e2m1x2_to_f16x2(w & 0xff), b = e2m1x2_to_f16x2(w >> 8);
    x[0] = half_of(a, 0) * s; x[1] = half_of(a, 1) * s; x[2] = half_of(b, 0) * s; x[3] = half_of(b, 1) * s;
  }
}

__global__ void __launch_bounds__(kWarps * 32) window_attend_kernel(const WindowArgs a) {
  const int row = blockIdx.x, h = blockIdx.y, g = h / a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int req, pos;
  if (a.cu_seqlens_q != nullptr) {
    if (row >= __ldg(a.cu_seqlens_q + a.num_reqs)) return;  // behind the last request
    prefill_position(row, a.cu_seqlens_q, a.num_reqs, a.seq_lens, req, pos);
  } else {
    decode_position(row, a.decode_query_len, a.seq_lens, req, pos);
  }
  const int low = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int head = pos < 0 ? 0 : min(a.num_sinks, low);
  const int count = pos < 0 ? 0 : head + pos - low + 1;
  const uint16_t* qp = a.q + row * a.q_row_stride + h * a.q_head_stride + 4 * lane;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __uint_as_float(static_cast<uint32_t>(qp[i]) << 16);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = warp; i < count; i += kWarps) {
    const int n = i < head ? i : low + i - head;
    const int b = n / kSparseBlock;
    if (b >= a.max_blocks) {
      set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
      continue;
    }
    const int phys = __ldg(a.page_table + req * a.pt_row_stride + b);
    const int64_t page = static_cast<int64_t>(phys) * a.block_page_stride + n % kSparseBlock / kPageRows;
    if (phys < 0 || page >= a.num_pages) {
      set_err(a.err_word, PBS_DEVERR_PAGE_OOB);
      continue;
    }
    const uint8_t* base = a.kv_cache + page * a.page_stride_bytes;
    float k[4], v[4];
    load4(base, a.kv_dtype, g, n % kPageRows, 0, lane, k);
    load4(base, a.kv_dtype, g, n % kPageRows, 1, lane, v);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - mu), p = ex2(s - mu);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = o[j] * f + p * v[j];
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kHeadDim];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) so[warp][4 * lane + j] = o[j];
  __syncthreads();
  float M = -INFINITY, L = 0.f, O = 0.f;
  const int d = threadIdx.x;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  if (M != -INFINITY)
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sm[w] - M);
      L += f * sl[w];
      O += f * so[w][d];
    }
  const float r = L != 0.f ? a.v_scale * O / L : 0.f;
  uint16_t bits;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(r));
  a.out[row * a.out_row_stride + h * a.out_head_stride + d] = bits;
  if (a.lse != nullptr && d == 0) a.lse[row * a.lse_row_stride + h] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_window_attend(const WindowArgs& a, cudaStream_t stream) {
  window_attend_kernel<<<dim3(a.num_rows, a.num_heads), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pbs
