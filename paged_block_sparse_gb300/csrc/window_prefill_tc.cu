// Window attend with sinks, varlen prefill, on the 5th-generation tensor cores (tcgen05 + TMEM). For a
// token at position p of its request, out = v_scale * softmax(softmax_scale * k_scale * q K^T) V over the
// keys 0 <= n <= p with n > p - window (any n when window is 0) or n < num_sinks.
//
// 1. convert_kernel: K and V of every 128-key block that some token of its request sees, per kv head, as
//    the 32 KiB shared-memory images of the MMA operands ([64-dim half][128 keys][128 B], 128B swizzle): K
//    in bf16 (exact for every format), V in fp16 times 2^-e with the block's largest finite |V| at
//    2^14..2^15 (exact: bf16 has 8 significant bits, fp16 keeps 28 binades below its largest value). It
//    resolves the page table once, dequantises once, and clears the keys that nobody sees, so that the
//    attend streams images with plain bulk copies. HBM-bound.
// 2. attend: persistent, one CTA per SM. A tile is 2 T consecutive tokens of one request (T = 128 / G) and
//    one kv head: two 128-row MMA tiles A and B (row = token * G + head) that share every K and V block, so
//    a block is read once per 256 rows, and the tensor cores work on one while the softmax of the other
//    runs. Bound by the tensor pipe and, next, by the softmax warps' issue slots.
//      warp 2     schedules: the next tile's description in one of two slots, and its Q (tensor map)
//      warp 0     loads: K and V images through one ring of 4 stages
//      warp 1     issues the MMAs, in the order PV_A(n-1) S_A(n) PV_B(n-1) S_B(n) over the blocks of all its tiles
//      warp 3     waits for the ring on warp 1's behalf
//      warps 4-7  softmax and output of A, one thread per row; warps 8-11 of B
//    TMEM: S_A, S_B, O_A, O_B, 128 fp32 columns each. A row's thread reads its 128 scores, writes P as fp16
//    over the first 64 of those columns (the A operand of PV). MMAs of one thread run in issue order, so
//    S(i + 1) may overwrite P(i) as soon as PV(i) has been issued.
//    P is rounded to fp16 (2^-11; bf16's 2^-8 would double the error of a bf16 output), sums stay in fp32.
//    Online softmax in base 2: the reference moves, and O is rescaled, only when the row maximum passes
//    it by 2^8. Each row keeps the exponent E of its O (O holds sum(P V) * 2^-E); a block of exponent e
//    enters as P * 2^(e - E), and E moves when e - E leaves [-8, 7] (down only as far as O's fp32 has room).
//    Infinities and NaN in V are cleared in the images (0 * NaN would reach rows that do not see them) and
//    added, after the output, to the rows that do.
// Blocks are masked per row only where a row's border crosses them; a block that no row of A (or B) sees is
// skipped for it. Multiplying just the 32-key parts of a crossed block that some row sees cost more in the MMA
// thread and the softmax's code than it saved (703 -> 744 us); so did two threads per row (972 us: 96 to 104
// registers a thread spill).
//
// Measured (events, L2 flushed): prompts of 2k-8k tokens, bf16, 64 / 8 heads, window 1024 + 64 sinks 703 us =
// 1032 TFLOP/s on the keys that are seen, 53 % of the measured dense rate (38 us of it the images); 2 x 4096
// tokens after 16k and 32k, NVFP4, 64 / 4 heads, window 4096 + 128 sinks 775 us = 1463 TFLOP/s, 75 %. A step (one
// block, both tiles) takes 2.9k clk for 2048 clk of MMAs: each tile's chain is its softmax (1300), PV and S
// (512 each) and 600 of barrier and MMA latency. A tile's end costs 5k clk.
#include "mbar_wait.cuh"
#include "pbs_device.cuh"
#include "pbs_internal.h"
#include "tc_device.cuh"

namespace pbs {
namespace {

constexpr int kRows = 128;
constexpr int kThreadsTc = 384;
constexpr int kImage = 32768;          // bytes of one K or V image
constexpr int kHalf = kImage / 2;      // its first 64 dims
constexpr int kQTile = kRows * kHeadDim * 2;
constexpr int kRing = 4;
constexpr int kOutStage = 8 * 4096;   // 32 rows x 64 dims of bf16 per softmax warp
constexpr float kLazyLog2 = 8.0f;
constexpr int kExpUp = 7, kExpDown = -8;
constexpr int kNoExp = -1000;  // E before the row's first block (far from any)
constexpr unsigned long long kWaitNs = 100000000ull;
// block info word: V exponent + 128 in the low byte (0: no finite V but zeros), valid pages in the next,
// then whether some V is infinite or NaN
constexpr int kInfoBias = 128;
constexpr int kMaxConvertCtas = 16384;  // 27 waves of the GPU: no call pays for more empty slots than that
constexpr int kInfoOdd = 1 << 16;
__device__ __forceinline__ int info_pages(int info) { return (info >> 8) & 0xff; }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// What a request needs of the cache: blocks [0, head) and [first, last].
struct Span {
  int head, first, count;  // count: blocks in all
};

__device__ __forceinline__ Span span_of(const WindowArgs& a, int p0, int p1) {
  Span s = {0, 0, 0};
  if (p1 < 0) return s;
  const int low = a.window > 0 ? max(0, max(p0, 0) - a.window + 1) : 0;
  const int head = min(a.num_sinks, low);
  // blocks past the page table are left out (the images' workspace has no room for them)
  const int end = min(p1 / kSparseBlock + 1, a.max_blocks);
  s.first = min(low / kSparseBlock, end);
  s.head = min((head + kSparseBlock - 1) / kSparseBlock, s.first);
  s.count = s.head + end - s.first;
  return s;
}

// Query tokens of request r (the padding of q does not count) and its first position.
__device__ __forceinline__ int tokens_of(const WindowArgs& a, int r, int* c0, int* p0) {
  *c0 = __ldg(a.cu_seqlens_q + r);
  const int n = __ldg(a.cu_seqlens_q + r + 1) - *c0;
  *p0 = __ldg(a.seq_lens + r) - n;
  return *c0 < 0 ? 0 : max(0, min(n, a.num_rows - *c0));
}

// The request that holds entry `index` when request r has count(r) entries, in order; `at` its entry there.
// -1: none. A whole warp.
template <typename Count>
__device__ __forceinline__ int find_request(const WindowArgs& a, int index, int lane, int* at, Count count) {
  int before = 0;
  for (int r0 = 0; r0 < a.num_reqs; r0 += 32) {
    const int n = r0 + lane < a.num_reqs ? count(r0 + lane) : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    const int x = index - before - (incl - n);
    const uint32_t hit = __ballot_sync(0xffffffffu, x >= 0 && x < n);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      *at = __shfl_sync(0xffffffffu, x, src);
      return r0 + src;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return -1;
}

__device__ __forceinline__ int blocks_of(const WindowArgs& a, int r) {
  int c0, p0;
  const int n = tokens_of(a, r, &c0, &p0);
  return n > 0 ? span_of(a, p0, p0 + n - 1).count : 0;
}

__device__ __forceinline__ float exp2i(int n) {  // 2^n, 0 below fp32's normal range
  return n < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + n) << 23);
}

// ---- images ------------------------------------------------------------------------------------

__device__ __forceinline__ float f16_lo(uint32_t x) {
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(x));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t x) {
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, hi;\n\t}" : "=f"(f) : "r"(x));
  return f;
}

// One quarter (32 dims) of a key's K or V as stored.
template <int FMT>
struct Quarter {
  uint4 w[FMT == PBS_KV_BF16 ? 4 : FMT == PBS_KV_FP8_E4M3 ? 2 : 1];
  uint32_t scales;  // NVFP4: the two e4m3 block scales
};

template <int FMT>
__device__ __forceinline__ Quarter<FMT> load_quarter(const uint8_t* page, int g, int row, int side, int quarter) {
  Quarter<FMT> q;
  q.scales = 0;
  if (FMT == PBS_KV_NVFP4) {
    const uint8_t* sl = page + (2 * g + side) * 1152;
    q.w[0] = __ldg(reinterpret_cast<const uint4*>(sl + row * 64) + quarter);
    q.scales = __ldg(reinterpret_cast<const uint16_t*>(sl + 1024 + row * 8) + quarter);
  } else {
    constexpr int kRow = FMT == PBS_KV_BF16 ? 512 : 256;
    constexpr int kN = FMT == PBS_KV_BF16 ? 4 : 2;
    const uint4* p = reinterpret_cast<const uint4*>(page + (g * kPageRows + row) * kRow + side * (kRow / 2)) + quarter * kN;
#pragma unroll
    for (int i = 0; i < kN; ++i) q.w[i] = __ldg(p + i);
  }
  return q;
}

// Elements 8c .. 8c + 7 of the quarter as float (exact).
template <int FMT>
__device__ __forceinline__ void eight(const Quarter<FMT>& q, int c, float (&v)[8]) {
  if (FMT == PBS_KV_BF16) {
    const uint32_t u[4] = {q.w[c].x, q.w[c].y, q.w[c].z, q.w[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(u[i]);
      v[2 * i + 1] = bf16_hi(u[i]);
    }
  } else if (FMT == PBS_KV_FP8_E4M3) {
    const uint4& w = q.w[c >> 1];
    const uint32_t lo = (c & 1) ? w.z : w.x, hi = (c & 1) ? w.w : w.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = e4m3x2_to_f16x2((i < 2 ? lo : hi) >> (16 * (i & 1)));
      v[2 * i] = f16_lo(h);
      v[2 * i + 1] = f16_hi(h);
    }
  } else {
    const uint32_t w = c == 0 ? q.w[0].x : c == 1 ? q.w[0].y : c == 2 ? q.w[0].z : q.w[0].w;
    const float s = f16_lo(e4m3x2_to_f16x2((q.scales >> (8 * (c >> 1))) & 0xffu));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = e2m1x2_to_f16x2((w >> (8 * i)) & 0xffu);
      v[2 * i] = f16_lo(h) * s;
      v[2 * i + 1] = f16_hi(h) * s;
    }
  }
}

// CTA (slot, kv head), 512 threads: thread t converts dims 32 (t % 4) .. of key t / 4, so that a warp reads
// whole rows of eight keys. The slots in use come first; a page table far wider than its requests has many that
// are not, so a CTA of a large grid takes every gridDim.x-th slot until it meets one.
template <int FMT>
__global__ void __launch_bounds__(512) convert_kernel(const WindowArgs a) {
  __shared__ int s_req, s_block;
  __shared__ float s_max[16];
  __shared__ uint32_t s_pages;
  __shared__ int s_odd;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = blockIdx.y;
  if (t == 0 && blockIdx.x == 0 && g == 0) *a.next_tile = 0;
  for (int slot = blockIdx.x; slot < a.image_slots; slot += gridDim.x) {
    if (warp == 0) {
      int at = 0;
      const int r = find_request(a, slot, lane, &at, [&](int i) { return blocks_of(a, i); });
      if (lane == 0) {
        s_req = r;
        s_pages = 0;
        s_odd = 0;
        if (r >= 0) {
          int c0, p0;
          const int n = tokens_of(a, r, &c0, &p0);
          const Span s = span_of(a, p0, p0 + n - 1);
          s_block = at < s.head ? at : s.first + at - s.head;
          if (at == 0 && (p0 + n - 1) / kSparseBlock >= a.max_blocks) set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
        }
      }
    }
    __syncthreads();
    const int r = s_req;
    if (r < 0) return;
    const int b = s_block, key = t >> 2, quarter = t & 3;
    int c0, p0;
    const int n_tok = tokens_of(a, r, &c0, &p0);
    const int n = b * kSparseBlock + key;
    bool live = n < p0 + n_tok && (a.window == 0 || n > max(p0, 0) - a.window || n < a.num_sinks);
    const uint8_t* page = a.kv_cache;
    const int phys = __ldg(a.page_table + static_cast<int64_t>(r) * a.pt_row_stride + b);
    const int64_t p = static_cast<int64_t>(phys) * a.block_page_stride + key / kPageRows;
    if (phys < 0 || p >= a.num_pages) {
      if (live) set_err(a.err_word, PBS_DEVERR_PAGE_OOB);
      live = false;
    } else {
      page += p * a.page_stride_bytes;
      if (t % 64 == 0) atomicOr(&s_pages, 1u << (key / kPageRows));
    }
    Quarter<FMT> kq, vq;
    if (live) {
      kq = load_quarter<FMT>(page, g, key % kPageRows, 0, quarter);
      vq = load_quarter<FMT>(page, g, key % kPageRows, 1, quarter);
    }
    const int64_t image = static_cast<int64_t>(slot) * a.num_kv_heads + g;
    uint8_t* kdst = a.k_images + image * kImage;
    uint8_t* vdst = a.v_images + image * kImage;
    float mx = 0.f;
    bool odd = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float v[8] = {};
      if (live) eight<FMT>(kq, c, v);
      const int c16 = quarter * 4 + c;  // 16-byte chunk of the key's 256 bytes
      *reinterpret_cast<uint4*>(kdst + (c16 >> 3) * kHalf + key * 128 + (((c16 & 7) ^ (key & 7)) << 4)) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      if (live) {
        eight<FMT>(vq, c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mx = fmaxf(mx, finite(v[i]) ? fabsf(v[i]) : 0.f);
          odd |= !finite(v[i]);
        }
      }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if (lane == 0) s_max[warp] = mx;
    if (odd) s_odd = 1;
    __syncthreads();
    odd = s_odd != 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) mx = fmaxf(mx, s_max[w]);
    int e = mx > 0.f ? static_cast<int>((__float_as_uint(mx) >> 23) & 0xffu) - 127 - 14 : 0;
    e = max(-100, min(100, e));
    const float sc = exp2i(-e);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float v[8] = {};
      if (live) eight<FMT>(vq, c, v);
      if (odd)  // 0 * infinity would reach the rows that do not see it: the attend adds these for those that do
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = finite(v[i]) ? v[i] : 0.f;
      const int c16 = quarter * 4 + c;
      *reinterpret_cast<uint4*>(vdst + (c16 >> 3) * kHalf + key * 128 + (((c16 & 7) ^ (key & 7)) << 4)) =
          make_uint4(pack_f16(v[0] * sc, v[1] * sc), pack_f16(v[2] * sc, v[3] * sc), pack_f16(v[4] * sc, v[5] * sc),
                     pack_f16(v[6] * sc, v[7] * sc));
    }
    if (t == 0) a.image_info[image] = (mx > 0.f ? e + kInfoBias : 0) | (static_cast<int>(s_pages) << 8) | (odd ? kInfoOdd : 0);
    __syncthreads();
  }
}

// ---- attend -------------------------------------------------------------------------------------

struct Tile {
  int end;            // no tile: the list is done
  int req, g, t0, n_tok;  // request, kv head, first row of q, tokens
  int p0;             // position of the first
  int head, first, count;
  int slot0, req_head, req_first;  // the request's first image slot, and its span: block b's slot is
                                   // slot0 + (b < req_head ? b : req_head + b - req_first)
};

struct Ctl {
  uint64_t q_full[2], q_empty[2];  // of A, of B
  uint64_t full[kRing], empty[kRing];
  uint64_t s_full[2], p_full[2];
  uint64_t pv_done[2];    // the tile's last PV
  uint64_t drained;       // every MMA of the CTA
  uint64_t tile_full[2], tile_empty[2];
  uint32_t tmem;
  int32_t abort;
  Tile tile[2];
};

constexpr size_t kSmemTc = 2 * kQTile + kRing * kImage + kOutStage + sizeof(Ctl);
static_assert(kSmemTc <= 232448, "shared memory exceeds 227 KiB");
constexpr uint32_t kTileUsers = 3 + 8;  // loads, MMAs, gate, the softmax warps

__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, Ctl* ctl, int32_t* err) {
  if (mbar_wait_quick(bar, parity, kWaitNs)) return true;
  set_err(err, PBS_DEVERR_TIMEOUT);
  atomicExch(&ctl->abort, 1);
  return false;
}
__device__ __forceinline__ bool warp_wait_on(uint64_t* bar, uint32_t parity, Ctl* ctl, int32_t* err) {
  return __all_sync(0xffffffffu, wait_on(bar, parity, ctl, err));
}
__device__ __forceinline__ bool aborted(Ctl* ctl) { return *reinterpret_cast<volatile int32_t*>(&ctl->abort) != 0; }

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// One thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// The i-th block of a tile's list.
__device__ __forceinline__ int tile_block(const Tile& t, int i) { return i < t.head ? i : t.first + i - t.head; }

// Positions of the first and last live token of MMA tile x (0: A, 1: B); last < first: none.
template <int kG>
__device__ __forceinline__ void tile_rows(const Tile& t, int x, int* pa, int* pb) {
  constexpr int T = kRows / kG;
  *pa = t.p0 + x * T;
  *pb = t.p0 + min(t.n_tok, (x + 1) * T) - 1;
}

// Entries of a tile's list that MMA tile x works on: all i < t.head, and x .. y (y < 0: it has no rows).
template <int kG>
__device__ __forceinline__ int2 seen_range(const WindowArgs& a, const Tile& t, int x) {
  int pa, pb;
  tile_rows<kG>(t, x, &pa, &pb);
  if (pb < pa || pb < 0) return make_int2(0, -1);
  const int low = a.window > 0 ? max(0, max(pa, 0) - a.window + 1) : 0;
  // the block of the first key in the window, or t.first when the sinks reach past t.first
  const int lo = a.window > 0 && a.num_sinks > t.first * kSparseBlock ? t.first : max(t.first, low / kSparseBlock);
  return make_int2(t.head + lo - t.first, min(t.count - 1, t.head + pb / kSparseBlock - t.first));
}

// Which of the keys base .. base + 31 a row at position p sees; pages: valid bits of the two pages.
__device__ __forceinline__ uint32_t row_bits(const WindowArgs& a, int base, int p, bool live, int pages) {
  const int behind = p - base;
  uint32_t w = !live || behind < 0 ? 0u : behind >= 31 ? 0xffffffffu : (2u << behind) - 1u;
  if (a.window > 0) {
    const int lo = p - a.window + 1 - base, s = a.num_sinks - base;
    const uint32_t in = lo <= 0 ? 0xffffffffu : lo > 31 ? 0u : 0xffffffffu << lo;
    const uint32_t sink = s <= 0 ? 0u : s >= 32 ? 0xffffffffu : (1u << s) - 1u;
    w &= in | sink;
  }
  return w & (((pages & 1) ? 0xffffu : 0u) | ((pages & 2) ? 0xffff0000u : 0u));
}

// The last entry tile x works on (-1: none).
__device__ __forceinline__ int last_seen(int2 r, int head) { return r.y < 0 ? -1 : r.y >= r.x ? r.y : head - 1; }

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// 32 lanes x 16 consecutive TMEM columns.
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// out[d] += v_scale * V[d] where V of a key is infinite or NaN (its weight, above zero, leaves those as they are).
template <int FMT>
__device__ __forceinline__ void add_odd_values(const uint8_t* page, int g, int row, float v_scale, uint16_t* out) {
#pragma unroll 1
  for (int quarter = 0; quarter < 4; ++quarter) {
    const Quarter<FMT> q = load_quarter<FMT>(page, g, row, 1, quarter);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float v[8];
      eight<FMT>(q, c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint16_t* o = out + quarter * 32 + c * 8 + i;
        if (!finite(v[i])) *o = static_cast<uint16_t>(pack_bf16(bf16_lo(*o) + v_scale * v[i], 0.f));
      }
    }
  }
}

// add_odd_values for the keys that a row at position p sees, over its MMA tile's blocks.
__device__ __noinline__ void add_odd_blocks(const WindowArgs& a, const Tile& t, int2 range, int p, uint16_t* own) {
#pragma unroll 1
  for (int i = 0; i < t.count; ++i) {
    if (i >= t.head && (i < range.x || i > range.y)) continue;
    const int b = tile_block(t, i);
    const int info = __ldg(a.image_info + static_cast<int64_t>(t.slot0 + (b < t.req_head ? b : t.req_head + b - t.req_first)) *
                                              a.num_kv_heads + t.g);
    if (!(info & kInfoOdd)) continue;
    const int64_t p0 = static_cast<int64_t>(__ldg(a.page_table + static_cast<int64_t>(t.req) * a.pt_row_stride + b)) *
                       a.block_page_stride;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t w = row_bits(a, b * kSparseBlock + 32 * c, p, true, info >> (8 + 2 * c));
#pragma unroll 1
      for (; w != 0; w &= w - 1) {
        const int key = 32 * c + __ffs(w) - 1;
        const uint8_t* page = a.kv_cache + (p0 + key / kPageRows) * a.page_stride_bytes;
        switch (a.kv_dtype) {
          case PBS_KV_BF16: add_odd_values<PBS_KV_BF16>(page, t.g, key % kPageRows, a.v_scale, own); break;
          case PBS_KV_FP8_E4M3: add_odd_values<PBS_KV_FP8_E4M3>(page, t.g, key % kPageRows, a.v_scale, own); break;
          default: add_odd_values<PBS_KV_NVFP4>(page, t.g, key % kPageRows, a.v_scale, own);
        }
      }
    }
  }
}

template <int kG>
__global__ void __launch_bounds__(kThreadsTc, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ WindowArgs a) {
  constexpr int T = kRows / kG;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled operands need it
    if (threadIdx.x == 0 && blockIdx.x == 0) set_err(a.err_word, PBS_DEVERR_TIMEOUT);
    return;
  }
  uint8_t* q_s = smem;
  uint8_t* ring = smem + 2 * kQTile;
  uint8_t* out_s = ring + kRing * kImage;
  Ctl* ctl = reinterpret_cast<Ctl*>(out_s + kOutStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ctl->abort = 0;
    mbar_init(&ctl->drained, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 2);  // the MMAs and the gate
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], i == 0 ? 5 : 4);  // A's: the softmax warps and the gate
      mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->tile_full[i], 1);
      mbar_init(&ctl->tile_empty[i], kTileUsers);
    }
    fence_mbar_init();
  }
  if (warp == 2) tc::alloc(&ctl->tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem;  // S_A, S_B, O_A, O_B

  // the softmax warps hold a row's 128 scores in registers: 128 x 88 + 256 x 208 = the launch's 384 x 168
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------------ softmax and output
    const int x = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const int tok = row / kG, h = row % kG;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + x * 128 + lane_off, to = tmem + 256 + x * 128 + lane_off;
    const float sl2 = a.scale_log2;
    int ns = 0;     // blocks of this MMA tile over the CTA's tiles
    int tiles = 0;  // tiles that had any
    bool ok = true;
    Tile t;
    const auto next_tile = [&](int k) {  // false: a wait gave up
      if (!warp_wait_on(&ctl->tile_full[k & 1], (k >> 1) & 1, ctl, a.err_word)) return false;
      t = ctl->tile[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->tile_empty[k & 1]);
      return true;
    };
    ok = next_tile(0);
    for (int k = 0; ok && !t.end && !aborted(ctl); ++k) {
      int pa, pb;
      tile_rows<kG>(t, x, &pa, &pb);
      const bool live = x * T + tok < t.n_tok;
      const int p = pa + tok;
      // positions of the warp's rows (those without a token count: they are not written)
      const int pw0 = pa + quad * 32 / kG, pw1 = pa + (quad * 32 + 31) / kG;
      float m = -INFINITY, l = 0.f;
      int E = kNoExp;
      int top = 0;  // at E's last move: the largest V (its e) that O held, by weight
      bool started = false;  // the tile has had a block: O holds something
      int odd = 0;           // kInfoOdd: one of them has infinities or NaN in V
      const int2 range = seen_range<kG>(a, t, x);
      for (int i = 0; i < t.count && range.y >= 0; ++i) {
        if (i >= t.head && (i < range.x || i > range.y)) continue;
        const int b = tile_block(t, i), n0 = b * kSparseBlock;
        const int info = __ldg(a.image_info + static_cast<int64_t>(t.slot0 + (b < t.req_head ? b : t.req_head + b - t.req_first)) *
                                                  a.num_kv_heads + t.g);
        odd |= info;
        const bool whole = info_pages(info) == 0xff && n0 + kSparseBlock - 1 <= pa &&
                           (a.window == 0 || n0 > pb - a.window || n0 + kSparseBlock <= a.num_sinks);
        if (!warp_wait_on(&ctl->s_full[x], ns & 1, ctl, a.err_word)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * c]));
        tc::wait_ld();
        bool any = live;  // does this row see a key of the block
        if (!whole) {
          const bool pages = info_pages(info) == 0xff;
          const bool low_free = a.window == 0 || n0 > pb - a.window || n0 + kSparseBlock <= a.num_sinks;
          if (pages && (low_free || (n0 >= a.num_sinks && n0 + kSparseBlock - 1 <= pa))) {
            // One border crosses the block: the row's own position (keys j <= edge stay) or the window's far end
            // (j >= edge). min with (edge + 1/2 - j) * inf = +-inf clears without a predicate per key.
            const int edge = low_free ? p - n0 : p - a.window + 1 - n0;
            const float sign = low_free ? 1.f : -1.f;
            // (a row without a token may keep what it likes: it is not written)
            const float at = sign * static_cast<float>(edge) + 0.5f;
            any = live && (low_free ? edge >= 0 : edge < kSparseBlock);
            const float2 inf = make_float2(INFINITY, INFINITY), step = make_float2(-8.f * sign, -8.f * sign);
            // keys that every row of the warp keeps: j <= keep (j >= keep for the far end)
            const int keep = low_free ? pw0 - n0 : pw1 - a.window + 1 - n0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (low_free ? keep >= 32 * c + 31 : keep <= 32 * c) continue;
              float2 b[4];  // (edge + 1/2 - j) * sign for j = 32c + 0, 1 | 2, 3 | 4, 5 | 6, 7, then 8 further
#pragma unroll
              for (int q = 0; q < 4; ++q) b[q] = make_float2(at - sign * (32 * c + 2 * q), at - sign * (32 * c + 2 * q + 1));
#pragma unroll
              for (int j = 32 * c; j < 32 * c + 32; j += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 w = mul2(b[q], inf);
                  v[j + 2 * q] = __float_as_uint(fminf(__uint_as_float(v[j + 2 * q]), w.x));
                  v[j + 2 * q + 1] = __float_as_uint(fminf(__uint_as_float(v[j + 2 * q + 1]), w.y));
                  b[q] = add2(b[q], step);
                }
            }
          } else {
            any = false;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = row_bits(a, n0 + 32 * c, p, live, info >> (8 + 2 * c));
              any |= w != 0u;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(w & (1u << j))) v[32 * c + j] = 0xff800000u;  // -inf
            }
          }
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = __uint_as_float(v[j]);
#pragma unroll
        for (int j = 4; j < 124; j += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(v[j + 2 * q]), __uint_as_float(v[j + 2 * q + 1])));
#pragma unroll
        for (int j = 124; j < 128; ++j) mx[j - 124] = fmaxf(mx[j - 124], __uint_as_float(v[j]));
        const float mxs = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;  // sl2 > 0
        // move the reference and the exponent, rescale O
        float f = 1.f;
        if (any && mxs > m + kLazyLog2) {
          f = ex2(m - mxs);  // 0 on the row's first keys
          l *= f;
          m = mxs;
        }
        const int e = info & 0xff;
        const bool some = any && e != 0;
        int de = some ? e - kInfoBias - E : 0;
        const bool moves = static_cast<uint32_t>(de - kExpDown) > static_cast<uint32_t>(kExpUp - kExpDown);  // not in [-8, 7]
        if (__any_sync(0xffffffffu, f != 1.f || moves)) {
          if (some) {
            const int lost = f > 0.f ? static_cast<int>(-log2f(f)) : 512;
            const int held = max(top, E + kInfoBias) - lost;  // largest V that O holds, by weight (within 2^7)
            if (E == kNoExp || f == 0.f) {  // nothing of the row
              E += de;
              de = 0;
              top = e;
            } else if (de > kExpUp || (de < kExpDown && de >= -120 && e >= held - 40)) {
              f *= exp2i(-de);  // (no lower than 40 below what O holds: it cannot overflow)
              E += de;
              de = 0;
              top = max(held, e);
            }
          }
          // (S(i) complete: so is the tile's PV(i - 1), issued before it)
          if (started && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {  // few registers: the scores stay in theirs
              uint32_t o[16];
              ld16(to + c, o);
              tc::wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc::st16(to + c, o);
            }
          }
        }
        de = max(de, -60);  // V that far below O adds nothing; the row sum still counts its keys
        // P * 2^de, and the row sum
        const float mu = (m == -INFINITY ? 0.f : m) - static_cast<float>(de);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        const float2 sc = make_float2(sl2, sl2), off = make_float2(-mu, -mu);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int i0 = 32 * c + 2 * j;
            float2 z = fma2(make_float2(__uint_as_float(v[i0]), __uint_as_float(v[i0 + 1])), sc, off);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            if (j & 1) sum1 = add2(sum1, z);
            else sum0 = add2(sum0, z);
            pk[j] = pack_f16(z.x, z.y);
          }
          tc::st16(ts + 16 * c, pk);
        }
        started = true;
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[x]);
        l += (sum0.x + sum0.y + sum1.x + sum1.y) * exp2i(-de);
        ++ns;
      }
      if (!ok) break;
      // ---- output; the next tile's description first (its S is on the way meanwhile)
      uint8_t* stage = out_s + (warp - 4) * 4096;
      const int rest = t.n_tok - x * T;  // the MMA tile's tokens
      const int64_t row0 = t.t0 + x * T;
      const int head0 = t.g * kG;
      odd = (odd & kInfoOdd) != 0;
      if (!odd && !next_tile(k + 1)) break;
      const bool blocks = __any_sync(0xffffffffu, started);
      if (blocks && !warp_wait_on(&ctl->pv_done[x], tiles++ & 1, ctl, a.err_word)) break;
      tc::fence_after_sync();
      // O * 2^E * v_scale / l. The factor stays in fp32's range for |E| <= 60; beyond, 2^E goes in two steps.
      const float inv = l != 0.f ? a.v_scale / l : 0.f;
      if (E == kNoExp) E = 0;
      const int e1 = max(-60, min(60, E));
      const float f1 = inv * exp2i(e1), f2 = exp2i(E - e1);
      const bool far = __any_sync(0xffffffffu, E != e1);
      const bool empty = __any_sync(0xffffffffu, l == 0.f);  // a row without a key: zeros
      // 64 dims at a time through shared memory (16-byte chunk c of row r at chunk c ^ (r % 8)), so that eight
      // lanes write one row's 128 bytes; a thread's own row alone would cost 32 lines per store
      const int i8 = lane >> 3;  // row 4q + i8 of the warp's 32 in store q
      uint16_t* dst = a.out + (row0 + (quad * 32) / kG + i8 / kG) * a.out_row_stride +
                      static_cast<int64_t>(head0 + (quad * 32) % kG + i8 % kG) * a.out_head_stride + 8 * (lane & 7);
      const int tok0 = (quad * 32) / kG + i8 / kG;
#pragma unroll 1
      for (int half = 0; half < 2 && blocks; ++half) {
        uint32_t o[64];
        tc::ld32(to + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
        tc::ld32(to + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
        tc::wait_ld();
        if (far)
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f2);
        if (empty && l == 0.f)
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j] = 0u;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = 8 * q + 2 * j;
            const float2 y = mul2(make_float2(__uint_as_float(o[d]), __uint_as_float(o[d + 1])), make_float2(f1, f1));
            w[j] = pack_bf16(y.x, y.y);
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int r = 4 * q + i8;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (tok0 + 4 * q / kG < rest)
            *reinterpret_cast<uint4*>(dst + (4 * q / kG) * a.out_row_stride + (4 * q % kG) * a.out_head_stride + 64 * half) = w;
        }
        __syncwarp();
      }
      if (!blocks && live) {  // no block: no row of the tile sees a key
        uint16_t* own = a.out + (row0 + tok) * a.out_row_stride + static_cast<int64_t>(head0 + h) * a.out_head_stride;
        for (int d = 0; d < kHeadDim; d += 8) *reinterpret_cast<uint4*>(own + d) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (live && a.lse != nullptr)
        a.lse[(row0 + tok) * a.lse_row_stride + head0 + h] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      if (odd) {
        __syncwarp();
        uint16_t* own = a.out + (row0 + tok) * a.out_row_stride + static_cast<int64_t>(head0 + h) * a.out_head_stride;
        if (live) add_odd_blocks(a, t, range, p, own);
        __syncwarp();
        if (!next_tile(k + 1)) break;
      }
      tc::fence_before_sync();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 2) {
    // ------------------------------------------------------------------ scheduler
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&q_map)) : "memory");
    int total = 0;  // request tiles
    for (int r0 = 0; r0 < a.num_reqs; r0 += 32) {
      int c0, p0;
      const int n = r0 + lane < a.num_reqs ? tokens_of(a, r0 + lane, &c0, &p0) : 0;
      total += __reduce_add_sync(0xffffffffu, static_cast<uint32_t>((n + 2 * T - 1) / (2 * T)));
    }
    const int flat = total * a.num_kv_heads;
    int nq[2] = {0, 0};
    for (int k = 0;; ++k) {
      // from the end: a request's last tiles see the most keys. A CTA takes its next tile when it has room for
      // its description (a fixed deal left 2-8 % of the CTAs' time unused)
      int f = static_cast<int>(blockIdx.x);
      bool go = true;
      if (lane == 0 && k >= 2) go = wait_on(&ctl->tile_empty[k & 1], ((k >> 1) - 1) & 1, ctl, a.err_word);
      if (lane == 0 && k > 0 && go) f = static_cast<int>(gridDim.x) + atomicAdd(a.next_tile, 1);
      f = __shfl_sync(0xffffffffu, f, 0);
      go = __shfl_sync(0xffffffffu, go && !aborted(ctl), 0);
      Tile* t = &ctl->tile[k & 1];
      const bool last = !go || f >= flat;
      if (!last) {
        int at = 0;
        const int r = find_request(a, total - 1 - f / a.num_kv_heads, lane, &at, [&](int i) {
          int c0, p0;
          return (tokens_of(a, i, &c0, &p0) + 2 * T - 1) / (2 * T);
        });
        int slot0 = 0;
        for (int r0 = 0; r0 < r; r0 += 32)
          slot0 += __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(r0 + lane < r ? blocks_of(a, r0 + lane) : 0));
        if (lane == 0) {
          int c0, p0;
          const int n = tokens_of(a, r, &c0, &p0);
          const Span whole = span_of(a, p0, p0 + n - 1);
          t->req = r;
          t->g = f % a.num_kv_heads;
          t->t0 = c0 + at * 2 * T;
          t->n_tok = min(2 * T, n - at * 2 * T);
          t->p0 = p0 + at * 2 * T;
          const Span s = span_of(a, t->p0, t->p0 + t->n_tok - 1);
          const bool held = slot0 >= 0 && slot0 + whole.count <= a.image_slots;  // always, if cu_seqlens_q does not decrease
          if (!held) set_err(a.err_word, PBS_DEVERR_TABLE);
          t->head = s.head;
          t->first = s.first;
          t->count = held ? s.count : 0;
          t->slot0 = slot0;
          t->req_head = whole.head;
          t->req_first = whole.first;
        }
      }
      if (lane == 0) {
        t->end = last;
        mbar_arrive(&ctl->tile_full[k & 1]);
        // the tile's Q: A's when the last S of A of the tile before has read its own, then B's
        for (int x = 0; !last && x < 2; ++x) {
          if (k > 0 && !wait_on(&ctl->q_empty[x], (k - 1) & 1, ctl, a.err_word)) break;
          if (x == 1 && t->n_tok <= T) {  // no B
            mbar_arrive(&ctl->q_full[1]);
            break;
          }
          mbar_arrive_expect_tx(&ctl->q_full[x], kQTile);
          tma_load_3d(q_s + x * kQTile, &q_map, &ctl->q_full[x], 0, t->g * kG, t->t0 + x * T);
          tma_load_3d(q_s + x * kQTile + kHalf, &q_map, &ctl->q_full[x], 64, t->g * kG, t->t0 + x * T);
          ++nq[x];
        }
      }
      __syncwarp();
      if (last) {
        // every copy must land before the CTA exits
        if (lane == 0 && k > 0) {
          for (int x = 0; x < 2; ++x)
            if (nq[x] > 0 && !mbar_wait_quick(&ctl->q_full[x], (k - 1) & 1, kWaitNs)) set_err(a.err_word, PBS_DEVERR_TIMEOUT);
        }
        break;
      }
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      int n = 0;  // images issued
      bool go = true;
      for (int k = 0; go; ++k) {
        if (!wait_on(&ctl->tile_full[k & 1], (k >> 1) & 1, ctl, a.err_word)) break;
        const Tile t = ctl->tile[k & 1];
        mbar_arrive(&ctl->tile_empty[k & 1]);
        if (t.end) break;
        for (int i = 0; go && i < t.count; ++i) {
          const int b = tile_block(t, i);
          const int64_t image =
              static_cast<int64_t>(t.slot0 + (b < t.req_head ? b : t.req_head + b - t.req_first)) * a.num_kv_heads + t.g;
          for (int side = 0; side < 2; ++side, ++n) {
            const int st = n % kRing;
            if (n >= kRing && !wait_on(&ctl->empty[st], ((n / kRing) - 1) & 1, ctl, a.err_word)) go = false;
            if (!go || aborted(ctl)) {
              go = false;
              break;
            }
            mbar_arrive_expect_tx(&ctl->full[st], kImage);
            bulk_load(ring + st * kImage, (side ? a.v_images : a.k_images) + image * kImage, kImage, &ctl->full[st]);
          }
        }
      }
      // every copy must land before the CTA exits
      for (int i = max(0, n - kRing); i < n; ++i)
        if (!mbar_wait_quick(&ctl->full[i % kRing], (i / kRing) & 1, kWaitNs)) set_err(a.err_word, PBS_DEVERR_TIMEOUT);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ gate
    // Waits for a step's V(i - 1) and K(i) and adds the last arrival to A's P barrier, so that the MMA thread,
    // whose every barrier read is on the critical path, reads one barrier for the three.
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0, n = 0;
      bool ok = true, pend = false;
      auto pass = [&]() {  // the next ring entry is loaded (and not loaded again behind the gate's back)
        if (!wait_on(&ctl->full[st], ph, ctl, a.err_word)) return false;
        mbar_arrive(&ctl->empty[st]);
        if (++st == kRing) {
          st = 0;
          ph ^= 1;
        }
        return true;
      };
      auto open = [&]() {  // A's pending PV may go; one arrival a phase
        if (!pend) return true;
        mbar_arrive(&ctl->p_full[0]);
        return wait_on(&ctl->p_full[0], n++ & 1, ctl, a.err_word);
      };
      bool first_step = true;
      for (int k = 0; ok; ++k) {
        if (!wait_on(&ctl->tile_full[k & 1], (k >> 1) & 1, ctl, a.err_word)) break;
        const Tile* t = &ctl->tile[k & 1];
        const bool end = t->end != 0;
        const int count = t->count, head = t->head;
        int2 r = {0, -1};
        if (!end) r = seen_range<kG>(a, *t, 0);
        mbar_arrive(&ctl->tile_empty[k & 1]);
        for (int i = 0; ok && i < (end ? 1 : count); ++i) {
          ok = (first_step || pass()) && (end || pass()) && open();  // V(n - 1), K(n)
          first_step = false;
          pend = r.y >= 0 && (i < head || (i >= r.x && i <= r.y));
        }
        if (end) break;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    // Step n of the CTA's block sequence, over its tiles: PV_A(n - 1) S_A(n) PV_B(n - 1) S_B(n).
    if (elect_one()) {
      constexpr uint32_t kIdescS = tc::idesc_f16(128, 128, true, false, false);
      constexpr uint32_t kIdescPV = tc::idesc_f16(128, 128, false, false, true);
      const uint64_t q_desc = tc::smem_desc_sw128(smem_u32(q_s), 16, 1024);
      const uint64_t k_desc = tc::smem_desc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t v_desc = tc::smem_desc_sw128(smem_u32(ring), kHalf, 1024);
      int st = 0;             // ring stage and phase of the next entry: K(0), V(0), K(1), V(1), ..
      uint32_t ph = 0;
      uint32_t done[2] = {0, 0};  // PVs of A and of B
      bool pend[2] = {false, false}, fresh[2] = {true, true}, final[2] = {false, false};
      int k = -1, i = -1, count = 0, head = 0;  // tile, block of its list, blocks
      int2 r[2] = {};
      bool ok = true, end = false, first_step = true;
      while (ok && !end) {
        const bool next_tile = i + 1 >= count;
        i = next_tile ? 0 : i + 1;
        int vst = 0;
        bool k_ready = false;
        if (!first_step) {  // V(n - 1); with a PV of A pending, its P barrier stands for it and for K(n) (the gate)
          vst = st;
          k_ready = pend[0];
          if (!pend[0] && !wait_on(&ctl->full[st], ph, ctl, a.err_word)) break;
          if (++st == kRing) {
            st = 0;
            ph ^= 1;
          }
        }
        const uint64_t vd = v_desc + static_cast<uint32_t>(vst * kImage >> 4);
        const uint64_t kd = k_desc + static_cast<uint32_t>(st * kImage >> 4);
        auto pv = [&](const int x) {  // O += P V
          if (!pend[x]) return true;
          if (!wait_on(&ctl->p_full[x], done[x] & 1, ctl, a.err_word)) return false;
          tc::fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_ts(tmem + 256 + x * 128, tmem + x * 128 + ks * 8, vd + (ks * 2048 >> 4), kIdescPV, !(fresh[x] && ks == 0));
          if (final[x]) tc::commit(&ctl->pv_done[x]);
          ++done[x];
          fresh[x] = false;
          pend[x] = false;
          return true;
        };
        auto qk = [&](const int x) {  // S = Q K^T
          pend[x] = r[x].y >= 0 && (i < head || (i >= r[x].x && i <= r[x].y));
          final[x] = i == last_seen(r[x], head);
          if (pend[x]) {
            tc::fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t at = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
              tc::mma_ss(tmem + x * 128, q_desc + (x * kQTile >> 4) + at, kd + at, kIdescS, ks > 0);
            }
            tc::commit(&ctl->s_full[x]);
          }
          if (i == count - 1) tc::commit(&ctl->q_empty[x]);  // the tile's last S (or none)
        };
        if (!next_tile) {
          ok = pv(0) && (k_ready || wait_on(&ctl->full[st], ph, ctl, a.err_word));
          if (!ok) break;
          qk(0);
          ok = pv(1);
          if (!ok) break;
          qk(1);
        } else {
          // S_A of the next tile goes before PV_B, unless its description is late or it has no blocks (the wait for the
          // tile after it could depend on PV_B)
          const auto enter = [&](const Tile* t) {
            count = t->count;
            head = t->head;
            r[0] = seen_range<kG>(a, *t, 0);
            r[1] = seen_range<kG>(a, *t, 1);
            mbar_arrive(&ctl->tile_empty[k & 1]);
          };
          ok = pv(0);
          if (!ok) break;
          const Tile* next = &ctl->tile[(k + 1) & 1];
          if (mbar_try_wait(&ctl->tile_full[(k + 1) & 1], ((k + 1) >> 1) & 1) && !next->end && next->count > 0 &&
              wait_on(&ctl->q_full[0], (k + 1) & 1, ctl, a.err_word)) {
            ++k;
            enter(next);
            fresh[0] = true;
            ok = k_ready || wait_on(&ctl->full[st], ph, ctl, a.err_word);
            if (!ok) break;
            qk(0);
            ok = pv(1);
            fresh[1] = true;
            ok = ok && wait_on(&ctl->q_full[1], k & 1, ctl, a.err_word);
            if (!ok) break;
            qk(1);
          } else {
            ok = pv(1);
            while (ok) {  // the next tile, skipping those without blocks
              ++k;
              ok = wait_on(&ctl->tile_full[k & 1], (k >> 1) & 1, ctl, a.err_word);
              if (!ok) break;
              const Tile* t = &ctl->tile[k & 1];
              end = t->end != 0;
              if (end) break;
              enter(t);
              ok = wait_on(&ctl->q_full[0], k & 1, ctl, a.err_word);
              if (!ok || count > 0) break;
              ok = wait_on(&ctl->q_full[1], k & 1, ctl, a.err_word);
              mbar_arrive(&ctl->q_empty[0]);
              mbar_arrive(&ctl->q_empty[1]);
            }
            if (!ok) break;
            if (!end) {
              fresh[0] = fresh[1] = true;
              ok = k_ready || wait_on(&ctl->full[st], ph, ctl, a.err_word);
              if (!ok) break;
              qk(0);
              ok = wait_on(&ctl->q_full[1], k & 1, ctl, a.err_word);
              if (!ok) break;
              qk(1);
            }
          }
        }
        if (!ok) break;
        if (!first_step) tc::commit(&ctl->empty[vst]);
        if (!end) {
          tc::commit(&ctl->empty[st]);
          if (++st == kRing) {
            st = 0;
            ph ^= 1;
          }
        }
        first_step = false;
      }
      // every MMA must complete before TMEM is released
      tc::commit(&ctl->drained);
      mbar_wait_quick(&ctl->drained, 0, kWaitNs);
    }
  }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 2) tc::dealloc(tmem, 512);
}

template <int kG>
cudaError_t launch_g(const WindowArgs& a, const CUtensorMap& q_map, int sms, cudaStream_t stream) {
  auto kern = prefill_kernel<kG>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemTc));
  if (e != cudaSuccess) return e;
  const int64_t tiles = (static_cast<int64_t>(a.num_rows) / (2 * kRows / kG) + a.num_reqs) * a.num_kv_heads;
  kern<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kThreadsTc, kSmemTc, stream>>>(q_map, a);
  return cudaGetLastError();
}

}  // namespace

int64_t window_image_slots(int64_t total_q, int64_t num_reqs, int64_t max_blocks, int64_t window, int64_t num_sinks) {
  // a request's span: its tokens' and the window's blocks with a border block at each end, and the sinks'
  const int64_t per_token = total_q / kSparseBlock;
  const int64_t rest = (window + kSparseBlock - 1) / kSparseBlock + 2 + (num_sinks + kSparseBlock - 1) / kSparseBlock;
  const int64_t by_window = per_token + num_reqs * rest, by_table = num_reqs * max_blocks;
  return window > 0 && by_window < by_table ? by_window : by_table;
}

size_t window_prefill_workspace(int64_t slots, int64_t num_kv_heads) {
  const int64_t images = slots * num_kv_heads;
  return static_cast<size_t>(images) * 2 * kImage + static_cast<size_t>((images * 4 + 4 + 255) / 256 * 256);
}

void window_attach_images(WindowArgs* a, void* workspace, int64_t slots) {
  const int64_t images = slots * a->num_kv_heads;
  a->image_slots = static_cast<int32_t>(slots);
  a->k_images = static_cast<uint8_t*>(workspace);
  a->v_images = a->k_images + images * kImage;
  a->image_info = reinterpret_cast<int32_t*>(a->v_images + images * kImage);
  a->next_tile = a->image_info + images;
}

cudaError_t launch_window_prefill_tc(const WindowArgs& a, const CUtensorMap& q_map, int sms, cudaStream_t stream) {
  const int most = kMaxConvertCtas / a.num_kv_heads;
  const dim3 grid(static_cast<unsigned>(max(1, min(a.image_slots, most))), static_cast<unsigned>(a.num_kv_heads));
  switch (a.kv_dtype) {
    case PBS_KV_BF16: convert_kernel<PBS_KV_BF16><<<grid, 512, 0, stream>>>(a); break;
    case PBS_KV_FP8_E4M3: convert_kernel<PBS_KV_FP8_E4M3><<<grid, 512, 0, stream>>>(a); break;
    case PBS_KV_NVFP4: convert_kernel<PBS_KV_NVFP4><<<grid, 512, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  switch (a.group) {
    case 1: return launch_g<1>(a, q_map, sms, stream);
    case 2: return launch_g<2>(a, q_map, sms, stream);
    case 4: return launch_g<4>(a, q_map, sms, stream);
    case 8: return launch_g<8>(a, q_map, sms, stream);
    case 16: return launch_g<16>(a, q_map, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pbs
