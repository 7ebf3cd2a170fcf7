// Window attend with sinks over the paged cache, mma.sync kernel: decode rows, and prefill tokens
// where the tcgen05 kernel does not run. For a query at position p of its request,
//   out = v_scale * softmax(softmax_scale * k_scale * q K^T) V  over the keys
//   0 <= n <= p with n > p - window (any n when window is 0) or n < num_sinks.
//
// Units. A group is up to 8 NT / G consecutive rows of one request (G query heads per kv head): its
// rows x heads are the 8 NT columns of the MMAs, so the rows of a request share every K / V read. An
// item is a group. Keys are taken in pairs of pages (32 keys, aligned, so a pair never leaves its block):
// an item's list is the pairs that hold sinks and then those of the window up to the last row's own. A unit
// is (item, kv head).
//
// Work split. Bound by HBM (bf16, fp8) or by the dequantisation's issue slots (NVFP4), and lengths are
// ragged, so with a workspace the pairs of all units form one sequence that is cut into equal parts, one
// per resident CTA: every CTA streams the same number of pairs, whatever the batch. A CTA's part may end
// one unit, hold whole ones and begin another; a unit cut between CTAs leaves one partial (max, sum, O)
// per CTA in the workspace, and the CTA that draws the unit's last ticket merges them in pair order
// (the same bits whoever is last) and clears the ticket. Without a workspace a CTA takes one unit.
//
// CTA. One producer warp: page-table entries of 32 pairs at a time, then one tensor copy per pair into a ring
// of stages; it runs ahead across unit borders. (Issuing is its cost: with two copies and four warp exchanges
// a pair, some 700 clocks, it held NVFP4 back.) The consumer warps take pairs in turn (a stage always belongs
// to one warp), each with its own online softmax (base 2, lazy reference: O is rescaled when the maximum
// passes it by 2^8); their partials meet in shared memory at the end of a unit. S^T = K Q^T and
// O^T += V^T P^T with keys as MMA rows (window_page.cuh).
//
// Measured (64 / 8 heads, events, L2 flushed): bf16, 64 requests, window 4096 + 128 sinks 172 us = 6.45 TB/s,
// 95 % of the measured copy rate; fp8, 128 requests of two rows, window 8191 339 us = 6.40 TB/s, 94 %; NVFP4,
// 32 requests of 8k-64k keys, no window 271 us = 5.0 TB/s, 74 %, bound by 310 warp instructions per page.
#include "mbar_wait.cuh"
#include "pbs_device.cuh"
#include "pbs_internal.h"
#include "window_page.cuh"

namespace pbs {
namespace {

constexpr int kPair = 2;               // pages per stage and consumer iteration
constexpr float kLazyLog2 = 8.0f;
constexpr int kOPitch = kHeadDim + 4;  // floats: rows 4 banks apart (conflict-free partial writes)
// CTAs per SM, consumer warps and stages per CTA. bf16 and fp8 are bound by HBM: 2 x 4 (fp8, with converts to do:
// 2 x 5) warps keep up, 128 to 160 KiB per SM in flight. NVFP4 is bound by the pipe that converts (and compares,
// selects and packs) at 16 lanes a clock and by the chains of its warps: 32 requests of 8k-64k keys took 294 us
// with 3 CTAs of 4 consumers, 323 with 3 of 3, 281 with 4 of 3, 357 with 2 of 7. Two fp8 rows of 128 requests:
// 344 us with 2 of 5, 356 with 2 of 4, 464 with 3 of 4 and half the stages.
template <int FMT, int NT>
struct Cfg {
  static constexpr int kWarps = FMT == PBS_KV_FP8_E4M3 ? 5 : FMT == PBS_KV_NVFP4 && NT == 1 ? 3 : 4;
  static constexpr int kStages = FMT == PBS_KV_BF16 ? 4 : 2 * kWarps;
  static constexpr int kCtas = FMT == PBS_KV_NVFP4 && NT == 1 ? 4 : 2;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static_assert(kStages % kWarps == 0, "each stage must belong to one consumer warp");
};

// The warps' partials of one column tile.
template <int W>
struct Merge {
  float o[W][8][kOPitch];
  float m[W][8];
  float l[W][8];
};

// One group of rows and its list of pairs.
struct Item {
  int req, row0, rows;  // first of its rows in q, how many
  int p0, p1;           // their positions
  int head;             // pairs [0, head), then
  int first;            // pairs first ..
  int real;             // pairs of the list
  int pairs;            // as scheduled: one at least
};

// What a unit costs beside its pairs (Q, the pairs its borders cross, the merge), in pairs: the sequence that is
// dealt out holds so many empty places behind each unit's pairs. 44 requests of up to 1.6k keys (three rows, 16
// heads per kv head): 201 us without them, as the short requests' CTAs end last.
constexpr int kUnitCost = 12;

template <int NS>
struct Ctl {
  uint64_t full[NS];
  uint64_t empty[NS];
  int32_t ok[NS];  // bit i: the stage holds page i of its pair (else padding, or not in the cache)
  int32_t abort;
  int32_t last;
  int32_t item;    // where this CTA's part begins
  Item it;
  int64_t offset;
  int32_t ids[32]; // first physical page of the producer's next pairs
  uint2 q[16][32]; // two column tiles: the unit's Q fragments, [tile * 8 + k-step][lane]
};

template <int FMT, int NT>
constexpr size_t kSmem = 1024 + size_t(Cfg<FMT, NT>::kStages) * kPair * wp::kPageBytes<FMT> +
                         sizeof(Merge<Cfg<FMT, NT>::kWarps>) + sizeof(Ctl<Cfg<FMT, NT>::kStages>);

constexpr int kPairKeys = kPair * kPageRows;
constexpr int kPairsPerBlock = kSparseBlock / kPairKeys;

__device__ __forceinline__ void pair_list(const WindowArgs& a, Item& it) {
  it.head = it.first = it.real = 0;
  if (it.p1 >= 0) {
    const int low = a.window > 0 ? max(0, max(it.p0, 0) - a.window + 1) : 0;
    const int head = min(a.num_sinks, low);
    it.first = low / kPairKeys;
    it.head = min((head + kPairKeys - 1) / kPairKeys, it.first);
    it.real = it.head + it.p1 / kPairKeys - it.first + 1;
  }
  it.pairs = max(1, it.real);
}

__device__ __forceinline__ Item decode_item(const WindowArgs& a, int item) {
  Item it;
  it.req = a.groups_per_req == 1 ? item : item / a.groups_per_req;
  const int r0 = (item - it.req * a.groups_per_req) * a.rows_per_group;
  it.rows = min(a.rows_per_group, a.decode_query_len - r0);
  it.row0 = it.req * a.decode_query_len + r0;
  it.p0 = __ldg(a.seq_lens + it.req) - a.decode_query_len + r0;
  it.p1 = it.p0 + it.rows - 1;
  pair_list(a, it);
  return it;
}

// Group `item` of the prefill tokens, counting each request's groups of rows_per_group in order; rows
// 0: there is no such group. One warp.
__device__ __forceinline__ Item prefill_item(const WindowArgs& a, int item, int lane) {
  Item it = {};
  int before = 0;
  for (int r0 = 0; r0 < a.num_reqs; r0 += 32) {
    const int r = r0 + lane;
    const int c0 = r < a.num_reqs ? __ldg(a.cu_seqlens_q + r) : 0;
    const int n = r < a.num_reqs ? __ldg(a.cu_seqlens_q + r + 1) - c0 : 0;
    const int groups = n > 0 && c0 >= 0 ? (n + a.rows_per_group - 1) / a.rows_per_group : 0;
    int incl = groups;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    const int at = item - before - (incl - groups);
    const uint32_t hit = __ballot_sync(0xffffffffu, at >= 0 && at < groups);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      const int n_of = __shfl_sync(0xffffffffu, n, src), c_of = __shfl_sync(0xffffffffu, c0, src);
      const int first = __shfl_sync(0xffffffffu, at, src) * a.rows_per_group;
      it.req = r0 + src;
      it.rows = min(a.rows_per_group, min(n_of - first, a.num_rows - c_of - first));
      it.row0 = c_of + first;
      it.p0 = __ldg(a.seq_lens + it.req) - n_of + first;
      it.p1 = it.p0 + it.rows - 1;
      if (it.rows > 0) pair_list(a, it);
      return it;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return it;
}

// Keys n0 .. n0 + 15 that rows at positions p_low .. p_high see between them, bit n - n0.
__device__ __forceinline__ uint32_t seen_bits(const WindowArgs& a, int n0, int p_high, int p_low) {
  const int behind = p_high - n0;  // causal: bits 0 .. behind
  if (behind < 0) return 0u;
  uint32_t m = behind >= 15 ? 0xffffu : (2u << behind) - 1u;
  if (a.window > 0) {
    const int lo = max(p_low, 0) - a.window + 1 - n0;
    const uint32_t in = lo <= 0 ? 0xffffu : lo > 15 ? 0u : (0xffffu << lo) & 0xffffu;
    const int s = a.num_sinks - n0;
    const uint32_t sink = s <= 0 ? 0u : s >= 16 ? 0xffffu : (1u << s) - 1u;
    m &= in | sink;
  }
  return m;
}

// One pair: both pages' K and V of kv head g.
template <int FMT>
__device__ __forceinline__ void load_pair(void* dst, const void* tmap, uint64_t* bar, int g, int page) {
  if (FMT == PBS_KV_NVFP4)
    tma_load_4d(dst, tmap, bar, 0, 0, g, page);
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(0), "r"(g), "r"(page)
        : "memory");
}

template <int W>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
}

__device__ __forceinline__ void add4(float4& o, float f, const float4& x) {
  o.x += f * x.x;
  o.y += f * x.y;
  o.z += f * x.z;
  o.w += f * x.w;
}

// The sequence of `total` pairs in `parts` parts: the first `more` have `each` + 1 pairs, the others `each`.
struct Cut {
  int64_t each;
  int more;
  __device__ __forceinline__ Cut(int64_t total, int parts) {
    if (total < (int64_t(1) << 31)) {  // 32-bit divisions are the cheap ones
      each = static_cast<uint32_t>(total) / static_cast<uint32_t>(parts);
      more = static_cast<int>(static_cast<uint32_t>(total) % static_cast<uint32_t>(parts));
    } else {
      each = total / parts;
      more = static_cast<int>(total % parts);
    }
  }
  __device__ __forceinline__ int64_t first(int c) const { return each * c + min(c, more); }
  // the part that holds pair x
  __device__ __forceinline__ int of(int64_t x) const {
    const int64_t wide = (each + 1) * more, y = x < wide ? x : x - wide, d = x < wide ? each + 1 : each;
    const int q = y < (int64_t(1) << 31) ? static_cast<int>(static_cast<uint32_t>(y) / static_cast<uint32_t>(d))
                                          : static_cast<int>(y / d);
    return x < wide ? q : more + q;
  }
};

// Output dims 4 lane .. and log-sum-exp of one row and head, from the merged maximum, sum and O.
__device__ __forceinline__ void store_out(const WindowArgs& a, int row, int head, int lane, float M, float L,
                                          const float4& O) {
  const float r = L != 0.f ? a.v_scale / L : 0.f;  // L is 0 only without keys (O too); NaN goes through
  uint16_t* out = a.out + static_cast<int64_t>(row) * a.out_row_stride + static_cast<int64_t>(head) * a.out_head_stride + 4 * lane;
  const uint32_t lo = pack_bf16(O.x * r, O.y * r), hi = pack_bf16(O.z * r, O.w * r);
  if (a.out_vec) {
    *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
  } else {
    out[0] = static_cast<uint16_t>(lo);
    out[1] = static_cast<uint16_t>(lo >> 16);
    out[2] = static_cast<uint16_t>(hi);
    out[3] = static_cast<uint16_t>(hi >> 16);
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[static_cast<int64_t>(row) * a.lse_row_stride + head] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int FMT, int NT>
__global__ void __launch_bounds__(Cfg<FMT, NT>::kThreads, Cfg<FMT, NT>::kCtas)
    window_attend_kernel(const __grid_constant__ CUtensorMap tmap, const WindowArgs a) {
  constexpr int kWarps = Cfg<FMT, NT>::kWarps, kThreads = Cfg<FMT, NT>::kThreads, NS = Cfg<FMT, NT>::kStages;
  constexpr int kPage = wp::kPageBytes<FMT>, kStage = kPair * kPage;
  constexpr int kCols = 8 * NT;
  constexpr int kSlot = kCols * (kHeadDim + 2);  // floats of a workspace partial: O, then m, then l
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Merge<kWarps>* mg = reinterpret_cast<Merge<kWarps>*>(stages + NS * kStage);
  Ctl<NS>* ctl = reinterpret_cast<Ctl<NS>*>(mg + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool split = a.split_ws != nullptr;
  const int H = a.num_kv_heads;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }

  // ---- this CTA's part of the sequence: `left` places from place `off` of unit (item, g)
  int item, g;
  int off = 0;
  int64_t left, start = 0;
  Cut cut(1, 1);
  Item it;
  if (split) {
    const int n_items = a.num_reqs * a.groups_per_req;
    const int per = (n_items + kThreads - 1) / kThreads;
    const int i0 = min(static_cast<int>(threadIdx.x) * per, n_items), i1 = min(i0 + per, n_items);
    int64_t mine = 0, total = 0;  // an item has up to 2^26 pairs: sums in 64 bits
    for (int i = i0; i < i1; ++i) mine += (decode_item(a, i).pairs + kUnitCost);
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    __shared__ int64_t sums[kWarps + 1];
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    for (int w = 0; w < kWarps + 1; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    total *= H;
    const int parts = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(int64_t(1), total >> a.min_pairs_log2)));
    if (static_cast<int>(blockIdx.x) >= parts) return;
    cut = Cut(total, parts);
    start = cut.first(blockIdx.x);
    left = cut.first(blockIdx.x + 1) - start;
    if (start >= before * H && start < (before + mine) * H) {
      int64_t at = before * H;
      for (int i = i0; i < i1; ++i) {
        const Item x = decode_item(a, i);
        const int64_t w = static_cast<int64_t>(x.pairs + kUnitCost) * H;
        if (start < at + w) {
          ctl->item = i;
          ctl->it = x;
          ctl->offset = start - at;
          break;
        }
        at += w;
      }
    }
    __syncthreads();
    item = ctl->item;
    it = ctl->it;
    // the offset lies inside the item: kv heads (at most 65535) x places (2^26)
    const int64_t offset = ctl->offset;
    const int places = it.pairs + kUnitCost;
    if (offset < (int64_t(1) << 31)) {
      g = static_cast<int>(static_cast<uint32_t>(offset) / static_cast<uint32_t>(places));
    } else {
      g = static_cast<int>(offset / places);
    }
    off = static_cast<int>(offset - static_cast<int64_t>(g) * places);
  } else {
    __syncthreads();
    item = blockIdx.x;
    g = blockIdx.y;
    it = a.cu_seqlens_q != nullptr ? prefill_item(a, item, lane) : decode_item(a, item);
    if (it.rows <= 0) return;
    left = it.pairs;
  }

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    int st = 0, issued = 0;  // the next pair's stage; pairs issued
    uint32_t ph = 1;         // phase of its empty barrier (the first round finds the stages empty)
    bool go = true;
    while (go && left > 0) {
      const int end = static_cast<int>(min(static_cast<int64_t>(it.pairs), off + left));
      const int32_t* pt_row = a.page_table + static_cast<int64_t>(it.req) * a.pt_row_stride;
      auto page_of = [&](int i) -> int {  // first physical page of entry i of the unit's list, -1: none
        if (i >= min(end, it.real)) return -1;
        const int pn = i < it.head ? i : it.first + (i - it.head);
        const int b = pn / kPairsPerBlock;
        if (b >= a.max_blocks) {
          set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
          return -1;
        }
        const int phys = __ldg(pt_row + b);
        const int64_t page = static_cast<int64_t>(phys) * a.block_page_stride + pn % kPairsPerBlock * kPair;
        // (the second page may lie behind the last key: then it is not missed)
        if (phys < 0 || page >= a.num_pages || (page + 1 >= a.num_pages && pn * kPairKeys + kPageRows <= it.p1))
          set_err(a.err_word, PBS_DEVERR_PAGE_OOB);
        return phys < 0 || page >= a.num_pages ? -1 : static_cast<int>(page);
      };
      int next = page_of(off + lane);
      for (int base = off; go && base < end; base += 32) {
        __syncwarp();
        ctl->ids[lane] = next;
        __syncwarp();
        if (base + 32 < end) next = page_of(base + 32 + lane);
        if (lane == 0) {
          const int n = min(32, end - base);
          for (int j = 0; j < n; ++j) {
            if (!mbar_wait_quick(&ctl->empty[st], ph, kWaitLimitNs)) {
              set_err(a.err_word, PBS_DEVERR_TIMEOUT);
              atomicExch(&ctl->abort, 1);
            }
            if (*reinterpret_cast<volatile int32_t*>(&ctl->abort) != 0) {
              go = false;
              break;
            }
            const int page = ctl->ids[j];
            ctl->ok[st] = page < 0 ? 0 : page + 1 < a.num_pages ? 3 : 1;
            if (page < 0) {
              mbar_arrive(&ctl->full[st]);
            } else {
              mbar_arrive_expect_tx(&ctl->full[st], kStage);
              load_pair<FMT>(stages + st * kStage, &tmap, &ctl->full[st], g, page);
            }
            ++issued;
            if (++st == NS) {
              st = 0;
              ph ^= 1;
            }
          }
        }
        go = __shfl_sync(0xffffffffu, go, 0);
      }
      left -= min(static_cast<int64_t>(it.pairs + kUnitCost - off), left);
      off = 0;
      if (left > 0 && ++g == H) {
        g = 0;
        it = decode_item(a, ++item);
      }
    }
    // every copy issued must land before the shared memory goes away
    if (lane == 0)
      for (int p = max(0, issued - NS); p < issued; ++p)
        if (!mbar_wait_quick(&ctl->full[p % NS], (p / NS) & 1, kWaitLimitNs)) {
          set_err(a.err_word, PBS_DEVERR_TIMEOUT);
          break;
        }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int hh = lane >> 2, c = lane & 3;
  const int G = a.group, gshift = __ffs(G) - 1;  // a power of two
  const float sl2 = a.scale_log2;
  int64_t s = 0;            // places of the CTA's part before this unit
  int mine = warp;          // this warp's next pair, counted from the unit's first
  int st = warp;            // its stage and phase
  uint32_t ph = 0;
  for (;;) {
    const int first = off, end = static_cast<int>(min(static_cast<int64_t>(it.pairs), off + left));
    const int n = end - first;
    const int64_t u0 = start + s - first;  // the unit's first place in the sequence
    if (n > 0) {  // (else the part begins behind the unit's pairs)
    // Q fragments and each column's row. One tile's stay in registers; two tiles' (32 registers) go to shared
    // memory, in fragment order.
    uint2 qf[NT == 1 ? 8 : 1];
    int row_of[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int col = 8 * t + hh;  // the B fragment's column
      const int r = col >> gshift;
      const bool live = r < it.rows;
      const uint32_t* q32 = reinterpret_cast<const uint32_t*>(
          a.q + static_cast<int64_t>(it.row0 + (live ? r : 0)) * a.q_row_stride +
          static_cast<int64_t>(g * G + (live ? col & (G - 1) : 0)) * a.q_head_stride);
      const auto word = [&](int j, int w) {
        const uint32_t x = live ? __ldg(q32 + (wp::q_dim<FMT>(j, w, c) >> 1)) : 0u;
        return FMT == PBS_KV_BF16 ? x : bf16x2_to_f16x2(x);
      };
      if (NT == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) qf[NT == 1 ? j : 0] = make_uint2(word(j, 0), word(j, 1));
      } else {
        for (int j = warp; j < 8; j += kWarps) ctl->q[8 * t + j][lane] = make_uint2(word(j, 0), word(j, 1));
      }
      row_of[t][0] = (8 * t + 2 * c) >> gshift;
      row_of[t][1] = (8 * t + 2 * c + 1) >> gshift;
    }
    if (NT > 1) consumers_sync<kWarps>();  // (the last unit's readers passed its merge)
    const auto q_frag = [&](int t, int j) { return NT == 1 ? qf[NT == 1 ? j : 0] : ctl->q[8 * t + j][lane]; };
    float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }

    // Entries of the list whose 32 keys every row of the group sees: [plain0, plain1) in the window (behind
    // the first row's position or before the last row's window they are not) and [0, plain_s) of the sinks.
    const int jump = it.first - it.head;
    int plain0 = 0, plain1 = 0, plain_s = 0;
    if (it.p0 >= 0) {
      const int whole1 = (it.p0 + 1) / kPairKeys;  // pairs before it end at p0 or earlier
      plain1 = whole1 - jump;
      plain0 = (a.window > 0 && it.p1 >= a.window ? (it.p1 - a.window) / kPairKeys + 1 : 0) - jump;
      plain_s = min(min(it.head, whole1), a.num_sinks / kPairKeys);
    }
    // this warp's pairs of the unit: the CTA's pairs are dealt in turn, over all its units
    for (; mine < n; mine += kWarps) {
      const int e = first + mine;
      bool ok = mbar_try_wait(&ctl->full[st], ph);
      if (!ok && *reinterpret_cast<volatile int32_t*>(&ctl->abort) == 0)
        ok = mbar_wait_quick(&ctl->full[st], ph, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, ok)) {  // a wait that gave up leaves the pair out
        set_err(a.err_word, PBS_DEVERR_TIMEOUT);
        atomicExch(&ctl->abort, 1);
      }
      const uint32_t real = ok ? ctl->ok[st] : 0u;
      const uint32_t whole = (e >= plain0 && e < plain1) || e < plain_s ? real : 0u;
      const uint32_t stp[kPair] = {smem_u32(stages) + st * kStage, smem_u32(stages) + st * kStage + kPage};

      float sc[kPair][NT][4];
      wp::page_scores<FMT, kPair, NT>(stp, q_frag, lane, sc);
      float mx[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) mx[t][0] = mx[t][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPair; ++i) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[i][t][x] *= sl2;
        if (!((whole >> i) & 1u)) {
          const int n0 = ((e < it.head ? e : e + jump) * kPair + i) * kPageRows;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int p = it.p0 + row_of[t][w];
              const uint32_t b = ((real >> i) & 1u) && row_of[t][w] < it.rows ? seen_bits(a, n0, p, p) : 0u;
              if (!((b >> hh) & 1u)) sc[i][t][w] = -INFINITY;
              if (!((b >> (hh + 8)) & 1u)) sc[i][t][w + 2] = -INFINITY;
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mx[t][0] = fmaxf(mx[t][0], fmaxf(sc[i][t][0], sc[i][t][2]));
          mx[t][1] = fmaxf(mx[t][1], fmaxf(sc[i][t][1], sc[i][t][3]));
        }
      }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mx[t][0] = fmaxf(mx[t][0], __shfl_xor_sync(0xffffffffu, mx[t][0], d));
          mx[t][1] = fmaxf(mx[t][1], __shfl_xor_sync(0xffffffffu, mx[t][1], d));
        }
      bool moved = false;
      float al[NT][2], mu[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const bool grow = mx[t][w] > m[t][w] + kLazyLog2;
          al[t][w] = grow ? ex2(m[t][w] - mx[t][w]) : 1.f;
          m[t][w] = grow ? mx[t][w] : m[t][w];
          mu[t][w] = m[t][w] == -INFINITY ? 0.f : m[t][w];
          moved |= grow;
        }
#pragma unroll
      for (int i = 0; i < kPair; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[i][t][x] = ex2(sc[i][t][x] - mu[t][x & 1]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float add = 0.f;
#pragma unroll
          for (int i = 0; i < kPair; ++i) add += sc[i][t][w] + sc[i][t][w + 2];
          l[t][w] = l[t][w] * al[t][w] + add;
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[t][i][x] *= al[t][x & 1];
      }
#pragma unroll
      for (int i = 0; i < kPair; ++i) {
        if ((whole >> i) & 1u) {
          wp::page_pv<FMT, NT>(stp[i], sc[i], lane, o);
        } else if ((real >> i) & 1u) {
          const int n0 = ((e < it.head ? e : e + jump) * kPair + i) * kPageRows;
          // consecutive rows see together the last row's end of the keys and the first row's window; a key that
          // rows between see and neither border row does cannot be (a page is as long as a group is at most)
          const int p0 = it.p0;
          const uint32_t any = seen_bits(a, n0, it.p1, p0);
          const bool same = it.rows == 1 || (any == seen_bits(a, n0, p0, p0) && any == seen_bits(a, n0, it.p1, it.p1));
          wp::page_pv_masked<FMT, NT>(stp[i], sc[i], lane, o, any, same, it.rows,
                                      [&](int r) { return seen_bits(a, n0, p0 + r, p0 + r); }, row_of);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[st]);
      st += kWarps;
      if (st >= NS) {
        st -= NS;
        ph ^= 1;
      }
    }
    mine -= n;

    // ---- the warps' partials meet, one column tile at a time
    const bool whole_unit = first == 0 && end == it.pairs;
    const int cols = it.rows * G;
    float* part = nullptr;
    if (!whole_unit) part = a.split_ws + (2 * static_cast<int64_t>(blockIdx.x) + (first == 0 ? 1 : 0)) * kSlot;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[t][0] += __shfl_xor_sync(0xffffffffu, l[t][0], x);
        l[t][1] += __shfl_xor_sync(0xffffffffu, l[t][1], x);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) mg->o[warp][2 * c + (x & 1)][wp::o_dim<FMT>(i, x >> 1, hh)] = o[t][i][x];
      if (hh == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          mg->m[warp][2 * c + w] = m[t][w];
          mg->l[warp][2 * c + w] = l[t][w];
        }
      }
      consumers_sync<kWarps>();
      // a warp takes a column, a lane four dims
      const int n_cols = min(8, cols - 8 * t);
      for (int q = warp; q < n_cols; q += kWarps) {
        float M = mg->m[0][q];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, mg->m[w][q]);
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          // without a maximum every weight is 0 (or NaN, which has to stay)
          const float f = M == -INFINITY ? 1.f : ex2(mg->m[w][q] - M);
          add4(O, f, *reinterpret_cast<const float4*>(&mg->o[w][q][4 * lane]));
          L += f * mg->l[w][q];
        }
        const int col = 8 * t + q;
        if (whole_unit) {
          store_out(a, it.row0 + (col >> gshift), g * G + (col & (G - 1)), lane, M, L, O);
        } else {
          *reinterpret_cast<float4*>(part + col * kHeadDim + 4 * lane) = O;
          if (lane == 0) {
            part[kCols * kHeadDim + col] = M;
            part[kCols * (kHeadDim + 1) + col] = L;
          }
        }
      }
      consumers_sync<kWarps>();  // the buffer is free for the next tile or unit
    }
    if (!whole_unit) {
      // publish, draw a ticket; the unit's last CTA merges its parts in pair order
      const int c0 = cut.of(u0), c1 = cut.of(u0 + it.pairs - 1);
      const int64_t unit = static_cast<int64_t>(item) * H + g;
      if (threadIdx.x == 0) {  // (released with the warps' stores, which came before the barrier)
        int before;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.split_tickets + unit) : "memory");
        ctl->last = before == c1 - c0;
      }
      consumers_sync<kWarps>();
      if (ctl->last) {
        for (int col = warp; col < cols; col += kWarps) {
          // lane p holds part c0 + p's maximum and sum, 32 parts at a time
          const auto slot = [&](int c) { return a.split_ws + (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * kSlot; };
          const float* s0 = slot(min(c0 + lane, c1));
          const float m0 = __ldcg(s0 + kCols * kHeadDim + col), l0 = __ldcg(s0 + kCols * (kHeadDim + 1) + col);
          float M = m0;
          for (int c = c0 + 32 + lane; c <= c1; c += 32) M = fmaxf(M, __ldcg(slot(c) + kCols * kHeadDim + col));
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
          float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
          float L = 0.f;
          for (int base = c0; base <= c1; base += 32) {
            const int n_parts = min(32, c1 - base + 1);
            float f = 0.f, l_of = 0.f;
            if (lane < n_parts) {
              const float* s = slot(base + lane);
              const float mp = base == c0 ? m0 : __ldcg(s + kCols * kHeadDim + col);
              f = M == -INFINITY ? 1.f : ex2(mp - M);
              l_of = f * (base == c0 ? l0 : __ldcg(s + kCols * (kHeadDim + 1) + col));
            }
#pragma unroll 8
            for (int p = 0; p < n_parts; ++p) {
              L += __shfl_sync(0xffffffffu, l_of, p);
              add4(O, __shfl_sync(0xffffffffu, f, p),
                   __ldcg(reinterpret_cast<const float4*>(slot(base + p) + col * kHeadDim + 4 * lane)));
            }
          }
          store_out(a, it.row0 + (col >> gshift), g * G + (col & (G - 1)), lane, M, L, O);
        }
        if (threadIdx.x == 0) a.split_tickets[unit] = 0;
      }
    }
    }
    const int64_t took = min(static_cast<int64_t>(it.pairs + kUnitCost - first), left);
    left -= took;
    if (left <= 0) break;
    s += took;
    off = 0;
    if (++g == H) {
      g = 0;
      it = decode_item(a, ++item);
    }
  }
}

template <int FMT, int NT>
cudaError_t launch_one(const WindowArgs& a, const CUtensorMap& tmap, int sms, cudaStream_t stream) {
  constexpr size_t smem = kSmem<FMT, NT>;
  static_assert((smem + 1024) * Cfg<FMT, NT>::kCtas <= 228 * 1024, "the CTAs of an SM exceed its shared memory");
  auto kern = window_attend_kernel<FMT, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  dim3 grid;
  if (a.split_ws != nullptr) {
    grid = dim3(static_cast<unsigned>(sms * Cfg<FMT, NT>::kCtas));
  } else {
    const int64_t groups = a.cu_seqlens_q != nullptr
                               ? static_cast<int64_t>(a.num_rows) / a.rows_per_group + a.num_reqs
                               : static_cast<int64_t>(a.num_reqs) * a.groups_per_req;
    grid = dim3(static_cast<unsigned>(groups), static_cast<unsigned>(a.num_kv_heads));
  }
  kern<<<grid, Cfg<FMT, NT>::kThreads, smem, stream>>>(tmap, a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_cols(const WindowArgs& a, const CUtensorMap& tmap, int sms, cudaStream_t stream) {
  return a.rows_per_group * a.group > 8 ? launch_one<FMT, 2>(a, tmap, sms, stream) : launch_one<FMT, 1>(a, tmap, sms, stream);
}

constexpr int kMaxCtas = 4;  // per SM, of any configuration
constexpr size_t kMaxPartialBytes = 16 * (kHeadDim + 2) * sizeof(float);

}  // namespace

size_t window_workspace_bytes(int sms, int64_t units) {
  return static_cast<size_t>(sms) * kMaxCtas * 2 * kMaxPartialBytes + static_cast<size_t>(units) * sizeof(int32_t);
}

void window_geometry(WindowArgs* a, int max_rows) {
  // 8 columns while the rows at hand fit them, else 16
  const int cols = static_cast<int64_t>(max_rows) * a->group <= 8 ? 8 : 16;
  a->rows_per_group = max_rows < cols / a->group ? max_rows : cols / a->group;
  a->groups_per_req = (a->decode_query_len + a->rows_per_group - 1) / a->rows_per_group;
}

cudaError_t launch_window_attend(const WindowArgs& a, const CUtensorMap& tmap, int sms, cudaStream_t stream) {
  switch (a.kv_dtype) {
    case PBS_KV_BF16: return launch_cols<PBS_KV_BF16>(a, tmap, sms, stream);
    case PBS_KV_FP8_E4M3: return launch_cols<PBS_KV_FP8_E4M3>(a, tmap, sms, stream);
    case PBS_KV_NVFP4: return launch_cols<PBS_KV_NVFP4>(a, tmap, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pbs
