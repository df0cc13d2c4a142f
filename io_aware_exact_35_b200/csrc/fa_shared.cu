// fa_shared.cu - decode of a batch whose sequences share a long prefix.
//
// Sequences come in groups of consecutive batch entries; group g shares a
// prefix of L_g keys held once in the pages of the cache, and sequence b has
// L_b keys of its own behind it.  One query per (b, head) attends both parts:
//   o = softmax(scale q [K_prefix; K_own]^T) [V_prefix; V_own].
// Softmax splits over keys: each part (and each split of a part) gives a state
// (m, l, acc) in log2 units, and the states are merged as in the decode
// kernels: M = max m_s, o = sum 2^(m_s - M) acc_s / sum 2^(m_s - M) l_s.
//
// Own keys are few per sequence and of unlike number; their kernel is described
// below.  The prefix is read once for all: the queries of a group that share a key/value head, n_g x (H / Hkv)
// rows, form a dense tile, S = Q K^T and O += P V, on the tensor cores.  With
// up to 128 rows the reads of K and V bound it (128 flops per byte and row
// against 253 of the card); with more rows the products do.
//
// One CTA: a tile of rows of one (group, key/value head) against one split of
// the prefix, in key tiles of 128.  A single chain S -> softmax -> P V is
// serial, so two run side by side, each with its own S, O, m and l:
//   PAIR   256 rows, chain c takes rows 128 c ..; a K / V tile serves both.
//   else   128 rows, chain c takes the key tiles j = c mod 2; the two are merged
//          at the end.
//   warps 0-3, 4-7  softmax of chain 0, 1: thread t owns row t.
//   warps 8-11      producers.  Rows of a page are contiguous, so a whole key
//                   tile comes as TMA boxes of one page each (or 128 rows of
//                   it), issued by the threads that own their first rows.  A
//                   tile with keys past the prefix or on a bad page, and pages
//                   of fewer than 8 rows, come row by row with 16-byte
//                   asynchronous copies that fill such keys with zeros (stale
//                   rows of a page may hold anything, and 0 x NaN would spread).
//   warp 12         tensor memory and the MMA issue; ring order
//                   PAIR K0 V0 K1 V1 .., else K0 K1 | V0 K2 | V1 K3 | ..
// Tensor memory (512 columns): S_0, S_1 [0, 256), O_0, O_1 [256, 512); P_c
// overwrites the first half of S_c as bf16.
//
// Measured: a key tile against 256 rows takes 1.9 us, 0.79 of the card's rate of
// products; a CTA's start and end about 9 us.  128 sequences over 32K shared keys
// 105 to 112 us a call, 33 over two prompts 41, 3 over 1000 keys 12.
//
// Scores, maxima, sums and O are in 32 bits.  P is rounded to bf16, the operand type
// of the product with V (half a step, 2^-8 of a probability; l is summed before it):
// such errors add up at random, so that O is 1.3 to 1.4 times as far from 64 bits as
// with P in 32 bits (0.0021-0.0023 against 0.0016-0.0017 over these shapes).
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

namespace shared {

constexpr int ROWS = 128;
constexpr int KEYS = 128;
constexpr int THREADS = 512;
constexpr int INFO = 8;                // key tiles whose pages and masks are kept
constexpr int TMA_ROWS = 8;            // smallest page that TMA fetches: a swizzle atom
constexpr int PRODUCERS = 128;
constexpr int WARP_MMA = 12;
// setmaxnreg split: 256 x 176 + 256 x 80 = the 512 x 128 launched.
constexpr int REGS_SOFTMAX = 176;
constexpr int REGS_OTHER = 80;
static_assert(256 * REGS_SOFTMAX + 256 * REGS_OTHER <= 65536,
              "setmaxnreg.inc would wait forever: the split exceeds the launch's registers");
constexpr int PANEL = 128 * 128;       // 128 rows x 64 bf16
constexpr float STALE_MAX = 8.0f;      // log2 units: O and l are rescaled beyond
constexpr int SM_COUNT = 148;          // sizes the splits (and so the workspace) alone

template <int D, bool PAIR>
struct Smem {
  static constexpr int TILE = D / 64 * PANEL;
  static constexpr int NSLOT = PAIR ? 4 : 5;                    // ring tiles
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = (PAIR ? 2 : 1) * TILE;
  static constexpr int PAGES_OFF = RING_OFF + NSLOT * TILE;     // int [INFO][KEYS]
  static constexpr int MASK_OFF = PAGES_OFF + INFO * KEYS * 4;  // unsigned [INFO][4]
  static constexpr int STAT_OFF = MASK_OFF + INFO * 16;         // m, l of both chains
  static constexpr int BAR_OFF = STAT_OFF + 4 * ROWS * 4;
  static constexpr int NBAR = 2 * NSLOT + 4 + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SUMS_OFF = MISC_OFF + 16;                // sums over the lengths
  static constexpr int BYTES = SUMS_OFF + 32 * 4;
  // one CTA (and its 512 tensor-memory columns) per SM
  static constexpr int ALLOC = BYTES > 118784 ? BYTES : 118784;
  // after the last product Q and the ring hold the output rows, padded to keep
  // the 16-byte accesses of neighbouring rows on different banks
  static constexpr int OUT_ROW = D + 4;
  static_assert((PAIR ? 2 : 1) * ROWS * OUT_ROW * 4 <= PAGES_OFF, "the output rows fit");
};

// The combine kernel waits for the grid before it and reads the partials of both
// kernels, so the later of the two ends no earlier than the other: its last CTA
// waits.  (Nothing to wait for where the launch was an ordinary one.)
__device__ __forceinline__ void outlast(bool last) {
  if (last) asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct Params {
  const __nv_bfloat16 *q, *kpages, *vpages;
  const int* table;       // [G][stride]
  const int* lens;        // [G]
  const int* cu;          // [G + 1]; null: one group of all B
  float* po;              // prefix partials [B * H][S][D]
  float2* pml;            // [B * H][S] (m, l)
  float* own_po;          // own partials [B * H][slots][D]
  float2* own_pml;        // [B * H][slots]
  int* own_count;         // own partials of each (sequence, head tile), if it has own keys
  long long table_stride;
  int* splits;            // the number of splits taken, where it is chosen here
  const int* own_lens;    // [B], at most Lmax
  int B, H, Hkv, G, S;
  int choose;             // 1: at most S splits, as the lengths ask
  int units, own_ctas;    // prefix CTAs per split, at least; CTAs of the own keys
  float key_kb;           // K and V of a key, as a part of each of those
  int Lmax;
  int pages, log2_page, num_pages;
  int box;                // rows of a TMA box; 0: copies row by row
  rope::Quotient by_r;    // by H / Hkv
  float scale_log2;
};

// First and last batch entry of group g; false (and reported, and first = -1) if it
// leaves the batch or runs backwards.
__device__ __forceinline__ bool group_range(const int* cu, int B, int g, int& b0, int& b1) {
  b0 = cu == nullptr ? 0 : cu[g];
  b1 = cu == nullptr ? B : cu[g + 1];
  if (b0 >= 0 && b1 >= b0 && b1 <= B) return true;
  record_error(1 /* FA_ERR_INVALID_ARG */);
  b0 = b1 = -1;
  return false;
}

// Each group begins where the one before it ends, so they are disjoint until one is
// refused, which is taken as empty; from then on a group begins no earlier than the
// largest end so far.  An entry therefore has one group, whose CTAs alone write its
// partials, and there are no more row tiles than the grid has.  A search that meets
// what it looks for before any refused group needs none of this; the others take the
// ranges from here, one warp, 32 groups at a time in their order (g0 = 0, 32, ..; lane i
// takes group g0 + i).
struct GroupsBehind {
  int end = 0;  // the largest end of the groups before g0
  __device__ __forceinline__ void take(const int* cu, int B, int G, int g0, int& b0, int& b1) {
    const int lane = threadIdx.x & 31;
    b0 = b1 = 0;
    if (g0 + lane < G) group_range(cu, B, g0 + lane, b0, b1);
    int upto = b1;  // the largest end up to this lane, then before it
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) upto = max(upto, __shfl_up_sync(0xffffffffu, upto, off));
    const int before = __shfl_up_sync(0xffffffffu, upto, 1);
    b0 = max(b0, max(end, lane == 0 ? 0 : before));
    b1 = max(b0, b1);
    end = max(end, __shfl_sync(0xffffffffu, upto, 31));
  }
};

__device__ __forceinline__ int prefix_len(const int* lens, int g, int pages, int log2_page) {
  const long long cap = static_cast<long long>(pages) << log2_page;
  return static_cast<int>(min(static_cast<long long>(max(lens[g], 0)), cap));
}

// Key tiles of split s: [first, last) of nt.
__device__ __forceinline__ int split_begin(int s, int S, int nt) {
  return static_cast<int>(static_cast<long long>(s) * nt / S);
}

// With own keys beside it the prefix does better on fewer SMs.  A prefix CTA
// takes a whole SM and the own keys' CTAs, three to an SM, come in rounds on those
// that are left; rounds that have not begun when the prefix ends run behind it, so
// that the time jumps where one more is needed.  The time of a call with S splits,
// in us, from the longest prefix of nt tiles and the own keys' kilobytes per CTA:
// the prefix in waves of `tile` a key tile and `start` a CTA; a round of n CTAs in
// 3 and the slower of 22 KB/us a CTA and 6.2 GB/ms in all; 6 for a round behind the
// prefix.  The constants were fitted to 12 shapes, of which the split taken is at
// most 5 % behind the best.  Measured, GPU time: 128 sequences with 230 keys on
// average over 32K: 7 splits 91.7, 8 101.2, 9 (all SMs) 103.8, all SMs with the own
// keys first 99.3; with 32 keys on average 7 splits 88.0, 8 81.1, 9 80.4.  Choosing
// costs about 2 us, which a batch that has no own keys pays too (73.3 against 71.4).
__device__ __forceinline__ float split_cost(const Params& p, int S, int nt, float own_kb,
                                            float tile, float start) {
  const int busy = p.units * S;
  // quotients of small numbers, rounded up past the error of the division
  auto up = [](float a, float b) { return ceilf(a / b * 0.99999f); };
  const float prefix = up(busy, SM_COUNT) * (tile * up(nt, S) + start);
  if (own_kb == 0.f) return prefix;
  auto round = [&](int n) { return 3.f + own_kb * fmaxf(1.f / 22.f, n * (1.f / 6200.f)); };
  const float behind = prefix + 6.f;
  const int slots = 3 * max(SM_COUNT - busy, 0);
  if (slots == 0) return behind + round(p.own_ctas);
  const float t = round(min(slots, p.own_ctas));
  const float all = up(p.own_ctas, slots) * t;
  if (all <= prefix) return prefix;
  const float left = p.own_ctas - slots * up(prefix, t);  // begun behind the prefix
  return left > 0.f ? behind + round(static_cast<int>(left)) : all;
}

// The number of splits, the same in every CTA: the CTA's warps sum up the lengths
// (sums are added in one order), and behind a barrier each of them chooses.
// first: own_lens[threadIdx.x]; sums: 32 words of shared memory.
__device__ __forceinline__ void sum_lengths(const Params& p, int first, float* sums) {
  const int lane = threadIdx.x & 31;
  int nt = 0;
  float keys = static_cast<float>(min(max(first, 0), p.Lmax));
  for (int b = threadIdx.x + THREADS; b < p.B; b += THREADS)
    keys += static_cast<float>(min(max(p.own_lens[b], 0), p.Lmax));
  for (int g = threadIdx.x; g < p.G; g += THREADS)
    nt = max(nt, (prefix_len(p.lens, g, p.pages, p.log2_page) + KEYS - 1) / KEYS);
  nt = __reduce_max_sync(0xffffffffu, nt);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) keys += __shfl_xor_sync(0xffffffffu, keys, off);
  if (lane == 0) {
    sums[threadIdx.x >> 5] = keys;
    sums[16 + (threadIdx.x >> 5)] = __int_as_float(nt);
  }
}

__device__ __forceinline__ int choose_splits(const Params& p, const float* sums, float tile,
                                             float start) {
  const int lane = threadIdx.x & 31;
  float keys = sums[lane & 15];
  const int nt = __reduce_max_sync(0xffffffffu, __float_as_int(sums[16 + (lane & 15)]));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) keys += __shfl_xor_sync(0xffffffffu, keys, off);
  const float own_kb = keys * p.key_kb;
  float best = INFINITY;
  int S = p.S;
  for (int s = lane + 1; s <= p.S; s += 32) {
    const float c = split_cost(p, s, nt, own_kb, tile, start);
    if (c < best) {
      best = c;
      S = s;
    }
  }
  // the least cost (not negative: it orders as its bits do), then the fewest splits
  const unsigned bits = __float_as_uint(best);
  const unsigned least = __reduce_min_sync(0xffffffffu, bits);
  return __reduce_min_sync(0xffffffffu, bits == least ? S : p.S);
}

// One warp: the group of the flat tile index, the row tile within it, the
// group's batch entries and its prefix length.  BEHIND: a refused group lies before.
template <bool BEHIND = false>
__device__ __forceinline__ bool find_tile(const Params& p, int r, int tile, int tile_rows,
                                          int& local, int& g, int& b0, int& b1, int& len) {
  constexpr int MANY = 1 << 25;  // more tiles than there are; 32 of them are no overflow
  const int lane = threadIdx.x & 31;
  int before = 0;
  GroupsBehind ranges;
  for (int g0 = 0; g0 < p.G; g0 += 32) {
    int n = 0, first = 0, last = 0, length = 0;
    if (BEHIND) ranges.take(p.cu, p.B, p.G, g0, first, last);
    if (g0 + lane < p.G) {
      length = prefix_len(p.lens, g0 + lane, p.pages, p.log2_page);
      const bool ok = BEHIND || group_range(p.cu, p.B, g0 + lane, first, last);
      n = (static_cast<int>(static_cast<long long>(last - first) * r) + tile_rows - 1) / tile_rows;
      n = ok ? n : MANY;
    }
    int upto = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > tile);
    if (hit != 0u) {
      const int at = __ffs(hit) - 1;
      b0 = __shfl_sync(0xffffffffu, first, at);
      if (!BEHIND && b0 < 0) return find_tile<true>(p, r, tile, tile_rows, local, g, b0, b1, len);
      g = g0 + at;
      local = tile - before - __shfl_sync(0xffffffffu, upto - n, at);
      b1 = __shfl_sync(0xffffffffu, last, at);
      len = __shfl_sync(0xffffffffu, length, at);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// One warp: the prefix length of the group that batch entry b belongs to; 0 without
// one.
template <bool BEHIND = false>
__device__ __forceinline__ int entry_prefix(const Params& p, int b) {
  const int lane = threadIdx.x & 31;
  GroupsBehind ranges;
  for (int g0 = 0; g0 < p.G; g0 += 32) {
    bool mine = false;
    int len = 0, b0, b1;
    if (BEHIND) ranges.take(p.cu, p.B, p.G, g0, b0, b1);
    if (g0 + lane < p.G) {
      len = prefix_len(p.lens, g0 + lane, p.pages, p.log2_page);
      if (!BEHIND && !group_range(p.cu, p.B, g0 + lane, b0, b1)) len = -1;
      mine = (b >= b0 && b < b1) || len < 0;
    }
    const unsigned m = __ballot_sync(0xffffffffu, mine);
    if (m != 0u) {
      len = __shfl_sync(0xffffffffu, len, __ffs(m) - 1);
      return !BEHIND && len < 0 ? entry_prefix<true>(p, b) : len;
    }
  }
  return 0;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    fa_shared_prefix_kernel(const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const Params p) {
  using L = Smem<D, PAIR>;
  constexpr int NSLOT = L::NSLOT;
  constexpr int CTA_ROWS = PAIR ? 2 * ROWS : ROWS;
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = blockIdx.x;
  const int hk = blockIdx.z;
  const int r = p.H / p.Hkv;
  const int own_len0 = p.choose && threadIdx.x < p.B ? p.own_lens[threadIdx.x] : 0;
  int g = 0, local = 0, b0 = 0, b1 = 0, len = 0;
  const bool found = find_tile(p, r, blockIdx.y, CTA_ROWS, local, g, b0, b1, len);
  const int row0 = local * CTA_ROWS;
  const int rows = min(CTA_ROWS, (b1 - b0) * r - row0);
  const int nt = (len + KEYS - 1) / KEYS;
  int j0 = split_begin(split, p.S, nt);
  int n = found ? split_begin(split + 1, p.S, nt) - j0 : 0;  // key tiles of this CTA
  const bool aligned = (smem_u32(smem) & 1023u) == 0;        // the swizzled tiles need it
  if (!aligned) {
    if (threadIdx.x == 0) record_error(2 /* FA_ERR_UNSUPPORTED */);
    n = 0;
  }
  const bool last = blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 &&
                    blockIdx.z == gridDim.z - 1;
  if (n <= 0 && !p.choose) {
    outlast(last);
    return;
  }

  int* pages = reinterpret_cast<int*>(smem + L::PAGES_OFF);
  unsigned* masks = reinterpret_cast<unsigned*>(smem + L::MASK_OFF);
  float* stat = reinterpret_cast<float*>(smem + L::STAT_OFF);
  float* sums = reinterpret_cast<float*>(smem + L::SUMS_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* empty = full + NSLOT;
  uint64_t* s_full = empty + NSLOT;  // [2]
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* mma_final = p_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  int* fetched = reinterpret_cast<int*>(smem + L::MISC_OFF + 8);  // ring tiles begun by any producer

  if (threadIdx.x == 0) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&full[s], PRODUCERS);
      mbar_init(&empty[s], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&s_full[c], 1);
      mbar_init(&p_full[c], 4);
    }
    mbar_init(mma_final, 1);
    *abort_flag = 0;
    *fetched = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 8 * 32 && p.box > 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (p.choose) sum_lengths(p, own_len0, sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (p.choose) {
    const int S = choose_splits(p, sums, PAIR ? 1.75f : 1.0f, PAIR ? 12.f : 9.f);
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) *p.splits = S;
    j0 = split_begin(split, S, nt);
    n = found && aligned && split < S ? split_begin(split + 1, S, nt) - j0 : 0;
    if (n <= 0) {
      if (warp == WARP_MMA) tmem_dealloc(tmem_base, 512);
      outlast(last);
      return;
    }
  }

  int begun = 0;  // ring tiles that this producer has arrived for
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == WARP_MMA) {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t IDESC_S = idesc_bf16_f32(ROWS, KEYS, false, false);
      constexpr uint32_t IDESC_O = idesc_bf16_f32(ROWS, D, false, true);
      const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + L::Q_OFF));
      const uint64_t kd0 = sdesc_kmajor_sw128(smem_u32(smem + L::RING_OFF));
      const uint64_t vd0 = sdesc_mnmajor_sw128(smem_u32(smem + L::RING_OFF), PANEL);
      int pcount[2] = {0, 0};
      // ring tile u has arrived
      auto ready = [&](int u) {
        const bool ok = mbar_wait_warp(&full[u % NSLOT], (u / NSLOT) & 1, abort_flag);
        tc_fence_after();
        return ok;
      };
      // S_c = Q K^T with the keys in ring tile u
      auto issue_s = [&](int c, int u) {
        const uint64_t qc = qd + static_cast<uint64_t>(((PAIR ? c : 0) * L::TILE) >> 4);
        const uint64_t kd = kd0 + static_cast<uint64_t>((u % NSLOT * L::TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * PANEL + (kk & 3) * 32) >> 4);
          mma_bf16_ss_w(tmem_base + c * 128, qc + off, kd + off, IDESC_S, kk > 0 ? 1u : 0u);
        }
        mma_commit_w(&s_full[c]);
      };
      // O_c (+)= P_c V with the values in ring tile u
      auto issue_pv = [&](int c, int u, bool first) {
        if (!mbar_wait_warp(&p_full[c], pcount[c] & 1, abort_flag)) return false;
        ++pcount[c];
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>((u % NSLOT * L::TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < KEYS / 16; ++kk)
          mma_bf16_ts_w(tmem_base + 256 + c * 128, tmem_base + c * 128 + kk * 8,
                        vd + static_cast<uint64_t>((kk * 2048) >> 4), IDESC_O,
                        (!first || kk > 0) ? 1u : 0u);
        return true;
      };
      auto release = [&](int u) { mma_commit_w(&empty[u % NSLOT]); };
      named_barrier(3, 2 * ROWS + 32);  // Q is in shared memory
      bool ok;
      if constexpr (PAIR) {  // K_j is ring tile 2 j, V_j ring tile 2 j + 1
        ok = ready(0);
        if (ok) {
          issue_s(0, 0);
          issue_s(1, 0);
          release(0);
        }
        for (int j = 0; ok && j < n; ++j) {
          const bool more = j + 1 < n;
          const int v = 2 * j + 1, k = 2 * j + 2;
          ok = ready(v) && issue_pv(0, v, j == 0) && (!more || ready(k));
          if (ok && more) issue_s(0, k);
          ok = ok && issue_pv(1, v, j == 0);
          if (ok) release(v);
          if (ok && more) {
            issue_s(1, k);
            release(k);
          }
        }
      } else {
        int u = 0;
        auto keys = [&](int c) {
          if (!ready(u)) return false;
          issue_s(c, u);
          release(u++);
          return true;
        };
        ok = keys(0) && (n < 2 || keys(1));
        for (int j = 0; ok && j < n; ++j) {
          ok = ready(u) && issue_pv(j & 1, u, j < 2);
          if (ok) release(u++);
          if (ok && j + 2 < n) ok = keys(j & 1);
        }
      }
      mma_commit_w(mma_final);
      mbar_wait_drain(mma_final, 0);
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    // ------------------------------------------------------------ producers
    const int t = threadIdx.x - 8 * 32;
    const int page_mask = (1 << p.log2_page) - 1;
    const long long page_elems = (static_cast<long long>(p.Hkv) << p.log2_page) * D;
    const long long head_elems = (static_cast<long long>(hk) << p.log2_page) * D;
    const int* table = p.table + g * p.table_stride;
    // Row-by-row copies in flight behind the newest tile.  One tile fewer than
    // the ring waits for: with PAIR a value tile is released only once the next
    // key tile has been handed over, one tile later.
    constexpr int LAG = NSLOT - 2;
    constexpr int CH = D / 8;            // 16-byte pieces per row
    constexpr int STEP = PRODUCERS / CH;  // rows per step
    const int ch = t % CH;
    const uint32_t ring = smem_u32(smem + L::RING_OFF);
    auto entry = [&](int j) {  // page of key t of tile j; -1 past the prefix
      const int key = (j0 + j) * KEYS + t;
      return j < n && key < len ? table[key >> p.log2_page] : -1;
    };
    int ahead = entry(0);
    // pages of tile j (-1: masked) and its mask
    auto look_up = [&](int j) {
      int page = ahead;
      ahead = entry(j + 1);  // in flight until the next tile
      if ((j0 + j) * KEYS + t < len && (page < 0 || page >= p.num_pages)) {
        record_error(1 /* FA_ERR_INVALID_ARG */);
        page = -1;
      }
      pages[(j % INFO) * KEYS + t] = page;
      const unsigned m = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) masks[(j % INFO) * 4 + (t >> 5)] = m;
      named_barrier(1, PRODUCERS);
    };
    int& u = begun;
    auto load = [&](const CUtensorMap& map, const __nv_bfloat16* pool, int j) {
      const int slot = u % NSLOT;
      if (u >= NSLOT && !mbar_wait(&empty[slot], (u / NSLOT - 1) & 1, abort_flag)) return false;
      ++u;
      const int* pj = pages + (j % INFO) * KEYS;
      const uint4 mk = *reinterpret_cast<const uint4*>(masks + (j % INFO) * 4);
      if (p.box > 0 && (mk.x & mk.y & mk.z & mk.w) == 0xffffffffu) {
        if ((t & (p.box - 1)) == 0) {
          mbar_arrive_expect_tx(&full[slot], p.box * D * 2);
          const int outer = pj[t] * p.Hkv + hk;
          const int row = ((j0 + j) * KEYS + t) & page_mask;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(smem + L::RING_OFF + slot * L::TILE + c * PANEL + t * 128, &map, &full[slot],
                        c * 64, row, outer);
        } else {
          mbar_arrive(&full[slot]);
        }
        return true;
      }
      const uint32_t dst = ring + slot * L::TILE + (ch >> 3) * PANEL;
#pragma unroll
      for (int i = 0; i < KEYS / STEP; ++i) {
        const int row = i * STEP + t / CH;
        const int page = pj[row];
        const long long off =
            page * page_elems + head_elems + (((j0 + j) * KEYS + row) & page_mask) * D;
        copy16(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4), pool + (page >= 0 ? off : 0) + ch * 8,
               page >= 0);
      }
      copy_commit();
      if (p.box > 0) {  // one of few such tiles
        copy_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&full[slot]);
      } else if (u > LAG) {
        // the tile LAG before this one has landed: hand it to the tensor core
        copy_wait<LAG>();
        fence_proxy_async_smem();
        mbar_arrive(&full[(u - 1 - LAG) % NSLOT]);
      }
      return true;
    };
    bool ok = true;
    if constexpr (PAIR) {
      for (int j = 0; j < n; ++j) {
        look_up(j);
        ok = ok && load(kmap, p.kpages, j) && load(vmap, p.vpages, j);
      }
    } else {
      look_up(0);
      ok = load(kmap, p.kpages, 0);
      if (n > 1) {
        look_up(1);
        ok = ok && load(kmap, p.kpages, 1);
      }
      for (int j = 0; j < n; ++j) {
        ok = ok && load(vmap, p.vpages, j);
        if (j + 2 < n) {
          look_up(j + 2);
          ok = ok && load(kmap, p.kpages, j + 2);
        }
      }
    }
    if (p.box == 0) {
      copy_wait<0>();
      fence_proxy_async_smem();
      if (ok)
        for (int v = max(0, u - LAG); v < u; ++v) mbar_arrive(&full[v % NSLOT]);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ------------------------------------------------------------ softmax
    // Query rows, 128-byte swizzle, while the first keys are on their way; rows
    // that do not exist are zero.
    {
      constexpr int CH = D / 8, STEP = 2 * ROWS / CH, N = CTA_ROWS / STEP;
      const int ch = threadIdx.x % CH, r0 = threadIdx.x / CH;
      uint4 v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int rr = row0 + r0 + i * STEP;
        v[i] = make_uint4(0, 0, 0, 0);
        if (rr - row0 < rows) {
          const int bq = p.by_r(rr);
          const size_t at =
              (static_cast<size_t>(b0 + bq) * p.H + hk * r + (rr - bq * r)) * D + ch * 8;
          if (dbg_ok(at + 8 <= static_cast<size_t>(p.B) * p.H * D))
            v[i] = *reinterpret_cast<const uint4*>(p.q + at);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = r0 + i * STEP;
        *reinterpret_cast<uint4*>(smem + L::Q_OFF + (row / ROWS) * L::TILE + (ch >> 3) * PANEL +
                                  (row % ROWS) * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v[i];
      }
      fence_proxy_async_smem();
      named_barrier(3, 2 * ROWS + 32);
    }
    const int c = warp >> 2;
    const int row = threadIdx.x & (ROWS - 1);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem_base + c * 128 + lane_off;
    const uint32_t tO = tmem_base + 256 + c * 128 + lane_off;
    const int first = PAIR ? c * ROWS : 0;                 // of the chain's rows
    const bool idle = first + (warp & 3) * 32 >= rows;     // none of this warp's rows exists
    constexpr int STRIDE = PAIR ? 1 : 2;                   // the chain's key tiles
    const float sl2 = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    int phase = 0;
    for (int j = PAIR ? 0 : c; j < n; j += STRIDE, phase ^= 1) {
      if (!mbar_wait_warp(&s_full[c], phase, abort_flag)) break;
      if (idle) {  // rows of a product are independent: theirs may hold anything
        if (lane == 0) mbar_arrive(&p_full[c]);
        continue;
      }
      tc_fence_after();
      uint32_t sr[128];
      tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
      tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
      const uint4 mk = *reinterpret_cast<const uint4*>(masks + (j % INFO) * 4);
      tmem_ld_wait();
      // Masked keys get -inf after the scale; so does the rare scale that is
      // not positive, where the largest product is not the largest score.
      const bool whole = (mk.x & mk.y & mk.z & mk.w) == 0xffffffffu;
      float mul = sl2;
      if (!whole || sl2 <= 0.f) {
        const unsigned mw[4] = {mk.x, mk.y, mk.z, mk.w};
#pragma unroll
        for (int i = 0; i < 128; ++i)
          sr[i] = ((mw[i >> 5] >> (i & 31)) & 1u)
                      ? __float_as_uint(__uint_as_float(sr[i]) * sl2) : __float_as_uint(-INFINITY);
        mul = 1.f;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 128; i += 2)
        mx[(i >> 1) & 3] = fmax3(mx[(i >> 1) & 3], __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
      const float hi = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
      const float m_new = fmaxf(m, hi);
      const bool grow = __any_sync(0xffffffffu, (m_new - m) > STALE_MAX);
      const float m_use = grow ? m_new : m;
      const float m_ref = (m_use == -INFINITY) ? 0.f : m_use;
      const float alpha = grow ? ex2_approx(m - m_ref) : 1.f;
      if (grow && j >= STRIDE) {
        // complete: S of this tile was issued after O += P V of the chain's last one
#pragma unroll 1
        for (int i = 0; i < D; i += 8) {
          uint32_t o[8];
          fwd::tmem_ld8(tO + i, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          fwd::tmem_st8(tO + i, o);
        }
      }
      const uint64_t sl2_2 = fwd::pack_f32x2(mul, mul);
      const uint64_t neg_m = fwd::pack_f32x2(-m_ref, -m_ref);
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 128; i += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1;
          fwd::fma_f32x2(x0, x1, __uint_as_float(sr[i + e]), __uint_as_float(sr[i + e + 1]), sl2_2,
                         neg_m);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          fwd::add_f32x2(sum[(e >> 1) & 3], p0, p1);
          pk[e >> 1] = pack_bf16x2(p0, p1);
        }
        tmem_st16(tS + (i >> 1), pk);
      }
      l = l * alpha + ((fwd::sum_f32x2(sum[0]) + fwd::sum_f32x2(sum[1])) +
                       (fwd::sum_f32x2(sum[2]) + fwd::sum_f32x2(sum[3])));
      m = m_use;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[c]);
    }
    stat[c * ROWS + row] = m;
    stat[(2 + c) * ROWS + row] = l;
    // Every product has completed: merge the chains.  Only these warps, which
    // hold the registers for it, take part.
    const bool done = mbar_wait_warp(mma_final, 0, abort_flag);
    tc_fence_after();
    named_barrier(2, 2 * ROWS);
    float* out = reinterpret_cast<float*>(smem);
    float w = 1.f;
    if constexpr (!PAIR) {
      const float m0 = stat[row], m1 = stat[ROWS + row], mine = c == 0 ? m0 : m1;
      w = mine == -INFINITY ? 0.f : ex2_approx(mine - fmaxf(m0, m1));
    }
    auto rows_out = [&](bool add) {
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
        uint32_t o[32];
        tmem_ld32(tO + i, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4* at = reinterpret_cast<float4*>(out + (first + row) * L::OUT_ROW + i + e);
          float4 v = add ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
          v.x = fmaf(w, __uint_as_float(o[e]), v.x);
          v.y = fmaf(w, __uint_as_float(o[e + 1]), v.y);
          v.z = fmaf(w, __uint_as_float(o[e + 2]), v.z);
          v.w = fmaf(w, __uint_as_float(o[e + 3]), v.w);
          *at = v;
        }
      }
    };
    if constexpr (PAIR) {
      if (done && !idle) rows_out(false);
    } else {
      if (done && n > 1 && c == 1 && !idle) rows_out(false);
      named_barrier(2, 2 * ROWS);
      if (done && c == 0 && !idle) rows_out(n > 1);
    }
    named_barrier(2, 2 * ROWS);
    // Rows warp, warp + 8, .. by the warp; lane k knows where the k-th goes.
    long long mine;
    {
      const int rr = row0 + min(warp + lane * 8, rows - 1);
      const int bq = p.by_r(rr);
      mine = (static_cast<long long>(b0 + bq) * p.H + hk * r + (rr - bq * r)) * p.S + split;
    }
    const int count = done ? (rows - warp + 7) / 8 : 0;
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
      const long long at = __shfl_sync(0xffffffffu, mine, k);
      if (lane * 4 < D && dbg_ok(at < static_cast<long long>(p.B) * p.H * p.S))
        *reinterpret_cast<float4*>(p.po + at * D + lane * 4) =
            *reinterpret_cast<const float4*>(out + (warp + k * 8) * L::OUT_ROW + lane * 4);
    }
    if (lane < count && dbg_ok(mine < static_cast<long long>(p.B) * p.H * p.S)) {
      const int i = warp + lane * 8;
      if constexpr (PAIR) {  // row i of the tile is row i % 128 of chain i / 128
        p.pml[mine] = make_float2(stat[i], stat[2 * ROWS + i]);
      } else {
        const float a = stat[i], b = stat[ROWS + i];
        const float top = fmaxf(a, b);
        const float wa = a == -INFINITY ? 0.f : ex2_approx(a - top);
        const float wb = b == -INFINITY ? 0.f : ex2_approx(b - top);
        p.pml[mine] = make_float2(top, fmaf(wa, stat[2 * ROWS + i], wb * stat[3 * ROWS + i]));
      }
    }
  }
  tmem_ld_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  // Every copy issued must land before this CTA's shared memory is freed.  The
  // products asked for all of them, unless a wait gave up: then producers that gave up
  // earlier arrive for the tiles that others began (at most one per slot: to begin a
  // tile, the one before it in its slot was complete), and each slot's last tile is
  // waited for.  (Row-by-row copies have been waited for by their threads.)
  if (*abort_flag && p.box > 0) {  // no wait is left that could raise it
    const bool producer = warp >= 8 && warp < 12;
    if (producer) atomicMax(fetched, begun);
    __syncthreads();
    if (producer) {
      const int all = *static_cast<volatile int*>(fetched), t = threadIdx.x - 8 * 32;
      for (; begun < all; ++begun) mbar_arrive(&full[begun % NSLOT]);
      if (t < NSLOT && t < all) mbar_wait_drain(&full[t], ((all - 1 - t) / NSLOT) & 1);
    }
  }
  outlast(last);
}

// ------------------------------------------------------------------ own keys
// The own keys of all sequences as one list of steps of 16 keys: sequence by
// sequence, and within it key/value head by head (and by tiles of 16 query
// heads, for larger groups).  The resident warps share the list out evenly, so
// short and long sequences alike keep every warp busy to the end (the split-KV
// kernel, one CTA per (sequence, head, 512 keys), reads 128 x 8 heads of 256
// keys on average at 2.9 TB/s; this one at 3.6).  A warp streams its steps
// through a ring of its own in shared memory, fetched ahead by 16-byte
// asynchronous copies across the ends of rows, heads and sequences; where it
// leaves a (sequence, head) it writes one partial state.
//
// S = Q K^T and O^T += V^T P^T run on mma.sync m16n8k16 with the query heads of
// the group as rows (tcgen05 needs at least 64 rows; these are few), operands
// assigned to fragments as in the grouped decode kernel: every lane takes whole
// 16-byte pieces, lane (g, c) = (lane / 4, lane % 4)
//   K   of key g (and g + 8), d 32 i + 8 c ..;
//   V   of keys 2c, 2c + 1, 2c + 8, 2c + 9, d 64 i + 8 g ..
// A row's pieces are stored at piece ^ swizzle(row), which makes both patterns
// free of bank conflicts.
struct OwnParams {
  const __nv_bfloat16 *q, *kpages, *vpages;
  const int* table;       // [B][stride]
  const int* seqlens;
  float* po;              // [B * H][slots][D]
  float2* pml;
  int* count;             // [B][Hkv * tiles] partials
  long long table_stride;
  int B, H, Hkv, r, tiles;  // r query heads per key/value head in tiles of 16
  int Lmax, log2_page, num_pages, slots, min_steps;
  float scale_log2;
};

constexpr int OWN_WARPS = 4;
constexpr int OWN_CTAS = 3;            // resident per SM
constexpr int OWN_KEYS = 16;           // keys of a step
constexpr int OWN_INFO = 16;           // steps whose description is kept (a power of two)

template <int D>
struct OwnSmem {
  static constexpr int HALF = OWN_KEYS * D * 2;  // keys, or values, of a step
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int WARP = STAGES * 2 * HALF + OWN_INFO * 16;
  static constexpr int BYTES = OWN_WARPS * WARP;
};

__device__ __forceinline__ int own_len(const int* seqlens, int b, int Lmax) {
  return min(max(seqlens[b], 0), Lmax);
}
__device__ __forceinline__ int own_steps(int len) { return (len + OWN_KEYS - 1) / OWN_KEYS; }
__device__ __forceinline__ int own_swizzle(int row) { return (row & 6) ^ ((row & 1) << 2); }

template <int D, bool HI>
__global__ void __launch_bounds__(OWN_WARPS * 32, OWN_CTAS)
    fa_shared_own_kernel(const OwnParams p) {
  using L = OwnSmem<D>;
  constexpr int STAGES = L::STAGES;
  constexpr int NT = OWN_WARPS * 32;
  constexpr int NH = HI ? 2 : 1;     // 8-head column tiles of O^T
  constexpr int KS = D / 16;         // k-steps of S = Q K^T
  constexpr int MT = D / 16;         // m-tiles of O^T
  constexpr int NKL = D / 32;        // 16-byte pieces per K row per lane
  constexpr int NVL = D / 64;        // 16-byte pieces per V row per lane
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long sums[NT + 1];
  __shared__ int lens[NT];           // with up to NT sequences: one per thread
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cols = p.Hkv * p.tiles;

  // Steps before each thread's stretch of sequences, and in all.
  const int stretch = (p.B + NT - 1) / NT;
  {
    long long mine = 0;
    for (int i = 0; i < stretch; ++i) {
      const int b = threadIdx.x * stretch + i;
      if (b < p.B) {
        const int len = own_len(p.seqlens, b, p.Lmax);
        lens[threadIdx.x] = len;
        mine += own_steps(len);
      }
    }
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    __shared__ long long warps[OWN_WARPS];
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += warps[w];
    sums[threadIdx.x] = before + upto - mine;
    if (threadIdx.x == NT - 1) sums[NT] = before + upto;
    __syncthreads();
  }
  const long long total = sums[NT] * cols;
  const long long warps_all = static_cast<long long>(gridDim.x) * OWN_WARPS;
  const long long share = (total + warps_all - 1) / warps_all;
  const long long per = share > p.min_steps ? share : p.min_steps;
  const long long wid = static_cast<long long>(blockIdx.x) * OWN_WARPS + warp;
  const long long f0 = wid * per;
  const bool last = blockIdx.x == gridDim.x - 1 && warp == OWN_WARPS - 1;
  if (f0 >= total) {
    outlast(last);
    return;
  }
  const long long count = min(per, total - f0);

  // The sequence of the first step: the stretch, then within it.
  int b, len;
  long long base;  // steps of the sequences before b
  {
    int stretches = 0;
#pragma unroll
    for (int i = 0; i < NT; i += 32)
      stretches += __popc(__ballot_sync(0xffffffffu, sums[i + lane] * cols <= f0));
    b = (stretches - 1) * stretch;
    base = sums[stretches - 1];
    while (stretch > 1) {
      const int at_len = b + lane < p.B ? own_len(p.seqlens, b + lane, p.Lmax) : 0;
      const int n = own_steps(at_len);
      int upto = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, (base + upto) * cols > f0);
      if (hit != 0u || b + 32 >= p.B) {
        const int at = hit != 0u ? __ffs(hit) - 1 : 0;
        base += __shfl_sync(0xffffffffu, upto - n, at);
        b += at;
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
      b += 32;
    }
    len = stretch > 1 ? own_len(p.seqlens, b, p.Lmax) : lens[b];
  }
  // Cursor of the step that is looked up next.
  constexpr int CH = D / 8;      // 16-byte pieces per row
  constexpr int RP = 32 / CH;    // rows per copy instruction
  const int ch = lane % CH, rr = lane / CH;
  int n = own_steps(len);
  int col = static_cast<int>((f0 - base * cols) / n);
  int step = static_cast<int>(f0 - base * cols - static_cast<long long>(col) * n);
  // Partial of the first (sequence, head): the warps that hold its earlier steps
  // come before this one.  All others begin here.
  int slot = step == 0 ? 0 : static_cast<int>(wid - (base * cols + static_cast<long long>(col) * n) / per);
  long long looked = 0;   // steps looked up so far
  bool fresh = true;      // the next step begins a (sequence, head)
  const long long page_elems = (static_cast<long long>(p.Hkv) << p.log2_page) * D;
  const int page_mask = (1 << p.log2_page) - 1;
  auto head_offset = [&](int at) {  // of the lane's piece in row 0 of a page
    return (static_cast<long long>(at / p.tiles) << p.log2_page) * D + ch * 8;
  };
  long long head = head_offset(col);

  uint8_t* ring = smem + warp * L::WARP;
  const uint32_t ring_at = smem_u32(ring);
  int4* info = reinterpret_cast<int4*>(ring + STAGES * 2 * L::HALF);
  // The step after the last one issued: its page entries (lanes 0-15) and place.
  int page = -1, key0 = 0, at_b = 0, at_col = 0, at_len = 0, flags = 0;
  long long at_head = 0;
  bool pending = false;
  auto look_up = [&] {
    pending = looked < count;
    if (!pending) return;
    key0 = step * OWN_KEYS;
    at_b = b;
    at_col = col;
    at_len = len;
    at_head = head;
    const int key = key0 + (lane & 15);
    page = key < len ? p.table[b * p.table_stride + (key >> p.log2_page)] : -1;
    ++looked;
    flags = fresh ? 1 : 0;
    fresh = false;
    if (step + 1 == n) {
      fresh = true;
      flags |= 2 | 4;  // the last of its (sequence, head)
      if (looked < count) {
        step = 0;
        if (++col == cols) {
          col = 0;
          base += n;
          do {  // there is a further step, so a further sequence
            ++b;
            len = stretch > 1 ? own_len(p.seqlens, b, p.Lmax) : lens[b];
            n = own_steps(len);
          } while (n == 0);
        }
        head = head_offset(col);
      }
    } else {
      ++step;
      if (looked == count) flags |= 2;  // the last of it here
    }
  };
  int in = 0, issued = 0;  // byte offset of the stage that is filled next
  // where the lane's piece of row rr goes; row i RP + rr is i * 512 bytes on, its
  // swizzle own_swizzle(i RP) ^ own_swizzle(rr)
  const uint32_t to = ((ch ^ own_swizzle(rr)) << 4) + rr * (D * 2);
  const bool one_page = p.log2_page >= 4;  // 16 aligned keys lie in one page
  auto issue = [&] {
    if (pending) {
      const bool exists = key0 + (lane & 15) < at_len;
      if (exists && (page < 0 || page >= p.num_pages)) {
        record_error(1 /* FA_ERR_INVALID_ARG */);
        page = -1;
      }
      const unsigned live = __ballot_sync(0xffffffffu, exists && page >= 0) & 0xffffu;
      if (lane == 0)
        info[issued & (OWN_INFO - 1)] = make_int4(at_b, at_col, static_cast<int>(live), flags);
      ++issued;
      const uint32_t dst = ring_at + in + to;
      if (one_page && live == 0xffffu) {
        const long long off = __shfl_sync(0xffffffffu, page, 0) * page_elems + at_head +
                              ((key0 & page_mask) + rr) * D;
        const __nv_bfloat16 *k = p.kpages + off, *v = p.vpages + off;
#pragma unroll
        for (int i = 0; i < OWN_KEYS / RP; ++i) {
          const uint32_t at = (dst ^ (own_swizzle(i * RP) << 4)) + i * 512;
          copy16(at, k + i * 256, true);
          copy16(at + L::HALF, v + i * 256, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < OWN_KEYS / RP; ++i) {
          const int row = i * RP + rr;
          const int pg = __shfl_sync(0xffffffffu, page, row);
          const long long off =
              at_head + (pg >= 0 ? pg * page_elems + ((key0 + row) & page_mask) * D : 0);
          const uint32_t at = (dst ^ (own_swizzle(i * RP) << 4)) + i * 512;
          copy16(at, p.kpages + off, pg >= 0);
          copy16(at + L::HALF, p.vpages + off, pg >= 0);
        }
      }
    }
    copy_commit();
    in = in + 2 * L::HALF == STAGES * 2 * L::HALF ? 0 : in + 2 * L::HALF;
    look_up();
  };
  const int first_b = b, first_col = col;
  look_up();
#pragma unroll 1
  for (int i = 0; i < STAGES; ++i) issue();

  const int g = lane >> 2;
  const int c = lane & 3;
  // offsets in a stage of the lane's pieces of K row g (even and odd pieces 4 i +
  // c) and of V rows 2c and 2c + 1 (piece g)
  const uint32_t k_even = g * (D * 2) + ((c ^ own_swizzle(g)) << 4), k_odd = k_even ^ 64u;
  const uint32_t v_even = L::HALF + 2 * c * (D * 2) + ((g ^ own_swizzle(2 * c)) << 4);
  const uint32_t v_odd = L::HALF + (2 * c + 1) * (D * 2) + ((g ^ own_swizzle(2 * c + 1)) << 4);
  uint32_t qa[KS][2], qb[KS][2];
  float o[NH][MT][4];
  float m[2] = {-INFINITY, -INFINITY};  // heads g, g + 8 (log2 units, stale)
  float l[2] = {0.f, 0.f};              // this lane's share of their sums
  int out = 0;                          // byte offset of the stage that is read next
  auto load_q = [&](int qb_, int qcol) {
    const int h0 = qcol / p.tiles * p.r + qcol % p.tiles * 16;  // first query head
    const int heads = min(16, p.r - qcol % p.tiles * 16);
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(
        p.q + (static_cast<size_t>(qb_) * p.H + h0 + g) * D);
    const uint32_t* q1 = q0 + 4 * D;  // eight heads on
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int w0 = (32 * (s >> 1) + 8 * c + 4 * (s & 1)) >> 1;
      qa[s][0] = g < heads ? q0[w0] : 0u;
      qa[s][1] = g < heads ? q0[w0 + 1] : 0u;
      qb[s][0] = (HI && g + 8 < heads) ? q1[w0] : 0u;
      qb[s][1] = (HI && g + 8 < heads) ? q1[w0 + 1] : 0u;
    }
  };
  load_q(first_b, first_col);           // in flight beside the first keys
#pragma unroll 1
  for (long long done = 0; done < count; ++done) {
    copy_wait<STAGES - 1>();
    __syncwarp();
    const int4 at = info[done & (OWN_INFO - 1)];
    if (at.w & 1) {
      if (done > 0) load_q(at.x, at.y);
#pragma unroll
      for (int i = 0; i < NH; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    const uint8_t* stage = ring + out;
    // S = Q K^T for keys 0 .. 7 (half 0) and 8 .. 15 (half 1) of the step, each
    // in two accumulators (a single chain of products would wait for itself)
    float sc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float s2[4] = {0.f, 0.f, 0.f, 0.f};
      sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
      for (int i = 0; i < NKL; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(stage + ((i & 1) ? k_odd : k_even) +
                                                        t * 8 * D * 2 + (i >> 1) * 128);
        dec::mma_bf16_16816(sc[t], qa[2 * i][0], qb[2 * i][0], qa[2 * i][1], qb[2 * i][1], u.x, u.y);
        dec::mma_bf16_16816(s2, qa[2 * i + 1][0], qb[2 * i + 1][0], qa[2 * i + 1][1],
                            qb[2 * i + 1][1], u.z, u.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[t][e] += s2[e];
    }
    uint4 vr[4][NVL];  // V rows 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NVL; ++j)
        vr[i][j] = *reinterpret_cast<const uint4*>(stage + ((i & 1) ? v_odd : v_even) +
                                                   (i >> 1) * 8 * D * 2 + j * 128);

    uint32_t pb[2][2] = {{0u, 0u}, {0u, 0u}};  // P^T as the B operand: [head half][key half]
    float alpha[2] = {1.f, 1.f};
    bool grew = false;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
      float x[2][2];
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool live = (at.z >> (8 * t + 2 * c + j)) & 1;
          x[t][j] = live ? sc[t][2 * r + j] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, x[t][j]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[r], mx);
      if (m_new - m[r] > STALE_MAX) {  // also when m = -inf < m_new
        alpha[r] = ex2_approx(m[r] - m_new);
        l[r] *= alpha[r];
        m[r] = m_new;
        grew = true;
      }
      const float mref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = ex2_approx(x[t][0] - mref);
        const float p1 = ex2_approx(x[t][1] - mref);
        l[r] += p0 + p1;
        pb[r][t] = pack_bf16x2(p0, p1);
      }
    }
    if (__any_sync(0xffffffffu, grew)) {
      // column j of head tile i is head 8i + 2c + j, whose factor lane
      // 4 (2c + j) computed
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const float a0 = __shfl_sync(0xffffffffu, alpha[i], 8 * c);
        const float a1 = __shfl_sync(0xffffffffu, alpha[i], 8 * c + 4);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          o[i][t][0] *= a0;
          o[i][t][1] *= a1;
          o[i][t][2] *= a0;
          o[i][t][3] *= a1;
        }
      }
    }
    // bf16 pair (row i, row i + 1) at entry e of the lane's V list
    auto vpair = [&](int i, int e) -> uint32_t {
      const uint4 &ua = vr[i][e >> 3], &ub = vr[i + 1][e >> 3];
      const int w = (e & 7) >> 1;
      const uint32_t wa = w == 0 ? ua.x : w == 1 ? ua.y : w == 2 ? ua.z : ua.w;
      const uint32_t wb = w == 0 ? ub.x : w == 1 ? ub.y : w == 2 ? ub.z : ub.w;
      return __byte_perm(wa, wb, (e & 1) ? 0x7632u : 0x5410u);
    };
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint32_t a0 = vpair(0, t), a1 = vpair(0, t + MT), a2 = vpair(2, t), a3 = vpair(2, t + MT);
#pragma unroll
      for (int i = 0; i < NH; ++i) dec::mma_bf16_16816(o[i][t], a0, a1, a2, a3, pb[i][0], pb[i][1]);
    }
    __syncwarp();  // the stage has been read by every lane
    out = out + 2 * L::HALF == STAGES * 2 * L::HALF ? 0 : out + 2 * L::HALF;
    issue();

    if (at.w & 2) {  // the state of this (sequence, head)
      const int sb = at.x, scol = at.y;
      const int h0 = scol / p.tiles * p.r + scol % p.tiles * 16;
      const int heads = min(16, p.r - scol % p.tiles * 16);
      // Where it begins here, this warp says how many partials there are: one, or
      // all the warps up to that of its last step (the cursor still stands on it).
      if (slot == 0 && lane == 0)
        p.count[static_cast<size_t>(sb) * cols + scol] =
            (at.w & 4) != 0
                ? 1
                : static_cast<int>((base * cols + static_cast<long long>(col + 1) * n - 1) / per - wid) + 1;
      if (dbg_ok(slot >= 0 && slot < p.slots)) {
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          float sum = l[r];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (c == 0 && 8 * r + g < heads)
            p.pml[(static_cast<size_t>(sb) * p.H + h0 + 8 * r + g) * p.slots + slot] =
                make_float2(m[r], sum);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = 8 * r + 2 * c + j;
            if (h >= heads) continue;
            float* po = p.po + ((static_cast<size_t>(sb) * p.H + h0 + h) * p.slots + slot) * D + 8 * g;
            // entries 0 .. D/16-1 and D/16 .. D/8-1 of the lane's list, d = 64 (e / 8) + 8 g + e % 8
#pragma unroll
            for (int t = 0; t < MT; t += 4) {
              *reinterpret_cast<float4*>(po + t) =
                  make_float4(o[r][t][j], o[r][t + 1][j], o[r][t + 2][j], o[r][t + 3][j]);
              *reinterpret_cast<float4*>(po + (MT == 8 ? 64 : 4) + t) = make_float4(
                  o[r][t][2 + j], o[r][t + 1][2 + j], o[r][t + 2][2 + j], o[r][t + 3][2 + j]);
            }
          }
        }
      }
      slot = 0;
    }
  }
  outlast(last);
}

// Each row (b, h) by WPR warps, each lane with D/32 columns: merges the S prefix
// splits and the own partials.  A warp takes every WPR-th eight partials; lane i
// weighs partial i, and eight partials are read at once.  One warp a row when
// there are many rows, four when there are few (and so perhaps many splits).
constexpr int COMBINE_WARPS = 4;
template <int D, int WPR>
__global__ void __launch_bounds__(COMBINE_WARPS * 32)
    fa_shared_combine_kernel(const Params p, const int* __restrict__ seqlens, int Lmax, int slots,
                             int tiles, __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long bh = static_cast<long long>(blockIdx.x) * (COMBINE_WARPS / WPR) + warp / WPR;
  const int part = warp % WPR;
  dec::wait_for_splits();
  if (WPR == 1 && bh >= static_cast<long long>(p.B) * p.H) return;
  const int b = static_cast<int>(bh / p.H);
  const int S = p.choose ? *p.splits : p.S;
  int own = 0, own_keys = 0;
  if (slots > 0) {
    const int r = p.H / p.Hkv, h = static_cast<int>(bh - static_cast<long long>(b) * p.H);
    own = p.own_count[static_cast<size_t>(b) * p.Hkv * tiles + h / r * tiles + h % r / 16];
    own_keys = own_len(seqlens, b, Lmax);
  }
  const int length = entry_prefix(p, b);
  const int nt = (length + KEYS - 1) / KEYS;
  const int np = nt > 0 ? S : 0;
  const int n = np + (own_keys > 0 ? own : 0);  // nothing is written for no keys
  const float* base = p.own_po + static_cast<size_t>(bh) * slots * D;
  const float* pre = p.po + static_cast<size_t>(bh) * p.S * D;
  auto state = [&](int i) -> float2 {
    if (i >= n) return make_float2(-INFINITY, 0.f);
    if (i < np) {
      if (split_begin(i, S, nt) == split_begin(i + 1, S, nt))
        return make_float2(-INFINITY, 0.f);  // a split of no keys writes nothing
      return p.pml[static_cast<size_t>(bh) * p.S + i];
    }
    return p.own_pml[static_cast<size_t>(bh) * slots + (i - np)];
  };
  // Eight partials of this lane's columns, read whether or not they were written
  // (a split of no keys writes nothing; its weight is zero and it is passed over).
  auto read = [&](int i0, float (&v)[8][V]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = min(i0 + k, n - 1);
      const float* at = (i < np ? pre + static_cast<size_t>(i) * D
                                : base + static_cast<size_t>(i - np) * D) + lane * V;
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(at + e);
        v[k][e] = x.x;
        v[k][e + 1] = x.y;
      }
    }
  };
  float M = -INFINITY, l = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  // eights part, part + WPR, ..: four of them (32 partials) share a maximum
  for (int i0 = part * 8; i0 < n; i0 += 4 * WPR * 8) {
    float v[8][V];
    read(i0, v);  // in flight together with the states
    const float2 s = state(i0 + (lane >> 3) * (WPR * 8) + (lane & 7));
    float top = s.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    top = fmaxf(M, top);
    const float alpha = M == -INFINITY ? 0.f : ex2_approx(M - top);
    M = top;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= alpha;
    const float w = s.x == -INFINITY ? 0.f : ex2_approx(s.x - M);
    l += w * s.y;  // of this lane's partials; added over the lanes below
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int at = i0 + q * WPR * 8;
      if (at >= n) break;
      if (q > 0) read(at, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, q * 8 + k);  // zero past the last
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = wk != 0.f ? fmaf(wk, v[k][e], acc[e]) : acc[e];
      }
    }
  }
  // the lanes' l carry the same factors, so they add up
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if constexpr (WPR > 1) {  // one row a CTA: the warps' states, added by every warp
    __shared__ float shared_acc[WPR][D];
    __shared__ float2 shared_ml[WPR];
#pragma unroll
    for (int e = 0; e < V; ++e) shared_acc[part][lane * V + e] = acc[e];
    if (lane == 0) shared_ml[part] = make_float2(M, l);
    __syncthreads();
    if (part != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WPR; ++w) top = fmaxf(top, shared_ml[w].x);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float2 ml = shared_ml[w];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int e = 0; e < V; ++e)
        acc[e] = f != 0.f ? fmaf(f, shared_acc[w][lane * V + e], acc[e]) : acc[e];
    }
    M = top;
  }
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(o + bh * D + lane * V + e) =
        l != 0.f ? pack_bf16x2(acc[e] / l, acc[e + 1] / l) : 0u;
  if (lane == 0 && lse != nullptr)
    lse[bh] = l != 0.f ? (M + lg2_approx(l)) * 0.6931471805599453f : -INFINITY;
}

// A launch that may start before the one ahead of it in the stream has ended.
template <typename... A>
fa_status launch_early(void (*kern)(A...), dim3 grid, int threads, int smem, bool early,
                       cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

// Splits of the prefix.  A CTA costs its key tiles plus about three tiles'
// time to start and to write its rows; CTAs run one per SM, so the splits that
// minimise waves x (tiles per split + 3) are taken, by the capacity of the
// prefix tables and the fewest row tiles that the groups can have.  busy: CTAs;
// longest: key tiles one after the other.
int prefix_splits(int B, int H, int Hkv, int G, int tile_rows, long long cap, long long* busy,
                  long long* longest) {
  const long long nt = (cap + KEYS - 1) / KEYS;
  if (nt <= 0) return 0;
  const long long rows = static_cast<long long>(B) * (H / Hkv);
  long long tiles = (rows + tile_rows - 1) / tile_rows;
  if (tiles < G) tiles = G;
  tiles *= Hkv;
  long long best = 1, cost = -1;
  for (long long s = 1; s <= nt && s <= SM_COUNT; ++s) {
    const long long waves = (tiles * s + SM_COUNT - 1) / SM_COUNT;
    const long long c = waves * ((nt + s - 1) / s + 3);
    if (cost < 0 || c < cost) {
      cost = c;
      best = s;
    }
  }
  *busy = tiles * best;
  *longest = (*busy + SM_COUNT - 1) / SM_COUNT * ((nt + best - 1) / best);
  return static_cast<int>(best);
}

// Whether CTAs take 256 rows: once the groups have more than 128 on average.
// (32K shared keys, 512 rows a head: 128 rows per CTA read every key four times
// through L2.)
bool paired(int B, int H, int Hkv, int G) {
  return static_cast<long long>(B) * (H / Hkv) > static_cast<long long>(G) * ROWS;
}

struct Layout {
  int S;                   // prefix splits
  long long busy;          // prefix CTAs with work, at least
  long long longest;       // key tiles one after the other
  int slots, min_steps;    // own partials per row; steps a warp takes at least
  size_t pml, own, own_pml, count, splits, total;  // byte offsets behind the prefix partials
};

Layout layout(int B, int H, int Hkv, int G, long long cap, long long Lmax, int d) {
  Layout w = {};
  w.S = G > 0
            ? prefix_splits(B, H, Hkv, G, paired(B, H, Hkv, G) ? 2 * ROWS : ROWS, cap,
                             &w.busy, &w.longest)
             : 0;
  if (Lmax > 0) {
    // A warp's steps are few where that costs little: at most 63 partials a row,
    // however long the rows of the table are, and 64 MB of them in all (with
    // fewer than 9 a row the limit would begin to lengthen short sequences).
    const long long steps = (Lmax + OWN_KEYS - 1) / OWN_KEYS;
    const long long room = (64ll << 20) / (static_cast<long long>(B) * H * d * 4) - 1;
    const long long most = room < 8 ? 8 : (room < 62 ? room : 62);
    w.min_steps = static_cast<int>((steps + most - 1) / most);
    w.slots = static_cast<int>((steps + w.min_steps - 1) / w.min_steps) + 1;
  }
  const size_t bh = static_cast<size_t>(B) * H;
  w.pml = align_up(bh * w.S * d * sizeof(float), 256);
  w.own = w.pml + align_up(bh * w.S * sizeof(float2), 256);
  w.own_pml = w.own + align_up(bh * w.slots * d * sizeof(float), 256);
  w.count = w.own_pml + align_up(bh * w.slots * sizeof(float2), 256);
  // one count per (sequence, head tile): at most one per head
  w.splits = w.count + (w.slots > 0 ? align_up(bh * sizeof(int), 256) : 0);
  w.total = w.splits + (w.slots > 0 && w.S > 1 ? 256 : 0);
  return w;
}

// CTAs of the own keys: the resident ones, or fewer where these would leave warps
// without a step.
int own_grid(const OwnParams& p) {
  const long long steps = static_cast<long long>(p.B) * p.Hkv * p.tiles *
                          ((p.Lmax + OWN_KEYS - 1) / OWN_KEYS);
  const long long want = (steps + OWN_WARPS * p.min_steps - 1) / (OWN_WARPS * p.min_steps);
  const long long most = static_cast<long long>(OWN_CTAS) * rope::sm_count();
  return static_cast<int>(want < most ? want : most);
}

template <int D, bool HI>
fa_status launch_own(const OwnParams& p, bool early, cudaStream_t stream) {
  using L = OwnSmem<D>;
  static SmemOptIn opt_in;
  if (const fa_status st = opt_in.ensure(fa_shared_own_kernel<D, HI>, L::BYTES); st != FA_OK)
    return st;
  return launch_early(fa_shared_own_kernel<D, HI>, dim3(own_grid(p)), OWN_WARPS * 32, L::BYTES,
                      early, stream, p);
}

template <int D, bool PAIR>
fa_status launch_prefix(Params& p, bool early, cudaStream_t stream) {
  using L = Smem<D, PAIR>;
  constexpr int CTA_ROWS = PAIR ? 2 * ROWS : ROWS;
  static SmemOptIn opt_in;
  if (const fa_status st = opt_in.ensure(fa_shared_prefix_kernel<D, PAIR>, L::ALLOC); st != FA_OK)
    return st;
  // row tiles: each group may end inside one
  const long long tiles = (static_cast<long long>(p.B) * (p.H / p.Hkv) +
                           static_cast<long long>(p.G) * (CTA_ROWS - 1)) / CTA_ROWS;
  // one box per page, or 128 rows of it
  const int page = 1 << p.log2_page;
  const long long outer = static_cast<long long>(p.num_pages) * p.Hkv;
  p.box = page >= TMA_ROWS && outer <= 0x7fffffffLL ? (page < KEYS ? page : KEYS) : 0;
  CUtensorMap kmap = {}, vmap = {};
  if (p.box > 0) {
    fa_status st = make_tmap_bf16_3d(&kmap, p.kpages, D, page, outer, p.box);
    if (st == FA_OK) st = make_tmap_bf16_3d(&vmap, p.vpages, D, page, outer, p.box);
    if (st != FA_OK) return st;
  }
  main_kernel_begin(stream);
  const fa_status st = launch_early(
      fa_shared_prefix_kernel<D, PAIR>, dim3(p.S, static_cast<unsigned>(tiles), p.Hkv), THREADS,
      L::ALLOC, early, stream, (const CUtensorMap)kmap, (const CUtensorMap)vmap, (const Params)p);
  if (st != FA_OK) return st;
  main_kernel_end(stream);
  return FA_OK;
}

template <int D>
fa_status launch(Params& p, const int* table, long long stride, const int* seqlens, int own_pages,
                 __nv_bfloat16* o, float* lse, const Layout& w, char* ws, cudaStream_t stream) {
  p.po = reinterpret_cast<float*>(ws);
  p.pml = reinterpret_cast<float2*>(ws + w.pml);
  p.own_po = reinterpret_cast<float*>(ws + w.own);
  p.own_pml = reinterpret_cast<float2*>(ws + w.own_pml);
  p.own_count = reinterpret_cast<int*>(ws + w.count);
  const int Lmax = own_pages << p.log2_page;
  const bool own = w.slots > 0 && p.num_pages > 0;
  const bool prefix = w.S > 0 && p.num_pages > 0;
  const int r = p.H / p.Hkv, tiles = (r + 15) / 16;
  // The prefix goes first and the own keys' CTAs run on the SMs that it leaves, with
  // as many splits as suit both.  Where own keys are by far the larger part (tables
  // taken as half used), they go first on all SMs.  (128 sequences, 32 key/value
  // heads, 8192 shared and 230 own keys on average, ratio 2.8: 114.6, prefix first
  // 122.5; 64 sequences, 8 heads, 16384 and 1015, ratio 1.9: 77.8, prefix first 73.6.)
  p.S = prefix ? w.S : 0;
  if (!prefix) p.G = 0;
  const bool pair = paired(p.B, p.H, p.Hkv, p.G);
  const float own_us = 0.5f * p.B * Lmax * p.Hkv * (D * 4.f / 6.2e6f);
  const float prefix_us = w.longest * (pair ? 1.75f : 1.0f) + 10.f;
  const bool prefix_first = own_us < 2.25f * prefix_us;
  const OwnParams op{p.q, p.kpages, p.vpages, table, seqlens, p.own_po, p.own_pml, p.own_count,
                     stride, p.B, p.H, p.Hkv, r, tiles, Lmax, p.log2_page, p.num_pages, w.slots,
                     w.min_steps, p.scale_log2};
  // Nothing to choose where the own keys have half of the SMs in any case, or none.
  p.choose = own && prefix && prefix_first && p.S > 1 && w.busy * 2 > SM_COUNT &&
             w.busy <= static_cast<long long>(p.S) * SM_COUNT;
  if (p.choose) {
    p.splits = reinterpret_cast<int*>(ws + w.splits);
    p.own_lens = seqlens;
    p.Lmax = Lmax;
    p.units = static_cast<int>(w.busy / w.S);
    p.own_ctas = own_grid(op);
    p.key_kb = D * 4 * 1e-3f * p.Hkv / p.own_ctas;
  }
  auto run_prefix = [&](bool early) {
    return pair ? launch_prefix<D, true>(p, early, stream) : launch_prefix<D, false>(p, early, stream);
  };
  auto run_own = [&](bool early) {
    return r > 8 ? launch_own<D, true>(op, early, stream) : launch_own<D, false>(op, early, stream);
  };
  fa_status st = FA_OK;
  if (prefix && prefix_first) st = run_prefix(false);
  if (own && st == FA_OK) st = run_own(prefix && prefix_first);
  if (prefix && !prefix_first && st == FA_OK) st = run_prefix(own);
  if (st != FA_OK) return st;
  // One warp a row for many rows, four for few.  GPU time of the call, one and four:
  // 128 rows 16.6 and 14.2 us, 512 19.5 and 17.2, 1056 27.8 and 28.0, 1184 23.7 and 24.4,
  // 1536 26.2 and 28.7, 2048 26.7 and 30.2, 4096 38.2 and 46.7 (4096 shared keys, up to
  // 256 of their own; 1056: 8192).
  const int rows = p.B * p.H;
  if (rows > 8 * SM_COUNT)
    return launch_early(fa_shared_combine_kernel<D, 1>, dim3((rows - 1) / COMBINE_WARPS + 1),
                        COMBINE_WARPS * 32, 0, prefix || own, stream, (const Params)p, seqlens, Lmax,
                        own ? w.slots : 0, tiles, o, lse);
  return launch_early(fa_shared_combine_kernel<D, COMBINE_WARPS>, dim3(rows), COMBINE_WARPS * 32, 0,
                      prefix || own, stream, (const Params)p, seqlens, Lmax, own ? w.slots : 0, tiles,
                      o, lse);
}

fa_status check_sizes(int B, int H, int Hkv, int G, int page_size, int prefix_pages,
                      int pages_per_seq, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || G < 0 || prefix_pages < 0 || pages_per_seq < 0)
    return FA_ERR_INVALID_ARG;
  if (B > 65535 || H > 65535 || G > 65535 ||
      static_cast<long long>(B) * H > 0x7fffffffLL)
    return FA_ERR_INVALID_ARG;
  if (page_size < 1 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(prefix_pages) * page_size > 0x7fffffffLL - KEYS ||
      static_cast<long long>(pages_per_seq) * page_size > 0x7fffffffLL - KEYS)
    return FA_ERR_INVALID_ARG;
  // row tiles: each group may end inside one
  if ((static_cast<long long>(B) * (H / Hkv) + static_cast<long long>(G) * (ROWS - 1)) / ROWS > 65535)
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace shared

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_decode_shared_workspace_size(int B, int H, int Hkv, int G, int page_size,
                                       int prefix_pages, int pages_per_seq, int d) {
  if (shared::check_sizes(B, H, Hkv, G, page_size, prefix_pages, pages_per_seq, d) != FA_OK)
    return 0;
  return shared::layout(B, H, Hkv, G, static_cast<long long>(prefix_pages) * page_size,
                        static_cast<long long>(pages_per_seq) * page_size, d)
      .total;
}

fa_status fa_decode_shared(const void* q, const void* kpages, const void* vpages,
                           const int* prefix_table, long long prefix_stride,
                           const int* prefix_lens, const int* cu_batch, const int* block_table,
                           long long table_stride, const int* seqlens, void* o, float* lse, int B,
                           int H, int Hkv, int G, int page_size, int prefix_pages,
                           int pages_per_seq, int num_pages, int d, float scale, void* workspace,
                           size_t ws_bytes, fa_stream_t stream) {
  Range nvtx_range("fa_decode_shared");
  fa_status st = shared::check_sizes(B, H, Hkv, G, page_size, prefix_pages, pages_per_seq, d);
  if (st != FA_OK) return st;
  if (num_pages < 0 || prefix_stride < prefix_pages || table_stride < pages_per_seq ||
      table_stride > 0x7fffffff)
    return FA_ERR_INVALID_ARG;
  if (!q || !o || (G > 0 && !prefix_lens) || (G > 1 && !cu_batch) ||
      (G > 0 && prefix_pages > 0 && !prefix_table) ||
      (pages_per_seq > 0 && (!block_table || !seqlens)) ||
      (num_pages > 0 && (!kpages || !vpages)))
    return FA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(kpages, 16) || !al(vpages, 16) || !al(o, 16) || !al(lse, 4) ||
      !al(prefix_table, 4) || !al(prefix_lens, 4) || !al(cu_batch, 4) || !al(block_table, 4) ||
      !al(seqlens, 4))
    return FA_ERR_INVALID_ARG;
  if (!(scale == scale)) return FA_ERR_INVALID_ARG;
  const shared::Layout w =
      shared::layout(B, H, Hkv, G, static_cast<long long>(prefix_pages) * page_size,
                     static_cast<long long>(pages_per_seq) * page_size, d);
  if (w.total > 0 && (!workspace || !aligned256(workspace) || ws_bytes < w.total))
    return FA_ERR_WORKSPACE;
  if ((st = check_device()) != FA_OK) return st;
  shared::Params p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kpages = static_cast<const __nv_bfloat16*>(kpages);
  p.vpages = static_cast<const __nv_bfloat16*>(vpages);
  p.table = prefix_table;
  p.table_stride = prefix_stride;
  p.lens = prefix_lens;
  p.cu = cu_batch;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.G = G;
  p.pages = prefix_pages;
  p.num_pages = num_pages;
  while ((1 << p.log2_page) < page_size) ++p.log2_page;
  p.by_r = rope::Quotient(H / Hkv);
  p.scale_log2 = scale * 1.4426950408889634f;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (d == 128)
    return shared::launch<128>(p, block_table, table_stride, seqlens, pages_per_seq,
                               static_cast<__nv_bfloat16*>(o), lse, w, ws, s);
  return shared::launch<64>(p, block_table, table_stride, seqlens, pages_per_seq,
                            static_cast<__nv_bfloat16*>(o), lse, w, ws, s);
}

}  // extern "C"
