// fa_rope.cu - per-head norm of queries and keys with the position rotation in
// the same pass, its gradient, and the serving form that writes new keys and
// values into the pages of a cache.
//
// For a row x of d values (one token, one head), weight w and eps:
//   r = 1 / sqrt(mean(x^2) + eps),   y = x r w        (no weight: y = x)
//   the first R values of y are rotated in pairs (i, i + R/2), or (2i, 2i+1)
//   interleaved, by the angle a_i = position * inv_freq[i]:
//   o_1 = y_1 cos a - y_2 sin a,   o_2 = y_2 cos a + y_1 sin a.
// Backward, from x and g = dL/do (nothing is saved by the forward):
//   dy = the rotation of g by -a,   c = mean(w dy x r),
//   dx = r (w dy - x r c),          dw = sum over rows of dy x r.
//
// Every value is read once and written once and costs about ten flops, so the
// passes are bound by HBM, if the instructions are few enough.  d/16 lanes
// share a row and each holds both values of eight pairs (two 16-byte pieces of
// the row), so a pair is turned within its lane; products are packed f32x2.  (A
// first form with eight values per lane and the partners exchanged by
// shuffles issued 2.5 times the instructions and stood at 40% of the copy
// bandwidth.)  A group of lanes keeps one token and walks over its heads, so the
// rotation and the weight fold into four factors per pair that stay in registers:
//   out_1 = r (x_1 w_1 cos - x_2 w_2 sin),  out_2 = r (x_2 w_2 cos + x_1 w_1 sin).
// Angles are formed once per token (fa_angle.h).  A frequency is held as the fraction of a
// turn per position in 64-bit fixed point, so the product with a position wraps
// around whole turns by itself and positions of millions lose nothing; the sine
// and cosine of what is left are 32-bit series.  (With products in double
// precision and the library's sincospif the backward of 16K tokens took 82.5 us
// instead of 80.1.)
//
// The CTAs are resident and walk over the tokens.  Each thread fetches its own
// pieces of the rows ahead with 16-byte asynchronous copies into shared memory
// that only it reads, so the copies run on across rows, heads and tokens
// without a barrier and without registers.
// Sums are in 32 bits; the only rounding to bf16 is that of the outputs.
//
// Measured (three inputs in turn): forward of 8K tokens x 40 heads x 128, 168 MB,
// 34.3 us a call (31.5 in a graph; a copy of as many bytes 28.4), backward of 16K
// tokens x 32 heads, 403 MB, 75.6 to 76.5, 8.9K tokens into pages, 218 MB, 40.8.
#include <type_traits>

#include "fa_angle.h"
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

namespace rope {

constexpr int THREADS = 128;
constexpr int FWD_STAGES = 4;   // rows fetched ahead per group, forward
constexpr int BWD_STAGES = 4;   // backward (two inputs per row)
constexpr int FWD_CTAS = 4;     // resident CTAs per SM
constexpr int BWD_CTAS = 4;
constexpr int MAX_BWD_CTAS = 2048;

struct Rows {  // one tensor of rows: element strides of batch, head and token
  long long b, h, n;
};

// t / n for 0 <= t < 2^31: with s = ceil(log2 n) and m = ceil(2^(31+s) / n),
// m n exceeds 2^(31+s) by less than n <= 2^s, so t m / 2^(31+s) exceeds t / n by
// less than 1 / n and has the same whole part.
struct Quotient {
  unsigned m;
  int shift;
  Quotient(int n = 1) {
    int s = 0;
    while ((1ll << s) < n) ++s;
    shift = s - 1;
    m = s == 0 ? 0u : static_cast<unsigned>(((1ull << (31 + s)) + n - 1) / n);
  }
  __device__ __forceinline__ int operator()(int t) const {
    return shift < 0 ? t : static_cast<int>(__umulhi(static_cast<unsigned>(t), m) >> shift);
  }
};

struct Params {
  const __nv_bfloat16 *q, *k, *v;
  const __nv_bfloat16 *gq, *gk;  // backward: gradients of the outputs
  __nv_bfloat16 *qo, *ko;        // outputs (backward: gradients of q and k)
  Rows sq, sk, sv, sgq, sgk, sqo, sko;
  const void *wq, *wk;           // [d] float32 or bf16; null: no norm
  const int* pos;
  long long pos_b;
  const float* inv_freq;
  float* part;                   // backward: [CTAs][d] partial weight gradients
  int w_f32;
  int T, N, H, Hkv, R;           // T = B * N tokens
  Quotient batch;                // by N
  int gpt;                       // lane groups per token, a power of two
  int gpt_k, q_ctas;             // backward: gpt is q's; CTAs that take q, the others k
  float eps;
  // append: pages of a cache
  __nv_bfloat16 *kpages, *vpages;
  const int* table;              // [B][table_stride]
  const int* batch_idx;          // [T]; null: token t belongs to sequence t
  const int* slots;              // [T] positions in the cache; null: pos
  long long table_stride;
  int B, pages_per_seq, log2_page, num_pages;
};

__device__ __forceinline__ void fetch16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void fetch_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A weight into shared memory as 32-bit values (1 where there is none).
// Interleaved, the first values of a lane's eight pairs come before the second
// ones, as the lane holds them.
template <int D, bool INTER>
__device__ __forceinline__ void stage_weight(const void* w, int w_f32, float* dst) {
  for (int i = threadIdx.x; i < D; i += THREADS) {
    const int in = i & (D / 2 - 1);  // place in its half of the row
    const int at = INTER ? (in >> 3) * 16 + (i & 1) * 8 + i / (D / 2) * 4 + ((in & 7) >> 1) : i;
    dst[at] = w == nullptr ? 1.f
              : w_f32      ? static_cast<const float*>(w)[i]
                           : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
  }
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_make(v, v); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_split(v, a, b);
  return a + b;
}

// Where a lane's eight pairs stand in the row.  Neighbouring lanes hold
// neighbouring 16-byte pieces (pieces 32 bytes apart would ask for every 32-byte
// sector twice: 35.6 us instead of 27.6 for a backward of 7.3K tokens).
//   half split   pair i of the lane is (c0 + i, c0 + away + i), away = R / 2;
//   interleaved  pairs 0-3 are the piece at c0, pairs 4-7 the piece at c0 + D / 2.
// Behind the rotated part the "pairs" are any values, left unturned.
// FULL: the whole row is rotated (R = D), so the distance of the pieces is known.
template <int D, bool INTER, bool FULL>
struct Lane {
  static constexpr int LPR = D / 16;
  int c0;               // first element of the lane's first 16-byte piece
  int away;             // from the first piece to the second
  bool turned0, turned1;  // pairs 0-3 and 4-7 inside the rotated part
  __device__ __forceinline__ Lane(int lane, int R) {
    const int sub = lane % LPR;
    if (INTER) {
      c0 = sub * 8;
      away = D / 2;
      turned0 = c0 < R;
      turned1 = c0 + D / 2 < R;
    } else {
      turned0 = turned1 = sub * 16 < R;
      c0 = turned0 ? sub * 8 : R + (sub - R / 16) * 8;
      away = turned0 ? R / 2 : (D - R) / 2;
    }
  }
  // whether the two pairs of packed operand i are turned
  __device__ __forceinline__ bool rot(int i) const { return FULL || (i < 2 ? turned0 : turned1); }
  __device__ __forceinline__ int delta() const { return FULL || INTER ? D / 2 : away; }
};

// Eight consecutive 32-bit values from shared memory as four pairs.
__device__ __forceinline__ void eight(const float* p, uint64_t (&v)[4]) {
  const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(p);
  const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(p + 4);
  v[0] = lo.x;
  v[1] = lo.y;
  v[2] = hi.x;
  v[3] = hi.y;
}

// The first (a) and second (b) values of a lane's eight pairs, two pairs to a
// packed operand, from the lane's two pieces.
template <bool INTER>
__device__ __forceinline__ void unpack(const uint4& u, const uint4& v, uint64_t (&a)[4],
                                       uint64_t (&b)[4]) {
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      a[i] = f2_make(lo(w[2 * i]), lo(w[2 * i + 1]));
      b[i] = f2_make(hi(w[2 * i]), hi(w[2 * i + 1]));
    } else {
      a[i] = f2_make(lo(w[i]), hi(w[i]));
      b[i] = f2_make(lo(w[4 + i]), hi(w[4 + i]));
    }
  }
}

template <bool INTER>
__device__ __forceinline__ void pack(const uint64_t (&a)[4], const uint64_t (&b)[4], uint4& u,
                                     uint4& v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    f2_split(a[i], a0, a1);
    f2_split(b[i], b0, b1);
    if constexpr (INTER) {
      w[2 * i] = pack_bf16x2(a0, b0);
      w[2 * i + 1] = pack_bf16x2(a1, b1);
    } else {
      w[i] = pack_bf16x2(a0, a1);
      w[4 + i] = pack_bf16x2(b0, b1);
    }
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  v = make_uint4(w[4], w[5], w[6], w[7]);
}

// The lane's share of a weight staged in shared memory.
template <int D, bool INTER, bool FULL>
__device__ __forceinline__ void lane_weight(const Lane<D, INTER, FULL>& L, const float* w,
                                            uint64_t (&a)[4], uint64_t (&b)[4]) {
  eight(w + (INTER ? 2 * L.c0 : L.c0), a);
  eight(w + (INTER ? 2 * L.c0 + 8 : L.c0 + L.delta()), b);
}

// cos and sin of the lane's pairs, from the token's tables.
template <int D, bool INTER, bool FULL>
__device__ __forceinline__ void lane_angles(const Lane<D, INTER, FULL>& L, const float* cs,
                                            const float* sn, uint64_t (&c)[4], uint64_t (&s)[4]) {
  auto four = [](const float* p, bool turned, uint64_t& v0, uint64_t& v1, float none) {
    if (turned) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
      v0 = u.x;
      v1 = u.y;
    } else {
      v0 = v1 = f2_both(none);
    }
  };
  const int p0 = INTER ? L.c0 / 2 : L.c0, p1 = INTER ? p0 + D / 4 : p0 + 4;
  four(cs + p0, L.rot(0), c[0], c[1], 1.f);
  four(cs + p1, L.rot(2), c[2], c[3], 1.f);
  four(sn + p0, L.rot(0), s[0], s[1], 0.f);
  four(sn + p1, L.rot(2), s[2], s[3], 0.f);
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Shared memory: the pieces fetched ahead (conflict-free: piece-major, a
// thread's 16 bytes side by side), then the angles of the CTA's tokens, twice.
template <int STAGES, int PIECES>
struct Ahead {
  static_assert((STAGES & (STAGES - 1)) == 0, "the stage wraps by a mask");
  static constexpr int STEP = PIECES * THREADS * 16;
  static constexpr int BYTES = STAGES * STEP;
  unsigned char* own;
  int in = 0, out = 0;  // byte offsets of the stages that are filled and read next
  __device__ __forceinline__ explicit Ahead(unsigned char* smem) : own(smem + threadIdx.x * 16) {}
  __device__ __forceinline__ void put(int piece, const void* src) const {
    fetch16(own + in + piece * (THREADS * 16), src);
  }
  __device__ __forceinline__ void filled() {
    fetch_commit();
    in = (in + STEP) & (BYTES - 1);
  }
  __device__ __forceinline__ void wait() const { fetch_wait<STAGES - 1>(); }
  __device__ __forceinline__ uint4 get(int piece) const {
    return *reinterpret_cast<const uint4*>(own + out + piece * (THREADS * 16));
  }
  __device__ __forceinline__ void used() { out = (out + STEP) & (BYTES - 1); }
};

// Where a thread stands: group hg of the gpt groups that share token `slot` of
// a tile of `tokens` tokens.
template <int D>
struct Place {
  static constexpr int LPR = D / 16;
  static constexpr int GROUPS = THREADS / LPR;
  int gpt, tokens, slot, hg;
  __device__ __forceinline__ explicit Place(int gpt_) : gpt(gpt_) {
    const int group = threadIdx.x / LPR;
    tokens = GROUPS / gpt;
    slot = group / gpt;
    hg = group & (gpt - 1);
  }
  // The threads of a token: one warp or a part of it, or several warps.
  __device__ __forceinline__ void sync() const {
    if (gpt * LPR <= 32) __syncwarp();
    else __syncthreads();
  }
  // cos and sin of the token's angles, each of its threads some of them.
  __device__ __forceinline__ void angles(int pos, const unsigned long long* inv, int half,
                                         float* cs, float* sn) const {
    for (int a = hg * LPR + threadIdx.x % LPR; a < half; a += gpt * LPR)
      turn(pos, inv[a], cs[a], sn[a]);
  }
};

// One row: norm and rotation of the lane's pairs by the factors w cos, w sin.
template <int D, bool INTER, bool FULL>
__device__ __forceinline__ void row_fwd(const Lane<D, INTER, FULL>& L, const uint64_t (&ac)[4],
                                        const uint64_t (&bs)[4], const uint64_t (&bc)[4],
                                        const uint64_t (&as)[4], bool norm, float eps, uint4& x0,
                                        uint4& x1) {
  uint64_t a[4], b[4], oa[4], ob[4];
  unpack<INTER>(x0, x1, a, b);
  uint64_t ss = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ss = f2_fma(b[i], b[i], f2_fma(a[i], a[i], ss));
    oa[i] = f2_mul(a[i], ac[i]);
    ob[i] = f2_mul(b[i], bc[i]);
    if (L.rot(i)) {  // behind it the partner is not looked at (it may be inf)
      oa[i] = f2_fma(b[i], bs[i], oa[i]);
      ob[i] = f2_fma(a[i], as[i], ob[i]);
    }
  }
  if (norm) {
    const uint64_t r = f2_both(rsqrtf(row_sum<D>(f2_sum(ss)) * (1.f / D) + eps));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      oa[i] = f2_mul(oa[i], r);
      ob[i] = f2_mul(ob[i], r);
    }
  }
  pack<INTER>(oa, ob, x0, x1);
}

template <int D, bool INTER, bool FULL, bool APPEND>
__global__ void __launch_bounds__(THREADS, FWD_CTAS) fa_qk_norm_rope_kernel(const Params p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float weights[2][D];
  __shared__ unsigned long long inv[D / 2];
  const Place<D> at(p.gpt);
  const Lane<D, INTER, FULL> L(threadIdx.x & 31, p.R);
  Ahead<FWD_STAGES, 2> ahead(smem);
  const int half = p.R / 2;
  float* tables = reinterpret_cast<float*>(smem + ahead.BYTES) + at.slot * 2 * half;
  const int nq = (p.H + at.gpt - 1) / at.gpt, nk = (p.Hkv + at.gpt - 1) / at.gpt;
  const int tiles = (p.T + at.tokens - 1) / at.tokens;

  // The rows fetched next: the heads of q, of k (and of v) of the group's
  // token in tile `ft`.  Heads that do not exist are passed over (what the
  // stage holds then is computed with but not stored), tokens past the last
  // repeat it.
  int ft = blockIdx.x - gridDim.x, part = APPEND ? 2 : 1, fh = at.hg, fheads = 0;
  const __nv_bfloat16 *fp = nullptr, *fk = nullptr, *fv = nullptr;
  long long fstep = 0;
  auto fetch = [&] {
    if (fh - at.hg >= fheads) {  // the next part that has heads (the same for every thread)
      if (part == 0 && p.Hkv > 0) {
        part = 1;
        fp = fk;
        fstep = p.sk.h * at.gpt;
        fheads = p.Hkv;
      } else if (APPEND && part == 1) {
        part = 2;
        fp = fv;
        fstep = p.sv.h * at.gpt;
      } else {
        ft += gridDim.x;
        const int t = min(ft * at.tokens + at.slot, p.T - 1);
        const int b = p.batch(t), n = t - b * p.N;
        fk = p.k + b * p.sk.b + n * p.sk.n + at.hg * p.sk.h + L.c0;
        if constexpr (APPEND) fv = p.v + n * p.sv.n + at.hg * p.sv.h + L.c0;
        part = p.H > 0 ? 0 : 1;
        fp = part == 0 ? p.q + b * p.sq.b + n * p.sq.n + at.hg * p.sq.h + L.c0 : fk;
        fstep = (part == 0 ? p.sq.h : p.sk.h) * at.gpt;
        fheads = part == 0 ? p.H : p.Hkv;
      }
      fh = at.hg;
    }
    if (ft < tiles && fh < fheads) {
      ahead.put(0, fp);
      ahead.put(1, fp + L.delta());
    }
    fp += fstep;
    fh += at.gpt;
    ahead.filled();
  };
#pragma unroll 1
  for (int i = 0; i < FWD_STAGES; ++i) fetch();

  stage_weight<D, INTER>(p.wq, p.w_f32, weights[0]);
  stage_weight<D, INTER>(p.wk, p.w_f32, weights[1]);
  for (int i = threadIdx.x; i < half; i += THREADS) inv[i] = turns(p.inv_freq[i]);
  __syncthreads();
  int buf = 0;  // the tables alternate: one synchronisation a token
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int t = tile * at.tokens + at.slot;
    const int tt = min(t, p.T - 1);
    const int b = p.batch(tt), n = tt - b * p.N;
    bool live = t < p.T;
    int place = 0;
    if constexpr (APPEND) {
      place = (p.slots != nullptr ? p.slots : p.pos)[tt];
      live = live && place >= 0;          // a negative place marks padding
    }
    float* cs = tables + buf * at.tokens * 2 * half;
    float* sn = cs + half;
    at.angles(half > 0 ? p.pos[b * p.pos_b + n] : 0, inv, half, cs, sn);
    at.sync();
    uint64_t c[4], s[4];
    lane_angles(L, cs, sn, c, s);
    auto normed_rows = [&](const float* w, bool norm, int count, int heads, __nv_bfloat16* dst,
                           long long dh) {
      uint64_t ac[4], bs[4], bc[4], as[4], wa[4], wb[4];
      lane_weight(L, w, wa, wb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ac[i] = f2_mul(wa[i], c[i]);
        bc[i] = f2_mul(wb[i], c[i]);
        as[i] = f2_mul(wa[i], s[i]);
        bs[i] = f2_mul(f2_mul(wb[i], s[i]), f2_both(-1.f));
      }
      const int mine = live ? heads - at.hg : 0;  // rows to store: h < heads
      dst += at.hg * dh + L.c0;
      dh *= at.gpt;
#pragma unroll 1
      for (int i = 0; i < count; ++i, dst += dh) {
        ahead.wait();
        uint4 x0 = ahead.get(0), x1 = ahead.get(1);
        ahead.used();
        row_fwd(L, ac, bs, bc, as, norm, p.eps, x0, x1);
        fetch();
        if (i * at.gpt < mine) {
          *reinterpret_cast<uint4*>(dst) = x0;
          *reinterpret_cast<uint4*>(dst + L.delta()) = x1;
        }
      }
    };
    normed_rows(weights[0], p.wq != nullptr, nq, p.H, p.qo + b * p.sqo.b + n * p.sqo.n, p.sqo.h);
    __nv_bfloat16* ko;
    __nv_bfloat16* vo = nullptr;
    long long kh;
    if constexpr (!APPEND) {
      ko = p.ko + b * p.sko.b + n * p.sko.n;
      kh = p.sko.h;
    } else {
      // the token's row in the pages
      const int seq = p.batch_idx != nullptr ? p.batch_idx[tt] : tt;
      const int lp = place >> p.log2_page;
      int page = -1;
      if (live && seq >= 0 && seq < p.B && lp < p.pages_per_seq)
        page = p.table[seq * p.table_stride + lp];
      if (live && (page < 0 || page >= p.num_pages)) {
        record_error(1 /* FA_ERR_INVALID_ARG */);
        live = false;
      }
      const long long page_rows = 1ll << p.log2_page;
      kh = page_rows * D;
      const long long off = live ? page * (p.Hkv * kh) + (place & (page_rows - 1)) * D : 0;
      ko = p.kpages + off;
      vo = p.vpages + off;
    }
    normed_rows(weights[1], p.wk != nullptr, nk, p.Hkv, ko, kh);
    if constexpr (APPEND) {
      vo += at.hg * kh + L.c0;
#pragma unroll 1
      for (int i = 0; i < nk; ++i, vo += kh * at.gpt) {
        ahead.wait();
        const uint4 x0 = ahead.get(0), x1 = ahead.get(1);
        ahead.used();
        if (live && i * at.gpt < p.Hkv - at.hg) {
          *reinterpret_cast<uint4*>(vo) = x0;
          *reinterpret_cast<uint4*>(vo + L.delta()) = x1;
        }
        fetch();
      }
    }
  }
}

// The first q_ctas CTAs take q and the others k (one weight and one gradient of
// it in registers); each ends with one partial weight gradient, and a second
// kernel adds those in a fixed order (no atomics: the same call gives the same
// bits).
template <int D, bool INTER, bool FULL>
__global__ void __launch_bounds__(THREADS, BWD_CTAS) fa_qk_norm_rope_bwd_kernel(const Params p) {
  constexpr int LPR = D / 16;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float weight[D];
  __shared__ unsigned long long inv[D / 2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool is_q = static_cast<int>(blockIdx.x) < p.q_ctas;
  const int cta = is_q ? blockIdx.x : blockIdx.x - p.q_ctas;
  const int ctas = is_q ? p.q_ctas : gridDim.x - p.q_ctas;
  const int heads = is_q ? p.H : p.Hkv;
  const void* wp = is_q ? p.wq : p.wk;
  const bool norm = wp != nullptr;
  const __nv_bfloat16* src = is_q ? p.q : p.k;
  const __nv_bfloat16* grad = is_q ? p.gq : p.gk;
  __nv_bfloat16* dst = is_q ? p.qo : p.ko;
  const Rows sx = is_q ? p.sq : p.sk, sg = is_q ? p.sgq : p.sgk, so = is_q ? p.sqo : p.sko;
  const Place<D> at(is_q ? p.gpt : p.gpt_k);
  const Lane<D, INTER, FULL> L(threadIdx.x & 31, p.R);
  Ahead<BWD_STAGES, 4> ahead(smem);
  const int half = p.R / 2;
  float* tables = reinterpret_cast<float*>(smem + ahead.BYTES) + at.slot * 2 * half;
  const int rows = (heads + at.gpt - 1) / at.gpt;
  const int tiles = (p.T + at.tokens - 1) / at.tokens;

  int ft = cta - ctas, fh = heads + at.hg;
  const __nv_bfloat16 *fg = nullptr, *fx = nullptr;
  const long long gstep = sg.h * at.gpt, xstep = norm ? sx.h * at.gpt : 0;
  auto fetch = [&] {
    if (fh - at.hg >= heads) {  // the next token (the same for every thread)
      ft += ctas;
      const int t = min(ft * at.tokens + at.slot, p.T - 1);
      const int b = p.batch(t), n = t - b * p.N;
      fg = grad + b * sg.b + n * sg.n + at.hg * sg.h + L.c0;
      if (norm) fx = src + b * sx.b + n * sx.n + at.hg * sx.h + L.c0;
      fh = at.hg;
    }
    if (ft < tiles && fh < heads) {
      ahead.put(0, fg);
      ahead.put(1, fg + L.delta());
      if (norm) {
        ahead.put(2, fx);
        ahead.put(3, fx + L.delta());
      }
    }
    fg += gstep;
    fx += xstep;
    fh += at.gpt;
    ahead.filled();
  };
#pragma unroll 1
  for (int i = 0; i < BWD_STAGES; ++i) fetch();

  stage_weight<D, INTER>(wp, p.w_f32, weight);
  for (int i = threadIdx.x; i < half; i += THREADS) inv[i] = turns(p.inv_freq[i]);
  __syncthreads();
  uint64_t dwa[4], dwb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dwa[i] = dwb[i] = 0;
  int buf = 0;
  for (int tile = cta; tile < tiles; tile += ctas, buf ^= 1) {
    const int t = tile * at.tokens + at.slot;
    const int tt = min(t, p.T - 1);
    const int b = p.batch(tt), n = tt - b * p.N;
    __nv_bfloat16* dr = dst + b * so.b + n * so.n + at.hg * so.h + L.c0;
    const long long dstep = so.h * at.gpt;
    float* cs = tables + buf * at.tokens * 2 * half;
    float* sn = cs + half;
    at.angles(half > 0 ? p.pos[b * p.pos_b + n] : 0, inv, half, cs, sn);
    at.sync();
    uint64_t c[4], s[4];
    lane_angles(L, cs, sn, c, s);
    const int mine = t < p.T ? heads - at.hg : 0;
#pragma unroll 1
    for (int i = 0; i < rows; ++i, dr += dstep) {
      const bool real = i * at.gpt < mine;
      uint64_t ga[4], gb[4];
      ahead.wait();
      unpack<INTER>(ahead.get(0), ahead.get(1), ga, gb);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!L.rot(e)) continue;
        const uint64_t ga0 = ga[e];  // the rotation by -a
        ga[e] = f2_fma(gb[e], s[e], f2_mul(ga0, c[e]));
        gb[e] = f2_fma(f2_mul(ga0, f2_both(-1.f)), s[e], f2_mul(gb[e], c[e]));
      }
      if (norm) {
        uint64_t xa[4], xb[4], wa[4], wb[4];
        unpack<INTER>(ahead.get(2), ahead.get(3), xa, xb);
        lane_weight(L, weight, wa, wb);
        uint64_t ss = 0, sd = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ss = f2_fma(xb[e], xb[e], f2_fma(xa[e], xa[e], ss));
          wa[e] = f2_mul(wa[e], ga[e]);
          wb[e] = f2_mul(wb[e], gb[e]);
          sd = f2_fma(wb[e], xb[e], f2_fma(wa[e], xa[e], sd));
        }
        const float r = rsqrtf(row_sum<D>(f2_sum(ss)) * (1.f / D) + p.eps);
        const float k = r * r * row_sum<D>(f2_sum(sd)) * (1.f / D);  // mean(w dy x r) r
        const uint64_t r2 = f2_both(r), rk = f2_both(-r * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (real) {  // rows that do not exist add nothing
            dwa[e] = f2_fma(f2_mul(xa[e], r2), ga[e], dwa[e]);
            dwb[e] = f2_fma(f2_mul(xb[e], r2), gb[e], dwb[e]);
          }
          ga[e] = f2_fma(xa[e], rk, f2_mul(wa[e], r2));
          gb[e] = f2_fma(xb[e], rk, f2_mul(wb[e], r2));
        }
      }
      ahead.used();
      fetch();
      if (real) {
        uint4 y0, y1;
        pack<INTER>(ga, gb, y0, y1);
        *reinterpret_cast<uint4*>(dr) = y0;
        *reinterpret_cast<uint4*>(dr + L.delta()) = y1;
      }
    }
  }
  if (!norm) return;  // no weight: no sums
  // the lanes with the same values, within the warp and then over the warps
  __shared__ float red[THREADS / 32][D];
  const int lane = threadIdx.x & 31;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2_split(dwa[i], dw[0][2 * i], dw[0][2 * i + 1]);
    f2_split(dwb[i], dw[1][2 * i], dw[1][2 * i + 1]);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float& v = dw[e >> 3][e & 7];
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane < LPR) {
      const int i = L.c0 + (INTER ? ((e & 4) ? D / 2 : 0) + 2 * (e & 3) + (e >> 3)
                                  : (e < 8 ? 0 : L.delta()) + (e & 7));
      red[threadIdx.x >> 5][i] = v;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += THREADS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) v += red[w][i];
    p.part[static_cast<size_t>(blockIdx.x) * D + i] = v;
  }
}

// Adds the partials: q's from rows 0 .. nq-1, k's from rows nq .. n-1.  32
// columns per CTA, 32 partials at a time.  The kernel is resident while the partials
// are still being written, so they are no read-only memory (no __restrict__).
__global__ void __launch_bounds__(1024)
    fa_weight_grad_kernel(const float* part, int nq, int n, int d, float* dwq, float* dwk) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const bool is_q = static_cast<int>(blockIdx.x) < d / 32;
  float* dw = is_q ? dwq : dwk;
  if (dw == nullptr) return;
  const int c0 = (static_cast<int>(blockIdx.x) - (is_q ? 0 : d / 32)) * 32;
  float v = 0.f;
  const int end = is_q ? nq : n;
  for (int r = (is_q ? 0 : nq) + y; r < end; r += 16 * 32) {
    float u[16];  // in flight at once: as many partials as there are as a rule
#pragma unroll
    for (int i = 0; i < 16; ++i)
      u[i] = r + 32 * i < end ? part[static_cast<size_t>(r + 32 * i) * d + c0 + x] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += u[i];
  }
  red[y][x] = v;
  __syncthreads();
  v = red[x][y];  // column y of this CTA, partials x, x + 32, ...
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (x == 0) dw[c0 + y] = v;
}

// Lane groups per token.  A CTA takes `groups` / gpt tokens at a time; per token
// a group pays for the angles and factors, about four rows' time, and then for
// its rows; and neighbouring groups read neighbouring heads, which is worth half
// of the time against one group a token and a seventh against two (40 heads of
// 8K tokens: 34.4 us with 4 groups, 35.9 with 1; 9 heads: 14.1 and 11.9).  The gpt
// of the shortest total over the CTAs' rounds is taken.
int groups_per_token(int T, int H, int Hkv, int groups, int lanes, int ctas) {
  int best = 1;
  long long least = -1;
  for (int gpt = 1; gpt <= groups; gpt *= 2) {
    const int tokens = groups / gpt;
    const long long tiles = (static_cast<long long>(T) + tokens - 1) / tokens;
    const long long rounds = (tiles + ctas - 1) / ctas;
    // threads of a token in several warps meet at a CTA barrier
    const long long rows = 4 + (gpt * lanes > 32 ? 1 : 0) + (H + gpt - 1) / gpt + (Hkv + gpt - 1) / gpt;
    const long long cost = rounds * rows * (gpt == 1 ? 30 : gpt == 2 ? 23 : 20);
    if (least < 0 || cost < least) {
      least = cost;
      best = gpt;
    }
  }
  return best;
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <int D, bool INTER, bool FULL, bool APPEND>
fa_status launch_fwd(Params& p, cudaStream_t stream) {
  constexpr int GROUPS = THREADS / (D / 16);
  const int sms = sm_count();
  p.gpt = groups_per_token(p.T, p.H, APPEND ? 2 * p.Hkv : p.Hkv, GROUPS, D / 16, FWD_CTAS * sms);
  const int tokens = GROUPS / p.gpt;
  const int tiles = (p.T + tokens - 1) / tokens;
  const int grid = tiles < FWD_CTAS * sms ? tiles : FWD_CTAS * sms;
  // 16 KB of rows and at most 16 KB of angles, below the 48 KB that need no opt-in
  const int smem = Ahead<FWD_STAGES, 2>::BYTES + 2 * tokens * p.R * static_cast<int>(sizeof(float));
  fa_qk_norm_rope_kernel<D, INTER, FULL, APPEND><<<grid, THREADS, smem, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

template <int D, bool INTER, bool FULL>
fa_status launch_bwd(Params& p, float* dwq, float* dwk, cudaStream_t stream) {
  constexpr int GROUPS = THREADS / (D / 16);
  const int sms = sm_count();
  // CTAs of q and of k by their rows, as many as are resident at once
  const int most = BWD_CTAS * sms < MAX_BWD_CTAS ? BWD_CTAS * sms : MAX_BWD_CTAS;
  int nq = static_cast<int>(static_cast<long long>(most) * p.H / (p.H + p.Hkv));
  if (p.H > 0 && nq < 1) nq = 1;
  if (p.Hkv > 0 && nq > most - 1) nq = most - 1;
  int nk = most - nq;
  p.gpt = groups_per_token(p.T, p.H, 0, GROUPS, D / 16, nq > 0 ? nq : 1);
  p.gpt_k = groups_per_token(p.T, p.Hkv, 0, GROUPS, D / 16, nk > 0 ? nk : 1);
  const int tq = GROUPS / p.gpt, tk = GROUPS / p.gpt_k;
  if ((p.T + tq - 1) / tq < nq) nq = (p.T + tq - 1) / tq;
  if ((p.T + tk - 1) / tk < nk) nk = (p.T + tk - 1) / tk;
  if (p.H == 0) nq = 0;
  if (p.Hkv == 0) nk = 0;
  p.q_ctas = nq;
  const int smem = Ahead<BWD_STAGES, 4>::BYTES +
                   2 * (tq > tk ? tq : tk) * p.R * static_cast<int>(sizeof(float));
  static SmemOptIn opt_in;
  if (const fa_status st =
          opt_in.ensure(fa_qk_norm_rope_bwd_kernel<D, INTER, FULL>,
                        Ahead<BWD_STAGES, 4>::BYTES + 2 * GROUPS * D * static_cast<int>(sizeof(float)));
      st != FA_OK)
    return st;
  fa_qk_norm_rope_bwd_kernel<D, INTER, FULL><<<nq + nk, THREADS, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (dwq == nullptr && dwk == nullptr) return FA_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const float* part = p.part;
  if (cudaLaunchKernelEx(&cfg, fa_weight_grad_kernel, part, nq, nq + nk, D, dwq, dwk) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

// Calls launch with the head dimension, the pairing and whether the whole row is
// rotated as constants.
template <typename F>
fa_status by_shape(int d, int interleaved, bool full, F launch) {
  constexpr std::integral_constant<int, 64> d64;
  constexpr std::integral_constant<int, 128> d128;
  auto on_full = [&](auto D, auto I) {
    return full ? launch(D, I, std::true_type()) : launch(D, I, std::false_type());
  };
  auto on_pairs = [&](auto D) {
    return interleaved ? on_full(D, std::true_type()) : on_full(D, std::false_type());
  };
  return d == 128 ? on_pairs(d128) : on_pairs(d64);
}

}  // namespace rope

namespace {

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides of a tensor of rows: multiples of 8 elements (16-byte loads).
bool take(const long long* s, rope::Rows& r) {
  r = rope::Rows{s[0], s[1], s[2]};
  return ((s[0] | s[1] | s[2]) & 7) == 0;
}

// What the three entry points check alike.  rotary_dim is a multiple of 16,
// so that the two halves are whole 16-byte vectors.
fa_status check_rope(const void* q, const void* k, const void* wq, const void* wk,
                     int weight_type, const int* positions, const float* inv_freq, long long T,
                     int H, int Hkv, int d, int rotary_dim, int interleaved, float eps) {
  if (T < 0 || T > 0x7fffffff - 65535 || H < 0 || Hkv < 0 || H + Hkv < 1 || H > 65535 || Hkv > 65535)
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rotary_dim < 0 || rotary_dim > d) return FA_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (weight_type != FA_WEIGHT_BF16 && weight_type != FA_WEIGHT_F32) return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || !(eps >= 0.f)) return FA_ERR_INVALID_ARG;
  if (T > 0 && ((H > 0 && !q) || (Hkv > 0 && !k))) return FA_ERR_INVALID_ARG;
  if (T > 0 && rotary_dim > 0 && (!positions || !inv_freq)) return FA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(k, 16) || !al(wq, weight_type == FA_WEIGHT_F32 ? 4 : 2) ||
      !al(wk, weight_type == FA_WEIGHT_F32 ? 4 : 2) || !al(positions, 4) || !al(inv_freq, 4))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_qk_norm_rope(const void* q, const void* k, const void* q_weight,
                          const void* k_weight, int weight_type, const int* positions,
                          long long pos_batch_stride, const float* inv_freq, void* q_out,
                          void* k_out, const long long* strides, int B, int H, int Hkv, int N,
                          int d, int rotary_dim, int interleaved, float eps,
                          fa_stream_t stream) {
  Range nvtx_range("fa_qk_norm_rope");
  if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
  const long long T = static_cast<long long>(B) * N;
  fa_status st = check_rope(q, k, q_weight, k_weight, weight_type, positions, inv_freq, T, H, Hkv,
                            d, rotary_dim, interleaved, eps);
  if (st != FA_OK) return st;
  rope::Params p = {};
  if (T > 0 && ((H > 0 && !q_out) || (Hkv > 0 && !k_out))) return FA_ERR_INVALID_ARG;
  if (!al(q_out, 16) || !al(k_out, 16)) return FA_ERR_INVALID_ARG;
  if (!strides || (H > 0 && (!take(strides, p.sq) || !take(strides + 6, p.sqo))) ||
      (Hkv > 0 && (!take(strides + 3, p.sk) || !take(strides + 9, p.sko))))
    return FA_ERR_INVALID_ARG;
  if ((st = check_device()) != FA_OK) return st;
  if (T == 0) return FA_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.qo = static_cast<__nv_bfloat16*>(q_out);
  p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.wq = q_weight;
  p.wk = k_weight;
  p.w_f32 = weight_type == FA_WEIGHT_F32;
  p.pos = positions;
  p.pos_b = pos_batch_stride;
  p.inv_freq = inv_freq;
  p.T = static_cast<int>(T);
  p.N = N;
  p.batch = rope::Quotient(N);
  p.H = H;
  p.Hkv = Hkv;
  p.R = rotary_dim;
  p.eps = eps;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return rope::by_shape(d, interleaved, rotary_dim == d, [&](auto D, auto I, auto F) {
    return rope::launch_fwd<D(), I(), F(), false>(p, s);
  });
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return static_cast<size_t>(rope::MAX_BWD_CTAS) * d * sizeof(float);
}

fa_status fa_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out,
                              const void* dk_out, const void* q_weight, const void* k_weight,
                              int weight_type, const int* positions, long long pos_batch_stride,
                              const float* inv_freq, void* dq, void* dk, float* dq_weight,
                              float* dk_weight, const long long* strides, int B, int H, int Hkv, int N, int d,
                              int rotary_dim, int interleaved, float eps, void* workspace,
                              size_t ws_bytes, fa_stream_t stream) {
  Range nvtx_range("fa_qk_norm_rope_bwd");
  if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
  const long long T = static_cast<long long>(B) * N;
  // without a weight the gradient does not depend on the values
  const bool need_q = H > 0 && q_weight != nullptr, need_k = Hkv > 0 && k_weight != nullptr;
  fa_status st = check_rope(need_q ? q : dq_out, need_k ? k : dk_out, q_weight, k_weight,
                            weight_type, positions, inv_freq, T, H, Hkv, d, rotary_dim,
                            interleaved, eps);
  if (st != FA_OK) return st;
  rope::Params p = {};
  if (T > 0 && ((H > 0 && (!dq_out || !dq)) || (Hkv > 0 && (!dk_out || !dk))))
    return FA_ERR_INVALID_ARG;
  if ((need_q && !dq_weight) || (need_k && !dk_weight)) return FA_ERR_INVALID_ARG;
  if (!al(dq_out, 16) || !al(dk_out, 16) || !al(dq, 16) || !al(dk, 16) || !al(dq_weight, 4) ||
      !al(dk_weight, 4))
    return FA_ERR_INVALID_ARG;
  if (!strides || (H > 0 && (!take(strides + 6, p.sgq) || !take(strides + 12, p.sqo))) ||
      (Hkv > 0 && (!take(strides + 9, p.sgk) || !take(strides + 15, p.sko))) ||
      (need_q && !take(strides, p.sq)) || (need_k && !take(strides + 3, p.sk)))
    return FA_ERR_INVALID_ARG;
  if ((need_q || need_k) && (workspace == nullptr || !aligned256(workspace) ||
                             ws_bytes < fa_qk_norm_rope_bwd_workspace_size(d)))
    return FA_ERR_WORKSPACE;
  if ((st = check_device()) != FA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // sums over no rows
  if ((T == 0 || H == 0) && q_weight != nullptr && dq_weight != nullptr &&
      cudaMemsetAsync(dq_weight, 0, d * sizeof(float), s) != cudaSuccess)
    return FA_ERR_CUDA;
  if ((T == 0 || Hkv == 0) && k_weight != nullptr && dk_weight != nullptr &&
      cudaMemsetAsync(dk_weight, 0, d * sizeof(float), s) != cudaSuccess)
    return FA_ERR_CUDA;
  if (T == 0) return FA_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.gq = static_cast<const __nv_bfloat16*>(dq_out);
  p.gk = static_cast<const __nv_bfloat16*>(dk_out);
  p.qo = static_cast<__nv_bfloat16*>(dq);
  p.ko = static_cast<__nv_bfloat16*>(dk);
  p.wq = need_q ? q_weight : nullptr;
  p.wk = need_k ? k_weight : nullptr;
  p.w_f32 = weight_type == FA_WEIGHT_F32;
  p.pos = positions;
  p.pos_b = pos_batch_stride;
  p.inv_freq = inv_freq;
  p.part = (need_q || need_k) ? static_cast<float*>(workspace) : nullptr;
  p.T = static_cast<int>(T);
  p.N = N;
  p.batch = rope::Quotient(N);
  p.H = H;
  p.Hkv = Hkv;
  p.R = rotary_dim;
  p.eps = eps;
  float* dwq = need_q ? dq_weight : nullptr;
  float* dwk = need_k ? dk_weight : nullptr;
  return rope::by_shape(d, interleaved, rotary_dim == d, [&](auto D, auto I, auto F) {
    return rope::launch_bwd<D(), I(), F()>(p, dwq, dwk, s);
  });
}

fa_status fa_append_paged(const void* q, const void* k, const void* v, const void* q_weight,
                          const void* k_weight, int weight_type, const int* positions,
                          const int* cache_positions, const int* batch_idx,
                          const float* inv_freq, void* q_out, void* kpages, void* vpages,
                          const int* block_table, const long long* strides, int T, int H,
                          int Hkv, int d, int rotary_dim, int interleaved, float eps, int B, int page_size,
                          int pages_per_seq, long long table_stride, int num_pages,
                          fa_stream_t stream) {
  Range nvtx_range("fa_append_paged");
  fa_status st = check_rope(q, k, q_weight, k_weight, weight_type, positions, inv_freq, T, H, Hkv,
                            d, rotary_dim, interleaved, eps);
  if (st != FA_OK) return st;
  if (Hkv < 1 || B < 0 || pages_per_seq < 0 || num_pages < 0 || table_stride < pages_per_seq)
    return FA_ERR_INVALID_ARG;
  if (page_size < 1 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
    return FA_ERR_INVALID_ARG;
  if (batch_idx == nullptr && T > B) return FA_ERR_INVALID_ARG;  // token t is of sequence t
  if (positions == nullptr && cache_positions == nullptr && T > 0) return FA_ERR_INVALID_ARG;
  rope::Params p = {};
  if (T > 0 && (!v || (H > 0 && !q_out) || (B > 0 && pages_per_seq > 0 && !block_table) ||
                (num_pages > 0 && (!kpages || !vpages))))
    return FA_ERR_INVALID_ARG;
  if (!al(v, 16) || !al(q_out, 16) || !al(kpages, 16) || !al(vpages, 16) || !al(block_table, 4) ||
      !al(cache_positions, 4) || !al(batch_idx, 4))
    return FA_ERR_INVALID_ARG;
  if (!strides || (H > 0 && (!take(strides, p.sq) || !take(strides + 9, p.sqo))) ||
      !take(strides + 3, p.sk) || !take(strides + 6, p.sv))
    return FA_ERR_INVALID_ARG;
  if ((st = check_device()) != FA_OK) return st;
  if (T == 0) return FA_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.qo = static_cast<__nv_bfloat16*>(q_out);
  p.wq = q_weight;
  p.wk = k_weight;
  p.w_f32 = weight_type == FA_WEIGHT_F32;
  p.pos = positions;
  p.slots = cache_positions;
  p.batch_idx = batch_idx;
  p.inv_freq = inv_freq;
  p.kpages = static_cast<__nv_bfloat16*>(kpages);
  p.vpages = static_cast<__nv_bfloat16*>(vpages);
  p.table = block_table;
  p.table_stride = table_stride;
  p.B = pages_per_seq > 0 ? B : 0;  // a table of no pages has no entries to read
  p.pages_per_seq = pages_per_seq;
  p.num_pages = num_pages;
  while ((1 << p.log2_page) < page_size) ++p.log2_page;
  p.T = T;
  p.N = T;
  p.batch = rope::Quotient(T);
  p.H = H;
  p.Hkv = Hkv;
  p.R = rotary_dim;
  p.eps = eps;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return rope::by_shape(d, interleaved, rotary_dim == d, [&](auto D, auto I, auto F) {
    return rope::launch_fwd<D(), I(), F(), true>(p, s);
  });
}

}  // extern "C"
