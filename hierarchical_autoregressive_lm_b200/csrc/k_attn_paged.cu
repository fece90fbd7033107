// Attention of one new token per sequence over a caller's paged KV cache.
//
//   o[b, h] = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m),
//   s_t = scale log2(e) q[b, h] . k_t,  m = max_t s_t,
// over one pass of the positions: a warp carries m, the sum and the
// accumulator in fp32 and multiplies the two by 2^(m_old - m_new) when m
// grows.
//
// A unit is (sequence, key head, up to eight of its query heads); its
// positions are cut into steps.  The rows of a page are read once for all
// heads of a unit, so the kernel is bound by the cache's bytes; 4 flops per
// element and head are far below what the tensor cores take.
//
// Split.  Lengths live on the device, so the host cannot deal them out.
//  * Shares: one CTA per resident slot takes an equal share of all steps of
//    all units, in unit order, from a prefix sum over the lengths: every CTA
//    reads the same number of rows, however uneven the sequences.  A unit that
//    falls into several CTAs leaves parts (accumulator, maximum, sum), which a
//    second kernel joins in the order of the positions.
//  * Clusters: a thread-block cluster of one to eight CTAs divides each unit
//    and joins it through distributed shared memory: one launch, no scratch.
// Which one a call takes: see choose().
//
// Measured on a B200 (copy rate 6.54 TB/s): 64 sequences of 512 to 4096
// positions, 32 heads over 8 of 128, bf16 pages: 98 us for 605 MB (6.2 TB/s).
// Two of 131072, e4m3 pages: 93 us for 554 MB (6.0 TB/s; the tile's
// instructions and the products' latency take the rest).  fp32 pages, 1024
// units of 4096 positions of 64: 350 us for 2.15 GB.  One sequence of 257
// positions, 16 heads of 64: 4.7 us, the latency of length, table, rows and join.
#include <cmath>
#include <type_traits>

#include "kv_pages.cuh"
#include "launch.cuh"
#include "ptx_sm100.cuh"

namespace photon {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kHeadsMax = 8;  // query heads of a unit
constexpr int kClusterMax = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How a launch deals out its work; parts are [cta][2][kHeadsMax].
struct Plan {
  int chunks;      // units per key head
  int ctas;        // 0: a cluster per unit
  int cluster;
  int min_steps;   // least steps worth a CTA
  float* acc;      // [cta][2][kHeadsMax][D]
  float2* ml;      // maximum and sum
  int4* meta;      // [cta]: sequence, unit within it, last CTA of the unit that starts here (-1: none)
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
// c[16 x 8] += a[16 x 16] b[16 x 8] (tf32: a[16 x 8] b[8 x 8]), fp32 accumulators.
#define PHOTON_MMA(shape, type)                                                                                    \
  asm("mma.sync.aligned." shape ".row.col.f32." type "." type ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};" \
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  PHOTON_MMA("m16n8k16", "bf16");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  PHOTON_MMA("m16n8k16", "f16");
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  PHOTON_MMA("m16n8k8", "tf32");
}
#undef PHOTON_MMA

// An 8 x 8 matrix of 16-bit elements, two of row g in lane 4 g + t, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ld_shared(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// 2^x to 2^-22 of itself, 0 below fp32's normal numbers.
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Codes as fp16 pairs, exact: pairs of bytes 0, 1 and 2, 3, or (SKIP) 0, 2 and 1, 3.
template <bool SKIP>
__device__ __forceinline__ void codes_f16(uint32_t& lo, uint32_t& hi, uint32_t w, e4m3) {
  if (SKIP) w = __byte_perm(w, 0, 0x3120);
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
template <bool SKIP>
__device__ __forceinline__ void codes_f16(uint32_t& lo, uint32_t& hi, uint32_t w, int8_t) {
  // code + 128 in the low bits of 1024
  w ^= 0x80808080u;
  const uint32_t a = __byte_perm(w, 0x64646464u, SKIP ? 0x4240 : 0x4140), b = __byte_perm(w, 0x64646464u, SKIP ? 0x4341 : 0x4342);
  const __half2 c = __floats2half2_rn(1152.f, 1152.f);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), c), y = __hsub2(*reinterpret_cast<const __half2*>(&b), c);
  lo = *reinterpret_cast<const uint32_t*>(&x), hi = *reinterpret_cast<const uint32_t*>(&y);
}

// x as the sum of two tf32 numbers (the upper 19 bits of fp32): the first is
// rounded, what it leaves is at most 2^12 units of x's last place, so that
// cutting it to 11 bits drops one unit at most, and has either sign.  Rounding
// by an addition carries a NaN's bits anywhere, but the remainder of what is
// not finite is NaN, and stays one.  Numbers that would round to infinity are
// cut off; SMALL: there are none.  Of numbers below 2^-104 the second part is
// not a normal one, and may count as zero.
template <bool SMALL = false>
__device__ __forceinline__ void split_tf32(uint32_t& hi, uint32_t& lo, float x) {
  uint32_t up = __float_as_uint(x);
  if (SMALL || fabsf(x) < __uint_as_float(0x7f7ff000u)) up += 0x1000u;
  hi = up & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

// What a unit's positions are.
struct Unit {
  int b, kh, h0, nh;  // sequence, key head, first query head and their number (at most kHeadsMax)
  int first, len;     // positions first .. len - 1
  const int* table;
};

// Results of the warps over their positions, before they are joined.
template <int D>
struct Joint {
  static constexpr int kPitch = D + 8;
  float o[kWarps][kHeadsMax][kPitch];
  float m[kWarps][kHeadsMax], l[kWarps][kHeadsMax];
};

// The same of a whole CTA, for the other CTAs of its cluster.
template <int D>
struct Joined {
  float o[kHeadsMax][D];
  float m[kHeadsMax], l[kHeadsMax];
};

// A warp's tiles of TP positions on their way through a ring of cp.async
// stages of its own, so that no barrier stands between load and use.  The
// 16-byte chunks of a row are permuted so that the rows that one instruction
// reads fall into different banks.
template <typename C, int D>
struct Ring {
  static constexpr bool kNarrow = KvKind<C>::narrow;
  static constexpr int kRow = D * sizeof(C), kChunks = kRow / 16;
  // 8 KB of keys and values a stage, where 16 to 64 positions make that
  static constexpr int TP = kRow > 512 ? 8 : 4096 / kRow < 16 ? 16 : 4096 / kRow > 64 ? 64 : 4096 / kRow;
  static constexpr int kTile = TP * kRow;  // bytes of K (and of V)
  static constexpr int kMeta = 16 + (kNarrow ? 12 * TP : 0);  // which positions exist, their scales and log2 of V's
  // 18 KB a warp, two stages at least: three CTAs an SM hold more bytes in flight
  // and hide more of the products' latency than two with deeper rings (1024
  // units of 4096 positions: bf16 319 us against 330, e4m3 186 against 203)
  static constexpr int kFit = 18432 / (2 * kTile + kMeta);
  static constexpr int kStages = kFit < 2 ? 2 : kFit;
  static constexpr int kBytes = kWarps * kStages * (2 * kTile + kMeta);
  static constexpr int kCtas = 3 * kBytes <= 222 * 1024 ? 3 : 2 * kBytes <= 222 * 1024 ? 2 : 1;
  static constexpr int PL = (TP + 31) / 32;  // positions a lane looks up
  static_assert(kTile % 128 == 0, "tiles start at a bank line");

  // Byte of chunk c of row r of a tile: eight rows' chunks c lie in different banks.
  static __device__ __forceinline__ uint32_t place(int r, int c) {
    if constexpr (kChunks >= 8) {
      return r * kRow + ((c ^ (r & 7)) << 4);
    } else {
      constexpr int RPL = 8 / kChunks;  // rows of a 128-byte line
      const int line = r / RPL;
      return line * 128 + ((((r % RPL) * kChunks + c) ^ (line & (kChunks - 1))) << 4);
    }
  }
  // fp32 values are read by element, two neighbouring chunks of rows 0, 2, 4, 6 or 1, 3, 5, 7 at a time.
  static __device__ __forceinline__ uint32_t place_v(int r, int c) {
    if constexpr (sizeof(C) == 4)
      return r * kRow + ((c ^ (r & 6)) << 4);
    else
      return place(r, c);
  }

  const PagedAttnArgs& a;
  const Unit& u;
  int p0, p1, w, lane, mine;  // mine: tiles of this warp
  uint32_t tiles;
  unsigned char* metas;
  int* err;
  static constexpr uint32_t kNone = 0xffffffffu;

  __device__ __forceinline__ Ring(const PagedAttnArgs& a_, const Unit& u_, int p0_, int p1_, unsigned char* smem, int* err_)
      : a(a_), u(u_), p0(p0_), p1(p1_), w(threadIdx.x >> 5), lane(threadIdx.x & 31), err(err_) {
    const int all = (p1 - p0 + TP - 1) / TP;
    mine = all > w ? (all - w + kWarps - 1) / kWarps : 0;
    tiles = ptx::smem_u32(smem) + w * (kStages * 2 * kTile);
    metas = smem + kWarps * (kStages * 2 * kTile) + w * (kStages * kMeta);
  }
  __device__ __forceinline__ uint32_t keys(int i) const { return tiles + i % kStages * 2 * kTile; }
  __device__ __forceinline__ const unsigned* exists(int i) const { return reinterpret_cast<const unsigned*>(metas + i % kStages * kMeta); }
  __device__ __forceinline__ const float* scales(int i) const { return reinterpret_cast<const float*>(metas + i % kStages * kMeta + 16); }

  // Pages of the warp's tile i.
  __device__ __forceinline__ void look_up(int (&page)[PL], int i) const {
    const KvPoolArgs& p = a.pool;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const int pos = p0 + (w + i * kWarps) * TP + j * 32 + lane % TP;
      page[j] = -1;
      if (i < mine && pos < p1) {
        page[j] = u.table[div_fast((uint32_t)pos, p.div)];
        if ((uint32_t)page[j] >= (uint32_t)p.pages) report_error(err, DEV_BAD_PLACE), page[j] = -1;
      }
    }
  }
  // Starts its copies; rows that do not exist become zeros.  Rows are found by
  // 32-bit offsets in the pool's units.
  __device__ __forceinline__ void issue(const int (&page)[PL], int i) const {
    const KvPoolArgs& p = a.pool;
    if (i < mine) {
      uint32_t off[PL];
      unsigned char* const meta = metas + i % kStages * kMeta;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        const int pos = p0 + (w + i * kWarps) * TP + j * 32 + lane % TP;
        const int row = pos - (int)div_fast((uint32_t)pos, p.div) * p.rows;
        const bool ok = page[j] >= 0;
        off[j] = ok ? (uint32_t)page[j] * p.page_u + (uint32_t)row * p.row_u + (uint32_t)u.kh * p.head_u : kNone;
        const unsigned mask = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) reinterpret_cast<unsigned*>(meta)[j] = mask;
        if (kNarrow && lane < TP) {
          const long long s = ok ? page[j] * p.scale_page + row * p.scale_row + u.kh * p.scale_head : 0;
          const uint32_t dst = ptx::smem_u32(meta + 16) + (j * 32 + lane) * 4;
          cp4(dst, p.k_scale + s, ok);
          cp4(dst + 4 * TP, p.v_scale + s, ok);
        }
      }
      const uint32_t dst = keys(i);
#pragma unroll
      for (int n = 0; n < TP * kChunks / 32; ++n) {
        const int id = n * 32 + lane, r = id / kChunks, c = id % kChunks;
        // all lanes of one copy read rows of the same half of the tile
        const uint32_t o = __shfl_sync(0xffffffffu, off[n * 32 / kChunks / 32], r % 32);
        const bool ok = o != kNone;
        const unsigned long long at = (unsigned long long)(ok ? o : 0u) * p.unit + 16 * c;
        cp16(dst + place(r, c), (const char*)p.k + at, ok);
        cp16(dst + kTile + place_v(r, c), (const char*)p.v + at, ok);
      }
    }
    cp_commit();
  }
  // The first stages; `page` holds the pages of the tile after them.
  __device__ __forceinline__ void start(int (&page)[PL]) const {
    int pages[kStages - 1][PL];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) look_up(pages[i], i);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(pages[i], i);
    look_up(page, kStages - 1);
  }
  // Waits for tile i and starts the tile that takes the place of tile i - 1.
  __device__ __forceinline__ void next(int (&page)[PL], int i) const {
    cp_wait<kStages - 2>();
    __syncwarp();  // every lane's copies of tile i are here, and tile i - 1 has been read
    issue(page, i + kStages - 1);
    look_up(page, i + kStages);
  }
};

// Positions of a tile that do not exist get no weight: s[n][e] is position 8 n + 2 t + e.
template <int N>
__device__ __forceinline__ void mask_scores(float (&s)[N][2], const unsigned* exists, int t) {
#pragma unroll
  for (int j = 0; j < (N + 3) / 4; ++j) {
    const unsigned mask = exists[j];
    if (mask != 0xffffffffu) {
#pragma unroll
      for (int n = 0; n < (N < 4 ? N : 4); ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!((mask >> (8 * n + 2 * t + e)) & 1)) s[4 * j + n][e] = -INFINITY;
    }
  }
}
// The larger of m and a head's scores, which four lanes share.
template <int N>
__device__ __forceinline__ float largest_score(const float (&s)[N][2], float m) {
  float x = -INFINITY;
#pragma unroll
  for (int n = 0; n < N; ++n) x = fmaxf(x, fmaxf(s[n][0], s[n][1]));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  return fmaxf(x, m);
}
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }
template <int N>
__device__ __forceinline__ void scale_all(float (&o)[N][4], float f) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[n][k] *= f;
}

// Attention of a unit's query heads on the tensor cores (m16n8k16): positions
// or elements of the rows are the products' 16, the heads their 8 columns, so
// little is wasted on heads of one token each; the cache's bytes are the
// bound, not the products.  The weights' columns become the second product's
// right side by a transposition within the warp.  With up to four heads
// (PACK) the other four columns carry what rounding leaves behind, at no
// cost; else that takes products of its own.
//
// bf16 pages: q, K and V are multiplied as they are; a weight goes in as the
// sum of two bf16 numbers, off by 2^-17 (one would be off by 2^-9, as much as
// the result's own rounding).
//
// 8-bit pages: both products run in fp16, which holds every code exactly.  q
// is divided by the power of two at its largest element; what fp16 cannot
// hold of it follows times 2^24, so q keeps 22 bits.  A weight p times its
// scale v has fp32's range, which fp16 has not: p v 2^(15 - x), with a power of
// two 2^x above every p |v| so far (x = ceil(z) for the running maximum z of
// (s - m) + log2 |v|, in this order: s may be so large that log2 |v| would be
// lost in its rounding), is at most 2^15, and what fp16 cannot hold of it follows.
// Weights keep 22 bits down to 2^-17 of the largest, and steps of 2^-38 of the
// largest below that.
template <typename T_, typename C, int D, bool PACK>
struct Half {
  using T = T_;
  using R = Ring<C, D>;
  static constexpr bool kNarrow = KvKind<C>::narrow;
  static constexpr int kStep = kWarps * R::TP;
  static constexpr int kSmem = R::kBytes;
  static constexpr int kCtas = R::kCtas;
  static_assert(kSmem >= (int)(sizeof(Joint<D>) + sizeof(Joined<D>)), "the ring is reused for the join");
  static constexpr int KS = D / 16;        // k steps of the first product, row tiles of the second
  static constexpr int SUB = R::TP / 16;
  static constexpr int QP = kNarrow && !PACK ? 2 : 1;  // parts of q that take products of their own

  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kNarrow)
      mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
    else
      mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (kNarrow) return pack_f16(x, y);
    else return pack_bf16(x, y);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    if constexpr (kNarrow) return unpack_f16(w);
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }

  // q as the right side of the first product, in the order of k that the keys
  // come in: column g.  Returns what turns its products into log2 weights.
  static __device__ __forceinline__ float load_q(uint32_t (&qb)[KS][QP][2], const PagedAttnArgs& a, const Unit& u, int g, int t) {
    const int head = PACK ? g & 3 : g;
    const T* q = (const T*)a.q + u.b * a.q_seq + (u.h0 + head) * a.q_head;
    const bool there = head < u.nh;
    float to_log2 = a.scale * kLog2e;
    if constexpr (kNarrow) {
      float x[KS][4];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k][i] = there ? ld_f(q + 16 * k + 4 * t + i) : 0.f;
          top = max(top, __float_as_uint(x[k][i]) & 0x7fffffffu);
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = min(max(top >> 23, 1u), 253u);
      to_log2 *= __uint_as_float(e << 23);
      const float down = __uint_as_float((254 - e) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float y = x[k][2 * i] * down, z = x[k][2 * i + 1] * down;
          const uint32_t h = pack_f16(y, z);
          const float2 f = unpack_f16(h);
          const uint32_t l = pack_f16(isfinite(y) ? (y - f.x) * 0x1p24f : 0.f, isfinite(z) ? (z - f.y) * 0x1p24f : 0.f);
          qb[k][0][i] = PACK && g >= 4 ? l : h;
          if constexpr (QP == 2) qb[k][1][i] = l;
        }
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qb[k][0][i] = there ? pack_bf16(ld_f(q + 16 * k + 8 * i + 2 * t), ld_f(q + 16 * k + 8 * i + 2 * t + 1)) : 0u;
    }
    return to_log2;
  }

  // Largest over a column pair's positions, which eight lanes share, and x.
  static __device__ __forceinline__ void largest_of(float (&m)[2], const float (&s)[2 * SUB][2], const float (&x)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y = s[0][e];
#pragma unroll
      for (int n = 1; n < 2 * SUB; ++n) y = fmaxf(y, s[n][e]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
      m[e] = fmaxf(x[e], y);
    }
  }

  static __device__ __forceinline__ void run(const PagedAttnArgs& a, const Unit& u, int p0, int p1, unsigned char* smem,
                                             int* err) {
    const R ring(a, u, p0, p1, smem, err);
    const int w = ring.w, lane = ring.lane, g = lane >> 2, t = lane & 3;
    int page[R::PL];
    ring.start(page);
    uint32_t qb[KS][QP][2];
    float to_log2[2];  // of columns 2 t, 2 t + 1
    {
      const float f = load_q(qb, a, u, g, t);
#pragma unroll
      for (int e = 0; e < 2; ++e) to_log2[e] = __shfl_sync(0xffffffffu, f, (2 * t + e) * 4);
    }
    // columns 2 t, 2 t + 1: maxima of s and of s - m + log2 |v|, x, sums; rows g, g + 8 of the row tiles
    float m[2] = {-INFINITY, -INFINITY}, z[2] = {-INFINITY, -INFINITY}, x2[2] = {0.f, 0.f}, l[2] = {0.f, 0.f}, o[KS][4];
#pragma unroll
    for (int n = 0; n < KS; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

    for (int i = 0; i < ring.mine; ++i) {
      ring.next(page, i);
      const uint32_t kt = ring.keys(i), vt = kt + R::kTile;
      const float* const scales = ring.scales(i);
      if constexpr (kNarrow) {
        // log2 |v| of every position; below -120 it is raised, so that no power of two leaves fp32
#pragma unroll
        for (int j = 0; j < R::PL; ++j)
          if (j * 32 + lane < R::TP) {
            const float lv = __log2f(fabsf(scales[R::TP + j * 32 + lane]));
            const_cast<float*>(scales)[2 * R::TP + j * 32 + lane] = fminf(fmaxf(lv, -120.f), 128.f);
          }
        __syncwarp();
      }
      // scores s[n]: position 8 n + g
      float s[2 * SUB][2];
#pragma unroll
      for (int u16 = 0; u16 < SUB; ++u16) {
        float c[QP][4] = {};
        const int r = u16 * 16 + (lane & 15);
        if constexpr (kNarrow) {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t x[4];
            ldsm(x, kt + R::place(r, k + (lane >> 4)));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              uint32_t f[4];
              codes_f16<false>(f[0], f[2], x[2 * kk], C());
              codes_f16<false>(f[1], f[3], x[2 * kk + 1], C());
#pragma unroll
              for (int j = 0; j < QP; ++j) mma(c[j], f, qb[k + kk][j][0], qb[k + kk][j][1]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t x[4];
            ldsm(x, kt + R::place(r, 2 * k + (lane >> 4)));
            mma(c[0], x, qb[k][0][0], qb[k][0][1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float ks = kNarrow ? scales[u16 * 16 + 8 * j + g] : 1.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = c[0][2 * j + e];
            if constexpr (kNarrow && PACK) {  // the other part is two lanes away
              const float y = __shfl_xor_sync(0xffffffffu, x, 2);
              x = t < 2 ? x + y * 0x1p-24f : y + x * 0x1p-24f;
            }
            if constexpr (QP == 2) x += c[QP - 1][2 * j + e] * 0x1p-24f;
            s[2 * u16 + j][e] = x * (to_log2[e] * ks);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < R::PL; ++j) {
        const unsigned mask = ring.exists(i)[j];
        if (mask != 0xffffffffu) {
#pragma unroll
          for (int n = 4 * j; n < (2 * SUB < 4 * j + 4 ? 2 * SUB : 4 * j + 4); ++n)
            if (!((mask >> (8 * (n - 4 * j) + g)) & 1)) s[n][0] = s[n][1] = -INFINITY;
        }
      }

      float m_new[2], moved[2], grow[2], up[2];  // up: 2^(15 - x)
      bool grown = false;
      largest_of(m_new, s, m);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float base = finite_base(m_new[e]);
        moved[e] = m[e] - base;
#pragma unroll
        for (int n = 0; n < 2 * SUB; ++n) s[n][e] -= base;
      }
      if constexpr (kNarrow) {
        float sv[2 * SUB][2];
#pragma unroll
        for (int n = 0; n < 2 * SUB; ++n) {
          const float lv = scales[2 * R::TP + 8 * n + g];
          sv[n][0] = s[n][0] + lv, sv[n][1] = s[n][1] + lv;
        }
        const float old[2] = {z[0] + moved[0], z[1] + moved[1]};
        largest_of(z, sv, old);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float by = moved[e];
        if constexpr (kNarrow) {
          const float x = fminf(fmaxf(ceilf(z[e]), -110.f), 129.f);
          up[e] = __int_as_float((142 - (int)x) << 23);
          by += x2[e] - x;
          grown |= x != x2[e];
          x2[e] = x;
        }
        grown |= m_new[e] != m[e];
        grow[e] = pow2(by);
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int n = 0; n < KS; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[n][k] *= grow[k & 1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] *= pow2(moved[e]), m[e] = m_new[e];

      // the second product's right side: weights of positions 2 t, 2 t + 1 (+ 8) of 16, column g
      auto weights = [&](int u16, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = 2 * u16 + j;
          float x = pow2(s[n][0]), y = pow2(s[n][1]);
          l[0] += x, l[1] += y;
          if constexpr (kNarrow) {
            const float vs = scales[R::TP + 8 * n + g];
            x = x * vs * up[0], y = y * vs * up[1];
          }
          hi[j] = pack(x, y);
          const float2 f = unpack(hi[j]);
          lo[j] = pack(x - f.x, y - f.y);
          if constexpr (PACK) {
            hi[j] = transpose8(t < 2 ? hi[j] : lo[j]);
          } else {
            hi[j] = transpose8(hi[j]), lo[j] = transpose8(lo[j]);
          }
        }
      };
      // chunks c, c + 1 of 16 positions: two row tiles of 8-bit elements, one of bf16
      auto product = [&](int u16, int c, const uint32_t (&hi)[2], const uint32_t (&lo)[2], float (*acc)[4]) {
        const int r = u16 * 16 + (kNarrow ? lane & 15 : (lane & 7) + (lane >> 4) * 8);
        uint32_t x[4];
        ldsm_t(x, vt + R::place_v(r, c + (kNarrow ? lane >> 4 : (lane >> 3) & 1)));
        if constexpr (kNarrow) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // rows g: elements 2 g of the chunk, rows g + 8: 2 g + 1
            uint32_t f[4];
            codes_f16<true>(f[0], f[1], x[2 * j], C());
            codes_f16<true>(f[2], f[3], x[2 * j + 1], C());
            mma(acc[j], f, hi[0], hi[1]);
            if constexpr (!PACK) mma(acc[j], f, lo[0], lo[1]);
          }
        } else {
          mma(acc[0], x, hi[0], hi[1]);
          if constexpr (!PACK) mma(acc[0], x, lo[0], lo[1]);
        }
      };
      if constexpr (std::is_same<T, float>::value) {
        // the tensor cores cut a sum off where an addition rounds it; fp32
        // results get each tile's sum by an addition
        uint32_t hi[SUB][2], lo[SUB][2];
#pragma unroll
        for (int u16 = 0; u16 < SUB; ++u16) weights(u16, hi[u16], lo[u16]);
#pragma unroll
        for (int c = 0; c < R::kChunks; c += 2) {
          float sum[2][4] = {};
#pragma unroll
          for (int u16 = 0; u16 < SUB; ++u16) product(u16, c, hi[u16], lo[u16], sum);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[c + k / 4][k % 4] += sum[k / 4][k % 4];
        }
      } else {
#pragma unroll
        for (int u16 = 0; u16 < SUB; ++u16) {
          uint32_t hi[2], lo[2];
          weights(u16, hi, lo);
#pragma unroll
          for (int c = 0; c < R::kChunks; c += 2) product(u16, c, hi, lo, &o[kNarrow ? c : c / 2]);
        }
      }
    }
    cp_wait<0>();
    __syncthreads();  // all rings have been read
    Joint<D>& joint = *reinterpret_cast<Joint<D>*>(smem);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
      if (g == 0 && (!PACK || t < 2)) joint.m[w][2 * t + e] = m[e], joint.l[w][2 * t + e] = l[e];
      const float f = kNarrow ? __int_as_float((112 + (int)x2[e]) << 23) : 1.f;  // 2^(x - 15)
#pragma unroll
      for (int n = 0; n < KS; ++n) {
        float x = o[n][e] * f, y = o[n][2 + e] * f;
        if constexpr (PACK) x += __shfl_xor_sync(0xffffffffu, x, 2), y += __shfl_xor_sync(0xffffffffu, y, 2);
        if (PACK && t >= 2) continue;
        float* const row = joint.o[w][2 * t + e] + 16 * n;
        if constexpr (kNarrow)
          *reinterpret_cast<float2*>(row + 2 * g) = make_float2(x, y);
        else
          row[g] = x, row[g + 8] = y;
      }
    }
    __syncthreads();
  }
};

// fp32 pages: q, K, V and the weights each as the sum of two tf32 numbers
// (m16n8k8), 22 bits of them; the products of the two smaller parts come along.
// The tensor cores cut a sum off where an addition rounds it (8192 positions
// of one sign in one accumulator came out 2^-16 too small), so their sums stay
// short: a score's in three parts, an output's over a tile.
template <int D>
struct Full {
  using T = float;
  using R = Ring<float, D>;
  static constexpr int kStep = kWarps * R::TP;
  static constexpr int KS = D / 8, NT = D / 8, N8 = R::TP / 8;
  static constexpr int kSmem = R::kBytes + KS * 32 * 16;  // the ring, and q
  static constexpr int kCtas = 2 * kSmem <= 220 * 1024 ? 2 : 1;
  static_assert(R::kBytes >= (int)(sizeof(Joint<D>) + sizeof(Joined<D>)), "the ring is reused for the join");

  static __device__ __forceinline__ void run(const PagedAttnArgs& a, const Unit& u, int p0, int p1, unsigned char* smem,
                                             int* err) {
    const R ring(a, u, p0, p1, smem, err);
    const int w = ring.w, lane = ring.lane, g = lane >> 2, t = lane & 3;
    uint4* const qs = reinterpret_cast<uint4*>(smem + R::kBytes);  // [k step][lane]
    int page[R::PL];
    ring.start(page);
    {
      const float* q = (const float*)a.q + u.b * a.q_seq + (u.h0 + g) * a.q_head;
      for (int k = w; k < KS; k += kWarps) {
        uint4 x;
        split_tf32(x.x, x.y, g < u.nh ? q[8 * k + t] : 0.f);
        split_tf32(x.z, x.w, g < u.nh ? q[8 * k + 4 + t] : 0.f);
        qs[k * 32 + lane] = x;
      }
    }
    __syncthreads();
    const float to_log2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f, o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

    for (int i = 0; i < ring.mine; ++i) {
      ring.next(page, i);
      const uint32_t kt = ring.keys(i), vt = kt + R::kTile;
      float c[N8][3][4] = {};  // of even and odd k steps, and of the smaller parts
#pragma unroll
      for (int k = 0; k < KS; k += 2) {
        const uint4 q0 = qs[k * 32 + lane], q1 = qs[k * 32 + 32 + lane];
#pragma unroll
        for (int n = 0; n < N8; ++n) {
          uint32_t x[4], hi[4], lo[4];
          ldsm(x, kt + R::place(8 * n + (lane & 7), 2 * k + (lane >> 3)));
#pragma unroll
          for (int j = 0; j < 4; ++j) split_tf32(hi[j], lo[j], __uint_as_float(x[j]));
          mma_tf32(c[n][0], q0.x, q0.y, q0.z, q0.w, hi[0], hi[1]);
          mma_tf32(c[n][2], q0.x, q0.y, q0.z, q0.w, lo[0], lo[1]);
          mma_tf32(c[n][1], q1.x, q1.y, q1.z, q1.w, hi[2], hi[3]);
          mma_tf32(c[n][2], q1.x, q1.y, q1.z, q1.w, lo[2], lo[3]);
        }
      }
      float s[N8][2];
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          s[n][e] = (c[n][0][e] + c[n][1][e] + (c[n][2][e] + (c[n][0][2 + e] + c[n][1][2 + e] + c[n][2][2 + e]))) * to_log2;
      mask_scores(s, ring.exists(i), t);
      const float m_new = largest_score(s, m), base = finite_base(m_new);
      if (__any_sync(0xffffffffu, m_new != m)) {
        const float grow = pow2(m - base);
        l *= grow;
        scale_all(o, grow);
      }
      m = m_new;
      uint32_t pa[N8][4];  // k t of the product is position 2 t, k t + 4 is position 2 t + 1
#pragma unroll
      for (int n = 0; n < N8; ++n) {
        const float x = pow2(s[n][0] - base), y = pow2(s[n][1] - base);
        l += x + y;
        split_tf32<true>(pa[n][0], pa[n][1], x);  // at most 1
        split_tf32<true>(pa[n][2], pa[n][3], y);
      }
#pragma unroll
      for (int d = 0; d < NT; ++d) {
        float sum[4] = {};
#pragma unroll
        for (int n = 0; n < N8; ++n) {
          const int r = 8 * n + 2 * t, chunk = 2 * d + (g >> 2);
          uint32_t h0, h1, l0, l1;
          split_tf32(h0, l0, ld_shared(vt + R::place_v(r, chunk) + (g & 3) * 4));
          split_tf32(h1, l1, ld_shared(vt + R::place_v(r + 1, chunk) + (g & 3) * 4));
          mma_tf32(sum, pa[n][0], pa[n][1], pa[n][2], pa[n][3], h0, h1);
          mma_tf32(sum, pa[n][0], pa[n][1], pa[n][2], pa[n][3], l0, l1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) o[d][k] += sum[k];
      }
    }
    cp_wait<0>();
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    __syncthreads();  // all rings have been read
    Joint<D>& joint = *reinterpret_cast<Joint<D>*>(smem);
    if (t == 0) joint.m[w][g] = m, joint.l[w][g] = l;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float2*>(joint.o[w][g] + 8 * n + 2 * t) = make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
    __syncthreads();
  }
};

// ------------------------------------------------------------------ split

__device__ __forceinline__ int length_of(const PagedAttnArgs& a, int b, int* err) {
  const int cap = a.width * a.pool.rows, len = a.len[b];
  if (len >= 0 && len <= cap) return len;
  report_error(err, DEV_BAD_LENGTH);
  return len < 0 ? 0 : cap;
}
__device__ __forceinline__ int first_of(const PagedAttnArgs& a, int len) {
  return a.window > 0 ? max(0, len - a.window) : 0;
}
// Steps of each unit of sequence b; one without positions takes one, that writes its zeros.
template <int STEP>
__device__ __forceinline__ int steps_of(const PagedAttnArgs& a, int b) {
  const int len = length_of(a, b, nullptr);
  return max(1, (len - first_of(a, len) + STEP - 1) / STEP);
}

struct Share {
  int b, unit, step;    // where the CTA starts
  long long steps, all;  // how many steps it takes, and how many there are
  int ctas;              // that take any
};

// CTA c's share of all steps.
template <int STEP>
__device__ __forceinline__ void share_of(const PagedAttnArgs& a, const Plan& plan, int c, Share* out) {
  __shared__ long long warp_sum[kWarps];
  const int tid = threadIdx.x, per = (a.seqs + kThreads - 1) / kThreads;
  const int lo = min(a.seqs, tid * per), hi = min(a.seqs, lo + per);
  const int units = a.pool.heads * plan.chunks;
  long long mine = 0;
  for (int b = lo; b < hi; ++b) mine += steps_of<STEP>(a, b);
  mine *= units;
  long long upto = mine;  // inclusive prefix over the threads
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if ((tid & 31) >= o) upto += x;
  }
  if ((tid & 31) == 31) warp_sum[tid >> 5] = upto;
  __syncthreads();
  long long all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < tid >> 5) upto += warp_sum[w];
    all += warp_sum[w];
  }
  const long long worth = (all + plan.min_steps - 1) / plan.min_steps;
  const int ctas = (int)(worth < plan.ctas ? worth : plan.ctas);
  const long long x0 = c * all / ctas, x1 = (c + 1) * all / ctas;
  if (tid == 0) out->steps = c < ctas ? x1 - x0 : 0, out->all = all, out->ctas = ctas;
  if (c < ctas && x0 >= upto - mine && x0 < upto) {
    long long x = x0 - (upto - mine);
    for (int b = lo; b < hi; ++b) {
      const int n = steps_of<STEP>(a, b);
      if (x < (long long)n * units) {
        out->b = b, out->unit = (int)(x / n), out->step = (int)(x % n);
        break;
      }
      x -= (long long)n * units;
    }
  }
  __syncthreads();
}

// Element e of head h over n results of the same unit, as accumulator,
// maximum and sum; get(k, &m, &l, &o) fetches the k-th.
struct Total {
  float o, m, l;
};
template <int N, typename F>
__device__ __forceinline__ Total total_of(int n, F&& get) {
  float m[N], l[N], o[N];
  Total t = {0.f, -INFINITY, 0.f};
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k < n) get(k, m[k], l[k], o[k]), t.m = fmaxf(t.m, m[k]);
  const float base = t.m == -INFINITY ? 0.f : t.m;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k < n) {
      const float f = pow2(m[k] - base);
      t.l += f * l[k];
      t.o += f * o[k];
    }
  return t;
}
template <int D>
__device__ __forceinline__ Total over_warps(const Joint<D>& joint, int h, int e) {
  return total_of<kWarps>(kWarps, [&](int k, float& m, float& l, float& o) {
    m = joint.m[k][h], l = joint.l[k][h], o = joint.o[k][h][e];
  });
}
template <class E>
__device__ __forceinline__ void put(const PagedAttnArgs& a, const Unit& u, int h, int e, const Total& t) {
  st_f((typename E::T*)a.o + u.b * a.o_seq + (u.h0 + h) * a.o_head + e, t.l == 0.f ? 0.f : t.o / t.l);
  if (a.lse && e == 0)
    a.lse[(long long)u.b * a.q_heads + u.h0 + h] =
        t.l == 0.f ? -INFINITY : ((t.m == -INFINITY ? 0.f : t.m) + log2f(t.l)) * kLn2;
}
// The cluster's CTAs have attended to a unit: each writes its share of the outputs.
template <class E, int D>
__device__ __forceinline__ void put_cluster(const PagedAttnArgs& a, const Unit& u, const Joint<D>& joint, Joined<D>& mine,
                                            int rank, int ranks) {
  for (int i = threadIdx.x; i < u.nh * D; i += kThreads) {
    const int h = i / D, e = i % D;
    const Total t = over_warps(joint, h, e);
    mine.o[h][e] = t.o;
    if (e == 0) mine.m[h] = t.m, mine.l[h] = t.l;
  }
  ptx::cluster_sync();
  const uint32_t o = ptx::smem_u32(mine.o), m = ptx::smem_u32(mine.m), l = ptx::smem_u32(mine.l);
  for (int i = rank * kThreads + threadIdx.x; i < u.nh * D; i += ranks * kThreads) {
    const int h = i / D, e = i % D;
    put<E>(a, u, h, e, total_of<kClusterMax>(ranks, [&](int k, float& pm, float& pl, float& po) {
      pm = ptx::ld_shared_cluster_f32(ptx::map_shared_rank(m + 4 * h, k));
      pl = ptx::ld_shared_cluster_f32(ptx::map_shared_rank(l + 4 * h, k));
      po = ptx::ld_shared_cluster_f32(ptx::map_shared_rank(o + 4 * i, k));
    }));
  }
  ptx::cluster_sync();  // no CTA leaves while others read its shared memory
}

__device__ __forceinline__ Unit unit_of(const PagedAttnArgs& a, const Plan& plan, int b, int unit, int* err) {
  const int group = a.q_heads / a.pool.heads, skip = unit % plan.chunks * kHeadsMax;
  Unit u;
  u.b = b, u.kh = unit / plan.chunks;
  u.h0 = u.kh * group + skip, u.nh = min(kHeadsMax, group - skip);
  u.len = length_of(a, b, err), u.first = first_of(a, u.len);
  u.table = a.table + b * a.table_stride;
  return u;
}

template <class E, int D>
__global__ void __launch_bounds__(kThreads, E::kCtas) k_attn_paged(const PagedAttnArgs a, const Plan plan, int* err) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Share share;
  pdl_wait();
  pdl_trigger();
  const int units = a.pool.heads * plan.chunks;
  const Joint<D>& joint = *reinterpret_cast<const Joint<D>*>(smem);
  if (plan.ctas == 0) {
    const int at = blockIdx.x / plan.cluster, rank = blockIdx.x % plan.cluster;
    const Unit u = unit_of(a, plan, at / units, at % units, err);
    const int steps = (u.len - u.first + E::kStep - 1) / E::kStep;
    const int s0 = (int)((long long)steps * rank / plan.cluster), s1 = (int)((long long)steps * (rank + 1) / plan.cluster);
    E::run(a, u, u.first + s0 * E::kStep, min(u.len, u.first + s1 * E::kStep), smem, err);
    if (plan.cluster > 1) {
      put_cluster<E, D>(a, u, joint, *reinterpret_cast<Joined<D>*>(smem + sizeof(Joint<D>)), rank, plan.cluster);
    } else {
      for (int i = threadIdx.x; i < u.nh * D; i += kThreads) put<E>(a, u, i / D, i % D, over_warps(joint, i / D, i % D));
    }
    return;
  }
  share_of<E::kStep>(a, plan, blockIdx.x, &share);
  if (threadIdx.x == 0) plan.meta[blockIdx.x] = make_int4(0, 0, -1, 0);
  int b = share.b, unit = share.unit, step = share.step;
  for (long long left = share.steps; left > 0;) {
    const Unit u = unit_of(a, plan, b, unit, err);
    const int steps = max(1, (u.len - u.first + E::kStep - 1) / E::kStep);
    const int n = (int)min((long long)(steps - step), left);
    E::run(a, u, u.first + step * E::kStep, n < steps - step ? u.first + (step + n) * E::kStep : u.len, smem, err);
    const long long slot = blockIdx.x * 2ll + (step == 0);
    if (n < steps && step == 0 && threadIdx.x == 0) {
      // steps up to and with the unit's last: they end in the share that holds it
      const long long upto = (long long)blockIdx.x * share.all / share.ctas + (share.steps - left) + steps;
      plan.meta[blockIdx.x] = make_int4(b, unit, (int)((upto * share.ctas - 1) / share.all), 0);
    }
    for (int i = threadIdx.x; i < u.nh * D; i += kThreads) {
      const int h = i / D, e = i % D;
      const Total t = over_warps(joint, h, e);
      if (n == steps) {
        put<E>(a, u, h, e, t);
      } else {
        plan.acc[(slot * kHeadsMax + h) * D + e] = t.o;
        if (e == 0) plan.ml[slot * kHeadsMax + h] = make_float2(t.m, t.l);
      }
    }
    left -= n, step = 0;
    if (++unit == units) unit = 0, ++b;
    __syncthreads();
  }
}

// Joins the parts of the unit that starts in CTA blockIdx.x, head blockIdx.y.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const PagedAttnArgs a, const Plan plan) {
  constexpr int L = D / 4, G = kJoinThreads / L;  // lanes of a part, parts at a time
  __shared__ float red[kJoinThreads / 32];
  __shared__ float4 so[G][L];
  __shared__ float sl[G];
  // what follows starts after this kernel: the next call's shares would wait
  // here in the places of its blocks (two calls in a row 113 us each, not 101)
  pdl_wait();
  const int c = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, group = a.q_heads / a.pool.heads;
  const int4 meta = plan.meta[c];
  const int skip = meta.y % plan.chunks * kHeadsMax;
  if (meta.z < 0 || h >= min(kHeadsMax, group - skip)) return;
  const int parts = meta.z - c + 1;
  // the first part is slot 1 of CTA c, the others slot 0 of the CTAs after it
  auto slot = [&](int i) { return ((long long)(c + i) * 2 + (i == 0)) * kHeadsMax + h; };
  float mx = -INFINITY;
  for (int i = tid; i < parts; i += kJoinThreads) mx = fmaxf(mx, plan.ml[slot(i)].x);
  mx = warp_max(mx);
  if ((tid & 31) == 0) red[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, red[w]);
  const float base = mx == -INFINITY ? 0.f : mx;
  const int e = tid % L, g = tid / L;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int i = g; i < parts; i += G) {
    const float2 ml = plan.ml[slot(i)];
    const float4 x = reinterpret_cast<const float4*>(plan.acc + slot(i) * D)[e];
    const float f = pow2(ml.x - base);
    l += f * ml.y;
    o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
  }
  so[g][e] = o;
  if (e == 0) sl[g] = l;
  __syncthreads();
  if (tid < D) {
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) sum += sl[k], x += reinterpret_cast<const float*>(so[k])[tid];
    const int head = meta.y / plan.chunks * group + skip + h;
    st_f((T*)a.o + meta.x * a.o_seq + head * a.o_head + tid, sum == 0.f ? 0.f : x / sum);
    if (a.lse && tid == 0) a.lse[(long long)meta.x * a.q_heads + head] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
  }
}

// ------------------------------------------------------------------ host

// Clusters of 2^log2 CTAs of k_attn_paged<E, D> that the current device holds at once.
template <class E, int D>
int resident(int log2) {
  static PerDevice cache[4];
  return cache[log2].get([=] {
    cudaFuncSetAttribute(k_attn_paged<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, E::kSmem);
    int n = 0;
    if (log2 == 0) {
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_attn_paged<E, D>, kThreads, E::kSmem);
      n *= device_sm_count();
    } else {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 1 << log2;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.gridDim = dim3(1 << log2), cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = E::kSmem;
      cfg.attrs = &attr, cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, k_attn_paged<E, D>, &cfg) != cudaSuccess) n = 0, cudaGetLastError();
    }
    return n > 0 ? n : log2 == 0 ? 1 : 0;
  });
}

constexpr int kMinSteps = 2;   // of a share
constexpr int kJoinSteps = 8;  // what shares cost beyond their steps: the prefix sum, the parts, the join

// Clusters are as large as one wave of them allows.  They win while their
// longest CTA takes few steps, shares where every slot has to read (bf16
// pages, heads of 128, us by clusters and by shares: 8 units of 1024
// positions 5.5 and 8.7, of 8192 15.4 and 15.1; 32 of 4096 13.0 and 16.4; 512
// of 512 31 and 33, of 4096 191 and 167).  A step reads about 32 KB whatever
// the type, so one constant serves them all.  `steps` are those of the table's
// width or the window, all that the host knows of the lengths: shorter ones
// behind a wide table take shares where clusters would win (8 units of 1024
// behind 16384 8.8 us, 128 units 16.4 where clusters take 12.3).
// Sets plan.cluster, and plan.ctas where shares are better.
template <class E, int D>
void choose(Plan& plan, long long units, long long steps) {
  int log2 = 0;
  while (log2 < 3 && (2 << log2) <= steps && units <= resident<E, D>(log2 + 1)) ++log2;
  const int slots = resident<E, D>(0);
  plan.cluster = 1 << log2;
  const long long waves = (units + slots - 1) / slots;
  const long long alone = (log2 ? 1 : waves) * ((steps + plan.cluster - 1) / plan.cluster);
  const long long shared = (units * steps + slots - 1) / slots + kJoinSteps;
  if (alone > shared) plan.ctas = (int)(units * steps < slots ? units * steps : slots);
}

template <class E, int D>
cudaError_t attn_e(const PagedAttnArgs& a, int* err, cudaStream_t s, size_t* need) {
  const int group = a.q_heads / a.pool.heads;
  Plan plan = {};
  plan.chunks = (group + kHeadsMax - 1) / kHeadsMax;
  plan.min_steps = kMinSteps;
  const long long units = (long long)a.seqs * a.pool.heads * plan.chunks;
  long long most = (long long)a.width * a.pool.rows;  // positions of a unit
  if (a.window > 0 && a.window < most) most = a.window;
  choose<E, D>(plan, units, (most + E::kStep - 1) / E::kStep);
  if (plan.ctas == 0) {
    // CTAs that start while a predecessor's last blocks still run fill the SMs
    // unevenly: only a grid that leaves SMs free starts early (us early and not:
    // 128 units of 2048 positions in e4m3 20.8 and 17.1, 8 of 1024 in bf16 5.6
    // and 5.9)
    const long long grid = units * plan.cluster;
    launch_kernel_cluster(k_attn_paged<E, D>, (unsigned)grid, kThreads, E::kSmem, s, plan.cluster,
                          grid <= device_sm_count(), a, plan, err);
    return cudaGetLastError();
  }
  const size_t parts = (size_t)plan.ctas * 2 * kHeadsMax;
  const size_t bytes = parts * (D * sizeof(float) + sizeof(float2)) + plan.ctas * sizeof(int4);
  float* scratch = (float*)a.scratch;
  cudaError_t e = cudaSuccess;
  if (a.scratch_bytes == 0) {
    e = scratch_malloc((void**)&scratch, bytes, s);
    if (e != cudaSuccess) return e;
  } else if (a.scratch_bytes < (long long)bytes) {
    *need = bytes;
    return cudaSuccess;
  }
  plan.acc = scratch;
  plan.ml = (float2*)(scratch + parts * D);
  plan.meta = (int4*)(plan.ml + parts);
  launch_kernel(k_attn_paged<E, D>, (unsigned)plan.ctas, kThreads, E::kSmem, s, a, plan, err);
  launch_kernel(k_attn_join<typename E::T, D>, dim3(plan.ctas, group < kHeadsMax ? group : kHeadsMax), kJoinThreads, 0, s, a, plan);
  e = cudaGetLastError();
  if (a.scratch_bytes == 0) {
    const cudaError_t f = cudaFreeAsync(scratch, s);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

template <typename T, typename C, int D>
cudaError_t attn_h(const PagedAttnArgs& a, int* err, cudaStream_t s, size_t* need) {
  return a.q_heads / a.pool.heads <= 4 ? attn_e<Half<T, C, D, true>, D>(a, err, s, need) : attn_e<Half<T, C, D, false>, D>(a, err, s, need);
}
template <typename C, int D>
cudaError_t attn_d(int dt, const PagedAttnArgs& a, int* err, cudaStream_t s, size_t* need) {
  if constexpr (std::is_same<C, float>::value) {
    return attn_e<Full<D>, D>(a, err, s, need);
  } else {
    if constexpr (KvKind<C>::narrow)
      if (dt == DT_F32) return attn_h<float, C, D>(a, err, s, need);
    return attn_h<bf16, C, D>(a, err, s, need);
  }
}

template <typename C>
cudaError_t attn_c(int dt, const PagedAttnArgs& a, int* err, cudaStream_t s, size_t* need) {
  switch (a.pool.dh) {
    case 32: return attn_d<C, 32>(dt, a, err, s, need);
    case 64: return attn_d<C, 64>(dt, a, err, s, need);
    case 128: return attn_d<C, 128>(dt, a, err, s, need);
    default: return attn_d<C, 256>(dt, a, err, s, need);
  }
}

}  // namespace

cudaError_t launch_attn_paged(int dt, const PagedAttnArgs& a, int* err, cudaStream_t s, size_t* need) {
  switch (a.pool.kind) {
    case 0: return attn_c<float>(dt, a, err, s, need);
    case 1: return attn_c<bf16>(dt, a, err, s, need);
    case 2: return attn_c<e4m3>(dt, a, err, s, need);
    default: return attn_c<int8_t>(dt, a, err, s, need);
  }
}

}  // namespace photon
