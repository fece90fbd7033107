// Rotary positions, and the write and read of a caller's paged KV cache.
//
// All three move rows once and are bound by memory.  A block takes a few
// tokens; it finds their places and the sines and cosines of their positions
// once, in shared memory, while the first rows are on their way, and then
// walks over (token, head, part of the row) with a thread on 16 elements:
// two vectors of eight that hold both elements of every pair, so that a
// rotation needs no other thread's data and may run in place.
//
// Measured on a B200 (copy rate 6.54 TB/s): rotation of 8191 tokens, 40 heads
// of 128, bf16: 27.1 us for 168 MB; 32255 tokens, 8 heads of 128, bf16 into
// int8 pages: 38.7 us for 201 MB, as much bound by the instructions that
// narrow 16 elements (about 200 a warp) as by bytes; 65536 tokens out of e4m3
// pages: 64.6 us for 408 MB; 64 tokens, 32 heads of 64: 1.5 us.
//
// Angles.  A pair turns by pos * f turns, f a 64-bit binary fraction.  The
// product modulo 2^64 drops whole turns without rounding; its upper 32 bits,
// as a signed number of half-turns in [-1, 1), go to sincospif, whose
// argument is then off by at most 2^-25 half-turns, and by what f was off times
// the position (2^-28 half-turns at the last one; fp32 pos * f would be off by
// whole radians near a million).
#include "kv_pages.cuh"
#include "launch.cuh"

namespace photon {

namespace {

// Small blocks: a block's rows wait for its places and angles, and the more
// blocks an SM holds the less that shows (rotation of 168 MB, 64 tokens into
// e4m3: 27.1 and 2.6 us with 128 threads, 28.0 and 2.9 with 256, 31.4 and 3.5
// with 512).
constexpr int kThreads = 128;
constexpr int kBlocks = 8;                    // an SM holds of them
constexpr int kTokensMax = 256;               // of a block
constexpr int kAnglesMax = 16 * kThreads;     // sines and cosines of a block: one token for every row it takes at a time

__device__ __forceinline__ void turn(unsigned long long freq, int pos, float scale, float* s, float* c) {
  const int half_turns = (int)(((unsigned long long)(long long)pos * freq) >> 32);
  sincospif((float)half_turns * 0x1p-31f, s, c);
  *s *= scale;
  *c *= scale;
}

// The split of one tensor's rows [tokens][heads].  `chunks` threads share a
// row, always the same part of it; a block's kThreads / chunks groups of them
// take `hp` heads of `tp` tokens at a time, so that a thread stays with one
// head and its addresses move by constants.  `parts` blocks share a token's
// heads; a block takes `tokens` tokens.
struct Split {
  int heads, chunks, hp, tp, parts, tokens, blocks;
  FastDiv by_chunks, by_hp, by_half, by_parts;
};

// work: threads' rows in the whole launch.
Split split_rows(int n, int heads, int chunks, int rot, long long work) {
  Split s = {};
  const int groups = kThreads / chunks;
  s.heads = heads, s.chunks = chunks;
  // as few idle groups as up to four more blocks a token allow
  const int least = (heads + groups - 1) / groups;
  long long best = -1;
  for (int parts = least; parts <= least + 4; ++parts) {
    const int hp = (heads + parts - 1) / parts, tp = groups / hp;
    const long long busy = (1ll << 20) * heads * tp / ((long long)parts * groups);
    if (busy > best) best = busy, s.parts = parts, s.hp = hp, s.tp = tp;
  }
  // up to four rows a thread, which share the block's angles and keep bytes in
  // flight, as long as one wave of blocks is full (us with one, two, four and
  // six, in blocks of 256: rotation of 168 MB 37.5, 29.5, 28.2, 27.8; read of
  // 408 MB 106, 77, 65, 66; write of 201 MB 43.5, 39.9, 39.1, 40.1)
  const long long wave = (long long)kBlocks * kThreads * device_sm_count();
  s.tokens = (int)(work >= 4 * wave ? 4 : work <= wave ? 1 : (work + wave - 1) / wave) * s.tp;
  if (s.tokens > kTokensMax) s.tokens = kTokensMax / s.tp * s.tp;
  if (rot && s.tokens > kAnglesMax / rot) s.tokens = kAnglesMax / rot / s.tp * s.tp;
  s.blocks = (n + s.tokens - 1) / s.tokens * s.parts;
  s.by_chunks = fast_div((uint32_t)chunks);
  s.by_hp = fast_div((uint32_t)s.hp);
  s.by_half = fast_div(rot ? (uint32_t)rot / 2 : 1u);
  s.by_parts = fast_div((uint32_t)s.parts);
  return s;
}

// What a block does of it: tokens t0 .. t0 + n - 1; this thread part c of one
// head of every tp-th of them from `first` on.  The loops run alike in all
// threads and guard the accesses, so that whole warps meet in the shuffles.
struct Range {
  int t0, n, first, head, c;
  bool active;
};
__device__ __forceinline__ Range range_of(const Split& s, int block, int tokens) {
  Range r;
  const int group = (int)div_fast((uint32_t)block, s.by_parts);
  r.t0 = group * s.tokens;
  r.n = min(s.tokens, tokens - r.t0);
  const int mine = (int)div_fast(threadIdx.x, s.by_chunks);
  r.c = threadIdx.x - mine * s.chunks;
  r.first = (int)div_fast((uint32_t)mine, s.by_hp);
  r.head = (block - group * s.parts) * s.hp + (mine - r.first * s.hp);
  r.active = r.first < s.tp && r.head < s.heads;
  return r;
}

// Cosines [rot / 2], then sines, of each of the block's tokens.
__device__ __forceinline__ void fill_angles(float* angles, const RopeArgs& r, const Split& s, const Range& range,
                                            const int* pos, bool back) {
  const int half = r.rot / 2;
  for (int i = threadIdx.x; i < range.n * half; i += kThreads) {
    const int t = (int)div_fast((uint32_t)i, s.by_half), f = i - t * half;
    float sn, cs;
    turn(r.freq[f], pos[range.t0 + t], r.scale, &sn, &cs);
    angles[t * r.rot + f] = cs;
    angles[t * r.rot + half + f] = back ? -sn : sn;
  }
}

// The elements of thread c of a row.  VEC: eight from e0 and eight from e1;
// with c < rot / 16 they are pairs, (e0 + i, e1 + i) or neighbours, else
// they pass through.  Otherwise one pair each of 8 c ... 8 c + 7 (or of c).
__device__ __forceinline__ void vectors_of(int& e0, int& e1, int c, int rot, int dh) {
  const int turned = rot / 16;
  if (c < turned) {
    e0 = 8 * c, e1 = e0 + rot / 2;
  } else {
    e0 = rot + 8 * (c - turned), e1 = e0 + (dh - rot) / 2;
  }
}
__device__ __forceinline__ void pair_of(int& e0, int& e1, int pair, const RopeArgs& r) {
  const bool split = pair < r.rot / 2 && !r.interleaved;
  e0 = split ? pair : 2 * pair;
  e1 = split ? pair + r.rot / 2 : 2 * pair + 1;
}

__device__ __forceinline__ void rotate(float& a, float& b, float cs, float sn) {
  const float x = a;
  a = x * cs - b * sn;
  b = x * sn + b * cs;
}
__device__ __forceinline__ void load4(float* v, const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
// Rotates thread c's two vectors of a row (c < rot / 16).
__device__ __forceinline__ void rotate16(float (&x)[8], float (&y)[8], int c, const float* angles, const RopeArgs& r) {
  const int half = r.rot / 2;
  float cs[8], sn[8];
  // neighbours: pairs 4 c .. of the first vector, then 4 c + rot / 4 .. of the second
  const int f0 = r.interleaved ? 4 * c : 8 * c, f1 = r.interleaved ? f0 + half / 2 : f0 + 4;
  load4(cs, angles + f0), load4(cs + 4, angles + f1);
  load4(sn, angles + half + f0), load4(sn + 4, angles + half + f1);
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
      rotate(y[2 * i], y[2 * i + 1], cs[4 + i], sn[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate(x[i], y[i], cs[i], sn[i]);
  }
}

// Eight elements as they lie in memory.
template <typename T> struct Raw8 {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) == 1) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x, w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) {
      if constexpr (sizeof(T) == 1)
        unpack4(v + 4 * i, w[i], T());
      else if constexpr (sizeof(T) == 2)
        unpack_bf16(v + 2 * i, w[i]);
      else
        v[i] = __uint_as_float(w[i]);
    }
  }
};

// Rows a thread has in flight: 64 bytes of its parts.
template <typename T> constexpr int kAhead = 4 / sizeof(T);

// A block's rows of one tensor, rotated.  Padding tokens (negative positions)
// are left out if `padded`.
template <typename T, bool VEC>
__device__ __forceinline__ void rotate_rows(float* angles, const RopeArgs& r, const int* pos, int n, int dh,
                                            const HeadsArgs& t, const Split& s, int block, bool back, bool padded) {
  const Range range = range_of(s, block, n);
  const T* const in = (const T*)t.in + range.t0 * t.in_tok + range.head * t.in_head;
  T* const out = (T*)t.out + range.t0 * t.out_tok + range.head * t.out_head;
  if constexpr (VEC) {
    constexpr int U = kAhead<T>;
    int e0, e1;
    vectors_of(e0, e1, range.c, r.rot, dh);
    Raw8<T> x[U], y[U];
    auto fetch = [&](int lo) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = lo + u * s.tp + range.first;
        if (range.active && i < range.n) {
          const T* p = in + i * t.in_tok;
          x[u].load(p + e0), y[u].load(p + e1);
        }
      }
    };
    fetch(0);
    fill_angles(angles, r, s, range, pos, back);
    __syncthreads();
    for (int lo = 0; lo < range.n; lo += U * s.tp) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = lo + u * s.tp + range.first;
        if (!range.active || i >= range.n || (padded && pos[range.t0 + i] < 0)) continue;
        float v[8], w[8];
        x[u].get(v), y[u].get(w);
        if (range.c < r.rot / 16) rotate16(v, w, range.c, angles + i * r.rot, r);
        T* p = out + i * t.out_tok;
        store8<true>(p + e0, v);
        store8<true>(p + e1, w);
      }
      fetch(lo + U * s.tp);
    }
  } else {
    fill_angles(angles, r, s, range, pos, back);
    __syncthreads();
    if (!range.active) return;
    for (int i = range.first; i < range.n; i += s.tp) {
      if (padded && pos[range.t0 + i] < 0) continue;
      const T* p = in + i * t.in_tok;
      T* o = out + i * t.out_tok;
      for (int pair = range.c; pair < dh / 2; pair += s.chunks) {
        int e0, e1;
        pair_of(e0, e1, pair, r);
        float x = ld_f(p + e0), y = ld_f(p + e1);
        const float* f = angles + i * r.rot + pair;
        if (pair < r.rot / 2) rotate(x, y, f[0], f[r.rot / 2]);
        st_f(o + e0, x), st_f(o + e1, y);
      }
    }
  }
}

// Blocks below sa.blocks take rows of a, the others of b.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocks) k_rope(const RopeArgs r, const int* __restrict__ pos, int n, int dh,
                                                      const HeadsArgs a, const HeadsArgs b, bool back, const Split sa,
                                                      const Split sb) {
  __shared__ __align__(16) float angles[kAnglesMax];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < sa.blocks)
    rotate_rows<T, VEC>(angles, r, pos, n, dh, a, sa, blockIdx.x, back, false);
  else
    rotate_rows<T, VEC>(angles, r, pos, n, dh, b, sb, blockIdx.x - sa.blocks, back, false);
}

// Where the block's tokens go: element and scale offsets, -1 for padding and
// for places that do not exist.
struct Places {
  long long at[kTokensMax], scale[kTokensMax];
};
__device__ __forceinline__ void fill_places(Places& out, const KvPoolArgs& p, const KvPlaceArgs& pl, const Range& range,
                                            int* err) {
  for (int i = threadIdx.x; i < range.n; i += kThreads) {
    const int t = range.t0 + i, pos = pl.pos[t], seq = pl.seq ? pl.seq[t] : t;
    int page, row;
    out.at[i] = -1;
    if (pos < 0) continue;
    if ((uint32_t)seq >= (uint32_t)pl.seqs) {
      report_error(err, DEV_BAD_PLACE);
    } else if (page_of(pl.table + seq * pl.table_stride, pl.width, p, pos, &page, &row, err)) {
      out.at[i] = page * p.page + row * p.row;
      out.scale[i] = page * p.scale_page + row * p.scale_row;
    }
  }
}

// x and y, a row's share of this thread, as codes: the row's threads (a group
// of `lanes` of the warp, at least two) agree on its scale.  `m` is the
// largest of this thread's magnitudes as bits: the order of unsigned numbers
// is that of magnitudes, with infinities and NaN above every number.  The
// group's first thread divides for the scale, which is returned there, the
// others for the codes, in one instruction sequence.
template <typename C>
__device__ __forceinline__ float quantise16(float (&x)[8], float (&y)[8], uint32_t m, int lanes, bool first) {
  for (int o = lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float amax = fmaxf(__uint_as_float(m), 1e-30f), top = KvKind<C>::top;
  const float q = (first ? amax : top) / (first ? top : amax);
  const float inv = __shfl_sync(0xffffffffu, q, (threadIdx.x & 31 & ~(lanes - 1)) + 1);
  const bool fine = m < 0x7f800000u;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= inv, y[i] *= inv;
  if (!fine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
  }
  return fine ? q : __uint_as_float(0x7fffffffu);
}
__device__ __forceinline__ uint32_t largest(const float (&x)[8], const float (&y)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(y[i]) & 0x7fffffffu));
  return m;
}
// The same of bf16 pairs as they were loaded, two at a time.
__device__ __forceinline__ uint32_t largest(const Raw8<bf16>& x, const Raw8<bf16>& y) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, __vmaxu2(x.w[i] & 0x7fff7fffu, y.w[i] & 0x7fff7fffu));
  return max(m << 16, m & 0xffff0000u);
}

// Blocks below sk.blocks take rows of k and v, which share a place, the
// others rows of q, which are rotated into q.out.
template <typename T, typename C, bool VEC, bool ROPE>
__global__ void __launch_bounds__(kThreads, kBlocks) k_kv_write(const KvPoolArgs p, const KvPlaceArgs pl, const HeadsArgs k,
                                                          const HeadsArgs v, const RopeArgs r, const HeadsArgs q,
                                                          const Split sk, const Split sq, int* err) {
  __shared__ __align__(16) float angles[ROPE ? kAnglesMax : 1];
  __shared__ Places places;
  pdl_wait();
  pdl_trigger();
  if (ROPE && (int)blockIdx.x >= sk.blocks) {
    rotate_rows<T, VEC>(angles, r, pl.pos, pl.tokens, p.dh, q, sq, blockIdx.x - sk.blocks, false, true);
    return;
  }
  const Range range = range_of(sk, blockIdx.x, pl.tokens);
  const T* const k_in = (const T*)k.in + range.t0 * k.in_tok + range.head * k.in_head;
  const T* const v_in = (const T*)v.in + range.t0 * v.in_tok + range.head * v.in_head;
  Raw8<T> raw[4];
  int e0 = 0, e1 = 0;
  if constexpr (VEC) vectors_of(e0, e1, range.c, r.rot, p.dh);
  auto fetch = [&](int lo) {
    const int i = lo + range.first;
    if (VEC && range.active && i < range.n) {
      const T* from = k_in + i * k.in_tok;
      raw[0].load(from + e0), raw[1].load(from + e1);
      from = v_in + i * v.in_tok;
      raw[2].load(from + e0), raw[3].load(from + e1);
    }
  };
  fetch(0);
  if constexpr (ROPE) fill_angles(angles, r, sk, range, pl.pos, false);
  fill_places(places, p, pl, range, err);
  __syncthreads();
  const long long head = range.head * p.head, scale_head = range.head * p.scale_head;
  for (int lo = 0; lo < range.n; lo += sk.tp) {
    const bool mine = range.active && lo + range.first < range.n;
    const int i = mine ? lo + range.first : 0;
    const long long at = places.at[i];
    const bool ok = mine && at >= 0;
#pragma unroll
    for (int n = 0; n < 2; ++n) {  // k, v
      float x[8], y[8];
      const float* f = angles + i * r.rot;
      if constexpr (VEC) {
        raw[2 * n].get(x), raw[2 * n + 1].get(y);
        if (ROPE && n == 0 && range.c < r.rot / 16) rotate16(x, y, range.c, f, r);
      } else {
        const T* from = n ? v_in + i * v.in_tok : k_in + i * k.in_tok;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int pair = 8 * range.c + j;
          pair_of(e0, e1, pair, r);
          x[j] = mine ? ld_f(from + e0) : 0.f, y[j] = mine ? ld_f(from + e1) : 0.f;
          if (ROPE && n == 0 && pair < r.rot / 2) rotate(x[j], y[j], f[pair], f[r.rot / 2 + pair]);
        }
      }
      if constexpr (KvKind<C>::narrow) {
        uint32_t m;
        if constexpr (VEC && sizeof(T) == 2)
          m = ROPE && n == 0 ? largest(x, y) : largest(raw[2 * n], raw[2 * n + 1]);
        else
          m = largest(x, y);
        const float scale = quantise16<C>(x, y, m, sk.chunks, range.c == 0);
        if (ok && range.c == 0) (n ? p.v_scale : p.k_scale)[places.scale[i] + scale_head] = scale;
      }
      C* out = (C*)(n ? p.v : p.k) + at + head;
      if constexpr (VEC) {
        if (ok) store8<true>(out + e0, x), store8<true>(out + e1, y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          pair_of(e0, e1, 8 * range.c + j, r);
          if (ok) store1(out + e0, x[j]), store1(out + e1, y[j]);
        }
      }
    }
    fetch(lo + sk.tp);
  }
}

// Blocks below s.blocks take key rows, the others value rows.
template <typename T, typename C, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvPoolArgs p, const KvPlaceArgs pl, const HeadsArgs k,
                                                      const HeadsArgs v, const Split s, int* err) {
  __shared__ Places places;
  pdl_wait();
  pdl_trigger();
  const bool value = (int)blockIdx.x >= s.blocks;
  const HeadsArgs t = value ? v : k;
  const Range range = range_of(s, value ? blockIdx.x - s.blocks : blockIdx.x, pl.tokens);
  fill_places(places, p, pl, range, err);
  __syncthreads();
  constexpr int U = kAhead<C>;
  const C* const pages = (const C*)(value ? p.v : p.k) + range.head * p.head + 8 * range.c;
  const float* const scales = (value ? p.v_scale : p.k_scale) + range.head * p.scale_head;
  T* const base = (T*)t.out + range.t0 * t.out_tok + range.head * t.out_head + 8 * range.c;
  for (int lo = 0; lo < range.n; lo += U * s.tp) {
    Raw8<C> rx[U], ry[U];
    float scale[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = lo + u * s.tp + range.first;
      ok[u] = range.active && i < range.n && places.at[i] >= 0;
      if (ok[u]) {
        const C* in = pages + places.at[i];
        rx[u].load(in), ry[u].load(in + p.dh / 2);
        if constexpr (KvKind<C>::narrow) scale[u] = scales[places.scale[i]];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      float x[8], y[8];
      rx[u].get(x), ry[u].get(y);
      if constexpr (KvKind<C>::narrow) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= scale[u], y[j] *= scale[u];
      }
      T* out = base + (lo + u * s.tp + range.first) * t.out_tok;
      store8<VEC>(out, x), store8<VEC>(out + p.dh / 2, y);
    }
  }
}

// Whether a tensor's rows can be taken 16 bytes at a time.
template <typename T>
bool aligned(const void* p, long long tok, long long head) {
  const long long n = 16 / sizeof(T);
  return (uintptr_t)p % 16 == 0 && tok % n == 0 && head % n == 0;
}
template <typename T>
bool aligned(const HeadsArgs& a) {
  return a.heads == 0 || ((!a.in || aligned<T>(a.in, a.in_tok, a.in_head)) &&
                          (!a.out || aligned<T>(a.out, a.out_tok, a.out_head)));
}
// Whether rows of dh elements fall into vectors of eight with whole pairs.
template <typename T>
bool rope_vectors(const RopeArgs& r, int dh, const HeadsArgs& a, const HeadsArgs& b) {
  return r.rot % 16 == 0 && dh % 16 == 0 && aligned<T>(a) && aligned<T>(b);
}

// Threads of a row: of 16 elements each in vectors, else of a pair at a time.
inline int rope_chunks(bool vec, int dh) { return vec ? dh / 16 : dh / 2 < 32 ? dh / 2 : 32; }

template <typename T>
void rope_t(const RopeArgs& r, const int* pos, int n, int dh, const HeadsArgs& a, const HeadsArgs& b, bool back,
            cudaStream_t s) {
  const bool vec = rope_vectors<T>(r, dh, a, b);
  const int chunks = rope_chunks(vec, dh);
  const long long work = (long long)n * (a.heads + b.heads) * chunks;
  const Split sa = split_rows(n, a.heads, chunks, r.rot, work);
  const Split sb = b.heads ? split_rows(n, b.heads, chunks, r.rot, work) : Split();
  launch_kernel(vec ? k_rope<T, true> : k_rope<T, false>, sa.blocks + sb.blocks, kThreads, 0, s, r, pos, n, dh, a, b,
                back, sa, sb);
}

template <typename T, typename C>
void write_t(const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v, const RopeArgs* r,
             const HeadsArgs& q, int* err, cudaStream_t s) {
  const RopeArgs rope = r ? *r : RopeArgs();
  // one choice for the whole launch: rows of k, v and q all in vectors, or none
  const bool vec = aligned<T>(k) && rope_vectors<T>(rope, p.dh, v, q);
  const int chunks = p.dh / 16, q_chunks = rope_chunks(vec, p.dh);
  const long long work = (long long)pl.tokens * (2ll * p.heads * chunks + (long long)q.heads * q_chunks);
  const Split sk = split_rows(pl.tokens, p.heads, chunks, rope.rot, work);
  const Split sq = q.heads ? split_rows(pl.tokens, q.heads, q_chunks, rope.rot, work) : Split();
  auto* kernel = rope.rot ? (vec ? k_kv_write<T, C, true, true> : k_kv_write<T, C, false, true>)
                          : (vec ? k_kv_write<T, C, true, false> : k_kv_write<T, C, false, false>);
  launch_kernel(kernel, sk.blocks + sq.blocks, kThreads, 0, s, p, pl, k, v, rope, q, sk, sq, err);
}

template <typename T, typename C>
void read_t(const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v, int* err,
            cudaStream_t s) {
  const int chunks = p.dh / 16;
  const Split sp = split_rows(pl.tokens, p.heads, chunks, 0, 2ll * pl.tokens * p.heads * chunks);
  const bool vec = aligned<T>(k) && aligned<T>(v);
  launch_kernel(vec ? k_kv_read<T, C, true> : k_kv_read<T, C, false>, 2 * sp.blocks, kThreads, 0, s, p, pl, k, v, sp, err);
}

}  // namespace

void launch_rope(int dt, const RopeArgs& r, const int* pos, int tokens, int dh, const HeadsArgs& a,
                 const HeadsArgs& b, bool backward, cudaStream_t s) {
  if (dt == DT_F32)
    rope_t<float>(r, pos, tokens, dh, a, b, backward, s);
  else
    rope_t<bf16>(r, pos, tokens, dh, a, b, backward, s);
}

void launch_kv_write(int dt, const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v,
                     const RopeArgs* r, const HeadsArgs& q, int* err, cudaStream_t s) {
  if (dt == DT_F32) {
    if (p.kind == 0) write_t<float, float>(p, pl, k, v, r, q, err, s);
    if (p.kind == 2) write_t<float, e4m3>(p, pl, k, v, r, q, err, s);
    if (p.kind == 3) write_t<float, int8_t>(p, pl, k, v, r, q, err, s);
  } else {
    if (p.kind == 1) write_t<bf16, bf16>(p, pl, k, v, r, q, err, s);
    if (p.kind == 2) write_t<bf16, e4m3>(p, pl, k, v, r, q, err, s);
    if (p.kind == 3) write_t<bf16, int8_t>(p, pl, k, v, r, q, err, s);
  }
}

void launch_kv_read(int dt, const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v,
                    int* err, cudaStream_t s) {
  if (dt == DT_F32) {
    if (p.kind == 0) read_t<float, float>(p, pl, k, v, err, s);
    if (p.kind == 2) read_t<float, e4m3>(p, pl, k, v, err, s);
    if (p.kind == 3) read_t<float, int8_t>(p, pl, k, v, err, s);
  } else {
    if (p.kind == 1) read_t<bf16, bf16>(p, pl, k, v, err, s);
    if (p.kind == 2) read_t<bf16, e4m3>(p, pl, k, v, err, s);
    if (p.kind == 3) read_t<bf16, int8_t>(p, pl, k, v, err, s);
  }
}

}  // namespace photon
