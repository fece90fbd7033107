// Rotary positions, and the write and read of a caller's paged KV cache.
//
// All three move rows once and are bound by memory.  A block takes a few
// tokens; it finds their places and the sines and cosines of their positions
// once, in shared memory, while the first rows are on their way, and then
// walks over (token, head, part of the row) with a thread on 16 elements:
// two vectors of eight that hold both elements of every pair, so that a
// rotation needs no other thread's data and may run in place.
//
// Angles.  A pair turns by pos * f turns, f a 64-bit binary fraction.  The
// product modulo 2^64 drops whole turns without rounding; its upper 32 bits,
// as a signed number of half-turns in [-1, 1), go to sincospif, whose
// argument is then off by at most 2^-25 half-turns at any position (fp32
// pos * f would be off by whole radians near a million).
#include "kv_pages.cuh"
#include "launch.cuh"

namespace photon {

namespace {

constexpr int kThreads = 256;
constexpr int kTokensMax = 256;   // of a block
constexpr int kAnglesMax = 4096;  // sines and cosines of a block

__device__ __forceinline__ void turn(unsigned long long freq, int pos, float scale, float* s, float* c) {
  const int half_turns = (int)(((unsigned long long)(long long)pos * freq) >> 32);
  sincospif((float)half_turns * 0x1p-31f, s, c);
  *s *= scale;
  *c *= scale;
}

// One launch's split: a block takes `tokens` tokens of `items` threads' work
// each (rows * chunks), or one of `parts` spans of one token's items.
struct Split {
  int tokens, items, chunks, parts, span, blocks;
  FastDiv by_items, by_chunks, by_half, by_parts;
};

Split split_rows(int n, int rows, int chunks, int rot) {
  // 1024 items a block (four a thread) keep enough bytes in flight; calls too
  // small to give every SM two such blocks take 256
  Split s = {};
  s.items = rows * chunks, s.chunks = chunks;
  s.span = (long long)n * s.items >= 2048ll * device_sm_count() ? 4 * kThreads : kThreads;
  s.tokens = s.span / s.items < 1 ? 1 : s.span / s.items;
  if (s.tokens > kTokensMax) s.tokens = kTokensMax;
  if (rot && s.tokens > kAnglesMax / rot) s.tokens = kAnglesMax / rot;
  if (s.tokens > n) s.tokens = n;
  s.parts = s.tokens > 1 ? 1 : (s.items + s.span - 1) / s.span;
  if (s.parts == 1) s.span = s.tokens * s.items;
  s.blocks = (n + s.tokens - 1) / s.tokens * s.parts;
  s.by_items = fast_div((uint32_t)s.items);
  s.by_chunks = fast_div((uint32_t)chunks);
  s.by_half = fast_div(rot ? (uint32_t)rot / 2 : 1u);
  s.by_parts = fast_div((uint32_t)s.parts);
  return s;
}

// What a block does of it: tokens t0 .. t0 + n - 1, items lo .. hi - 1 of them.
struct Range {
  int t0, n, lo, hi;
};
__device__ __forceinline__ Range range_of(const Split& s, int block, int tokens) {
  Range r;
  const int group = (int)div_fast((uint32_t)block, s.by_parts);
  r.t0 = group * s.tokens;
  r.n = min(s.tokens, tokens - r.t0);
  r.lo = (block - group * s.parts) * s.span;
  r.hi = min(r.n * s.items, r.lo + s.span);
  return r;
}
struct Item {
  int token, row, c;  // token within the block
};
__device__ __forceinline__ Item item_of(const Split& s, int i) {
  Item it;
  it.token = (int)div_fast((uint32_t)i, s.by_items);
  const uint32_t rest = i - it.token * s.items;
  it.row = (int)div_fast(rest, s.by_chunks);
  it.c = (int)rest - it.row * s.chunks;
  return it;
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

// Items a thread has in flight: 64 bytes of rows.
template <typename T> constexpr int kAhead = 4 / sizeof(T);

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_rope(const RopeArgs r, const int* __restrict__ pos, int n, int dh,
                                                   const HeadsArgs a, const HeadsArgs b, bool back, const Split s) {
  __shared__ __align__(16) float angles[kAnglesMax];
  pdl_wait();
  pdl_trigger();
  const Range range = range_of(s, blockIdx.x, n);
  auto row_in = [&](const Item& it) {
    const HeadsArgs& t = it.row < a.heads ? a : b;
    const int h = it.row < a.heads ? it.row : it.row - a.heads;
    return (const T*)t.in + (range.t0 + it.token) * t.in_tok + h * t.in_head;
  };
  auto row_out = [&](const Item& it) {
    const HeadsArgs& t = it.row < a.heads ? a : b;
    const int h = it.row < a.heads ? it.row : it.row - a.heads;
    return (T*)t.out + (range.t0 + it.token) * t.out_tok + h * t.out_head;
  };
  if constexpr (VEC) {
    constexpr int U = kAhead<T>;
    Raw8<T> x[U], y[U];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= range.hi) continue;
        const Item it = item_of(s, i);
        int e0, e1;
        vectors_of(e0, e1, it.c, r.rot, dh);
        const T* p = row_in(it);
        x[u].load(p + e0), y[u].load(p + e1);
      }
    };
    int i0 = range.lo + threadIdx.x;
    fetch(i0);
    fill_angles(angles, r, s, range, pos, back);
    __syncthreads();
    while (i0 < range.hi) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= range.hi) continue;
        const Item it = item_of(s, i);
        int e0, e1;
        vectors_of(e0, e1, it.c, r.rot, dh);
        float v[8], w[8];
        x[u].get(v), y[u].get(w);
        if (it.c < r.rot / 16) rotate16(v, w, it.c, angles + it.token * r.rot, r);
        T* p = row_out(it);
        store8<true>(p + e0, v);
        store8<true>(p + e1, w);
      }
      i0 += U * kThreads;
      fetch(i0);
    }
  } else {
    fill_angles(angles, r, s, range, pos, back);
    __syncthreads();
    for (int i = range.lo + threadIdx.x; i < range.hi; i += kThreads) {
      const Item it = item_of(s, i);
      int e0, e1;
      pair_of(e0, e1, it.c, r);
      const T* p = row_in(it);
      float x = ld_f(p + e0), y = ld_f(p + e1);
      const float* f = angles + it.token * r.rot + it.c;
      if (it.c < r.rot / 2) rotate(x, y, f[0], f[r.rot / 2]);
      T* o = row_out(it);
      st_f(o + e0, x), st_f(o + e1, y);
    }
  }
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
// of `lanes` of the warp) agree on its scale.  |x| is compared as bits: the
// order of unsigned numbers is that of magnitudes, with infinities and NaN
// above every number.
template <typename C>
__device__ __forceinline__ void quantise16(float (&x)[8], float (&y)[8], float* scale, int lanes, bool first) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(y[i]) & 0x7fffffffu));
  const unsigned mask = ((1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
  for (int o = lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
  const float amax = fmaxf(__uint_as_float(m), 1e-30f);
  const bool fine = m < 0x7f800000u;
  const float inv = fine ? KvKind<C>::top / amax : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = fine ? x[i] * inv : 0.f;
    y[i] = fine ? y[i] * inv : 0.f;
  }
  if (first) *scale = fine ? amax / KvKind<C>::top : __uint_as_float(0x7fffffffu);
}

// Rows of a token: key heads, value heads, query heads (rotated into q.out).
template <typename T, typename C, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvPoolArgs p, const KvPlaceArgs pl, const HeadsArgs k,
                                                       const HeadsArgs v, const RopeArgs r, const HeadsArgs q,
                                                       const Split s, int* err) {
  __shared__ __align__(16) float angles[kAnglesMax];
  __shared__ Places places;
  pdl_wait();
  pdl_trigger();
  const Range range = range_of(s, blockIdx.x, pl.tokens);
  auto row_in = [&](const Item& it) {
    const HeadsArgs& t = it.row < p.heads ? k : it.row < 2 * p.heads ? v : q;
    const int h = it.row < p.heads ? it.row : it.row < 2 * p.heads ? it.row - p.heads : it.row - 2 * p.heads;
    return (const T*)t.in + (range.t0 + it.token) * t.in_tok + h * t.in_head;
  };
  auto turns = [&](const Item& it) { return r.rot > 0 && (it.row < p.heads || it.row >= 2 * p.heads); };
  constexpr int U = VEC ? kAhead<T> : 1;
  Raw8<T> rx[U], ry[U];
  auto fetch = [&](int i0) {
    if constexpr (VEC) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= range.hi) continue;
        const Item it = item_of(s, i);
        int e0, e1;
        vectors_of(e0, e1, it.c, r.rot, p.dh);
        const T* in = row_in(it);
        rx[u].load(in + e0), ry[u].load(in + e1);
      }
    }
  };
  int i0 = range.lo + threadIdx.x;
  fetch(i0);
  if (r.rot) fill_angles(angles, r, s, range, pl.pos, false);
  fill_places(places, p, pl, range, err);
  __syncthreads();
  while (i0 < range.hi) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= range.hi) continue;
      const Item it = item_of(s, i);
      const bool query = it.row >= 2 * p.heads;
      // a query follows its position alone, whether or not its place exists
      if (query ? pl.pos[range.t0 + it.token] < 0 : places.at[it.token] < 0) continue;
      float x[8], y[8];
      int e0[VEC ? 1 : 8], e1[VEC ? 1 : 8];
      const float* f = angles + it.token * r.rot;
      if constexpr (VEC) {
        vectors_of(e0[0], e1[0], it.c, r.rot, p.dh);
        rx[u].get(x), ry[u].get(y);
        if (it.c < r.rot / 16 && turns(it)) rotate16(x, y, it.c, f, r);
      } else {
        const T* in = row_in(it);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int pair = 8 * it.c + j;
          pair_of(e0[j], e1[j], pair, r);
          x[j] = ld_f(in + e0[j]), y[j] = ld_f(in + e1[j]);
          if (pair < r.rot / 2 && turns(it)) rotate(x[j], y[j], f[pair], f[r.rot / 2 + pair]);
        }
      }
      if (query) {
        T* out = (T*)q.out + (range.t0 + it.token) * q.out_tok + (it.row - 2 * p.heads) * q.out_head;
        if constexpr (VEC) {
          store8<true>(out + e0[0], x), store8<true>(out + e1[0], y);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) st_f(out + e0[j], x[j]), st_f(out + e1[j], y[j]);
        }
        continue;
      }
      const bool value = it.row >= p.heads;
      const int h = value ? it.row - p.heads : it.row;
      if constexpr (KvKind<C>::narrow)
        quantise16<C>(x, y, (value ? p.v_scale : p.k_scale) + places.scale[it.token] + h * p.scale_head, s.chunks, it.c == 0);
      C* out = (C*)(value ? p.v : p.k) + places.at[it.token] + h * p.head;
      if constexpr (VEC) {
        store8<true>(out + e0[0], x), store8<true>(out + e1[0], y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) store1(out + e0[j], x[j]), store1(out + e1[j], y[j]);
      }
    }
    i0 += U * kThreads;
    fetch(i0);
  }
}

template <typename T, typename C, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvPoolArgs p, const KvPlaceArgs pl, const HeadsArgs k,
                                                      const HeadsArgs v, const Split s, int* err) {
  __shared__ Places places;
  pdl_wait();
  pdl_trigger();
  const Range range = range_of(s, blockIdx.x, pl.tokens);
  fill_places(places, p, pl, range, err);
  __syncthreads();
  constexpr int U = kAhead<C>;
  for (int i0 = range.lo + threadIdx.x; i0 < range.hi; i0 += U * kThreads) {
    Raw8<C> rx[U], ry[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kThreads >= range.hi) continue;
      const Item it = item_of(s, i0 + u * kThreads);
      if (places.at[it.token] < 0) continue;
      const bool value = it.row >= p.heads;
      const int h = value ? it.row - p.heads : it.row;
      const C* in = (const C*)(value ? p.v : p.k) + places.at[it.token] + h * p.head + 8 * it.c;
      rx[u].load(in), ry[u].load(in + p.dh / 2);
      if constexpr (KvKind<C>::narrow) scale[u] = (value ? p.v_scale : p.k_scale)[places.scale[it.token] + h * p.scale_head];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kThreads >= range.hi) continue;
      const Item it = item_of(s, i0 + u * kThreads);
      if (places.at[it.token] < 0) continue;
      const bool value = it.row >= p.heads;
      const int h = value ? it.row - p.heads : it.row;
      float x[8], y[8];
      rx[u].get(x), ry[u].get(y);
      if constexpr (KvKind<C>::narrow) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= scale[u], y[j] *= scale[u];
      }
      const HeadsArgs& t = value ? v : k;
      T* out = (T*)t.out + (range.t0 + it.token) * t.out_tok + h * t.out_head + 8 * it.c;
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

template <typename T>
void rope_t(const RopeArgs& r, const int* pos, int n, int dh, const HeadsArgs& a, const HeadsArgs& b, bool back,
            cudaStream_t s) {
  const bool vec = rope_vectors<T>(r, dh, a, b);
  const Split sp = split_rows(n, a.heads + b.heads, vec ? dh / 16 : dh / 2, r.rot);
  launch_kernel(vec ? k_rope<T, true> : k_rope<T, false>, sp.blocks, kThreads, 0, s, r, pos, n, dh, a, b, back, sp);
}

template <typename T, typename C>
void write_t(const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v, const RopeArgs* r,
             const HeadsArgs& q, int* err, cudaStream_t s) {
  const RopeArgs rope = r ? *r : RopeArgs();
  const Split sp = split_rows(pl.tokens, 2 * p.heads + q.heads, p.dh / 16, rope.rot);
  // one choice for the whole launch: rows of k, v and q all in vectors, or none
  const bool vec = aligned<T>(k) && rope_vectors<T>(rope, p.dh, v, q);
  launch_kernel(vec ? k_kv_write<T, C, true> : k_kv_write<T, C, false>, sp.blocks, kThreads, 0, s, p, pl, k, v, rope, q,
                sp, err);
}

template <typename T, typename C>
void read_t(const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v, int* err,
            cudaStream_t s) {
  const Split sp = split_rows(pl.tokens, 2 * p.heads, p.dh / 16, 0);
  const bool vec = aligned<T>(k) && aligned<T>(v);
  launch_kernel(vec ? k_kv_read<T, C, true> : k_kv_read<T, C, false>, sp.blocks, kThreads, 0, s, p, pl, k, v, sp, err);
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
