// Rotary positions, and the write and read of a caller's paged KV cache.
//
// All three move rows once and are bound by memory: a thread holds eight
// elements (or two vectors of a rotated head) and walks over heads of one
// token, so that the token's angles and place are found once for all of them.
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
constexpr int kHeads = 8;  // most heads of one token a thread walks over

__device__ __forceinline__ void turn(unsigned long long freq, int pos, float scale, float* s, float* c) {
  const int half_turns = (int)(((unsigned long long)(long long)pos * freq) >> 32);
  sincospif((float)half_turns * 0x1p-31f, s, c);
  *s *= scale;
  *c *= scale;
}

// PP consecutive elements; PP is one 16-byte vector or a single element.
template <typename T, int PP>
__device__ __forceinline__ void load_pp(float (&v)[PP], const T* p) {
  if constexpr (PP == 1) {
    v[0] = ld_f(p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
    load8<true>(v, p);
  }
}
template <typename T, int PP>
__device__ __forceinline__ void store_pp(T* p, const float (&v)[PP]) {
  if constexpr (PP == 1) {
    st_f(p, v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    store8<true>(p, v);
  }
}

// One launch's split of tokens x heads x chunks over threads: a block takes
// `tokens` tokens, a token `items` = slots * chunks threads, and a thread the
// heads slot, slot + slots, ... of its token.
struct Split {
  int tokens, items, slots, chunks;
  FastDiv by_items, by_chunks;
  int blocks;
};

Split split_heads(int n, int heads, int chunks) {
  // enough threads for every SM first, then more heads a thread
  const long long rows = (long long)n * heads * chunks;
  long long hpt = rows / ((long long)device_sm_count() * 1024);
  hpt = hpt < 1 ? 1 : hpt > kHeads ? kHeads : hpt;
  Split s;
  s.slots = (int)((heads + hpt - 1) / hpt);
  s.chunks = chunks;
  s.items = s.slots * chunks;
  s.tokens = s.items < kThreads ? kThreads / s.items : 1;
  s.by_items = fast_div((uint32_t)s.items);
  s.by_chunks = fast_div((uint32_t)chunks);
  s.blocks = (int)(((long long)n + s.tokens - 1) / s.tokens);
  return s;
}

// Rotation of one (slot, chunk) of a token over its heads.  Chunk c < the
// rotated ones holds pairs c * PP ..: elements [c PP, +PP) and [c PP + rot/2,
// +PP), or [2 c PP, + 2 PP) when interleaved; later chunks copy 2 PP elements.
template <typename T, int PP>
__device__ __forceinline__ void rope_item(const RopeArgs& r, int pos, long long token, const HeadsArgs& a,
                                          const HeadsArgs& b, int slot, int slots, int c, bool back) {
  const int turned = r.rot / (2 * PP);
  float sn[PP], cs[PP];
  int e0, e1;
  if (c < turned) {
    e0 = r.interleaved ? 2 * c * PP : c * PP;
    e1 = r.interleaved ? e0 + PP : e0 + r.rot / 2;
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      turn(r.freq[c * PP + i], pos, r.scale, &sn[i], &cs[i]);
      if (back) sn[i] = -sn[i];
    }
  } else {
    e0 = 2 * c * PP, e1 = e0 + PP;
  }
  const int heads = a.heads + b.heads;
#pragma unroll 4
  for (int h = slot; h < heads; h += slots) {
    const bool second = h >= a.heads;
    const HeadsArgs& t = second ? b : a;
    const int hh = second ? h - a.heads : h;
    const T* in = (const T*)t.in + token * t.in_tok + hh * t.in_head;
    T* out = (T*)t.out + token * t.out_tok + hh * t.out_head;
    float x[PP], y[PP], u[PP], v[PP];
    load_pp<T, PP>(x, in + e0);
    load_pp<T, PP>(y, in + e1);
    if (c >= turned) {
#pragma unroll
      for (int i = 0; i < PP; ++i) u[i] = x[i], v[i] = y[i];
    } else if (!r.interleaved) {
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        u[i] = x[i] * cs[i] - y[i] * sn[i];
        v[i] = x[i] * sn[i] + y[i] * cs[i];
      }
    } else if constexpr (PP == 1) {
      u[0] = x[0] * cs[0] - y[0] * sn[0];
      v[0] = x[0] * sn[0] + y[0] * cs[0];
    } else {
#pragma unroll
      for (int i = 0; i < PP / 2; ++i) {
        u[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
        u[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
        v[2 * i] = y[2 * i] * cs[PP / 2 + i] - y[2 * i + 1] * sn[PP / 2 + i];
        v[2 * i + 1] = y[2 * i] * sn[PP / 2 + i] + y[2 * i + 1] * cs[PP / 2 + i];
      }
    }
    store_pp<T, PP>(out + e0, u);
    store_pp<T, PP>(out + e1, v);
  }
}

// Every item of a block's tokens: f(token, slot, chunk).
template <typename F>
__device__ __forceinline__ void for_items(const Split& s, int block, int n, F&& f) {
  if (s.items <= kThreads) {
    const uint32_t tl = div_fast(threadIdx.x, s.by_items);
    const long long token = (long long)block * s.tokens + tl;
    if ((int)tl >= s.tokens || token >= n) return;
    const uint32_t i = threadIdx.x - tl * s.items, slot = div_fast(i, s.by_chunks);
    f((int)token, (int)slot, (int)(i - slot * s.chunks));
  } else {
    for (uint32_t i = threadIdx.x; i < (uint32_t)s.items; i += kThreads) {
      const uint32_t slot = div_fast(i, s.by_chunks);
      f(block, (int)slot, (int)(i - slot * s.chunks));
    }
  }
}

template <typename T, int PP>
__global__ void __launch_bounds__(kThreads) k_rope(const RopeArgs r, const int* __restrict__ pos, int n,
                                                   const HeadsArgs a, const HeadsArgs b, bool back, const Split s) {
  pdl_wait();
  pdl_trigger();
  for_items(s, blockIdx.x, n, [&](int token, int slot, int c) {
    rope_item<T, PP>(r, pos[token], token, a, b, slot, s.slots, c, back);
  });
}

// Place of token t; false for padding and for places that do not exist.
__device__ __forceinline__ bool place_of(const KvPoolArgs& p, const KvPlaceArgs& pl, int t, int* page, int* row,
                                         int* err) {
  const int pos = pl.pos[t];
  if (pos < 0) return false;
  const int seq = pl.seq ? pl.seq[t] : t;
  if ((uint32_t)seq >= (uint32_t)pl.seqs) return report_error(err, DEV_BAD_PLACE), false;
  return page_of(pl.table + seq * pl.table_stride, pl.width, p, pos, page, row, err);
}

// x (elements e0 .. e0 + 7 of a row) rotated; the partners of the half layout
// come from the row itself.
template <typename T, bool VEC>
__device__ __forceinline__ void rotate8(float (&x)[8], const T* row, int e0, const RopeArgs& r, const float (&sn)[8],
                                        const float (&cs)[8]) {
  if (e0 >= r.rot) return;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e0 + 2 * i < r.rot) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * cs[i] - b * sn[i];
        x[2 * i + 1] = a * sn[i] + b * cs[i];
      }
    }
    return;
  }
  const int half = r.rot / 2;
  if (VEC && half % 8 == 0) {
    float y[8];
    const bool low = e0 < half;
    load8<VEC>(y, row + (low ? e0 + half : e0 - half));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = low ? x[i] * cs[i] - y[i] * sn[i] : y[i] * sn[i] + x[i] * cs[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      if (e < r.rot) {
        const bool low = e < half;
        const float y = ld_f(row + (low ? e + half : e - half));
        x[i] = low ? x[i] * cs[i] - y * sn[i] : y * sn[i] + x[i] * cs[i];
      }
    }
  }
}

// Stores one row's eight elements; the dh / 8 lanes of a row share its scale.
// |x| is compared as bits: the order of unsigned numbers is that of
// magnitudes, with infinities and NaN above every number.
template <typename C>
__device__ __forceinline__ void put8(float (&x)[8], C* dst, float* scale, int lanes, unsigned mask, bool first) {
  if constexpr (KvKind<C>::narrow) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    for (int o = lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
    const float amax = fmaxf(__uint_as_float(m), 1e-30f);
    const bool fine = m < 0x7f800000u;
    const float inv = KvKind<C>::top / amax;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fine ? x[i] * inv : 0.f;
    if (first) *scale = fine ? amax / KvKind<C>::top : __uint_as_float(0x7fffffffu);
  }
  store8<true>(dst, x);
}

template <typename T, typename C, bool VEC, int PP>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvPoolArgs p, const KvPlaceArgs pl, const HeadsArgs k,
                                                       const HeadsArgs v, const RopeArgs r, const HeadsArgs q,
                                                       const Split s, const Split sq, int* err) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= s.blocks) {  // rotation of q
    for_items(sq, blockIdx.x - s.blocks, pl.tokens, [&](int token, int slot, int c) {
      const int pos = pl.pos[token];
      if (pos >= 0) rope_item<T, PP>(r, pos, token, q, HeadsArgs(), slot, sq.slots, c, false);
    });
    return;
  }
  for_items(s, blockIdx.x, pl.tokens, [&](int token, int slot, int c) {
    int page, row;
    if (!place_of(p, pl, token, &page, &row, err)) return;
    const int lanes = s.chunks;
    const unsigned mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
    float sn[8], cs[8];
    if (8 * c < r.rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = 8 * c + i, half = r.rot / 2;
        const int f = r.interleaved ? 4 * c + i : e < half ? e : e - half;
        if (f < half && (i < 4 || !r.interleaved)) turn(r.freq[f], pl.pos[token], r.scale, &sn[i], &cs[i]);
      }
    }
    const long long at = page * p.page + row * p.row + 8 * c, sat = page * p.scale_page + row * p.scale_row;
#pragma unroll 2
    for (int h = slot; h < p.heads; h += s.slots) {
      const T* kr = (const T*)k.in + token * k.in_tok + h * k.in_head;
      const T* vr = (const T*)v.in + token * v.in_tok + h * v.in_head;
      float x[8], y[8];
      load8<VEC>(x, kr + 8 * c);
      load8<VEC>(y, vr + 8 * c);
      if (r.rot) rotate8<T, VEC>(x, kr, 8 * c, r, sn, cs);
      put8(x, (C*)p.k + at + h * p.head, p.k_scale + sat + h * p.scale_head, lanes, mask, c == 0);
      put8(y, (C*)p.v + at + h * p.head, p.v_scale + sat + h * p.scale_head, lanes, mask, c == 0);
    }
  });
}

template <typename T, typename C, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvPoolArgs p, const KvPlaceArgs pl, const HeadsArgs k,
                                                      const HeadsArgs v, const Split s, int* err) {
  pdl_wait();
  pdl_trigger();
  for_items(s, blockIdx.x, pl.tokens, [&](int token, int slot, int c) {
    int page, row;
    if (!place_of(p, pl, token, &page, &row, err)) return;
    const long long at = page * p.page + row * p.row + 8 * c, sat = page * p.scale_page + row * p.scale_row;
#pragma unroll 4
    for (int h = slot; h < p.heads; h += s.slots) {
      float x[8], y[8];
      load8<true>(x, (const C*)p.k + at + h * p.head);
      load8<true>(y, (const C*)p.v + at + h * p.head);
      if constexpr (KvKind<C>::narrow) {
        const float a = p.k_scale[sat + h * p.scale_head], b = p.v_scale[sat + h * p.scale_head];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= a, y[i] *= b;
      }
      store8<VEC>((T*)k.out + token * k.out_tok + h * k.out_head + 8 * c, x);
      store8<VEC>((T*)v.out + token * v.out_tok + h * v.out_head + 8 * c, y);
    }
  });
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
template <typename T>
bool rope_vectors(const RopeArgs& r, int dh, const HeadsArgs& a, const HeadsArgs& b) {
  const int two = 2 * 16 / sizeof(T);
  return r.rot % two == 0 && dh % two == 0 && aligned<T>(a) && aligned<T>(b);
}
bool in_place(const HeadsArgs& a) { return a.heads == 0 || a.in == a.out; }

// Chunks of a rotated head: what passes through is left alone in place.
int rope_chunks(const RopeArgs& r, int dh, const HeadsArgs& a, const HeadsArgs& b, int pp) {
  return (in_place(a) && in_place(b) ? r.rot : dh) / (2 * pp);
}

template <typename T>
void rope_t(const RopeArgs& r, const int* pos, int n, int dh, const HeadsArgs& a, const HeadsArgs& b, bool back,
            cudaStream_t s) {
  constexpr int PP = 16 / sizeof(T);
  if (rope_vectors<T>(r, dh, a, b)) {
    const Split sp = split_heads(n, a.heads + b.heads, rope_chunks(r, dh, a, b, PP));
    launch_kernel(k_rope<T, PP>, sp.blocks, kThreads, 0, s, r, pos, n, a, b, back, sp);
  } else {
    const Split sp = split_heads(n, a.heads + b.heads, rope_chunks(r, dh, a, b, 1));
    launch_kernel(k_rope<T, 1>, sp.blocks, kThreads, 0, s, r, pos, n, a, b, back, sp);
  }
}

template <typename T, typename C>
void write_t(const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v, const RopeArgs* r,
             const HeadsArgs& q, int* err, cudaStream_t s) {
  constexpr int PP = 16 / sizeof(T);
  const RopeArgs rope = r ? *r : RopeArgs();
  const Split sp = split_heads(pl.tokens, p.heads, p.dh / 8);
  // one choice for the whole launch: rows of k, v and q all in vectors, or none
  const bool vec = aligned<T>(k) && aligned<T>(v) && (q.heads == 0 || rope_vectors<T>(rope, p.dh, q, HeadsArgs()));
  Split sq = Split();
  if (q.heads) sq = split_heads(pl.tokens, q.heads, rope_chunks(rope, p.dh, q, HeadsArgs(), vec ? PP : 1));
  if (vec)
    launch_kernel(k_kv_write<T, C, true, PP>, sp.blocks + sq.blocks, kThreads, 0, s, p, pl, k, v, rope, q, sp, sq, err);
  else
    launch_kernel(k_kv_write<T, C, false, 1>, sp.blocks + sq.blocks, kThreads, 0, s, p, pl, k, v, rope, q, sp, sq, err);
}

template <typename T, typename C>
void read_t(const KvPoolArgs& p, const KvPlaceArgs& pl, const HeadsArgs& k, const HeadsArgs& v, int* err,
            cudaStream_t s) {
  const Split sp = split_heads(pl.tokens, p.heads, p.dh / 8);
  if (aligned<T>(k) && aligned<T>(v))
    launch_kernel(k_kv_read<T, C, true>, sp.blocks, kThreads, 0, s, p, pl, k, v, sp, err);
  else
    launch_kernel(k_kv_read<T, C, false>, sp.blocks, kThreads, 0, s, p, pl, k, v, sp, err);
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
