// Attention of one new token per sequence over a caller's paged KV cache.
//
//   o[b, h] = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m),
//   s_t = scale log2(e) q[b, h] . k_t,  m = max_t s_t,
// over one pass of the positions: a warp carries m, the sum and the
// accumulator in fp32 and multiplies the two by 2^(m_old - m_new) when m
// grows.
//
// One CTA of four warps per (sequence, key head, up to GH of its query
// heads).  The warps take tiles of 16 positions in turn; their results are
// joined in shared memory.
#include <cmath>

#include "kv_pages.cuh"
#include "launch.cuh"

namespace photon {

namespace {

constexpr int kWarps = 4;
constexpr int kTile = 16;  // positions a warp takes at a time

__device__ __forceinline__ float one_f(float x) { return x; }
__device__ __forceinline__ float one_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float one_f(int8_t x) { return (float)x; }
__device__ __forceinline__ float one_f(e4m3 x) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(x.x, __NV_E4M3)));
}
// N consecutive elements (at most 16 bytes a load) as fp32.
template <int N, typename C>
__device__ __forceinline__ void load_n(float (&v)[N], const C* p) {
  constexpr int M = N * sizeof(C) > 16 ? 16 / (int)sizeof(C) : N;
  struct alignas(M * sizeof(C)) Raw {
    C x[M];
  };
#pragma unroll
  for (int j = 0; j < N; j += M) {
    const Raw r = *reinterpret_cast<const Raw*>(p + j);
#pragma unroll
    for (int i = 0; i < M; ++i) v[j + i] = one_f(r.x[i]);
  }
}

template <typename T, typename C, int D, int GH>
__global__ void __launch_bounds__(kWarps * 32) k_attn_paged(const PagedAttnArgs a, const int chunks, int* err) {
  constexpr int VPL = D / 32;  // output elements of a lane
  __shared__ __align__(16) float sq[GH][D];
  __shared__ __align__(16) float so[kWarps][GH][D];
  __shared__ __align__(16) float sp[kWarps][kTile][GH];
  __shared__ long long soff[kWarps][kTile];
  __shared__ float sm[kWarps][GH], sl[kWarps][GH];
  pdl_wait();
  pdl_trigger();
  const KvPoolArgs& p = a.pool;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.x / (p.heads * chunks), rest = blockIdx.x % (p.heads * chunks);
  const int kh = rest / chunks, group = a.q_heads / p.heads;
  const int h0 = kh * group + rest % chunks * GH, nh = min(GH, (kh + 1) * group - h0);
  const int cap = a.width * p.rows;
  int len = a.len[b];
  if (len < 0 || len > cap) {
    report_error(err, DEV_BAD_LENGTH);
    len = len < 0 ? 0 : cap;
  }
  const int first = a.window > 0 ? max(0, len - a.window) : 0;
  for (int i = tid; i < GH * D; i += kWarps * 32) {
    const int h = i / D, e = i % D;
    sq[h][e] = 0.f;
    if (h < nh) sq[h][e] = ld_f((const T*)a.q + b * a.q_seq + (h0 + h) * a.q_head + e) * (a.scale * 1.4426950408889634f);
  }
  __syncthreads();
  const int* table = a.table + b * a.table_stride;
  float m[GH], l[GH], acc[GH][VPL];
#pragma unroll
  for (int h = 0; h < GH; ++h) {
    m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[h][i] = 0.f;
  }
  for (int t0 = first + w * kTile; t0 < len; t0 += kWarps * kTile) {
    // lanes 0..15 (and 16..31 again): place of one position, -1 where there is none
    long long off = -1;
    float ks = 1.f, vs = 1.f;
    {
      const int pos = t0 + lane % kTile;
      int page, row;
      if (pos < len && page_of(table, a.width, p, pos, &page, &row, err)) {
        off = page * p.page + row * p.row + kh * p.head;
        if constexpr (KvKind<C>::narrow) {
          const long long s = page * p.scale_page + row * p.scale_row + kh * p.scale_head;
          ks = p.k_scale[s], vs = p.v_scale[s];
        }
      }
      if (lane < kTile) soff[w][lane] = off;
    }
    __syncwarp();
    // lane (g, t): positions g and g + 8, every fourth group of eight elements
    float s[2][GH];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const long long o = soff[w][g + 8 * r];
#pragma unroll
      for (int h = 0; h < GH; ++h) s[r][h] = 0.f;
      if (o >= 0) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = (t + 4 * i) * 8;
          float x[8];
          load8<true>(x, (const C*)p.k + o + e);
#pragma unroll
          for (int h = 0; h < GH; ++h) {
            const float4 q0 = *reinterpret_cast<const float4*>(&sq[h][e]);
            const float4 q1 = *reinterpret_cast<const float4*>(&sq[h][e + 4]);
            s[r][h] += x[0] * q0.x + x[1] * q0.y + x[2] * q0.z + x[3] * q0.w + x[4] * q1.x + x[5] * q1.y +
                       x[6] * q1.z + x[7] * q1.w;
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool seen = soff[w][g + 8 * r] >= 0;
      const float k_scale = __shfl_sync(0xffffffffu, ks, g + 8 * r);
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        s[r][h] += __shfl_xor_sync(0xffffffffu, s[r][h], 1);
        s[r][h] += __shfl_xor_sync(0xffffffffu, s[r][h], 2);
        s[r][h] = seen ? s[r][h] * k_scale : -INFINITY;
      }
    }
    const float v0 = __shfl_sync(0xffffffffu, vs, g), v1 = __shfl_sync(0xffffffffu, vs, g + 8);
#pragma unroll
    for (int h = 0; h < GH; ++h) {
      float mx = fmaxf(s[0][h], s[1][h]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(mx, m[h]);
      const float base = mx == -INFINITY ? 0.f : mx, grow = exp2f(m[h] - base);
      const float p0 = exp2f(s[0][h] - base), p1 = exp2f(s[1][h] - base);
      m[h] = mx;
      l[h] = l[h] * grow + (p0 + p1);
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[h][i] *= grow;
      if (t == 0) sp[w][g][h] = p0 * v0, sp[w][g + 8][h] = p1 * v1;
    }
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < kTile; ++j) {
      const long long o = soff[w][j];
      if (o < 0) continue;
      float x[VPL];
      load_n<VPL>(x, (const C*)p.v + o + lane * VPL);
#pragma unroll
      for (int h = 0; h < GH; ++h)
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[h][i] += sp[w][j][h] * x[i];
    }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < GH; ++h) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
    if (lane == 0) sm[w][h] = m[h], sl[w][h] = l[h];
#pragma unroll
    for (int i = 0; i < VPL; ++i) so[w][h][lane * VPL + i] = acc[h][i];
  }
  __syncthreads();
  for (int i = tid; i < nh * D; i += kWarps * 32) {
    const int h = i / D, e = i % D;
    float mx = sm[0][h], sum = 0.f, o = 0.f;
#pragma unroll
    for (int k = 1; k < kWarps; ++k) mx = fmaxf(mx, sm[k][h]);
    const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float f = exp2f(sm[k][h] - base);
      sum += f * sl[k][h];
      o += f * so[k][h][e];
    }
    st_f((T*)a.o + b * a.o_seq + (h0 + h) * a.o_head + e, sum == 0.f ? 0.f : o / sum);
    if (a.lse && e == 0)
      a.lse[(long long)b * a.q_heads + h0 + h] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
  }
}

template <typename T, typename C, int D>
void attn_d(const PagedAttnArgs& a, int* err, cudaStream_t s) {
  const int group = a.q_heads / a.pool.heads;
  const int gh = group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8, chunks = (group + gh - 1) / gh;
  const unsigned grid = (unsigned)((long long)a.seqs * a.pool.heads * chunks);
  if (gh == 1) launch_kernel(k_attn_paged<T, C, D, 1>, grid, kWarps * 32, 0, s, a, chunks, err);
  if (gh == 2) launch_kernel(k_attn_paged<T, C, D, 2>, grid, kWarps * 32, 0, s, a, chunks, err);
  if (gh == 4) launch_kernel(k_attn_paged<T, C, D, 4>, grid, kWarps * 32, 0, s, a, chunks, err);
  if (gh == 8) launch_kernel(k_attn_paged<T, C, D, 8>, grid, kWarps * 32, 0, s, a, chunks, err);
}

template <typename T, typename C>
void attn_c(const PagedAttnArgs& a, int* err, cudaStream_t s) {
  switch (a.pool.dh) {
    case 32: return attn_d<T, C, 32>(a, err, s);
    case 64: return attn_d<T, C, 64>(a, err, s);
    case 128: return attn_d<T, C, 128>(a, err, s);
    case 256: return attn_d<T, C, 256>(a, err, s);
  }
}

}  // namespace

void launch_attn_paged(int dt, const PagedAttnArgs& a, int* err, cudaStream_t s) {
  if (dt == DT_F32) {
    if (a.pool.kind == 0) attn_c<float, float>(a, err, s);
    if (a.pool.kind == 2) attn_c<float, e4m3>(a, err, s);
    if (a.pool.kind == 3) attn_c<float, int8_t>(a, err, s);
  } else {
    if (a.pool.kind == 1) attn_c<bf16, bf16>(a, err, s);
    if (a.pool.kind == 2) attn_c<bf16, e4m3>(a, err, s);
    if (a.pool.kind == 3) attn_c<bf16, int8_t>(a, err, s);
  }
}

}  // namespace photon
