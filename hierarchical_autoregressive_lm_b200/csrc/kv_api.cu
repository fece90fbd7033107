// C entry points of the operators around a caller's paged KV cache: argument
// checks, then the launches of k_kv_pages.cu and k_attn_paged.cu.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kernels.h"
#include "photon.h"

using namespace photon;

static int refuse(const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_error_message(buf);
  return PHOTON_ERR_ARG;
}

static int result(cudaError_t e) {
  if (e == cudaSuccess) return PHOTON_OK;
  set_error_message(cudaGetErrorString(e));
  return e == cudaErrorMemoryAllocation ? PHOTON_ERR_OOM : PHOTON_ERR_CUDA;
}
static int launched() { return result(cudaGetLastError()); }

static bool aligned_to(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

// Each check returns PHOTON_OK or the refusal.
static int check_rope(const photon_rope_table* r, int head_dim, RopeArgs* out) {
  if (!r->d_freq || !aligned_to(r->d_freq, 8)) return refuse("rope: d_freq must be an 8-byte aligned device array");
  if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > head_dim)
    return refuse("rope: rot_dim %d must be even, 2..head_dim = %d", r->rot_dim, head_dim);
  out->freq = (const unsigned long long*)r->d_freq;
  out->rot = r->rot_dim;
  out->interleaved = r->interleaved != 0;
  out->scale = r->scale;
  return PHOTON_OK;
}

static int check_rows(const char* name, int dtype, const void* p) {
  if (!p) return refuse("%s: NULL buffer", name);
  if (!aligned_to(p, dtype_size(dtype))) return refuse("%s: not aligned to its elements", name);
  return PHOTON_OK;
}

static int check_pool(const photon_kv_pages* p, int dtype, KvPoolArgs* out) {
  if (!p) return refuse("pages: NULL");
  if (p->kind < PHOTON_KV_F32 || p->kind > PHOTON_KV_INT8) return refuse("pages: unknown kind %d", p->kind);
  if ((p->kind == PHOTON_KV_F32 && dtype != 0) || (p->kind == PHOTON_KV_BF16 && dtype != 1))
    return refuse("pages: a wide cache holds the type of q, k and v");
  if (p->pages <= 0 || p->page_rows <= 0 || p->heads <= 0) return refuse("pages: empty shape");
  if (p->head_dim != 32 && p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return refuse("pages: head_dim %d (32, 64, 128 or 256)", p->head_dim);
  if (!p->k || !p->v) return refuse("pages: NULL buffer");
  const int narrow = p->kind >= PHOTON_KV_E4M3;
  if (narrow && (!p->k_scale || !p->v_scale)) return refuse("pages: a narrow cache needs k_scale and v_scale");
  const int64_t per16 = p->kind == PHOTON_KV_F32 ? 4 : p->kind == PHOTON_KV_BF16 ? 8 : 16;
  if (!aligned_to(p->k, 16) || !aligned_to(p->v, 16) || p->page_stride % per16 || p->head_stride % per16 ||
      p->row_stride % per16)
    return refuse("pages: bases and strides must be multiples of 16 bytes");
  if (narrow && (!aligned_to(p->k_scale, 4) || !aligned_to(p->v_scale, 4))) return refuse("pages: scales not aligned");
  out->k = p->k, out->v = p->v;
  out->k_scale = narrow ? p->k_scale : nullptr;
  out->v_scale = narrow ? p->v_scale : nullptr;
  out->page = p->page_stride, out->head = p->head_stride, out->row = p->row_stride;
  out->scale_page = p->scale_page, out->scale_head = p->scale_head, out->scale_row = p->scale_row;
  out->kind = p->kind, out->pages = p->pages, out->rows = p->page_rows, out->heads = p->heads;
  out->dh = p->head_dim;
  out->div = fast_div((uint32_t)p->page_rows);
  return PHOTON_OK;
}

static int check_table(const photon_kv_pages* p, const int32_t* table, int32_t seqs, int32_t width) {
  if (seqs <= 0 || width <= 0) return refuse("table: empty shape [%d, %d]", seqs, width);
  if (!table || !aligned_to(table, 4)) return refuse("table: NULL or misaligned");
  if ((int64_t)width * p->page_rows > (1 << 30)) return refuse("table: more than 2^30 positions a sequence");
  return PHOTON_OK;
}

static int check_tokens(int32_t tokens, int64_t heads, const int32_t* pos, const int32_t* seq) {
  if (heads > (1 << 20)) return refuse("more than 2^20 heads");
  if (tokens < 0 || tokens > (1 << 30) || tokens * heads > INT32_MAX)
    return refuse("tokens * heads must be below 2^31 (%d tokens)", tokens);
  if (tokens > 0 && (!pos || !aligned_to(pos, 4) || !aligned_to(seq, 4))) return refuse("positions: NULL or misaligned");
  return PHOTON_OK;
}

#define CHECK(x)                    \
  do {                              \
    const int rc_ = (x);            \
    if (rc_ != PHOTON_OK) return rc_; \
  } while (0)

extern "C" {

int photon_rope_frequencies(const photon_rope_config* c, uint64_t* h_freq, float* h_scale) {
  set_error_message("");
  if (!c || !h_freq || !h_scale) return refuse("rope: NULL argument");
  if (c->rot_dim < 2 || c->rot_dim > 512 || c->rot_dim % 2) return refuse("rope: rot_dim %d must be even, 2..512", c->rot_dim);
  if (c->scaling < PHOTON_ROPE_PLAIN || c->scaling > PHOTON_ROPE_YARN) return refuse("rope: unknown scaling %d", c->scaling);
  if (!(c->theta > 0) || !std::isfinite(c->theta)) return refuse("rope: theta must be positive");
  if (!std::isfinite(c->attn_scale)) return refuse("rope: attn_scale must be finite");
  const bool scaled = c->scaling != PHOTON_ROPE_PLAIN;
  if (scaled && (!(c->factor >= 1) || !std::isfinite(c->factor))) return refuse("rope: factor must be at least 1");
  if (c->scaling == PHOTON_ROPE_NTK && c->rot_dim < 4) return refuse("rope: NTK scaling needs rot_dim >= 4");
  if (c->scaling == PHOTON_ROPE_YARN && (c->original_len <= 0 || !(c->beta > c->alpha) || !std::isfinite(c->beta - c->alpha)))
    return refuse("rope: YARN needs original_len > 0 and beta > alpha");
  const double two_pi = 6.283185307179586476925286766559;
  const double d = c->rot_dim, theta = c->scaling == PHOTON_ROPE_NTK ? c->theta * pow(c->factor, d / (d - 2)) : c->theta;
  for (int i = 0; i < c->rot_dim / 2; ++i) {
    double f = pow(theta, -2.0 * i / d);
    if (c->scaling == PHOTON_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == PHOTON_ROPE_YARN) {
      double g = (c->original_len * f / two_pi - c->alpha) / (c->beta - c->alpha);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = f * g + f / c->factor * (1 - g);
    }
    if (!std::isfinite(f)) return refuse("rope: frequency %d is not finite", i);
    double turns = f / two_pi;
    turns -= floor(turns);
    const double scaled_up = rint(turns * 0x1p64);
    h_freq[i] = scaled_up >= 0x1p64 ? 0 : (uint64_t)scaled_up;
  }
  *h_scale = (float)(c->attn_scale != 0 ? c->attn_scale : c->scaling == PHOTON_ROPE_YARN ? 0.1 * log(c->factor) + 1 : 1.0);
  return PHOTON_OK;
}

int photon_rope(int32_t dtype, const photon_rope_table* rope, const int32_t* d_pos, int32_t tokens, int32_t head_dim,
                const void* d_x, int64_t x_token, int64_t x_head, int32_t heads, void* d_y, int64_t y_token,
                int64_t y_head, const void* d_x2, int64_t x2_token, int64_t x2_head, int32_t heads2, void* d_y2,
                int64_t y2_token, int64_t y2_head, int32_t backward, void* stream) {
  set_error_message("");
  if (dtype != 0 && dtype != 1) return refuse("dtype must be 0 or 1");
  if (!rope) return refuse("rope: NULL");
  if (head_dim < 2 || head_dim > 512 || head_dim % 2) return refuse("head_dim %d must be even, 2..512", head_dim);
  if (heads <= 0 || heads2 < 0) return refuse("heads: %d and %d", heads, heads2);
  RopeArgs r;
  CHECK(check_rope(rope, head_dim, &r));
  CHECK(check_tokens(tokens, (int64_t)heads + heads2, d_pos, nullptr));
  if (tokens == 0) return PHOTON_OK;
  CHECK(check_rows("x", dtype, d_x));
  CHECK(check_rows("y", dtype, d_y));
  HeadsArgs a, b;
  a = {d_x, d_y, x_token, x_head, y_token, y_head, heads};
  if (heads2) {
    CHECK(check_rows("x2", dtype, d_x2));
    CHECK(check_rows("y2", dtype, d_y2));
    b = {d_x2, d_y2, x2_token, x2_head, y2_token, y2_head, heads2};
  }
  if ((d_x == d_y && (x_token != y_token || x_head != y_head)) ||
      (heads2 && d_x2 == d_y2 && (x2_token != y2_token || x2_head != y2_head)))
    return refuse("in place needs equal strides");
  launch_rope(dtype, r, d_pos, tokens, head_dim, a, b, backward != 0, (cudaStream_t)stream);
  return launched();
}

int photon_kv_write(const photon_kv_pages* pages, int32_t dtype, const int32_t* d_table, int64_t table_stride,
                    int32_t seqs, int32_t width, const int32_t* d_seq, const int32_t* d_pos, int32_t tokens,
                    const void* d_k, int64_t k_token, int64_t k_head, const void* d_v, int64_t v_token,
                    int64_t v_head, const photon_rope_table* rope, const void* d_q, int64_t q_token, int64_t q_head,
                    int32_t q_heads, void* d_q_out, int64_t qo_token, int64_t qo_head, int32_t* d_err, void* stream) {
  set_error_message("");
  if (dtype != 0 && dtype != 1) return refuse("dtype must be 0 or 1");
  KvPoolArgs p;
  CHECK(check_pool(pages, dtype, &p));
  if (q_heads < 0) return refuse("q_heads: %d", q_heads);
  CHECK(check_tokens(tokens, (int64_t)p.heads + q_heads, d_pos, d_seq));
  RopeArgs r;
  if (rope) CHECK(check_rope(rope, p.dh, &r));
  if (q_heads && !rope) return refuse("q is rotated, so it needs rope");
  if (tokens == 0) return PHOTON_OK;
  CHECK(check_table(pages, d_table, seqs, width));
  CHECK(check_rows("k", dtype, d_k));
  CHECK(check_rows("v", dtype, d_v));
  const KvPlaceArgs pl = {d_table, table_stride, seqs, width, d_seq, d_pos, tokens};
  HeadsArgs k, v, q;
  k = {d_k, nullptr, k_token, k_head, 0, 0, p.heads};
  v = {d_v, nullptr, v_token, v_head, 0, 0, p.heads};
  if (q_heads) {
    CHECK(check_rows("q", dtype, d_q));
    CHECK(check_rows("q_out", dtype, d_q_out));
    if (d_q == d_q_out && (q_token != qo_token || q_head != qo_head)) return refuse("in place needs equal strides");
    q = {d_q, d_q_out, q_token, q_head, qo_token, qo_head, q_heads};
  }
  launch_kv_write(dtype, p, pl, k, v, rope ? &r : nullptr, q, d_err, (cudaStream_t)stream);
  return launched();
}

int photon_kv_read(const photon_kv_pages* pages, int32_t dtype, const int32_t* d_table, int64_t table_stride,
                   int32_t seqs, int32_t width, const int32_t* d_seq, const int32_t* d_pos, int32_t tokens, void* d_k,
                   int64_t k_token, int64_t k_head, void* d_v, int64_t v_token, int64_t v_head, int32_t* d_err,
                   void* stream) {
  set_error_message("");
  if (dtype != 0 && dtype != 1) return refuse("dtype must be 0 or 1");
  KvPoolArgs p;
  CHECK(check_pool(pages, dtype, &p));
  CHECK(check_tokens(tokens, p.heads, d_pos, d_seq));
  if (tokens == 0) return PHOTON_OK;
  CHECK(check_table(pages, d_table, seqs, width));
  CHECK(check_rows("k", dtype, d_k));
  CHECK(check_rows("v", dtype, d_v));
  const KvPlaceArgs pl = {d_table, table_stride, seqs, width, d_seq, d_pos, tokens};
  HeadsArgs k, v;
  k = {nullptr, d_k, 0, 0, k_token, k_head, p.heads};
  v = {nullptr, d_v, 0, 0, v_token, v_head, p.heads};
  launch_kv_read(dtype, p, pl, k, v, d_err, (cudaStream_t)stream);
  return launched();
}

int photon_attn_decode_paged(const photon_kv_pages* pages, int32_t dtype, const int32_t* d_table,
                             int64_t table_stride, int32_t seqs, int32_t width, const int32_t* d_len,
                             const void* d_q, int64_t q_seq, int64_t q_head, int32_t q_heads, int32_t window,
                             float scale, void* d_o, int64_t o_seq, int64_t o_head, float* d_lse, int32_t* d_err,
                             void* stream) {
  set_error_message("");
  if (dtype != 0 && dtype != 1) return refuse("dtype must be 0 or 1");
  PagedAttnArgs a;
  CHECK(check_pool(pages, dtype, &a.pool));
  if (seqs == 0) return PHOTON_OK;
  CHECK(check_table(pages, d_table, seqs, width));
  if (q_heads <= 0 || q_heads % a.pool.heads) return refuse("q_heads %d must be a multiple of heads %d", q_heads, a.pool.heads);
  if ((int64_t)seqs * q_heads > INT32_MAX) return refuse("seqs * q_heads must be below 2^31");
  if (window < 0) return refuse("window: %d", window);
  if (!std::isfinite(scale)) return refuse("scale must be finite");
  if (!d_len || !aligned_to(d_len, 4)) return refuse("d_len: NULL or misaligned");
  CHECK(check_rows("q", dtype, d_q));
  CHECK(check_rows("o", dtype, d_o));
  if (!aligned_to(d_lse, 4)) return refuse("d_lse: misaligned");
  a.table = d_table, a.table_stride = table_stride, a.seqs = seqs, a.width = width, a.len = d_len;
  a.q = d_q, a.q_seq = q_seq, a.q_head = q_head, a.q_heads = q_heads;
  a.window = window, a.scale = scale;
  a.o = d_o, a.o_seq = o_seq, a.o_head = o_head, a.lse = d_lse;
  return result(launch_attn_paged(dtype, a, d_err, (cudaStream_t)stream));
}

}  // extern "C"
