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

// A process's first call may be a captured one: loading kernels and creating
// the memory pool are no stream work, and are allowed during the call.
struct RelaxedCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

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
  if (p->page_stride < 0 || p->head_stride < 0 || p->row_stride < 0) return refuse("pages: negative stride");
  // rows are found by 32-bit offsets in the largest power of two of bytes that divides every stride
  const int64_t size = p->kind == PHOTON_KV_F32 ? 4 : p->kind == PHOTON_KV_BF16 ? 2 : 1, limit = INT64_MAX / 32;
  if (p->page_stride > limit || p->head_stride > limit || p->row_stride > limit) return refuse("pages: stride out of range");
  int64_t unit = 16;
  while (unit < (1 << 20) && ((p->page_stride | p->head_stride | p->row_stride) * size) % (2 * unit) == 0) unit *= 2;
  const double last = ((double)p->page_stride * (p->pages - 1) + (double)p->head_stride * (p->heads - 1) +
                       (double)p->row_stride * (p->page_rows - 1)) * size / unit;
  if (last >= 4294967295.0) return refuse("pages: too large for offsets in units of %d bytes", (int)unit);
  out->unit = (uint32_t)unit;
  out->page_u = (uint32_t)(p->page_stride * size / unit), out->head_u = (uint32_t)(p->head_stride * size / unit);
  out->row_u = (uint32_t)(p->row_stride * size / unit);
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

static int check_table(const photon_kv_pages* p, const int32_t* table, int64_t seqs, int64_t width) {
  if (seqs <= 0 || seqs > INT32_MAX || width <= 0) return refuse("table: shape [%lld, %lld]", (long long)seqs, (long long)width);
  if (!table || !aligned_to(table, 4)) return refuse("table: NULL or misaligned");
  if (width > (1 << 30) || width * p->page_rows > (1 << 30)) return refuse("table: more than 2^30 positions a sequence");
  return PHOTON_OK;
}

static int check_tokens(int64_t tokens, int64_t heads, const int32_t* pos, const int32_t* seq) {
  if (heads > (1 << 20)) return refuse("more than 2^20 heads");
  if (tokens < 0 || tokens > (1 << 30) || tokens * heads > INT32_MAX)
    return refuse("tokens * heads must be below 2^31 (%lld tokens)", (long long)tokens);
  if (tokens > 0 && (!pos || !aligned_to(pos, 4) || !aligned_to(seq, 4))) return refuse("positions: NULL or misaligned");
  return PHOTON_OK;
}

// Rows in, rows out.
static HeadsArgs rows_of(const photon_rows* in, const photon_rows* out, int64_t heads) {
  HeadsArgs h;
  if (in) h.in = in->p, h.in_tok = in->token, h.in_head = in->head;
  if (out) h.out = out->p, h.out_tok = out->token, h.out_head = out->head;
  h.heads = (int)heads;
  return h;
}
static int check_in_place(const photon_rows& x, const photon_rows& y) {
  if (x.p == y.p && (x.token != y.token || x.head != y.head)) return refuse("in place needs equal strides");
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
  // the fractions have 64 bits, and a position has 31: in doubles f's own
  // rounding would be as large at the last positions as that of the angle
  const long double two_pi = 6.283185307179586476925286766559005768L, factor = c->factor, alpha = c->alpha;
  const long double d = c->rot_dim;
  const long double theta = c->scaling == PHOTON_ROPE_NTK ? c->theta * powl(factor, d / (d - 2)) : (long double)c->theta;
  for (int i = 0; i < c->rot_dim / 2; ++i) {
    long double f = powl(theta, -2 * i / d);
    if (c->scaling == PHOTON_ROPE_LINEAR) f /= factor;
    if (c->scaling == PHOTON_ROPE_YARN) {
      long double g = (c->original_len * f / two_pi - alpha) / (c->beta - alpha);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = f * g + f / factor * (1 - g);
    }
    if (!std::isfinite((double)f)) return refuse("rope: frequency %d is not finite", i);
    long double turns = f / two_pi;
    turns -= floorl(turns);
    const long double scaled_up = rintl(ldexpl(turns, 64));
    h_freq[i] = scaled_up >= 0x1p64L ? 0 : (uint64_t)scaled_up;
  }
  *h_scale = (float)(c->attn_scale != 0 ? c->attn_scale : c->scaling == PHOTON_ROPE_YARN ? 0.1 * log(c->factor) + 1 : 1.0);
  return PHOTON_OK;
}

int photon_rope(const photon_rope_args* args, void* stream) {
  set_error_message("");
  if (!args) return refuse("args: NULL");
  const photon_rope_args& c = *args;
  if (c.dtype != 0 && c.dtype != 1) return refuse("dtype must be 0 or 1");
  if (!c.rope) return refuse("rope: NULL");
  if (c.head_dim < 2 || c.head_dim > 512 || c.head_dim % 2) return refuse("head_dim must be even, 2..512");
  if (c.heads <= 0 || c.heads2 < 0 || c.heads > (1 << 20) || c.heads2 > (1 << 20)) return refuse("heads out of range");
  RopeArgs r;
  CHECK(check_rope(c.rope, (int)c.head_dim, &r));
  CHECK(check_tokens(c.tokens, c.heads + c.heads2, c.d_pos, nullptr));
  if (c.tokens == 0) return PHOTON_OK;
  const int dt = (int)c.dtype;
  CHECK(check_rows("x", dt, c.x.p));
  CHECK(check_rows("y", dt, c.y.p));
  CHECK(check_in_place(c.x, c.y));
  HeadsArgs b;
  if (c.heads2) {
    CHECK(check_rows("x2", dt, c.x2.p));
    CHECK(check_rows("y2", dt, c.y2.p));
    CHECK(check_in_place(c.x2, c.y2));
    b = rows_of(&c.x2, &c.y2, c.heads2);
  }
  RelaxedCapture relaxed;
  launch_rope(dt, r, c.d_pos, (int)c.tokens, (int)c.head_dim, rows_of(&c.x, &c.y, c.heads), b, c.backward != 0,
              (cudaStream_t)stream);
  return launched();
}

// What the write and the read check alike; *go: there is work to do.
static int check_kv(const photon_kv_args* c, KvPoolArgs* p, KvPlaceArgs* pl, bool* go) {
  *go = false;
  if (!c) return refuse("args: NULL");
  if (c->dtype != 0 && c->dtype != 1) return refuse("dtype must be 0 or 1");
  CHECK(check_pool(c->pages, (int)c->dtype, p));
  if (c->q_heads < 0 || c->q_heads > (1 << 20)) return refuse("q_heads out of range");
  CHECK(check_tokens(c->tokens, p->heads + c->q_heads, c->d_pos, c->d_seq));
  if (!aligned_to(c->d_err, 4)) return refuse("d_err: misaligned");
  if (c->tokens == 0) return PHOTON_OK;
  CHECK(check_table(c->pages, c->d_table, c->seqs, c->width));
  CHECK(check_rows("k", (int)c->dtype, c->k.p));
  CHECK(check_rows("v", (int)c->dtype, c->v.p));
  *pl = {c->d_table, c->table_stride, (int)c->seqs, (int)c->width, c->d_seq, c->d_pos, (int)c->tokens};
  *go = true;
  return PHOTON_OK;
}

int photon_kv_write(const photon_kv_args* args, void* stream) {
  set_error_message("");
  KvPoolArgs p;
  KvPlaceArgs pl;
  bool go;
  CHECK(check_kv(args, &p, &pl, &go));
  const photon_kv_args& c = *args;
  RopeArgs r;
  if (c.rope) CHECK(check_rope(c.rope, p.dh, &r));
  if (c.q_heads && !c.rope) return refuse("q is rotated, so it needs rope");
  if (p.k == p.v || (p.k_scale && p.k_scale == p.v_scale)) return refuse("pages: keys and values share memory");
  if (!go) return PHOTON_OK;
  const int dt = (int)c.dtype;
  HeadsArgs q;
  if (c.q_heads) {
    CHECK(check_rows("q", dt, c.q.p));
    CHECK(check_rows("q_out", dt, c.q_out.p));
    CHECK(check_in_place(c.q, c.q_out));
    q = rows_of(&c.q, &c.q_out, c.q_heads);
  }
  RelaxedCapture relaxed;
  launch_kv_write(dt, p, pl, rows_of(&c.k, nullptr, p.heads), rows_of(&c.v, nullptr, p.heads), c.rope ? &r : nullptr, q,
                  c.d_err, (cudaStream_t)stream);
  return launched();
}

int photon_kv_read(const photon_kv_args* args, void* stream) {
  set_error_message("");
  KvPoolArgs p;
  KvPlaceArgs pl;
  bool go;
  CHECK(check_kv(args, &p, &pl, &go));
  if (args->rope || args->q_heads) return refuse("a read takes no rope and no q");
  if (!go) return PHOTON_OK;
  RelaxedCapture relaxed;
  launch_kv_read((int)args->dtype, p, pl, rows_of(nullptr, &args->k, p.heads), rows_of(nullptr, &args->v, p.heads),
                 args->d_err, (cudaStream_t)stream);
  return launched();
}

int photon_attn_decode_paged(const photon_attn_paged_args* args, void* stream) {
  set_error_message("");
  if (!args) return refuse("args: NULL");
  const photon_attn_paged_args& c = *args;
  if (c.dtype != 0 && c.dtype != 1) return refuse("dtype must be 0 or 1");
  PagedAttnArgs a;
  CHECK(check_pool(c.pages, (int)c.dtype, &a.pool));
  if (c.seqs == 0) return PHOTON_OK;
  CHECK(check_table(c.pages, c.d_table, c.seqs, c.width));
  if (c.q_heads <= 0 || c.q_heads % a.pool.heads) return refuse("q_heads must be a multiple of heads %d", a.pool.heads);
  if (c.q_heads > (1 << 20) || c.seqs * c.q_heads > INT32_MAX / 8) return refuse("seqs * q_heads must be below 2^28");
  if (c.window < 0 || c.window > INT32_MAX) return refuse("window out of range");
  const float scale = (float)c.scale;
  if (!std::isfinite(scale)) return refuse("scale must be finite");
  if (!c.d_len || !aligned_to(c.d_len, 4)) return refuse("d_len: NULL or misaligned");
  CHECK(check_rows("q", (int)c.dtype, c.q.p));
  CHECK(check_rows("o", (int)c.dtype, c.o.p));
  if (c.o.p == c.q.p) return refuse("o must not be q");
  if (!aligned_to(c.d_lse, 4) || !aligned_to(c.d_err, 4)) return refuse("d_lse, d_err: misaligned");
  a.table = c.d_table, a.table_stride = c.table_stride, a.seqs = (int)c.seqs, a.width = (int)c.width, a.len = c.d_len;
  a.q = c.q.p, a.q_seq = c.q.token, a.q_head = c.q.head, a.q_heads = (int)c.q_heads;
  a.window = (int)c.window, a.scale = scale;
  a.o = c.o.p, a.o_seq = c.o.token, a.o_head = c.o.head, a.lse = c.d_lse;
  RelaxedCapture relaxed;
  a.scratch = c.d_scratch, a.scratch_bytes = c.scratch_bytes;
  if (c.scratch_bytes > 0 && (!c.d_scratch || !aligned_to(c.d_scratch, 16))) return refuse("d_scratch: NULL or misaligned");
  size_t need = 0;
  CHECK(result(launch_attn_paged((int)c.dtype, a, c.d_err, (cudaStream_t)stream, &need)));
  if (need && c.scratch_bytes > 0) return refuse("scratch_bytes %lld, needs %zu", (long long)c.scratch_bytes, need);
  return (int)need;
}

}  // extern "C"
