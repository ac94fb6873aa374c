// C entry points of the operators that work on the caller's device buffers
// (include/fs.h): the 8-bit paged KV cache, draft verification, and what differs from
// request to request in a step (pages, rotary positions, adapters, sampling). They check
// their arguments on the host and enqueue on the caller's stream.

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "../../include/fs.h"
#include "fs_internal.h"

using namespace fsk;

namespace {

int refuse(int code, const char* why) {
  set_null_error(why);
  return code;
}

constexpr int kMaxTokens = 1 << 30;  // token + split arithmetic stays in 32 bits

int x_type(int32_t dtype) {
  return dtype == FS_DTYPE_F32 ? X_F32 : dtype == FS_DTYPE_BF16 ? X_BF16 : -1;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Null if every pointer is memory of the current device.
const char* not_here(std::initializer_list<const void*> ptrs) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return "no CUDA device";
  for (const void* p : ptrs) {
    if (!p) continue;
    cudaPointerAttributes at{};
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return "not a device pointer";
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
      return "not a device pointer";
    if (at.type == cudaMemoryTypeDevice && at.device != dev) return "memory of another device";
  }
  return nullptr;
}

const char* bad_cache(const fs_kv_q8* c) {
  if (!c) return "NULL cache";
  if (!kv_q8_supports(c->head_dim)) return "head_dim must be 64, 128 or 256";
  if (c->n_kv_heads < 1 || c->page_size < 1 || c->max_pages < 1)
    return "n_kv_heads, page_size and max_pages must be positive";
  if ((int64_t)c->max_pages * c->page_size > kMaxTokens) return "a lane may hold 2^30 tokens";
  if (c->n_pages > 0 && (int64_t)c->n_kv_heads * c->page_size > (((int64_t)1 << 32) - 2) / c->n_pages)
    return "the cache may hold 2^32 - 2 rows";
  return nullptr;
}
const char* bad_buffers(const fs_kv_q8* c) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table) return "NULL cache buffer";
  if (c->n_pages < 1 || c->n_lanes < 1) return "n_pages and n_lanes must be positive";
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return "codes must be 16-byte aligned";
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->page_table, 4))
    return "scales and page table must be 4-byte aligned";
  return nullptr;
}

KvQ8 view(const fs_kv_q8* c) {
  KvQ8 v;
  v.k = c->k;
  v.v = c->v;
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.page_table = c->page_table;
  v.n_pages = c->n_pages;
  v.Hkv = c->n_kv_heads;
  v.page_size = c->page_size;
  v.hd = c->head_dim;
  v.n_lanes = c->n_lanes;
  v.max_pages = c->max_pages;
  v.by_page = FastDiv((uint32_t)c->page_size);
  v.by_head = FastDiv((uint32_t)c->n_kv_heads);
  return v;
}

const char* bad_rows(const void* p, int64_t stride, int64_t width, int xt) {
  if (!p) return "NULL rows";
  if (!aligned(p, xt == X_F32 ? 4 : 2)) return "rows must be aligned to their type";
  if (stride < width) return "rows overlap (stride below the row's width)";
  return nullptr;
}

const char* bad_rope(const float* c, const float* s, int32_t len) {
  if (!c != !s) return "rope_cos and rope_sin go together";
  if (c && (len < 1 || !aligned(c, 4) || !aligned(s, 4))) return "bad rotation tables";
  return nullptr;
}

// Blocks a grid may have along x is 2^31 - 1; rows and KV heads share it.
bool grid_fits(int64_t n, int64_t heads) { return n * heads <= (int64_t)INT32_MAX; }

int launched(const Launched& l) {
  if (l.error != cudaSuccess) {
    cudaGetLastError();  // reported here
    return refuse(FS_ERR_CUDA, cudaGetErrorString(l.error));
  }
  return l.kernels > 0 ? FS_OK : refuse(FS_ERR_CUDA, "no kernel for this shape");
}

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Bytes from the first value of n rows to the end of the last.
struct Span {
  const char* from;
  int64_t stride, width, bytes;  // stride and width of a row, in bytes
  Span(const void* p, int64_t stride_, int64_t width_, int64_t n, int64_t e)
      : from(static_cast<const char*>(p)), stride(stride_ * e), width(width_ * e),
        bytes(n > 0 ? (n - 1) * stride_ * e + width_ * e : 0) {}
};
// Whether a value of one lies in the other. Rows of one stride may interleave (columns of
// one panel); spans of two strides that meet count as overlapping.
bool overlap(const Span& a, const Span& b) {
  if (!a.from || !b.from || a.bytes == 0 || b.bytes == 0) return false;
  const Span& lo = a.from <= b.from ? a : b;
  const Span& hi = a.from <= b.from ? b : a;
  const int64_t d = hi.from - lo.from;
  if (d >= lo.bytes) return false;
  if (lo.stride != hi.stride) return true;
  const int64_t r = d % lo.stride;
  return r < lo.width || r + hi.width > lo.stride;
}

struct AttnPlan {
  int max_len, split_len, n_splits;
  int64_t bytes;
};

// Splits and workspace of one attention call; why is set when it is refused.
int plan_attention(const fs_kv_q8* c, int32_t n, int32_t n_heads, int32_t max_len,
                   int32_t split_len, AttnPlan* p) {
  if (const char* why = bad_cache(c)) return refuse(FS_ERR_ARG, why);
  if (n < 0 || n > 65535) return refuse(FS_ERR_ARG, "n outside [0, 65535]");
  if (n_heads < 1 || n_heads % c->n_kv_heads || n_heads / c->n_kv_heads > 8)
    return refuse(FS_ERR_ARG, "n_heads must be 1 to 8 times n_kv_heads");
  if (n_heads > 65535) return refuse(FS_ERR_ARG, "too many heads");
  if (max_len < 0) return refuse(FS_ERR_ARG, "negative max_len");
  if (split_len < 0 || split_len % 64 || split_len > kMaxTokens)
    return refuse(FS_ERR_ARG, "split_len must be a multiple of 64, at most 2^30");
  const int cap = c->max_pages * c->page_size;
  p->max_len = max_len == 0 ? cap : std::min<int>(max_len, cap);
  p->split_len = split_len;
  if (!split_len) {
    const int sms = device_sms();
    if (!sms) return refuse(FS_ERR_CUDA, "no CUDA device");
    p->split_len = attn_q8_split_len(n, c->n_kv_heads, c->head_dim, p->max_len, sms);
    // a lane of more than 8192 splits: longer ones
    const int64_t least = ((int64_t)p->max_len + kMaxQ8Splits - 1) / kMaxQ8Splits;
    if (p->split_len < least) p->split_len = (int)((least + 127) / 128 * 128);
  }
  const int64_t ns = ((int64_t)p->max_len + p->split_len - 1) / p->split_len;
  if (ns > kMaxQ8Splits) return refuse(FS_ERR_ARG, "split_len too small for max_len (8192 splits)");
  p->n_splits = (int)ns;
  p->bytes = ns <= 1 ? 0 : (int64_t)n * ns * n_heads * (c->head_dim + 2) * 4;
  return FS_OK;
}

}  // namespace

extern "C" {

int fs_kv_q8_append(const fs_kv_q8* cache, const void* k, const void* v, int64_t k_stride,
                    int64_t v_stride, int32_t dtype, const int32_t* lanes,
                    const int32_t* positions, int32_t n, const float* rope_cos,
                    const float* rope_sin, int32_t rope_len, void* stream) {
  const char* why = bad_cache(cache);
  if (!why) why = bad_buffers(cache);
  if (why) return refuse(FS_ERR_ARG, why);
  const int xt = x_type(dtype);
  if (xt < 0) return refuse(FS_ERR_ARG, "dtype must be F32 or BF16");
  if (n < 0) return refuse(FS_ERR_ARG, "negative n");
  if ((why = bad_rope(rope_cos, rope_sin, rope_len))) return refuse(FS_ERR_ARG, why);
  if (n == 0) return FS_OK;
  const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
  if ((why = bad_rows(k, k_stride, width, xt)) || (why = bad_rows(v, v_stride, width, xt)))
    return refuse(FS_ERR_ARG, why);
  if (!lanes || !positions || !aligned(lanes, 4) || !aligned(positions, 4))
    return refuse(FS_ERR_ARG, "NULL or misaligned lanes or positions");
  if (!grid_fits(n, cache->n_kv_heads)) return refuse(FS_ERR_ARG, "too many rows");
  if ((why = not_here({cache->k, cache->v, cache->k_scale, cache->v_scale, cache->page_table, k, v,
                       lanes, positions, rope_cos, rope_sin})))
    return refuse(FS_ERR_ARG, why);
  return launched(launch_kv_q8_append(view(cache), k, v, k_stride, v_stride, xt, false, lanes,
                                      positions, n, rope_cos, rope_sin, rope_len, (cudaStream_t)stream));
}

int fs_kv_q8_read(const fs_kv_q8* cache, const int32_t* lanes, const int32_t* positions,
                  int32_t n, void* k_out, void* v_out, int64_t k_stride, int64_t v_stride,
                  int32_t dtype, void* stream) {
  const char* why = bad_cache(cache);
  if (!why) why = bad_buffers(cache);
  if (why) return refuse(FS_ERR_ARG, why);
  const int xt = x_type(dtype);
  if (xt < 0) return refuse(FS_ERR_ARG, "dtype must be F32 or BF16");
  if (n < 0) return refuse(FS_ERR_ARG, "negative n");
  if (n == 0 || (!k_out && !v_out)) return FS_OK;
  const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
  if ((k_out && (why = bad_rows(k_out, k_stride, width, xt))) ||
      (v_out && (why = bad_rows(v_out, v_stride, width, xt))))
    return refuse(FS_ERR_ARG, why);
  if (!lanes || !positions || !aligned(lanes, 4) || !aligned(positions, 4))
    return refuse(FS_ERR_ARG, "NULL or misaligned lanes or positions");
  if (!grid_fits(n, cache->n_kv_heads)) return refuse(FS_ERR_ARG, "too many rows");
  if ((why = not_here({cache->k, cache->v, cache->k_scale, cache->v_scale, cache->page_table,
                       k_out, v_out, lanes, positions})))
    return refuse(FS_ERR_ARG, why);
  return launched(launch_kv_q8_read(view(cache), lanes, positions, n, k_out, v_out, k_stride,
                                    v_stride, xt, (cudaStream_t)stream));
}

int64_t fs_kv_q8_attention_workspace(const fs_kv_q8* cache, int32_t n, int32_t n_heads,
                                     int32_t max_len, int32_t split_len) {
  AttnPlan p{};
  const int rc = plan_attention(cache, n, n_heads, max_len, split_len, &p);
  return rc ? rc : p.bytes;
}

int fs_kv_q8_attention(const fs_kv_q8* cache, const void* q, int64_t q_stride,
                       const int32_t* lanes, const int32_t* lengths, int32_t n,
                       int32_t n_heads, int32_t max_len, float scale, const float* rope_cos,
                       const float* rope_sin, int32_t rope_len, void* out, int64_t out_stride,
                       int32_t dtype, int32_t split_len, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  const char* why = bad_cache(cache);
  if (!why) why = bad_buffers(cache);
  if (why) return refuse(FS_ERR_ARG, why);
  const int xt = x_type(dtype);
  if (xt < 0) return refuse(FS_ERR_ARG, "dtype must be F32 or BF16");
  if (!std::isfinite(scale)) return refuse(FS_ERR_ARG, "scale must be finite");
  if ((why = bad_rope(rope_cos, rope_sin, rope_len))) return refuse(FS_ERR_ARG, why);
  AttnPlan p{};
  if (const int rc = plan_attention(cache, n, n_heads, max_len, split_len, &p)) return rc;
  if (n == 0) return FS_OK;
  if (rope_cos && p.max_len > rope_len)
    return refuse(FS_ERR_ARG, "max_len exceeds the rotation tables");
  const int64_t width = (int64_t)n_heads * cache->head_dim;
  if ((why = bad_rows(q, q_stride, width, xt)) || (why = bad_rows(out, out_stride, width, xt)))
    return refuse(FS_ERR_ARG, why);
  if (!lanes || !lengths || !aligned(lanes, 4) || !aligned(lengths, 4))
    return refuse(FS_ERR_ARG, "NULL or misaligned lanes or lengths");
  if (cache->n_kv_heads > 65535 || p.n_splits < 1) return refuse(FS_ERR_ARG, "too many KV heads");
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes))
    return refuse(FS_ERR_SCRATCH, "workspace smaller than fs_kv_q8_attention_workspace says");
  if (p.bytes > 0 && !aligned(workspace, 16))
    return refuse(FS_ERR_ARG, "workspace must be 16-byte aligned");
  if ((why = not_here({cache->k, cache->v, cache->k_scale, cache->v_scale, cache->page_table, q,
                       out, lanes, lengths, rope_cos, rope_sin, p.bytes ? workspace : nullptr})))
    return refuse(FS_ERR_ARG, why);
  AttnQ8 a{};
  a.kv = view(cache);
  a.q = q; a.q_stride = q_stride;
  a.lanes = lanes; a.lens = lengths;
  a.n = n; a.H = n_heads; a.max_len = p.max_len; a.scale = scale;
  a.rc = rope_cos; a.rs = rope_sin;
  a.out = out; a.out_stride = out_stride;
  a.split_len = p.split_len; a.n_splits = p.n_splits;
  a.part_acc = static_cast<float*>(workspace);
  a.part_ml = a.part_acc ? a.part_acc + (int64_t)n * p.n_splits * n_heads * cache->head_dim : nullptr;
  const int sms = device_sms();
  if (!sms) return refuse(FS_ERR_CUDA, "no CUDA device");
  return launched(launch_attention_q8(a, xt, xt, false, sms, (cudaStream_t)stream));
}

int fs_verify_draft(const float* logits, int64_t logits_stride, int32_t n_rows, int32_t vocab,
                    const int32_t* row_start, int32_t n_seqs, const int32_t* draft,
                    const float* draft_probs, int64_t probs_stride, const float* temps,
                    const float* u_accept, const float* u_sample, int32_t* n_accepted,
                    int32_t* next_token, void* stream) {
  if (n_rows < 0 || n_seqs < 0) return refuse(FS_ERR_ARG, "negative n_rows or n_seqs");
  if (vocab < 1 || vocab > kMaxTokens) return refuse(FS_ERR_ARG, "vocab outside [1, 2^30]");
  if (n_seqs > INT32_MAX / 8) return refuse(FS_ERR_ARG, "too many sequences");
  if (n_seqs == 0) return FS_OK;
  if (n_rows > 0) {
    const char* why = bad_rows(logits, logits_stride, vocab, X_F32);
    if (!why && draft_probs) why = bad_rows(draft_probs, probs_stride, vocab, X_F32);
    if (why) return refuse(FS_ERR_ARG, why);
    if (!draft || !u_accept) return refuse(FS_ERR_ARG, "NULL draft or u_accept");
  }
  if (!row_start || !temps || !u_sample || !n_accepted || !next_token)
    return refuse(FS_ERR_ARG, "NULL argument array");
  for (const void* p : {(const void*)row_start, (const void*)draft, (const void*)temps,
                        (const void*)u_accept, (const void*)u_sample, (const void*)n_accepted,
                        (const void*)next_token})
    if (!aligned(p, 4)) return refuse(FS_ERR_ARG, "arrays must be 4-byte aligned");
  if (const char* why = not_here({logits, row_start, draft, draft_probs, temps, u_accept, u_sample,
                                  n_accepted, next_token}))
    return refuse(FS_ERR_ARG, why);
  VerifyArgs a{};
  a.logits = logits; a.ld_logits = logits_stride; a.n_rows = n_rows; a.V = vocab;
  a.row_start = row_start; a.n_seqs = n_seqs;
  a.draft = draft; a.probs = draft_probs; a.ld_probs = probs_stride;
  a.temps = temps; a.u_accept = u_accept; a.u_sample = u_sample;
  a.n_accepted = n_accepted; a.next_token = next_token;
  const int sms = device_sms();
  if (!sms) return refuse(FS_ERR_CUDA, "no CUDA device");
  return launched(launch_verify(a, sms, (cudaStream_t)stream));
}

int fs_pages_update(int32_t* holders, int32_t n_pages, int32_t* page_table, int32_t* lengths,
                    int32_t n_lanes, int32_t max_pages, int32_t page_size, const int32_t* keep,
                    const int32_t* grow, int32_t* row_start, int32_t* row_lane,
                    int32_t* row_position, int32_t* row_length, int64_t* row_slot,
                    int32_t max_rows, int32_t* status, void* stream) {
  if (n_pages < 1 || max_pages < 1 || page_size < 1)
    return refuse(FS_ERR_ARG, "n_pages, max_pages and page_size must be positive");
  if ((int64_t)max_pages * page_size > kMaxTokens) return refuse(FS_ERR_ARG, "a lane may hold 2^30 tokens");
  if (n_lanes < 1 || n_lanes > kMaxPageLanes) return refuse(FS_ERR_ARG, "n_lanes outside [1, 8192]");
  if (max_rows < 0) return refuse(FS_ERR_ARG, "negative max_rows");
  if (!holders || !page_table || !lengths || !grow || !row_start || !status)
    return refuse(FS_ERR_ARG, "NULL argument array");
  for (const void* p : {(const void*)holders, (const void*)page_table, (const void*)lengths,
                        (const void*)keep, (const void*)grow, (const void*)row_start,
                        (const void*)row_lane, (const void*)row_position, (const void*)row_length,
                        (const void*)status})
    if (!aligned(p, 4)) return refuse(FS_ERR_ARG, "arrays must be 4-byte aligned");
  if (!aligned(row_slot, 8)) return refuse(FS_ERR_ARG, "row_slot must be 8-byte aligned");
  const Span rw[] = {{holders, n_pages, n_pages, 1, 4}, {page_table, max_pages, max_pages, n_lanes, 4},
                     {lengths, n_lanes, n_lanes, 1, 4}, {row_start, n_lanes + 1, n_lanes + 1, 1, 4},
                     {row_lane, max_rows, max_rows, 1, 4}, {row_position, max_rows, max_rows, 1, 4},
                     {row_length, max_rows, max_rows, 1, 4}, {row_slot, max_rows, max_rows, 1, 8},
                     {status, 4, 4, 1, 4}};
  const Span ro[] = {{keep, n_lanes, n_lanes, 1, 4}, {grow, n_lanes, n_lanes, 1, 4}};
  const int n_rw = (int)(sizeof(rw) / sizeof(rw[0]));
  for (int i = 0; i < n_rw; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(rw[i], rw[j])) return refuse(FS_ERR_ARG, "arrays overlap");
    if (overlap(rw[i], ro[0]) || overlap(rw[i], ro[1])) return refuse(FS_ERR_ARG, "arrays overlap");
  }
  if (const char* why = not_here({holders, page_table, lengths, keep, grow, row_start, row_lane,
                                  row_position, row_length, row_slot, status}))
    return refuse(FS_ERR_ARG, why);
  PagesArgs a{};
  a.holders = holders; a.table = page_table; a.lengths = lengths; a.keep = keep; a.grow = grow;
  a.n_pages = n_pages; a.n_lanes = n_lanes; a.max_pages = max_pages; a.page_size = page_size;
  a.by_page = FastDiv((uint32_t)page_size);
  a.row_start = row_start; a.row_lane = row_lane; a.row_position = row_position;
  a.row_length = row_length; a.row_slot = row_slot; a.max_rows = max_rows; a.status = status;
  a.code_full = FS_ERR_KV_FULL; a.code_rows = FS_ERR_SCRATCH; a.code_shared = FS_ERR_STATE;
  return launched(launch_pages(a, (cudaStream_t)stream));
}

int fs_rope_frequencies(int32_t rotary_dim, double theta, const fs_rope_scaling* scaling,
                        double* inv_freq, double* factor_out) {
  if (!inv_freq || !factor_out) return refuse(FS_ERR_ARG, "NULL output");
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > kMaxRotary)
    return refuse(FS_ERR_ARG, "rotary_dim must be even, 2 to 512");
  if (!(theta > 0) || !std::isfinite(theta)) return refuse(FS_ERR_ARG, "theta must be positive");
  const int kind = scaling ? scaling->kind : FS_ROPE_SCALING_NONE;
  if (kind < FS_ROPE_SCALING_NONE || kind > FS_ROPE_SCALING_BANDS)
    return refuse(FS_ERR_ARG, "unknown kind of scaling");
  const double by = kind ? scaling->factor : 1.0;
  if (!(by > 0) || !std::isfinite(by)) return refuse(FS_ERR_ARG, "the scaling's factor must be positive");
  const bool parts = kind == FS_ROPE_SCALING_RAMP || kind == FS_ROPE_SCALING_BANDS;
  if (parts && (scaling->original < 1 || !(scaling->low > 0) || !(scaling->low < scaling->high) ||
                !std::isfinite(scaling->high)))
    return refuse(FS_ERR_ARG, "the scaling needs original > 0 and 0 < low < high");
  if (kind == FS_ROPE_SCALING_RAMP && !(theta > 1)) return refuse(FS_ERR_ARG, "a ramp needs theta > 1");
  const double pi = 3.14159265358979323846, r = rotary_dim;
  const double base = kind == FS_ROPE_SCALING_BASE && rotary_dim > 2
                          ? theta * std::pow(by, r / (r - 2)) : theta;
  double lo = 0, hi = 1;  // of the ramp
  if (kind == FS_ROPE_SCALING_RAMP) {
    auto pair_with = [&](double turns) {
      return r * std::log(scaling->original / (2 * pi * turns)) / (2 * std::log(theta));
    };
    lo = std::max(std::floor(pair_with(scaling->high)), 0.0);
    hi = std::min(std::ceil(pair_with(scaling->low)), r - 1);
    if (!(hi > lo)) hi = lo + 0.001;
  }
  for (int j = 0; j < rotary_dim / 2; ++j) {
    const double f = std::pow(base, -2.0 * j / r);
    double keep = 1;  // the part of f that is not scaled
    if (kind == FS_ROPE_SCALING_LINEAR) keep = 0;
    if (kind == FS_ROPE_SCALING_RAMP) keep = 1 - std::min(1.0, std::max(0.0, (j - lo) / (hi - lo)));
    if (kind == FS_ROPE_SCALING_BANDS) {
      const double turns = scaling->original * f / (2 * pi);
      keep = std::min(1.0, std::max(0.0, (turns - scaling->low) / (scaling->high - scaling->low)));
    }
    inv_freq[j] = f / by * (1 - keep) + f * keep;
  }
  *factor_out = kind == FS_ROPE_SCALING_RAMP && by > 1 ? 0.1 * std::log(by) + 1 : 1.0;
  return FS_OK;
}

int fs_rope(const void* q, int64_t q_stride, int32_t n_heads, const void* k, int64_t k_stride,
            int32_t n_kv_heads, int32_t n, int32_t head_dim, int32_t dtype,
            const int32_t* positions, const double* inv_freq, int32_t rotary_dim, double factor,
            int32_t flags, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
            void* stream) {
  const int xt = x_type(dtype);
  if (xt < 0) return refuse(FS_ERR_ARG, "dtype must be F32 or BF16");
  if (n < 0) return refuse(FS_ERR_ARG, "negative n");
  if (n_heads < 1 || n_heads > 65535) return refuse(FS_ERR_ARG, "n_heads outside [1, 65535]");
  if (k ? n_kv_heads < 1 || n_kv_heads > 65535 : n_kv_heads != 0 || k_out)
    return refuse(FS_ERR_ARG, "k, k_out and n_kv_heads go together");
  if (head_dim < 2 || head_dim > 1024) return refuse(FS_ERR_ARG, "head_dim outside [2, 1024]");
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim || rotary_dim > kMaxRotary)
    return refuse(FS_ERR_ARG, "rotary_dim must be even, 2 to head_dim and at most 512");
  if (flags & ~(FS_ROPE_INTERLEAVED | FS_ROPE_INVERSE)) return refuse(FS_ERR_ARG, "unknown flag");
  if (!std::isfinite(factor) || !std::isfinite((float)factor))
    return refuse(FS_ERR_ARG, "factor must be a finite f32 number");
  if (!inv_freq) return refuse(FS_ERR_ARG, "NULL inv_freq");
  for (int j = 0; j < rotary_dim / 2; ++j)
    if (!(std::fabs(inv_freq[j]) <= 1 << 20)) return refuse(FS_ERR_ARG, "inv_freq must be within 2^20");
  if (n == 0) return FS_OK;
  const int64_t e = xt == X_F32 ? 4 : 2;
  const int64_t qw = (int64_t)n_heads * head_dim, kw = (int64_t)n_kv_heads * head_dim;
  const char* why = bad_rows(q, q_stride, qw, xt);
  if (!why) why = bad_rows(q_out, q_out_stride, qw, xt);
  if (!why && k) why = bad_rows(k, k_stride, kw, xt);
  if (!why && k) why = bad_rows(k_out, k_out_stride, kw, xt);
  if (why) return refuse(FS_ERR_ARG, why);
  if (!positions || !aligned(positions, 4)) return refuse(FS_ERR_ARG, "NULL or misaligned positions");
  if ((q_out == q && n > 1 && q_out_stride != q_stride) || (k && k_out == k && n > 1 && k_out_stride != k_stride))
    return refuse(FS_ERR_ARG, "in place the strides must be the same");
  const Span qi(q, q_stride, qw, n, e), qo(q_out, q_out_stride, qw, n, e), ki(k, k_stride, kw, n, e),
      ko(k_out, k_out_stride, kw, n, e), at(positions, n, n, 1, 4);
  if ((q_out != q && overlap(qi, qo)) || (k_out != k && overlap(ki, ko)) || overlap(qo, ko) ||
      overlap(qo, ki) || overlap(ko, qi) || overlap(qo, at) || overlap(ko, at))
    return refuse(FS_ERR_ARG, "buffers overlap");
  if ((why = not_here({q, k, q_out, k_out, positions}))) return refuse(FS_ERR_ARG, why);
  RopeArgs a{};
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.qo_stride = q_out_stride; a.ko_stride = k_out_stride;
  a.positions = positions;
  a.n = n; a.H = n_heads; a.Hkv = n_kv_heads; a.hd = head_dim; a.rot = rotary_dim;
  a.factor = (float)factor;
  a.inverse = (flags & FS_ROPE_INVERSE) != 0;
  // f / (2 pi) as a fraction of 2^64: the product by a pair of doubles, then its bits
  const double ih = 0.15915494309189535, il = -9.839338337591243e-18;  // 1 / (2 pi)
  for (int j = 0; j < rotary_dim / 2; ++j) {
    const double f = inv_freq[j], p = f * ih, pe = std::fma(f, ih, -p) + f * il;
    const double part = p - std::trunc(p);  // exact
    // the top 32 bits of the fraction, then what is left of it and pe
    const double top = std::floor(part * 0x1p32);
    const double rest = (part * 0x1p32 - top) * 0x1p32 + pe * 0x1p64;
    a.F[j] = ((uint64_t)(int64_t)top << 32) + (uint64_t)(int64_t)std::llrint(rest);
  }
  const int sms = device_sms();
  if (!sms) return refuse(FS_ERR_CUDA, "no CUDA device");
  return launched(launch_rope(a, xt, (flags & FS_ROPE_INTERLEAVED) != 0, sms, (cudaStream_t)stream));
}

int fs_lora_add(const void* x, int64_t x_stride, int32_t x_dtype, const int32_t* adapter,
                int32_t n, int32_t K, int32_t N, const uint16_t* A, const uint16_t* B,
                const float* scale, int32_t n_adapters, int32_t rank, const void* base,
                int64_t base_stride, void* out, int64_t out_stride, int32_t y_dtype,
                void* stream) {
  const int xt = x_type(x_dtype), yt = x_type(y_dtype);
  if (xt < 0 || yt < 0) return refuse(FS_ERR_ARG, "x_dtype and y_dtype must be F32 or BF16");
  if (n < 0) return refuse(FS_ERR_ARG, "negative n");
  if (n_adapters < 1) return refuse(FS_ERR_ARG, "n_adapters must be positive");
  if (rank < 8 || rank % 8 || rank > 128) return refuse(FS_ERR_ARG, "rank must be a multiple of 8, 8 to 128");
  if (K < 8 || K % 8 || K > (1 << 24)) return refuse(FS_ERR_ARG, "K must be a multiple of 8, 8 to 2^24");
  if (N < 1 || N > (1 << 24)) return refuse(FS_ERR_ARG, "N outside [1, 2^24]");
  if (n == 0) return FS_OK;
  const int64_t ex = xt == X_F32 ? 4 : 2, ey = yt == X_F32 ? 4 : 2;
  const char* why = bad_rows(x, x_stride, K, xt);
  if (!why) why = bad_rows(out, out_stride, N, yt);
  if (!why && base) why = bad_rows(base, base_stride, N, yt);
  if (why) return refuse(FS_ERR_ARG, why);
  if (!adapter || !A || !B || !scale) return refuse(FS_ERR_ARG, "NULL adapter array");
  if (!aligned(adapter, 4) || !aligned(scale, 4) || !aligned(A, 16) || !aligned(B, 16))
    return refuse(FS_ERR_ARG, "adapter and scale must be 4-byte, A and B 16-byte aligned");
  if (base == out && n > 1 && base_stride != out_stride)
    return refuse(FS_ERR_ARG, "in place the strides must be the same");
  const Span o(out, out_stride, N, n, ey);
  const int64_t low = (int64_t)n_adapters * rank;
  if ((base != out && overlap(o, Span(base, base_stride, N, n, ey))) ||
      overlap(o, Span(x, x_stride, K, n, ex)) || overlap(o, Span(adapter, n, n, 1, 4)) ||
      overlap(o, Span(scale, n_adapters, n_adapters, 1, 4)) || overlap(o, Span(A, low * K, low * K, 1, 2)) ||
      overlap(o, Span(B, low * N, low * N, 1, 2)))
    return refuse(FS_ERR_ARG, "buffers overlap");
  if ((why = not_here({x, adapter, A, B, scale, base, out}))) return refuse(FS_ERR_ARG, why);
  LoraArgs a{};
  a.x = x; a.x_stride = x_stride; a.adapter = adapter;
  a.n = n; a.K = K; a.N = N;
  a.A = reinterpret_cast<const __nv_bfloat16*>(A);
  a.B = reinterpret_cast<const __nv_bfloat16*>(B);
  a.scale = scale; a.n_adapters = n_adapters; a.rank = rank;
  a.base = base; a.base_stride = base_stride; a.out = out; a.out_stride = out_stride;
  const int sms = device_sms();
  if (!sms) return refuse(FS_ERR_CUDA, "no CUDA device");
  return launched(launch_lora(a, xt, yt, sms, (cudaStream_t)stream));
}

int fs_sample_filtered(const float* logits, int64_t logits_stride, int32_t n, int32_t vocab,
                       const float* temps, const int32_t* top_k, const float* top_p,
                       const float* min_p, const float* u, int32_t* tokens, int32_t* kept,
                       void* stream) {
  if (n < 0 || n > INT32_MAX / 8) return refuse(FS_ERR_ARG, "n outside [0, 2^28)");
  if (vocab < 1 || vocab > (1 << 20)) return refuse(FS_ERR_ARG, "vocab outside [1, 2^20]");
  if (n == 0) return FS_OK;
  if (const char* why = bad_rows(logits, logits_stride, vocab, X_F32)) return refuse(FS_ERR_ARG, why);
  if (!temps || !u || !tokens) return refuse(FS_ERR_ARG, "NULL argument array");
  for (const void* p : {(const void*)temps, (const void*)top_k, (const void*)top_p, (const void*)min_p,
                        (const void*)u, (const void*)tokens, (const void*)kept})
    if (!aligned(p, 4)) return refuse(FS_ERR_ARG, "arrays must be 4-byte aligned");
  const Span t(tokens, n, n, 1, 4), k(kept, n, n, 1, 4), z(logits, logits_stride, vocab, n, 4);
  if (overlap(t, k) || overlap(t, z) || overlap(k, z)) return refuse(FS_ERR_ARG, "arrays overlap");
  for (const void* p : {(const void*)temps, (const void*)top_k, (const void*)top_p, (const void*)min_p,
                        (const void*)u})
    if (overlap(t, Span(p, n, n, 1, 4)) || overlap(k, Span(p, n, n, 1, 4)))
      return refuse(FS_ERR_ARG, "arrays overlap");
  if (const char* why = not_here({logits, temps, top_k, top_p, min_p, u, tokens, kept}))
    return refuse(FS_ERR_ARG, why);
  FilteredArgs a{};
  a.logits = logits; a.ld = logits_stride; a.n = n; a.V = vocab;
  a.temps = temps; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p; a.u = u;
  a.tokens = tokens; a.kept = kept;
  const int sms = device_sms();
  if (!sms) return refuse(FS_ERR_CUDA, "no CUDA device");
  return launched(launch_sample_filtered(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
