// C entry points of the operators that work on the caller's device buffers
// (include/fs.h): the 8-bit paged KV cache and draft verification. They check
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

}  // extern "C"
