// attn_paged_api.cu -- the C ABI of include/attn_paged.h: argument checks and
// launches.  Every check runs before anything is queued; nothing here
// allocates memory.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_internal.h"
#include "attn_testing.h"

namespace attnpipe {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

attn_status_t take_cache(const attn_kv_cache_t* c, KvCache* out) {
  if (!c || !c->k || !c->v || !c->block_table) return ATTN_ERR_INVALID_ARG;
  if (c->B <= 0 || c->H_kv <= 0 || c->D <= 0 || c->num_pages <= 0 || c->page_size <= 0 ||
      c->max_blocks <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (c->format != ATTN_KV_BF16 && c->format != ATTN_KV_INT4) return ATTN_ERR_INVALID_ARG;
  if (c->page_size % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->B > 65535 || c->H_kv > 32767) return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)c->max_blocks * c->page_size >= (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  // pages times heads index the pool's tensor map
  if ((int64_t)c->num_pages * c->H_kv >= (1ll << 31)) return ATTN_ERR_UNSUPPORTED;
  // byte offsets are 64-bit; the pool must fit them
  if ((int64_t)c->num_pages * c->H_kv >= (1ll << 46) / ((int64_t)c->page_size * 256))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->block_table))
    return ATTN_ERR_MISALIGNED;
  out->k = static_cast<const uint8_t*>(c->k);
  out->v = static_cast<const uint8_t*>(c->v);
  out->table = c->block_table;
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->blocks_per_page = c->page_size / 16;
  out->max_blocks = c->max_blocks;
  out->B = c->B;
  out->H_kv = c->H_kv;
  out->capacity = c->max_blocks * c->page_size;
  return ATTN_OK;
}

// The strides of dimensions of size 1 are not looked at (and stored as 0).
attn_status_t take_tensor(const attn_bhsd_t* t, int B, int H, int S, KvTensor* out) {
  if (!t || !t->data) return ATTN_ERR_INVALID_ARG;
  out->data = static_cast<const uint16_t*>(t->data);
  out->sb = B > 1 ? t->stride_b : 0;
  out->sh = H > 1 ? t->stride_h : 0;
  out->ss = S > 1 ? t->stride_s : 0;
  if (!aligned16(t->data) || out->sb % 8 != 0 || out->sh % 8 != 0 || out->ss % 8 != 0)
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

// Query rows to a tile: the smallest that holds a KV head's rows, at most 64.
int tile_rows(int group, int S_q) {
  const int64_t rows = (int64_t)group * S_q;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

constexpr size_t kLeastWorkspace = 256;   // reported where none is used: 0 says invalid

// CTAs that may write parts to the workspace: none where an item is kept whole.
int64_t part_ctas(int64_t B, int64_t H_kv, int64_t rows, int tile, int64_t max_keys) {
  if (max_keys <= kPagedWholeKeys) return 0;
  const int64_t units =
      B * H_kv * ((rows + tile - 1) / tile) * ((max_keys + kPagedUnit - 1) / kPagedUnit);
  return units < kPagedMaxCtas ? units : kPagedMaxCtas;
}

size_t part_bytes(int64_t ctas, int tile, int D) {
  return (size_t)ctas * (2 * tile * (D + 1) * sizeof(float) + sizeof(int4));
}

// The sizes of a paged attention: ATTN_OK where its rows and tiles can be
// indexed.
attn_status_t check_rows(int B, int H_q, int H_kv, int S_q) {
  if (B <= 0 || H_q <= 0 || H_kv <= 0 || S_q <= 0 || H_q % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)(H_q / H_kv) * S_q;
  if (rows >= (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  // items, with what each counts for apart from its keys, are counted in an int
  const int tile = tile_rows(H_q / H_kv, S_q);
  if (((rows + tile - 1) / tile) * H_kv * B * (kPagedItemKeys / kPagedUnit + 1) >=
      (1ll << 31))
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn_status_t paged_impl(const attn_kv_cache_t* cache, const attn_bhsd_t* q, void* o, float* lse,
                         const int* lens, const int* q_lens, void* workspace,
                         size_t workspace_bytes, int H_q, int S_q, int causal, float scale,
                         attn_stream_t stream, int drop_stage = -1,
                         unsigned long long timeout_ns = kDefaultTimeoutNs) {
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  attn_status_t st = take_cache(cache, &p.cache);
  if (st != ATTN_OK) return st;
  if (!o || !lse || !lens) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if ((st = check_rows(cache->B, H_q, cache->H_kv, S_q)) != ATTN_OK) return st;
  if ((st = take_tensor(q, cache->B, H_q, S_q, &p.q)) != ATTN_OK) return st;
  if (!aligned16(o) || !aligned4(lse) || !aligned4(lens) || !aligned4(q_lens) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return ATTN_ERR_MISALIGNED;
  p.group = H_q / cache->H_kv;
  const int rows = tile_rows(p.group, S_q);
  const int64_t parts = part_ctas(cache->B, cache->H_kv, (int64_t)p.group * S_q, rows,
                                  p.cache.capacity);
  if (parts > 0 && (!workspace || workspace_bytes < part_bytes(parts, rows, cache->D)))
    return ATTN_ERR_INVALID_ARG;
  if ((st = check_device()) != ATTN_OK) return st;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.lens = lens;
  p.q_lens = q_lens;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + (size_t)2 * parts * rows * cache->D;
  p.shared = reinterpret_cast<int4*>(p.part_lse + (size_t)2 * parts * rows);
  p.H_q = H_q;
  p.S_q = S_q;
  p.causal = causal;
  // (kept finite)
  const double scale_log2 = (double)scale * 1.4426950408889634;
  p.scale_log2 = (float)std::fmin(std::fmax(scale_log2, -(double)FLT_MAX), (double)FLT_MAX);
  int bits = 0;   // 2^bits >= capacity
  while ((1 << bits) < p.cache.capacity) ++bits;
  p.max_prob = std::ldexp(1.f, -bits);
  p.lead = (float)(bits + 8);
  p.code_base_low = 0x64006400u;
  p.code_base_high = 0x54005400u;
  p.timeout_ns = timeout_ns;
  p.fault_drop_stage = drop_stage;
  if (cache->format == ATTN_KV_BF16) {
    const uint64_t heads = (uint64_t)cache->num_pages * cache->H_kv;
    if (!encode_bf16_map_3d(&p.tm_k, cache->k, cache->D, cache->page_size, heads, 16) ||
        !encode_bf16_map_3d(&p.tm_v, cache->v, cache->D, cache->page_size, heads, 16))
      return ATTN_ERR_CUDA;
  }
  return launch_attn_paged(p, cache->D, cache->format == ATTN_KV_INT4, rows,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attnpipe

using namespace attnpipe;

extern "C" {

attn_status_t attn_kv_append(const attn_kv_cache_t* cache, const attn_bhsd_t* q, void* q_out,
                             const attn_bhsd_t* k, const attn_bhsd_t* v, const int* start,
                             const int* new_lens, const float* cos, const float* sin,
                             int rope_rows, int rot_dim, int interleaved, int H_q, int S,
                             attn_stream_t stream) {
  KvAppendParams p;
  std::memset(&p, 0, sizeof(p));
  attn_status_t st = take_cache(cache, &p.cache);
  if (st != ATTN_OK) return st;
  if (!start || S <= 0 || H_q < 0 || (H_q > 0) != (q != nullptr) || (H_q > 0) != (q_out != nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > cache->D || rot_dim % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!cos || !sin || rope_rows <= 0)) return ATTN_ERR_INVALID_ARG;
  // one grid column a token, one row of blocks per few heads
  if ((int64_t)cache->B * S >= (1ll << 31) || H_q > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!aligned4(start) || !aligned4(new_lens) ||
      (rot_dim > 0 && (!aligned16(cos) || !aligned16(sin))))
    return ATTN_ERR_MISALIGNED;
  if (H_q > 0) {
    if ((st = take_tensor(q, cache->B, H_q, S, &p.q)) != ATTN_OK) return st;
    if (!aligned16(q_out)) return ATTN_ERR_MISALIGNED;
  }
  if ((st = take_tensor(k, cache->B, cache->H_kv, S, &p.k)) != ATTN_OK) return st;
  if ((st = take_tensor(v, cache->B, cache->H_kv, S, &p.v)) != ATTN_OK) return st;
  if ((st = check_device()) != ATTN_OK) return st;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.start = start;
  p.new_lens = new_lens;
  p.cos = cos;
  p.sin = sin;
  p.rope_rows = rope_rows;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved;
  p.H_q = H_q;
  p.S = S;
  return launch_kv_append(p, cache->D, cache->format == ATTN_KV_INT4,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

attn_status_t attn_kv_read(const attn_kv_cache_t* cache, void* k_out, void* v_out,
                           const int* lens, const int* start, int S, attn_stream_t stream) {
  KvReadParams p;
  std::memset(&p, 0, sizeof(p));
  attn_status_t st = take_cache(cache, &p.cache);
  if (st != ATTN_OK) return st;
  if (!k_out || !v_out || !lens || S <= 0) return ATTN_ERR_INVALID_ARG;
  if ((int64_t)cache->B * S >= (1ll << 31)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(lens) || !aligned4(start))
    return ATTN_ERR_MISALIGNED;
  if ((st = check_device()) != ATTN_OK) return st;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.lens = lens;
  p.start = start;
  p.S = S;
  return launch_kv_read(p, cache->D, cache->format == ATTN_KV_INT4,
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

size_t attn_paged_workspace_bytes(int B, int H_q, int H_kv, int S_q, int D, int max_keys) {
  if (check_rows(B, H_q, H_kv, S_q) != ATTN_OK || (D != 64 && D != 128) || max_keys <= 0) return 0;
  const int group = H_q / H_kv, tile = tile_rows(group, S_q);
  const size_t n = part_bytes(part_ctas(B, H_kv, (int64_t)group * S_q, tile, max_keys), tile, D);
  return n < kLeastWorkspace ? kLeastWorkspace : n;
}

attn_status_t attn_fwd_paged(const attn_kv_cache_t* cache, const attn_bhsd_t* q, void* o,
                             float* lse, const int* lens, const int* q_lens, void* workspace,
                             size_t workspace_bytes, int H_q, int S_q, int causal, float scale,
                             attn_stream_t stream) {
  return paged_impl(cache, q, o, lse, lens, q_lens, workspace, workspace_bytes, H_q, S_q, causal,
                    scale, stream);
}

attn_status_t attn_fwd_paged_timeout_test(const attn_kv_cache_t* cache, const attn_bhsd_t* q,
                                          void* o, float* lse, const int* lens,
                                          const int* q_lens, void* workspace,
                                          size_t workspace_bytes, int H_q, int S_q, int causal,
                                          float scale, int drop_stage,
                                          unsigned long long wait_budget_ns,
                                          attn_stream_t stream) {
  if (drop_stage < 0) return ATTN_ERR_INVALID_ARG;
  if (wait_budget_ns < 1000000ull || wait_budget_ns > kDefaultTimeoutNs)
    return ATTN_ERR_INVALID_ARG;
  return paged_impl(cache, q, o, lse, lens, q_lens, workspace, workspace_bytes, H_q, S_q, causal,
                    scale, stream, drop_stage, wait_budget_ns);
}

}  // extern "C"
