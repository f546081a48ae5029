// attn_packed_api.cu -- the C ABI of include/attn_packed.h: argument checks and
// launches.  Every check runs before anything is queued; nothing here
// allocates memory.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_internal.h"
#include "attn_testing.h"

namespace attnpipe {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A [T, H, D] tensor whose strides of dimensions of size 1 are replaced by ones that
// any use of them accepts.
struct Thd {
  uint16_t* data;
  int64_t st, sh;
};

attn_status_t take(const attn_thd_t* t, int T, int H, int D, Thd* out) {
  if (!t || !t->data) return ATTN_ERR_INVALID_ARG;
  out->data = static_cast<uint16_t*>(t->data);
  out->sh = H > 1 ? t->stride_h : D;
  out->st = T > 1 ? t->stride_t : (int64_t)H * out->sh;
  if (!aligned(t->data, 16) || out->st % 8 != 0 || out->sh % 8 != 0) return ATTN_ERR_MISALIGNED;
  // (what a tensor map takes)
  if (out->st <= 0 || out->sh <= 0 || out->st >= (1ll << 38) || out->sh >= (1ll << 38))
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Query tokens of a 128-row tile: as many whole groups of heads as fit, such that a
// tile's first row is a multiple of 4 in the row vectors (copies of 16 bytes).  0 where
// there is no such number.
int tile_positions(int group) {
  if (group > 128 || (group > 32 && group % 4 != 0)) return 0;
  return group % 4 == 0 ? 128 / group : 32 / group * 4;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

attn_status_t check_sizes(const attn_packed_t* s) {
  if (!s || s->B <= 0 || s->T_q <= 0 || s->T_k <= 0 || s->H_q <= 0 || s->H_kv <= 0 || s->D <= 0 ||
      s->H_q % s->H_kv != 0)
    return ATTN_ERR_INVALID_ARG;
  if ((s->causal != 0 && s->causal != 1) || !std::isfinite(s->scale)) return ATTN_ERR_INVALID_ARG;
  if (s->D != 64 && s->D != 128) return ATTN_ERR_UNSUPPORTED;
  const int positions = tile_positions(s->H_q / s->H_kv);
  if (positions == 0 || s->B > 65535 || s->H_kv > 65535) return ATTN_ERR_UNSUPPORTED;
  // tokens and what is counted of them stay within ints
  if (s->T_q >= (1 << 30) || s->T_k >= (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  if (packed_tile_room(s->T_q, s->B, positions, s->H_kv) * 2 * s->H_kv >= INT_MAX ||
      packed_key_room(s->T_k, s->B, s->H_kv) * s->H_kv >= INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  // thread blocks of the backward's row kernels (16 rows each, at least)
  if ((int64_t)s->T_q * s->H_q / 16 >= INT_MAX) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Where the parts of the workspace begin.
struct Layout {
  size_t seq_q, seq_k, first, tiles, keys, tile_parts, tile_lse, key_parts, tile_counters, key_counters;
  size_t group_at;
  size_t nlse, ndelta, dq_acc, end;
  int64_t vec_stride;
  int slots;   // of a K/V head's parts, of each list
};

Layout layout_of(const attn_packed_t& s, bool backward, bool deterministic) {
  const int group = s.H_q / s.H_kv, positions = tile_positions(group);
  Layout l{};
  size_t at = sizeof(PackedHeader);
  const auto part = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  l.seq_q = part((size_t)(s.B + 1) * sizeof(int));
  l.seq_k = part((size_t)(s.B + 1) * sizeof(int));
  l.first = part((size_t)(s.B + 1) * 2 * sizeof(int));
  // Slots for parts, if any entry can be cut.
  const auto cut = [](int64_t blocks, int least) { return 2 * blocks >= 3 * least; };
  const int64_t key_blocks = ((int64_t)s.T_k + 127) / 128;
  const int64_t query_tiles = ((int64_t)s.T_q + positions - 1) / positions;
  l.slots = packed_slots(s.H_kv);
  const size_t heads = (size_t)l.slots * s.H_kv, counters = heads * kPackedCounters * sizeof(int);
  if (!backward || deterministic) {
    l.tiles = part((size_t)packed_tile_room(s.T_q, s.B, positions, s.H_kv) * sizeof(PackedTile));
    l.tile_counters = part(counters);
    if (cut(key_blocks, kPackedLeastTile)) {
      l.tile_parts = part(heads * 256 * s.D * sizeof(float));
      if (!backward) l.tile_lse = part(heads * 256 * sizeof(float));
    }
  }
  if (backward) {
    l.keys = part((size_t)packed_key_room(s.T_k, s.B, s.H_kv) * sizeof(PackedKeys));
    l.group_at = part((size_t)packed_key_room(s.T_k, s.B, s.H_kv) * sizeof(int));
    l.key_counters = part(counters);
    if (cut(query_tiles, packed_least_keys(s.D))) l.key_parts = part(heads * 2 * 128 * s.D * sizeof(float));
    // every sequence's rows from packed_vec0 on, and what a copy of 128 reads past them
    l.vec_stride = (((int64_t)s.T_q + 4ll * s.B + 4) * group + 128 + 3) & ~3ll;
    l.nlse = part((size_t)s.H_kv * l.vec_stride * sizeof(float));
    l.ndelta = part((size_t)s.H_kv * l.vec_stride * sizeof(float));
    if (!deterministic) l.dq_acc = part((size_t)s.T_q * s.H_q * s.D * sizeof(float));
  }
  l.end = at;
  return l;
}

// The sequences' bounds and the workspace, and the plan over them.
attn_status_t take_plan(const attn_packed_t& s, const int* cu_q, const int* cu_k, void* workspace,
                        size_t bytes, const Layout& l, PackedPlan* plan, PackedShape* shape) {
  if (!cu_q || !workspace || bytes < l.end) return ATTN_ERR_INVALID_ARG;
  if (!cu_k && s.T_k != s.T_q) return ATTN_ERR_INVALID_ARG;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(workspace, 256))
    return ATTN_ERR_MISALIGNED;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  const int group = s.H_q / s.H_kv;
  plan->cu_q = cu_q;
  plan->cu_k = cu_k ? cu_k : cu_q;
  plan->B = s.B;
  plan->T_q = s.T_q;
  plan->T_k = s.T_k;
  plan->positions = tile_positions(group);
  plan->over_positions = ((1ull << 40) + plan->positions - 1) / plan->positions;
  plan->over_tile = ((1ull << 40) + 2 * plan->positions - 1) / (2 * plan->positions);
  plan->causal = s.causal;
  plan->head = reinterpret_cast<PackedHeader*>(ws);
  plan->seq_q = reinterpret_cast<int*>(ws + l.seq_q);
  plan->seq_k = cu_k ? reinterpret_cast<int*>(ws + l.seq_k) : plan->seq_q;
  plan->H_kv = s.H_kv;
  plan->least_keys = packed_least_keys(s.D);
  plan->early = 0;
  // (a part that the layout does not have begins at 0, where the header is)
  const auto at = [&](size_t offset) { return offset ? ws + offset : nullptr; };
  plan->first[0] = reinterpret_cast<int*>(ws + l.first);
  plan->first[1] = plan->first[0] + s.B + 1;
  plan->tiles = reinterpret_cast<PackedTile*>(at(l.tiles));
  plan->keys = reinterpret_cast<PackedKeys*>(at(l.keys));
  plan->group_at = reinterpret_cast<int*>(at(l.group_at));
  shape->over_positions = plan->over_positions;
  shape->over_group = ((1ull << 40) + group - 1) / group;
  shape->over_group64 = ~0ull / (unsigned)group + 1;
  plan->counters[0] = reinterpret_cast<int*>(at(l.tile_counters));
  plan->counters[1] = reinterpret_cast<int*>(at(l.key_counters));
  plan->n_counters = l.slots * s.H_kv * kPackedCounters;
  shape->tile_parts = reinterpret_cast<float*>(at(l.tile_parts));
  shape->tile_lse = reinterpret_cast<float*>(at(l.tile_lse));
  shape->key_parts = reinterpret_cast<float*>(at(l.key_parts));
  shape->tile_counters = plan->counters[0];
  shape->key_counters = plan->counters[1];
  shape->head = plan->head;
  shape->next = plan->head->next;
  shape->tiles = plan->tiles;
  shape->keys = plan->keys;
  shape->group = group;
  shape->positions = plan->positions;
  shape->inv_group = (65536 + group - 1) / group;
  shape->T_q = s.T_q;
  shape->T_k = s.T_k;
  return ATTN_OK;
}

bool map_rows(CUtensorMap* map, const Thd& t, const attn_packed_t& s, const PackedShape& sh) {
  return encode_bf16_map_thd(map, t.data, s.D, s.H_q, s.T_q, t.sh, t.st, sh.group, sh.positions);
}
bool map_keys(CUtensorMap* map, const Thd& t, const attn_packed_t& s) {
  return encode_bf16_map_thd(map, t.data, s.D, s.H_kv, s.T_k, t.sh, t.st, 1, 128);
}

attn_status_t done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

attn_status_t fwd_impl(const attn_packed_t* s, const attn_thd_t* q, const attn_thd_t* k,
                       const attn_thd_t* v, const attn_thd_t* o, float* lse,
                       const int* cu_q, const int* cu_k, void* workspace,
                       size_t workspace_bytes, attn_stream_t stream, int drop_block = -1,
                       unsigned long long timeout_ns = kDefaultTimeoutNs) {
  attn_status_t st = check_sizes(s);
  if (st != ATTN_OK) return st;
  Thd tq, tk, tv, to;
  if ((st = take(q, s->T_q, s->H_q, s->D, &tq)) != ATTN_OK ||
      (st = take(k, s->T_k, s->H_kv, s->D, &tk)) != ATTN_OK ||
      (st = take(v, s->T_k, s->H_kv, s->D, &tv)) != ATTN_OK ||
      (st = take(o, s->T_q, s->H_q, s->D, &to)) != ATTN_OK)
    return st;
  if (!lse) return ATTN_ERR_INVALID_ARG;
  if (!aligned(lse, 4)) return ATTN_ERR_MISALIGNED;
  PackedPlan plan;
  PackedFwdParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  const Layout l = layout_of(*s, false, false);
  if ((st = take_plan(*s, cu_q, cu_k, workspace, workspace_bytes, l, &plan, &p.sh)) != ATTN_OK)
    return st;
  if ((st = check_device()) != ATTN_OK) return st;
  if (!map_rows(&p.tm_q, tq, *s, p.sh) || !map_keys(&p.tm_k, tk, *s) || !map_keys(&p.tm_v, tv, *s))
    return ATTN_ERR_CUDA;
  // 32 rows of a tile: whole groups of heads of one token or more, or 32 heads of one
  const int group = p.sh.group, box_heads = group < 32 ? group : 32;
  p.sh.o_boxes = packed_o_boxes(group, p.sh.positions);
  if (p.sh.o_boxes > 0 && !encode_bf16_map_thd(&p.tm_o, to.data, s->D, s->H_q, s->T_q, to.sh, to.st,
                                         box_heads, 32 / box_heads))
    return ATTN_ERR_CUDA;
  p.o = to.data;
  p.o_st = to.st;
  p.o_sh = to.sh;
  p.lse = lse;
  p.B = s->B;
  p.H_q = s->H_q;
  p.H_kv = s->H_kv;
  p.causal = s->causal;
  // (a negative scale runs as -Q K^T times |scale|, as in attn_fwd)
  p.neg_scores = std::signbit(s->scale) ? 1 : 0;
  p.scale_log2 = scale_log2_of(std::fabs(s->scale));
  p.timeout_ns = timeout_ns;
  p.fault_drop_block = drop_block;
  p.num_tiles = (int)(packed_tile_room(s->T_q, s->B, p.sh.positions, s->H_kv) * s->H_kv);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (packed_without_plan(s->B, s->T_q, s->T_k, s->H_kv, p.sh.positions)) {
    p.sh.head = nullptr;
    p.cu_q = plan.cu_q;
    p.cu_k = plan.cu_k;
    p.num_tiles = (int)((s->T_q / (2 * p.sh.positions) + s->B) * s->H_kv);
    return done(launch_attn_fwd_packed(p, s->D, cs));
  }
  const cudaError_t e = launch_packed_plan(plan, cs);
  return done(e != cudaSuccess ? e : launch_attn_fwd_packed(p, s->D, cs));
}

attn_status_t bwd_impl(const attn_packed_t* s, const attn_thd_t* q, const attn_thd_t* k,
                       const attn_thd_t* v, const attn_thd_t* o, const float* lse,
                       const attn_thd_t* dout, const attn_thd_t* dq, const attn_thd_t* dk,
                       const attn_thd_t* dv, const int* cu_q, const int* cu_k,
                       void* workspace, size_t workspace_bytes, int deterministic,
                       attn_stream_t stream, int drop_item = -1,
                       unsigned long long timeout_ns = kDefaultTimeoutNs) {
  attn_status_t st = check_sizes(s);
  if (st != ATTN_OK) return st;
  if (deterministic != 0 && deterministic != 1) return ATTN_ERR_INVALID_ARG;
  Thd tq, tk, tv, to, tdo, tdq, tdk, tdv;
  if ((st = take(q, s->T_q, s->H_q, s->D, &tq)) != ATTN_OK ||
      (st = take(k, s->T_k, s->H_kv, s->D, &tk)) != ATTN_OK ||
      (st = take(v, s->T_k, s->H_kv, s->D, &tv)) != ATTN_OK ||
      (st = take(o, s->T_q, s->H_q, s->D, &to)) != ATTN_OK ||
      (st = take(dout, s->T_q, s->H_q, s->D, &tdo)) != ATTN_OK ||
      (st = take(dq, s->T_q, s->H_q, s->D, &tdq)) != ATTN_OK ||
      (st = take(dk, s->T_k, s->H_kv, s->D, &tdk)) != ATTN_OK ||
      (st = take(dv, s->T_k, s->H_kv, s->D, &tdv)) != ATTN_OK)
    return st;
  if (!lse) return ATTN_ERR_INVALID_ARG;
  if (!aligned(lse, 4)) return ATTN_ERR_MISALIGNED;
  PackedPlan plan;
  PackedBwdParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  const Layout l = layout_of(*s, true, deterministic != 0);
  if ((st = take_plan(*s, cu_q, cu_k, workspace, workspace_bytes, l, &plan, &p.sh)) != ATTN_OK)
    return st;
  if ((st = check_device()) != ATTN_OK) return st;
  if (!map_rows(&p.tm_q, tq, *s, p.sh) || !map_rows(&p.tm_do, tdo, *s, p.sh) ||
      !map_keys(&p.tm_k, tk, *s) || !map_keys(&p.tm_v, tv, *s))
    return ATTN_ERR_CUDA;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.nlse2 = reinterpret_cast<float*>(ws + l.nlse);
  p.ndelta = reinterpret_cast<float*>(ws + l.ndelta);
  p.dq_acc = deterministic ? nullptr : reinterpret_cast<float*>(ws + l.dq_acc);
  p.vec_stride = l.vec_stride;
  p.seq_q = plan.seq_q;
  p.dq = tdq.data;
  p.dk = tdk.data;
  p.dv = tdv.data;
  p.o_st = to.st, p.o_sh = to.sh;
  p.do_st = tdo.st, p.do_sh = tdo.sh;
  p.dq_st = tdq.st, p.dq_sh = tdq.sh;
  p.dk_st = tdk.st, p.dk_sh = tdk.sh;
  p.dv_st = tdv.st, p.dv_sh = tdv.sh;
  p.B = s->B;
  p.H_q = s->H_q;
  p.H_kv = s->H_kv;
  p.causal = s->causal;
  p.scale = s->scale;
  p.scale_log2 = scale_log2_of(s->scale);
  p.timeout_ns = timeout_ns;
  p.fault_drop_item = drop_item;
  // (the row vectors of up to 31 sequences need no plan, which then runs beside them)
  plan.early = s->B < 32 ? 1 : 0;
  p.cu_q = plan.early ? plan.cu_q : nullptr;
  return done(launch_attn_bwd_packed(p, plan, s->D, to.data, tdo.data, lse,
                                     (int)packed_tile_room(s->T_q, s->B, p.sh.positions, s->H_kv),
                                     (int)packed_key_room(s->T_k, s->B, s->H_kv),
                                     static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace attnpipe

using namespace attnpipe;

extern "C" {

size_t attn_packed_workspace_bytes(const attn_packed_t* s) {
  return check_sizes(s) == ATTN_OK ? layout_of(*s, false, false).end : 0;
}

size_t attn_packed_bwd_workspace_bytes(const attn_packed_t* s, int deterministic) {
  if (check_sizes(s) != ATTN_OK || (deterministic != 0 && deterministic != 1)) return 0;
  return layout_of(*s, true, deterministic != 0).end;
}

attn_status_t attn_fwd_packed(const attn_packed_t* s, const attn_thd_t* q, const attn_thd_t* k,
                              const attn_thd_t* v, const attn_thd_t* o, float* lse,
                              const int* cu_q, const int* cu_k, void* workspace,
                              size_t workspace_bytes, attn_stream_t stream) {
  return fwd_impl(s, q, k, v, o, lse, cu_q, cu_k, workspace, workspace_bytes, stream);
}

attn_status_t attn_bwd_packed(const attn_packed_t* s, const attn_thd_t* q, const attn_thd_t* k,
                              const attn_thd_t* v, const attn_thd_t* o, const float* lse,
                              const attn_thd_t* dout, const attn_thd_t* dq, const attn_thd_t* dk,
                              const attn_thd_t* dv, const int* cu_q, const int* cu_k,
                              void* workspace, size_t workspace_bytes, int deterministic,
                              attn_stream_t stream) {
  return bwd_impl(s, q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, workspace, workspace_bytes,
                  deterministic, stream);
}

attn_status_t attn_fwd_packed_timeout_test(const attn_packed_t* s, const attn_thd_t* q,
                                           const attn_thd_t* k, const attn_thd_t* v,
                                           const attn_thd_t* o, float* lse, const int* cu_q,
                                           const int* cu_k, void* workspace,
                                           size_t workspace_bytes, int drop_block,
                                           unsigned long long wait_budget_ns,
                                           attn_stream_t stream) {
  if (drop_block < 0 || wait_budget_ns < 1000000ull || wait_budget_ns > kDefaultTimeoutNs)
    return ATTN_ERR_INVALID_ARG;
  return fwd_impl(s, q, k, v, o, lse, cu_q, cu_k, workspace, workspace_bytes, stream, drop_block,
                  wait_budget_ns);
}

attn_status_t attn_bwd_packed_timeout_test(
    const attn_packed_t* s, const attn_thd_t* q, const attn_thd_t* k, const attn_thd_t* v,
    const attn_thd_t* o, const float* lse, const attn_thd_t* dout, const attn_thd_t* dq,
    const attn_thd_t* dk, const attn_thd_t* dv, const int* cu_q, const int* cu_k, void* workspace,
    size_t workspace_bytes, int deterministic, int drop_item, unsigned long long wait_budget_ns,
    attn_stream_t stream) {
  if (drop_item < 0 || wait_budget_ns < 1000000ull || wait_budget_ns > kDefaultTimeoutNs)
    return ATTN_ERR_INVALID_ARG;
  return bwd_impl(s, q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, workspace, workspace_bytes,
                  deterministic, stream, drop_item, wait_budget_ns);
}

int attn_fwd_packed_o_boxes(const attn_packed_t* s) {
  if (check_sizes(s) != ATTN_OK) return -1;
  const int group = s->H_q / s->H_kv;
  return packed_o_boxes(group, tile_positions(group));
}

attn_status_t attn_rope_packed(const attn_thd_t* q, const attn_thd_t* q_out, const attn_thd_t* k,
                               const attn_thd_t* k_out, const int* positions, const int* sections,
                               int axes, const float* cos, const float* sin, int rope_rows,
                               int rot_dim, int interleaved, int inverse, int T, int H_q, int H_kv,
                               int D, attn_stream_t stream) {
  if (T <= 0 || H_q < 0 || H_kv < 0 || H_q + (int64_t)H_kv <= 0 || D <= 0 || rope_rows <= 0 ||
      !positions || !sections || !cos || !sin)
    return ATTN_ERR_INVALID_ARG;
  if ((H_q > 0) != (q != nullptr) || (H_q > 0) != (q_out != nullptr) ||
      (H_kv > 0) != (k != nullptr) || (H_kv > 0) != (k_out != nullptr))
    return ATTN_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return ATTN_ERR_INVALID_ARG;
  if (axes < 1 || axes > 4 || rot_dim <= 0 || rot_dim > D || rot_dim % 16 != 0)
    return ATTN_ERR_INVALID_ARG;
  RopePackedParams p;
  std::memset(&p, 0, sizeof(p));
  int64_t end = 0;
  for (int a = 0; a < 4; ++a) {
    if (a < axes) {
      if (sections[a] <= 0) return ATTN_ERR_INVALID_ARG;
      end += sections[a];
    }
    p.ends[a] = end <= D ? (int)end : D;
  }
  if (end != rot_dim / 2) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (T >= (1 << 30) || H_q > 32767 || H_kv > 32767) return ATTN_ERR_UNSUPPORTED;
  attn_status_t st;
  Thd tq{}, tk{}, tqo{}, tko{};
  if (H_q > 0 && ((st = take(q, T, H_q, D, &tq)) != ATTN_OK ||
                  (st = take(q_out, T, H_q, D, &tqo)) != ATTN_OK))
    return st;
  if (H_kv > 0 && ((st = take(k, T, H_kv, D, &tk)) != ATTN_OK ||
                   (st = take(k_out, T, H_kv, D, &tko)) != ATTN_OK))
    return st;
  if (!aligned(positions, 4) || !aligned(cos, 16) || !aligned(sin, 16)) return ATTN_ERR_MISALIGNED;
  if ((st = check_device()) != ATTN_OK) return st;
  p.q = tq.data, p.q_st = tq.st, p.q_sh = tq.sh;
  p.k = tk.data, p.k_st = tk.st, p.k_sh = tk.sh;
  p.q_out = tqo.data, p.qo_st = tqo.st, p.qo_sh = tqo.sh;
  p.k_out = tko.data, p.ko_st = tko.st, p.ko_sh = tko.sh;
  p.positions = positions;
  p.cos = cos;
  p.sin = sin;
  p.rope_rows = rope_rows;
  p.rot_dim = rot_dim;
  p.inverse = inverse;
  p.axes = axes;
  p.T = T;
  p.H_q = H_q;
  p.H_kv = H_kv;
  return done(launch_rope_packed(p, D, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
