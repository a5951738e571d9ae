// C-ABI entry points of the serving-step operators: page plans and rotary positions with the cache
// writes.  Every argument error is caught here, before any CUDA call.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "internal.h"

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int32_t shift_of(int32_t v) {
  for (int32_t s = 0; s < 31; ++s)
    if ((int32_t{1} << s) == v) return s;
  return -1;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr int32_t kMaxQHeads = 16384, kMaxKvHeads = 8192;   // blockIdx.y holds a share of the q, k and v heads
constexpr int32_t kMaxHeadDim = 16384;

// The rotation's own arguments (rope may be null where nothing turns).
qsa_status rope_args(const qsa_rope_spec* rope, int32_t head_dim, qsa::RopeParams* p) {
  p->magnitude = 1.0f;
  p->sin_sign = 1.0f;
  if (!rope) return QSA_OK;
  if (rope->rot_dim < 0 || rope->rot_dim % 2 != 0 || rope->rot_offset < 0 ||
      static_cast<int64_t>(rope->rot_dim) + rope->rot_offset > head_dim ||
      (rope->layout != QSA_ROPE_HALF && rope->layout != QSA_ROPE_INTERLEAVED) ||
      (rope->transpose != 0 && rope->transpose != 1) || !std::isfinite(rope->magnitude))
    return QSA_ERR_INVALID_ARG;
  if (rope->rot_dim > 0 && !rope->steps) return QSA_ERR_INVALID_ARG;
  if (rope->rot_dim / 2 > qsa::kRopeMaxPairs) return QSA_ERR_UNSUPPORTED;
  p->rot_dim = rope->rot_dim;
  p->rot_offset = rope->rot_dim > 0 ? rope->rot_offset : 0;
  p->interleaved = rope->layout == QSA_ROPE_INTERLEAVED;
  p->magnitude = rope->magnitude;
  p->sin_sign = rope->transpose ? -rope->magnitude : rope->magnitude;
  if (rope->rot_dim > 0) std::memcpy(p->steps, rope->steps, sizeof(uint64_t) * (rope->rot_dim / 2));
  return QSA_OK;
}

qsa_status run_rope(qsa::RopeParams& p, const qsa_rope_spec* rope, int32_t dtype, bool fp4, void* stream) {
  if (p.n_rows < 0 || p.n_qheads < 0 || p.n_kvheads < 0 || p.head_dim < 1 ||
      (dtype != QSA_BF16 && dtype != QSA_FP16))
    return QSA_ERR_INVALID_ARG;
  if (p.n_qheads + static_cast<int64_t>(p.n_kvheads) < 1) return QSA_ERR_INVALID_ARG;
  if (p.n_qheads > kMaxQHeads || p.n_kvheads > kMaxKvHeads || p.head_dim > kMaxHeadDim ||
      p.n_rows > INT32_MAX)
    return QSA_ERR_UNSUPPORTED;
  const int64_t q_width = static_cast<int64_t>(p.n_qheads) * p.head_dim;
  if (p.n_qheads > 0) {
    if (!p.q || !p.q_out || p.q_stride < 0 || p.q_out_stride < q_width) return QSA_ERR_INVALID_ARG;
    if (p.q == p.q_out && p.q_stride != p.q_out_stride) return QSA_ERR_INVALID_ARG;
    if (!aligned_to(p.q, 2) || !aligned_to(p.q_out, 2)) return QSA_ERR_INVALID_ARG;
  }
  if (p.n_kvheads > 0) {
    if (!p.k || !p.k_cache || !p.slots || p.k_stride < 0 || p.n_slots < 0) return QSA_ERR_INVALID_ARG;
    if ((p.v == nullptr) != (p.v_cache == nullptr) || (p.v && p.v_stride < 0)) return QSA_ERR_INVALID_ARG;
    if (!aligned_to(p.k, 2) || !aligned_to(p.v, 2)) return QSA_ERR_INVALID_ARG;
    if (!fp4 && (!aligned_to(p.k_cache, 2) || !aligned_to(p.v_cache, 2))) return QSA_ERR_INVALID_ARG;
  }
  p.n_vheads = p.v ? p.n_kvheads : 0;
  const qsa_status st = rope_args(rope, p.head_dim, &p);
  if (st != QSA_OK) return st;
  if (p.rot_dim > 0 && !p.positions) return QSA_ERR_INVALID_ARG;
  if (fp4) {
    // 16-dim blocks of aligned rows; rotated halves have to fill whole blocks
    if (p.head_dim % 32 != 0 || p.rot_offset % 16 != 0 || p.rot_dim % (p.interleaved ? 16 : 32) != 0)
      return QSA_ERR_UNSUPPORTED;
    if (!qsa::rope_is_aligned(p)) return QSA_ERR_INVALID_ARG;
  }
  if (p.n_rows == 0) return QSA_OK;
  int32_t sms = 0;
  const qsa_status ds = qsa::device_sms(&sms);
  if (ds != QSA_OK) return ds;
  if (qsa::launch_rope(p, dtype == QSA_FP16, fp4, sms, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return QSA_ERR_CUDA;
  qsa::count_launches(1);
  return QSA_OK;
}

// How the units of a call are dealt out, by a model of its time in key tiles.  A unit takes its tiles and about
// three tiles' time of its own (query tile, first softmax, output).  Whole units: blocks that become free take the
// next one, and about half a unit's time passes while the last ones finish.  Equal shares divide that time evenly,
// but a block then has one more unit begun or ended, writes up to two partial ones in fp32 (a tile's worth of bytes
// each when all 128 rows are in use) that the join reads again, and the join is one more launch, about three tiles
// long.  Shares are taken where the model gives them 7 %.  The lengths behind the page table are not known here: every
// unit is taken to see as many keys as the table has room for (or the window).  Where that is far from the lengths, the
// choice can fall on the slower way: prompts of 1024 and 2048 rows, 32/8 heads of 128 dims, take 21 and 43 us in a table
// of just their length (whole units), 33 and 64 in one four times as wide or more (shares); 24/2 heads of 256 dims 25
// and 50, and 39 and 68.  Measured (us, whole / shares): 128 decode rows with contexts of 1k
// to 8k, 24/2 heads of 256 dims, window 4096: 146 / 127; 48 decode rows over 16k to 32k keys in 4 bits: 449 / 224; a
// chunk of 512 rows at 8000, 256 dims: 103 / 89, 128 dims, 32/8 heads: 67 / 74; the last 8192 rows of a 32k prompt:
// 150 / 153; 256 decode rows of 1k to 4k, 128 dims: 338 / 356; a prompt of 2048 rows: 44 / 60.
struct WindowPlan {
  int32_t tile_tokens, n_tiles, shares, unit_cost;
  int32_t key_tiles;             // a unit has at most as many
  int64_t n_units;
};
constexpr int32_t kMaxShareTiles = 1 << 14;    // every block sums all units' tiles
WindowPlan plan_window(int64_t n_rows, int32_t n_requests, int32_t n_kvheads, int32_t group, int32_t tile_rows,
                       int64_t max_keys, int32_t window, int32_t n_sink, int32_t sms) {
  WindowPlan w{};
  w.tile_tokens = tile_rows / group;
  w.n_tiles = static_cast<int32_t>(n_rows / w.tile_tokens + n_requests);
  w.n_units = static_cast<int64_t>(w.n_tiles) * n_kvheads;
  // units with rows: every request has at most one partial tile
  int64_t tiles = (n_rows + w.tile_tokens - 1) / w.tile_tokens + n_requests - 1;
  if (tiles > n_rows) tiles = n_rows;
  int64_t keys = max_keys;
  if (window > 0) {
    const int64_t seen = static_cast<int64_t>(window) + w.tile_tokens + n_sink + 64;
    if (seen < keys) keys = seen;
  }
  const int64_t kt = (keys + qsa::kWinTile - 1) / qsa::kWinTile;
  const int64_t items = tiles * n_kvheads;
  w.key_tiles = static_cast<int32_t>(kt);
  if (kt <= 1 || w.n_tiles > kMaxShareTiles) return w;
  const int64_t rows_per = n_rows < tiles * w.tile_tokens ? (n_rows + tiles - 1) / tiles : w.tile_tokens;
  const double partial = static_cast<double>(rows_per * group) / qsa::kWinTile;
  const double load = static_cast<double>(items) / sms, unit = kt + 3.0;
  const double whole = load > 1.0 ? (load + 0.5) * unit : unit;
  const int64_t shares = items * kt < sms ? items * kt : sms;
  const double even = static_cast<double>(items) * unit / shares + 3.0 + 6.0 * partial + 3.0;
  if (even < 0.93 * whole) {
    w.shares = static_cast<int32_t>(shares);
    // with fewer units than shares, every share has one or two, and the tiles are divided
    w.unit_cost = items > shares ? 3 : 0;
  }
  return w;
}

// Rows of the query tile (WinCfg::kRows of the kernels).
int32_t window_tile_rows(int32_t head_dim, bool fp4) { return fp4 && head_dim == 256 ? 64 : qsa::kWinTile; }

// Partial outputs, their log-sum-exps and the join records of a call in equal shares.
size_t window_ws_bytes(int32_t head_dim, int32_t shares) {
  return static_cast<size_t>(shares) * (2 * qsa::kWinTile * (static_cast<size_t>(head_dim) + 1) * 4 + sizeof(qsa::JoinRecord));
}

struct Fp4Cache {
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  float k_global, v_global;
};

qsa_status check_window(int64_t n_rows, int32_t n_requests, int32_t pages_per_req, int32_t page_size,
                        int64_t n_pages, int32_t n_qheads, int32_t n_kvheads, int32_t head_dim,
                        int32_t window, int32_t n_sink, bool fp4) {
  if (n_rows < 0 || n_requests < 1 || pages_per_req < 1 || page_size < 1 || n_pages < 1 || n_qheads < 1 ||
      n_kvheads < 1 || n_qheads % n_kvheads != 0 || window < 0 || n_sink < 0)
    return QSA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return QSA_ERR_UNSUPPORTED;
  if (n_qheads / n_kvheads > window_tile_rows(head_dim, fp4)) return QSA_ERR_UNSUPPORTED;
  if (n_rows >= INT32_MAX - n_requests) return QSA_ERR_UNSUPPORTED;
  // positions, rounded up to whole key tiles, are held in 32 bits
  if (static_cast<int64_t>(pages_per_req) * page_size > INT32_MAX - 2 * qsa::kWinTile) return QSA_ERR_UNSUPPORTED;
  if (n_pages > INT32_MAX / page_size || n_pages * page_size > (INT32_MAX - 1) / n_kvheads)
    return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

qsa_status run_window(const void* q, const void* k_cache, const void* v_cache, const Fp4Cache* fp4,
                      const int32_t* cu_seqlens_q, const int32_t* kv_lens, const int32_t* page_table,
                      void* out, float* lse, int64_t n_rows, int32_t n_requests, int32_t pages_per_req,
                      int32_t page_size, int64_t n_pages, int32_t n_qheads, int32_t n_kvheads,
                      int32_t head_dim, float scale, int32_t window, int32_t n_sink, int32_t dtype,
                      void* workspace, size_t workspace_bytes, void* stream_v) {
  if (!q || !k_cache || !v_cache || !cu_seqlens_q || !kv_lens || !page_table || !out) return QSA_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
      !aligned_to(cu_seqlens_q, 4) || !aligned_to(kv_lens, 4) || !aligned_to(page_table, 4) ||
      !aligned_to(lse, 4))
    return QSA_ERR_INVALID_ARG;
  // (scale log2(e), with a 4-bit cache's scale, is what the kernel multiplies by)
  const float scale_log2 = scale * 1.4426950408889634f * (fp4 ? fp4->k_global : 1.0f);
  if (!(scale > 0.0f) || !(scale_log2 > 0.0f) || !std::isfinite(scale_log2) || (dtype != QSA_BF16 && dtype != QSA_FP16))
    return QSA_ERR_INVALID_ARG;
  qsa_status st = check_window(n_rows, n_requests, pages_per_req, page_size, n_pages, n_qheads, n_kvheads,
                               head_dim, window, n_sink, fp4 != nullptr);
  if (st != QSA_OK) return st;
  if (n_rows == 0) return QSA_OK;
  int32_t sms = 0;
  st = qsa::device_sms(&sms);
  if (st != QSA_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  const int32_t group = n_qheads / n_kvheads;
  const WindowPlan w = plan_window(n_rows, n_requests, n_kvheads, group, window_tile_rows(head_dim, fp4 != nullptr),
                                   static_cast<int64_t>(pages_per_req) * page_size, window, n_sink, sms);
  if (w.n_units > INT32_MAX) return QSA_ERR_UNSUPPORTED;
  qsa::WindowParams p{};
  p.q = q;
  p.out = out;
  p.lse = lse;
  if (qsa::device_status_address(&p.status) != cudaSuccess) return QSA_ERR_CUDA;
  p.pa.page_table = page_table;
  p.pa.cu_seqlens_q = cu_seqlens_q;
  p.pa.kv_lens = kv_lens;
  p.pa.n_requests = n_requests;
  p.pa.pages_per_req = pages_per_req;
  p.pa.page_size = page_size;
  p.pa.page_shift = shift_of(page_size);
  p.pa.n_pages = n_pages;
  p.n_rows = n_rows;
  p.n_units = w.n_units;
  p.n_qheads = n_qheads;
  p.n_kvheads = n_kvheads;
  p.group = group;
  p.tile_tokens = w.tile_tokens;
  p.n_tiles = w.n_tiles;
  p.shares = w.shares;
  p.unit_cost = w.unit_cost;
  p.wait_ns = qsa::kWinWaitNs + qsa::kWinWaitNsPerTile * static_cast<unsigned long long>(w.key_tiles);
  p.out_32 = aligned_to(out, 32);
  p.window = window;
  p.n_sink = n_sink;
  int32_t box = 1;      // keys per copy: the largest power of two <= 64 that divides the page size
  while (box < 64 && page_size % (2 * box) == 0) box *= 2;
  p.box = box >= 8 ? box : 0;
  p.n_slots = static_cast<int32_t>(n_pages * page_size);
  p.scale_log2 = scale_log2;
  p.v_mult = 1.0f;
  if (fp4) {
    p.k_codes = static_cast<const uint8_t*>(k_cache);
    p.v_codes = static_cast<const uint8_t*>(v_cache);
    p.k_scale = fp4->k_scale;
    p.v_scale = fp4->v_scale;
    p.v_mult = fp4->v_global;
  }
  if (qsa::log_geometry())
    std::fprintf(stderr,
                 "qsa: window d=%d rows=%lld requests=%d heads=%d/%d window=%d sinks=%d%s -> tile_tokens=%d "
                 "box=%d shares=%d units=%lld\n",
                 head_dim, static_cast<long long>(n_rows), n_requests, n_qheads, n_kvheads, window, n_sink,
                 fp4 ? " fp4" : "", p.tile_tokens, p.box, p.shares, static_cast<long long>(p.n_units));
  void* ws = workspace;
  bool own = false;
  const size_t need = window_ws_bytes(head_dim, p.shares);
  if (need > 0) {
    if (ws) {
      if (workspace_bytes < need || !aligned_to(ws, 256)) return QSA_ERR_WORKSPACE;
    } else {
      if (qsa::ws_alloc(&ws, need, stream) != cudaSuccess) return QSA_ERR_CUDA;
      own = true;
    }
    p.part_o = static_cast<float*>(ws);
    p.part_lse = p.part_o + static_cast<size_t>(p.shares) * 2 * qsa::kWinTile * head_dim;
    p.joins = reinterpret_cast<qsa::JoinRecord*>(p.part_lse + static_cast<size_t>(p.shares) * 2 * qsa::kWinTile);
  }
  p.stall_first_item = qsa::take_stall_request() ? 1 : 0;
  const cudaError_t e = qsa::launch_window(p, head_dim, dtype == QSA_FP16, fp4 != nullptr, k_cache, v_cache,
                                           stream);
  if (own) cudaFreeAsync(ws, stream);
  if (e != cudaSuccess) return QSA_ERR_CUDA;
  qsa::count_launches(p.shares > 0 ? 2 : 1);
  return QSA_OK;
}

}  // namespace

extern "C" {

size_t qsa_window_workspace_bytes(int64_t n_rows, int32_t n_requests, int32_t pages_per_req,
                                  int32_t page_size, int32_t n_qheads, int32_t n_kvheads,
                                  int32_t head_dim, int32_t window, int32_t n_sink, int32_t fp4,
                                  int32_t num_sms) {
  if (check_window(n_rows, n_requests, pages_per_req, page_size, 1, n_qheads, n_kvheads, head_dim, window,
                   n_sink, fp4 != 0) != QSA_OK || n_rows == 0)
    return 0;
  if (num_sms <= 0 && qsa::device_sms(&num_sms) != QSA_OK) return 0;
  const WindowPlan w = plan_window(n_rows, n_requests, n_kvheads, n_qheads / n_kvheads, window_tile_rows(head_dim, fp4 != 0),
                                   static_cast<int64_t>(pages_per_req) * page_size, window, n_sink, num_sms);
  return window_ws_bytes(head_dim, w.shares);
}

qsa_status qsa_window_attention_paged(const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                                      const int32_t* page_table, void* out, float* lse, int64_t n_rows,
                                      int32_t n_requests, int32_t pages_per_req, int32_t page_size,
                                      int64_t n_pages, int32_t n_qheads, int32_t n_kvheads,
                                      int32_t head_dim, float scale, int32_t window, int32_t n_sink,
                                      int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return run_window(q, k_cache, v_cache, nullptr, cu_seqlens_q, kv_lens, page_table, out, lse, n_rows, n_requests,
                    pages_per_req, page_size, n_pages, n_qheads, n_kvheads, head_dim, scale, window, n_sink,
                    dtype, workspace, workspace_bytes, stream);
}

qsa_status qsa_window_attention_fp4_paged(const void* q, const void* k_cache, const uint8_t* k_scale,
                                          const void* v_cache, const uint8_t* v_scale, float k_global,
                                          float v_global, const int32_t* cu_seqlens_q,
                                          const int32_t* kv_lens, const int32_t* page_table, void* out,
                                          float* lse, int64_t n_rows, int32_t n_requests,
                                          int32_t pages_per_req, int32_t page_size, int64_t n_pages,
                                          int32_t n_qheads, int32_t n_kvheads, int32_t head_dim,
                                          float scale, int32_t window, int32_t n_sink, int32_t dtype,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!k_scale || !v_scale || !aligned_to(k_scale, 16) || !aligned_to(v_scale, 16)) return QSA_ERR_INVALID_ARG;
  if (!(k_global > 0.0f) || !(v_global > 0.0f) || !std::isfinite(k_global) || !std::isfinite(v_global))
    return QSA_ERR_INVALID_ARG;
  const Fp4Cache f{k_scale, v_scale, k_global, v_global};
  return run_window(q, k_cache, v_cache, &f, cu_seqlens_q, kv_lens, page_table, out, lse, n_rows, n_requests,
                    pages_per_req, page_size, n_pages, n_qheads, n_kvheads, head_dim, scale, window, n_sink,
                    dtype, workspace, workspace_bytes, stream);
}

qsa_status qsa_page_plan(const int32_t* past_lens, const int32_t* new_lens, int32_t* page_table,
                         const int32_t* free_pages, int64_t n_free, const int32_t* free_head,
                         int32_t* free_head_out, int32_t* cu_seqlens_q, int32_t* kv_lens,
                         int32_t* positions, int32_t* slots, int32_t* shortfall, int32_t n_requests,
                         int32_t pages_per_req, int32_t page_size, int64_t n_pages, int64_t max_rows,
                         void* stream) {
  if (!past_lens || !new_lens || !page_table || !free_head || !free_head_out || !cu_seqlens_q || !kv_lens ||
      (n_free > 0 && !free_pages))
    return QSA_ERR_INVALID_ARG;
  if (n_requests < 1 || pages_per_req < 1 || page_size < 1 || n_pages < 0 || n_free < 0 || max_rows < 0)
    return QSA_ERR_INVALID_ARG;
  for (const void* a : {static_cast<const void*>(past_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(page_table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(free_head), static_cast<const void*>(free_head_out),
                        static_cast<const void*>(cu_seqlens_q), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(positions), static_cast<const void*>(slots),
                        static_cast<const void*>(shortfall)})
    if (!aligned_to(a, 4)) return QSA_ERR_INVALID_ARG;
  // the kernel numbers a step's fresh pages in 32 bits: no more than the table has entries
  if (n_requests > qsa::kPlanMaxRequests || max_rows > INT32_MAX || n_free > INT32_MAX ||
      static_cast<int64_t>(n_requests) * pages_per_req > INT32_MAX)
    return QSA_ERR_UNSUPPORTED;
  int32_t sms = 0;
  const qsa_status st = qsa::device_sms(&sms);
  if (st != QSA_OK) return st;
  qsa::PagePlanParams p{};
  p.past_lens = past_lens;
  p.new_lens = new_lens;
  p.page_table = page_table;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.free_head_out = free_head_out;
  p.cu_seqlens_q = cu_seqlens_q;
  p.kv_lens = kv_lens;
  p.positions = positions;
  p.slots = slots;
  p.shortfall = shortfall;
  p.n_free = n_free;
  p.n_pages = n_pages;
  p.max_rows = max_rows;
  p.n_requests = n_requests;
  p.pages_per_req = pages_per_req;
  p.page_size = page_size;
  p.page_shift = shift_of(page_size);
  p.vec_rows = aligned_to(positions, 16) && aligned_to(slots, 16);
  if (qsa::launch_page_plan(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) return QSA_ERR_CUDA;
  qsa::count_launches(1);
  return QSA_OK;
}

qsa_status qsa_rope_steps(const qsa_rope_scaling* scaling, int32_t rot_dim, double base, uint64_t* steps,
                          float* magnitude) {
  if (!steps || !magnitude || rot_dim < 2 || rot_dim % 2 != 0 || !std::isfinite(base) || base <= 0.0)
    return QSA_ERR_INVALID_ARG;
  if (rot_dim / 2 > qsa::kRopeMaxPairs) return QSA_ERR_UNSUPPORTED;
  const qsa_rope_scaling none{QSA_ROPE_SCALE_NONE, 1.0, 0.0, 0.0, 0.0};
  const qsa_rope_scaling& s = scaling ? *scaling : none;
  const double f = s.kind == QSA_ROPE_SCALE_NONE ? 1.0 : s.factor;
  if (!std::isfinite(f) || f <= 0.0) return QSA_ERR_INVALID_ARG;
  const bool ramp = s.kind == QSA_ROPE_SCALE_YARN || s.kind == QSA_ROPE_SCALE_TURNS;
  if (ramp && (!(s.original_len > 0.0) || !std::isfinite(s.original_len) || !(s.beta_slow > 0.0) ||
               !(s.beta_fast > s.beta_slow) || !std::isfinite(s.beta_fast)))
    return QSA_ERR_INVALID_ARG;
  double low = 0.0, high = 0.0, b = base;
  switch (s.kind) {
    case QSA_ROPE_SCALE_NONE:
    case QSA_ROPE_SCALE_LINEAR:
    case QSA_ROPE_SCALE_TURNS: break;
    case QSA_ROPE_SCALE_NTK:
      if (rot_dim < 4) return QSA_ERR_INVALID_ARG;
      b = base * std::pow(f, static_cast<double>(rot_dim) / (rot_dim - 2));
      if (!std::isfinite(b)) return QSA_ERR_INVALID_ARG;
      break;
    case QSA_ROPE_SCALE_YARN: {
      if (base <= 1.0) return QSA_ERR_INVALID_ARG;
      // the pair that makes t turns over the original length
      auto pair_at = [&](double t) {
        return rot_dim * std::log(s.original_len / (kTwoPi * t)) / (2.0 * std::log(base));
      };
      low = std::fmax(std::floor(pair_at(s.beta_fast)), 0.0);
      high = std::fmin(std::ceil(pair_at(s.beta_slow)), rot_dim - 1.0);
      break;
    }
    default: return QSA_ERR_INVALID_ARG;
  }
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(b, -2.0 * i / rot_dim);      // radians per token
    double keep = 1.0;                               // share of the unscaled frequency
    if (s.kind == QSA_ROPE_SCALE_LINEAR) keep = 0.0;
    if (s.kind == QSA_ROPE_SCALE_YARN)
      keep = 1.0 - std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
    if (s.kind == QSA_ROPE_SCALE_TURNS)
      keep = std::fmin(std::fmax((s.original_len * w / kTwoPi - s.beta_slow) / (s.beta_fast - s.beta_slow),
                                 0.0), 1.0);
    w = keep * w + (1.0 - keep) * w / f;
    const double turns = w / kTwoPi;
    steps[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
  }
  *magnitude = s.kind == QSA_ROPE_SCALE_YARN && f > 1.0 ? static_cast<float>(0.1 * std::log(f) + 1.0) : 1.0f;
  return QSA_OK;
}

qsa_status qsa_rope(const void* x, void* out, const int32_t* positions, const qsa_rope_spec* rope,
                    int64_t n_rows, int32_t n_heads, int32_t head_dim, int64_t x_stride,
                    int64_t out_stride, int32_t dtype, void* stream) {
  if (!rope || !positions) return QSA_ERR_INVALID_ARG;
  qsa::RopeParams p{};
  p.q = x;
  p.q_out = out;
  p.positions = positions;
  p.n_rows = n_rows;
  p.n_qheads = n_heads;
  p.head_dim = head_dim;
  p.q_stride = x_stride;
  p.q_out_stride = out_stride;
  return run_rope(p, rope, dtype, false, stream);
}

qsa_status qsa_rope_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                           void* v_cache, const int32_t* positions, const int32_t* slots,
                           const qsa_rope_spec* rope, int64_t n_rows, int64_t n_slots, int32_t n_qheads,
                           int32_t n_kvheads, int32_t head_dim, int64_t q_stride, int64_t q_out_stride,
                           int64_t k_stride, int64_t v_stride, int32_t dtype, void* stream) {
  if (n_kvheads < 1) return QSA_ERR_INVALID_ARG;
  qsa::RopeParams p{};
  p.q = q;
  p.q_out = q_out;
  p.k = k;
  p.v = v;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.positions = positions;
  p.slots = slots;
  p.n_rows = n_rows;
  p.n_slots = n_slots;
  p.n_qheads = n_qheads;
  p.n_kvheads = n_kvheads;
  p.head_dim = head_dim;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return run_rope(p, rope, dtype, false, stream);
}

qsa_status qsa_rope_append_fp4(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                               uint8_t* k_scale, void* v_cache, uint8_t* v_scale, float k_global,
                               float v_global, void* k_seen, void* v_seen, const int32_t* positions,
                               const int32_t* slots, const qsa_rope_spec* rope, int64_t n_rows,
                               int64_t n_slots, int32_t n_qheads, int32_t n_kvheads, int32_t head_dim,
                               int64_t q_stride, int64_t q_out_stride, int64_t k_stride,
                               int64_t v_stride, int32_t dtype, void* stream) {
  if (n_kvheads < 1 || !v || !k_scale || !v_scale) return QSA_ERR_INVALID_ARG;
  if (!(k_global > 0.0f) || !(v_global > 0.0f) || !std::isfinite(k_global) || !std::isfinite(v_global))
    return QSA_ERR_INVALID_ARG;
  qsa::RopeParams p{};
  p.q = q;
  p.q_out = q_out;
  p.k = k;
  p.v = v;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_seen = k_seen;
  p.v_seen = v_seen;
  p.k_global = k_global;
  p.v_global = v_global;
  p.positions = positions;
  p.slots = slots;
  p.n_rows = n_rows;
  p.n_slots = n_slots;
  p.n_qheads = n_qheads;
  p.n_kvheads = n_kvheads;
  p.head_dim = head_dim;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return run_rope(p, rope, dtype, true, stream);
}

}  // extern "C"
