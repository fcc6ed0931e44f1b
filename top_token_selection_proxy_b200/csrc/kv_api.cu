// kv_api.cu -- host side of the pivot_kv_* calls of include/pivot.h: argument checks and launches.  Nothing is
// allocated and no call synchronises the host.
#include <algorithm>
#include <cmath>

#include "kv.cuh"

using namespace pivot;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kFar = 1ll << 62;  // more tokens than there can be; positions, which may lie below 0, less it fit 64 bits

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

pivot_status check_cache(const pivot_kv_cache* c) {
  if (!c || !c->k || !c->v || !c->k_exp || !c->v_exp) return PIVOT_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->kv_heads <= 0 || c->page_size <= 0 || c->page_size % PIVOT_KV_BLOCK)
    return PIVOT_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return PIVOT_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) || c->kv_heads > 1024) return PIVOT_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)c->num_pages * c->kv_heads > (int64_t)0x7FFFFFFFll / c->page_size) return PIVOT_ERR_UNSUPPORTED_SHAPE;
  return PIVOT_OK;
}

pivot_status check_step(const pivot_kv_step* s, const pivot_kv_cache* c) {
  if (!s || !s->block_table || !s->row_offsets || !s->lens) return PIVOT_ERR_INVALID_ARG;
  if (s->B <= 0 || s->rows < 0 || s->table_width <= 0 || s->table_stride < s->table_width) return PIVOT_ERR_INVALID_ARG;
  if (s->rows >= 0x7FFFFFF0ll || (int64_t)s->table_width * c->page_size >= 0x7FFFFFF0ll)
    return PIVOT_ERR_UNSUPPORTED_SHAPE;
  return PIVOT_OK;
}

// Row tensors [rows, heads, d]: rows `stride` elements apart, each on a 16-byte boundary.
pivot_status check_rows(const void* p, int64_t stride, int64_t heads, int d, pivot_dtype dt) {
  const int64_t esz = dt == PIVOT_BF16 ? 2 : 4;
  if (!p || stride < heads * d || !aligned(p, 16) || stride * esz % 16) return PIVOT_ERR_INVALID_ARG;
  return PIVOT_OK;
}

// Whether the outputs share memory with the queries (which cut items read again after others were written) or with one
// another.
bool out_overlaps(const pivot_kv_cache& c, const pivot_kv_step& s, const void* q, int64_t q_stride, int q_heads,
                  pivot_dtype dt, const void* out, const float* lse) {
  const int64_t esz = dt == PIVOT_BF16 ? 2 : 4, row = (int64_t)q_heads * c.d;
  const int64_t q_bytes = ((s.rows - 1) * q_stride + row) * esz, out_bytes = s.rows * row * esz;
  const int64_t lse_bytes = s.rows * q_heads * (int64_t)sizeof(float);
  auto meet = [](const void* a, int64_t na, const void* b, int64_t nb) {
    const char *p = static_cast<const char*>(a), *r = static_cast<const char*>(b);
    return p < r + nb && r < p + na;
  };
  return meet(out, out_bytes, q, q_bytes) ||
         (lse && (meet(lse, lse_bytes, q, q_bytes) || meet(lse, lse_bytes, out, out_bytes)));
}

KvCache device_cache(const pivot_kv_cache& c) {
  return {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_exp, c.v_exp, c.num_pages, c.kv_heads,
          c.page_size, c.d};
}

KvStep device_step(const pivot_kv_step& s) {
  return {s.block_table, s.row_offsets, s.lens, s.table_stride, s.rows, s.table_width, s.B};
}

int sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

// The payload as rows of 128 bytes, in boxes of one block's 16 tokens, 128-byte swizzle.
bool payload_map(CUtensorMap* m, const void* base, int64_t rows) {
  typedef CUresult (*Fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                         const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                         CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Fn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<Fn>(p)
               : nullptr;
  }();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, PIVOT_KV_BLOCK}, each[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether a call may go to the tcgen05 kernel.
bool many_rows(int64_t rows, int B, int q_heads, int kv_heads, int d, pivot_dtype dt) {
  return dt == PIVOT_BF16 && d == 128 && rows * (q_heads / kv_heads) > 16 * (int64_t)B;
}

// Whether it pays there, by the most work that there can be, in tiles of 128 tokens by 16 query rows: that kernel
// needs some 14 us more for its launches and first tiles, and takes a tile of 128 rows in the time of about 1.5 of 16.
// Measured (16 against 128 rows an item, us): 1 sequence of 4000, 8 key heads of 64 rows (1024) 32 against 41, of 128
// rows (2048) 43 against 41; 16 of 500, 4 heads of 24 rows (512) 26 against 29; 16 of 4000, 4 heads of 20 rows (4096)
// 63 against 50; 16 of 32000, 2 heads of 64 rows (32000) 395 against 114.  These are batches of equal sequences under
// tables of their length, and the rule knows no others: with a wider table, or one long sequence among short ones, the
// call as a whole still goes one way, and may pay those 14 us, or take many rows 16 at a time.
bool much_work(const pivot_kv_cache& c, const pivot_kv_step& s, int q_heads, int64_t window, int64_t sinks) {
  const int64_t group = q_heads / c.kv_heads, cap = (int64_t)s.table_width * c.page_size;
  int64_t seen = cap;
  if (window > 0 && window < cap && sinks < cap) seen = std::min(cap, window + sinks + s.rows / s.B);
  return (s.rows * group / 16 + s.B) * c.kv_heads * (seen / 128 + 1) >= 1536;
}

// Checks that the attention calls share, and the argument block they launch with.
pivot_status attention_args(const pivot_kv_cache* cache, const pivot_kv_step* step, const void* q, int64_t q_stride,
                            int q_heads, pivot_dtype dt, float scale, void* out, void* ws, KvAttnArgs* a) {
  pivot_status st = check_cache(cache);
  if (st == PIVOT_OK) st = check_step(step, cache);
  if (st != PIVOT_OK) return st;
  if (dt != PIVOT_BF16 && dt != PIVOT_F32) return PIVOT_ERR_INVALID_ARG;
  if (q_heads <= 0 || q_heads % cache->kv_heads || !out || !aligned(out, 16) || !ws || !aligned(ws, 256) ||
      !std::isfinite(scale * kLog2e))
    return PIVOT_ERR_INVALID_ARG;
  st = check_rows(q, q_stride, q_heads, cache->d, dt);
  if (st != PIVOT_OK) return st;
  if (q_heads > 1024) return PIVOT_ERR_UNSUPPORTED_SHAPE;
  a->c = device_cache(*cache);
  a->st = device_step(*step);
  a->q = q;
  a->out = out;
  a->q_stride = q_stride;
  a->hq = q_heads;
  a->group = q_heads / cache->kv_heads;
  a->scale2 = scale * kLog2e;
  a->is_bf16 = dt == PIVOT_BF16;
  return PIVOT_OK;
}

}  // namespace

extern "C" {

pivot_status pivot_kv_append(const pivot_kv_cache* cache, const pivot_kv_step* step, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, pivot_dtype dt, const float* cos, const float* sin,
                             int64_t n_pos, int rot, int interleaved, const void* q, int64_t q_stride, int q_heads,
                             void* q_out, int64_t q_out_stride, pivot_stream_t stream) {
  clear_cuda_error();
  pivot_status st = check_cache(cache);
  if (st == PIVOT_OK) st = check_step(step, cache);
  if (st != PIVOT_OK) return st;
  if (dt != PIVOT_BF16 && dt != PIVOT_F32) return PIVOT_ERR_INVALID_ARG;
  st = check_rows(k, k_stride, cache->kv_heads, cache->d, dt);
  if (st == PIVOT_OK) st = check_rows(v, v_stride, cache->kv_heads, cache->d, dt);
  if (st != PIVOT_OK) return st;
  if (rot < 0 || rot > cache->d || rot % 16 || (interleaved != 0 && interleaved != 1)) return PIVOT_ERR_INVALID_ARG;
  if (rot && (!cos || !sin || !aligned(cos, 16) || !aligned(sin, 16) ||
              n_pos < (int64_t)step->table_width * cache->page_size))
    return PIVOT_ERR_INVALID_ARG;
  if (q) {
    if (q_heads <= 0 || (q_out == q && q_out_stride != q_stride)) return PIVOT_ERR_INVALID_ARG;
    st = check_rows(q, q_stride, q_heads, cache->d, dt);
    if (st == PIVOT_OK) st = check_rows(q_out, q_out_stride, q_heads, cache->d, dt);
    if (st != PIVOT_OK) return st;
  }
  if (step->rows == 0) return PIVOT_OK;
  KvAppendArgs a{};
  a.c = device_cache(*cache);
  a.st = device_step(*step);
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_out = q_out;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.cos = cos;
  a.sin = sin;
  a.n_pos = n_pos;
  a.rot = rot;
  a.interleaved = interleaved;
  a.hq = q_heads;
  a.is_bf16 = dt == PIVOT_BF16;
  const cudaError_t e = launch_kv_append(a, sms(), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PIVOT_OK : record_cuda_error(e, "kv append kernel");
}

size_t pivot_kv_workspace_size(int64_t rows, int B, int q_heads, int kv_heads, int d, int topk, pivot_dtype dt) {
  if (rows < 0 || rows >= 0x7FFFFFF0ll || B <= 0 || kv_heads <= 0 || q_heads <= 0 || q_heads > 1024 ||
      q_heads % kv_heads || (d != 64 && d != 128) || topk < 0 || topk > 65536 || (dt != PIVOT_BF16 && dt != PIVOT_F32))
    return 0;
  return topk == 0 && many_rows(rows, B, q_heads, kv_heads, d, dt) ? kv_attn_tc_workspace(sms(), d)
                                                                 : kv_attn_workspace(sms(), d);
}

pivot_status pivot_kv_attention(const pivot_kv_cache* cache, const pivot_kv_step* step, const void* q,
                                int64_t q_stride, int q_heads, pivot_dtype dt, float scale, int64_t window,
                                int64_t sinks, void* out, float* lse_opt, void* ws, size_t ws_bytes,
                                pivot_stream_t stream) {
  clear_cuda_error();
  KvAttnArgs a{};
  const pivot_status st = attention_args(cache, step, q, q_stride, q_heads, dt, scale, out, ws, &a);
  if (st != PIVOT_OK) return st;
  if (window < 0 || sinks < 0) return PIVOT_ERR_INVALID_ARG;
  if (ws_bytes < pivot_kv_workspace_size(step->rows, step->B, q_heads, cache->kv_heads, cache->d, 0, dt))
    return PIVOT_ERR_WORKSPACE_TOO_SMALL;
  a.lse = lse_opt;
  a.window = std::min(window, kFar);
  a.sinks = std::min(sinks, kFar);
  if (step->rows == 0) return PIVOT_OK;
  if (out_overlaps(*cache, *step, q, q_stride, q_heads, dt, out, lse_opt)) return PIVOT_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (many_rows(step->rows, step->B, q_heads, cache->kv_heads, cache->d, dt) &&
      much_work(*cache, *step, q_heads, a.window, a.sinks)) {
    const int64_t slots = (int64_t)cache->num_pages * cache->kv_heads * cache->page_size;
    CUtensorMap kmap, vmap;
    if (!payload_map(&kmap, cache->k, slots) || !payload_map(&vmap, cache->v, slots))
      return record_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    e = launch_kv_attn_tc(a, kmap, vmap, sms(), ws, device_timeout_ns(), debug_flags() & 1, s);
  } else {
    e = launch_kv_attn(a, sms(), ws, nullptr, s);
  }
  return e == cudaSuccess ? PIVOT_OK : record_cuda_error(e, "kv attention kernel");
}

pivot_status pivot_kv_attention_selected(const pivot_kv_cache* cache, const pivot_kv_step* step, const void* q,
                                         int64_t q_stride, int q_heads, pivot_dtype dt, float scale,
                                         const int32_t* indices, int64_t index_stride, int topk, void* out,
                                         float* lse_opt, void* ws, size_t ws_bytes, pivot_stream_t stream) {
  clear_cuda_error();
  KvAttnArgs a{};
  const pivot_status st = attention_args(cache, step, q, q_stride, q_heads, dt, scale, out, ws, &a);
  if (st != PIVOT_OK) return st;
  if (!indices || topk <= 0 || index_stride < topk) return PIVOT_ERR_INVALID_ARG;
  if (topk > 65536) return PIVOT_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < pivot_kv_workspace_size(step->rows, step->B, q_heads, cache->kv_heads, cache->d, topk, dt))
    return PIVOT_ERR_WORKSPACE_TOO_SMALL;
  a.lse = lse_opt;
  a.indices = indices;
  a.idx_stride = index_stride;
  a.topk = topk;
  if (step->rows == 0) return PIVOT_OK;
  if (out_overlaps(*cache, *step, q, q_stride, q_heads, dt, out, lse_opt)) return PIVOT_ERR_INVALID_ARG;
  const cudaError_t e = launch_kv_attn(a, sms(), ws, nullptr, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PIVOT_OK : record_cuda_error(e, "kv selected attention kernel");
}

}  // extern "C"
