// kv.cuh -- what the kernels of the paged 8-bit key/value cache share: the cache and the step as the device sees
// them, e4m3 conversions and the search for a row's sequence.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "kernels.cuh"
#include "ptx.cuh"

namespace pivot {

constexpr int kKvBlock = PIVOT_KV_BLOCK;

struct KvCache {
  uint8_t *k, *v;      // e4m3 [pages, hk, ps, d]
  int8_t *ke, *ve;     // [pages, hk, ps / 16]
  int pages, hk, ps, d;
};

struct KvStep {
  const int32_t* table;  // [B, width], rows `stride` apart
  const int64_t* off;    // [B+1]
  const int64_t* lens;   // [B]
  int64_t stride, rows;
  int width, B;
};

struct KvAppendArgs {
  KvCache c;
  KvStep st;
  const void *k, *v, *q;
  void* q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;  // elements
  const float *cos, *sin;  // [n_pos, rot / 2]
  int64_t n_pos;
  int rot, interleaved, hq, rows_per_cta, kv_slices;
  bool is_bf16;
};

struct KvAttnArgs {
  KvCache c;
  KvStep st;
  const void* q;
  void* out;
  float* lse;             // or null
  int64_t q_stride;
  int hq, group;          // query heads; query heads of one key head
  float scale2;           // scale * log2(e): scores in units of log 2
  int64_t window, sinks;  // window 0: none
  const int32_t* indices; // selected form: [rows, topk], rows idx_stride apart; else null
  int64_t idx_stride;
  int topk;
  bool is_bf16;
};

cudaError_t launch_kv_append(const KvAppendArgs& a, int sms, cudaStream_t s);
// What a CTA leaves for the merge when it began an item that others end.  The work of an attention call is a line
// of tiles, item after item, of which every CTA takes an equal stretch.
struct alignas(16) KvOpen {
  int64_t row0;                            // first query row's index
  int32_t stretch, head0, rr0, valid, open;  // open: how many CTAs' results make the item (0: none was begun)
};

// The CTA after the last one whose stretch reaches into an item that ends at place `item_end` of the line: stretch j
// begins at total * j / ctas.
__device__ __forceinline__ int kv_parts(int64_t item_end, int64_t total, int64_t ctas) {
  return (int)((item_end * ctas + total - 1) / total);
}

struct KvLine {
  int* status;
  const int* gate;  // null, or: run only where it is not 0
  bool whole;       // items are not cut: each is one place of the line
  KvOpen* open;     // [ctas]
  float* part;      // [ctas][2][kv_part_floats]: of an item that the stretch ends, of one that it begins
};

// Partial result of an item of `rows` query rows: sums [rows][d], then (reference, l, 0, 0) of each row.
__host__ __device__ constexpr size_t kv_part_floats(int rows, int d) { return (size_t)rows * (d + 4); }

// Lets a kernel use its dynamic shared memory, once on each device.
template <auto kKernel>
cudaError_t kv_allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

size_t kv_attn_workspace(int sms, int d);
cudaError_t launch_kv_attn(const KvAttnArgs& a, int sms, void* ws, const int* gate, cudaStream_t s);
cudaError_t launch_kv_merge(const KvAttnArgs& a, const KvLine& line, int ctas, int rows, bool many, float lift,
                            cudaStream_t s);
size_t kv_attn_tc_workspace(int sms, int d);
cudaError_t launch_kv_attn_tc(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms, void* ws,
                              uint64_t timeout_ns, bool stall, cudaStream_t s);

// The sequence b with off[b] <= r < off[b+1], or -1.
__device__ __forceinline__ int kv_sequence_of(const KvStep& st, int64_t r) {
  if (r >= st.off[st.B]) return -1;
  int lo = 0, hi = st.B;  // off[lo] <= r < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (st.off[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x * 2^e, e <= 0, where 2^e alone may lie below fp32's normal range: sums over tokens whose values' scales lie far apart.
__device__ __forceinline__ float kv_down(float x, float e) {
  return x * ex2(fmaxf(e, -126.f)) * ex2(fminf(e + 126.f, 0.f));
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t two) {  // two e4m3 bytes to two fp16
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The page of a position below 2^31, or -1 where it is absent.
__device__ __forceinline__ int kv_page(const KvStep& st, const KvCache& c, int b, uint32_t pos) {
  const uint32_t i = pos / (uint32_t)c.ps;
  if (i >= (uint32_t)st.width) return -1;
  const int pg = __ldg(st.table + (int64_t)b * st.stride + i);
  return pg >= 0 && pg < c.pages ? pg : -1;
}

__device__ __forceinline__ float kv_e4m3_to_f32(uint8_t x) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(x, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// Four consecutive output values.
__device__ __forceinline__ void kv_store4(const KvAttnArgs& a, int64_t at, float x, float y, float z, float w,
                                          bool bf16) {
  if (bf16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x, y), hi = __floats2bfloat162_rn(z, w);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(x, y, z, w);
  }
}

// 2^e for an integer e in [-126, 127].
__device__ __forceinline__ float kv_exp2i(int e) { return __int_as_float((e + 127) << 23); }

// A score's scale 2^e of a cache exponent (any int8: below -126 it is 2^-126).
__device__ __forceinline__ float kv_scale(int e) { return kv_exp2i(max(e, -126)); }

}  // namespace pivot
