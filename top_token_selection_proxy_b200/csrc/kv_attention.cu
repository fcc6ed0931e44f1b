// kv_attention.cu -- attention over the paged 8-bit cache: every visible position of a sequence, or each row's own
// list of positions.
//
// o = sum_s p_s v_s / sum_s p_s, p_s = exp2(scale2 * q . k_s - m), one pass with a running maximum m.
#include "kv.cuh"

namespace pivot {
namespace {

constexpr int kSimple = 128;

// One CTA for a row and query head: 128 positions at a time, a thread scores one and then sums one output dim.
template <bool BF16, bool SEL>
__global__ void __launch_bounds__(kSimple) kv_attn_simple_kernel(const KvAttnArgs a) {
  __shared__ float qs[128], w[kSimple];
  __shared__ int64_t at[kSimple];
  __shared__ float red[kSimple / 32];
  const int64_t r = blockIdx.x;
  const int j = blockIdx.y, tid = threadIdx.x, d = a.c.d, head = j / a.group;
  const int b = kv_sequence_of(a.st, r);
  if (b < 0) return;
  const int64_t pos = a.st.lens[b] - a.st.off[b + 1] + r;
  const int64_t cap = (int64_t)a.st.width * a.c.ps;
  const int64_t n = SEL ? (pos < 0 ? 0 : a.topk) : min64(pos + 1, cap);
  if (tid < d) {
    const int64_t qi = r * a.q_stride + (int64_t)j * d + tid;
    qs[tid] = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[qi])
                   : reinterpret_cast<const float*>(a.q)[qi];
  }
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int64_t i0 = 0; i0 < n; i0 += kSimple) {
    __syncthreads();
    const int64_t i = i0 + tid;
    int64_t s = -1;
    if (i < n) s = SEL ? (int64_t)a.indices[r * a.idx_stride + i] : i;
    bool seen = s >= 0 && s <= pos && s < cap;
    if (!SEL && a.window > 0) seen = seen && (s > pos - a.window || s < a.sinks);
    int64_t slot = -1;
    float x = -INFINITY;
    if (seen) {
      const int pg = kv_page(a.st, a.c, b, (uint32_t)s);
      if (pg >= 0) {
        const int in = (int)(s % a.c.ps);
        const int64_t ph = (int64_t)pg * a.c.hk + head;
        slot = ph * a.c.ps + in;
        const uint8_t* k = a.c.k + slot * d;
        float dot = 0.f;
        for (int e = 0; e < d; ++e) dot = fmaf(qs[e], kv_e4m3_to_f32(k[e]), dot);
        x = dot * kv_scale(a.c.ke[ph * (a.c.ps / kKvBlock) + in / kKvBlock]) * a.scale2;
      }
    }
    float t = x;
#pragma unroll
    for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o));
    if (tid % 32 == 0) red[tid / 32] = t;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
    w[tid] = slot < 0 ? 0.f : exp2f(x - mn);
    at[tid] = slot;
    __syncthreads();
    l *= f;
    acc *= f;
    m = mn;
    for (int e = 0; e < kSimple; ++e) {
      if (at[e] < 0) continue;
      l += w[e];
      if (tid < d) {
        const int64_t ph = at[e] / a.c.ps, in = at[e] % a.c.ps;
        acc = fmaf(w[e], kv_e4m3_to_f32(a.c.v[at[e] * d + tid]) *
                             kv_scale(a.c.ve[ph * (a.c.ps / kKvBlock) + in / kKvBlock]), acc);
      }
    }
  }
  if (tid < d) {
    const float o = l == 0.f ? 0.f : acc / l;
    const int64_t oi = (r * a.hq + j) * (int64_t)d + tid;
    if (BF16) reinterpret_cast<__nv_bfloat16*>(a.out)[oi] = __float2bfloat16_rn(o);
    else reinterpret_cast<float*>(a.out)[oi] = o;
  }
  if (a.lse && tid == 0) a.lse[r * a.hq + j] = l == 0.f ? -INFINITY : 0.6931471805599453f * m + logf(l);
}

}  // namespace

cudaError_t launch_kv_attn_simple(const KvAttnArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.st.rows, (unsigned)a.hq);
  if (a.indices)
    a.is_bf16 ? kv_attn_simple_kernel<true, true><<<grid, kSimple, 0, s>>>(a)
              : kv_attn_simple_kernel<false, true><<<grid, kSimple, 0, s>>>(a);
  else
    a.is_bf16 ? kv_attn_simple_kernel<true, false><<<grid, kSimple, 0, s>>>(a)
              : kv_attn_simple_kernel<false, false><<<grid, kSimple, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pivot
