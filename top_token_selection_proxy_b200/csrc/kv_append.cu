// kv_append.cu -- new keys and values into the paged 8-bit cache: rotation by position, the scale of each block
// of 16 tokens and head, e4m3 rounding; the queries rotated beside them.
//
// The mathematics: y = rotated x; e = the least integer with max|y| <= 448 * 2^e over the block's new tokens
// (a block that holds earlier tokens keeps the larger of e and its own exponent, and rounds them again to the
// new scale); payload = e4m3(y * 2^-e).  A power of two as the scale makes y * 2^-e exact, so each value is
// rounded once, and rounding held values again changes only those that leave e4m3's normal range.
//
// What bounds it: bytes (a key row is read once at 2 or 4 bytes an element and written at 1, a query row is read
// and written).  A block is one warp's work for one head and one of k and v: its (up to 16) token rows stay in
// registers between the maximum and the rounding, so nothing is read twice; 8 elements a lane, 16-byte loads.
// Query rows are other CTAs' work: a warp keeps a row's angles and takes its heads in batches of loads.
#include "kv.cuh"

namespace pivot {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kE = 8;  // elements a lane holds of a row

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[kE]) {
  if (BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[kE]) {
  if (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Where a lane's 8 elements stand in the rotation: which cos/sin entries they take, which lane holds the
// other half of their pairs, and the sign of its term.
struct Turn {
  bool on, split;  // within `rot`; pairs across lanes (halves) or within the lane (interleaved)
  int entry, peer;
  float sign;
};

template <int D>
__device__ __forceinline__ Turn turn_of(int rot, int interleaved, int lane) {
  constexpr int kLanes = D / kE;
  const int sub = lane % kLanes, e0 = sub * kE;
  Turn t;
  t.on = e0 < rot;
  t.split = !interleaved;
  t.entry = t.peer = 0;
  t.sign = 1.f;
  if (!t.on) {
    t.peer = lane;
  } else if (interleaved) {
    t.entry = e0 / 2;
    t.peer = lane;
  } else {
    const bool low = e0 < rot / 2;
    t.entry = low ? e0 : e0 - rot / 2;
    t.peer = low ? lane + rot / (2 * kE) : lane - rot / (2 * kE);
    t.sign = low ? -1.f : 1.f;
  }
  return t;
}

// The angles that a lane's 8 elements take at one position.
struct Angles {
  float c[kE], s[kE];
};

__device__ __forceinline__ Angles angles_at(const Turn& t, bool go, const float* cos, const float* sin, int64_t pos,
                                            int half) {
  Angles a;
#pragma unroll
  for (int i = 0; i < kE; ++i) a.c[i] = 1.f, a.s[i] = 0.f;
  if (go) {
    const float4* pc = reinterpret_cast<const float4*>(cos + pos * half + t.entry);
    const float4* ps = reinterpret_cast<const float4*>(sin + pos * half + t.entry);
    const float4 c0 = __ldg(pc), s0 = __ldg(ps);
    a.c[0] = c0.x, a.c[1] = c0.y, a.c[2] = c0.z, a.c[3] = c0.w;
    a.s[0] = s0.x, a.s[1] = s0.y, a.s[2] = s0.z, a.s[3] = s0.w;
    if (t.split) {
      const float4 c1 = __ldg(pc + 1), s1 = __ldg(ps + 1);
      a.c[4] = c1.x, a.c[5] = c1.y, a.c[6] = c1.z, a.c[7] = c1.w;
      a.s[4] = s1.x, a.s[5] = s1.y, a.s[6] = s1.z, a.s[7] = s1.w;
    }
  }
  return a;
}

// a c + b s in fp32.
__device__ __forceinline__ float turned(float a, float c, float b, float s) { return fmaf(b, s, a * c); }

// a c + b s rounded to odd at 24 bits: the exact value's neighbour whose last bit is set, unless it is exact.  A
// later rounding to fewer bits, and a comparison with a power of two times 448, then give what the exact value
// gives.  The products' and the sum's own errors are exact fp32 values (fused multiply-add; Knuth's two-sum).
__device__ __forceinline__ float turned_odd(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
  const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(b, s, -q);
  const float sum = __fadd_rn(p, q), v = __fsub_rn(sum, p);
  const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, v)), __fsub_rn(q, v));
  const float low = __fadd_rn(es, __fadd_rn(ep, eq));
  const float hi = __fadd_rn(sum, low);
  const float rest = __fsub_rn(low, __fsub_rn(hi, sum));
  const int bits = __float_as_int(hi);
  if ((rest > 0.f || rest < 0.f) && !(bits & 1)) return __int_as_float((rest > 0.f) == (hi > 0.f) ? bits + 1 : bits - 1);
  return hi;  // exact, odd already, or not finite
}

// x turned: F(a, c, b, s) forms each element.  All lanes of the warp take part.
template <typename F>
__device__ __forceinline__ void rotate(float (&x)[kE], const Turn& t, const Angles& a, F form) {
  if (t.split) {
    const float sign = t.on ? t.sign : 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float other = __shfl_sync(~0u, x[i], t.peer);
      x[i] = t.on ? form(x[i], a.c[i], other, sign * a.s[i]) : x[i];
    }
  } else if (t.on) {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      const float u = x[2 * i], w = x[2 * i + 1];
      x[2 * i] = form(u, a.c[i], w, -a.s[i]);
      x[2 * i + 1] = form(w, a.c[i], u, a.s[i]);
    }
  }
}

// The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), within the range of a scale.
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u);
  return min(max(e, PIVOT_KV_EXP_MIN), PIVOT_KV_EXP_MAX);  // zero and subnormals: the least
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float finite_abs(float y) {
  const float a = fabsf(y);
  return a <= 3.402823466e38f ? a : 0.f;  // NaN and infinities do not set the scale
}

// One block of one sequence and head: new tokens [p0, p1) at rows row0 .., earlier ones [base, p0).
template <int D, bool BF16>
__device__ void append_block(const KvAppendArgs& a, bool is_key, int head, int page, int64_t row0, uint32_t base,
                             uint32_t p0, uint32_t p1, int lane) {
  constexpr int kLanes = D / kE, kRows = 32 / kLanes, kPasses = kKvBlock / kRows;
  const int sub = lane % kLanes, slot = lane / kLanes;
  const void* src = is_key ? a.k : a.v;
  const int64_t stride = is_key ? a.k_stride : a.v_stride;
  const int rot = is_key ? a.rot : 0;
  const Turn t = turn_of<D>(rot, a.interleaved, lane);
  float y[kPasses][kE];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {  // all loads first: they are independent
    const uint32_t p = base + i * kRows + slot;
    if (p >= p0 && p < p1) {
      load8<BF16>(src, (row0 + (p - p0)) * stride + head * D + sub * kE, y[i]);
    } else {
#pragma unroll
      for (int j = 0; j < kE; ++j) y[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t p = base + i * kRows + slot;
    if (rot)
      rotate(y[i], t, angles_at(t, t.on && p >= p0 && p < p1, a.cos, a.sin, p, a.rot / 2), turned_odd);
#pragma unroll
    for (int j = 0; j < kE; ++j) amax = fmaxf(amax, finite_abs(y[i][j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  int e = exponent_of(amax);
  uint8_t* dst = is_key ? a.c.k : a.c.v;
  int8_t* exps = is_key ? a.c.ke : a.c.ve;
  const int64_t ph = (int64_t)page * a.c.hk + head;
  const int in_page = base % (uint32_t)a.c.ps;
  int8_t* exp_at = exps + ph * (a.c.ps / kKvBlock) + in_page / kKvBlock;
  uint8_t* rows = dst + (ph * a.c.ps + in_page) * D;
  if (p0 > base) {  // earlier tokens of the sequence: their exponent, and their payload at the new one
    const int was = *exp_at;
    if (was >= e) {
      e = was;
    } else {
      const float f = was - e < -126 ? 0.f : kv_exp2i(was - e);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t p = base + i * kRows + slot;
        if (p < p0) {
          uint2* at = reinterpret_cast<uint2*>(rows + (int64_t)(p - base) * D + sub * kE);
          const uint2 r = *at;
          float z[kE];
#pragma unroll
          for (int j = 0; j < kE; ++j) z[j] = kv_e4m3_to_f32((uint8_t)((j < 4 ? r.x : r.y) >> (8 * (j & 3)))) * f;
          *at = make_uint2(pack4(z[0], z[1], z[2], z[3]), pack4(z[4], z[5], z[6], z[7]));
        }
      }
    }
  }
  const float inv = kv_exp2i(-min(max(e, -126), 126));
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t p = base + i * kRows + slot;
    if (p >= p0 && p < p1) {
      const float(&z)[kE] = y[i];
      *reinterpret_cast<uint2*>(rows + (int64_t)(p - base) * D + sub * kE) =
          make_uint2(pack4(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv),
                     pack4(z[4] * inv, z[5] * inv, z[6] * inv, z[7] * inv));
    }
  }
  __syncwarp();  // every lane has read the old exponent
  if (lane == 0) *exp_at = (int8_t)e;
}

// A CTA takes `rows_per_cta` rows.  The first `kv_slices` of each such group append the blocks whose first new token
// is among them (a block's other rows may follow behind), a warp for each of 8 of the heads of k and v; the others
// rotate the query rows.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 2) kv_append_kernel(const KvAppendArgs a) {
  constexpr int kLanes = D / kE, kHeads = 32 / kLanes, kBatch = 4;  // heads a warp takes at a time; times this
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_cta;
  const int64_t total = min64(a.st.off[a.st.B], a.st.rows);
  const int64_t r1 = min64(r0 + a.rows_per_cta, total);
  if (r0 >= r1) return;
  const int64_t cap = (int64_t)a.st.width * a.c.ps;
  int b = kv_sequence_of(a.st, r0);
  int64_t begin = a.st.off[b], end = a.st.off[b + 1], len = a.st.lens[b];
  auto follow = [&](int64_t r) {  // the sequence of a later row; its position
    while (r >= end && b + 1 < a.st.B) {
      ++b;
      begin = end;
      end = a.st.off[b + 1];
      len = a.st.lens[b];
    }
    return len - end + r;
  };
  if (blockIdx.y < a.kv_slices) {
    const int job = (int)blockIdx.y * kWarps + warp;
    if (job >= 2 * a.c.hk) return;
    for (int64_t r = r0; r < r1; ++r) {
      const int64_t p64 = follow(r);
      if (p64 < 0 || p64 >= cap || (p64 % kKvBlock && r != begin)) continue;
      const uint32_t p = (uint32_t)p64, base = p / kKvBlock * kKvBlock;
      const uint32_t p1 = (uint32_t)min64(min64((int64_t)base + kKvBlock, len), min64(p64 + (total - r), cap));
      const int page = kv_page(a.st, a.c, b, p);
      if (page >= 0)
        append_block<D, BF16>(a, job < a.c.hk, job < a.c.hk ? job : job - a.c.hk, page, r, base, p, p1, lane);
    }
    return;
  }
  // A row's heads are one warp's, or, where the rows are few, several warps'.
  const int split = a.rows_per_cta >= kWarps ? 1 : kWarps / a.rows_per_cta;
  const int per = ((a.hq + split - 1) / split + kHeads - 1) / kHeads * kHeads;
  const Turn t = turn_of<D>(a.rot, a.interleaved, lane);
  for (int64_t r = r0 + warp / split; r < r1; r += kWarps / split) {
    const int64_t p = follow(r);
    if (p < 0 || p >= cap) continue;
    const Angles an = angles_at(t, t.on, a.cos, a.sin, p, a.rot / 2);
    const int h1 = min(a.hq, (warp % split + 1) * per);
    for (int h0 = warp % split * per; h0 < h1; h0 += kBatch * kHeads) {
      float x[kBatch][kE];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * kHeads + lane / kLanes;
#pragma unroll
        for (int j = 0; j < kE; ++j) x[i][j] = 0.f;
        if (h < h1) load8<BF16>(a.q, r * a.q_stride + (int64_t)h * D + lane % kLanes * kE, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * kHeads + lane / kLanes;
        rotate(x[i], t, an, turned);
        if (h < h1) store8<BF16>(a.q_out, r * a.q_out_stride + (int64_t)h * D + lane % kLanes * kE, x[i]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& args, int sms, cudaStream_t s) {
  KvAppendArgs a = args;
  int per = kKvBlock;  // fewer where that leaves SMs without work
  while (per > 1 && (a.st.rows + per - 1) / per < 2 * sms) per /= 2;
  a.rows_per_cta = per;
  a.kv_slices = (2 * a.c.hk + kWarps - 1) / kWarps;
  const dim3 grid((unsigned)((a.st.rows + per - 1) / per), (unsigned)(a.kv_slices + (a.q ? 1 : 0)));
  if (a.c.d == 128)
    a.is_bf16 ? kv_append_kernel<128, true><<<grid, kThreads, 0, s>>>(a)
              : kv_append_kernel<128, false><<<grid, kThreads, 0, s>>>(a);
  else
    a.is_bf16 ? kv_append_kernel<64, true><<<grid, kThreads, 0, s>>>(a)
              : kv_append_kernel<64, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pivot
