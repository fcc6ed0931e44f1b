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
#include "kv.cuh"

namespace pivot {
namespace {

constexpr int kThreads = 256;
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

// x turned by the angles of one position, in T's arithmetic (float, or double where an exponent is in doubt).
// All lanes of the warp take part; `live` lanes have a row.
template <typename T>
__device__ __forceinline__ void rotate(const float (&x)[kE], T (&y)[kE], const Turn& t, bool live, const float* cos,
                                       const float* sin, int64_t pos, int half) {
  float c[kE], s[kE];
  const bool go = live && t.on;
  if (go) {
    const float4* pc = reinterpret_cast<const float4*>(cos + pos * half + t.entry);
    const float4* ps = reinterpret_cast<const float4*>(sin + pos * half + t.entry);
    const float4 c0 = __ldg(pc), s0 = __ldg(ps);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w;
    if (t.split) {
      const float4 c1 = __ldg(pc + 1), s1 = __ldg(ps + 1);
      c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
      s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
    }
  }
  if (t.split) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float other = __shfl_sync(~0u, x[i], t.peer);
      y[i] = go ? (T)x[i] * (T)c[i] + (T)(t.sign * other) * (T)s[i] : (T)x[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      const T a = x[2 * i], b = x[2 * i + 1];
      y[2 * i] = go ? a * (T)c[i] - b * (T)s[i] : a;
      y[2 * i + 1] = go ? b * (T)c[i] + a * (T)s[i] : b;
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
    const bool live = p >= p0 && p < p1;
    if (rot) {
      float x[kE];
#pragma unroll
      for (int j = 0; j < kE; ++j) x[j] = y[i][j];
      rotate<float>(x, y[i], t, live, a.cos, a.sin, p, a.rot / 2);
    }
#pragma unroll
    for (int j = 0; j < kE; ++j) amax = fmaxf(amax, finite_abs(y[i][j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  int e = exponent_of(amax);
  // A rotated maximum carries a rounding error of a few units; within 16 of a step between two exponents
  // (1 block in 3 * 10^5) the step is decided in 64 bits.
  const int near = (int)(__float_as_uint(amax) & 0x7FFFFFu) - 0x600000;
  if (rot && near >= -16 && near <= 16) {
    double m = 0.0;
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t p = base + i * kRows + slot;
      const bool live = p >= p0 && p < p1;
      float x[kE];
      double z[kE];
#pragma unroll
      for (int j = 0; j < kE; ++j) x[j] = 0.f;
      if (live) load8<BF16>(src, (row0 + (p - p0)) * stride + head * D + sub * kE, x);
      rotate<double>(x, z, t, live, a.cos, a.sin, p, a.rot / 2);
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        const double w = fabs(z[j]);
        if (w <= 3.402823466e38 && w > m) m = w;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double w = __shfl_xor_sync(~0u, m, o);
      m = w > m ? w : m;
    }
    const int low = exponent_of(__uint_as_float((__float_as_uint(amax) & 0xFF800000u) | 0x600000u));  // at the step
    e = low;
    if (low < PIVOT_KV_EXP_MAX && m > 448.0 * (double)kv_exp2i(low)) e = low + 1;
  }
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

// A CTA takes `rows_per_cta` rows: the blocks whose first new token is among them (a block's other rows may
// follow behind), and the rotation of their query rows.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
  constexpr int kLanes = D / kE, kRows = 32 / kLanes;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kWarps = kThreads / 32;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_cta;
  const int64_t total = min64(a.st.off[a.st.B], a.st.rows);
  const int64_t r1 = min64(r0 + a.rows_per_cta, total);
  if (r0 >= r1) return;
  const uint32_t cap = (uint32_t)a.st.width * (uint32_t)a.c.ps;
  int b = kv_sequence_of(a.st, r0);
  int64_t begin = a.st.off[b], end = a.st.off[b + 1], len = a.st.lens[b];
  int turn = 0;  // jobs go round the warps
  for (int64_t r = r0; r < r1; ++r) {
    while (r >= end && b + 1 < a.st.B) {
      ++b;
      begin = end;
      end = a.st.off[b + 1];
      len = a.st.lens[b];
    }
    const int64_t p64 = len - end + r;
    if (p64 < 0 || p64 >= (int64_t)cap) continue;
    const uint32_t p = (uint32_t)p64;
    if (p % kKvBlock == 0 || r == begin || p == 0) {
      const uint32_t base = p / kKvBlock * kKvBlock;
      const uint32_t p1 = (uint32_t)min64(min64((int64_t)base + kKvBlock, len), min64(p64 + (total - r), cap));
      const int page = kv_page(a.st, a.c, b, p);
      if (page >= 0) {
        for (int j = 0; j < 2 * a.c.hk; ++j, ++turn)
          if (turn % kWarps == warp)
            append_block<D, BF16>(a, j < a.c.hk, j < a.c.hk ? j : j - a.c.hk, page, r, base, p, p1, lane);
      }
    }
    if (a.q) {  // kRows heads of this row a pass
      const Turn t = turn_of<D>(a.rot, a.interleaved, lane);
      for (int h0 = 0; h0 < a.hq; h0 += kRows, ++turn) {
        if (turn % kWarps != warp) continue;
        const int h = h0 + lane / kLanes;
        const bool live = h < a.hq;
        const int64_t at = (int64_t)h * D + lane % kLanes * kE;
        float x[kE], y[kE];
#pragma unroll
        for (int j = 0; j < kE; ++j) x[j] = 0.f;
        if (live) load8<BF16>(a.q, r * a.q_stride + at, x);
        rotate<float>(x, y, t, live, a.cos, a.sin, p, a.rot / 2);
        if (live) store8<BF16>(a.q_out, r * a.q_out_stride + at, y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& args, int sms, cudaStream_t s) {
  KvAppendArgs a = args;
  int per = kKvBlock;
  while (per > 1 && (a.st.rows + per - 1) / per < 8 * sms) per /= 2;
  a.rows_per_cta = per;
  const unsigned grid = (unsigned)((a.st.rows + per - 1) / per);
  if (a.c.d == 128)
    a.is_bf16 ? kv_append_kernel<128, true><<<grid, kThreads, 0, s>>>(a)
              : kv_append_kernel<128, false><<<grid, kThreads, 0, s>>>(a);
  else
    a.is_bf16 ? kv_append_kernel<64, true><<<grid, kThreads, 0, s>>>(a)
              : kv_append_kernel<64, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pivot
