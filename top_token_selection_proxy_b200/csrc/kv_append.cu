// kv_append.cu -- new keys and values into the paged 8-bit cache: rotation by position, the scale of each block
// of 16 tokens and head, e4m3 rounding; the queries rotated beside them.
//
// The mathematics: y = rotated x; e = the least integer with max|y| <= 448 * 2^e over the block's new tokens
// (a block that holds earlier tokens keeps the larger of e and its own exponent, and rounds them again to the
// new scale); payload = e4m3(y * 2^-e).  A power of two as the scale makes y * 2^-e exact, so each value is
// rounded once, and rounding held values again changes only those that leave e4m3's normal range.
//
// What bounds it: bytes (a key row is read once at 2 or 4 bytes an element and written at 1, a query row is read
// and written).  A block is two warps' work for one head and one of k and v: its (up to 16) token rows stay in
// registers between the maximum and the rounding, so nothing is read twice; 8 elements a lane, 16-byte loads.  (A block
// that holds something not finite is read and rotated once more, with fp64 where fp32 gives no number.)
// Query rows are other CTAs' work: a warp keeps a row's angles and takes its heads in batches of loads.
//
// Measured: a prompt of 8192 tokens, 8 key heads and 64 query heads of 128, bf16: 80 us, 4.0 TB/s (61 % of the measured
// copy bandwidth); 9 prompts of up to 1900 tokens, 24 and 3 heads, together: 27 us (49 %); one token for each of 32
// sequences: 5 us on the GPU, which is latency.  The next bound is the issue slots (47 to 53 % of their peak): the keys'
// two-float rotation takes some 15 operations an element, where a plain fp32 one would now and then land on the wrong
// side of an e4m3 tie.
#include "kv.cuh"

namespace pivot {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kE = 8;  // elements a lane holds of a row
constexpr float kMax = 3.402823466e38f;  // the largest finite fp32

// 8 elements as they lie in memory, and as fp32.
template <bool BF16>
struct Raw {
  uint4 v[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void* p, int64_t at, bool live) {
  Raw<BF16> r;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
  return r;
}

template <bool BF16>
__device__ __forceinline__ void widen(const Raw<BF16>& r, float (&x)[kE]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.v[i].x), x[4 * i + 1] = __uint_as_float(r.v[i].y);
      x[4 * i + 2] = __uint_as_float(r.v[i].z), x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
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
#pragma unroll
      for (int i = 0; i < kE; ++i) a.s[i] *= t.sign;  // the lower half's pairs take -sin
    }
  }
  return a;
}

// a c + b s in fp32.
struct Turned {
  __device__ float operator()(float a, float c, float b, float s) const { return fmaf(b, s, a * c); }
};

// a c + b s rounded to odd at 24 bits: the exact value's neighbour whose last bit is set, unless it is exact.  A
// later rounding to fewer bits, and a comparison with a power of two times 448, then give what the exact value
// gives.  The products' and the sum's own errors are exact fp32 values (fused multiply-add; Knuth's two-sum); their sum
// is rounded, so a remainder under 2^-47 of the terms may not show in the last bit (2 of 2e8 random rotations).
struct TurnedOdd {
  __device__ float operator()(float a, float c, float b, float s) const {
    const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
    const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(b, s, -q);
    const float sum = __fadd_rn(p, q), v = __fsub_rn(sum, p);
    const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, v)), __fsub_rn(q, v));
    const float low = __fadd_rn(es, __fadd_rn(ep, eq));
    const float hi = __fadd_rn(sum, low);
    const float rest = __fsub_rn(low, __fsub_rn(hi, sum));
    const int bits = __float_as_int(hi);
    if ((rest > 0.f || rest < 0.f) && !(bits & 1)) return __int_as_float((rest > 0.f) == (hi > 0.f) ? bits + 1 : bits - 1);
    return hi;  // exact or odd already; NaN wherever a product or the sum is not finite
  }
};

// The same where the value's terms may leave fp32.  fp64 holds every product of two fp32 values: NaN and infinities are
// the formula's, and a finite value that no fp32 holds becomes the largest one, which is past every scale.
struct TurnedFar {
  __device__ float operator()(float a, float c, float b, float s) const {
    const float near = TurnedOdd{}(a, c, b, s);
    if (fabsf(near) <= kMax) return near;
    const double v = fma((double)a, (double)c, (double)b * (double)s);
    return isfinite(v) ? (float)fmin(fmax(v, -(double)kMax), (double)kMax) : (float)v;
  }
};

// The elements of r, turned: form(a, c, b, s) = a c + b s.  All lanes of the warp take part.
template <bool BF16, typename F>
__device__ __forceinline__ void rotate(const Raw<BF16>& r, float (&x)[kE], const Turn& t, const Angles& a, F form) {
  widen<BF16>(r, x);
  if (t.split) {
    Raw<BF16> other;  // exchanged as it lies in memory: two bf16 a word
    float y[kE];
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i)
      other.v[i] = make_uint4(__shfl_sync(~0u, r.v[i].x, t.peer), __shfl_sync(~0u, r.v[i].y, t.peer),
                              __shfl_sync(~0u, r.v[i].z, t.peer), __shfl_sync(~0u, r.v[i].w, t.peer));
    widen<BF16>(other, y);
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = t.on ? form(x[i], a.c[i], y[i], a.s[i]) : x[i];
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
  return a <= kMax ? a : 0.f;  // NaN and infinities do not set the scale
}

__device__ __forceinline__ float max_or_nan(float a, float b) {  // NaN where either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What the two warps of a block tell each other: the largest value of each half.  One set for each block in turn
// of two, so that one barrier a block is enough.
struct Pair {
  float amax[2][2];
};

// One block of one sequence and head, by two warps of 8 tokens each: new tokens [p0, p1) at rows row0 .., earlier
// ones [base, p0).  `half`: which of the two this warp is.
template <int D, bool BF16>
__device__ __forceinline__ void append_block(const KvAppendArgs& a, Pair& pair, int bar, int turn, bool is_key, int head, int b,
                             int64_t row0, uint32_t base, uint32_t p0, uint32_t p1, int half, int lane) {
  constexpr int kLanes = D / kE, kRows = 32 / kLanes, kPasses = kKvBlock / 2 / kRows;
  const int sub = lane % kLanes, slot = half * (kKvBlock / 2) + lane / kLanes;
  const void* src = is_key ? a.k : a.v;
  const int64_t stride = is_key ? a.k_stride : a.v_stride;
  const int rot = is_key ? a.rot : 0;
  const Turn t = turn_of<D>(rot, a.interleaved, lane);
  const int page = kv_page(a.st, a.c, b, p0);  // not needed before the rows have come
  Raw<BF16> raw[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {  // all loads first: they are independent
    const uint32_t p = base + i * kRows + slot;
    raw[i] = load8<BF16>(src, (row0 + (p - p0)) * stride + head * D + sub * kE, p >= p0 && p < p1);
  }
  float y[kPasses][kE], amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t p = base + i * kRows + slot;
    if (rot) rotate<BF16>(raw[i], y[i], t, angles_at(t, t.on && p >= p0 && p < p1, a.cos, a.sin, p, a.rot / 2), TurnedOdd{});
    else widen<BF16>(raw[i], y[i]);
#pragma unroll
    for (int j = 0; j < kE; ++j) amax = max_or_nan(amax, fabsf(y[i][j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = max_or_nan(amax, __shfl_xor_sync(~0u, amax, o));
  if (!(amax <= kMax)) {  // rare: the rows once more, with care for what is not finite, which does not set the scale
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t p = base + i * kRows + slot;
      const bool live = p >= p0 && p < p1;
      const Raw<BF16> again = load8<BF16>(src, (row0 + (p - p0)) * stride + head * D + sub * kE, live);
      if (rot) rotate<BF16>(again, y[i], t, angles_at(t, t.on && live, a.cos, a.sin, p, a.rot / 2), TurnedFar{});
#pragma unroll
      for (int j = 0; j < kE; ++j) amax = fmaxf(amax, finite_abs(y[i][j]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  }
  const int64_t ph = (int64_t)max(page, 0) * a.c.hk + head;
  const int in_page = base % (uint32_t)a.c.ps;
  int8_t* exp_at = (is_key ? a.c.ke : a.c.ve) + ph * (a.c.ps / kKvBlock) + in_page / kKvBlock;
  const bool held = p0 > base;  // earlier tokens of the sequence: their exponent may be the larger
  const int was = held && page >= 0 ? *exp_at : 0;
  if (lane == 0) pair.amax[turn & 1][half] = amax;
  named_bar_sync(bar, 64);  // both halves' maxima; and both have read the exponent
  int e = exponent_of(fmaxf(pair.amax[turn & 1][0], pair.amax[turn & 1][1]));
  if (page < 0) return;
  uint8_t* rows = (is_key ? a.c.k : a.c.v) + (ph * a.c.ps + in_page) * D;
  if (held && was >= e) e = was;
  if (held && was < e) {  // their payload at the new scale
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
  const float inv = kv_exp2i(-min(max(e, -126), 126));
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t p = base + i * kRows + slot;
    const float(&z)[kE] = y[i];
    if (p >= p0 && p < p1)
      *reinterpret_cast<uint2*>(rows + (int64_t)(p - base) * D + sub * kE) =
          make_uint2(pack4(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv),
                     pack4(z[4] * inv, z[5] * inv, z[6] * inv, z[7] * inv));
  }
  if (lane == 0 && half == 0) *exp_at = (int8_t)e;
}

// A CTA takes `rows_per_cta` rows.  The first `kv_slices` of each such group append the blocks whose first new token
// is among them (a block's other rows may follow behind), two warps for each of 4 of the heads of k and v; the
// others rotate the query rows.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 3 : 2) kv_append_kernel(const KvAppendArgs a) {
  constexpr int kLanes = D / kE, kHeads = 32 / kLanes;  // heads a warp takes at a time
  constexpr int kBatch = 8;                 // ... and loads of them under way
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
    __shared__ Pair pairs[kWarps / 2];
    const int job = (int)blockIdx.y * (kWarps / 2) + warp / 2;
    if (job >= 2 * a.c.hk) return;
    int turn = 0;
    for (int64_t r = r0; r < r1;) {
      const int64_t p64 = follow(r);
      const int in = (int)p64 & (kKvBlock - 1);
      const int64_t next = p64 < 0 ? r - p64 : p64 < cap ? r + kKvBlock - in : end;  // row of the next block's first token
      if (p64 >= 0 && p64 < cap && (in == 0 || r == begin)) {
        const uint32_t p = (uint32_t)p64, base = p - in;
        const uint32_t p1 = (uint32_t)min64(min64((int64_t)base + kKvBlock, len), min64(p64 + (total - r), cap));
        append_block<D, BF16>(a, pairs[warp / 2], 1 + warp / 2, turn++, job < a.c.hk,
                              job < a.c.hk ? job : job - a.c.hk, b, r, base, p, p1, warp & 1, lane);
      }
      r = max64(min64(next, end), r + 1);
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
    for (int h0 = warp % split * per + lane / kLanes; h0 - lane / kLanes < h1; h0 += kBatch * kHeads) {
      Raw<BF16> raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        raw[i] = load8<BF16>(a.q, r * a.q_stride + (int64_t)(h0 + i * kHeads) * D + lane % kLanes * kE, h0 + i * kHeads < h1);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[kE];
        rotate<BF16>(raw[i], x, t, an, Turned{});
        if (h0 + i * kHeads < h1)
          store8<BF16>(a.q_out, r * a.q_out_stride + (int64_t)(h0 + i * kHeads) * D + lane % kLanes * kE, x);
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
  a.kv_slices = (2 * a.c.hk + kWarps / 2 - 1) / (kWarps / 2);
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
