// kv_attention.cu -- attention over the paged 8-bit cache with few query rows for a key head: every visible
// position of a sequence, or each row's own list of positions.
//
// o = sum_s p_s v_s / sum_s p_s, p_s = 2^(z_s - m), z = scale2 * q . k (units of log 2), one pass over the keys.
// A key is payload * 2^e with one e for 16 tokens and head, so z = (q . payload) * 2^e scale2, and the output sum
// takes weights p * 2^e.  Both sums are kept relative to a reference u of each row, a value of z + e that may lag
// behind the largest by as much as fp16 holds: weights enter the product as fp16 values of 2^(z + e - u + 2), the
// denominator adds 2^(z - u) in fp32, which holds it for all scales there are (|e| <= 60).  fp16 keeps 11 bits of a weight
// where a bf16 output keeps 8 of their sum; fp32 calls multiply what it leaves as a second fp16 (21 bits), a second product.
//
// What bounds it: the cache's bytes (2 d and a little for each token and key head, read once for up to 16 query
// rows).  So the payload goes to registers in the order in which the matrix instruction wants it, without a
// detour: in a product the order of the summed index is free, hence a lane that holds 16 consecutive dims of a key
// holds the operands of 4 steps of m16n8k16, and a lane that holds 16 consecutive dims of a value those of 16
// column tiles.  Each lane copies exactly the 16-byte pieces that it will use itself into its own places of shared
// memory (cp.async), so the ring needs no barrier: every warp runs through its own tokens alone.
//
// Work is cut evenly whatever the lengths are: all tiles of 128 tokens of all (sequence, key head, 16 query rows)
// stand in one line, each item behind a few places for what it costs beside its tiles, and every CTA takes an equal
// stretch of it.  A stretch that begins or ends inside an item leaves a partial result, which kv_merge_kernel joins in
// a fixed order.  (The places: 48 sequences of 1 to 32768 tokens, window 1024, d = 64: 60 us without them, 35 us with.)
//
// Measured: 16 sequences of 32000 tokens, 8 key heads, one row of 8 query heads each: d = 128 bf16 251 us (4.19 TB/s,
// 64 % of the measured copy bandwidth), fp32 339 us; d = 64 130 us (62 %).  1 of 200000: 109 us (57 %).  Not DRAM but
// the warps' own latency holds it there (few warps fit beside the registers that the sums take; 25 % of the tensor
// pipe's cycles): conversions to fp16, exponentials and products follow one another within a warp.  Selected rows (1024
// rows of 64 query heads over 2048 tokens each): 484 us; each of the 4 groups of 16 heads gathers the list for itself,
// from L2.
#include <type_traits>

#include "kv.cuh"

namespace pivot {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRowsT = 16;              // query rows of an item
constexpr int kWTok = 32;               // tokens a warp takes at a time (two blocks)
constexpr int kTile = kWTok * kWarps;   // tokens of a tile
constexpr int kItemCost = 4;            // what an item costs beside its tiles, in tiles
constexpr int kWholeTiles = 2;          // items of so few tiles are not cut
constexpr float kRest = 2048.f;         // fp32: what a weight's fp16 leaves goes into the product times 2^11
constexpr float kLift = 2.f;            // a weight of the row's reference is 2^2 in fp16

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Values that are not to be computed with before this point.
__device__ __forceinline__ void stay(float (&z)[4][4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) asm volatile("" : "+f"(z[j][0]), "+f"(z[j][1]), "+f"(z[j][2]), "+f"(z[j][3]));
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
  return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(~0u, x, 1);
  return x + __shfl_xor_sync(~0u, x, 2);
}

// 16 (or 8) bytes to shared memory; nothing is read and zeros are written where `live` is false.
template <int N>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, bool live) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0) : "memory");
}

// ---------------------------------------------------------------- the line of tiles
struct Extent {      // of one sequence
  int64_t first;     // position of its first row
  int hi;            // last position there is (-1: none)
  int sink_tiles, lo_tile, tiles, row_tiles;
};

__device__ __forceinline__ Extent extent_of(const KvAttnArgs& a, int b) {
  Extent e;
  const int64_t n = a.st.off[b + 1] - a.st.off[b], len = a.st.lens[b];
  const int64_t cap = (int64_t)a.st.width * a.c.ps;
  e.first = len - n;
  e.hi = (int)max64(min64(len, cap) - 1, -1);
  int64_t lo = 0;
  if (a.window > 0) lo = min64(max64(e.first - a.window + 1, 0), max64(e.hi, 0));
  e.lo_tile = (int)(lo / kTile);
  e.sink_tiles = a.window > 0 ? (int)min64((min64(a.sinks, e.hi + 1) + kTile - 1) / kTile, e.lo_tile) : 0;
  e.tiles = e.sink_tiles + max(e.hi, 0) / kTile - e.lo_tile + 1;
  e.row_tiles = n > 0 ? (int)((n * a.group + kRowsT - 1) / kRowsT) : 0;
  return e;
}

// Places of an item in the line.
__device__ __forceinline__ int places(const KvLine& line, int tiles) { return line.whole ? 1 : tiles + kItemCost; }

__device__ __forceinline__ int64_t weight_of(const KvAttnArgs& a, const KvLine& line, int b) {
  if (b >= a.st.B) return 0;
  const Extent e = extent_of(a, b);
  return (int64_t)a.c.hk * e.row_tiles * places(line, e.tiles);
}

// Where a CTA stands in the line: kept in shared memory while it works on an item, for the loop needs the registers.
struct Place {
  int64_t at, stop, total, ctas, row0, row;
  int t0, t1, t, end, rr0, h, valid, x, b, per_b;
  Extent e;
};

// ---------------------------------------------------------------- the kernel
template <int D, bool BF16, bool SEL>
struct Shape {
  // CTAs an SM holds, and stages of a warp's ring.  Dense rows of 128 need 255 registers: two CTAs of three stages take
  // 251 us where three of two take 397 (16 sequences of 32000, bf16).  Selected ones wait for a gather behind two
  // look-ups, so more warps count for more: three CTAs 480 us, two 542 (1024 rows of 64 heads, lists of 2048; lists of 512
  // for 64 rows of 8 heads: 24.3 and 22.6).  d = 64: three CTAs 129 us, four 164.
  static constexpr int kCtas = !BF16 || (D == 128 && !SEL) ? 2 : 3;
  static constexpr int kStages = D == 64 ? 4 : SEL && BF16 ? 2 : 3;
  static constexpr int kKPieces = 4 * (D / 64);         // 16-byte pieces of keys a lane holds of 32 tokens
  static constexpr int kVBytes = D / 8;                 // bytes of a value a lane holds
  static constexpr int kStageBytes = 32 * (kKPieces * 16 + 8 * kVBytes + 4);  // a warp's; 4: the tokens' scales
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQParts = BF16 ? 1 : 3;
  static constexpr int kQBytes = kQParts * (D / 16) * 32 * 16;  // the query rows' operands, the same for all warps
  static constexpr size_t kBytes = kRing + kQBytes + 64 * sizeof(float) * kWarps;
  static constexpr int kSumStride = D + 16;  // floats of a row of the warps' sums
  static_assert(kWarps * kRowsT * kSumStride * 4 <= kRing, "the warps' sums take the ring's place");
};

template <int D, bool BF16, bool SEL>
__global__ void __launch_bounds__(kThreads, Shape<D, BF16, SEL>::kCtas) kv_attn_kernel(const KvAttnArgs a, const KvLine line) {
  using S = Shape<D, BF16, SEL>;
  constexpr int NK = D / 16, NT = D / 8, kStages = S::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Place place;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, tig = lane % 4;
  float* const stats = reinterpret_cast<float*>(smem + S::kRing + S::kQBytes);  // [warp][16 rows][u, l]
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStageBytes;
  if (line.gate) {
    if (*line.gate == 0) return;
  } else if (blockIdx.x == 0 && tid == 0) {
    *line.status = 0;
  }

  // this CTA's stretch of the line
  int64_t total = 0, sel_rows = 0, w_first = 0;  // w_first: of the lane's first sequence
  const int sel_rt = (a.group + kRowsT - 1) / kRowsT, sel_tiles = (a.topk + kTile - 1) / kTile;
  if (SEL) {
    sel_rows = max64(min64(a.st.off[a.st.B], a.st.rows), 0);
    total = sel_rows * a.c.hk * sel_rt * places(line, sel_tiles);
  } else {
    for (int b = lane; b < a.st.B; b += 32) {
      const int64_t w = weight_of(a, line, b);
      if (b < 32) w_first = w;
      total += w;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  }
  int64_t ctas = min64(gridDim.x, total);
  KvOpen* const open = line.open + blockIdx.x;
  if (tid == 0 && !line.whole) open->open = 0;
  if (blockIdx.x >= ctas) return;
  int64_t at = total * blockIdx.x / ctas;
  int64_t stop = total * (blockIdx.x + 1) / ctas;

  // the item that holds place `at`: sequence b, item x of it, place t of the item
  int b = 0, x = 0, t = 0, per_b = 0;
  int64_t row = 0;
  Extent e{};
  if (SEL) {
    const int64_t item = at / places(line, sel_tiles);
    t = (int)(at - item * places(line, sel_tiles));
    per_b = a.c.hk * sel_rt;
    row = item / per_b;
    x = (int)(item - row * per_b);
    e.tiles = sel_tiles;
    e.row_tiles = sel_rt;
    b = kv_sequence_of(a.st, row);
  } else {
    int64_t run = 0;
    for (int b0 = 0;; b0 += 32) {
      if (b0 >= a.st.B) return;  // only where the lengths changed under the call
      const int64_t w = b0 ? weight_of(a, line, b0 + lane) : w_first;
      int64_t inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += up;
      }
      const unsigned hit = __ballot_sync(~0u, run + inc > at);
      if (hit) {
        const int l = __ffs(hit) - 1;
        b = b0 + l;
        at -= run + __shfl_sync(~0u, inc - w, l);  // tiles into the sequence, for a moment
        break;
      }
      run += __shfl_sync(~0u, inc, 31);
    }
    e = extent_of(a, b);
    per_b = a.c.hk * e.row_tiles;
    x = (int)(at / places(line, e.tiles));
    t = (int)(at - (int64_t)x * places(line, e.tiles));
    at = total * blockIdx.x / ctas;
  }

  while (at < stop) {
    int end = (int)min64(places(line, e.tiles), t + (stop - at));  // places [t, end) of the item
    int t0 = line.whole ? 0 : max(t - kItemCost, 0);               // its tiles among them
    int t1 = line.whole ? e.tiles : max(end - kItemCost, 0);
    if (t1 > t0) {  // else the item begins in the next stretch
    int h = x / e.row_tiles, rr0 = (x - h * e.row_tiles) * kRowsT;  // key head, first of its query rows
    int64_t row0, first;
    int n, hi;
    if (SEL) {
      row0 = row;
      n = 1;
      first = b < 0 ? -1 : a.st.lens[b] - a.st.off[b + 1] + row;
      hi = (int)max64(min64(first, (int64_t)a.st.width * a.c.ps - 1), -1);
    } else {
      row0 = a.st.off[b];
      n = (int)(a.st.off[b + 1] - row0);
      first = e.first;
      hi = e.hi;
    }
    int valid = (int)min64(kRowsT, (int64_t)n * a.group - rr0);
    if (tid == 0) place = {at, stop, total, ctas, row0, row, t0, t1, t, end, rr0, h, valid, x, b, per_b, e};
    // What this lane's two rows see, and what all rows of the item do, as positions that fit 32 bits: up to sees_upto,
    // from sees_from on or among the first `sinks`.  (64-bit positions in the loop would cost it its registers.)
    auto small = [](int64_t v) { return (int)min64(max64(v, -1), 0x7FFFFFF0); };
    const bool windowed = !SEL && a.window > 0;
    const int64_t p_lo = first + rr0 / a.group, p_hi = first + (rr0 + valid - 1) / a.group;
    int sees_upto[2], sees_from[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t p = first + (rr0 + min(g + 8 * i, valid - 1)) / a.group;
      sees_upto[i] = small(min64(p, hi));
      sees_from[i] = windowed ? max(small(p - a.window + 1), 0) : 0;
    }
    const int whole_upto = small(min64(p_lo, hi)), whole_from = windowed ? max(small(p_hi - a.window + 1), 0) : 0;
    const int sinks = windowed ? small(a.sinks) : 0;

    // q: this lane's operands, scaled by a power of two so that the row's largest lies in [2^14, 2^15): one fp16 holds
    // a bf16's 8 bits (down to 2^-31 of the largest), three hold an fp32's 24.
    float unit[2];  // |scale2| / that power
    {
      float v[2][2 * NK * 2];
      uint4* const qs = reinterpret_cast<uint4*>(smem + S::kRing);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = rr0 + g + 8 * i, in = g + 8 * i;
        const int64_t r = row0 + rr / a.group;
        const bool live = in < valid && r < a.st.rows;
        const int64_t base = r * a.q_stride + (int64_t)(h * a.group + rr % a.group) * D + 16 * tig;
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (live) {
              if (BF16) {
                const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.q) + base + 64 * c + j);
                f[0] = __uint_as_float(w.x << 16), f[1] = __uint_as_float(w.x & 0xFFFF0000u);
                f[2] = __uint_as_float(w.y << 16), f[3] = __uint_as_float(w.y & 0xFFFF0000u);
              } else {
                const float4 w = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + base + 64 * c + j);
                f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[i][16 * c + j + k] = f[k];
              top = fmaxf(top, fabsf(f[k]));
            }
          }
        top = quad_max(top);
        const bool finite = top <= 3.402823466e38f;
        const int ex = top > 0.f && finite ? max((int)(__float_as_uint(top) >> 23) - 127 - 14, -100) : 0;
        unit[i] = fabsf(a.scale2) * kv_exp2i(ex);
        const float down = a.scale2 < 0.f ? -kv_exp2i(-ex) : kv_exp2i(-ex);
#pragma unroll
        for (int k = 0; k < D / 4; ++k) v[i][k] *= down;
      }
      if (warp == 0) {
#pragma unroll
        for (int ks = 0; ks < NK; ++ks)
#pragma unroll
          for (int part = 0; part < S::kQParts; ++part) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // a0: row g, a1: row g + 8, a2, a3: the same rows' next two dims
              float* f = &v[k & 1][4 * ks + (k & 2)];
              w[k] = pack_f16(f[0], f[1]);
              const __half2 hh = *reinterpret_cast<const __half2*>(&w[k]);
              f[0] -= __low2float(hh);
              f[1] -= __high2float(hh);
            }
            qs[(part * NK + ks) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
          }
      }
      __syncthreads();
    }

    float o[NT][4], ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    // The tiles in which some row of the item can see something: of [t0, t1) those of the first tokens, then those
    // from w0 on.
    int tb = t1, w0 = t0, ahead = 0;
    if (!SEL) {
      const int last = (int)(min64(p_hi, hi) < 0 ? -1 : min64(p_hi, hi) / kTile);  // tile of the last position
      tb = min(tb, last < e.lo_tile ? min(e.sink_tiles, last + 1) : e.sink_tiles + last - e.lo_tile + 1);
      if (a.window > 0) {
        const int sinks_end = (int)((min64(a.sinks, hi + 1) + kTile - 1) / kTile);
        const int from = (int)(min64(max64(p_lo - a.window + 1, 0), max(hi, 0)) / kTile);
        ahead = max(min(tb, sinks_end) - t0, 0);
        w0 = max(max(t0, sinks_end), e.sink_tiles + from - e.lo_tile);
      }
    } else if (hi < 0) {
      tb = t0;
    }
    const int steps = ahead + max(tb - w0, 0);
    const int gap = w0 - ahead + (SEL ? 0 : e.lo_tile - e.sink_tiles);  // places in the line to tiles, past the first tokens'
    auto base_of = [&](int step) {  // first of this warp's tokens (positions, or places in the list)
      return (step < ahead ? t0 + step : gap + step) * kTile + warp * kWTok;
    };

    // Look-ups run ahead of the copies, a step between each and the next: list entries (selected), then pages, then the
    // copies and the scales.  What a load brings is not looked at before the step after.
    const int32_t* const list = SEL ? a.indices + row0 * a.idx_stride : nullptr;
    auto load_entry = [&](int step) -> int {  // a lane's position of a step, as the list has it
      int i = -1;
      if (step < steps) i = base_of(step) + lane;
      if (SEL) {
        int s = -1;
        if (i >= 0 && i < a.topk) s = __ldg(list + i);
        return s;
      }
      return i;
    };
    const int32_t* const table = a.st.table + (int64_t)max(b, 0) * a.st.stride;
    auto load_page = [&](int s) -> int {  // page of a lane's position, as the table has it; -1: there is none
      int page = -1;
      const uint32_t i = (uint32_t)max(s, 0) / (uint32_t)a.c.ps;
      if (s >= 0 && s <= hi && i < (uint32_t)a.st.width) page = __ldg(table + i);
      return page;
    };
    // The copies of one step, and the loads of the lane's token's scales.  They are kept beside the copies: ke + 127 in
    // the low byte, ve as bf16 in the upper half; 0 where the token is absent.
    int pend_ke = 0, pend_ve = 0;
    bool pend_there = false;
    uint32_t pend_at = 0;
    auto issue = [&](int step, int s, int page) {
      const uint32_t at_stage = (step % kStages) * S::kStageBytes;
      const uint32_t dst = ring + at_stage + lane * 16;
      uint32_t in = 0;
      int slot = -1;  // row of the cache
      pend_at = at_stage;
      pend_there = page >= 0 && page < a.c.pages;
      if (pend_there) {
        in = (uint32_t)s % (uint32_t)a.c.ps;
        const int ph = page * a.c.hk + h;
        slot = ph * a.c.ps + (int)in;
        const int64_t be = (int64_t)ph * (a.c.ps / kKvBlock) + in / kKvBlock;
        pend_ke = __ldg(a.c.ke + be);
        pend_ve = __ldg(a.c.ve + be);
      }
      const uint32_t vdst = ring + at_stage + S::kKPieces * 512 + lane * S::kVBytes;
      const uint8_t* const ksrc = a.c.k + 16 * tig;
      const uint8_t* const vsrc = a.c.v + S::kVBytes * g;
      auto copies = [&](auto every) {  // every token is there
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int sl = __shfl_sync(~0u, slot, 8 * j + g);
          const uint8_t* src = ksrc + (int64_t)(uint32_t)(every ? sl : max(sl, 0)) * D;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            cp_async_or_zero<16>(dst + (j * (D / 64) + c) * 512, src + 64 * c, every || sl >= 0);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int sl = __shfl_sync(~0u, slot, 16 * (j / 4) + 8 * (j / 2 % 2) + 2 * tig + j % 2);
          cp_async_or_zero<S::kVBytes>(vdst + j * 32 * S::kVBytes, vsrc + (int64_t)(uint32_t)(every ? sl : max(sl, 0)) * D,
                                       every || sl >= 0);
        }
      };
      if (__all_sync(~0u, slot >= 0)) copies(std::true_type{});
      else copies(std::false_type{});
    };
    // The scales of the copies issued last, one step later.
    auto settle = [&]() {
      const uint32_t ex = pend_there ? (uint32_t)(max(pend_ke, -126) + 127) | __float_as_uint((float)pend_ve) : 0u;
      *reinterpret_cast<uint32_t*>(smem + (ring - smem_u32(smem)) + pend_at + S::kKPieces * 512 + 256 * S::kVBytes + lane * 4) = ex;
    };

    // One loop for both ends: step + kStages is copied after step was computed, and the first kStages before any was.
    // (Its code is read once; a CTA's first pass through new code costs more than its work.)
    int s_next = load_entry(0), s_after = load_entry(1);
    int page_next = load_page(s_next);
#pragma unroll 1
    for (int step = -kStages; step < steps; ++step) {
     if (step >= 0) {
      cp_async_wait<kStages - 1>();  // a lane reads only what it copied itself; the scales are the warp's
      __syncwarp();
      const uint8_t* const kst = smem + (ring - smem_u32(smem)) + (step % kStages) * S::kStageBytes;
      const uint8_t* const vst = kst + S::kKPieces * 512;
      const uint32_t* const scales = reinterpret_cast<const uint32_t*>(vst + 256 * S::kVBytes);
      const int base = base_of(step);

      // scores: 4 tiles of 8 tokens
      float z[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j][0] = z[j][1] = z[j][2] = z[j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 kw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          kw[j] = *reinterpret_cast<const uint4*>(kst + (j * (D / 64) + c) * 512 + lane * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t b0[4], b1[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = k == 0 ? kw[j].x : k == 1 ? kw[j].y : k == 2 ? kw[j].z : kw[j].w;
            b0[j] = cvt_e4m3x2(w);
            b1[j] = cvt_e4m3x2(w >> 16);
          }
#pragma unroll
          for (int part = S::kQParts - 1; part >= 0; --part) {
            const uint4 w = reinterpret_cast<const uint4*>(smem + S::kRing)[(part * NK + 4 * c + k) * 32 + lane];
            const uint32_t aq[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16816(z[j], aq, b0[j], b1[j]);
          }
        }
      }

      // mask
      const bool whole = __all_sync(~0u, scales[lane] != 0) &&
                         (SEL || (base + kWTok - 1 <= whole_upto && (base >= whole_from || base + kWTok <= sinks)));
      uint32_t te[4][2];  // scales of the two tokens that this lane holds in each tile
      if (SEL) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 w = *reinterpret_cast<const uint2*>(scales + 8 * j + 2 * tig);
          te[j][0] = w.x, te[j][1] = w.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2)  // a block's tokens share one
          te[j][0] = te[j][1] = te[j + 1][0] = te[j + 1][1] = scales[8 * j];
      }
      if (!whole) {
        stay(z);  // or the compiler masks every step
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int s = base + 8 * j + 2 * tig + k;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool seen = te[j][k] && (SEL || (s <= sees_upto[i] && (s >= sees_from[i] || s < sinks)));
              if (!seen) z[j][2 * i + k] = -INFINITY;
            }
          }
      }
      // some row sees a token of this step that another does not
      const bool part_seen = !SEL && !whole;

      // weights: p for the sum, p * 2^(ve + 2) for the product.  Where a row's do not fit fp16, or it has no reference
      // yet, it takes a new one from the scores in hand, and its sums so far are scaled down.
      uint32_t pa[2][4], pb[2][4];  // operands of the two blocks; fp32: 2^11 times the rest of them
      float psum[2];
#pragma unroll 1
      for (bool fresh = true;; fresh = false) {
        const float r0 = ref[0] == -INFINITY ? 0.f : ref[0], r1 = ref[1] == -INFINITY ? 0.f : ref[1];
        float wsum[2] = {0.f, 0.f};
        psum[0] = psum[1] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float w[2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float ks = __uint_as_float(te[j][k] << 23), vs = ex2(__uint_as_float(te[j][k] & 0xFFFF0000u) + kLift);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // a factor of 0 would make a hidden score, -inf, NaN
              const float p = ex2(fmaf(z[j][2 * i + k], fmaxf(unit[i] * ks, 1e-37f), i ? -r1 : -r0));
              psum[i] += p;
              w[i][k] = p * vs;
              wsum[i] += w[i][k];
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t hw = pack_f16(w[i][0], w[i][1]);
            pa[j / 2][2 * (j % 2) + i] = hw;
            if (!BF16) {
              const __half2 hh = *reinterpret_cast<const __half2*>(&hw);
              pb[j / 2][2 * (j % 2) + i] = pack_f16((w[i][0] - __low2float(hh)) * kRest, (w[i][1] - __high2float(hh)) * kRest);
            }
          }
        }
        bool over[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) over[i] = wsum[i] > 32768.f || (fresh && ref[i] == -INFINITY);
        if (!__any_sync(~0u, over[0] || over[1])) break;
        stay(z);
        bool raised = false;
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              t = fmaxf(t, fmaf(z[j][2 * i + k], fmaxf(unit[i] * __uint_as_float(te[j][k] << 23), 1e-37f),
                                __uint_as_float(te[j][k] & 0xFFFF0000u)));
          t = quad_max(t);  // the four lanes of a row decide together
          const bool raise = quad_max(over[i] ? 1.f : 0.f) > 0.f && t > ref[i];
          const float down = raise && ref[i] != -INFINITY ? ref[i] - t : 0.f;
          f[i] = ex2(down);
          if (raise) ref[i] = t;
          l[i] = kv_down(l[i], down);
          raised |= raise;
        }
        if (!__any_sync(~0u, raised)) break;
        if (__any_sync(~0u, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int n8 = 0; n8 < NT; ++n8) o[n8][0] *= f[0], o[n8][1] *= f[0], o[n8][2] *= f[1], o[n8][3] *= f[1];
        }
      }
      l[0] += psum[0];
      l[1] += psum[1];

      // output sums: 16 tokens a block, NT tiles of 8 dims
      constexpr int VW = S::kVBytes / 4;  // words a lane holds of a value
      auto value = [&](int u, uint32_t (&w)[4][VW]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* at4 = vst + (4 * u + j) * 32 * S::kVBytes + lane * S::kVBytes;
          if (VW == 4) {
            const uint4 r = *reinterpret_cast<const uint4*>(at4);
            w[j][0] = r.x, w[j][1] = r.y, w[j][VW == 4 ? 2 : 0] = r.z, w[j][VW == 4 ? 3 : 1] = r.w;
          } else {
            const uint2 r = *reinterpret_cast<const uint2*>(at4);
            w[j][0] = r.x, w[j][1] = r.y;
          }
        }
      };
      // A weight of zero does not hide a NaN value from a matrix instruction.  Tokens that no row sees were zeroed
      // on the way in; one that some rows see and others do not gets its product row by row.
      bool odd = false;
      if (part_seen) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t w[4][VW];
          value(u, w);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < VW; ++k) odd |= __vcmpeq4(w[j][k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
        }
        odd = __any_sync(~0u, odd);
      }
      auto product = [&](auto by_row, int only) {  // by_row: of row `only` alone
        int upto = 0, from = 0;  // what that row sees: its lanes hold it
        if (by_row) {
          upto = __shfl_sync(~0u, only < 8 ? sees_upto[0] : sees_upto[1], only % 8 * 4);
          from = __shfl_sync(~0u, only < 8 ? sees_from[0] : sees_from[1], only % 8 * 4);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t w[4][VW];
          value(u, w);
          if (by_row) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int s = base + 16 * u + 8 * (j / 2) + 2 * tig + j % 2;
              if (!(s <= upto && (s >= from || s < sinks))) {
#pragma unroll
                for (int k = 0; k < VW; ++k) w[j][k] = 0u;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < VW; ++k) {
            const uint32_t l0 = __byte_perm(w[0][k], w[1][k], 0x5140), h0 = __byte_perm(w[0][k], w[1][k], 0x7362);
            const uint32_t l1 = __byte_perm(w[2][k], w[3][k], 0x5140), h1 = __byte_perm(w[2][k], w[3][k], 0x7362);
            const uint32_t b0[4] = {cvt_e4m3x2(l0), cvt_e4m3x2(l0 >> 16), cvt_e4m3x2(h0), cvt_e4m3x2(h0 >> 16)};
            const uint32_t b1[4] = {cvt_e4m3x2(l1), cvt_e4m3x2(l1 >> 16), cvt_e4m3x2(h1), cvt_e4m3x2(h1 >> 16)};
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              if (BF16 && !by_row) {
                mma16816(o[4 * k + q4], pa[u], b0[q4], b1[q4]);
              } else {  // fp32: a block's own sum first, then one addition
                float t4[4] = {0.f, 0.f, 0.f, 0.f};
                if (!BF16) {
                  mma16816(t4, pb[u], b0[q4], b1[q4]);
#pragma unroll
                  for (int i = 0; i < 4; ++i) t4[i] *= 1.f / kRest;
                }
                mma16816(t4, pa[u], b0[q4], b1[q4]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (!by_row || only == g + 8 * (i / 2)) o[4 * k + q4][i] += t4[i];
              }
            }
          }
        }
      };
      if (!odd) {
        product(std::false_type{}, 0);
      } else {
#pragma unroll 1
        for (int only = 0; only < valid; ++only) product(std::true_type{}, only);
      }
     }

      // the next copies go where this step's were; every lane is past its own reads, and the warp past the scales
      __syncwarp();
      if (step > -kStages) settle();
      if (step + kStages < steps) issue(step + kStages, s_next, page_next);
      cp_async_commit();
      page_next = load_page(s_after);
      s_next = s_after;
      s_after = load_entry(step + kStages + 2);
    }

    // the warps' results together, in shared memory
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) l[i] = quad_sum(l[i]);
    if (tig == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* st = stats + warp * 64 + (g + 8 * i) * 4;
        st[0] = ref[i], st[1] = l[i];
      }
    }
    __syncthreads();  // also: every warp is done with its ring
    {
      const volatile Place& p = place;
      at = p.at, stop = p.stop, total = p.total, ctas = p.ctas, row0 = p.row0, row = p.row;
      t0 = p.t0, t1 = p.t1, t = p.t, end = p.end, rr0 = p.rr0, h = p.h, valid = p.valid, x = p.x, b = p.b, per_b = p.per_b;
      e.first = p.e.first, e.hi = p.e.hi, e.sink_tiles = p.e.sink_tiles, e.lo_tile = p.e.lo_tile, e.tiles = p.e.tiles;
      e.row_tiles = p.e.row_tiles;
    }
    // [warp][16 rows], 4 dims a piece: the pieces that the four lanes of a row store at a time stand side by side
    float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w * 64 + r * 4]);
      // a row that saw nothing here has sums of zero, whatever its queries are
      const bool none = ref[i] == -INFINITY && l[i] == 0.f;
      const float f = ref[i] == -INFINITY ? 1.f : ex2(ref[i] - top);
      float* to = sums + (warp * kRowsT + r) * S::kSumStride + 4 * tig;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n8 = 0; n8 < NT; n8 += 4)
          *reinterpret_cast<float4*>(to + 4 * (k * NT + n8)) =
              make_float4(none ? 0.f : o[n8][2 * i + k] * f, none ? 0.f : o[n8 + 1][2 * i + k] * f,
                          none ? 0.f : o[n8 + 2][2 * i + k] * f, none ? 0.f : o[n8 + 3][2 * i + k] * f);
    }
    __syncthreads();
    const bool all = t0 == 0 && t1 == e.tiles;
    float* const part = line.part + ((int64_t)blockIdx.x * 2 + (t0 == 0)) * kv_part_floats(kRowsT, D);
    constexpr int kLanes = D / 4;  // threads of a row
    for (int r = tid / kLanes; r < valid; r += kThreads / kLanes) {
      const int c = tid % kLanes * 4;
      float top = -INFINITY, lt = 0.f;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        top = fmaxf(top, stats[w * 64 + r * 4]);
        const float4 v = *reinterpret_cast<const float4*>(sums + (w * kRowsT + r) * S::kSumStride +
                                                          4 * (c % (2 * NT)) + 4 * (c / (2 * NT)));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float rw = stats[w * 64 + r * 4], lw = stats[w * 64 + r * 4 + 1];
        lt += rw == -INFINITY ? lw : kv_down(lw, rw - top);  // -inf: zero, or NaN of a score
      }
      if (all) {
        const int64_t rr = row0 + (rr0 + r) / a.group;
        if (rr < a.st.rows) {
          const int j = h * a.group + (rr0 + r) % a.group;
          const float f = lt == 0.f ? 0.f : ex2(-kLift) / lt;
          kv_store4(a, (rr * a.hq + j) * (int64_t)D + c, s.x * f, s.y * f, s.z * f, s.w * f, BF16);
          if (a.lse && c == 0) a.lse[rr * a.hq + j] = lt == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(lt));
        }
      } else {
        *reinterpret_cast<float4*>(part + r * D + c) = s;
        if (c == 0) *reinterpret_cast<float4*>(part + kRowsT * D + r * 4) = make_float4(top, lt, 0.f, 0.f);
      }
    }
    if (!all && t0 == 0 && tid == 0)
      *open = {row0, (int)blockIdx.x, h * a.group, rr0, valid, kv_parts(at - t + e.tiles + kItemCost, total, ctas) - (int)blockIdx.x};
    __syncthreads();  // the ring is free again
    }

    at += end - t;
    t = 0;
    if (++x == per_b && at < stop) {
      x = 0;
      if (SEL) {
        ++row;
        if (row >= a.st.off[b + 1]) b = kv_sequence_of(a.st, row);
      } else {
        do e = extent_of(a, ++b);
        while (e.row_tiles == 0 && b + 1 < a.st.B);
        if (e.row_tiles == 0) break;  // as above
        per_b = a.c.hk * e.row_tiles;
      }
    }
  }
}

// Joins the partial results of an item that several CTAs worked on: blocks (c, y) those that CTA c began.  `per_row`
// warps take one of the item's rows together, lanes four dims; the order of the sums is fixed by the line alone.
constexpr int kMergeWarps = 8;
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kMergeWarps)
    kv_merge_kernel(const KvAttnArgs a, const KvLine line, const int rows, const float lift, const int per_row) {
  __shared__ float sums[kMergeWarps][D + 4];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (line.gate && *line.gate == 0) return;
  const KvOpen op = line.open[blockIdx.x];
  if (!op.open) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = warp % per_row;
  const int more = op.open - 1;  // CTAs c + 1 .. c + more work on the item's other tiles
  const int r = blockIdx.y * (kMergeWarps / per_row) + warp / per_row;
  if (per_row == 1 && r >= op.valid) return;
  auto part_of = [&](int i) {  // the first one stands in the place of an item begun, the others in that of one ended
    return line.part + ((int64_t)(op.stretch + i) * 2 + (i == 0)) * kv_part_floats(rows, D);
  };
  const int64_t stat_at = (int64_t)rows * D + (int64_t)min(r, rows - 1) * 4;
  float u = -INFINITY;  // the largest reference
  for (int i = lane; i <= more; i += 32) u = fmaxf(u, part_of(i)[stat_at]);
#pragma unroll
  for (int o = 16; o; o >>= 1) u = fmaxf(u, __shfl_xor_sync(~0u, u, o));
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool mine = lane * 4 < D && r < op.valid;
#pragma unroll 4
  for (int i = sub; i <= more; i += per_row) {
    const float* p = part_of(i);
    const float2 s = *reinterpret_cast<const float2*>(p + stat_at);
    const float4 v = mine ? *reinterpret_cast<const float4*>(p + r * D + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float f = s.x == -INFINITY ? (s.y == 0.f ? 0.f : 1.f) : ex2(s.x - u);  // no reference: nothing, or NaN of a score
    l = fmaf(s.y, f, l);
    if (f == 0.f) l += kv_down(s.y, s.x - u);  // l may count where 2^(s.x - u) alone lies below fp32's normal range
    else acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
  }
  if (per_row > 1) {
    if (lane * 4 < D) *reinterpret_cast<float4*>(&sums[warp][lane * 4]) = acc;
    if (lane == 0) sums[warp][D] = l;
    __syncthreads();
    if (sub) return;
    for (int w = 1; w < per_row; ++w) {
      l += sums[warp + w][D];
      if (lane * 4 < D) acc.x += sums[warp + w][lane * 4], acc.y += sums[warp + w][lane * 4 + 1],
                        acc.z += sums[warp + w][lane * 4 + 2], acc.w += sums[warp + w][lane * 4 + 3];
    }
  }
  const int64_t row = op.row0 + (op.rr0 + r) / a.group;
  if (r >= op.valid || row >= a.st.rows) return;
  const int j = op.head0 + (op.rr0 + r) % a.group;
  const float f = l == 0.f ? 0.f : ex2(-lift) / l;
  if (mine) kv_store4(a, (row * a.hq + j) * (int64_t)D + lane * 4, acc.x * f, acc.y * f, acc.z * f, acc.w * f, BF16);
  if (a.lse && lane == 0) a.lse[row * a.hq + j] = l == 0.f ? -INFINITY : 0.6931471805599453f * (u + log2f(l));
}

// The most items that a call can have, and tiles of each.
int64_t most_items(const KvAttnArgs& a) {
  return a.indices ? a.st.rows * a.c.hk * ((a.group + kRowsT - 1) / kRowsT)
                   : (a.st.B + a.st.rows * a.group / kRowsT) * (int64_t)a.c.hk;
}
int64_t most_tiles(const KvAttnArgs& a) {
  if (a.indices) return (a.topk + kTile - 1) / kTile;
  const int64_t cap = (int64_t)a.st.width * a.c.ps;
  return (cap + kTile - 1) / kTile + (a.window > 0 ? 1 : 0);
}

// Items of one or two tiles are not cut: a CTA takes whole ones, and no launch joins parts (a list of 97 for 8 rows:
// 6.6 us in a graph against 7.6).  With more the cut pays (512 tokens, 8 key heads, in 5 tiles: 15.3 us whole, 14.4 cut).
bool whole_items(const KvAttnArgs& a) { return most_tiles(a) <= kWholeTiles; }

// CTAs of the line: as many as the device holds at once, but no more than there can be places.
int line_ctas(int sms, const KvAttnArgs& a) {
  const int64_t per = !a.is_bf16 || (a.c.d == 128 && !a.indices) ? 2 : 3;
  const int64_t places = most_items(a) * (whole_items(a) ? 1 : most_tiles(a) + kItemCost);
  return (int)std::max<int64_t>(1, std::min<int64_t>(per * sms, places));
}

KvLine carve_line(void* ws, int ctas) {
  char* p = static_cast<char*>(ws);
  KvLine line;
  line.status = reinterpret_cast<int*>(p);
  line.open = reinterpret_cast<KvOpen*>(p + 256);
  line.part = reinterpret_cast<float*>(p + 256 + (size_t)ctas * sizeof(KvOpen));
  return line;
}

template <int D, bool BF16, bool SEL>
cudaError_t launch_line(const KvAttnArgs& a, int ctas, const KvLine& line, cudaStream_t s) {
  using Sh = Shape<D, BF16, SEL>;
  cudaError_t e = kv_allow_smem<kv_attn_kernel<D, BF16, SEL>>(Sh::kBytes);
  if (e != cudaSuccess) return e;
  kv_attn_kernel<D, BF16, SEL><<<ctas, kThreads, Sh::kBytes, s>>>(a, line);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1 || line.whole) return e;
  // Few items cut into many parts: all warps of a block for a row; else a warp.
  return launch_kv_merge(a, line, ctas, kRowsT, ctas > 8 * most_items(a), kLift, s);
}

}  // namespace

// Of the most CTAs an SM holds.
size_t kv_attn_workspace(int sms, int d) {
  return 256 + (size_t)3 * sms * (sizeof(KvOpen) + 2 * kv_part_floats(kRowsT, d) * sizeof(float));
}

cudaError_t launch_kv_merge(const KvAttnArgs& a, const KvLine& line, int ctas, int rows, bool many, float lift,
                            cudaStream_t s) {
  const int per_row = many ? kMergeWarps : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)(rows * per_row / kMergeWarps));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its launch overlaps the kernel before it
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (a.c.d == 128)
    return a.is_bf16 ? cudaLaunchKernelEx(&cfg, kv_merge_kernel<128, true>, a, line, rows, lift, per_row)
                     : cudaLaunchKernelEx(&cfg, kv_merge_kernel<128, false>, a, line, rows, lift, per_row);
  return a.is_bf16 ? cudaLaunchKernelEx(&cfg, kv_merge_kernel<64, true>, a, line, rows, lift, per_row)
                   : cudaLaunchKernelEx(&cfg, kv_merge_kernel<64, false>, a, line, rows, lift, per_row);
}

cudaError_t launch_kv_attn(const KvAttnArgs& a, int sms, void* ws, const int* gate, cudaStream_t s) {
  const int ctas = line_ctas(sms, a);
  KvLine line = carve_line(ws, ctas);
  line.gate = gate;
  line.whole = whole_items(a);
  const bool sel = a.indices != nullptr;
  if (a.c.d == 128) {
    if (a.is_bf16) return sel ? launch_line<128, true, true>(a, ctas, line, s) : launch_line<128, true, false>(a, ctas, line, s);
    return sel ? launch_line<128, false, true>(a, ctas, line, s) : launch_line<128, false, false>(a, ctas, line, s);
  }
  if (a.is_bf16) return sel ? launch_line<64, true, true>(a, ctas, line, s) : launch_line<64, true, false>(a, ctas, line, s);
  return sel ? launch_line<64, false, true>(a, ctas, line, s) : launch_line<64, false, false>(a, ctas, line, s);
}

}  // namespace pivot
