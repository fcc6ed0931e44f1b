// kv_attention_tc.cu -- attention over the paged 8-bit cache with many query rows for a key head (a group of draft
// tokens of many heads, a chunk of a prompt): bf16 queries, d = 128, on the tcgen05 tensor cores.
//
// The same sums as kv_attention.cu, for items of 128 query rows by tiles of 128 tokens:
//   S = Q K^T   kind::f8f6f4.  Keys are multiplied as they lie in the cache: TMA brings e4m3 pages into the swizzled
//               operand layout, nothing is converted.  A bf16 query has 8 bits: two e4m3 parts of 4 bits hold it
//               (scaled to [2^7, 2^8); what lies 2^-9 below a row's largest keeps fewer, and is off by up to 2^-17 of
//               that largest), two products into one sum.
//   O += P V    kind::f16.  Weights leave the softmax as fp16 and stay in tensor memory; four warps turn the values
//               into fp16 (an e4m3 product would leave the weights 4 bits).
// Two tiles are in work at a time, each with its own S, P and softmax warpgroup, into one O: while one is in the
// softmax, the tensor core multiplies for the other, and a tile's scores are there before its warpgroup has finished
// the weights of the tile before.  A row has one reference u, which lags behind its largest score by what fp16 holds;
// it passes from tile to tile in shared memory, in the tiles' order, so that results do not depend on timing.
//
// What bounds it: for full items the softmax (a tile's 128 x 128 exponentials are 1024 clocks of an SM, its products
// 1060, and what else the softmax warps issue comes on top); with half the rows or fewer the cache's bytes.
// Measured: rows 4096 .. 8191 of a prompt, 32 query and 4 key heads: 552 us, 746 TFLOP/s of the 4 d a visible pair
// (46 % of the measured bf16 burst).  32 sequences of 16000 to 200000 tokens, 4 rows of 32 heads on 2: 616 us, 3.1 TB/s
// (47 %; 592 to 630 us from one B200 to the next), where kv_attention.cu takes 3600.  Four softmax warpgroups, each with
// half the registers, took 995 and 714 us where two took 662 and 611; loops unrolled (past the instruction cache) twice as
// long.
#include <type_traits>

#include "kv.cuh"

namespace pivot {
namespace {

constexpr int D = 128, M = 128, kTok = 128;
constexpr int kKS = 4, kVS = 3, kMeta = 8;   // stages of keys, of raw values, of the blocks' scales
constexpr int kTileB = kTok * D;             // bytes of an e4m3 tile
constexpr int kSoft = 256, kConv = 128;      // threads: two softmax warpgroups, one of the converters
constexpr int kWConv = kSoft / 32, kWTma = kWConv + kConv / 32, kWQk = kWTma + 1, kWPv = kWQk + 1;
constexpr int kThreads = 32 * (kWPv + 1);
constexpr int kItemCost = 8;   // what an item costs beside its tiles, in tiles
constexpr float kLift = 2.f;  // a weight of the row's reference is 2^2 in fp16, the largest thus 2^2 to 2^3
// Values' exponents up to here are this kernel's.  It sums weights 2^(z + ve - u + 2) in fp32, 2^-ve times them for l: with
// exponents 76 apart at most (they begin at -60), a token of 2^-52 of the row's largest p still counts.
constexpr int kTopExp = 16;

struct Meta {  // of a tile's 8 blocks
  float ks[8], ve[8], iv[8];  // 2^ke, ve, 2^-ve
  uint32_t present;           // one bit a block
  uint32_t pad[7];
};

struct TcArgs {
  KvAttnArgs a;
  KvLine line;
  int* gate;            // set where kv_attn_kernel must compute the call again: a masked place holds a NaN value, a value's
                        // exponent is above kTopExp, or a wait ran out here
  int64_t slots;        // rows of the cache's tensor maps
  uint64_t timeout_ns;
  bool stall;           // test hook: the product waits for weights of a thread that there is not
};

// ---------------------------------------------------------------- items: 128 query rows of a sequence and key head
struct Item {
  int b, h, rt, row_tiles;
  int64_t row0, first, p_lo, p_hi;  // first row's index; positions of the sequence's first row, of the item's
  int hi, rr0, valid;               // last position there is; first query row, how many
  int ahead, w0, tiles;             // tiles of the first tokens, first tile after them, all
  __device__ int tile(int k) const { return k < ahead ? k : w0 + k - ahead; }
};

struct Seq {
  int64_t row0, first;
  int hi, row_tiles;
  int64_t n;
};

__device__ __forceinline__ Seq seq_of(const KvAttnArgs& a, int b) {
  Seq s{};
  if (b >= a.st.B) return s;
  s.row0 = a.st.off[b];
  s.n = max64(a.st.off[b + 1] - s.row0, 0);
  const int64_t len = a.st.lens[b];
  s.first = len - s.n;
  s.hi = (int)max64(min64(len, (int64_t)a.st.width * a.c.ps) - 1, -1);
  s.row_tiles = (int)((s.n * a.group + M - 1) / M);
  return s;
}

// Which tiles item rt of a sequence reads: those of the first tokens, then from w0 to its last position.
__device__ __forceinline__ int tiles_of(const KvAttnArgs& a, const Seq& s, int rt, Item* it = nullptr) {
  const int64_t rr0 = (int64_t)rt * M;
  const int valid = (int)min64(M, s.n * a.group - rr0);
  const int64_t p_lo = s.first + rr0 / a.group, p_hi = s.first + (rr0 + valid - 1) / a.group;
  const int64_t last = min64(p_hi, s.hi);
  int ahead = 0, w0 = 0, tiles = 1;
  if (last >= 0) {
    const int lt = (int)(last / kTok);
    if (a.window > 0) {
      ahead = min((int)((min64(a.sinks, s.hi + 1) + kTok - 1) / kTok), lt + 1);
      w0 = max(ahead, (int)(min64(max64(p_lo - a.window + 1, 0), last) / kTok));
      tiles = ahead + max(lt - w0 + 1, 0);
    } else {
      tiles = lt + 1;
    }
  }
  if (it) {
    it->rt = rt;
    it->row_tiles = s.row_tiles;
    it->row0 = s.row0;
    it->first = s.first;
    it->hi = s.hi;
    it->rr0 = (int)rr0;
    it->valid = valid;
    it->p_lo = p_lo;
    it->p_hi = p_hi;
    it->ahead = ahead;
    it->w0 = w0;
    it->tiles = tiles;
  }
  return tiles;
}

// Places in the line of a sequence and one key head: each item's tiles behind kItemCost.  `wide`: the warp's lanes share
// one sequence's items; else a lane has its own.
__device__ __forceinline__ int64_t seq_tiles(const KvAttnArgs& a, const Seq& s, bool wide, int lane) {
  int64_t t = 0;
  for (int rt = wide ? lane : 0; rt < s.row_tiles; rt += wide ? 32 : 1) t += tiles_of(a, s, rt) + kItemCost;
  if (wide) {
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
  }
  return t;
}

// The CTA's stretch of the line, walked by every role for itself (all lanes of a warp together).
struct Walk {
  int64_t at, stop, total, ctas;
  Item it;
  Seq s;
  int place, end;  // places [place, end) of the item in the stretch
  int t0, t1;      // its tiles among them
  bool live;

  // tiles of 32 sequences, one a lane
  __device__ int64_t weights(const KvAttnArgs& a, int b0, int lane) const {
    const Seq q = seq_of(a, b0 + lane);
    int64_t mine = 0;
    unsigned many = __ballot_sync(~0u, q.row_tiles > 8);
    if (q.row_tiles <= 8) mine = seq_tiles(a, q, false, lane);
    while (many) {
      const int l = __ffs(many) - 1;
      many &= many - 1;
      const int64_t t = seq_tiles(a, seq_of(a, b0 + l), true, lane);
      if (lane == l) mine = t;
    }
    return mine * a.c.hk;
  }

  __device__ void start(const KvAttnArgs& a, int lane) {
    total = 0;
    live = false;
    for (int b0 = 0; b0 < a.st.B; b0 += 32) total += weights(a, b0, lane);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    ctas = min64(gridDim.x, total);
    if (blockIdx.x >= ctas) return;
    at = total * blockIdx.x / ctas;
    stop = total * (blockIdx.x + 1) / ctas;
    int64_t run = 0;
    for (int b0 = 0; b0 < a.st.B; b0 += 32) {
      const int64_t w = weights(a, b0, lane);
      int64_t inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += up;
      }
      const unsigned hit = __ballot_sync(~0u, run + inc > at);
      if (hit) {
        const int l = __ffs(hit) - 1;
        int64_t in = at - run - __shfl_sync(~0u, inc - w, l);
        const int64_t per = __shfl_sync(~0u, w, l) / a.c.hk;
        it.b = b0 + l;
        it.h = (int)(in / per);
        in -= it.h * per;
        s = seq_of(a, it.b);
        for (int r0 = 0; r0 < s.row_tiles; r0 += 32) {  // the item: prefix over its sequence's row tiles
          const int64_t v = r0 + lane < s.row_tiles ? tiles_of(a, s, r0 + lane) + kItemCost : 0;
          int64_t pre = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(~0u, pre, o);
            if (lane >= o) pre += up;
          }
          const unsigned here = __ballot_sync(~0u, pre > in);
          if (here) {
            const int k = __ffs(here) - 1;
            tiles_of(a, s, r0 + k, &it);
            cut((int)(in - __shfl_sync(~0u, pre - v, k)));
            live = true;
            if (t1 <= t0) next(a);  // the item begins in the next stretch
            return;
          }
          in -= __shfl_sync(~0u, pre, 31);
        }
        return;  // only where the lengths changed under the call
      }
      run += __shfl_sync(~0u, inc, 31);
    }
  }

  __device__ void cut(int from) {
    place = from;
    end = (int)min64(it.tiles + kItemCost, place + (stop - at));
    t0 = max(place - kItemCost, 0);
    t1 = max(end - kItemCost, 0);
  }

  // To the next item of which the stretch has tiles.
  __device__ void next(const KvAttnArgs& a) {
    do {
      at += end - place;
      if (at >= stop) {
        live = false;
        return;
      }
      int rt = it.rt + 1;
      if (rt == s.row_tiles) {
        rt = 0;
        if (++it.h == a.c.hk) {
          it.h = 0;
          do {
            if (++it.b >= a.st.B) {
              live = false;
              return;
            }
            s = seq_of(a, it.b);
          } while (s.row_tiles == 0);
        }
      }
      tiles_of(a, s, rt, &it);
      cut(0);
    } while (t1 <= t0);
  }
};

struct Tail {
  uint64_t kf[kKS], ke[kKS], vf[kVS], ve[kVS], hf[2], he[2], sf[2], sc[2], pf[2], rf[2], od[2], mf[kMeta], qf, of, xf;
  uint32_t tmem_slot;
  volatile int abort_flag;
  Meta meta[kMeta];
  Walk walk[kWPv + 1];  // one for each warp: in registers it would crowd out the softmax
  float unit[M];
  float ref[M];          // each row's reference, settled tile after tile
  float stats[2][M][2];  // reference and l of each half's tiles
};

constexpr int kOffQ = 0, kOffK = 2 * M * D, kOffV = kOffK + kKS * kTileB, kOffH = kOffV + kVS * kTileB,
              kOffTail = kOffH + 2 * kTok * D * 2;
constexpr size_t kSmem = kOffTail + sizeof(Tail);
static_assert(kSmem <= 232448, "227 KB of dynamic shared memory per CTA");

// Two fp32 values in one register pair, for the packed instructions.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Values that are not to be computed with before this point.
__device__ __forceinline__ void stay(uint32_t (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7]));
}

// Whether every row of the item sees every token of a tile (where its pages are present).
__device__ __forceinline__ bool whole_tile(const KvAttnArgs& a, const Item& it, int base) {
  return base + kTok - 1 <= min64(it.p_lo, it.hi) &&
         (a.window <= 0 || base > it.p_hi - a.window || base + kTok <= a.sinks);
}

__global__ void __launch_bounds__(kThreads, 1)
    kv_attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const TcArgs args) {
  const KvAttnArgs& a = args.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail& T = *reinterpret_cast<Tail*>(smem + kOffTail);
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled operands need it; there is no room to align
    if (threadIdx.x == 0) atomicOr(args.line.status, DEV_ERR_BOUNDS), *args.gate = 1;
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kKS; ++i) mbar_init(&T.kf[i], 1), mbar_init(&T.ke[i], 1);
    for (int i = 0; i < kVS; ++i) mbar_init(&T.vf[i], 1), mbar_init(&T.ve[i], kConv);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&T.hf[i], kConv), mbar_init(&T.he[i], 1);
      mbar_init(&T.sf[i], 1), mbar_init(&T.sc[i], kSoft / 2), mbar_init(&T.pf[i], kSoft / 2 + args.stall);
      mbar_init(&T.rf[i], kSoft / 2), mbar_init(&T.od[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&T.mf[i], 1);
    mbar_init(&T.qf, kSoft);
    mbar_init(&T.of, 1);
    mbar_init(&T.xf, kSoft);
    T.abort_flag = 0;
    fence_mbar_init();
    args.line.open[blockIdx.x].open = 0;
  }
  if (warp == kWQk) {
    tmem_alloc(&T.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = T.tmem_slot;  // 128 columns each of S0, S1 and O, 64 each of P0, P1
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity, args.timeout_ns, &T.abort_flag)) return true;
    T.abort_flag = 1;
    atomicOr(args.line.status, DEV_ERR_TIMEOUT);
    return false;
  };

  Walk& w = T.walk[warp];
  {
    Walk v;
    v.start(a, lane);
    if (lane == 0) w = v;
    __syncwarp();
  }
  auto advance = [&]() {
    __syncwarp();
    if (lane == 0) w.next(a);
    __syncwarp();
  };

  if (warp == kWTma) {
    // ------------------------------------------------------------ copies: pages, scales
    // Lane l looks after block l % 8 of tile l / 8 of four; four tiles' look-ups are under way while the four
    // before them are copied.
    uint32_t n = 0;  // tiles so far
    bool ok = true;
    for (; w.live && ok; advance()) {
      const Item& it = w.it;
      const int nt = w.t1 - w.t0;
      auto position = [&](int k) {  // of this lane's block in the four tiles from k on; -1: none
        const int t = k + lane / 8;
        if (t >= nt) return -1;
        const int p = it.tile(w.t0 + t) * kTok + lane % 8 * kKvBlock;
        return p <= it.hi ? p : -1;
      };
      auto page_at = [&](int p) { return p < 0 ? -1 : kv_page(a.st, a.c, it.b, (uint32_t)p); };
      struct Block {
        int slot;
        int8_t ke, ve;
      };
      auto block_at = [&](int p, int page) {
        Block r{-1, 0, 0};
        if (page >= 0) {
          const int in = (int)((uint32_t)p % (uint32_t)a.c.ps);
          const int ph = page * a.c.hk + it.h;
          r.slot = ph * a.c.ps + in;
          const int64_t e = (int64_t)ph * (a.c.ps / kKvBlock) + in / kKvBlock;
          r.ke = __ldg(a.c.ke + e);
          r.ve = __ldg(a.c.ve + e);
        }
        return r;
      };
      int p1 = position(0);
      Block now = block_at(p1, page_at(p1)), then;
      p1 = position(4);
      int page1 = page_at(p1);
      for (int k = 0; k < nt; ++k, ++n) {
        if (k % 4 == 0) {
          if (k) now = then;
          then = block_at(p1, page1);
          p1 = position(k + 8);
          page1 = page_at(p1);
        }
        const int ks = n % kKS, vs = n % kVS, ms = n % kMeta;
        int good = 1;
        if (lane == 0) good = wait(&T.ke[ks], (n / kKS & 1) ^ 1) && wait(&T.ve[vs], (n / kVS & 1) ^ 1);
        good = __shfl_sync(~0u, good, 0);
        if (!good) {
          ok = false;
          break;
        }
        const bool mine = lane / 8 == k % 4;
        const unsigned there = __ballot_sync(~0u, mine && now.slot >= 0);
        if (mine) {
          Meta& m = T.meta[ms];
          const int i = lane % 8;
          m.ks[i] = kv_scale(now.ke);
          m.ve[i] = (float)now.ve;
          m.iv[i] = kv_exp2i(min(-(int)now.ve, 127));
          if (now.ve > kTopExp && now.slot >= 0) *args.gate = 1;
          if (i == 0) m.present = there >> (8 * (k % 4)) & 0xFFu;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&T.mf[ms]);
          mbar_arrive_expect_tx(&T.kf[ks], kTileB);
          mbar_arrive_expect_tx(&T.vf[vs], kTileB);
        }
        __syncwarp();
        if (mine) {
          const int y = now.slot >= 0 ? now.slot : (int)args.slots;  // behind the last row: zeros
          const int at = lane % 8 * kKvBlock * D;
          tma_load_2d(smem + kOffK + ks * kTileB + at, &kmap, &T.kf[ks], 0, y);
          tma_load_2d(smem + kOffV + vs * kTileB + at, &vmap, &T.vf[vs], 0, y);
        }
      }
    }
  } else if (warp == kWQk || warp == kWPv) {
    // ------------------------------------------------------------ products (one thread of each of two warps, so that
    // one's waits do not keep the other's products back)
    uint32_t n = 0, items = 0, before[2] = {0, 0};  // tiles, items; tiles of each half before this item
    bool ok = true;
    for (; w.live && ok; advance(), ++items) {
      const int nt = w.t1 - w.t0;
      if (lane == 0 && warp == kWQk) {
        const uint32_t qaddr = smem_u32(smem + kOffQ);
        ok = wait(&T.qf, items & 1);
        for (int k = 0; k < nt && ok; ++k) {  // S = Q K^T, once the half's last S has been read
          const uint32_t i = n + k;
          const int ks = i % kKS, s = k & 1;
          ok = (k < 2 || wait(&T.sc[s], (before[s] + (k - 2) / 2) & 1)) && wait(&T.kf[ks], i / kKS & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kaddr = smem_u32(smem + kOffK) + ks * kTileB;
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8(tmem + 128 * s, sw128_kmajor_desc(qaddr + part * M * D + kk * 32),
                      sw128_kmajor_desc(kaddr + kk * 32), idesc_e4m3_f32(M, kTok), part == 0 || kk > 0);
          umma_commit(&T.sf[s]);
          umma_commit(&T.ke[ks]);
        }
      } else if (lane == 0) {
        for (int k = 0; k < nt && ok; ++k) {  // O += P V
          const uint32_t i = n + k;
          const int s = k & 1, hb = i & 1;
          ok = wait(&T.hf[hb], i / 2 & 1) && wait(&T.pf[s], (before[s] + k / 2) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v = smem_u32(smem + kOffH) + hb * (kTok * D * 2);
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk)
            umma_f16_ts(tmem + 256, tmem + 384 + 64 * s + 8 * kk,
                        sw128_mnmajor_desc(v + kk * 16 * 128, kTok * 128, 1024), idesc_f16_f32_bmn(M, D), k > 0 || kk > 0);
          umma_commit(&T.od[s]);
          umma_commit(&T.he[hb]);
        }
        if (ok) umma_commit(&T.of);  // the item's scores were all read before its last weights came
      }
      n += nt;
      before[0] += (nt + 1) / 2;
      before[1] += nt / 2;
      ok = __shfl_sync(~0u, (int)ok, 0);
    }
  } else if (warp >= kWConv) {
    // ------------------------------------------------------------ values to fp16: a thread for a token
    const int t = tid - kSoft;
    uint32_t n = 0;
    bool ok = true;
    for (; w.live && ok; advance()) {
      const int nt = w.t1 - w.t0;
      for (int k = 0; k < nt; ++k, ++n) {
        const int vs = n % kVS, hb = n & 1;
        const int base = w.it.tile(w.t0 + k) * kTok;
        ok = wait(&T.vf[vs], n / kVS & 1) && wait(&T.he[hb], (n / 2 & 1) ^ 1);
        if (!ok) break;
        const uint8_t* src = smem + kOffV + vs * kTileB + t * 128;
        uint8_t* dst = smem + kOffH + hb * (kTok * D * 2) + t * 128;
        const bool look = !whole_tile(a, w.it, base);
        uint32_t odd = 0;
        auto put = [&](int c, uint4 lo, uint4 hi) {  // 16 dims of fp16; dims 0-63, then 64-127
          uint8_t* half = dst + (c / 4) * (kTok * 128);
          const int c2 = (c % 4) * 2;
          *reinterpret_cast<uint4*>(half + ((c2 ^ (t & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(half + (((c2 + 1) ^ (t & 7)) << 4)) = hi;
        };
        if (base + t > w.it.hi) {  // what lies behind the last token stays out of the product
#pragma unroll 1
          for (int c = 0; c < 8; ++c) put(c, make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0));
        } else {
#pragma unroll 4
          for (int c = 0; c < 8; ++c) {
            const uint4 r = *reinterpret_cast<const uint4*>(src + ((c ^ (t & 7)) << 4));
            put(c, make_uint4(cvt_e4m3x2(r.x), cvt_e4m3x2(r.x >> 16), cvt_e4m3x2(r.y), cvt_e4m3x2(r.y >> 16)),
                make_uint4(cvt_e4m3x2(r.z), cvt_e4m3x2(r.z >> 16), cvt_e4m3x2(r.w), cvt_e4m3x2(r.w >> 16)));
          }
          if (look) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              const uint4 r = *reinterpret_cast<const uint4*>(src + (c << 4));
              odd |= __vcmpeq4(r.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(r.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                     __vcmpeq4(r.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(r.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            }
          }
        }
        // A weight of zero does not hide a NaN: where some rows may not see this token, the call is computed again
        // by the kernel that goes row by row.
        if (odd) *args.gate = 1;
        fence_proxy_async_smem();
        mbar_arrive(&T.hf[hb]);
        mbar_arrive(&T.ve[vs]);
      }
      // One lane's wait may run out where another's did not: they leave together, or they would wait for one another at
      // different barriers.
      ok = __all_sync(~0u, ok);
    }
  } else {
    // ------------------------------------------------------------ softmax: a thread for a row, a warpgroup for a half
    const int s = warp / 4, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;  // lane 32 * (warp % 4) in an address' upper half
    const uint32_t sc = tmem + lanes + 128 * s, oc = tmem + lanes + 256, pc = tmem + lanes + 384 + 64 * s;
    // tiles of both halves; items; tiles of this half; of the other before this item
    uint32_t n = 0, items = 0, mine = 0, theirs = 0;
    bool ok = true;
    // after a failed wait the loop only keeps the barriers' count
    for (; w.live; advance(), ++items) {
      const Item& it = w.it;
      const int nt = w.t1 - w.t0;
      const int64_t pos = it.first + (it.rr0 + min(r, it.valid - 1)) / a.group;
      if (s == 0) {  // the query row in two parts
        const int rr = it.rr0 + r;
        const int64_t row = it.row0 + rr / a.group;
        const bool have = r < it.valid && row < a.st.rows;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + row * a.q_stride +
                              (int64_t)(it.h * a.group + rr % a.group) * D;
        auto load = [&](int c) {
          return have ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
        };
        float top = 0.f;
#pragma unroll 8
        for (int c = 0; c < 16; ++c) {
          const uint4 x = load(c);
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[j] << 16)), fabsf(__uint_as_float(v[j] & 0xFFFF0000u))));
        }
        const bool finite = top <= 3.402823466e38f;
        const int ex = top > 0.f && finite ? max((int)(__float_as_uint(top) >> 23) - 127 - 7, -100) : 0;
        const float f = !finite ? __int_as_float(0x7FC00000)  // e4m3 has no infinity: such a row is NaN
                        : a.scale2 < 0.f ? -kv_exp2i(-ex) : kv_exp2i(-ex);  // largest in [2^7, 2^8)
        T.unit[r] = fabsf(a.scale2) * kv_exp2i(ex);
#pragma unroll 2
        for (int c = 0; c < 8; ++c) {  // read again: 128 dims would not stay in registers
          const uint4 x[2] = {load(2 * c), load(2 * c + 1)};
          uint32_t w1[4], w2[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // 4 dims a word
            const uint4& q4 = x[j / 2];
            const uint32_t lo = j % 2 ? q4.z : q4.x, hi = j % 2 ? q4.w : q4.y;
            const float v[4] = {__uint_as_float(lo << 16) * f, __uint_as_float(lo & 0xFFFF0000u) * f,
                                __uint_as_float(hi << 16) * f, __uint_as_float(hi & 0xFFFF0000u) * f};
            uint32_t a1 = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
            a1 |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3) << 16;
            w1[j] = a1;
            const uint32_t h0 = cvt_e4m3x2(a1), h1 = cvt_e4m3x2(a1 >> 16);
            const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&h0)),
                         g1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
            uint32_t a2 =
                __nv_cvt_float2_to_fp8x2(make_float2(v[0] - g0.x, v[1] - g0.y), __NV_SATFINITE, __NV_E4M3);
            a2 |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2] - g1.x, v[3] - g1.y), __NV_SATFINITE, __NV_E4M3)
                  << 16;
            w2[j] = a2;
          }
          uint8_t* to = smem + kOffQ + r * 128 + ((c ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(to) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
          *reinterpret_cast<uint4*>(to + M * D) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();  // the item before: its sums have been read
      mbar_arrive(&T.qf);
      ok = __all_sync(~0u, ok && wait(&T.qf, items & 1));
      const float unit = T.unit[r];
      const bool idle = 32 * (warp % 4) >= it.valid;  // a warp without rows
      // what the row sees, and what all rows do, as positions that fit 32 bits (window and first tokens: all, where
      // there is no window)
      auto small = [](int64_t v) { return (int)min64(max64(v, -1), 0x7FFFFFF0); };
      const int sees_upto = small(min64(it.hi, pos)), whole_upto = small(min64(it.p_lo, it.hi));
      const int sees_from = a.window > 0 ? max(small(pos - a.window + 1), 0) : 0;
      const int whole_from = a.window > 0 ? max(small(it.p_hi - a.window + 1), 0) : 0;
      const int sinks = a.window > 0 ? small(a.sinks) : 0;
      const int tile0 = w.t0, ahead = it.ahead, gap = it.w0 - it.ahead;
      // u: the reference of the row's weights, 2^(z + ve - u + 2) in the product, 2^(z - u + 2) in the sum l
      float u = -INFINITY, l = 0.f;
      for (int k = s; k < nt; k += 2, ++mine) {
        const uint32_t i = n + k;
        if (!ok) continue;
        ok = __all_sync(~0u, wait(&T.mf[i % kMeta], i / kMeta & 1) && wait(&T.sf[s], mine & 1));
        if (!ok) continue;
        tc_fence_after();
        const Meta& me = T.meta[i % kMeta];
        const int kk = k + tile0, base = (kk < ahead ? kk : kk + gap) * kTok;
        const uint32_t present = me.present;
        const bool whole = present == 0xFFu && base + kTok - 1 <= whole_upto && (base >= whole_from || base + kTok <= sinks);
        auto hide = [&](int c, auto all, uint32_t (&x)[32]) {  // of 32 scores, hidden ones become -inf
          if (!all) {
            auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
            const int c0 = base + 32 * c;
            const uint32_t there = ((present >> (2 * c) & 1) ? 0xFFFFu : 0u) | ((present >> (2 * c + 1) & 1) ? 0xFFFF0000u : 0u);
            const uint32_t see = below(sees_upto - c0 + 1) & (~below(sees_from - c0) | below(sinks - c0)) & there;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(see >> j & 1)) x[j] = 0xFF800000u;
          }
        };
        // what a block's scores are multiplied by; never 0: a hidden score, -inf, times it stays -inf
        auto factor = [&](float ks) { return fmaxf(unit * ks, 1e-37f); };
        // One pass: weights relative to the reference u that this half settled on last.  It may lag behind the largest
        // score as long as fp16 holds the weights (32 of them sum to 2^15 at most); a row for which it does not,
        // or that has none yet, takes a new one from the scores in hand, and what it weighed before is scaled down.
        // After an item's first tiles that is rare.  (The loops are not unrolled, and masked tiles have code of their
        // own: the code then stays in the instruction cache.  Unrolled it ran at half the speed, and in one copy the
        // compiler masks every tile.)
        // This tile's first weights, times f: a power of two, so that no weight is rounded twice (a factor of 11 bits put all
        // of a tile's weights off by up to 2^-12 together).  One below fp16's normal range is applied as two: a weight of
        // 2^15 times it is still one that counts.  (Products in fp32 would be 64 instructions more in each of three places:
        // the whole kernel took 18 % longer, with two factors 4 %.)
        auto scale_weights = [&](int columns, float f) {
          const __half2 f1 = __float2half2_rn(fmaxf(f, 0x1p-14f)), f2 = __float2half2_rn(fminf(f * 0x1p14f, 1.f));
          tmem_wait_st();
#pragma unroll 1
          for (int q = 0; q < columns; q += 16) {
            uint32_t y[16];
            tmem_ld32x32b_x16(pc + q, y);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __half2 h = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&y[j]), f1), f2);
              y[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tmem_st32x32b_x16(pc + q, y);
          }
        };
        auto weigh = [&](auto all) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32], y[16];
            tmem_ld32x32b_x32(sc + 32 * c, x);
            const float2 ks = *reinterpret_cast<const float2*>(&me.ks[2 * c]), ve = *reinterpret_cast<const float2*>(&me.ve[2 * c]),
                         iv = *reinterpret_cast<const float2*>(&me.iv[2 * c]);
            const float cb[2] = {factor(ks.x), factor(ks.y)};
            tmem_wait_ld();
            stay(x);
            if (c == 3) {  // S may be overwritten
              tc_fence_before();
              mbar_arrive(&T.sc[s]);
            }
            hide(c, all, x);
            float part = 0.f;
#pragma unroll 1
            for (bool first = true;; first = false) {
              const float ref = u == -INFINITY ? 0.f : u;
              float total = 0.f;
              part = 0.f;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float off = (h ? ve.y : ve.x) - ref + kLift;
                const uint64_t off2 = two(off, off), cb2 = two(cb[h], cb[h]);
                uint64_t sum = two(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                  float d0, d1;
                  split(fma2(two(__uint_as_float(x[16 * h + j]), __uint_as_float(x[16 * h + j + 1])), cb2, off2), d0, d1);
                  d0 = ex2(d0);
                  d1 = ex2(d1);
                  sum = add2(sum, two(d0, d1));
                  y[8 * h + j / 2] = pack_f16(d0, d1);
                }
                float s0, s1;
                split(sum, s0, s1);
                total += s0 + s1;
                part = fmaf(s0 + s1, h ? iv.y : iv.x, part);
              }
              const bool over = total > 32768.f || (first && u == -INFINITY);
              if (!__any_sync(~0u, over)) break;
              stay(x);  // or the compiler takes the maxima of every tile
              float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                t0 = fmaxf(t0, __uint_as_float(x[j]));
                t1 = fmaxf(t1, __uint_as_float(x[16 + j]));
              }
              const float t = floorf(fmaxf(t0 * cb[0] + ve.x, t1 * cb[1] + ve.y));  // whole: factors are powers of two
              const bool raise = over && t > u;
              if (!__any_sync(~0u, raise)) break;
              const float f = raise && u != -INFINITY ? ex2(u - t) : 1.f;
              if (raise) u = t;
              l *= f;
              if (c > 0) scale_weights(16 * c, f);
            }
            l += part;
            if (c == 0 && k >= 2) {  // this half's weights of two tiles ago are used up
              ok = wait(&T.od[s], (mine - 1) & 1);
              tc_fence_after();
            }
            tmem_st32x32b_x16(pc + 16 * c, y);
          }
        };
        if (idle) {
          tc_fence_before();
          mbar_arrive(&T.sc[s]);
          // As the other warps: else it could count for two tiles in one phase of pf, before their weights are there.
          if (k >= 2) ok = wait(&T.od[s], (mine - 1) & 1);
        } else if (whole) {
          weigh(std::true_type{});
        } else {
          weigh(std::false_type{});
        }
        ok = __all_sync(~0u, ok);
        if (!ok) continue;
        // The rows' reference, settled tile after tile: the larger of the tile before's and this one's.
        float before = -INFINITY;
        if (k > 0) {
          ok = __all_sync(~0u, wait(&T.rf[s ^ 1], (theirs + (k - 1) / 2) & 1));
          if (!ok) continue;
          before = T.ref[r];
        }
        const float settled = fmaxf(u, before);
        const float fw = settled > u && u != -INFINITY ? ex2(u - settled) : 1.f;
        const float fo = settled > before && before != -INFINITY ? ex2(before - settled) : 1.f;
        T.ref[r] = settled;
        mbar_arrive(&T.rf[s]);
        if (__any_sync(~0u, fw != 1.f)) {
          l *= fw;
          scale_weights(64, fw);
        }
        u = settled;
        if (__any_sync(~0u, fo != 1.f)) {  // the sums so far, once the tile before has gone into them
          ok = __all_sync(~0u, wait(&T.od[s ^ 1], (theirs + (k - 1) / 2) & 1));
          if (!ok) continue;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D; q += 16) {
            uint32_t y[16];
            tmem_ld32x32b_x16(oc + q, y);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * fo);
            tmem_st32x32b_x16(oc + q, y);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&T.pf[s]);
      }
      theirs += s == 0 ? nt / 2 : (nt + 1) / 2;
      // the item's sums: each warpgroup takes half of the dims
      ok = __all_sync(~0u, ok && wait(&T.of, items & 1));
      tc_fence_after();
      T.stats[s][r][0] = u;
      T.stats[s][r][1] = l;
      mbar_arrive(&T.xf);
      ok = __all_sync(~0u, ok && wait(&T.xf, items & 1));
      if (ok && !idle) {
        const float ref = T.ref[r], u0 = T.stats[0][r][0], u1 = T.stats[1][r][0], l0 = T.stats[0][r][1], l1 = T.stats[1][r][1];
        // a half that saw nothing has l = 0, or NaN of a score
        const float lt = (u0 == -INFINITY ? l0 : l0 * ex2(u0 - ref)) + (u1 == -INFINITY ? l1 : l1 * ex2(u1 - ref));
        const bool none = ref == -INFINITY && lt == 0.f;  // the row saw nothing
        const bool all = w.t0 == 0 && w.t1 == it.tiles;
        const float g = all && !none ? 1.f / lt : 1.f;
        const int rr = it.rr0 + r;
        const int64_t row = it.row0 + rr / a.group;
        const int j = it.h * a.group + rr % a.group;
        const bool put = r < it.valid && row < a.st.rows;
        float* const part = args.line.part + ((int64_t)blockIdx.x * 2 + (w.t0 == 0)) * kv_part_floats(M, D);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int d0 = 64 * s + 32 * c;
          uint32_t x[32];
          tmem_ld32x32b_x32(oc + d0, x);
          tmem_wait_ld();
          if (put) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = none ? 0.f : __uint_as_float(x[e + q]) * g;
              if (all) kv_store4(a, (row * a.hq + j) * (int64_t)D + d0 + e, v[0], v[1], v[2], v[3], true);
              else *reinterpret_cast<float4*>(part + r * D + d0 + e) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        if (put && s == 0) {
          if (all) {
            if (a.lse) a.lse[row * a.hq + j] = none ? -INFINITY : 0.6931471805599453f * (ref - kLift + log2f(lt));
          } else {
            *reinterpret_cast<float4*>(part + M * D + r * 4) = make_float4(ref, lt * ex2(-kLift), 0.f, 0.f);
          }
        }
        if (tid == 0 && !all && w.t0 == 0)
          args.line.open[blockIdx.x] = {it.row0, (int)blockIdx.x, it.h * a.group, it.rr0, it.valid,
                                        kv_parts(w.at - w.place + it.tiles + kItemCost, w.total, w.ctas) - (int)blockIdx.x};
      }
      n += nt;
    }
  }

  __syncthreads();
  if (T.abort_flag) {  // let copies and products in flight end before tensor memory goes
    if (tid == 0) *args.gate = 1;  // what this CTA leaves undone is computed again, without waits
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  if (warp == kWQk) tmem_dealloc(tmem, 512);
}

}  // namespace

size_t kv_attn_tc_workspace(int sms, int d) {
  return 256 + (size_t)sms * (sizeof(KvOpen) + 2 * kv_part_floats(M, D) * sizeof(float)) + kv_attn_workspace(sms, d);
}

cudaError_t launch_kv_attn_tc(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms, void* ws,
                              uint64_t timeout_ns, bool stall, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, s);
  if (e != cudaSuccess) return e;
  char* p = static_cast<char*>(ws);
  TcArgs t{};
  t.a = a;
  t.line.status = reinterpret_cast<int*>(p);
  t.gate = reinterpret_cast<int*>(p + 64);
  t.line.open = reinterpret_cast<KvOpen*>(p + 256);
  t.line.part = reinterpret_cast<float*>(p + 256 + (size_t)sms * sizeof(KvOpen));
  t.slots = (int64_t)a.c.pages * a.c.hk * a.c.ps;
  t.timeout_ns = timeout_ns;
  t.stall = stall;
  e = kv_allow_smem<kv_attn_tc_kernel>(kSmem);
  if (e != cudaSuccess) return e;
  kv_attn_tc_kernel<<<sms, kThreads, kSmem, s>>>(kmap, vmap, t);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_kv_merge(a, t.line, sms, M, sms > 8 * (a.st.B + a.st.rows * a.group / M) * (int64_t)a.c.hk, kLift, s);
  if (e != cudaSuccess) return e;
  return launch_kv_attn(a, sms, p + 256 + (size_t)sms * (sizeof(KvOpen) + 2 * kv_part_floats(M, D) * sizeof(float)),
                        t.gate, s);
}

}  // namespace pivot
