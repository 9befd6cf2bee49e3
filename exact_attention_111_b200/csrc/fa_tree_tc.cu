// fa_tree_tc.cu -- attention of new tokens over the paged cache when a key head has many rows
// (drafted trees, chunks of a prompt): the same mathematics as fa_tree.cu on tcgen05 tensor cores.
//
// A unit's row tile is 256 rows (two 128-row MMA tiles that share every K/V tile); CTA c walks its part
// of the line of chunks (fa_cache.cuh), one chunk = one 128-key tile.  Warp roles (512 threads):
//   warps 0-3, 4-7  softmax groups 0, 1: Q rows into shared memory, then one row per thread
//   warps 8-11      correction: O_q <- alpha O_q in TMEM; makes the V tiles that hold new tokens safe;
//                   E4M3: expands V into the ring
//   warp  12        producer: the K/V ring by TMA, one box per page and 128-byte panel (E4M3: the codes)
//   warp  13        MMA issuer (one thread) and TMEM allocator
//   warps 14-15     E4M3: expand K into the ring
// Tensor memory (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+d), O1 [256+d,256+2d); P
// (16-bit) over the first 64 columns of its S.  Per tile u: O_q += P_q V(u-1), then S_q = Q_q K(u)^T, so
// a finished S_q(u) also says that O_q holds every earlier product.
//
// Why two query tiles: K and V come from L2 or HBM once for 256 rows, and one tile's softmax runs beside the
// other's products.  What bounds it: per 128 keys 2048 cycles of MMA and 2048 of exponentials (16 a clock);
// a tile pair takes 3550 to 3750 at 16 bits (softmax 1850 to 2000, then 1700 to 1750 until the next S: P V and S
// behind the other tile's).  Issue matters: the MMA warp walks converged with its operands in uniform
// registers (trees of 64 tokens 162 -> 156 us).  E4M3: 5300 to 5600 cycles (softmax 3000 to 3400 beside the
// expansions' issue, then 2250); K's staging and expansion, one after the other in one buffer (shared memory is full
// at d = 128), set the pace.
//
// Measured in captured graphs in bursts (at sustained load the clock falls: 185, 153 and 149 us): 8 trees of up to 64
// tokens over up to 16384 keys, 64 query and 8 key heads of 128, bf16: 157 us, 699 TFLOP/s; 2 chunks of 512 over 16000
// keys, 32 and 8 heads, fp16: 137 us, 760 TFLOP/s; 16 trees of up to 48 over up to 8000 E4M3 keys: 147 us, 361 TFLOP/s.
// Where the first's go: 9 to the merge kernel; the slowest CTA takes 1.16 times the median one (the parts are equal
// in chunks, not in rows: chunks 1.25, E4M3 trees 1.18), and the median one's 233000 cycles at 1.73 GHz are 206000 for
// 59 tiles, 15000 for Q and the first S of its segments, 12000 for their results, 2000 to find its part.
//
// A masked product is 0 * v, which is not 0 where v is not finite.  Tiles that hold new tokens (which some
// rows see and others do not) or reach past the end are therefore read once more by the correction
// warps before their product: rows past the sequence's end become zero, and values that are not
// finite do too, noted; the epilogue then adds those of such tiles to the rows that see them.
#include <climits>

#include "fa.h"
#include "fa_cache.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr float kLn2f = 0.693147180559945309f;

template <int D, bool kFp8>
struct BigCfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kPanelBytes = kTile * 128;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kCodes = kTile * D;                // one tile's E4M3 codes
  static constexpr int kSmem = 2 * kTileBytes + 2 * kStages * kTileBytes + (kFp8 ? 2 * kCodes : 0);
  static constexpr int kOCol = 256;
  static constexpr int kCorrWarp = 8, kLoadWarp = 12, kMmaWarp = 13;
  // 512 threads x 128 registers at launch, shared out again by setmaxnreg: the shares add up to
  // exactly the launch's, so every increase is satisfied.
  static constexpr int kLaunchRegs = 128, kRegSoftmax = 176, kRegCorr = 88, kRegOther = 72;
  static_assert(2 * kRegSoftmax + kRegCorr + kRegOther <= 4 * kLaunchRegs, "register shares");
};

// A segment: the CTA's run of tiles [kt0, kt0 + n) of one unit; nu of them can be seen by some row.
struct Seg {
  int g;                         // first chunk in the line
  SeqView s;
  int b, h, unit, row0, nrows, kt0, n, nu;
  bool from_start, to_end;
};

// A walk over the CTA's segments.
struct Walk {
  Cursor c;
  int g, left;
  Seg e;
  __device__ __forceinline__ void start(const Part& p) {
    c = p.at;
    g = p.lo;
    left = p.n;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if (left <= 0) return false;
    e.s = c.s;
    e.b = c.b;
    e.h = c.h;
    e.unit = c.u;
    e.row0 = (c.u - c.h * c.s.RT) * a.tile_rows;
    e.nrows = min(a.tile_rows, c.s.T * a.G - e.row0);
    e.kt0 = c.kt;
    e.n = min(c.s.KT - c.kt, left);
    e.nu = max(0, min(e.n, c.last / kChunk + 1 - c.kt));
    e.from_start = c.kt == 0;
    e.to_end = c.kt + e.n == c.s.KT;
    e.g = g;
    g += e.n;
    left -= e.n;
    if (left > 0) next_unit(a, c);
    return true;
  }
};

struct BigShared {
  uint64_t q_full[2], o_full[2];
  uint64_t k_full[4], v_full[4], k_empty[4], v_empty[4], v_ok[4];
  uint64_t s_full[2], p_full[2], alpha_full[2], o_ready[2];
  uint64_t c_full[2], c_empty[2];       // E4M3: staged codes of K and of V
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  // [group][its segments mod 2]: number + 1 of a segment with a value that was made safe.  The correction
  // warps reach a group's segment n + 2 only with all its alphas of segment n + 1, which it
  // publishes after it has read entry n.
  int odd[2][2];
  float alpha[2][kTile];
  // E4M3: staged scale codes of a tile (K's and V's with K, V's with V), and by tile mod 8 2^E of its K and
  // E of its V (kfac 0, vexp kWide: rows as they are).  Entry u is written again for tile u + 8, whose K slot is free only
  // after S of tile u + 8 - kStages, so of u + 4, which waited for both softmax groups to have finished u + 3.
  alignas(16) uint8_t scales[3][kTile];
  float kfac[8], vexp[8];
  Walk walk[8];                  // one per softmax warp, whose registers are full
};

// Whether tile kt holds new tokens or reaches past them.
__device__ __forceinline__ bool tail_tile(const Seg& e, int kt) { return (kt + 1) * kChunk > e.s.len; }

// E4M3 rows enter the fp16 products as code * 2^(scale - E) with E the largest scale of the tile's keys, exactly:
// a code has its last bit at 2^-9, fp16 at 2^-24, so scales may be 2^15 apart (K) and are let to be 2^8 apart (V).
// 2^E of K goes into the tile's score factor; E of V into the exponent of the weights, 2^(s + E - R), with a
// reference R of each row's own, which follows the largest max(s) + E of the row's tiles (visible keys only): R is
// moved (and O with it) when one is 2^15 above it, to 2^11 under it.  Weights keep fp16's eleven bits down to 2^-25
// of the row's largest, or 2^-17 where a tile puts R too high by a key of up to 2^8 the size that the row
// does not see.  A tile whose scales are further apart ("wide") keeps its rows as they are, and the softmax takes
// each key's scale from the cache, K's to the score and V's to the weight, so that no key's size depends on
// another's.  Rows of scale code 0 or 1 (zeros, and values below 2^-117) do not make a tile wide; they become zero beside
// others 2^25 as large.
//
// Warp 12 keeps one tile's codes of K and of V ahead in shared memory by TMA.  Warps 14 and 15 expand
// K into the ring; the correction warps expand V, one tile ahead of their rescales.  In tiles that hold
// new tokens V's rows past the end become zero and so do NaN codes, noted (see the top of the file).

// fp16 2^d twice, d <= 15; 0 below the type's last bit.
__device__ __forceinline__ uint32_t half2_pow2(int d) {
  const uint32_t h = d >= -14 ? (uint32_t)(min(d, 15) + 15) << 10 : d >= -24 ? 1u << (d + 24) : 0u;
  return h | (h << 16);
}

constexpr float kWide = 1000.f;          // vexp of a wide tile
constexpr int kRaw = -1000;              // expand_tile: rows as they are

// The largest of a tile's first `keys` scale codes, and whether the smallest above 1 is more than `apart` below; one warp.
__device__ __forceinline__ uint32_t top_scale(const uint8_t* scales, int keys, uint32_t apart, bool& wide) {
  const int lane = lane_id(), k = keys - 4 * lane;
  uint32_t x = *reinterpret_cast<const uint32_t*>(scales + 4 * lane);
  x &= k >= 4 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
  uint32_t top = 0, low = 255;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (x >> (8 * i)) & 0xFF;
    top = max(top, b);
    low = min(low, b > 1 ? b : 255u);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  wide = __any_sync(0xffffffffu, low + apart < top);
  return top;
}
constexpr uint32_t kApartK = 15, kApartV = 8;

// Expand one tile (128 rows of D codes, as TMA staged them) into a ring tile: warp wi of nW.  A pass
// of a warp is 32 / kLanes rows; row factors are computed once, two or one per lane, and
// shuffled (e = kRaw: 1).  clean (V): rows from `keys` on become zero and NaN codes too; returns whether there were.
// The caller releases the staging behind the stores and the proxy fence.  (Released behind the last loads,
// before their values were used, the next copy got in first: whole V tiles came out wrong.)
template <int D, int nW>
__device__ __forceinline__ bool expand_tile(const uint8_t* src0, uint8_t* dst0, const uint8_t* scales, int e, int wi,
                                            bool clean, int keys) {
  constexpr int kLanes = D / 16, kW = 32 / kLanes, kF = kTile / nW / 32, kPasses = kTile / (nW * kW);
  const int lane = lane_id();
  const int chunk = lane % kLanes, sub = lane / kLanes;
  uint32_t f[kF];
#pragma unroll
  for (int k = 0; k < kF; ++k) {
    const int j = k * 32 + lane;
    f[k] = e == kRaw ? half2_pow2(0) : half2_pow2((int)scales[(j / kW) * (nW * kW) + wi * kW + j % kW] - e);
  }
  bool odd = false;
  // chunk `chunk` of the codes (16) is chunks 2 chunk, 2 chunk + 1 of the row (8 values each); at d =
  // 128 half of the lanes start with the second, so that a quarter warp's stores hit all banks
  const int r0 = wi * kW + sub;
  const int c0 = (2 * chunk) & 7, sw = D == 128 ? (chunk >> 2) & 1 : 0;
  uint8_t* dst = dst0 + (chunk >> 2) * (kTile * 128);
  static_assert(kPasses % 2 == 0, "passes");
#pragma unroll 1
  for (int i0 = 0; i0 < kPasses; i0 += 2) {               // two passes in flight (four: 5 % slower, spills)
    uint2 x[2][2];
    uint32_t fi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = i0 + i, r = r0 + p * nW * kW;
      const uint8_t* src = src0 + (D == 64 ? r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4) : r * 128 + ((chunk ^ (r & 7)) << 4));
      x[i][0] = *reinterpret_cast<const uint2*>(src + 8 * sw);
      x[i][1] = *reinterpret_cast<const uint2*>(src + 8 - 8 * sw);
      fi[i] = __shfl_sync(0xffffffffu, kF > 1 && p * kW >= 32 ? f[kF - 1] : f[0], (p * kW) % 32 + sub);
    }
    if (clean) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool past = r0 + (i0 + i) * nW * kW >= keys;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t& y = (k & 1) ? x[i][k >> 1].y : x[i][k >> 1].x;
          if (past) y = 0;
          const uint32_t b = ((y & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // NaN: 0x7F + 1 carries into bit 7
          if (b != 0) {
            y &= ~((b >> 7) * 0xFFu);
            odd = true;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + (i0 + i) * nW * kW;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t y = j < 2 ? x[i][k].x : x[i][k].y;
          const uint32_t h = e4m3_to_f16x2((j & 1) ? y >> 16 : y);
          const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&fi[i]));
          o[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(dst + r * 128 + (((c0 + (k ^ sw)) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  return odd;
}

__device__ __forceinline__ void l2_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z) : "memory");
}

// Warp 12 with an E4M3 cache: K's codes with both sets of scale codes, V's codes with V's.
template <int D>
__device__ void stage_role(const TreeArgs& a, BigShared& sh, uint8_t* sC, const CUtensorMap* tm_k,
                           const CUtensorMap* tm_v, Walk& w) {
  constexpr int kCodes = kTile * D;
  const int lane = lane_id();
  const DevStatus st{a.c.status, a.timeout_ns};
  volatile int* abort_flag = &sh.abort_flag;
  const int R = 1 << a.c.page_shift, boxes = kTile / R;
  const Seg& e = w.e;
  int n[2] = {0, 0};
  bool ok = true;
  if (lane == 0) {
    prefetch_tmap(tm_k);
    prefetch_tmap(tm_v);
  }
  while (ok && w.next(a)) {
    for (int u = 0; u < e.nu && ok; ++u) {
      const int pos = (e.kt0 + u) * kChunk + lane * R;
      int row = (int)((long long)a.c.pages * a.c.Hk << a.c.page_shift);   // behind the last row: zeros
      bool valid = false;
      if (lane < boxes && pos < e.s.len + e.s.T) {
        const long long r = slot_row(a.c, e.b, e.h, pos);
        if (r >= 0) {
          row = (int)r;
          valid = true;
        }
      }
      const int nvalid = __popc(__ballot_sync(0xffffffffu, valid));
      if (valid) {                                        // one buffer each: have the copies start from L2
        l2_prefetch_3d(tm_k, 0, row, 0);
        l2_prefetch_3d(tm_v, 0, row, 0);
      }
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        if (ok && n[v] > 0) ok = mbar_wait(&sh.c_empty[v], (n[v] - 1) & 1, abort_flag, st);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.c_full[v], kCodes + (v == 0 ? 2 : 1) * nvalid * R);
        __syncwarp();
        if (lane < boxes) tma_load_3d(sC + v * kCodes + lane * R * D, v == 0 ? tm_k : tm_v, &sh.c_full[v], 0, row, 0);
        if (valid) {
          if (v == 0) bulk_load(&sh.scales[0][lane * R], a.c.ks + row, R, &sh.c_full[0]);
          bulk_load(&sh.scales[1 + v][lane * R], a.c.vs + row, R, &sh.c_full[v]);
        }
        ++n[v];
      }
    }
  }
  __syncwarp();
  // After a wait that ran out: copies in flight land before the shared memory goes away.
  if (*abort_flag && lane == 0)
    for (int v = 0; v < 2; ++v)
      if (n[v] > 0) mbar_wait_drain(&sh.c_full[v], (n[v] - 1) & 1, st);
  __syncwarp();
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Warps 14 and 15 with an E4M3 cache: K into the ring, and each tile's factors.
template <int D, int kStages>
__device__ void expand_k_role(const TreeArgs& a, BigShared& sh, uint8_t* sK, const uint8_t* sC, Walk& w, int wi) {
  const int lane = lane_id();
  const DevStatus st{a.c.status, a.timeout_ns};
  volatile int* abort_flag = &sh.abort_flag;
  const Seg& e = w.e;
  int n = 0;
  bool ok = true;
  while (ok && w.next(a)) {
    for (int u = 0; u < e.nu && ok; ++u, ++n) {
      const int s = n % kStages;
      ok = mbar_wait(&sh.c_full[0], n & 1, abort_flag, st);
      if (ok && n >= kStages) ok = mbar_wait(&sh.k_empty[s], ((n / kStages) - 1) & 1, abort_flag, st);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int keys = e.s.len + e.s.T - (e.kt0 + u) * kChunk;
      bool wide_k, wide_v;
      const uint32_t ek = top_scale(sh.scales[0], keys, kApartK, wide_k);
      const uint32_t ev = top_scale(sh.scales[1], keys, kApartV, wide_v);
      if (wi == 0 && lane == 0) {
        *reinterpret_cast<volatile float*>(&sh.kfac[n & 7]) = wide_k ? 0.f : scale_value(ek);
        *reinterpret_cast<volatile float*>(&sh.vexp[n & 7]) = wide_v ? kWide : (float)((int)ev - 127);
      }
      expand_tile<D, 2>(sC, sK + s * (kTile * D * 2), sh.scales[0], wide_k ? kRaw : (int)ek, wi, false, 0);
      fence_async_smem();
      mbar_arrive(&sh.k_full[s]);
      mbar_arrive(&sh.c_empty[0]);
    }
  }
}

// A Q row of bf16 pairs to fp16 (row_factor).  Returns the inverse factor, for the scores.
template <int N>
__device__ __forceinline__ float row_to_fp16(uint32_t* x) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 f = unpack2<false>(x[i]);
    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  const int k = row_factor(amax);
  const float f = scale_value(127 + k);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 v = unpack2<false>(x[i]);
    x[i] = pack2<true>(v.x * f, v.y * f);
  }
  return scale_value(127 - k);
}

// The scale codes of keys pos .. pos + 15 (zeros where there is no key, or no page).
__device__ __forceinline__ void load_codes(const TreeArgs& a, const Seg& e, int pos, uint4& ks, uint4& vs) {
  ks = vs = make_uint4(0, 0, 0, 0);
  if (pos >= e.s.len + e.s.T) return;
  const long long row = slot_row(a.c, e.b, e.h, pos);
  if (row < 0) return;
  ks = *reinterpret_cast<const uint4*>(a.c.ks + row);
  vs = *reinterpret_cast<const uint4*>(a.c.vs + row);
}
__device__ __forceinline__ uint32_t byte_of(const uint4& w, int i) {
  const uint32_t x = i < 4 ? w.x : i < 8 ? w.y : i < 12 ? w.z : w.w;
  return (x >> (8 * (i & 3))) & 0xFF;
}

// One row's softmax of an E4M3 tile in its general form: for a wide tile (kf 0: the scores lack K's scales; ve kWide:
// V's rows lack theirs), and where R and m are so far apart that the row sum needs exponentials of its
// own.  Rare and slow: scale codes come from the cache, each weight takes two exponentials, and the scores are read
// from tensor memory twice, 32 at a time, so that the usual path keeps its registers.  (P goes over
// scores that have been read: columns 16 h of 32 h.)
__device__ __forceinline__ void wide_tile(const TreeArgs& a, const Seg& e, int t, int kt, float sl2q, float kf, float ve,
                                          uint32_t tS, float& m, float& l, float& ref, float* alpha, uint64_t* alpha_full) {
  uint32_t s[32];                                         // 32 scores, masked and scaled
  float c[32];                                            // the keys' V exponents
  auto load = [&](int h) {
    __syncwarp();
    tmem_ld32_sync(tS + 32 * h, s);
    const uint32_t vis = visible32(a, e.s, t, kt * kChunk + 32 * h - e.s.len);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint4 ks, vs;
      load_codes(a, e, kt * kChunk + 32 * h + 16 * g, ks, vs);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 16 * g + i;
        const float x = __uint_as_float(s[j]) * (sl2q * (kf == 0.f ? scale_value(byte_of(ks, i)) : kf));
        s[j] = __float_as_uint((vis >> j) & 1u ? x : -INFINITY);
        c[j] = ve == kWide ? (float)((int)byte_of(vs, i) - 127) : ve;
      }
    }
  };
  float mx = -INFINITY, my = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    load(h);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      mx = fmaxf(mx, __uint_as_float(s[j]));
      my = fmaxf(my, __uint_as_float(s[j]) + c[j]);
    }
  }
  const float mn = fmaxf(m, mx), rn = my > ref + 15.f ? my - 11.f : ref;
  l *= mn == -INFINITY ? 1.f : ex2(m - mn);
  m = mn;
  *alpha = rn == ref ? 1.f : ex2(ref - rn);
  ref = rn;
  mbar_arrive(alpha_full);
  const float mneg = m == -INFINITY ? 0.f : -m, rneg = ref == -INFINITY ? 0.f : -ref;
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    load(h);
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = __uint_as_float(s[2 * i]), y = __uint_as_float(s[2 * i + 1]);
      l += ex2(x + mneg) + ex2(y + mneg);
      pk[i] = pack2<true>(ex2(x + c[2 * i] + rneg), ex2(y + c[2 * i + 1] + rneg));
    }
    __syncwarp();                                         // the store is the whole warp's
    tmem_st16(tS + 16 * h, pk);
    tmem_wait_st();
  }
}

// kFp16: type of q and o.  The products of a 16-bit cache are in that type, those of an E4M3 cache in fp16.
template <int D, bool kFp8, bool kFp16>
__global__ void __launch_bounds__(512, 1)
    tree_big_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const TreeArgs a) {
  using C = BigCfg<D, kFp8>;
  constexpr bool kMmaFp16 = kFp8 || kFp16;
  constexpr float kLift = kFp16 ? kFp16Lift : 0.f;      // 16-bit caches (an E4M3 cache's weights have a reference)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ BigShared sh;
  if ((smem_addr(smem_raw) & 1023u) != 0) {               // the tiles' swizzle needs it
    if (threadIdx.x == 0) atomicCAS(a.c.status, 0, kDevBadState);
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* sK = sQ + 2 * C::kTileBytes;
  uint8_t* sV = sK + C::kStages * C::kTileBytes;
  uint8_t* sC = sV + C::kStages * C::kTileBytes;          // E4M3: staged codes of K, then of V
  const int warp = warp_id(), lane = lane_id();
  const DevStatus st{a.c.status, a.timeout_ns};
  volatile int* abort_flag = &sh.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh.k_full[s], kFp8 ? 64 : 1);
      mbar_init(&sh.v_full[s], kFp8 ? 128 : 1);
      mbar_init(&sh.k_empty[s], 1);
      mbar_init(&sh.v_empty[s], 1);
      mbar_init(&sh.v_ok[s], 128);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&sh.q_full[q], 128);
      mbar_init(&sh.o_full[q], 1);
      mbar_init(&sh.s_full[q], 1);
      mbar_init(&sh.p_full[q], 128);
      mbar_init(&sh.alpha_full[q], 128);
      mbar_init(&sh.o_ready[q], 128);
      sh.odd[q][0] = sh.odd[q][1] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.c_full[i], 1);
      mbar_init(&sh.c_empty[i], i == 0 ? 64 : 128);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  grid_begin();
  const Part part = find_part(a, blockIdx.x == 0 && warp == 0);
  if (threadIdx.x == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp >= C::kLoadWarp) {
    reg_dec<C::kRegOther>();
    Walk w;
    w.start(part);
    const Seg& e = w.e;
    if (kFp8 && warp == C::kLoadWarp) {
      stage_role<D>(a, sh, sC, &tm_k, &tm_v, w);
    } else if (kFp8 && warp > C::kMmaWarp) {
      expand_k_role<D, C::kStages>(a, sh, sK, sC, w, warp - C::kMmaWarp - 1);
    } else if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------------- producer
      const int R = 1 << a.c.page_shift;                  // rows per box: one page
      const int boxes = kTile / R;
      int nk = 0, nv = 0;                                 // tiles whose copy was started
      bool ok = true;
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
      }
      while (ok && w.next(a)) {
        const int end = e.s.len + e.s.T;
        for (int u = 0; u < e.nu && ok; ++u) {
          const int s = nk % C::kStages;
          const uint32_t ph = ((nk / C::kStages) - 1) & 1;
          // a page past the end, or no page, reads as zeros: a row behind the tensor's last
          const int box = lane % boxes, panel = lane / boxes;
          const int pos = (e.kt0 + u) * kChunk + box * R;
          const bool mine = lane < boxes * C::kPanels;
          int row = (int)((long long)a.c.pages * a.c.Hk << a.c.page_shift);
          if (mine && pos < end) {
            const long long r = slot_row(a.c, e.b, e.h, pos);
            if (r >= 0) row = (int)r;
          }
          const int off = panel * C::kPanelBytes + box * R * 128;
          if (nk >= C::kStages) ok = mbar_wait(&sh.k_empty[s], ph, abort_flag, st);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[s], C::kTileBytes);
          __syncwarp();
          if (mine) tma_load_3d(sK + s * C::kTileBytes + off, &tm_k, &sh.k_full[s], 0, row, panel);
          ++nk;
          if (nv >= C::kStages) ok = mbar_wait(&sh.v_empty[s], ph, abort_flag, st);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&sh.v_full[s], C::kTileBytes);
          __syncwarp();
          if (mine) tma_load_3d(sV + s * C::kTileBytes + off, &tm_v, &sh.v_full[s], 0, row, panel);
          ++nv;
        }
      }
      __syncwarp();
      if (*abort_flag && lane == 0) {
        // every copy this warp started lands before the CTA's shared memory goes away
        for (int i = max(0, nk - C::kStages); i < nk; ++i)
          mbar_wait_drain(&sh.k_full[i % C::kStages], (i / C::kStages) & 1, st);
        for (int i = max(0, nv - C::kStages); i < nv; ++i)
          mbar_wait_drain(&sh.v_full[i % C::kStages], (i / C::kStages) & 1, st);
      }
      __syncwarp();
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      // The whole warp walks and waits, one elected lane issues: the operands are then the same in all
      // lanes, broadcast so that the compiler knows, and stay in uniform registers.
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(128, 128, kMmaFp16, false, false);
      const uint32_t idesc_pv = idesc_f16(128, D, kMmaFp16, false, true);
      // Operand descriptors: the upper half is constant, the lower a sum in the address field (16-byte
      // units).  (As 64-bit sums both halves go through registers: 167 -> 188 us at trees of 64.)
      constexpr uint64_t kHi = (uint64_t)((1024 >> 4) | (1 << 14) | (2 << 29)) << 32;   // see smem_desc_sw128
      const uint32_t lQ = (smem_addr(sQ) >> 4) | (16 >> 4) << 16, lK = (smem_addr(sK) >> 4) | (16 >> 4) << 16;
      const uint32_t lV = (smem_addr(sV) >> 4) | (C::kPanelBytes >> 4) << 16;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      int nt = 0;                                         // tiles before this segment
      int np[2] = {0, 0};                                 // P tiles consumed
      uint32_t tails = 0;                                 // bit s: parity of stage s's safe V tiles
      uint32_t nseg[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, st));
      };
      while (ok && w.next(a)) {
        const int nq = e.nrows > kTile ? 2 : 1;
        for (int u = 0; u <= e.nu && ok && e.nu > 0; ++u) {
          const int tp = nt + u - 1, tc = nt + u;
          const int sp = (tp + C::kStages) % C::kStages, sc = tc % C::kStages;
          bool v_ready = false, k_ready = false;
          auto pv = [&](int q) -> bool {
            if (u == 0 || q >= nq) return true;
            if (!v_ready) {
              if (!wait(&sh.v_full[sp], (tp / C::kStages) & 1)) return false;
              if (!kFp8 && tail_tile(e, e.kt0 + u - 1)) {
                if (!wait(&sh.v_ok[sp], (tails >> sp) & 1u)) return false;
                tails ^= 1u << sp;
              }
              v_ready = true;
            }
            const uint32_t lv = __shfl_sync(0xffffffffu, lV + (sp * C::kTileBytes >> 4), 0);
            const uint32_t more = __shfl_sync(0xffffffffu, u > 1 ? 1u : 0u, 0);
            if (!wait(&sh.p_full[q], np[q] & 1) || !wait(&sh.o_ready[q], np[q] & 1)) return false;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                mma_ts(tm + C::kOCol + q * D, tm + q * 128 + kk * 8, kHi | (lv + (kk * 2048 >> 4)), idesc_pv,
                       kk > 0 ? 1u : more);
            }
            ++np[q];
            return true;
          };
          auto sq = [&](int q) -> bool {
            if (u == e.nu || q >= nq) return true;
            if (!k_ready) {
              if (!wait(&sh.k_full[sc], (tc / C::kStages) & 1)) return false;
              k_ready = true;
            }
            if (u == 0) {
              if (!wait(&sh.q_full[q], nseg[q] & 1)) return false;
              ++nseg[q];
            }
            const uint32_t lk = __shfl_sync(0xffffffffu, lK + (sc * C::kTileBytes >> 4), 0);
            const uint32_t lq = __shfl_sync(0xffffffffu, lQ + (q * C::kTileBytes >> 4), 0);
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = ((kk >> 2) * C::kPanelBytes + (kk & 3) * 32) >> 4;
                mma_ss(tm + q * 128, kHi | (lq + koff), kHi | (lk + koff), idesc_s, kk > 0 ? 1u : 0u);
              }
              tc_commit(&sh.s_full[q]);
            }
            return true;
          };
          ok = pv(0) && sq(0) && pv(1);
          if (u > 0 && ok && leader) tc_commit(&sh.v_empty[sp]);
          ok = ok && sq(1);
          if (u < e.nu && ok && leader) tc_commit(&sh.k_empty[sc]);
        }
        nt += e.nu;
        if (ok && e.nu > 0 && leader)
          for (int q = 0; q < nq; ++q) tc_commit(&sh.o_full[q]);   // O_q holds every product
      }
      if (leader) {
        tc_commit(&sh.mma_done);
        mbar_wait_drain(&sh.mma_done, 0, st);
      }
      __syncwarp();
    }
  } else if (warp >= C::kCorrWarp) {
    // ------------------------------------------------------------------ correction warpgroup
    reg_dec<C::kRegCorr>();
    const int wq = warp & 3;
    const int r = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    int nt = 0, cq[2] = {0, 0};
    int seg[2] = {0, 0};
    bool ok = true;
    Walk w;
    w.start(part);
    const Seg& e = w.e;
    while (ok && w.next(a)) {
      const int nq = e.nrows > kTile ? 2 : 1;
      auto expand_v = [&](int u) -> bool {                // tile u of the segment
        const int n = nt + u, s = n % C::kStages;
        bool go = mbar_wait(&sh.c_full[1], n & 1, abort_flag, st);
        if (go && n >= C::kStages) go = mbar_wait(&sh.v_empty[s], ((n / C::kStages) - 1) & 1, abort_flag, st);
        if (!__all_sync(0xffffffffu, go)) return false;
        const int keys = e.s.len + e.s.T - (e.kt0 + u) * kChunk;
        bool wide;
        const uint32_t ev = top_scale(sh.scales[2], keys, kApartV, wide);
        if (expand_tile<D, 4>(sC + C::kCodes, sV + s * C::kTileBytes, sh.scales[2], wide ? kRaw : (int)ev, wq,
                              tail_tile(e, e.kt0 + u), keys))
          for (int q = 0; q < nq; ++q) *reinterpret_cast<volatile int*>(&sh.odd[q][seg[q] & 1]) = seg[q] + 1;
        fence_async_smem();
        mbar_arrive(&sh.v_full[s]);
        mbar_arrive(&sh.c_empty[1]);
        return true;
      };
      if constexpr (kFp8) {
        if (e.nu > 0) ok = expand_v(0);
      }
      for (int u = 0; u < e.nu && ok; ++u) {
        const int kt = e.kt0 + u;
        if (!kFp8 && tail_tile(e, kt)) {
          // this thread's V row (key): zero past the end, and where it is not finite
          const int t = nt + u, s = t % C::kStages;
          ok = mbar_wait(&sh.v_full[s], (t / C::kStages) & 1, abort_flag, st);
          if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
          uint8_t* vrow = sV + s * C::kTileBytes + r * 128;
          const bool past = kt * kChunk + r >= e.s.len + e.s.T;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint4* p = reinterpret_cast<uint4*>(vrow + (c >> 3) * C::kPanelBytes + (((c & 7) ^ (r & 7)) << 4));
            uint4 x = past ? make_uint4(0, 0, 0, 0) : *p;
            uint32_t* y = &x.x;
            bool odd = past;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              constexpr uint32_t ex = kFp16 ? 0x7C00u : 0x7F80u;
              if ((y[i] & ex) == ex) { y[i] &= 0xFFFF0000u; odd = true; }
              if (((y[i] >> 16) & ex) == ex) { y[i] &= 0xFFFFu; odd = true; }
            }
            if (odd) {
              *p = x;
              if (!past)
                for (int q = 0; q < nq; ++q) *reinterpret_cast<volatile int*>(&sh.odd[q][seg[q] & 1]) = seg[q] + 1;
            }
          }
          fence_async_smem();
          mbar_arrive(&sh.v_ok[s]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q >= nq) continue;
          ok = mbar_wait(&sh.alpha_full[q], cq[q] & 1, abort_flag, st);
          if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
          const float al = sh.alpha[q][r];
          if (u > 0 && __any_sync(0xffffffffu, al != 1.f)) {
            __syncwarp();
            tc_fence_after();
            const uint32_t tO = tmem + C::kOCol + q * D + lane_off;
#pragma unroll 2
            for (int cc = 0; cc < D; cc += 16) {          // 16 at a time: 32 spill beside the walk's state
              uint32_t o[16];
              tmem_ld16(tO + cc, o);
              tmem_wait_ld();
              reg_fence16(o);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 x = mul2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), make_float2(al, al));
                o[i] = __float_as_uint(x.x);
                o[i + 1] = __float_as_uint(x.y);
              }
              tmem_st16(tO + cc, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(&sh.o_ready[q]);
          ++cq[q];
        }
        if constexpr (kFp8) {
          if (ok && u + 1 < e.nu) ok = expand_v(u + 1);
        }
      }
      nt += e.nu;
      if (e.nu > 0)
        for (int q = 0; q < nq; ++q) ++seg[q];
    }
  } else {
    // ------------------------------------------------------------------ softmax groups
    reg_inc<C::kRegSoftmax>();
    const int q = warp >> 2;
    const int wq = warp & 3;
    const int rl = wq * 32 + lane;                        // row of the 128-row tile
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + q * 128 + lane_off;
    const uint32_t tO = tmem + C::kOCol + q * D + lane_off;
    int cs = 0, nseg = 0;
    int tile = 0;                                         // tiles of the CTA before this segment
    bool ok = true;
    Walk& w = sh.walk[warp];
    if (lane == 0) w.start(part);
    const Seg& e = w.e;
    while (ok) {
      __syncwarp();
      bool more = false;
      if (lane == 0) more = w.next(a);
      if (!__shfl_sync(0xffffffffu, more, 0)) break;
      __syncwarp();
      const int tile0 = tile;
      tile += e.nu;
      if (q == 1 && e.nrows <= kTile) continue;           // this group's tile has no rows
      const int r = q * kTile + rl;                       // row of the unit
      const bool live = r < e.nrows;
      const int R = e.row0 + (live ? r : 0);
      const int t = R / a.G;
      float sl2q = a.scale_log2;
      if (e.nu > 0) {
        // Q row into the swizzled tile (rows without a token: zeros)
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (e.s.cu0 + t) * a.q_tok + (e.h * a.G + (R - t * a.G)) * a.q_head);
        uint8_t* dst = sQ + q * C::kTileBytes + rl * 128;
        uint4 x[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x[c] = live ? src[c] : make_uint4(0, 0, 0, 0);
        if constexpr (kFp8 && !kFp16) sl2q *= row_to_fp16<D / 2>(&x[0].x);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kPanelBytes + (((c & 7) ^ (rl & 7)) << 4)) = x[c];
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.q_full[q]);
      }
      float m = -INFINITY, l = 0.f, ref = -INFINITY;      // ref: R, with an E4M3 cache
      for (int u = 0; u < e.nu; ++u) {
        const int kt = e.kt0 + u;
        ok = mbar_wait(&sh.s_full[q], cs & 1, abort_flag, st);
        if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
        __syncwarp();                                     // as at P's stores
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[32 * i]));
        float s[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(sr[i]);
        if (tail_tile(e, kt)) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t vis = visible32(a, e.s, t, kt * kChunk + 32 * h - e.s.len);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((vis >> i) & 1u)) s[32 * h + i] = -INFINITY;
          }
        }
        float sl2 = sl2q, alpha = 1.f, mneg, lfac = 1.f;
        if constexpr (kFp8) {
          const float kf = *reinterpret_cast<volatile float*>(&sh.kfac[(tile0 + u) & 7]);
          const float ve = *reinterpret_cast<volatile float*>(&sh.vexp[(tile0 + u) & 7]);
          sl2 = fmaxf(sl2q * kf, 0x1p-126f);              // never 0, which would make NaN of a masked score's -inf
          const float mx2 = row_max128(s) * sl2;
          const float mn = fmaxf(m, mx2), rn = mx2 + ve > ref + 15.f ? mx2 + ve - 11.f : ref;
          // 2^(s + ve - R) serves the products and, times 2^(R - ve - m), the row sum
          if (__any_sync(0xffffffffu, kf == 0.f || ve == kWide || rn - ve - mn > 90.f)) {
            wide_tile(a, e, t, kt, sl2q, kf, ve, tS, m, l, ref, &sh.alpha[q][rl], &sh.alpha_full[q]);
            tc_fence_before();
            mbar_arrive(&sh.p_full[q]);
            ++cs;
            continue;
          }
          alpha = mn == -INFINITY ? 1.f : ex2(m - mn);
          m = mn;
          sh.alpha[q][rl] = rn == ref ? 1.f : ex2(ref - rn);       // 0 when R = -inf
          ref = rn;
          mneg = rn == -INFINITY ? 0.f : ve - rn;
          lfac = m == -INFINITY ? 1.f : ex2(rn - ve - m);
        } else {
          // m is the running max less kLift: the largest P is 2^kLift
          const float mx2 = row_max128(s) * sl2 - kLift;
          if (mx2 > m) {
            alpha = ex2(m - mx2);                         // 0 when m = -inf
            m = mx2;
          }
          sh.alpha[q][rl] = alpha;
          mneg = (m == -INFINITY) ? 0.f : -m;
        }
        mbar_arrive(&sh.alpha_full[q]);
        const float2 sl2v = make_float2(sl2, sl2), mnegv = make_float2(mneg, mneg);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        __syncwarp();                                     // P's stores are the whole warp's: rows may have parted above
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = fma2(make_float2(s[32 * h + 2 * i], s[32 * h + 2 * i + 1]), sl2v, mnegv);
            // (a share on the FMA pipe's polynomial, as the dense forward has at d = 64, costs the LSE
            // three digits, and at d = 128 4 to 6 % of time)
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            acc[i & 3] = add2(acc[i & 3], p);
            pk[i] = pack2<kMmaFp16>(p.x, p.y);            // at most half a 16-bit step; the sum keeps 32 bits
          }
          tmem_st16(tS + 16 * h, pk);
        }
        const float2 sum = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
        l = l * alpha + (kFp8 ? (sum.x + sum.y) * lfac : sum.x + sum.y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.p_full[q]);
        ++cs;
      }
      // -------------------------------------------------------------- results
      if (e.nu > 0) {
        if (ok) ok = mbar_wait(&sh.o_full[q], nseg & 1, abort_flag, st);
        ++nseg;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const bool whole = e.from_start && e.to_end;
      const int slot = 2 * blockIdx.x + (e.from_start ? 1 : 0);
      if (q == 0 && rl == 0 && e.from_start && !e.to_end) {
        a.meta[2 * blockIdx.x] = make_int4(part.line.owner(e.g + e.s.KT - 1), e.nrows, e.s.cu0, e.h);
        a.meta[2 * blockIdx.x + 1] = make_int4(e.row0, 0, 0, 0);
      }
      const bool odd = e.nu > 0 && *reinterpret_cast<volatile int*>(&sh.odd[q][(nseg - 1) & 1]) == nseg;
      // E4M3: O's reference from R to m, 2^(R - m) in two steps: it may lie outside fp32's normal range
      const float half = !kFp8 ? 1.f : ref == -INFINITY ? 0.f : ex2(0.5f * (ref - m));
      const float inv = whole ? (l == 0.f ? 0.f : half / l) : half;
      const int hq = e.h * a.G + (R - t * a.G);
      const long long tk = e.s.cu0 + t;
      if (live) {
        if (whole) {
          a.lse[tk * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
        } else {
          float* ml = a.part_ml + ((long long)slot * a.slot_rows + r) * 2;
          ml[0] = m;
          ml[1] = l;
        }
      }
#pragma unroll
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t o[32];
        if (e.nu > 0) {
          __syncwarp();                                   // the load is the whole warp's; rows part below
          tmem_ld32_sync(tO + cc, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (live) {
          if constexpr (kFp8) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * half);
          }
          if (odd) {                                      // rare: see the top of the file
            // keys of the segment's tiles that were made safe; j < 0 is the prefix
            const int j1 = min(e.s.T, (e.kt0 + e.nu) * kChunk - e.s.len);
            for (int j = max(e.kt0, e.s.len / kChunk) * kChunk - e.s.len; j < j1; ++j) {
              if (!(visible32(a, e.s, t, j) & 1u)) continue;
              const long long row = slot_row(a.c, e.b, e.h, (long long)e.s.len + j);
              if (row < 0) continue;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if constexpr (kFp8) {
                  if ((a.c.v[row * D + cc + i] & 0x7F) == 0x7F) o[i] = 0x7FFFFFFFu;
                } else {
                  constexpr uint32_t ex = kFp16 ? 0x7C00u : 0x7F80u;
                  const uint32_t x = reinterpret_cast<const uint16_t*>(a.c.v)[row * D + cc + i];
                  if ((x & ex) == ex) o[i] = __float_as_uint(__uint_as_float(o[i]) + unpack2<kFp16>(x).x);
                }
              }
            }
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.o + tk * a.o_tok + hq * a.o_head + cc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 w;
              w.x = pack2<kFp16>(__uint_as_float(o[8 * i + 0]) * inv, __uint_as_float(o[8 * i + 1]) * inv);
              w.y = pack2<kFp16>(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv);
              w.z = pack2<kFp16>(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv);
              w.w = pack2<kFp16>(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv);
              dst[i] = w;
            }
          } else {
            // four columns of all rows, then the next four: a warp's stores are contiguous
            uint4* dst = reinterpret_cast<uint4*>(a.part_o) + ((long long)slot * (D / 4) + cc / 4) * a.slot_rows + r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if constexpr (kFp8) {
#pragma unroll
                for (int k = 0; k < 4; ++k) o[4 * i + k] = __float_as_uint(__uint_as_float(o[4 * i + k]) * inv);
              }
              dst[(long long)i * a.slot_rows] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
        }
      }
      tc_fence_before();                                  // O is read: the next segment may overwrite it
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kFp8, bool kFp16>
cudaError_t launch_big(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, cudaStream_t s) {
  using C = BigCfg<D, kFp8>;
  auto kern = tree_big_kernel<D, kFp8, kFp16>;
  static bool done[128];
  const cudaError_t e = prepare_kernel(kern, C::kSmem, C::kLaunchRegs, done);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(ctas), 512, C::kSmem, s, tk, tv, a);
}

template <int D>
cudaError_t launch_big_d(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, bool fp8, bool fp16, int ctas,
                         cudaStream_t s) {
  if (fp8) return fp16 ? launch_big<D, true, true>(tk, tv, a, ctas, s) : launch_big<D, true, false>(tk, tv, a, ctas, s);
  return fp16 ? launch_big<D, false, true>(tk, tv, a, ctas, s) : launch_big<D, false, false>(tk, tv, a, ctas, s);
}

}  // namespace

cudaError_t launch_tree_big(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, bool fp8, bool fp16,
                            int ctas, cudaStream_t s) {
  return a.c.d == 128 ? launch_big_d<128>(tk, tv, a, fp8, fp16, ctas, s) : launch_big_d<64>(tk, tv, a, fp8, fp16, ctas, s);
}

}  // namespace fa
